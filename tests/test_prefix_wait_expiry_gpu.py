"""Failure detection of the shared-prefix attention without a GPU fault: in a copy of the library built with a 1 ms
limit, the softmax warps withhold one hand-off (the probabilities of a CTA's fourth tile), so the waits for it cannot
end. The CTA's roles give up, the call returns, the kernels behind it run on what was written, the status word reports
the timeout, and both libraries still pass parity afterwards in the same process: the aborted CTAs freed their tensor
memory and had no copy in flight."""
import ctypes
import math
import os

import pytest
import torch

import hybrid_reference as H
import kda_recurrent_gb300 as K
import serving_reference as R
from helpers import assert_out_close
from kda_recurrent_gb300 import build as kbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)
TEST_LIB = os.path.join(kbuild.BUILD_DIR, "wait_limit_test", "libkda_gb300_wait_limit_test.so")


@pytest.fixture(scope="module")
def tlib():
    path = kbuild.build(extra_flags=["-DKDA_WAIT_LIMIT_NS=1000000ull", "-DKDA_TEST_WITHHOLD_HANDOFF=3"], lib_path=TEST_LIB)
    return K.bind(ctypes.CDLL(path))


def p(t):
    return ctypes.c_void_p(t.data_ptr())


def call(lib, q, c, out):
    B, Hq, _ = q.shape
    pages, Hkv, ps, _ = c["k_cache"].shape
    P, G = c["block_table"].shape[1], c["prefix_lens"].shape[0]
    ws = K.attn_prefix_decode_workspace(B, Hq, Hkv, P, ps, G, DEV)
    ws.fill_(0x7f)  # what an aborted CTA leaves unwritten
    stride = c["k_cache"].stride(0)
    return lib.kda_attn_prefix_decode(p(q), p(c["k_cache"]), p(c["v_cache"]), stride, stride, pages, ps, p(c["block_table"]), P,
                                      p(c["seq_lens"]), p(c["cu_groups"]), p(c["prefix_lens"]), G, p(out), None, B, Hq, Hkv, SCALE,
                                      p(ws), ws.numel(), ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)), ws


def status(lib):
    detail = ctypes.c_int32(0)
    return lib.kda_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ctypes.byref(detail))


def inputs(rows, prefix, Hkv, seed):
    c = R.prefix_inputs([0, rows], [prefix], [prefix + 5 + i for i in range(rows)], Hkv, 64, seed=seed, device=DEV)
    wide = torch.full((rows, 73 * 2**20 // (512 * 64 * Hkv * rows) + 2 + c["block_table"].shape[1]), -1, dtype=torch.int32, device=DEV)
    wide[:, :c["block_table"].shape[1]] = c["block_table"]
    return c, dict(c, block_table=wide)


@pytest.mark.parametrize("rows", [3, 20])
def test_wait_expiry_is_reported_and_the_context_stays_usable(tlib, rows):
    gen = torch.Generator().manual_seed(rows)
    q = torch.randn(rows, 32, 128, generator=gen).to(torch.bfloat16).to(DEV)
    out = torch.empty_like(q)
    assert status(tlib) == K.KDA_OK
    # no CTA has four tiles: the withheld hand-off is not reached
    small, wide = inputs(rows, 512, 2, 1)
    ref, _, _ = H.attn_decode(q, small, SCALE)
    st, _ = call(tlib, q, wide, out)
    assert st == K.KDA_OK and status(tlib) == K.KDA_OK
    assert_out_close(out, ref)
    # shares of many tiles, several of them to an item
    _, big = inputs(rows, 128 * 152 * 8, 2, 2)
    st, _ = call(tlib, q, big, torch.empty_like(q))
    assert st == K.KDA_OK
    torch.cuda.synchronize()
    assert status(tlib) == K.KDA_ERR_DEVICE_TIMEOUT
    assert status(tlib) == K.KDA_OK
    for lib in (tlib, K.load()):
        out.zero_()
        st, _ = call(lib, q, wide, out)
        assert st == K.KDA_OK and status(lib) == K.KDA_OK
        assert_out_close(out, ref)
