"""Attention behind a shared prefix whose CTAs give up when their loads have all been asked for: the warps that load have
nothing left to do by then, and still wait for the copies in flight before the CTA leaves. The copy of the library is that of
test_prefix_wait_expiry_gpu.py (a limit of 1 ms, the probabilities of a CTA's fourth tile withheld); there the shares are so
long that the loading warps give up themselves, here they end four to seven tiles in, within what the rings hold."""
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


def call(lib, q, c, out):
    def p(t):
        return ctypes.c_void_p(t.data_ptr())

    B, Hq, _ = q.shape
    pages, Hkv, ps, _ = c["k_cache"].shape
    P, G = c["block_table"].shape[1], c["prefix_lens"].shape[0]
    ws = K.attn_prefix_decode_workspace(B, Hq, Hkv, P, ps, G, DEV)
    ws.fill_(0x7f)  # what an aborted CTA leaves unwritten
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    st = lib.kda_attn_prefix_decode(p(q), p(c["k_cache"]), p(c["v_cache"]), c["k_cache"].stride(0), c["v_cache"].stride(0), pages, ps,
                                    p(c["block_table"]), P, p(c["seq_lens"]), p(c["cu_groups"]), p(c["prefix_lens"]), G, p(out), None,
                                    B, Hq, Hkv, SCALE, p(ws), ws.numel(), stream)
    detail = ctypes.c_int32(0)
    return st, lib.kda_device_status(stream, ctypes.byref(detail))


@pytest.mark.parametrize("rows", [32, 16])  # 256 query rows of the key head, a tile a step; 128, two tiles a step
@pytest.mark.parametrize("tiles", [4, 5, 6, 7])  # of a share
def test_shares_whose_loads_are_all_in_flight(tlib, rows, tiles):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    gen = torch.Generator().manual_seed(tiles)
    q = torch.randn(rows, 8, 128, generator=gen).to(torch.bfloat16).to(DEV)
    # every step of the prefix costs ten times a tile of the rest, of which there is one a row: all SMs but one have a share
    n = 128 * (sms - 1) * tiles * (1 if rows == 32 else 2)
    gen = torch.Generator(device=DEV).manual_seed(tiles)
    page = 1024
    kv = torch.randn(n // page + 1 + rows, 2, 1, page, 128, generator=gen, device=DEV).to(torch.bfloat16)
    shared, own = n // page, -(-(n % page + 9) // page)
    i32 = dict(dtype=torch.int32, device=DEV)
    table = torch.arange(shared, **i32).repeat(rows, 1)
    table = torch.cat([table, shared + torch.arange(rows, **i32)[:, None]], 1)
    assert own == 1
    kv[shared:, :, :, :n % page] = kv[shared:shared + 1, :, :, :n % page].clone()
    big = dict(k_cache=kv[:, 0], v_cache=kv[:, 1], block_table=table, seq_lens=torch.full((rows,), n + 9, **i32),
               cu_groups=torch.tensor([0, rows], **i32), prefix_lens=torch.tensor([n], **i32))
    assert call(tlib, q, big, torch.empty_like(q)) == (K.KDA_OK, K.KDA_ERR_DEVICE_TIMEOUT)
    # the SMs are as they were: a small call of both libraries, in wide tables, so that the prefix is shared
    small = R.prefix_inputs([0, rows], [384], [384 + 5 + i for i in range(rows)], 1, 64, seed=1, device=DEV)
    wide = torch.full((rows, (48 << 20) // (512 * 64 * rows) + 1), -1, **i32)
    wide[:, :small["block_table"].shape[1]] = small["block_table"]
    ref, _, _ = H.attn_decode(q, small, SCALE)
    for lib in (tlib, K.load()):
        out = torch.zeros_like(q)
        assert call(lib, q, dict(small, block_table=wide), out) == (K.KDA_OK, K.KDA_OK)
        assert_out_close(out, ref)
