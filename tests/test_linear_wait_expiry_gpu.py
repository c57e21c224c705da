"""Failure detection of the linear-attention prompt kernel without a GPU fault: in a copy of the library built
with a 1 ms limit, the state warps withhold one hand-off (the state of a CTA's fourth chunk), so the MMA
warp's wait for it cannot end. The watchdog warp gives up for the CTA, the call returns, the status word
reports the timeout, and the product library still passes parity afterwards in the same process: the aborted
CTAs freed their tensor memory and had no copy in flight."""
import ctypes
import math
import os

import pytest
import torch

import hybrid_reference as R
import kda_recurrent_gb300 as K
from helpers import assert_out_close, assert_state_close
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
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def call(lib, inp, out, fin, workspace=None):
    T, H, _ = inp["q"].shape
    N = inp["cu_seqlens"].shape[0] - 1
    return lib.kda_linear_prefill(p(inp["q"]), p(inp["k"]), p(inp["v"]), p(inp["log_decay"]), 0, p(inp["cu_seqlens"]),
                                  p(inp["init_state"]), p(out), p(fin), N, T, H, SCALE, p(workspace),
                                  0 if workspace is None else workspace.numel(),
                                  ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))


def status(lib):
    detail = ctypes.c_int32(0)
    return lib.kda_device_status(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream), ctypes.byref(detail))


@pytest.mark.parametrize("windows", [False, True])
def test_wait_expiry_is_reported_and_the_context_stays_usable(tlib, windows):
    assert status(tlib) == K.KDA_OK
    # 3 chunks do not reach the withheld hand-off
    inp = R.linear_inputs([384], 2, seed=71, decay="head", device=DEV)
    out, fin = torch.empty_like(inp["q"]), torch.empty_like(inp["init_state"])
    assert call(tlib, inp, out, fin) == K.KDA_OK and status(tlib) == K.KDA_OK
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    assert_out_close(out, ref_out)
    assert_state_close(fin, ref_fin, tol=2e-5)
    # 80 chunks do, in every chain and (with windows of more than three chunks) in every window
    T = 128 * 80
    big = R.linear_inputs([T], 8, seed=72, decay="head", device=DEV)
    out, fin = torch.empty_like(big["q"]), torch.empty_like(big["init_state"])
    ws = K.linear_prefill_workspace(1, T, 8, DEV) if windows else None
    assert call(tlib, big, out, fin, ws) == K.KDA_OK
    torch.cuda.synchronize()
    assert status(tlib) == K.KDA_ERR_DEVICE_TIMEOUT
    assert status(tlib) == K.KDA_OK
    out2, fin2 = K.linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], inp["init_state"],
                                  scale=SCALE)
    assert_out_close(out2, ref_out)
    assert_state_close(fin2, ref_fin, tol=2e-5)
    assert K.kda_device_status()[0] == K.KDA_OK
