"""Refusals of the operators beside KDA layers, on the host: every case fails validation before the
library touches the device (the pointers are plain integers that are never dereferenced), or in the
Python binding before the library is called."""
import math
import os
import re

import pytest
import torch

import kda_recurrent_gb300 as K
from kda_recurrent_gb300 import build as kbuild

A = 0x10000  # a 16-byte-aligned fake address (never dereferenced)
OK, INVALID, UNSUPPORTED, MISALIGNED = K.KDA_OK, K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_MISALIGNED


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return K.load()


def prefill(lib, **over):
    a = dict(q=A, k=A, v=A, g=A, per=0, cu=A, init=None, out=A, fin=None, N=1, T=32, H=2, scale=0.1, ws=None, nb=0)
    a.update(over)
    return lib.kda_linear_prefill(a["q"], a["k"], a["v"], a["g"], a["per"], a["cu"], a["init"], a["out"], a["fin"],
                                  a["N"], a["T"], a["H"], a["scale"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("over,want", [
    (dict(N=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(scale=math.nan), INVALID),
    (dict(scale=math.inf), INVALID), (dict(per=2), INVALID), (dict(N=0), INVALID), (dict(cu=None), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(out=None), INVALID), (dict(q=A + 8), MISALIGNED), (dict(k=A + 2), MISALIGNED), (dict(v=A + 4), MISALIGNED),
    (dict(out=A + 8), MISALIGNED), (dict(init=A + 4), MISALIGNED), (dict(fin=A + 4), MISALIGNED),
    (dict(g=A + 2), MISALIGNED), (dict(cu=A + 1), MISALIGNED), (dict(ws=A + 8, nb=1 << 30), MISALIGNED),
    (dict(T=2**31 - 1, H=100), UNSUPPORTED), (dict(N=2**30, H=100), UNSUPPORTED),
    (dict(N=0, T=0), OK), (dict(T=0), OK)])
def test_linear_prefill_arguments(lib, over, want):
    assert prefill(lib, **over) == want


def test_linear_prefill_workspace_size(lib):
    assert K.kda_linear_prefill_workspace_size(1, 8192, 8, sm_count=152) >= 0
    assert K.kda_linear_prefill_workspace_size(0, 0, 8, sm_count=152) == 0
    for bad in ((-1, 1, 1), (1, -1, 1), (1, 1, 0)):
        with pytest.raises(K.KdaError) as e:
            K.kda_linear_prefill_workspace_size(*bad, sm_count=152)
        assert e.value.status == INVALID


@pytest.mark.parametrize("N,T,H", [(2**30, 0, 100), (2**31 - 1, 2**31 - 1, 2**31 - 1), (1, 2**31 - 1, 100), (2**24, 5, 2)])
def test_linear_prefill_workspace_size_has_the_calls_limits(lib, N, T, H):
    assert lib.kda_linear_prefill_workspace_size(N, T, H, 152) == UNSUPPORTED == prefill(lib, N=N, T=T, H=H)


def decode(lib, **over):
    a = dict(q=A, k=A, v=A, g=A, per=0, slot=A, pool=A, slots=4, dt=0, out=A, R=3, H=2, scale=0.1)
    a.update(over)
    return lib.kda_linear_decode(a["q"], a["k"], a["v"], a["g"], a["per"], a["slot"], a["pool"], a["slots"], a["dt"],
                                 a["out"], a["R"], a["H"], a["scale"], None)


@pytest.mark.parametrize("over,want", [
    (dict(R=-1), INVALID), (dict(H=0), INVALID), (dict(slots=0), INVALID), (dict(dt=2), INVALID), (dict(per=-1), INVALID),
    (dict(scale=math.nan), INVALID), (dict(q=None), INVALID), (dict(g=None), INVALID), (dict(slot=None), INVALID),
    (dict(pool=None), INVALID), (dict(out=None), INVALID), (dict(k=A + 8), MISALIGNED), (dict(pool=A + 8), MISALIGNED),
    (dict(slot=A + 2), MISALIGNED), (dict(g=A + 2), MISALIGNED), (dict(R=2**31 - 1, H=64), UNSUPPORTED),
    (dict(slots=1 << 60), UNSUPPORTED), (dict(R=0), OK)])
def test_linear_decode_arguments(lib, over, want):
    assert decode(lib, **over) == want


def attn(lib, **over):
    a = dict(q=A, k=A, v=A, ks=2 * 16 * 128, vs=2 * 16 * 128, pages=10, ps=16, bt=A, P=4, sl=A, out=A, lse=None,
             w=None, B=2, Hq=4, Hkv=2, scale=0.1, ws=A, nb=1 << 40)
    a.update(over)
    return lib.kda_attn_decode(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["ps"], a["bt"], a["P"], a["sl"],
                               a["out"], a["lse"], a["w"], a["B"], a["Hq"], a["Hkv"], a["scale"], a["ws"], a["nb"], None)


CACHE = [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(pages=0), INVALID), (dict(P=0), INVALID),
    (dict(ps=0), INVALID), (dict(ps=4), UNSUPPORTED), (dict(ps=24, ks=1 << 20, vs=1 << 20), UNSUPPORTED),
    (dict(ps=2048, ks=1 << 30, vs=1 << 30), UNSUPPORTED), (dict(ks=4095), INVALID), (dict(vs=4000), INVALID),
    (dict(ks=4100), MISALIGNED), (dict(vs=4097), MISALIGNED), (dict(P=1 << 27), UNSUPPORTED),
    (dict(pages=1 << 32), UNSUPPORTED), (dict(ks=1 << 58), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(k=A + 8), MISALIGNED), (dict(v=A + 2), MISALIGNED),
    (dict(bt=A + 2), MISALIGNED), (dict(sl=A + 1), MISALIGNED), (dict(B=0), OK)]


@pytest.mark.parametrize("over,want", CACHE + [
    (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(q=A + 8), MISALIGNED), (dict(out=A + 8), MISALIGNED),
    (dict(ws=A + 8), MISALIGNED), (dict(lse=A + 2), MISALIGNED), (dict(w=A + 4), MISALIGNED),
    (dict(B=1 << 23, Hq=64, Hkv=64, ks=1 << 20, vs=1 << 20), UNSUPPORTED)])
def test_attn_decode_arguments(lib, over, want):
    assert attn(lib, **over) == want


def test_attn_decode_workspace_size(lib):
    assert K.kda_attn_decode_workspace_size(2, 8, 2, 10, 16, sm_count=152) >= 0
    assert (K.kda_attn_decode_workspace_size(2, 8, 2, 10, 16, True, sm_count=152)
            >= K.kda_attn_decode_workspace_size(2, 8, 2, 10, 16, False, sm_count=152))
    for bad in ((-1, 8, 2, 10, 16), (2, 7, 2, 10, 16), (2, 0, 2, 10, 16), (2, 8, 0, 10, 16), (2, 8, 2, 0, 16),
                (2, 8, 2, 10, 0)):
        with pytest.raises(K.KdaError) as e:
            K.kda_attn_decode_workspace_size(*bad, sm_count=152)
        assert e.value.status == INVALID


@pytest.mark.parametrize("B,Hq,Hkv,P,ps", [(2**31 - 1, 64, 64, 1 << 20, 1024), (1 << 23, 64, 1, 4, 16), (2, 4, 2, 1 << 27, 16),
                                           (2, 4, 2, 10, 4), (2, 4, 2, 10, 24), (2, 4, 2, 10, 2048), (1, 1 << 20, 1 << 20, 4, 1024)])
@pytest.mark.parametrize("weight", [0, 1])
def test_attn_decode_workspace_size_has_the_calls_limits(lib, B, Hq, Hkv, P, ps, weight):
    assert lib.kda_attn_decode_workspace_size(B, Hq, Hkv, P, ps, weight, 152) == UNSUPPORTED
    assert attn(lib, B=B, Hq=Hq, Hkv=Hkv, P=P, ps=ps, ks=1 << 40, vs=1 << 40) == UNSUPPORTED


def test_attn_decode_workspace_size_of_the_largest_calls(lib):
    # every size that the call takes has its bytes in 64 bits
    n = lib.kda_attn_decode_workspace_size((1 << 24) - 1, 1, 1, (1 << 20) - 1, 1024, 1, 152)
    assert n >= ((1 << 24) - 1) * ((1 << 20) - 1) * 1024 * 4


def evict(lib, **over):
    a = dict(k=A, v=A, ks=2 * 16 * 128, vs=2 * 16 * 128, pages=10, ps=16, bt=A, dt=None, P=4, sl=A, w=A, dw=A, nl=A,
             kept=A, B=2, Hkv=2, budget=20, sink=2, recent=5)
    a.update(over)
    return lib.kda_cache_evict(a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["ps"], a["bt"], a["dt"], a["P"], a["sl"],
                               a["w"], a["dw"], a["nl"], a["kept"], a["B"], a["Hkv"], a["budget"], a["sink"],
                               a["recent"], None)


@pytest.mark.parametrize("over,want", CACHE + [
    (dict(budget=0), INVALID), (dict(sink=-1), INVALID), (dict(recent=-1), INVALID), (dict(sink=16), INVALID),
    (dict(sink=2**31 - 1, recent=2**31 - 1), INVALID), (dict(w=None), INVALID), (dict(dw=None), INVALID),
    (dict(nl=None), INVALID), (dict(kept=None), INVALID), (dict(w=A + 4), MISALIGNED), (dict(dw=A + 4), MISALIGNED),
    (dict(nl=A + 2), MISALIGNED), (dict(kept=A + 2), MISALIGNED), (dict(dt=A + 2), MISALIGNED)])
def test_cache_evict_arguments(lib, over, want):
    assert evict(lib, **over) == want


@pytest.mark.parametrize("name", ["kda_linear_prefill", "kda_linear_decode", "kda_attn_decode", "kda_cache_evict"])
def test_kernels_wait_for_the_launch_before_they_touch_memory(name):
    """These kernels may start while the launch before them still runs. In each one's source the wait comes first:
    unconditionally, and before anything that reads or writes global memory."""
    text = open(os.path.join(kbuild.CSRC, name + ".cu")).read()
    bodies = re.findall(r"__global__ void.*?\n(.*?)\n}\n", text, re.S)
    assert len(bodies) == text.count("__global__ void") >= 1
    for body in bodies:
        before, wait, _ = body.partition("\n    wait_for_prior();")
        assert wait and body.count("wait_for_prior") == 1
        touches = [m for m in re.findall(r"\b(\w+)\(", before) if m in ("row_length", "load_block", "load", "__ldg", "__ldcs",
                                                                       "rank_sequences", "item_of", "tma_load", "next_item")]
        assert not touches, touches


# ---------------------------------------------------------------- the build


@pytest.mark.parametrize("fails", ["compile", "headers"])
def test_the_library_builds_without_the_compiled_binding(lib, monkeypatch, tmp_path, fails):
    """Who calls the C functions only, or the KDA calls, needs no Python or torch headers."""
    path = tmp_path / "binding.so"
    path.write_bytes(b"")
    os.utime(path, (0, 0))  # of older sources
    monkeypatch.setattr(kbuild, "BINDING_PATH", str(path))
    if fails == "compile":
        def refuse():
            raise RuntimeError("g++ failed on binding.cpp")
        monkeypatch.setattr(kbuild, "_compile_binding", refuse)
    else:
        monkeypatch.setattr(kbuild.sysconfig, "get_paths", lambda: {"include": str(tmp_path / "none")})
    with pytest.warns(UserWarning, match="binding"):
        assert kbuild.build() == kbuild.LIB_PATH
    assert kbuild.up_to_date() and not path.exists()
    monkeypatch.setattr(K, "_native", None)
    with pytest.raises(RuntimeError, match="binding not built"):
        K.linear_decode(*[torch.zeros(1, 1, 128, dtype=torch.bfloat16)] * 3, None, None, None, scale=1.0)


# ---------------------------------------------------------------- the binding's own checks


def bf16(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_host_tensors_are_refused():
    q, cu = bf16(4, 2, 128), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        K.linear_prefill(q, q, q, torch.zeros(2), cu, scale=1.0)
    with pytest.raises(ValueError, match="CUDA device"):
        K.linear_decode(q, q, q, torch.zeros(4, 2), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2, 128, 128),
                        scale=1.0)
    k, bt, n = bf16(3, 2, 16, 128), torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA device"):
        K.attn_decode(q, k, k, bt, n, scale=1.0)
    with pytest.raises(ValueError, match="CUDA device"):
        K.cache_evict(k, k, bt, n, torch.zeros(4, 2, 32), budget=8)


def test_shapes_and_types_are_checked():
    q, cu, g = bf16(4, 2, 128), torch.tensor([0, 4], dtype=torch.int32), torch.zeros(2)
    with pytest.raises(TypeError, match="k: expected"):
        K.linear_prefill(q, q.float(), q, g, cu, scale=1.0)
    with pytest.raises(ValueError, match="log_decay"):
        K.linear_prefill(q, q, q, torch.zeros(3), cu, scale=1.0)
    with pytest.raises(ValueError, match="log_decay"):
        K.linear_prefill(q, q, q, torch.zeros(2, 4), cu, scale=1.0)
    with pytest.raises(ValueError, match="q: expected shape"):
        K.linear_prefill(bf16(4, 2, 64), q, q, g, cu, scale=1.0)
    with pytest.raises(ValueError, match="contiguous"):
        K.linear_prefill(q, bf16(2, 4, 128).transpose(0, 1), q, g, cu, scale=1.0)
    with pytest.raises(ValueError, match="init_state"):
        K.linear_prefill(q, q, q, g, cu, torch.zeros(2, 2, 128, 128), scale=1.0)
    slot = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError, match="state_pool"):
        K.linear_decode(q, q, q, g, slot, torch.zeros(4, 2, 128, 128, dtype=torch.float16), scale=1.0)
    with pytest.raises(TypeError, match="slot_idx"):
        K.linear_decode(q, q, q, g, slot.long(), torch.zeros(4, 2, 128, 128), scale=1.0)
    k, bt, n = bf16(3, 2, 16, 128), torch.zeros(4, 2, dtype=torch.int32), torch.ones(4, dtype=torch.int32)
    out, ws = torch.zeros_like(q), torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="page must be contiguous"):
        K.kda_attn_decode(q, bf16(3, 16, 2, 128).transpose(1, 2), k, bt, n, out, 1.0, ws)
    with pytest.raises(ValueError, match="v_cache: expected shape"):
        K.kda_attn_decode(q, k, bf16(3, 2, 8, 128), bt, n, out, 1.0, ws)
    with pytest.raises(ValueError, match="block_table"):
        K.kda_attn_decode(q, k, k, bt[:3], n, out, 1.0, ws)
    with pytest.raises(ValueError, match="weight"):
        K.kda_attn_decode(q, k, k, bt, n, out, 1.0, ws, weight=torch.zeros(4, 2, 16))
    with pytest.raises(ValueError, match="lse"):
        K.kda_attn_decode(q, k, k, bt, n, out, 1.0, ws, lse=torch.zeros(4, 1))
    with pytest.raises(ValueError, match="kept"):
        K.kda_cache_evict(k, k, bt, n, torch.zeros(4, 2, 32), torch.zeros(4, dtype=torch.int32),
                          torch.zeros(4, 2, 7, dtype=torch.int32), 8)
