"""Refusals of the operators around the attention layer, on the host: every case fails validation before the library
touches the device (the pointers are plain integers that are never dereferenced), or in the Python binding."""
import math

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


def resize(lib, **over):
    a = dict(bt=A, sl=A, nl=A, ol=A, ring=A, st=A, os=A, F=10, ps=16, B=2, P=4, cu=A, slots=A, pos=A, rows=A, T=5)
    a.update(over)
    return lib.kda_page_resize(a["bt"], a["sl"], a["nl"], a["ol"], a["ring"], a["st"], a["os"], a["F"], a["ps"], a["B"], a["P"],
                               a["cu"], a["slots"], a["pos"], a["rows"], a["T"], None)


@pytest.mark.parametrize("over,want", [
    (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(nl=None), INVALID), (dict(ol=None), INVALID),
    (dict(ring=None), INVALID), (dict(st=None), INVALID), (dict(os=None), INVALID), (dict(F=0), INVALID), (dict(B=-1), INVALID),
    (dict(P=0), INVALID), (dict(ps=0), INVALID), (dict(T=-1), INVALID), (dict(ps=4), UNSUPPORTED), (dict(ps=24), UNSUPPORTED),
    (dict(ps=2048), UNSUPPORTED), (dict(F=1 << 30), UNSUPPORTED), (dict(P=1 << 27), UNSUPPORTED), (dict(bt=A + 2), MISALIGNED),
    (dict(slots=A + 4), MISALIGNED), (dict(cu=A + 1), MISALIGNED), (dict(os=A + 2), MISALIGNED), (dict(rows=A + 2), MISALIGNED)])
def test_page_resize_arguments(lib, over, want):
    assert resize(lib, **over) == want


def rope(lib, **over):
    a = dict(q=A, k=A, v=A, qs=512, ks=256, vs=256, pos=A, f=A, rot=128, il=0, m=1.0, wq=A, wk=A, bf=1, eps=1e-6, qo=A, qos=512,
             ko=None, kos=0, kc=A, vc=A, kps=2 * 16 * 128, vps=2 * 16 * 128, pages=10, ps=16, slots=A, T=3, Hq=4, Hkv=2)
    a.update(over)
    return lib.kda_qk_norm_rope(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["pos"], a["f"], a["rot"], a["il"], a["m"],
                                a["wq"], a["wk"], a["bf"], a["eps"], a["qo"], a["qos"], a["ko"], a["kos"], a["kc"], a["vc"],
                                a["kps"], a["vps"], a["pages"], a["ps"], a["slots"], a["T"], a["Hq"], a["Hkv"], None)


@pytest.mark.parametrize("over,want", [
    (dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(rot=-16), INVALID), (dict(rot=144), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(il=2), INVALID), (dict(bf=2), INVALID), (dict(m=math.nan), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.inf), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(qo=None), INVALID), (dict(pos=None), INVALID), (dict(f=None), INVALID),
    (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(slots=None), INVALID), (dict(slots=None, kc=None, vc=None), INVALID),
    (dict(qs=504), INVALID), (dict(ks=128), INVALID), (dict(vs=255), INVALID), (dict(qos=0), INVALID), (dict(ko=A, kos=8), INVALID),
    (dict(qs=513), MISALIGNED), (dict(vs=260), MISALIGNED), (dict(qs=1 << 60), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(kps=100), INVALID), (dict(vps=2 * 16 * 128 + 4), MISALIGNED), (dict(ps=12), UNSUPPORTED), (dict(q=A + 8), MISALIGNED),
    (dict(wq=A + 4), MISALIGNED), (dict(pos=A + 2), MISALIGNED), (dict(slots=A + 4), MISALIGNED), (dict(f=A + 1), MISALIGNED),
    (dict(Hq=70000, qs=70000 * 128, qos=70000 * 128), UNSUPPORTED), (dict(T=0), OK), (dict(T=0, q=None, slots=A), OK)])
def test_qk_norm_rope_arguments(lib, over, want):
    assert rope(lib, **over) == want


def prefix(lib, **over):
    a = dict(q=A, k=A, v=A, ks=2 * 16 * 128, vs=2 * 16 * 128, pages=10, ps=16, bt=A, P=4, sl=A, cu=A, pl=A, G=2, out=A, lse=None,
             B=2, Hq=4, Hkv=2, scale=0.1, ws=A, nb=1 << 40)
    a.update(over)
    return lib.kda_attn_prefix_decode(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["pages"], a["ps"], a["bt"], a["P"], a["sl"],
                                      a["cu"], a["pl"], a["G"], a["out"], a["lse"], a["B"], a["Hq"], a["Hkv"], a["scale"], a["ws"],
                                      a["nb"], None)


@pytest.mark.parametrize("over,want", [
    (dict(B=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=5), INVALID), (dict(G=-1), INVALID),
    (dict(P=0), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID), (dict(scale=math.nan), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(bt=None), INVALID), (dict(sl=None), INVALID), (dict(cu=None), INVALID),
    (dict(pl=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID), (dict(ks=100), INVALID), (dict(ps=12), UNSUPPORTED),
    (dict(ps=2048), UNSUPPORTED), (dict(ks=1 << 39, pages=1), UNSUPPORTED), (dict(B=2**23, Hq=4), UNSUPPORTED),
    (dict(vs=2 * 16 * 128 + 4), MISALIGNED), (dict(q=A + 8), MISALIGNED), (dict(k=A + 8), MISALIGNED), (dict(out=A + 2), MISALIGNED),
    (dict(ws=A + 8), MISALIGNED), (dict(cu=A + 2), MISALIGNED), (dict(pl=A + 1), MISALIGNED), (dict(lse=A + 2), MISALIGNED), (dict(B=0), OK)])
def test_attn_prefix_decode_arguments(lib, over, want):
    assert prefix(lib, **over) == want


def test_attn_prefix_decode_workspace_size(lib):
    n = [K.kda_attn_prefix_decode_workspace_size(B, 64, 8, 10, 64, 4, sm_count=152) for B in (1, 8, 512)]
    assert 0 < n[0] < n[1] < n[2] and all(x % 16 == 0 for x in n)
    assert n[0] > K.kda_attn_decode_workspace_size(1, 64, 8, 10, 64, sm_count=152)
    for bad, status in (((1, 4, 3, 4, 16, 1), INVALID), ((1, 4, 2, 4, 16, -1), INVALID), ((1, 4, 2, 4, 24, 1), UNSUPPORTED),
                        ((2**23, 4, 2, 4, 16, 1), UNSUPPORTED)):
        assert lib.kda_attn_prefix_decode_workspace_size(*bad, 152) == status
    assert lib.kda_attn_prefix_decode_workspace_size(1, 4, 2, 4, 16, 1, -1) == INVALID


def test_binding_refuses_tensors_that_do_not_fit():
    i32 = dict(dtype=torch.int32)
    t, l, r, s = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(5, **i32), torch.zeros(2, **i32)

    def page(**over):
        a = dict(block_table=t, seq_lens=l, new_lens=l, free_pages=r, free_state=s, page_size=8, out_lens=l, out_state=s)
        K.kda_page_resize(**{**a, **over})

    for over, error in ((dict(block_table=t.long()), TypeError), (dict(seq_lens=torch.zeros(3, **i32)), ValueError),
                        (dict(free_state=r), ValueError), (dict(cu_tokens=l), ValueError), (dict(slots=l), TypeError),
                        (dict(slots=torch.zeros(4, dtype=torch.int64), rows=torch.zeros(5, **i32)), ValueError),
                        (dict(block_table=torch.zeros(3, 2, **i32).T), ValueError), (dict(page_size=1 << 40), ValueError),
                        (dict(out_lens=None), TypeError), (dict(), ValueError)):  # (the last: not on a GPU)
        with pytest.raises(error):
            page(**over)

    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(3, 4, 128, **bf), torch.zeros(3, 2, 128, **bf)
    pos, f, cache, slots = torch.zeros(3, **i32), torch.ones(64), torch.zeros(2, 2, 8, 128, **bf), torch.zeros(3, dtype=torch.int64)

    def rope(**over):
        a = dict(q=q, k=k, positions=pos, inv_freq=f, q_out=q, k_out=k)
        K.kda_qk_norm_rope(**{**a, **over})

    for over, error in ((dict(q=q.float()), TypeError), (dict(q=q[:, 0]), ValueError), (dict(k=k[:2]), ValueError),
                        (dict(q=q.transpose(0, 1)), ValueError), (dict(q=torch.zeros(3, 4, 256, **bf)[..., ::2]), ValueError),
                        (dict(positions=pos.long()), TypeError), (dict(positions=None), TypeError), (dict(q_out=None), TypeError),
                        (dict(q_weight=torch.ones(64)), ValueError), (dict(q_weight=torch.ones(128), k_weight=torch.ones(128, **bf)), TypeError),
                        (dict(k_weight=torch.ones(128, dtype=torch.float16)), TypeError), (dict(v=k), TypeError),
                        (dict(v=k, k_cache=cache, v_cache=cache), TypeError), (dict(slots=slots), TypeError),
                        (dict(v=k, k_cache=cache, v_cache=cache[:1], slots=slots), ValueError),
                        (dict(v=k, k_cache=cache, v_cache=cache, slots=slots.int()), TypeError), (dict(), ValueError)):
        with pytest.raises(error):
            rope(**over)

    q1, table, lens = torch.zeros(2, 4, 128, **bf), torch.zeros(2, 3, **i32), torch.zeros(2, **i32)

    def attend(**over):
        a = dict(q=q1, k_cache=cache, v_cache=cache, block_table=table, seq_lens=lens, cu_groups=lens, prefix_lens=lens[:1], out=q1,
                 scale=1.0, workspace=None)
        K.kda_attn_prefix_decode(**{**a, **over})

    for over, error in ((dict(q=q), ValueError), (dict(cu_groups=lens[:1]), ValueError), (dict(prefix_lens=lens), ValueError),
                        (dict(prefix_lens=None), TypeError), (dict(cu_groups=lens.float()), TypeError), (dict(lse=torch.zeros(2)), ValueError),
                        (dict(out=None), TypeError), (dict(seq_lens=pos), ValueError), (dict(v_cache=cache[:1]), ValueError), (dict(), ValueError)):
        with pytest.raises(error):
            attend(**over)
