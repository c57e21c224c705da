"""Pages, norm and rotation into them, and attention behind a shared prefix, run together as a server uses them.

Tolerances: the example's as in its own test (relL2 of the logits <= 3e-2). Step by step against 64 bits: queries and keys
are rounded to BF16 once (2^-8), as the reference's are from its own 64-bit values, so a score differs by less than two such
roundings of its terms; with the attention's own 2 x 2^-8 that is relL2 <= 4 x 2^-8 = 1.6e-2."""
import math
import os
import sys

import pytest
import torch

import kda_recurrent_gb300 as K
import serving_reference as R
from helpers import rel_l2

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_example_with_a_shared_prefix_matches_a_plain_pass():
    import hybrid_serving
    r = hybrid_serving.serve(batch=3, new_tokens=4, budget=0, check=True, prefix=100)
    assert 0 < r["worst"] <= 3e-2, r["worst"]
    assert (r["table"][1:, :6] == r["table"][0, :6]).all()  # 96 tokens in common pages
    assert len(set(r["table"][:, 6].tolist())) == 3
    held = sum(-(-n // 16) for n in r["lens"]) - 2 * 6
    assert r["free"] + held == r["table"].numel()


def test_example_gives_the_pages_of_cut_rows_back():
    import hybrid_serving
    r = hybrid_serving.serve(batch=4, new_tokens=60, budget=64)
    assert r["evictions"] >= 1 and r["free"] + sum(-(-n // 16) for n in r["lens"]) == r["table"].numel()


@pytest.mark.parametrize("Hq,Hkv,ps", [(32, 8, 16), (24, 8, 64)])
def test_steps_of_a_batch_behind_a_prefix(Hq, Hkv, ps):
    # 40 rows in two groups, of more tokens than are read row by row; three steps of one token a row, one row padding
    i32 = dict(dtype=torch.int32, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(Hq)
    B, first, prefix, room = 40, [0, 25, 40], [768, 512], 128
    P = (768 + room) // ps
    assert B * Hkv * P * ps * 512 > 72 << 20
    pages = sum(prefix) // ps + B * (room // ps)
    free = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    state = torch.tensor([0, pages], **i32)
    table, lens = torch.full((B, P), -1, **i32), torch.zeros(B, **i32)
    cache = torch.full((pages, 2, Hkv, ps, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    inv_freq, magnitude = K.rope_frequencies(128, factor=4.0, original_length=512, device=DEV)
    wq, wk = (1 + 0.1 * torch.randn(128, generator=gen, device=DEV) for _ in range(2))
    keys, values = ([torch.empty(0, Hkv, 128, dtype=torch.float64) for _ in range(B)] for _ in range(2))

    def bf16(*shape):
        return torch.randn(*shape, generator=gen, device=DEV).to(torch.bfloat16)

    def write(new_lens, tokens, padding=0):
        """Grows the rows; returns the new tokens' queries in and out, and their rows."""
        _, slots, positions, rows = K.page_resize(table, lens, new_lens, free, state, ps, max_tokens=tokens + padding)
        qkv = bf16(tokens + padding, Hq + 2 * Hkv, 128)
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        out = K.qk_norm_rope(q, k, positions, inv_freq, q_weight=wq, k_weight=wk, magnitude=magnitude, v=v, k_cache=cache[:, 0],
                             v_cache=cache[:, 1], slots=slots)
        turned = R.qk_rope(k, wk, positions, inv_freq, 1e-6, magnitude, False)
        for t, b in enumerate(rows.tolist()):
            if b >= 0:
                keys[b], values[b] = torch.cat([keys[b], turned[t:t + 1]]), torch.cat([values[b], v[t:t + 1].cpu().double()])
        return q, positions, out, rows

    # the first row of each group writes the prefix; the others begin with its pages
    leaders = torch.zeros(B, **i32)
    for g in range(2):
        leaders[first[g]] = prefix[g]
    write(leaders, sum(prefix))
    for g in range(2):
        a, b = first[g], first[g + 1]
        table[a:b, :prefix[g] // ps] = table[a, :prefix[g] // ps]
        lens[a:b] = prefix[g]
        for r in range(a + 1, b):
            keys[r], values[r] = keys[a], values[a]
    # own prompts of odd lengths; one row ends, and is padding from then on
    own = torch.randint(1, 60, (B,), generator=gen, device=DEV).to(torch.int32)
    write(lens + own, int(own.sum()), padding=3)
    target = lens.clone()
    target[7] = prefix[0]
    K.page_resize(table, lens, target, free, state, ps, max_tokens=0)
    lens[7] = 0
    groups, prefix_lens = torch.tensor(first, **i32), torch.tensor(prefix, **i32)
    for _ in range(3):
        q, positions, out, rows = write(lens + (lens > 0).to(torch.int32), B - 1, padding=1)
        assert rows.tolist() == [b for b in range(B) if b != 7] + [-1]
        batch_q = torch.zeros(B, Hq, 128, dtype=torch.bfloat16, device=DEV)
        batch_q[rows[:-1].long()] = out[:-1]
        got, lse = K.attn_prefix_decode(batch_q, cache[:, 0], cache[:, 1], table, lens, groups, prefix_lens, scale=128 ** -0.5,
                                        want_lse=True)
        turned = R.qk_rope(q, wq, positions, inv_freq, 1e-6, magnitude, False)
        assert (got[7] == 0).all() and torch.isinf(lse[7]).all()
        ref = torch.zeros(B, Hq, 128, dtype=torch.float64)
        for t, b in enumerate(rows.tolist()[:-1]):
            assert int(lens[b]) == keys[b].shape[0]
            x = torch.einsum("hgd,nhd->hgn", turned[t].view(Hkv, -1, 128), keys[b]) * 128 ** -0.5
            ref[b] = torch.einsum("hgn,nhd->hgd", torch.softmax(x, -1), values[b]).reshape(Hq, 128)
        assert rel_l2(got, ref) <= 1.6e-2
    assert K.kda_device_status()[0] == K.KDA_OK
