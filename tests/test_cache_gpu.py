"""Attention of one token over a paged key-value cache, and eviction from it, against plain 64-bit
forms.

Tolerances: an output is rounded once to BF16 (2^-9), after products with probabilities rounded to at
least BF16 (2^-9 of each term): relL2 <= 2 x 2^-9 = 3.9e-3, under the library's 1e-2. A score is an FP32
sum of 128 products: for these inputs (sum of |q_i k_i| scale < 15) its error is at most 128 x 2^-24 x 15
= 1.2e-4, which bounds lse absolutely and the weights relatively (with lse's own: 2.4e-4). What eviction
chooses and moves is exact."""
import math

import pytest
import torch

import hybrid_reference as R
import kda_recurrent_gb300 as K
from helpers import assert_out_close, rel_l2, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)
LSE_TOL, WEIGHT_TOL = 1.2e-4, 2.4e-4


def queries(B, Hq, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(B, Hq, 128, generator=gen).to(torch.bfloat16).to(DEV)


def check(q, c, weight=True, scale=SCALE):
    B, Hq, _ = q.shape
    cap = c["block_table"].shape[1] * c["k_cache"].shape[2]
    start = torch.rand(B, c["k_cache"].shape[1], cap, device=DEV)
    w = start.clone() if weight else None
    out, lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=scale,
                             want_lse=True, weight=w)
    ref_out, ref_lse, ref_w = R.attn_decode(q, c, scale)
    assert_out_close(out, ref_out)
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse).cpu(), empty) and (out.cpu()[empty] == 0).all()
    assert (lse.cpu().double() - ref_lse)[~empty].abs().max().item() <= LSE_TOL if (~empty).any() else True
    if weight:
        grown = (w - start).cpu()
        assert (w[(ref_w == 0).to(DEV)] == start[(ref_w == 0).to(DEV)]).all()
        # start < 1: the sum's own rounding adds 2^-24
        assert ((grown - ref_w).abs() <= WEIGHT_TOL * ref_w + 2.0 ** -23).all()
    return out, lse, w


@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("page", [8, 64])
def test_attn_lengths(n, page):
    check(queries(1, 4, n), R.cache_inputs([n], 2, page, seed=n, device=DEV))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (8, 8), (16, 4), (12, 2), (20, 1), (32, 2), (48, 1),
                                    (64, 8)])
@pytest.mark.parametrize("weight", [True, False])
def test_attn_heads(Hq, Hkv, weight):
    check(queries(3, Hq, Hq), R.cache_inputs([100, 1, 333], Hkv, 16, seed=Hq, device=DEV), weight)


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
def test_attn_page_sizes(page):
    check(queries(4, 4, 5), R.cache_inputs([700, 0, 65, 2050], 2, page, seed=page, device=DEV))


@pytest.mark.parametrize("lens,Hkv", [([5000], 1), ([9000, 10, 3000], 2), ([0, 0], 2), ([1] * 40, 3),
                                      ([100 * i for i in range(30)], 2)])
def test_attn_ragged(lens, Hkv):
    check(queries(len(lens), 2 * Hkv, 6), R.cache_inputs(lens, Hkv, 16, seed=41, max_pages=600, device=DEV))


@pytest.mark.parametrize("lens,Hq,Hkv", [([60000], 3, 1), ([20000], 20, 1), ([0, 30000, 7], 16, 2)])
def test_attn_long_row_of_few_heads(lens, Hq, Hkv):
    # a row cut between many SMs: each leaves one part, and the parts are more than a warp joins alone
    check(queries(len(lens), Hq, 54), R.cache_inputs(lens, Hkv, 64, seed=54, device=DEV))


def test_attn_table_far_wider_than_the_rows():
    # so many tiles that a table could hold pass 32-bit products: the work is cut in 64 bits
    c = R.cache_inputs([300, 5000], 2, 64, seed=55, max_pages=1 << 21, device=DEV)
    q = queries(2, 8, 55)
    narrow = dict(c, block_table=c["block_table"][:, :80].contiguous())
    out, lse, _ = check(q, narrow, weight=False)
    wide, wide_lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE,
                                   want_lse=True)
    assert torch.equal(wide, out) and torch.equal(wide_lse, lse)


def test_attn_many_short_rows():
    lens = [(7 * i) % 40 for i in range(300)]
    check(queries(300, 8, 56), R.cache_inputs(lens, 4, 8, seed=56, device=DEV))


def test_attn_one_token_is_its_value():
    c = R.cache_inputs([1], 1, 16, seed=42, device=DEV)
    out, lse, _ = check(queries(1, 1, 42), c)
    assert torch.equal(out[0, 0], c["v_cache"][c["block_table"][0, 0].long(), 0, 0])


def test_attn_combined_cache():
    c = R.cache_inputs([300, 77], 2, 32, seed=43, combined=True, device=DEV)
    assert not c["k_cache"].is_contiguous()
    check(queries(2, 6, 43), c)


def test_cache_of_one_page_has_any_page_stride():
    c = R.cache_inputs([13], 2, 16, seed=60, extra_pages=0, device=DEV)
    k, v = (torch.empty(2, 1, 16, 128, dtype=torch.bfloat16, device=DEV).transpose(0, 1).copy_(c[n]) for n in ("k_cache", "v_cache"))
    assert k.shape[0] == 1 and k.stride(0) < k[0].numel()
    q = queries(1, 4, 60)
    args = (c["block_table"], c["seq_lens"])
    assert torch.equal(K.attn_decode(q, k, v, *args, scale=SCALE), K.attn_decode(q, c["k_cache"], c["v_cache"], *args, scale=SCALE))
    w = torch.rand(1, 2, 16, device=DEV)
    for cache in ((k, v), (c["k_cache"], c["v_cache"])):
        K.cache_evict(*cache, *args, w.clone(), budget=5)
    assert torch.equal(k[:, :, :5], c["k_cache"][:, :, :5]) and torch.equal(v[:, :, :5], c["v_cache"][:, :, :5])


def test_attn_missing_pages_are_masked():
    c = R.cache_inputs([200, 64, 500], 2, 16, seed=44, device=DEV)
    c["block_table"][0, 3] = -1
    c["block_table"][1, :] = -1  # nothing is left of the row
    c["block_table"][2, 10:] = -1
    check(queries(3, 4, 44), c)
    assert K.kda_device_status()[0] == K.KDA_OK


def test_attn_bad_tables_are_reported():
    q = queries(2, 2, 45)
    c = R.cache_inputs([40, 90], 1, 16, seed=45, device=DEV)
    c["block_table"][1, 2] = c["k_cache"].shape[0]
    check(q, c)
    assert K.kda_device_status() == (K.KDA_ERR_DEVICE_INPUT, 1)
    c = R.cache_inputs([96, 90], 1, 16, seed=45, device=DEV)
    c["seq_lens"][0], c["seq_lens"][1] = 5000, -3
    check(q, c)
    assert K.kda_device_status()[0] == K.KDA_ERR_DEVICE_INPUT


def test_attn_shared_prefix_pages():
    c = R.cache_inputs([128, 64], 2, 32, seed=46, device=DEV)
    c["block_table"][1, :2] = c["block_table"][0, :2]
    check(queries(2, 4, 46), c)


@pytest.mark.parametrize("scale", [0.0, 4.0, -SCALE])
def test_attn_scales(scale):
    # 4.0: scores of several hundred, all weight on few tokens; their error grows alike
    q, c = queries(2, 4, 47), R.cache_inputs([150, 1000], 2, 16, seed=47, device=DEV)
    out, lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=scale, want_lse=True)
    ref_out, ref_lse, _ = R.attn_decode(q, c, scale)
    assert_out_close(out, ref_out)
    assert (lse.cpu().double() - ref_lse).abs().max().item() <= LSE_TOL * max(1.0, abs(scale) / SCALE)


def test_attn_nan_stays_in_its_row():
    c = R.cache_inputs([100, 100], 2, 16, seed=48, device=DEV)
    q = queries(2, 4, 48)
    out, lse, _ = check(q, c)
    c["k_cache"][c["block_table"][1, 2].long(), 0, 3] = math.nan
    out2, lse2 = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE,
                               want_lse=True)
    assert torch.equal(out2[0], out[0]) and torch.equal(out2[1, 2:], out[1, 2:])
    assert torch.isnan(lse2[1, :2]).all() and torch.isnan(out2[1, :2]).all()


@pytest.mark.parametrize("page", [8, 16])
def test_attn_weights_of_missing_pages_are_not_written(page):
    # ... whatever lies there, also in a row that a NaN key makes NaN
    c = R.cache_inputs([100, 90, 40], 2, page, seed=57, device=DEV)
    q, p = queries(3, 4, 57), c["block_table"]
    p[0, 1], p[1, 0], p[2, :] = -1, -1, -1
    c["k_cache"][p[1, 3].long(), 0, 3] = math.nan
    for fill in (-0.0, math.nan, 0.5):
        w = torch.full((3, 2, p.shape[1] * page), fill, device=DEV)
        K.attn_decode(q, c["k_cache"], c["v_cache"], p, c["seq_lens"], scale=SCALE, weight=w)
        masked = (p < 0).repeat_interleave(page, 1)
        masked |= torch.arange(p.shape[1] * page, device=DEV) >= c["seq_lens"][:, None]
        got = w.transpose(0, 1)[:, masked]
        assert torch.equal(got.view(torch.int32), torch.full_like(got, fill).view(torch.int32))
        if fill == 0.5:
            assert torch.isnan(w[1, 0][~masked[1]]).all() and torch.isfinite(w[1, 1]).all()
            assert (w[0][:, ~masked[0]] > 0.5).all()


def test_attn_infinite_scores():
    # a key of -inf scores takes no weight; a row of them gives zeros
    c = R.cache_inputs([40, 20], 1, 16, seed=49, device=DEV)
    q = queries(2, 1, 49).abs() + 0.5
    p = c["block_table"]
    c["k_cache"][p[0, 1].long(), 0, 2] = -math.inf
    for j in range(20):
        c["k_cache"][p[1, j // 16].long(), 0, j % 16] = -math.inf
    out, lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE, want_lse=True)
    c0 = dict(c, seq_lens=c["seq_lens"][:1], block_table=p[:1])
    ref_out, ref_lse, _ = R.attn_decode(q[:1], c0, SCALE)
    assert_out_close(out[:1], ref_out)
    assert (lse[0].cpu().double() - ref_lse[0]).abs().max() <= LSE_TOL
    assert (out[1] == 0).all() and lse[1, 0].item() == -math.inf


@pytest.mark.parametrize("lens,Hq,Hkv", [([1, 40, 100], 4, 2), ([5000, 17], 2, 1), ([700] * 40, 8, 4), ([60000], 20, 1)])
def test_attn_infinite_values(lens, Hq, Hkv):
    # an infinite value makes its channel infinite, opposite ones or a NaN make it NaN; the others keep their bits
    c = R.cache_inputs(lens, Hkv, 16, seed=58, device=DEV)
    q, p = queries(len(lens), Hq, 58), c["block_table"].cpu()
    clean, lse, _ = check(q, c, weight=False)
    rows = torch.arange(len(lens))
    first, last = p[:, 0].long(), p[rows, torch.tensor([(n - 1) // 16 for n in lens])].long()
    at = torch.tensor([(n - 1) % 16 for n in lens])
    v = c["v_cache"]
    v[first, :, 0, 3] = math.inf
    v[last, :, at, 126] = -math.inf
    v[last, :, at, 64] = math.nan
    v[first, :, 0, 9], v[last, :, at, 9] = math.inf, -math.inf
    out, lse2 = K.attn_decode(q, c["k_cache"], v, c["block_table"], c["seq_lens"], scale=SCALE, want_lse=True)
    ref, _, _ = R.attn_decode(q, c, SCALE)
    odd = [3, 9, 64, 126]
    assert torch.equal(out[..., odd].cpu().double().nan_to_num(nan=7.0), ref[..., odd].nan_to_num(nan=7.0))
    assert not torch.isfinite(ref[..., odd]).any()
    keep = [i for i in range(128) if i not in odd]
    assert torch.equal(out[..., keep], clean[..., keep]) and torch.equal(lse2, lse)


def test_attn_no_score_above_minus_infinity_gives_zeros():
    c = R.cache_inputs([20, 5000], 1, 16, seed=59, device=DEV)
    q = queries(2, 1, 59).abs() + 0.5
    c["k_cache"][...] = -math.inf
    c["v_cache"][:, :, 3] = math.inf
    out, lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE, want_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()


def test_attn_repeats_bit_for_bit():
    c = R.cache_inputs([3000, 17, 900], 2, 16, seed=50, device=DEV)
    q = queries(3, 8, 50)
    a = [K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE, want_lse=True)
         for _ in range(3)]
    assert all(torch.equal(x, y) for r in a[1:] for x, y in zip(r, a[0]))


def test_attn_offsets_pass_32_bits():
    pages, Hkv, ps = 140000, 8, 16  # 2.3e9 elements each
    k = torch.empty(pages, Hkv, ps, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    small = R.cache_inputs([40], Hkv, ps, seed=51, device=DEV)
    used = small["block_table"][0].long()
    far = torch.tensor([139999, 5, 133000], device=DEV)
    k[far], v[far] = small["k_cache"][used], small["v_cache"][used]
    c = dict(k_cache=k, v_cache=v, block_table=far[None].to(torch.int32), seq_lens=small["seq_lens"])
    q = queries(1, 8, 51)
    out = K.attn_decode(q, k, v, c["block_table"], c["seq_lens"], scale=SCALE)
    ref_out, _, _ = R.attn_decode(q, small, SCALE)
    assert_out_close(out, ref_out)


def test_attn_workspace_too_small_is_refused():
    c = R.cache_inputs([40], 2, 16, seed=52, device=DEV)
    q = queries(1, 2, 52)
    with pytest.raises(K.KdaError) as e:
        K.kda_attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], torch.empty_like(q), SCALE,
                          torch.empty(0, dtype=torch.uint8, device=DEV))
    assert e.value.status == K.KDA_ERR_INVALID_ARG


def test_attn_on_another_stream_and_graph():
    c = R.cache_inputs([3000, 5], 2, 16, seed=53, device=DEV)
    q = queries(2, 8, 53)
    ref = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE)
    out = torch.zeros_like(q)
    ws = K.attn_decode_workspace(2, 8, 2, c["block_table"].shape[1], 16, False, DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    K.kda_attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], out, SCALE, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        K.kda_attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], out, SCALE, ws)
    out.zero_()
    c["seq_lens"][0] = 1000  # lengths are read on the device: one graph serves them all
    g.replay()
    torch.cuda.synchronize()
    ref = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE)
    assert torch.equal(out, ref)


# ---------------------------------------------------------------- eviction


def check_evict(lens, Hkv, page, budget, sink, recent, *, seed, weights=None, in_place=False, max_pages=None):
    dst_pages = 0 if in_place else len(lens) * -(-budget // page)
    c = R.cache_inputs(lens, Hkv, page, seed=seed, extra_pages=3 + dst_pages, max_pages=max_pages, device=DEV)
    B, P = c["block_table"].shape
    cap = P * page
    gen = torch.Generator().manual_seed(seed)
    w = torch.rand(B, Hkv, cap, generator=gen) ** 4 if weights is None else weights(B, Hkv, cap, gen)
    if in_place:
        dst_table, dst_weight = None, None
        to = c["block_table"].cpu()
    else:
        per = min(P, -(-budget // page))
        to = torch.full((B, P), -1, dtype=torch.int32)
        for b in range(B):
            to[b, :per] = torch.tensor(c["free"][b * per:(b + 1) * per], dtype=torch.int32)
        dst_table, dst_weight = to.to(DEV), torch.full((B, Hkv, cap), 7.0, device=DEV)
    k0, v0, table = c["k_cache"].cpu(), c["v_cache"].cpu(), c["block_table"].cpu()
    wd = w.to(DEV)
    new_lens, kept = K.cache_evict(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], wd, budget=budget,
                                   sink=sink, recent=recent, dst_table=dst_table, dst_weight=dst_weight)
    want_k, want_v = k0.clone(), v0.clone()
    want_w = w.clone() if in_place else torch.full((B, Hkv, cap), 7.0)
    want_kept = torch.full((B, Hkv, budget), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        m = min(n, budget)
        for h in range(Hkv):
            ids = R.evict_choice(w[b, h].tolist(), n, budget, sink, recent)
            assert len(ids) == m
            want_kept[b, h, :m] = torch.tensor(ids, dtype=torch.int32)
            want_w[b, h, :n] = 0
            want_w[b, h, :m] = w[b, h, ids]
            i, j = torch.arange(m), torch.tensor(ids, dtype=torch.long)
            src, dst = table[b, j // page].long(), to[b, i // page].long()
            want_k[dst, h, i % page] = k0[src, h, j % page]
            want_v[dst, h, i % page] = v0[src, h, j % page]
    assert new_lens.tolist() == [min(n, budget) for n in lens]
    assert torch.equal(kept.cpu(), want_kept)
    got_w = (wd if in_place else dst_weight).cpu()
    assert torch.equal(got_w.nan_to_num(nan=-5.0), want_w.nan_to_num(nan=-5.0))
    for got, want in ((c["k_cache"], want_k), (c["v_cache"], want_v)):
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    assert K.kda_device_status()[0] == K.KDA_OK


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,Hkv,page,budget,sink,recent", [
    ([100], 1, 16, 40, 4, 10), ([64, 65, 63], 2, 16, 64, 0, 0), ([300, 0, 1, 299], 3, 8, 33, 2, 31),
    ([500], 2, 64, 1, 0, 0), ([500], 2, 64, 1, 0, 1), ([500], 2, 64, 1, 1, 0), ([257], 1, 32, 256, 128, 128),
    ([1000, 2000], 2, 128, 700, 0, 700), ([5000, 4096, 4097], 2, 16, 3000, 16, 500), ([9000], 1, 64, 50, 0, 7)])
def test_evict(lens, Hkv, page, budget, sink, recent, in_place):
    check_evict(lens, Hkv, page, budget, sink, recent, seed=61, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,Hkv,page,budget,sink,recent", [
    ([40000], 2, 64, 9000, 16, 500), ([33000, 9, 70001], 1, 128, 20000, 3, 0), ([131072], 1, 256, 131071, 0, 1),
    ([131100], 1, 32, 700, 4, 100), ([36000] * 20, 1, 256, 300, 0, 10)])
def test_evict_long_rows(lens, Hkv, page, budget, sink, recent, in_place):
    check_evict(lens, Hkv, page, budget, sink, recent, seed=67, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long_row_of_ties(in_place):
    def weights(B, H, cap, gen):
        return (torch.rand(B, H, cap, generator=gen) * 3).floor()
    check_evict([50001], 2, 64, 30000, 5, 77, seed=68, in_place=in_place, weights=weights)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_many_heads(in_place):
    check_evict([200 + 10 * i for i in range(40)], 8, 16, 128, 4, 32, seed=62, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kind", ["equal", "few", "signs", "special", "low_bits"])
def test_evict_ties_and_special_weights(kind, in_place):
    def weights(B, H, cap, gen):
        r = torch.rand(B, H, cap, generator=gen)
        if kind == "equal":
            return torch.zeros(B, H, cap)
        if kind == "few":
            return (r * 3).floor()
        if kind == "signs":
            return torch.where(r < 0.3, torch.full_like(r, -0.0), torch.where(r < 0.6, torch.zeros_like(r), 1e-40 - r))
        if kind == "low_bits":
            return 1.0 + (r * 40).floor() * 2.0 ** -23
        w = r.clone()
        w[r < 0.2], w[(r > 0.2) & (r < 0.3)], w[(r > 0.3) & (r < 0.4)] = math.nan, math.inf, -math.inf
        return w

    check_evict([400, 90, 5000], 2, 16, 100, 3, 20, seed=63, weights=weights, in_place=in_place)


def test_evict_in_place_by_slices():
    # as many heads as the middle width of column slices takes
    check_evict([260 + 7 * i for i in range(10)], 5, 16, 200, 4, 50, seed=69, in_place=True)


@pytest.mark.parametrize("rows,Hkv", [(19, 1), (10, 2), (38, 1), (13, 3), (19, 4), (11, 7)])
def test_evict_in_place_beside_the_slices_limits(rows, Hkv):
    check_evict([230 + 11 * i for i in range(rows)], Hkv, 16, 200, 4, 50, seed=72, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_offsets_pass_32_bits(in_place):
    pages, ps = 140000, 16  # 2.3e9 elements each
    k = torch.empty(pages, 8, ps, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    at = torch.tensor([139999, 5, 133000], device=DEV)
    to = at if in_place else torch.tensor([139000, 6, 132000], device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(70)
    for x in (k, v):
        x[at] = torch.randn(3, 8, ps, 128, generator=gen, device=DEV).to(torch.bfloat16)
    before = [x[at].transpose(0, 1).reshape(8, 3 * ps, 128).clone() for x in (k, v)]
    w = torch.rand(1, 8, 3 * ps, generator=gen, device=DEV)
    lens = torch.tensor([45], dtype=torch.int32, device=DEV)
    new_lens, kept = K.cache_evict(k, v, at[None].to(torch.int32), lens, w, budget=33, sink=1, recent=3,
                                   dst_table=None if in_place else to[None].to(torch.int32))
    assert new_lens.item() == 33
    for x, old in zip((k, v), before):
        got = x[to].transpose(0, 1).reshape(8, 3 * ps, 128)[:, :33]
        assert torch.equal(got, old.gather(1, kept[0].long()[..., None].expand(8, 33, 128)))


def test_calls_without_waits_equal_calls_with_waits():
    """Launches overlap the work before them: every call here reads what the one before it writes."""
    def run(wait):
        c = R.cache_inputs([700, 300], 2, 16, seed=71, device=DEV)
        cap = c["block_table"].shape[1] * 16
        w, lens = torch.zeros(2, 2, cap, device=DEV), c["seq_lens"].clone()
        pool = torch.zeros(2, 8, 128, 128, device=DEV)
        slots, g = torch.arange(2, dtype=torch.int32, device=DEV), torch.full((8,), -0.1, device=DEV)
        cu = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
        x, seen = queries(2, 8, 71), []
        ws = K.attn_decode_workspace(2, 8, 2, c["block_table"].shape[1], 16, True, DEV)
        pause = torch.cuda.synchronize if wait else lambda: None
        for step in range(12):
            x = K.linear_decode(x, x, x, g, slots, pool, scale=0.3)
            pause()
            x = K.attn_decode(x, c["k_cache"], c["v_cache"], c["block_table"], lens, scale=SCALE, weight=w, workspace=ws)
            pause()
            x, state = K.linear_prefill(x, x, x, g, cu, pool, scale=0.3)
            pause()
            pool.copy_(state)
            if step % 4 == 3:
                lens, kept = K.cache_evict(c["k_cache"], c["v_cache"], c["block_table"], lens, w, budget=250 - 40 * (step // 4),
                                           sink=2, recent=30)
                pause()
                seen.append(kept)
            x = (x.float() / x.float().norm(dim=-1, keepdim=True)).to(torch.bfloat16)
        return [x, pool, w, lens, c["k_cache"], c["v_cache"], *seen]
    for a, b in zip(run(True), run(False)):
        assert torch.equal(a.nan_to_num(), b.nan_to_num())


def test_evict_new_lens_may_be_seq_lens():
    c = R.cache_inputs([100, 20], 2, 16, seed=64, device=DEV)
    w = torch.rand(2, 2, c["block_table"].shape[1] * 16, device=DEV)
    kept = torch.empty(2, 2, 50, dtype=torch.int32, device=DEV)
    K.kda_cache_evict(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], w, c["seq_lens"], kept, 50)
    assert c["seq_lens"].tolist() == [50, 20]
    assert (kept[1, :, :20] == torch.arange(20, device=DEV)).all()


def test_evict_missing_page_is_reported():
    c = R.cache_inputs([100], 1, 16, seed=65, device=DEV)
    c["block_table"][0, 2] = -1
    w = torch.ones(1, 1, c["block_table"].shape[1] * 16, device=DEV)
    K.cache_evict(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], w, budget=60, recent=60)
    assert K.kda_device_status() == (K.KDA_ERR_DEVICE_INPUT, 0)


def test_attention_then_eviction():
    """The weights one operator gathers are what the other chooses by."""
    c = R.cache_inputs([300, 250], 2, 16, seed=66, device=DEV)
    cap = c["block_table"].shape[1] * 16
    w = torch.zeros(2, 2, cap, device=DEV)
    for step in range(3):
        K.attn_decode(queries(2, 8, step), c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE,
                      weight=w)
    assert rel_l2(w.sum(-1), torch.full((2, 2), 12.0)) <= 1e-5  # 3 steps x 4 query heads
    q, seen = queries(2, 8, 9), w.cpu()
    new_lens, kept = K.cache_evict(c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], w, budget=100, recent=16)
    for b, n in enumerate((300, 250)):
        for h in range(2):
            assert kept[b, h].tolist() == R.evict_choice(seen[b, h].tolist(), n, 100, 0, 16)
    c["seq_lens"] = new_lens
    out = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], new_lens, scale=SCALE)
    ref_out, _, _ = R.attn_decode(q, c, SCALE)
    assert_out_close(out, ref_out)
    assert to_np(w[:, :, 100:]).max() == 0
