"""Attention of one token for rows that share a prefix, against the plain 64-bit form on the rows' own tables.

Tolerances: an output is rounded once to BF16 (2^-8 of it at most); the prefix's probabilities are rounded to BF16 each
(2^-8), which for independent values adds an error of at most 2^-8 of the output's norm: relL2 <= 2 x 2^-8 = 7.8e-3, under
the library's 1e-2. A score is an FP32 sum of 128 products: for these inputs (sum of |q_i k_i| scale < 15) its error is at
most 128 x 2^-24 x 15 = 1.2e-4, which bounds lse absolutely."""
import math

import pytest
import torch

import hybrid_reference as H
import kda_recurrent_gb300 as K
import serving_reference as R
from helpers import assert_out_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)
LSE_TOL = 1.2e-4


def queries(B, Hq, seed):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(B, Hq, 128, generator=gen).to(torch.bfloat16).to(DEV)


def widened(c, Hq):
    """With a table so wide that the call shares the prefix (it reads rows of narrow tables one by one)."""
    rows, width = c["block_table"].shape
    _, Hkv, page, _ = c["k_cache"].shape
    tokens = (73 << 20) // (512 * rows * Hkv * -(-Hq // Hkv // 16)) + page
    table = torch.full((rows, max(width, -(-tokens // page))), -1, dtype=torch.int32, device=DEV)
    table[:, :width] = c["block_table"]
    return dict(c, block_table=table)


def call(q, c, scale=SCALE, **kw):
    return K.attn_prefix_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], c["cu_groups"], c["prefix_lens"],
                                scale=scale, want_lse=True, **kw)


def check(q, c, scale=SCALE, lse_tol=LSE_TOL, status=K.KDA_OK, ref=None):
    K.kda_device_status()
    out, lse = call(q, widened(c, q.shape[1]), scale)
    assert K.kda_device_status()[0] == status
    ref_out, ref_lse, _ = ref or H.attn_decode(q, c, scale)
    empty = torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(lse).cpu(), empty) and (out.cpu()[empty] == 0).all()
    assert_out_close(out, ref_out)
    assert (lse.cpu().double() - ref_lse)[~empty].abs().max().item() <= lse_tol if (~empty).any() else True
    return out, lse


def inputs(first, prefix, tails, Hkv, page, seed, **kw):
    """Rows of their group's prefix and `tails` tokens more (less where negative)."""
    group = [g for g in range(len(prefix)) for _ in range(first[g], first[g + 1])]
    return R.prefix_inputs(first, prefix, [max(0, prefix[g] + t) for g, t in zip(group, tails)], Hkv, page, seed=seed, device=DEV, **kw)


@pytest.mark.parametrize("n", [0, 1, 16, 127, 128, 129, 200, 255, 256, 257, 384, 1000])
@pytest.mark.parametrize("page", [8, 64, 256])
def test_prefix_lengths(n, page):
    check(queries(3, 4, n), inputs([0, 3], [n], [1, 50, 7], 2, page, n + 1))


@pytest.mark.parametrize("tail", [0, 1, 15, 16, 17, 129, 700])
def test_prefix_tails(tail):
    check(queries(4, 4, tail), inputs([0, 4], [256], [tail] * 4, 2, 16, tail + 1))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (2, 2), (3, 1), (8, 8), (12, 2), (20, 1), (48, 1), (64, 8)])
@pytest.mark.parametrize("rows", [2, 9])
def test_prefix_heads(Hq, Hkv, rows):
    check(queries(rows, Hq, Hq), inputs([0, rows], [300], [10 + i for i in range(rows)], Hkv, 16, Hq))


@pytest.mark.parametrize("rows,group", [(16, 8), (17, 8), (31, 8), (32, 8), (33, 8), (48, 8), (49, 8), (43, 3), (86, 3), (130, 5)])
def test_prefix_tiles_of_query_rows(rows, group):
    # 128, 136, ... 650 query rows of a key head: one tile, two, and several pairs whose last has one or two
    check(queries(rows, group, rows), inputs([0, rows], [700], [(7 * i) % 40 for i in range(rows)], 1, 32, rows))


@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("combined", [False, True])
def test_prefix_page_sizes(page, combined):
    check(queries(6, 4, 5), inputs([0, 2, 6], [2100, 515], [3, 60, 0, 1, 2, 900], 2, page, page, combined=combined))


def test_prefix_rows_of_several_kinds():
    # groups of one row, of none, rows of no group, rows shorter than the prefix, rows of no tokens
    first, prefix = [2, 3, 3, 7, 7, 12], [300, 500, 640, 0, 200]
    lens = [100, 0, 333, 700, 640, 100, 0, 0, 200, 220, 150, 900, 5, 400]
    c = R.prefix_inputs(first, prefix, lens, 2, 16, seed=3, device=DEV)
    kinds = R.prefix_inputs([0, 2, 3, 3, 7, 7, 12, 14], [0, 300, 500, 640, 0, 200, 0], lens, 2, 16, seed=3, device=DEV)
    kinds["cu_groups"], kinds["prefix_lens"] = c["cu_groups"], c["prefix_lens"]  # (cu_groups then leaves out rows 0, 1, 12 and 13)
    check(queries(14, 8, 3), kinds)


def test_prefix_first_row_of_a_group_is_padding():
    c = R.prefix_inputs([0, 5], [512], [0, 100, 600, 512, 700], 2, 16, seed=4, device=DEV)
    c["block_table"][0] = 2**30  # a padding row's table may hold anything
    q = queries(5, 8, 4)
    out, lse = call(q, widened(c, 8))
    clean = dict(c, block_table=c["block_table"].clone())
    clean["block_table"][0] = -1
    ref_out, ref_lse, _ = H.attn_decode(q, clean, SCALE)
    assert_out_close(out, ref_out)
    assert (out[0] == 0).all() and (lse.cpu().double() - ref_lse)[1:].abs().max() <= LSE_TOL
    assert K.kda_device_status()[0] == K.KDA_OK


@pytest.mark.parametrize("lens", [[0, 0], [0, 100], [511, 16]])
def test_prefix_that_no_row_of_a_group_holds(lens):
    # behind a row's tokens its table may hold anything, and nobody's prefix is read there
    c = R.prefix_inputs([0, 2, 5], [512, 512], lens + [600, 512, 700], 2, 16, seed=5, device=DEV)
    clean = dict(c, block_table=c["block_table"].clone())
    for b, n in enumerate(lens):
        c["block_table"][b, -(-n // 16):] = 2**30
        clean["block_table"][b, -(-n // 16):] = -1
    q = queries(5, 8, 5)
    want = check(q, clean)
    got = call(q, widened(c, 8))
    assert K.kda_device_status()[0] == K.KDA_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefix_copies_instead_of_shared_pages():
    check(queries(4, 4, 6), inputs([0, 4], [400], [5, 0, 100, 30], 2, 64, 6, copies=True))


@pytest.mark.parametrize("groups", [1, 31, 400, 700])
def test_prefix_many_groups(groups):
    rows = [2 + g % 3 for g in range(groups)]
    first = [0] + torch.tensor(rows).cumsum(0).tolist()
    prefix = [128 * (g % 4) + g % 7 for g in range(groups)]
    check(queries(first[-1], 2, groups), inputs(first, prefix, [i % 5 for i in range(first[-1])], 1, 16, groups, max_pages=40))


@pytest.mark.parametrize("rows,Hq,Hkv,n", [(2, 1, 1, 40000), (3, 16, 2, 20000), (40, 8, 1, 9000)])
def test_prefix_cut_between_many_sms(rows, Hq, Hkv, n):
    check(queries(rows, Hq, n), inputs([0, rows], [n], [3] * rows, Hkv, 64, rows))


@pytest.mark.parametrize("page", [8, 16, 64, 128, 256])
def test_prefix_missing_pages_are_masked(page):
    c = inputs([0, 3, 5], [1100, 600], [50, 0, 300, 5, 40], 2, page, 8)
    for tokens in (0, 130, 256, 520, 521, 1000):  # of the first group, for all of its rows
        c["block_table"][:3, tokens // page] = -1
    c["block_table"][3:, :] = torch.where(torch.arange(c["block_table"].shape[1], device=DEV) * page < 600, -1, c["block_table"][3:])
    check(queries(5, 6, 8), c)


def test_prefix_pages_past_the_cache_are_recorded_and_masked():
    c = inputs([0, 3], [600], [50, 0, 300], 2, 64, 9)
    c["block_table"][:, 2] = c["k_cache"].shape[0]
    check(queries(3, 6, 9), c, status=K.KDA_ERR_DEVICE_INPUT)


@pytest.mark.parametrize("cu", [[0, 3, 2, 6], [-1, 3, 4, 6], [0, 3, 4, 7], [5, 4, 4, 6]])
def test_prefix_bad_groups_share_nothing(cu):
    c = inputs([0, 3, 4, 6], [300, 200, 260], [5] * 6, 2, 16, 10)
    c["cu_groups"] = torch.tensor(cu, dtype=torch.int32, device=DEV)
    check(queries(6, 4, 10), c, status=K.KDA_ERR_DEVICE_INPUT)


@pytest.mark.parametrize("n", [-5, 2**30])
def test_prefix_bad_prefix_lengths_are_clamped(n):
    c = inputs([0, 3], [300], [5] * 3, 2, 16, 11)
    c["prefix_lens"][0] = n
    check(queries(3, 4, 11), c, status=K.KDA_ERR_DEVICE_INPUT)


def test_prefix_bad_sequence_lengths_are_clamped():
    c = inputs([0, 3], [256], [0, 16, 0], 2, 16, 12)
    c = widened(c, 4)
    c["seq_lens"][1] = 2**30  # clamped to the table's tokens, of which only 272 are there
    K.kda_device_status()
    out, _ = call(queries(3, 4, 12), c)
    assert K.kda_device_status() == (K.KDA_ERR_DEVICE_INPUT, 1)
    c["seq_lens"][1] = 272
    assert_out_close(call(queries(3, 4, 12), c)[0], out.double().cpu())


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-3])
def test_prefix_scales(scale):
    check(queries(5, 8, 13), inputs([0, 5], [520], [5, 6, 0, 1, 130], 2, 16, 13), scale=scale)


@pytest.mark.parametrize("rows", [3, 40])
def test_prefix_growing_scores(rows):
    # the maximum grows over the tokens by far more than 2^8, then falls: what was summed is scaled down on the way
    c = inputs([0, rows], [1500], [20] * rows, 1, 16, 14)
    pages = c["block_table"][0, :1500 // 16].long()
    ramp = torch.linspace(0.1, 8.0, 1488, device=DEV)
    ramp[1000:] = 0.5
    k = c["k_cache"]
    k[pages] = (k[pages].float() * ramp.view(-1, 1, 16, 1)).to(torch.bfloat16)
    q = queries(1, 8, 14).expand(rows, 8, 128).contiguous()
    check(q, c, lse_tol=8 * LSE_TOL)


def test_prefix_infinite_and_nan_values_reach_their_channel_only():
    c = inputs([0, 4], [512], [20] * 4, 1, 16, 15)
    page = c["block_table"][0, 5].long()
    c["v_cache"][page, 0, 3, 17] = math.inf
    c["v_cache"][page, 0, 9, 40] = math.nan
    out, lse = call(queries(4, 4, 15), widened(c, 4))
    assert (out[:, :, 17] == math.inf).all() and torch.isnan(out[:, :, 40]).all()
    rest = [i for i in range(128) if i not in (17, 40)]
    assert torch.isfinite(out[:, :, rest]).all() and torch.isfinite(lse).all()


def test_prefix_nan_keys_and_infinite_scores():
    c = inputs([0, 4, 8], [512, 384], [20] * 8, 1, 16, 16)
    c["k_cache"][c["block_table"][0, 5].long(), 0, 3, 17] = math.nan
    out, _ = call(queries(8, 4, 16), widened(c, 4))
    assert torch.isnan(out[:4]).all() and torch.isfinite(out[4:]).all()
    # keys whose score is -inf have no weight
    c = inputs([0, 4], [512], [20] * 4, 1, 16, 17)
    q = queries(4, 4, 17)
    q[..., 0] = 1.0
    c["k_cache"][c["block_table"][0, 5].long(), 0, :, 0] = -math.inf
    out, lse = call(q, widened(c, 4))
    c["block_table"][:, 5] = -1
    ref_out, ref_lse, _ = H.attn_decode(q, c, SCALE)
    assert_out_close(out, ref_out)
    assert (lse.cpu().double() - ref_lse).abs().max() <= LSE_TOL


@pytest.mark.parametrize("groups", [0, 1])
def test_prefix_without_groups_or_of_few_tokens_is_the_plain_call(groups):
    c = inputs([0, 3], [300], [5, 6, 7], 2, 16, 18)
    q = queries(3, 4, 18)
    if groups == 0:
        c["cu_groups"], c["prefix_lens"] = c["cu_groups"][:1], c["prefix_lens"][:0]
        c = widened(c, 4)
    out, lse = call(q, c)
    plain, plain_lse = K.attn_decode(q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], scale=SCALE, want_lse=True)
    assert torch.equal(out, plain) and torch.equal(lse, plain_lse)


def test_prefix_wide_table():
    # so many tiles that a table could hold pass 32-bit products
    c = inputs([0, 3], [300], [5, 600, 7], 2, 64, 19)
    wide = dict(c, block_table=torch.full((3, 1 << 21), -1, dtype=torch.int32, device=DEV))
    wide["block_table"][:, :c["block_table"].shape[1]] = c["block_table"]
    q = queries(3, 8, 19)
    out, lse = check(q, c)
    got, got_lse = call(q, wide)
    assert torch.equal(out, got) and torch.equal(lse, got_lse)


@pytest.mark.parametrize("rows,Hq,Hkv,tokens", [(3, 2, 2, 16384), (3, 2, 2, 16392), (5, 40, 2, 4912), (5, 40, 2, 4920)])
def test_prefix_beside_the_limit_of_few_tokens(rows, Hq, Hkv, tokens):
    # 48 MiB are 98304 tokens of a row's key head and 16 query heads: rows x Hkv x ceil(group / 16) x table's tokens
    c = inputs([0, rows], [700], [3] * rows, Hkv, 8, rows, max_pages=-(-tokens // 8))
    q = queries(rows, Hq, 40)
    out, lse = call(q, c)
    ref_out, ref_lse, _ = H.attn_decode(q, dict(c, block_table=c["block_table"][:, :100].contiguous()), SCALE)
    assert_out_close(out, ref_out)
    assert (lse.cpu().double() - ref_lse).abs().max() <= LSE_TOL


def test_prefix_cache_offsets_pass_32_bits():
    Hkv, page = 4, 128
    pages = 2**31 // (2 * Hkv * page * 128) + 9
    cache = torch.empty(pages, 2, Hkv, page, 128, dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(20)
    cache[-8:] = torch.randn(8, 2, Hkv, page, 128, generator=gen, device=DEV).to(torch.bfloat16)
    i32 = dict(dtype=torch.int32, device=DEV)
    last = list(range(pages - 8, pages))
    table = torch.tensor([last[:5] + [-1], last[:4] + [last[5], last[6]]], **i32)
    small = dict(block_table=torch.where(table < 0, -1, table - (pages - 8)), seq_lens=torch.tensor([600, 650], **i32),
                 k_cache=cache[-8:, 0], v_cache=cache[-8:, 1], cu_groups=torch.tensor([0, 2], **i32), prefix_lens=torch.tensor([512], **i32))
    q = queries(2, 8, 20)
    want = check(q, small)
    got = call(q, widened(dict(small, block_table=table, k_cache=cache[:, 0], v_cache=cache[:, 1]), 8))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_prefix_same_bits_again_on_another_stream_and_in_a_graph():
    narrow = inputs([0, 20, 30], [1500, 700], [7 * i % 90 for i in range(30)], 2, 16, 21)
    c = widened(narrow, 16)
    q = queries(30, 16, 21)
    want = call(q, c)
    ws = K.attn_prefix_decode_workspace(30, 16, 2, c["block_table"].shape[1], 16, 2, DEV)
    ws.random_()
    for _ in range(3):
        got = call(q, c, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, lse = torch.empty_like(q), torch.empty(30, 16, device=DEV)
    args = (q, c["k_cache"], c["v_cache"], c["block_table"], c["seq_lens"], c["cu_groups"], c["prefix_lens"], out, SCALE, ws, lse)
    K.kda_attn_prefix_decode(*args, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_attn_prefix_decode(*args)
    for lens in ([7, 700], [1500, 0]):  # the captured call follows what its tensors hold
        c["prefix_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ref_out, ref_lse, _ = H.attn_decode(q, narrow, SCALE)
        assert_out_close(out, ref_out)
        assert (lse.cpu().double() - ref_lse).abs().max() <= LSE_TOL


def test_prefix_between_other_launches():
    # overlapping launches: lengths, groups and queries come from the launch just before, the output goes to the next
    c = widened(inputs([0, 8], [900], [30] * 8, 2, 16, 22), 8)
    q = queries(8, 8, 22)
    want = call(q, c)[0]
    ws = K.attn_prefix_decode_workspace(8, 8, 2, c["block_table"].shape[1], 16, 1, DEV)
    lens, prefix, groups = (torch.zeros_like(c[n]) for n in ("seq_lens", "prefix_lens", "cu_groups"))
    q2, out = torch.zeros_like(q), torch.empty_like(q)
    for _ in range(20):
        for x in (lens, prefix, groups, q2):
            x.zero_()
        lens.copy_(c["seq_lens"]), prefix.copy_(c["prefix_lens"]), groups.copy_(c["cu_groups"]), q2.copy_(q)
        K.kda_attn_prefix_decode(q2, c["k_cache"], c["v_cache"], c["block_table"], lens, groups, prefix, out, SCALE, ws)
        got = out + 0
        assert torch.equal(got, want)


def test_prefix_on_two_streams_beside_prompts_on_a_third():
    # kernels that all hold tensor memory, in flight together
    a = widened(inputs([0, 20, 30], [1500, 700], [7 * i % 90 for i in range(30)], 2, 16, 23), 16)
    b = widened(inputs([0, 8], [900], [30] * 8, 2, 64, 24), 8)
    qa, qb = queries(30, 16, 23), queries(8, 8, 24)
    want_a, want_b = call(qa, a), call(qb, b)
    gen = torch.Generator().manual_seed(25)
    q, k, v = (torch.randn(700, 4, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(3))
    decay = -torch.rand(700, 4, generator=gen).to(DEV)
    cu = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)

    def prompt(**kw):
        return K.linear_prefill(q, k, v, decay, cu, scale=SCALE, **kw)

    want_c = prompt()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        got.append((call(qa, a, stream=streams[0]), call(qb, b, stream=streams[1]), prompt(stream=streams[2])))
    torch.cuda.synchronize()
    assert K.kda_device_status()[0] == K.KDA_OK
    for x, y, z in got:
        assert all(torch.equal(g, w) for g, w in zip((*x, *y, *z), (*want_a, *want_b, *want_c)))
