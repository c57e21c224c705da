"""Pages handed out on the GPU, and queries and keys normed, rotated and written into them.

Pages, slots and lengths are exact. Tolerances of the rotation: a result is rounded once to BF16 (2^-8 of it at most);
before that x r w has five roundings of 2^-24 and the sum of 128 squares in the norm 128 x 2^-24 / 2 (relative to a
pair's length); sine and cosine are off by 2^-20 (the hardware's 2^-20.9 and the angle's 2^-32 of a turn), and with two products and a sum a pair
(a, b) gives an error of at most (2^-19 + 72 x 2^-24) magnitude |(a, b)| < 2^-17 magnitude |(a, b)|."""
import math

import pytest
import torch

import kda_recurrent_gb300 as K
import serving_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---------------------------------------------------------------- pages


def resize(table, old, new, ring, state, ps, max_tokens, in_place=False, expect_status=K.KDA_OK):
    i32 = dict(dtype=torch.int32, device=DEV)
    B = len(old)
    t = dict(table=torch.tensor(table, **i32).view(B, -1) if B else torch.empty(0, 1, **i32), old=torch.tensor(old, **i32),
             new=torch.tensor(new, **i32), ring=torch.tensor(ring, **i32), state=torch.tensor(state, **i32))
    lens, out_state = (t["old"], t["state"]) if in_place else (torch.full((B,), -9, **i32), torch.full((2,), -9, **i32))
    cu, slots = torch.full((B + 1,), -9, **i32), torch.full((max_tokens,), -9, dtype=torch.int64, device=DEV)
    positions, rows = torch.full((max_tokens,), -9, **i32), torch.full((max_tokens,), -9, **i32)
    K.kda_device_status()
    K.kda_page_resize(t["table"], t["old"], t["new"], t["ring"], t["state"], ps, lens, out_state, cu, slots, positions, rows)
    status = K.kda_device_status()
    assert status[0] == expect_status, status
    if not in_place:
        assert t["old"].tolist() == old and t["state"].tolist() == state
    return [x.tolist() for x in (t["table"], lens, t["ring"], out_state, cu, slots, positions, rows)]


def check_resize(old, new, ps, *, seed=1, spare=5, extra=3, in_place=False, max_pages=None, start=None, drop=0):
    table, ring, state = R.page_inputs(old, new, ps, seed=seed, spare=spare, max_pages=max_pages, start=start)
    state[1] -= drop
    T = sum(max(0, b - a) for a, b in zip(old, new)) + extra
    short = drop > spare
    got = resize(table, old, new, ring, state, ps, T, in_place, K.KDA_ERR_DEVICE_INPUT if short else K.KDA_OK)
    want = R.page_resize(table, old, new, ring, state, ps, T)
    for name, g, w in zip(("table", "lens", "ring", "state", "cu", "slots", "positions", "rows"), got, want):
        assert g == list(w), name
    return got


def lengths(n, lo, hi, seed):
    return torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("old,new", [([0], [1]), ([0], [0]), ([7], [8]), ([8], [9]), ([9], [8]), ([8], [0]), ([100], [3]),
                                     ([0, 0, 0], [0, 17, 0]), ([5, 16, 0, 40], [6, 17, 33, 0]), ([64, 1], [0, 64])])
@pytest.mark.parametrize("ps", [8, 16])
def test_pages_small(old, new, ps):
    check_resize(old, new, ps)


@pytest.mark.parametrize("B", [1, 31, 32, 33, 255, 256, 257, 1023, 1024, 1025, 2500])
def test_pages_row_counts(B):
    old = lengths(B, 0, 60, B)
    check_resize(old, [n + 1 for n in old], 8, seed=B)
    check_resize(old, lengths(B, 0, 60, B + 1), 8, seed=B, in_place=True)


@pytest.mark.parametrize("lens", [[5000], [1, 40000, 3], [9000] * 8, [20] * 1500])
@pytest.mark.parametrize("ps", [8, 64, 1024])
def test_pages_prompts_on_a_cluster(lens, ps):
    check_resize([0] * len(lens), lens, ps, seed=7)
    check_resize(lens, [0] * len(lens), ps, seed=8, in_place=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_given_back_in_many_rounds_by_a_cluster(in_place):
    # rows of both kinds, tokens enough for all of the GPU, more pages given back than one round holds
    old, new = [0, 60000, 33, 300000, 0, 5], [40000, 7, 33, 0, 900, 6]
    check_resize(old, new, 8, seed=9, in_place=in_place)
    old = lengths(1100, 0, 300, 34)  # rows of two rounds, too
    check_resize(old, [n + 100 if i % 2 else n // 3 for i, n in enumerate(old)], 16, seed=34, in_place=in_place)
    check_resize(old, [n + 100 if i % 2 else n // 3 for i, n in enumerate(old)], 16, seed=35, in_place=in_place, drop=700)


@pytest.mark.parametrize("in_place", [False, True])
def test_pages_of_wide_tables_on_a_cluster(in_place):
    # few new tokens, but tables that could give many pages back: one launch of a cluster does everything
    B = 200
    old = lengths(B, 0, 3000, 31)
    new = [n + 1 if i % 3 else n // 2 for i, n in enumerate(old)]
    check_resize(old, new, 8, seed=31, max_pages=400, in_place=in_place)
    check_resize([300000, 0, 300000, 9], [0, 50, 8, 10], 8, seed=32, in_place=in_place)  # three rounds of pages given back
    check_resize([100] * 4200, [101] * 4100 + [99] * 100, 8, seed=33, max_pages=16, in_place=in_place)


@pytest.mark.parametrize("tokens", [512, 513, 1024, 1025, 2048, 2049, 16384, 16385])  # of the maps: one CTA, a cluster, the whole GPU
@pytest.mark.parametrize("rows,max_pages", [(3, None), (3, 700), (300, None), (300, 109), (300, 110), (300, 218), (300, 219)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_beside_the_limits_of_few_tokens(tokens, rows, max_pages, in_place):
    # (300 rows: up to 32768 entries of the tables, up to 65536, more)
    old = lengths(rows, 0, 900, tokens)
    grow = tokens - 7  # (some of the maps stay empty)
    new = [n + grow // rows + (i < grow % rows) if i % 50 != 2 else n // 2 for i, n in enumerate(old)]
    T = sum(max(0, b - a) for a, b in zip(old, new))
    check_resize(old, new, 16, seed=tokens, extra=tokens - T, max_pages=max_pages, in_place=in_place)


@pytest.mark.parametrize("T", [30, 5000, 20000])
def test_pages_maps_at_odd_addresses(T):
    # maps that begin inside a 16-byte word, and are not written together
    i32 = dict(dtype=torch.int32, device=DEV)
    pages = -(-T // 16)
    table, lens, state = torch.full((2, pages), -1, **i32), torch.zeros(2, **i32), torch.tensor([0, pages + 1], **i32)
    ring = torch.arange(pages + 1, **i32).flip(0).contiguous()
    slots = torch.full((T + 9,), -9, dtype=torch.int64, device=DEV)
    positions, rows = (torch.full((T + 9,), -9, **i32) for _ in range(2))
    K.kda_page_resize(table, lens, torch.tensor([T - 3, 3], **i32), ring, state, 16, lens, state, None, slots[1:T + 5],
                      positions[3:T + 7], rows[2:T + 6])
    page = [pages - i for i in range(pages + 1)]
    first = -(-(T - 3) // 16)  # the second row's page
    want = [page[t // 16] * 16 + t % 16 for t in range(T - 3)] + [page[first] * 16 + t for t in range(3)] + [-1] * 4
    assert slots.tolist() == [-9] + want + [-9] * 4
    assert positions.tolist() == [-9] * 3 + list(range(T - 3)) + [0, 1, 2] + [0] * 4 + [-9] * 2
    assert rows.tolist() == [-9] * 2 + [0] * (T - 3) + [1] * 3 + [-1] * 4 + [-9] * 3


def test_pages_new_lens_become_the_lengths():
    i32 = dict(dtype=torch.int32, device=DEV)
    for n in (7, 6000, 30000):  # one CTA, a cluster, two launches
        table, state = torch.full((1, 1900), -1, **i32), torch.tensor([0, 1900], **i32)
        lens, new, after = torch.zeros(1, **i32), torch.tensor([n], **i32), torch.empty(2, **i32)
        slots = torch.empty(n, dtype=torch.int64, device=DEV)
        K.kda_page_resize(table, lens, new, torch.arange(1900, **i32), state, 16, new, after, slots=slots)
        assert new.tolist() == [n] and lens.tolist() == [0] and after.tolist() == [-(-n // 16), 1900 - -(-n // 16)]
        K.kda_page_resize(table, lens, new, torch.arange(1900, **i32), state, 16, torch.empty_like(new), state, slots=slots)
        assert state.tolist() == after.tolist()


def test_pages_ring_wraps():
    for start in (0, 1, 10, 21, 22):
        check_resize([40, 0, 80], [0, 60, 85], 8, seed=3, start=start % 23, spare=0)


@pytest.mark.parametrize("drop", [1, 2, 6, 9, 1000])
def test_pages_too_few_are_refused_in_order(drop):
    old, new = [3, 40, 8, 10, 0, 16], [9, 8, 30, 12, 40, 16]
    spare = 0
    need = sum(max(0, -(-m // 8) - -(-n // 8)) for n, m in zip(old, new))
    check_resize(old, new, 8, seed=4, spare=spare, drop=min(drop, need))


@pytest.mark.parametrize("B", [300, 1500])
def test_pages_too_few_in_a_large_batch(B):
    old, new = lengths(B, 0, 50, 1), lengths(B, 0, 90, 2)
    for drop in (1, 100, 400):
        check_resize(old, new, 8, seed=5, spare=0, drop=drop)


def test_pages_missing_ones_are_not_given_back():
    table, ring, state = R.page_inputs([64, 64, 64], [8, 0, 64], 8, seed=6)
    table[0][3] = table[1][0] = table[1][7] = table[2][1] = -1
    got = resize(table, [64, 64, 64], [8, 0, 64], ring, state, 8, 4)
    assert got == [list(x) for x in R.page_resize(table, [64, 64, 64], [8, 0, 64], ring, state, 8, 4)]
    # a new token on a missing page has no slot
    got = resize([[-1, 5]], [3], [10], [9, 9, 9, 1, 9, 9], [3, 1], 8, 8)
    assert got[5] == [-1] * 5 + [8, 9, -1] and got[0] == [[-1, 1]]


def test_pages_bad_lengths_states_and_pages():
    bad = K.KDA_ERR_DEVICE_INPUT
    got = resize([[0, 1]], [-4], [99], [2, 3, 4, 5], [0, 4], 8, 20, expect_status=bad)  # clamped to [0, 16]
    assert got[1] == [16] and got[0] == [[2, 3]] and got[4] == [0, 16]
    for state in ([4, 1], [-1, 1], [0, 5], [0, -1]):  # an empty ring
        got = resize([[0, 1]], [8], [9], [2, 3, 4, 5], state, 8, 2, expect_status=bad)
        assert got[1] == [8] and got[3] == [0, 0] and got[5] == [-1, -1]
    got = resize([[0, 1]], [8], [9], [7, 3, 4, 5], [0, 1], 8, 2, expect_status=bad)  # a page past the cache
    assert got[0] == [[0, -1]] and got[5] == [-1, -1]
    got = resize([[9, 1]], [4], [5], [0, 1, 2, 3], [0, 1], 8, 2, expect_status=bad)
    assert got[5] == [-1, -1]
    got = resize([[0, 1], [2, 3]], [16, 16], [0, 0], [0, 1, 2, 3], [1, 2], 8, 2, expect_status=bad)  # more than there are
    assert got[3] == [1, 4] and got[2] == [1, 1, 2, 0]


def test_pages_tokens_past_the_maps_are_left_out():
    got = resize([[-1] * 4] * 2, [0, 0], [9, 9], list(range(8)), [0, 8], 8, 12, expect_status=K.KDA_ERR_DEVICE_INPUT)
    assert got[4] == [0, 9, 18] and got[1] == [9, 9] and len(got[5]) == 12 and got[7] == [0] * 9 + [1] * 3


def test_pages_empty_batch_and_optional_maps():
    got = resize([], [], [], [4, 5], [1, 1], 8, 3)
    assert got[3] == [1, 1] and got[4] == [0] and got[5] == [-1] * 3 and got[6] == [0] * 3
    i32 = dict(dtype=torch.int32, device=DEV)
    table, lens, state = torch.full((1, 2), -1, **i32), torch.zeros(1, **i32), torch.tensor([0, 2], **i32)
    K.kda_page_resize(table, lens, torch.tensor([9], **i32), torch.tensor([1, 0], **i32), state, 8, lens, state)
    assert table.tolist() == [[1, 0]] and lens.tolist() == [9] and state.tolist() == [0, 0]


def test_pages_slots_pass_32_bits():
    i32 = dict(dtype=torch.int32, device=DEV)
    F = (1 << 22) + 3
    ring = torch.zeros(F, **i32)
    ring[F - 1] = F - 1
    table, lens, state = torch.full((1, 1), -1, **i32), torch.zeros(1, **i32), torch.tensor([F - 1, 1], **i32)
    cu, slots, positions, rows = K.page_resize(table, lens, torch.tensor([1024], **i32), ring, state, 1024, max_tokens=1024)
    assert slots.tolist() == [(F - 1) * 1024 + i for i in range(1024)] and state.tolist() == [0, 0]


def test_pages_in_a_graph_replayed_step_by_step():
    i32 = dict(dtype=torch.int32, device=DEV)
    old = [3, 16, 0, 30]
    table, ring, state = R.page_inputs(old, [n + 12 for n in old], 8, seed=12)
    t, lens, ring_t, st = (torch.tensor(x, **i32) for x in (table, old, ring, state))
    new = lens + 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        maps = [torch.empty(5, **i32), torch.empty(6, dtype=torch.int64, device=DEV), torch.empty(6, **i32), torch.empty(6, **i32)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            K.kda_page_resize(t, lens, new, ring_t, st, 8, lens, st, *maps)
            new.add_(1)
        for _ in range(12):
            want = R.page_resize(table, old, [n + 1 for n in old], ring, state, 8, 6)
            graph.replay()
            side.synchronize()
            got = [x.tolist() for x in (t, lens, ring_t, st, *maps)]
            assert got == [list(x) for x in want]
            table, old, ring, state = want[:4]


# ---------------------------------------------------------------- norm and rotation


def close(got, ref, inp, weight, inv_freq, eps, magnitude, interleaved):
    """Against FP64 with the bound above: a pair's length from the normed input."""
    x = R.qk_rope(inp, weight, None, None, eps, 1.0, False)
    half = 0 if inv_freq is None else inv_freq.numel()
    size = x.abs()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    pair = magnitude * torch.hypot(x[..., a], x[..., b])
    size[..., a] = size[..., b] = pair
    err = (got.cpu().double() - ref).abs()
    assert (err <= ref.abs() * 2.0 ** -8 * 1.001 + size * 2.0 ** -17).all(), (err / (size + 1e-30)).max()


def rope_check(T, Hq, Hkv, *, rot=128, interleaved=False, norm="bf16", ps=16, packed=False, cache=True, far=4096, magnitude=1.0,
               seed=0, weights=(True, True), k_out=False, eps=1e-6):
    gen = torch.Generator().manual_seed(seed + T)
    x = torch.randn(T, Hq + 2 * Hkv, 128, generator=gen).to(torch.bfloat16).to(DEV)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    if not packed:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    pos = torch.randint(0, far, (T,), generator=gen).to(torch.int32).to(DEV)
    f = K.rope_frequencies(rot, device=DEV)[0]
    kind = {"bf16": torch.bfloat16, "f32": torch.float32}.get(norm)
    wq, wk = ((1 + 0.2 * torch.randn(128, generator=gen)).to(kind).to(DEV) if kind and on else None for on in weights)
    args = dict(eps=eps, q_weight=wq, k_weight=wk, magnitude=magnitude, interleaved=interleaved)
    q_ref = R.qk_rope(q, wq, pos, f, eps, magnitude, interleaved)
    k_ref = R.qk_rope(k, wk, pos, f, eps, magnitude, interleaved)
    q_out = torch.full((T, Hq, 128), math.nan, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, Hkv, 128), math.nan, dtype=torch.bfloat16, device=DEV) if k_out or not cache else None
    kept = x.clone()
    if cache:
        pages = -(-T // ps) + 2
        kv = torch.full((pages, 2, Hkv, ps, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        slots = torch.randperm(pages * ps, generator=gen)[:T].to(DEV)
        slots[::5] = -1  # padding
        args.update(v=v, k_cache=kv[:, 0], v_cache=kv[:, 1], slots=slots)
    K.kda_qk_norm_rope(q, k, pos, f if rot else None, q_out, ko, **args)
    close(q_out, q_ref, q, wq, f, eps, magnitude, interleaved)
    if ko is not None:
        close(ko, k_ref, k, wk, f, eps, magnitude, interleaved)
    assert torch.equal(x, kept)
    if cache:
        on = (slots >= 0).cpu()
        page, at = slots[on.to(DEV)] // ps, slots[on.to(DEV)] % ps
        assert torch.equal(kv[page, 1, :, at], v[on.to(DEV)])
        close(kv[page, 0, :, at], k_ref[on], k[on.to(DEV)], wk, f, eps, magnitude, interleaved)
        rest = torch.ones(pages, ps, dtype=torch.bool, device=DEV)
        rest[page, at] = False
        assert (kv.permute(0, 3, 1, 2, 4)[rest] == 7.0).all()
    assert K.kda_device_status()[0] == K.KDA_OK
    return q_out


@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 80, 96, 112, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", ["none", "bf16", "f32"])
def test_rope_parts_of_the_head(rot, interleaved, norm):
    rope_check(9, 6, 2, rot=rot, interleaved=interleaved, norm=norm, seed=rot)


@pytest.mark.parametrize("T", [1, 2, 3, 31, 32, 33, 500, 4567])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (3, 1), (5, 5), (64, 8)])
def test_rope_tokens_and_heads(T, Hq, Hkv):
    rope_check(T, Hq, Hkv, packed=T % 2 == 1, ps=8 << (T % 4), seed=Hq)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_far_positions_and_scale(interleaved):
    # in 32 bits the angle of a position near 2^31 would be off by more than a turn
    rope_check(64, 4, 2, far=2**31 - 1, magnitude=1.25, interleaved=interleaved, norm="f32")


def test_rope_negative_positions_turn_back():
    gen = torch.Generator().manual_seed(3)
    q, k = (torch.randn(5, 2, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    f, _ = K.rope_frequencies(128, device=DEV)
    pos = torch.tensor([-1, -77, -100000, 0, -2**31], dtype=torch.int32, device=DEV)
    out, k_out = K.qk_norm_rope(q, k, pos, f)
    close(out, R.qk_rope(q, None, pos, f, 0, 1.0, False), q, None, f, 0, 1.0, False)
    close(k_out, R.qk_rope(k, None, pos, f, 0, 1.0, False), k, None, f, 0, 1.0, False)
    assert torch.equal(out[3], q[3])  # position 0


@pytest.mark.parametrize("weights", [(True, False), (False, True)])
def test_rope_norm_of_one_of_them(weights):
    rope_check(7, 4, 2, weights=weights, cache=False)
    rope_check(7, 4, 2, weights=weights, k_out=True)


def test_rope_in_place_and_strided_outputs():
    gen = torch.Generator().manual_seed(5)
    x = torch.randn(33, 12, 128, generator=gen).to(torch.bfloat16).to(DEV)
    q, k, v = x[:, :8], x[:, 8:10], x[:, 10:]
    pos = torch.arange(33, dtype=torch.int32, device=DEV) * 1000
    f, _ = K.rope_frequencies(128, device=DEV)
    w = torch.ones(128, device=DEV)
    want_q, want_k = K.qk_norm_rope(q, k, pos, f, q_weight=w, k_weight=w)
    kept = v.clone()
    K.kda_qk_norm_rope(q, k, pos, f, q, k, q_weight=w, k_weight=w)
    assert torch.equal(q, want_q) and torch.equal(k, want_k) and torch.equal(v, kept)


def test_rope_zeros_infinities_and_nan_stay_where_they_are():
    gen = torch.Generator().manual_seed(6)
    q, k = (torch.randn(4, 2, 128, generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2))
    q[0, 0] = 0
    q[1, 1, 100] = math.inf  # a channel that does not turn
    q[2, 0, 5] = math.nan
    pos = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=DEV)
    f, _ = K.rope_frequencies(64, device=DEV)
    out, _ = K.qk_norm_rope(q, k, pos, f)
    bad = ~torch.isfinite(out)
    assert bad.nonzero().tolist() == [[1, 1, 100], [2, 0, 5], [2, 0, 37]] and out[1, 1, 100] == math.inf
    out, _ = K.qk_norm_rope(q, k, pos, f, q_weight=torch.ones(128, device=DEV), k_weight=torch.ones(128, device=DEV))
    assert (out[0, 0] == 0).all() and torch.isfinite(out[[0, 3]]).all() and torch.isfinite(out[1, 0]).all() and torch.isfinite(out[2, 1]).all()


def test_rope_slots_past_the_cache_are_recorded():
    q, k, v = (torch.ones(3, 1, 128, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    cache = torch.zeros(2, 2, 1, 8, 128, dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([3, 16, -5], device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    K.kda_device_status()
    K.qk_norm_rope(q, k, pos, None, v=v, k_cache=cache[:, 0], v_cache=cache[:, 1], slots=slots)
    assert K.kda_device_status() == (K.KDA_ERR_DEVICE_INPUT, 1)
    assert cache.sum().item() == 2 * 128 and (cache[0, :, 0, 3] == 1).all()


@pytest.mark.parametrize("T", [5, 700])
def test_rope_on_another_stream_and_in_a_graph(T):
    gen = torch.Generator().manual_seed(T)
    q, k, v = (torch.randn(T, h, 128, generator=gen).to(torch.bfloat16).to(DEV) for h in (6, 2, 2))
    positions = torch.randint(0, 9000, (T,), generator=gen).to(torch.int32).to(DEV)
    slots = torch.randperm(T + 40, generator=gen)[:T].to(DEV)
    inv_freq, magnitude = K.rope_frequencies(96, factor=4.0, original_length=2048, device=DEV)
    weight = torch.randn(128, generator=gen).to(DEV)

    def caches():
        return [torch.zeros(-(-(T + 40) // 16), 2, 16, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]

    def run(kc, vc, **kw):
        return K.qk_norm_rope(q, k, positions, inv_freq, magnitude=magnitude, q_weight=weight, k_weight=weight, v=v, k_cache=kc,
                              v_cache=vc, slots=slots, **kw)

    want = caches()
    want.append(run(*want))
    got = caches()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got.append(run(*got, stream=side))
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    got = caches()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got.append(run(*got))
    positions2, slots2 = positions.flip(0).contiguous(), slots.flip(0).contiguous()
    q2, k2, v2 = (x.flip(0).contiguous() for x in (q, k, v))
    for x, y in ((positions, positions2), (slots, slots2), (q, q2), (k, k2), (v, v2)):  # other tokens in the same tensors
        x.copy_(y)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2].flip(0))


def test_rope_cache_offsets_pass_32_bits():
    ps, H = 1024, 8
    pages = 2**31 // (ps * H * 128) + 2
    cache = torch.empty(pages, 2, H, ps, 128, dtype=torch.bfloat16, device=DEV)
    q, k, v = (torch.randn(2, H, 128, device=DEV).to(torch.bfloat16) for _ in range(3))
    slots = torch.tensor([pages * ps - 1, 5], device=DEV)
    K.qk_norm_rope(q, k, torch.zeros(2, dtype=torch.int32, device=DEV), None, v=v, k_cache=cache[:, 0], v_cache=cache[:, 1], slots=slots)
    assert torch.equal(cache[-1, 0, :, -1], k[0]) and torch.equal(cache[-1, 1, :, -1], v[0])
    assert torch.equal(cache[0, 0, :, 5], k[1]) and torch.equal(cache[0, 1, :, 5], v[1])


def test_rope_frequencies():
    f, m = K.rope_frequencies(128, base=5e5, device="cpu")
    assert m == 1.0 and f[0] == 1.0 and torch.equal(f, (5e5 ** (-torch.arange(0, 128, 2).double() / 128)).float())
    f, m = K.rope_frequencies(64, factor=4.0, device="cpu")
    assert m == 1.0 and f[0] == 0.25
    g, m = K.rope_frequencies(64, factor=4.0, original_length=8192, device="cpu")
    assert g[0] == 1.0 and g[-1] == f[-1] and m == 1 + math.log(4.0) / 10
    with pytest.raises(ValueError):
        K.rope_frequencies(24)


def test_pages_then_rope_then_attention_step():
    """One step as they are used together: pages and slots for each row's new token, its key and value into them."""
    i32 = dict(dtype=torch.int32, device=DEV)
    old, ps, Hq, Hkv = [15, 0, 16, 40], 16, 4, 2
    table, ring, state = R.page_inputs(old, [n + 1 for n in old], ps, seed=20)
    t, lens, ring_t, st = (torch.tensor(x, **i32) for x in (table, old, ring, state))
    gen = torch.Generator().manual_seed(21)
    cache = torch.randn(len(ring), 2, Hkv, ps, 128, generator=gen).to(torch.bfloat16).to(DEV)
    q, k, v = (torch.randn(4, h, 128, generator=gen).to(torch.bfloat16).to(DEV) for h in (Hq, Hkv, Hkv))
    _, slots, positions, _ = K.page_resize(t, lens, lens + 1, ring_t, st, ps, max_tokens=4)
    f, _ = K.rope_frequencies(128, device=DEV)
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    qo = K.qk_norm_rope(q, k, positions, f, q_weight=w, k_weight=w, v=v, k_cache=cache[:, 0], v_cache=cache[:, 1], slots=slots)
    out = K.attn_decode(qo, cache[:, 0], cache[:, 1], t, lens, scale=128 ** -0.5)
    assert lens.tolist() == [n + 1 for n in old] and positions.tolist() == old
    for b, n in enumerate(old):
        page = t[b, n // ps].long()
        assert torch.equal(cache[page, 1, :, n % ps], v[b])
    assert torch.equal(out[1], v[1].repeat_interleave(Hq // Hkv, 0))  # the only token is its value
