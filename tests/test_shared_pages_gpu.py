"""Pages handed out and given back for rows that share pages with others: exact, against lists."""
import pytest
import torch

import kda_recurrent_gb300 as K
import serving_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = dict(dtype=torch.int32, device=DEV)


def reference(table, old, new, shared, ring, state, ps, max_tokens):
    """As R.page_resize, but that a row's first shared[b] pages stay where they are."""
    given = [list(r) for r in table]
    for b, n in enumerate(shared):
        given[b][:n] = [-1] * n  # (a missing page is not given back)
    out = R.page_resize(given, old, new, ring, state, ps, max_tokens)
    plain = R.page_resize(table, old, new, ring, state, ps, max_tokens)
    return (plain[0], out[1], out[2], out[3], *plain[4:])


def check(old, new, shared, ps, *, seed=1, max_pages=None, in_place=False, drop=0, extra=3, status=K.KDA_OK, given=None):
    table, ring, state = R.page_inputs(old, new, ps, seed=seed, spare=5, max_pages=max_pages)
    state[1] -= drop
    T = sum(max(0, b - a) for a, b in zip(old, new)) + extra
    want = reference(table, old, new, given or shared, ring, state, ps, T)
    t, lens, after, ring_t, st, sh = (torch.tensor(x, **I32) for x in (table, old, new, ring, state, shared))
    out_lens, out_state = (lens, st) if in_place else (torch.full_like(lens, -9), torch.full_like(st, -9))
    cu, slots = torch.full((len(old) + 1,), -9, **I32), torch.full((T,), -9, dtype=torch.int64, device=DEV)
    positions, rows = torch.full((T,), -9, **I32), torch.full((T,), -9, **I32)
    K.kda_device_status()
    K.kda_page_resize(t, lens, after, ring_t, st, ps, out_lens, out_state, cu, slots, positions, rows, shared_pages=sh)
    assert K.kda_device_status()[0] == status
    got = [x.tolist() for x in (t, out_lens, ring_t, out_state, cu, slots, positions, rows)]
    for name, g, w in zip(("table", "lens", "ring", "state", "cu", "slots", "positions", "rows"), got, want):
        assert g == list(w), name
    assert sh.tolist() == shared


def ints(n, lo, hi, seed):
    return torch.randint(lo, hi + 1, (n,), generator=torch.Generator().manual_seed(seed)).tolist()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shared", [0, 1, 3, 4, 5, 8])
def test_one_row_shrinks(shared, in_place):
    for new in (0, 1, 23, 24, 25, 31, 32, 33, 40):
        check([33], [new], [shared], 8, max_pages=8, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("rows,hi,max_pages,grow", [(7, 300, None, 5), (300, 900, None, 3), (300, 900, 300, 40), (1100, 300, None, 20),
                                                    (1100, 300, None, 70), (2500, 60, None, 1)])
def test_many_rows(rows, hi, max_pages, grow, in_place):
    # one CTA, one cluster, the whole GPU, two launches: rows that grow, shrink to anything and end, sharing any number
    old = ints(rows, 0, hi, rows)
    new = [n + grow if i % 3 == 0 else 0 if i % 7 == 1 else n // (1 + i % 4) for i, n in enumerate(old)]
    shared = [min(x, max_pages or 2) for x in ints(rows, 0, hi // 8, rows + 1)]
    wide = max_pages or max(-(-max(a, b) // 8) for a, b in zip(old, new))
    shared = [min(x, wide) for x in shared]
    check(old, new, shared, 8, seed=rows, max_pages=wide, in_place=in_place)
    check(old, new, [0] * rows, 8, seed=rows, max_pages=wide, in_place=in_place)


def test_numbers_out_of_range_are_clamped_and_recorded():
    bad = K.KDA_ERR_DEVICE_INPUT
    check([33, 33], [0, 0], [-1, 2], 8, max_pages=6, status=bad, given=[0, 2])
    check([33, 33], [0, 0], [1, 7], 8, max_pages=6, status=bad, given=[1, 6])
    check([33, 33], [0, 0], [1, 6], 8, max_pages=6)


def test_too_few_pages_with_shared_ones():
    check([40, 8, 64, 3], [41, 9, 0, 30], [5, 1, 4, 0], 8, drop=8, status=K.KDA_ERR_DEVICE_INPUT)


def test_numbers_in_the_tensor_of_the_lengths():
    # out_lens may be any of the inputs of a row each, this one too
    old, new = ints(300, 0, 900, 5), ints(300, 0, 900, 6)
    table, ring, state = R.page_inputs(old, new, 8, seed=5)
    shared = [min(x, len(table[0])) for x in ints(300, 0, 20, 7)]
    want = reference(table, old, new, shared, ring, state, 8, 0)
    t, lens, after, ring_t, st, sh = (torch.tensor(x, **I32) for x in (table, old, new, ring, state, shared))
    K.kda_page_resize(t, lens, after, ring_t, st, 8, sh, torch.empty_like(st), shared_pages=sh)
    assert sh.tolist() == want[1] and ring_t.tolist() == want[2] and t.tolist() == want[0]


def test_requests_behind_a_prefix_end_like_any_other():
    """Eight rows read 40 tokens' pages of row 0: they end at length 0 in any order, while the others go on, without a page
    of the prefix in the ring before its owner ends; what is handed out meanwhile is nobody else's."""
    ps, B, P, pages = 8, 8, 12, 80
    gen = torch.Generator().manual_seed(3)
    table, lens, state = torch.full((B, P), -1, **I32), torch.zeros(B, **I32), torch.tensor([0, pages], **I32)
    ring = torch.randperm(pages, generator=gen).to(torch.int32).to(DEV)
    new = torch.zeros(B, **I32)
    new[0] = 40
    K.page_resize(table, lens, new, ring, state, ps, max_tokens=40)
    table[1:, :5] = table[0, :5]
    lens[1:] = 40
    prefix = set(table[0, :5].tolist())
    shared = torch.tensor([0] + [5] * (B - 1), **I32)

    def resize(to):
        K.page_resize(table, lens, torch.tensor(to, **I32), ring, state, ps, max_tokens=400, shared_pages=shared)
        first, count = state.tolist()
        free = [ring.tolist()[(first + i) % pages] for i in range(count)]
        held = [table[b, :-(-n // ps)].tolist() for b, n in enumerate(lens.tolist())]
        mine = [x for b, row in enumerate(held) for x in row[int(shared[b]):]]
        owned = set(mine) | prefix
        assert len(set(free)) == len(free) and not owned & set(free)
        assert len(mine) == len(set(mine)) and len(owned) + len(free) == pages
        return free

    resize([40] + [60 + b for b in range(1, B)])
    alive = {b: 60 + b for b in range(1, B)}
    for b in (3, 1, 7, 2, 6, 5, 4):  # all but the owner end, the others take tokens
        del alive[b]
        for x in alive:
            alive[x] += 5
        resize([40] + [alive.get(i, 0) for i in range(1, B)])
        table[b] = -1
        shared[b] = 0  # the row is free for a request of its own
    prefix = set()
    assert sorted(resize([0] * B)) == list(range(pages)) and state.tolist()[1] == pages
    assert K.kda_device_status()[0] == K.KDA_OK


def test_in_a_graph():
    old, ps = [30, 30, 16, 40], 8
    table, ring, state = R.page_inputs(old, [n + 12 for n in old], ps, seed=12)
    t, lens, ring_t, st, shared = (torch.tensor(x, **I32) for x in (table, old, ring, state, [2, 2, 0, 1]))
    new = torch.zeros(4, **I32)
    slots = torch.empty(16, dtype=torch.int64, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        K.kda_page_resize(t, lens, new, ring_t, st, ps, lens, st, slots=slots, shared_pages=shared)
    for to, sh in (([31, 33, 18, 41], [2, 2, 0, 1]), ([0, 34, 2, 41], [2, 2, 0, 1]), ([0, 0, 0, 0], [0, 2, 0, 5])):
        new.copy_(torch.tensor(to, dtype=torch.int32))
        shared.copy_(torch.tensor(sh, dtype=torch.int32))
        want = reference(table, old, to, sh, ring, state, ps, 16)
        graph.replay()
        torch.cuda.synchronize()
        assert [x.tolist() for x in (t, lens, ring_t, st, slots)] == [list(want[i]) for i in (0, 1, 2, 3, 5)]
        table, old, ring, state = want[:4]
