"""Linear attention with a decay for each head, prompt and single-token form, against the token
recurrence in FP64.

Tolerances: the output is rounded once to BF16 (relative error <= 2^-9 an element), after products in
which the decayed scores and the state are each rounded to BF16 (<= 2^-9 of their part): relL2 <=
3 x 2^-9 = 5.9e-3, under the 1e-2 that this library's outputs are held to. The FP32 state keeps its
decayed keys to 16 bits (2^-17 = 7.6e-6) and sums in FP32: relL2 <= 2e-5. BF16 pool states are
rounded once: 2^-9."""
import math

import pytest
import torch

import hybrid_reference as R
import kda_recurrent_gb300 as K
from helpers import assert_out_close, assert_state_close, rel_l2

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)
STATE_TOL = 2e-5


def run(inp, workspace=False, want_final=True):
    N, (T, H, _) = inp["cu_seqlens"].shape[0] - 1, inp["q"].shape
    ws = K.linear_prefill_workspace(N, T, H, DEV) if workspace else None
    return K.linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], inp["init_state"],
                            scale=SCALE, want_final=want_final, workspace=ws)


def check(inp, workspace=False):
    out, fin = run(inp, workspace)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    assert_out_close(out, ref_out)
    assert_state_close(fin, ref_fin, tol=STATE_TOL)
    assert K.kda_device_status()[0] == K.KDA_OK
    return out, fin


@pytest.mark.parametrize("T", [1, 2, 15, 16, 31, 63, 64, 65, 127, 128, 129, 200, 256, 257, 511])
@pytest.mark.parametrize("decay,init", [("head", True), ("token", False)])
def test_prefill_lengths(T, decay, init):
    check(R.linear_inputs([T], 2, seed=T, decay=decay, init=init, device=DEV))


@pytest.mark.parametrize("lens,H", [([64, 45], 1), ([1, 0, 130, 128, 7], 3), ([300, 17, 256, 511, 1], 5),
                                    ([0, 0, 5], 2), ([129] * 7, 32)])
@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_varlen(lens, H, decay, workspace):
    check(R.linear_inputs(lens, H, seed=11, decay=decay, device=DEV), workspace)


@pytest.mark.parametrize("lens,H", [([1500], 1), ([2048], 2), ([700, 64, 1300], 3), ([1025, 0, 2000], 2)])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_prefill_windows(lens, H, decay):
    check(R.linear_inputs(lens, H, seed=12, decay=decay, device=DEV), workspace=True)


def test_prefill_workspace_is_used_for_few_chains():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert K.linear_prefill_workspace(1, 2048, 2, DEV) is not None
    assert K.linear_prefill_workspace(1, 2048, sms, DEV) is None
    assert K.linear_prefill_workspace(1, 256, 2, DEV) is None  # too short to gain


@pytest.mark.parametrize("final", [True, False])
def test_prefill_many_short_chains(final):
    # more items than SMs: every CTA takes over several, full and partial chunks in turn
    lens = [(37 * i) % 300 for i in range(60)]
    inp = R.linear_inputs(lens, 6, seed=22, decay="token", device=DEV)
    out, fin = run(inp, want_final=final)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    assert_out_close(out, ref_out)
    if final:
        assert_state_close(fin, ref_fin, tol=STATE_TOL)
    assert K.kda_device_status()[0] == K.KDA_OK


def test_prefill_more_sequences_than_are_ranked():
    lens = [1 + (13 * i) % 40 for i in range(300)]
    check(R.linear_inputs(lens, 1, seed=23, device=DEV))


def test_prefill_windowed_last_wave():
    # more chains than SMs, and a last wave of a few: whole chains and windows in one call
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H = sms + 3
    inp = R.linear_inputs([600], H, seed=13, decay="token", device=DEV)
    a, fa = run(inp)
    b, fb = run(inp, workspace=True)
    assert rel_l2(b, a) <= 1e-2 and rel_l2(fb, fa) <= STATE_TOL
    heads = [0, 1, sms - 1, sms, sms + 2]
    sub = {n: x for n, x in inp.items()}
    for n in ("q", "k", "v", "log_decay"):
        sub[n] = inp[n][:, heads].contiguous()
    sub["init_state"] = inp["init_state"][:, heads].contiguous()
    ref_out, ref_fin = R.linear_prefill(sub, SCALE)
    for out, fin in ((a, fa), (b, fb)):
        assert_out_close(out[:, heads], ref_out)
        assert_state_close(fin[:, heads], ref_fin, tol=STATE_TOL)


@pytest.mark.parametrize("workspace", [False, True])
@pytest.mark.parametrize("kind", ["none", "fast", "clear", "mixed"])
def test_prefill_extreme_decays(kind, workspace):
    T, H = 900, 2
    inp = R.linear_inputs([T], H, seed=14, decay="token", device=DEV)
    g = inp["log_decay"]
    if kind == "none":
        g.zero_()  # nothing is forgotten
    elif kind == "fast":
        g.fill_(-60.0)  # e^g at the edge of FP32 within two tokens
    elif kind == "clear":
        g[5::37] = -math.inf  # the state is cleared
    else:
        g[::3] = -200.0
        g[1::3] = 0.0
    check(inp, workspace)


def test_prefill_per_head_equals_per_token():
    inp = R.linear_inputs([333, 70], 4, seed=15, decay="head", device=DEV)
    a, fa = run(inp)
    inp["log_decay"] = inp["log_decay"].expand(403, 4).contiguous()
    b, fb = run(inp)
    assert rel_l2(b, a) <= 1e-2 and rel_l2(fb, fa) <= STATE_TOL


@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_split_and_carry(workspace):
    inp = R.linear_inputs([1000], 2, seed=16, decay="token", device=DEV)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    state, outs = inp["init_state"], []
    for a, b in ((0, 1), (1, 390), (390, 1000)):
        part = {n: inp[n][a:b].contiguous() for n in ("q", "k", "v", "log_decay")}
        part["cu_seqlens"] = torch.tensor([0, b - a], dtype=torch.int32, device=DEV)
        part["init_state"] = state
        out, state = run(part, workspace)
        outs.append(out)
    assert_out_close(torch.cat(outs), ref_out)
    assert_state_close(state, ref_fin, tol=3 * STATE_TOL)


@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_state_in_place_and_without_final(workspace):
    inp = R.linear_inputs([640, 0, 33], 2, seed=17, device=DEV)
    out, fin = run(inp, workspace)
    alone, none = run(inp, workspace, want_final=False)
    assert none is None and torch.equal(alone, out)
    state = inp["init_state"].clone()
    ws = K.linear_prefill_workspace(3, 673, 2, DEV) if workspace else None
    K.kda_linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], state, out, state, SCALE,
                         workspace=ws)
    assert torch.equal(state, fin)
    assert torch.equal(fin[1], inp["init_state"][1])  # the empty sequence


@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_sequences_do_not_touch(workspace):
    # NaN and infinity in one sequence stay there; the others' bits do not change
    lens = [70, 129, 200, 640]
    inp = R.linear_inputs(lens, 2, seed=18, device=DEV)
    out, fin = run(inp, workspace)
    bad = {n: None if x is None else x.clone() for n, x in inp.items()}
    a, b = 70, 199
    bad["q"][a:b], bad["k"][a:b], bad["v"][a:b] = math.nan, math.inf, math.nan
    out2, fin2 = run(bad, workspace)
    for lo, hi, n in ((0, 70, 0), (199, 399, 2), (399, 1039, 3)):
        assert torch.equal(out2[lo:hi], out[lo:hi]) and torch.equal(fin2[n], fin[n])


@pytest.mark.parametrize("lens,H,at,final", [([300], 2, 200, True), ([300], 2, 290, False), ([128], 1, 5, False),
                                             ([70, 129, 60], 3, 100, True), ([40] * 200, 2, 50, False),
                                             ([1500], 2, 700, True), ([2000], 1, 1990, False)])
@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_values_that_are_not_finite_stay_in_their_channel(lens, H, at, final, workspace):
    # ... and begin at their token: earlier outputs, other channels, sequences and heads do not see them
    inp = R.linear_inputs(lens, H, seed=29, decay="head", device=DEV)
    inp["log_decay"].fill_(-0.01)
    out, fin = run(inp, workspace, want_final=final)
    cu = inp["cu_seqlens"].tolist()
    n = max(i for i, a in enumerate(cu[:-1]) if a <= at)
    last = min(at + 20, cu[n + 1] - 1)
    bad = {m: None if x is None else x.clone() for m, x in inp.items()}
    places = ((at, 3, math.inf), (at, 70, -math.inf), (last, 127, math.nan), (at, 9, math.inf), (last, 9, -math.inf),
              (last, 71, math.inf))
    for t, c, x in places:
        bad["v"][t, H - 1, c] = x
    out2, fin2 = run(bad, workspace, want_final=final)
    odd = sorted({c for _, c, _ in places})
    one = {m: None if x is None else x[:, H - 1:].contiguous() if m in "qkv" else x[H - 1:] if m == "log_decay" else
           x[:, H - 1:] if m == "init_state" else x for m, x in bad.items()}
    ref_out, ref_fin = R.linear_prefill(one, SCALE)
    a, b = cu[n], cu[n + 1]
    got, ref = out2[a:b, H - 1][:, odd].cpu().double(), ref_out[a:b, 0][:, odd]
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)) and not torch.isfinite(ref[-1]).any()
    assert_out_close(got[torch.isfinite(ref)], ref[torch.isfinite(ref)])
    same = torch.ones(out.shape, dtype=torch.bool, device=DEV)
    same[a:b, H - 1, odd] = False
    assert torch.equal(out2[same], out[same])
    if final:
        assert torch.equal(fin2[n, H - 1][:, odd].cpu().double().nan_to_num(nan=7.0), ref_fin[n, 0][:, odd].nan_to_num(nan=7.0))
        fin2[n, H - 1][:, odd] = fin[n, H - 1][:, odd]
        assert torch.equal(fin2, fin)


@pytest.mark.parametrize("name,x", [("q", math.nan), ("q", math.inf), ("k", math.nan), ("k", -math.inf), ("log_decay", math.nan)])
@pytest.mark.parametrize("lens,at", [([300], 200), ([1500, 40], 700)])
@pytest.mark.parametrize("workspace", [False, True])
def test_prefill_nothing_that_is_not_finite_reaches_an_earlier_token(name, x, lens, at, workspace):
    inp = R.linear_inputs(lens, 2, seed=36, decay="token", device=DEV)
    out, fin = run(inp, workspace)
    inp[name] = inp[name].clone()
    inp[name][at, 1] = x
    out2, fin2 = run(inp, workspace)
    assert not torch.isfinite(out2[at, 1]).any()
    same = torch.ones(out.shape, dtype=torch.bool, device=DEV)
    same[at:lens[0] if name != "q" else at + 1, 1] = False
    assert torch.equal(out2[same], out[same])
    assert torch.equal(fin2[1:], fin[1:]) and torch.equal(fin2[0, 0], fin[0, 0])
    assert torch.equal(fin2[0, 1], fin[0, 1]) if name == "q" else not torch.isfinite(fin2[0, 1]).any()


def test_prefill_every_chunk_ends_in_nan():
    # every output but each chunk's last is formed again
    inp = R.linear_inputs([1280], 2, seed=37, device=DEV)
    clean, _ = run(inp)
    inp["v"][127::128] = math.nan
    out, fin = run(inp)
    assert_out_close(out[:127], clean[:127])
    assert torch.isnan(out[127:]).all() and torch.isnan(fin).all()


def test_prefill_all_values_nan():
    inp = R.linear_inputs([20, 400], 2, seed=30, device=DEV)
    inp["v"].fill_(math.nan)
    out, fin = run(inp)
    assert torch.isnan(out).all() and torch.isnan(fin).all()


def test_prefill_windows_in_place():
    # the initial state lies where the end state goes, which other windows' launches read before
    inp = R.linear_inputs([1400, 0, 1700], 2, seed=24, decay="token", device=DEV)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    state, out = inp["init_state"].clone(), torch.empty_like(inp["q"])
    ws = K.linear_prefill_workspace(3, 3100, 2, DEV)
    assert ws is not None
    K.kda_linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], state, out, state, SCALE,
                         workspace=ws)
    assert_out_close(out, ref_out)
    assert_state_close(state, ref_fin, tol=STATE_TOL)
    assert torch.equal(state[1], inp["init_state"][1])


def test_prefill_windows_do_not_touch():
    # windows end at multiples of a chunk inside a sequence; another sequence's NaN begins right behind it
    lens = [1300, 129, 1601]
    inp = R.linear_inputs(lens, 2, seed=25, device=DEV)
    assert K.linear_prefill_workspace(3, sum(lens), 2, DEV) is not None
    out, fin = run(inp, True)
    bad = {n: None if x is None else x.clone() for n, x in inp.items()}
    bad["q"][1300:1429], bad["k"][1300:1429], bad["v"][1300:1429] = math.nan, math.inf, math.nan
    out2, fin2 = run(bad, True)
    for lo, hi, n in ((0, 1300, 0), (1429, 3030, 2)):
        assert torch.equal(out2[lo:hi], out[lo:hi]) and torch.equal(fin2[n], fin[n])


def test_prefill_long_windowed_last_wave():
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H = sms + 2
    inp = R.linear_inputs([1450], H, seed=26, decay="token", device=DEV)
    assert K.linear_prefill_workspace(1, 1450, H, DEV) is not None
    out, fin = run(inp, workspace=True)
    heads = [0, sms - 1, sms, sms + 1]
    sub = {n: x for n, x in inp.items()}
    for n in ("q", "k", "v", "log_decay"):
        sub[n] = inp[n][:, heads].contiguous()
    sub["init_state"] = inp["init_state"][:, heads].contiguous()
    ref_out, ref_fin = R.linear_prefill(sub, SCALE)
    assert_out_close(out[:, heads], ref_out)
    assert_state_close(fin[:, heads], ref_fin, tol=STATE_TOL)


@pytest.mark.parametrize("lens,H", [([8192] * 5 + [300] * 15, 8), ([16384] + [2048] * 4, 32), ([1450], 154)])
def test_prefill_windowed_last_wave_in_place(lens, H):
    # A CTA takes its next item when it begins one: behind long chains a window's beginning may come long after
    # the end of its chain's last window, which stores the end state where the initial one lay.
    assert len(lens) * H - torch.cuda.get_device_properties(0).multi_processor_count in range(1, 51)
    inp = R.linear_inputs(lens, H, seed=27, decay="head", device=DEV)
    out, fin = run(inp, workspace=True)
    ws = K.linear_prefill_workspace(len(lens), sum(lens), H, DEV)
    assert ws is not None
    for _ in range(4):
        state, again = inp["init_state"].clone(), torch.empty_like(out)
        K.kda_linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], state, again, state,
                             SCALE, workspace=ws)
        assert torch.equal(again, out) and torch.equal(state, fin)


def test_prefill_windowed_calls_without_waits_equal_calls_with_waits():
    """Launches overlap the work before them: each call here reads what the one before it writes."""
    lens, H = [1400, 0, 1700], 2
    inp = R.linear_inputs(lens, H, seed=28, decay="head", device=DEV)
    ws = K.linear_prefill_workspace(len(lens), sum(lens), H, DEV)
    assert ws is not None

    def chain(wait):
        a, b, state = inp["v"].clone(), torch.empty_like(inp["v"]), inp["init_state"].clone()
        for step in range(20):
            K.kda_linear_prefill(inp["q"], inp["k"], a, inp["log_decay"], inp["cu_seqlens"], state, b, state, 1.0,
                                 workspace=ws)
            if wait:
                torch.cuda.synchronize()
            a, b = b, a
        return a, state
    for x, y in zip(chain(True), chain(False)):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def windowed(N, T, H):
    ws = K.linear_prefill_workspace(N, T, H, DEV)
    assert ws is not None
    return ws


@pytest.mark.parametrize("decay", ["head", "token"])
@pytest.mark.parametrize("lens,H", [([1024, 1, 2400], 2), ([2500, 0, 130, 128, 7], 3), ([40, 3000], 5), ([16 * 128, 16 * 128 + 1], 4)])
def test_prefill_windows_varlen(lens, H, decay):
    windowed(len(lens), sum(lens), H)
    inp = R.linear_inputs(lens, H, seed=38, decay=decay, init=decay == "token", device=DEV)
    out, fin = check(inp, workspace=True)
    alone, none = run(inp, workspace=True, want_final=False)
    assert none is None and torch.equal(alone, out)


def test_prefill_windows_split_and_carry():
    # the state goes from one windowed call to the next in place
    inp = R.linear_inputs([4300], 2, seed=39, decay="token", device=DEV)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    state, outs = inp["init_state"].clone(), []
    for a, b in ((0, 1300), (1300, 2900), (2900, 4300)):
        part = [inp[n][a:b].contiguous() for n in ("q", "k", "v", "log_decay")]
        outs.append(torch.empty_like(part[0]))
        K.kda_linear_prefill(*part, torch.tensor([0, b - a], dtype=torch.int32, device=DEV), state, outs[-1], state, SCALE,
                             workspace=windowed(1, b - a, 2))
    assert_out_close(torch.cat(outs), ref_out)
    assert_state_close(state, ref_fin, tol=3 * STATE_TOL)


def test_prefill_windows_on_another_stream_and_graph():
    inp = R.linear_inputs([2700, 50], 2, seed=40, device=DEV)
    ref, fref = run(inp, True)
    ws = windowed(2, 2750, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q, k, v = (inp[n].clone() for n in "qkv")  # on that stream, behind which the call has to wait
    out, fin = K.linear_prefill(q, k, v, inp["log_decay"], inp["cu_seqlens"], inp["init_state"], scale=SCALE, workspace=ws,
                                stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(fin, fref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        K.kda_linear_prefill(q, k, v, inp["log_decay"], inp["cu_seqlens"], inp["init_state"], out, fin, SCALE, workspace=ws)
    for _ in range(3):
        out.zero_(), fin.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(fin, fref)


def test_prefill_token_offsets_pass_32_bits():
    T, H = 69800, 256  # 2.3e9 elements each
    gen = torch.Generator(device=DEV).manual_seed(41)
    q, k, v = (torch.empty(T, H, 128, dtype=torch.bfloat16, device=DEV).normal_(0.0, s, generator=gen) for s in (0.1, 0.1, 1.0))
    g = -torch.rand(T, H, generator=gen, device=DEV)
    cu = torch.tensor([0, 68000, 69500, T], dtype=torch.int32, device=DEV)
    out, fin = K.linear_prefill(q, k, v, g, cu, scale=SCALE)
    a = 68000
    assert (a * H + 200) * 128 > 2 ** 31
    heads = [0, 200, 255]
    part = [x[a:, heads].contiguous() for x in (q, k, v, g)]
    small, fsmall = K.linear_prefill(*part, cu[1:] - a, scale=SCALE)
    assert torch.equal(out[a:, heads], small) and torch.equal(fin[1:, heads], fsmall)
    inp = dict(zip(("q", "k", "v", "log_decay"), part), cu_seqlens=cu[1:] - a, init_state=None)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    assert_out_close(small, ref_out)
    assert_state_close(fsmall, ref_fin, tol=STATE_TOL)


def test_prefill_state_offsets_pass_32_bits():
    N = 140000  # sequences of one token: 2.3e9 state elements, in place
    gen = torch.Generator(device=DEV).manual_seed(42)
    q, k, v = (torch.randn(N, 1, 128, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(3))
    g = torch.full((1,), -0.5, device=DEV)
    state = torch.full((N, 1, 128, 128), 0.25, device=DEV)
    cu = torch.arange(N + 1, dtype=torch.int32, device=DEV)
    out = torch.empty_like(q)
    K.kda_linear_prefill(q, k, v, g, cu, state, out, state, 0.01)
    for n in (0, 131071, 131072, N - 1):
        want = 0.25 * math.exp(-0.5) + k[n, 0].double()[:, None] * v[n, 0].double()
        assert_state_close(state[n, 0], want, tol=STATE_TOL)
        assert_out_close(out[n, 0], 0.01 * q[n, 0].double() @ want)
    assert K.kda_device_status()[0] == K.KDA_OK


def test_prefill_repeats_bit_for_bit():
    inp = R.linear_inputs([1500, 77], 3, seed=19, device=DEV)
    for ws in (False, True):
        a, fa = run(inp, ws)
        b, fb = run(inp, ws)
        assert torch.equal(a, b) and torch.equal(fa, fb)


def test_prefill_bad_cu_seqlens_are_clamped_and_reported():
    inp = R.linear_inputs([100, 60], 2, seed=20, device=DEV)
    inp["cu_seqlens"] = torch.tensor([0, 100, 900], dtype=torch.int32, device=DEV)
    run(inp)
    assert K.kda_device_status()[0] == K.KDA_ERR_DEVICE_INPUT
    assert K.kda_device_status()[0] == K.KDA_OK


def test_prefill_on_another_stream():
    inp = R.linear_inputs([700, 50], 2, seed=21, device=DEV)
    ref, fref = run(inp, True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out, fin = torch.empty_like(ref), torch.empty_like(fref)
    ws = K.linear_prefill_workspace(2, 750, 2, DEV)
    s.wait_stream(torch.cuda.current_stream())
    K.kda_linear_prefill(inp["q"], inp["k"], inp["v"], inp["log_decay"], inp["cu_seqlens"], inp["init_state"], out,
                         fin, SCALE, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(fin, fref)


# ---------------------------------------------------------------- one token


def token_inputs(rows, H, slots, state, decay, seed):
    inp = R.linear_inputs([rows], H, seed=seed, decay=decay, init=False, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    pool = (torch.randn(slots, H, 128, 128, generator=gen, device=DEV) * 0.1).to(
        torch.float32 if state == "f32" else torch.bfloat16)
    slot = torch.randperm(slots, generator=gen, device=DEV)[:rows].to(torch.int32)
    return inp, pool, slot


@pytest.mark.parametrize("rows,H", [(1, 1), (1, 8), (3, 5), (33, 8), (300, 3), (700, 2)])
@pytest.mark.parametrize("state", ["f32", "bf16"])
@pytest.mark.parametrize("decay", ["head", "token"])
def test_decode(rows, H, state, decay):
    inp, pool, slot = token_inputs(rows, H, rows + 9, state, decay, 31)
    before = pool.clone()
    out = K.linear_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], slot, pool, scale=SCALE)
    ref_out, ref_S = R.linear_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], before[slot.long()], SCALE)
    assert_out_close(out, ref_out)
    assert_state_close(pool[slot.long()], ref_S, tol=1e-6 if state == "f32" else 2.0 ** -9)
    rest = torch.ones(rows + 9, dtype=torch.bool, device=DEV)
    rest[slot.long()] = False
    assert torch.equal(pool[rest], before[rest])
    assert K.kda_device_status()[0] == K.KDA_OK


def test_decode_padding_and_bad_slots():
    inp, pool, slot = token_inputs(6, 2, 10, "f32", "head", 32)
    before = pool.clone()
    slot[1], slot[4] = -1, 10
    out = K.linear_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], slot, pool, scale=SCALE)
    assert (out[[1, 4]] == 0).all() and (out[[0, 2, 3, 5]] != 0).any()
    used = torch.zeros(10, dtype=torch.bool, device=DEV)
    used[slot[[0, 2, 3, 5]].long()] = True
    assert torch.equal(pool[~used], before[~used])
    assert K.kda_device_status() == (K.KDA_ERR_DEVICE_INPUT, 4)


def test_decode_continues_a_prefill():
    inp = R.linear_inputs([200], 4, seed=33, decay="token", device=DEV)
    ref_out, ref_fin = R.linear_prefill(inp, SCALE)
    head = {n: inp[n][:190].contiguous() for n in ("q", "k", "v", "log_decay")}
    head["cu_seqlens"] = torch.tensor([0, 190], dtype=torch.int32, device=DEV)
    head["init_state"] = inp["init_state"]
    _, pool = run(head)
    slot = torch.zeros(1, dtype=torch.int32, device=DEV)
    for t in range(190, 200):
        out = K.linear_decode(*(inp[n][t:t + 1].contiguous() for n in ("q", "k", "v", "log_decay")), slot, pool,
                              scale=SCALE)
        assert_out_close(out, ref_out[t:t + 1])
    assert_state_close(pool, ref_fin, tol=STATE_TOL)


def test_decode_slot_offsets_pass_32_bits():
    slots, H = 20000, 8  # 2.6e9 elements
    pool = torch.empty(slots, H, 128, 128, dtype=torch.bfloat16, device=DEV)
    slot = torch.tensor([19999, 3, 17000], dtype=torch.int32, device=DEV)
    pool[slot.long()] = 0.25
    inp, _, _ = token_inputs(3, H, 3, "bf16", "head", 34)
    ref_out, ref_S = R.linear_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], pool[slot.long()], SCALE)
    out = K.linear_decode(inp["q"], inp["k"], inp["v"], inp["log_decay"], slot, pool, scale=SCALE)
    assert_out_close(out, ref_out)
    assert_state_close(pool[slot.long()], ref_S, tol=2.0 ** -9)


def test_decode_replays_in_a_graph():
    inp, pool, slot = token_inputs(5, 8, 9, "f32", "token", 35)
    start, out = pool.clone(), torch.empty_like(inp["q"])
    args = (inp["q"], inp["k"], inp["v"], inp["log_decay"], slot, pool, out, SCALE)
    K.kda_linear_decode(*args)
    once = pool.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        K.kda_linear_decode(*args)
    pool.copy_(start)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, once)
