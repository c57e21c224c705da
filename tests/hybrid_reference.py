"""Plain 64-bit forms (CPU) of the operators beside KDA layers, and their input recipes."""
from __future__ import annotations

import math

import torch

D = 128


def linear_inputs(lens, H, *, seed, decay="token", init=True, device="cuda"):
    """q, k (L2-normalised), v BF16 [T, H, 128]; log_decay FP32 [H] or [T, H]; cu_seqlens; init_state."""
    gen = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)

    def randn(*shape):
        return torch.randn(*shape, generator=gen)

    def unit():
        x = randn(T, H, D)
        return (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    q, k, v = unit(), unit(), randn(T, H, D).to(torch.bfloat16)
    rate = torch.exp2(-1.0 - 7.0 * torch.rand(H, generator=gen))
    g = -rate if decay == "head" else -rate * torch.nn.functional.softplus(randn(T, H))
    cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    state = randn(N, H, D, D) * 0.1 if init else None
    out = dict(q=q, k=k, v=v, log_decay=g, cu_seqlens=cu, init_state=state)
    return {n: None if x is None else x.to(device) for n, x in out.items()}


def linear_prefill(inp, scale):
    """(out [T, H, 128], final_state) in FP64, token by token."""
    x = {n: None if t is None else t.cpu() for n, t in inp.items()}
    T, H, _ = x["q"].shape
    cu = x["cu_seqlens"].tolist()
    g = x["log_decay"].double().expand(T, H)
    out = torch.zeros(T, H, D, dtype=torch.float64)
    final = torch.zeros(len(cu) - 1, H, D, D, dtype=torch.float64)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        S = torch.zeros(H, D, D, dtype=torch.float64) if x["init_state"] is None else x["init_state"][n].double()
        for t in range(a, b):
            decay = torch.exp(g[t])[:, None, None]
            S = torch.where(decay == 0, torch.zeros_like(S), S * decay)
            S = S + x["k"][t].double()[:, :, None] * x["v"][t].double()[:, None, :]
            out[t] = scale * torch.einsum("hi,hij->hj", x["q"][t].double(), S)
        final[n] = S
    return out, final


def linear_decode(q, k, v, log_decay, states, scale):
    """(out, new states) in FP64 for gathered states [R, H, 128, 128]."""
    R, H, _ = q.shape
    g = log_decay.cpu().double().expand(R, H)
    S = states.cpu().double() * torch.exp(g)[..., None, None]
    S = S + k.cpu().double()[..., :, None] * v.cpu().double()[..., None, :]
    return scale * torch.einsum("rhi,rhij->rhj", q.cpu().double(), S), S


def cache_inputs(lens, Hkv, page_size, *, seed, extra_pages=3, max_pages=None, combined=False, device="cuda"):
    """A paged cache holding rows of the given lengths in shuffled pages, with NaN in every slot that no
    row owns."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    P = max(1, max(need)) if max_pages is None else max_pages
    pages = sum(need) + extra_pages
    order = torch.randperm(pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), P), -1, dtype=torch.int32)
    kv = torch.full((pages, 2, Hkv, page_size, D), math.nan, dtype=torch.bfloat16)
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        for i in range(need[b]):
            m = min(page_size, n - i * page_size)
            kv[order[at + i], :, :, :m] = torch.randn(2, Hkv, m, D, generator=gen).to(torch.bfloat16)
        at += need[b]
    kv = kv.to(device)
    k, v = kv[:, 0], kv[:, 1]
    if not combined:
        k, v = k.contiguous(), v.contiguous()
    return dict(k_cache=k, v_cache=v, block_table=table.to(device),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=device), free=order[at:].tolist())


def attn_decode(q, c, scale):
    """(out, lse, weight sums [B, Hkv, capacity]) in FP64; tokens of missing pages are masked."""
    B, Hq, _ = q.shape
    k, v, table = c["k_cache"].cpu().double(), c["v_cache"].cpu().double(), c["block_table"].cpu()
    _, Hkv, ps, _ = k.shape
    G, cap = Hq // Hkv, table.shape[1] * ps
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64)
    weight = torch.zeros(B, Hkv, cap, dtype=torch.float64)
    q = q.cpu().double()
    for b, n in enumerate(c["seq_lens"].tolist()):
        n = min(max(n, 0), cap)
        js = [j for j in range(n) if 0 <= int(table[b, j // ps]) < k.shape[0]]
        if not js:
            continue
        j = torch.tensor(js)
        p, s = table[b, j // ps].long(), j % ps
        for h in range(Hkv):
            heads = slice(h * G, (h + 1) * G)
            x = scale * q[b, heads] @ k[p, h, s].T
            lse[b, heads] = torch.logsumexp(x, -1)
            w = torch.softmax(x, -1)
            out[b, heads] = w @ v[p, h, s]
            weight[b, h, j] = w.sum(0)
    return out, lse, weight


def evict_choice(w, n, budget, sink, recent):
    """Positions kept of a row of n tokens with weights w (a list), by the definition."""
    if n <= budget:
        return list(range(n))
    free = sorted(range(sink, n - recent), key=lambda j: (-(-math.inf if math.isnan(w[j]) else w[j]), j))
    return sorted(list(range(sink)) + free[:budget - sink - recent] + list(range(n - recent, n)))
