"""Cases of the operators that a model with KDA layers needs beside them: linear attention with a decay
for each head (prompt and single-token form), attention of one new token over a paged key-value cache, and
eviction from that cache by accumulated attention weight.

``own`` selects the side: False computes each operator in its plain form (elementary torch operations in
32 bits, rounded once at the end), True calls the library.

    linear attention   S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t   (one 128 x 128 state a head)
    attention          o = sum_j p_j v_j,  p = softmax_j(scale q . k_j) over the cached tokens j of a sequence;
                       the weight of token j grows by p_j, summed over the query heads that share its key
    eviction           a sequence longer than `budget` keeps its first `sink` and last `recent` tokens and the
                       heaviest others (ties: the earlier token), packed in their order
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
CHUNK = 128  # of the plain chunked form


def listed():
    return [
        # the smallest prompt: one sequence, one head, half a chunk; a call's latency
        dict(name="linear_prompt_1x64_h1", op="linear_prefill", seqs=1, lo=64, hi=64, heads=1, decay="head",
             init=False, lens_seed=0),
        # one long prompt on few heads: the chains alone leave most of the GPU idle
        dict(name="linear_prompt_1x8192_h8", op="linear_prefill", seqs=1, lo=8192, hi=8192, heads=8, decay="head",
             init=True, lens_seed=0),
        # a packed batch of ragged prompts with gates that depend on the token
        dict(name="linear_prompt_16_ragged_h32", op="linear_prefill", seqs=16, lo=256, hi=4096, heads=32,
             decay="token", init=False, lens_seed=2),
        # the large prompt batch: bandwidth
        dict(name="linear_prompt_8x16384_h96", op="linear_prefill", seqs=8, lo=16384, hi=16384, heads=96,
             decay="head", init=True, lens_seed=0),
        # one user's next token
        dict(name="linear_token_1row_h8_f32", op="linear_decode", rows=1, heads=8, slots=64, state="f32",
             decay="head"),
        # an odd batch of rows on BF16 states, gates that depend on the token
        dict(name="linear_token_333rows_h32_bf16", op="linear_decode", rows=333, heads=32, slots=400, state="bf16",
             decay="token"),
        # a full serving batch on FP32 states
        dict(name="linear_token_4096rows_h8_f32", op="linear_decode", rows=4096, heads=8, slots=6144, state="f32",
             decay="head"),
        # one user's next token over a short cache: latency
        dict(name="attn_1x1000_h8", op="attn_decode", seqs=1, lo=1000, hi=1000, q_heads=8, kv_heads=8, page=64,
             weight=False, lens_seed=0),
        # a ragged batch with shared key heads and small pages, which also accumulates the weights
        dict(name="attn_16_ragged_h32_kv8_weight", op="attn_decode", seqs=16, lo=256, hi=4096, q_heads=32, kv_heads=8,
             page=16, weight=True, lens_seed=2),
        # long caches of a large batch: bandwidth
        dict(name="attn_64_long_h64_kv8", op="attn_decode", seqs=64, lo=4096, hi=32768, q_heads=64, kv_heads=8,
             page=64, weight=False, lens_seed=5),
        # two short caches cut to a small budget: latency
        dict(name="evict_2x1500_to_512_kv8", op="cache_evict", seqs=2, lo=1400, hi=1600, kv_heads=8, page=16,
             budget=512, sink=4, recent=128, lens_seed=6),
        # a batch of long caches cut to a quarter: bandwidth
        dict(name="evict_32_long_to_4096_kv8", op="cache_evict", seqs=32, lo=8192, hi=16384, kv_heads=8, page=64,
             budget=4096, sink=16, recent=1024, lens_seed=7),
    ]


def draw(rng):
    """One more case of these ranges, no dearer than the largest listed one of its kind."""
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["linear_prefill", "linear_decode", "attn_decode", "cache_evict"])
    seed = rng.randrange(1 << 20)
    if op == "linear_prefill":
        heads, hi = span(1, 96), span(1, 16384)
        seqs = max(1, min(span(1, 64), (4 << 20) // (heads * max(hi, CHUNK))))
        return dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi, heads=heads,
                    decay=rng.choice(["head", "token"]), init=rng.random() < 0.5, lens_seed=seed)
    if op == "linear_decode":
        heads = span(1, 96)
        rows = max(1, min(span(1, 4096), (4096 * 8) // heads))
        return dict(op=op, rows=rows, heads=heads, slots=rows + span(1, 1000), state=rng.choice(["f32", "bf16"]),
                    decay=rng.choice(["head", "token"]), lens_seed=seed)
    kv_heads, page = span(1, 32), rng.choice([16, 32, 64, 128])
    if op == "attn_decode":
        hi = span(1, 65536)
        seqs = max(1, min(span(1, 256), (8 << 20) // (kv_heads * max(hi, 64))))
        return dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 2, 16])), hi=hi,
                    q_heads=kv_heads * rng.choice([1, 2, 3, 4, 6, 8, 16]), kv_heads=kv_heads, page=page,
                    weight=rng.random() < 0.5, lens_seed=seed)
    hi = span(64, 32768)
    seqs = max(1, min(span(1, 64), (2 << 20) // (kv_heads * hi)))
    budget = max(8, int(hi * rng.uniform(0.1, 0.9)))
    return dict(op=op, seqs=seqs, lo=max(1, hi // rng.choice([1, 2, 4])), hi=hi, kv_heads=kv_heads, page=page,
                budget=budget, sink=rng.randrange(0, budget // 8 + 1), recent=rng.randrange(0, budget // 2 + 1),
                lens_seed=seed)


def lengths(case):
    """The sequences' lengths: part of the case, the same for every seed."""
    gen = torch.Generator(device="cpu").manual_seed(case["lens_seed"])
    return [int(n) for n in torch.randint(case["lo"], case["hi"] + 1, (case["seqs"],), generator=gen)]


def work(case):
    op = case["op"]
    if op == "linear_prefill":
        lens = lengths(case)
        tokens = sum(lens) * case["heads"]
        states = case["seqs"] * case["heads"] * D * D * 4
        gates = 4 * (case["heads"] if case["decay"] == "head" else tokens)
        return {"bytes": tokens * 4 * D * 2 + gates + states * (2 if case["init"] else 1), "flops": tokens * 4 * D * D}
    if op == "linear_decode":
        items = case["rows"] * case["heads"]
        return {"bytes": items * (2 * D * D * (4 if case["state"] == "f32" else 2) + 4 * D * 2), "flops": items * 4 * D * D}
    lens = lengths(case)
    cached = sum(lens) * case["kv_heads"]
    if op == "attn_decode":
        heads = case["seqs"] * case["q_heads"]
        return {"bytes": cached * (2 * D * 2 + (8 if case["weight"] else 0)) + heads * (2 * D * 2 + 4),
                "flops": 4 * D * sum(lens) * case["q_heads"]}
    kept = sum(min(n, case["budget"]) for n in lens) * case["kv_heads"]
    return {"bytes": cached * 4 + kept * (2 * 2 * D * 2 + 4 + 4), "flops": cached}


# ---------------------------------------------------------------- inputs


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def unit(*shape):  # L2-normalised queries and keys
        x = randn(*shape)
        return x.mul_(torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    s = dict(case)
    if case["op"] in ("linear_prefill", "linear_decode"):
        H = case["heads"]
        # slow and fast heads: e^g between about 1 - 2^-4 and 1 - 2^-12, per token scaled by softplus of a gate
        rate = torch.exp2(-4.0 - 8.0 * torch.rand(H, generator=gen, device=dev))
        if case["op"] == "linear_prefill":
            lens = lengths(case)
            T = sum(lens)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            s["lens"] = torch.tensor(lens, device=dev)
            s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            s["init_state"] = randn(case["seqs"], H, D, D) * 0.02 if case["init"] else None
            s["final_state"] = torch.empty(case["seqs"], H, D, D, device=dev)
            n = T
        else:
            n = case["rows"]
            pool = randn(case["slots"], H, D, D).mul_(0.02)
            s["pool"] = pool if case["state"] == "f32" else pool.to(torch.bfloat16)
            s["slot_idx"] = torch.randperm(case["slots"], generator=gen, device=dev)[:n].to(torch.int32)
        s["q"], s["k"] = unit(n, H, D), unit(n, H, D)
        s["v"] = randn(n, H, D).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["log_decay"] = -rate if case["decay"] == "head" else -rate * torch.nn.functional.softplus(randn(n, H))
        return s

    lens = lengths(case)
    B, Hkv, ps = case["seqs"], case["kv_heads"], case["page"]
    pages = [-(-n // ps) for n in lens]
    P = max(pages)
    dst = [-(-min(n, case["budget"]) // ps) for n in lens] if case["op"] == "cache_evict" else [0] * B
    total = sum(pages) + sum(dst)
    order = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    table, dst_table, at = torch.full((B, P), -1, dtype=torch.int32, device=dev), None, 0
    for b in range(B):
        table[b, :pages[b]] = order[at:at + pages[b]]
        at += pages[b]
    s["block_table"], s["seq_lens"] = table, torch.tensor(lens, dtype=torch.int32, device=dev)
    s["k_cache"] = randn(total, Hkv, ps, D).to(torch.bfloat16)
    s["v_cache"] = randn(total, Hkv, ps, D).to(torch.bfloat16)
    if case["op"] == "attn_decode":
        s["q"] = (randn(B, case["q_heads"], D) * 1.5).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, case["q_heads"], device=dev)
        s["weight_acc"] = torch.rand(B, Hkv, P * ps, generator=gen, device=dev) * 1e-2 if case["weight"] else None
        return s
    dst_table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
    for b in range(B):
        dst_table[b, :dst[b]] = order[at:at + dst[b]]
        at += dst[b]
    s["dst_table"] = dst_table
    # heavy-tailed weights; one token in sixteen was never looked at (ties)
    u = torch.rand(B, Hkv, P * ps, generator=gen, device=dev)
    s["weight_acc"] = torch.where(u < 1 / 16, torch.zeros_like(u), -torch.log(u).clamp_max(0) ** 3)
    s["dst_weight"] = torch.zeros_like(s["weight_acc"])
    s["new_lens"] = torch.empty(B, dtype=torch.int32, device=dev)
    s["kept"] = torch.empty(B, Hkv, case["budget"], dtype=torch.int32, device=dev)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return OWN[s["op"]](s)
    return PLAIN[s["op"]](s)


def own_linear_prefill(s):
    import kda_recurrent_gb300 as K
    if "workspace" not in s:  # kept for the state's later passes
        s["workspace"] = K.linear_prefill_workspace(s["seqs"], s["q"].shape[0], s["heads"], s["q"].device)
    K.kda_linear_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["cu_seqlens"], s["init_state"], s["out"],
                         s["final_state"], SCALE, workspace=s["workspace"])
    return {"out": s["out"], "final_state": s["final_state"]}


def own_linear_decode(s):
    import kda_recurrent_gb300 as K
    K.kda_linear_decode(s["q"], s["k"], s["v"], s["log_decay"], s["slot_idx"], s["pool"], s["out"], SCALE)
    return {"out": s["out"], "pool": s["pool"]}


def own_attn_decode(s):
    import kda_recurrent_gb300 as K
    if "workspace" not in s:  # kept for the state's later passes
        s["workspace"] = K.attn_decode_workspace(s["seqs"], s["q_heads"], s["kv_heads"], s["block_table"].shape[1],
                                                 s["page"], s["weight"], s["q"].device)
    K.kda_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["out"], SCALE,
                      s["workspace"], lse=s["lse"], weight=s["weight_acc"])
    return {"out": s["out"], "lse": s["lse"], "weight": s["weight_acc"]}


def own_cache_evict(s):
    import kda_recurrent_gb300 as K
    K.kda_cache_evict(s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["weight_acc"], s["new_lens"],
                      s["kept"], s["budget"], sink=s["sink"], recent=s["recent"], dst_table=s["dst_table"],
                      dst_weight=s["dst_weight"])
    return {"kept": s["kept"], "new_lens": s["new_lens"], "weight": s["dst_weight"], "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


OWN = {"linear_prefill": own_linear_prefill, "linear_decode": own_linear_decode, "attn_decode": own_attn_decode,
       "cache_evict": own_cache_evict}


def plain_linear_prefill(s):
    """Chunked form, every chunk at once: products inside a chunk under the decays between its tokens, each
    chunk's own state, the states' sums over earlier chunks by a matrix of decays between chunks."""
    N, H = s["seqs"], s["heads"]
    dev = s["q"].device
    C = -(-s["hi"] // CHUNK)
    t = torch.arange(C * CHUNK, device=dev)
    live = t < s["lens"][:, None]                                                       # [N, C CHUNK]
    at = (s["cu_seqlens"][:-1, None].long() + t).clamp_max(s["q"].shape[0] - 1)

    def chunks(x):
        x = x[at].float() * live[..., None, None]                                       # [N, C CHUNK, H, D]
        return x.view(N, C, CHUNK, H, -1).permute(0, 3, 1, 2, 4)                        # [N, H, C, CHUNK, D]

    q, k, v = chunks(s["q"]), chunks(s["k"]), chunks(s["v"])
    g = s["log_decay"].expand(s["q"].shape[0], H)
    g = (g[at] * live[..., None]).view(N, C, CHUNK, H).permute(0, 3, 1, 2)              # [N, H, C, CHUNK]
    G = g.cumsum(-1)
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    pair = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~causal, -math.inf))
    out = (q @ k.transpose(-1, -2) * pair) @ v
    del pair
    total = G[..., -1]                                                                  # [N, H, C]
    own_states = (k * torch.exp(total[..., None] - G)[..., None]).transpose(-1, -2) @ v  # [N, H, C, D, D]
    start = s["init_state"] if s["init_state"] is not None else torch.zeros(N, H, D, D, device=dev)
    source = torch.cat([start[:, :, None], own_states], 2).view(N, H, C + 1, D * D)
    del own_states
    # between[c, j] = sum of total[m] over j <= m < c
    m, j = torch.arange(C, device=dev)[:, None], torch.arange(C + 1, device=dev)
    between = (total[..., :, None] * (m >= j)).cumsum(-2)
    between = torch.cat([torch.zeros_like(between[..., :1, :]), between], -2)
    seen = torch.arange(C + 1, device=dev)[:, None] >= j
    states = (torch.exp(between) * seen @ source).view(N, H, C + 1, D, D)
    del source
    out += (q * torch.exp(G)[..., None]) @ states[:, :, :-1]
    out = (out * SCALE).permute(0, 2, 3, 1, 4).reshape(N, C * CHUNK, H, D)[live]
    return {"out": out.to(torch.bfloat16), "final_state": states[:, :, -1].clone()}


def plain_linear_decode(s):
    slots = s["slot_idx"].long()
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    decay = torch.exp(s["log_decay"].expand(s["rows"], s["heads"]))
    state = s["pool"][slots].float() * decay[..., None, None] + k[..., :, None] * v[..., None, :]
    out = (q[..., None, :] @ state)[..., 0, :] * SCALE
    s["pool"][slots] = state.to(s["pool"].dtype)
    return {"out": out.to(torch.bfloat16), "pool": s["pool"]}


def plain_attn_decode(s):
    B, Hq, Hkv, ps = s["seqs"], s["q_heads"], s["kv_heads"], s["page"]
    P = s["block_table"].shape[1]
    pages = s["block_table"].clamp_min(0).long()

    def rows(cache):
        return cache[pages].transpose(1, 2).reshape(B, Hkv, P * ps, D).float()

    live = torch.arange(P * ps, device=s["q"].device) < s["seq_lens"][:, None]          # [B, P ps]
    q = s["q"].float().view(B, Hkv, Hq // Hkv, D)
    x = (q @ rows(s["k_cache"]).transpose(-1, -2) * SCALE).masked_fill(~live[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    norm = p.sum(-1, keepdim=True)
    p = p / norm
    out = (p @ rows(s["v_cache"])).view(B, Hq, D).to(torch.bfloat16)
    if s["weight_acc"] is not None:
        s["weight_acc"] += p.sum(2)
    return {"out": out, "lse": (top + torch.log(norm)).view(B, Hq), "weight": s["weight_acc"]}


def plain_cache_evict(s):
    B, Hkv, ps, budget = s["seqs"], s["kv_heads"], s["page"], s["budget"]
    cap = s["block_table"].shape[1] * ps
    dev = s["k_cache"].device
    j = torch.arange(cap, device=dev)
    lens = s["seq_lens"].long()
    live = j < lens[:, None]
    safe = live & ((j < s["sink"]) | (j >= lens[:, None] - s["recent"]))
    kind = (safe.long() * 2 + (live & ~safe).long())[:, None].expand(B, Hkv, cap)      # 2: safe, 1: by weight, 0: none
    order = torch.argsort(s["weight_acc"], dim=-1, descending=True, stable=True)
    order = order.gather(-1, torch.argsort(kind.gather(-1, order), dim=-1, descending=True, stable=True))
    new_lens = lens.clamp_max(budget)
    i = torch.arange(budget, device=dev)
    used = (i < new_lens[:, None])[:, None].expand(B, Hkv, budget)
    order = torch.nn.functional.pad(order, (0, max(0, budget - cap)))[..., :budget]
    kept = order.masked_fill(~used, cap).sort(-1).values.masked_fill(~used, -1)
    b, h, n = used.nonzero(as_tuple=True)
    src = kept[b, h, n]
    from_page, to_page = s["block_table"][b, src // ps].long(), s["dst_table"][b, n // ps].long()
    for_h = (to_page, h, n % ps)
    s["k_cache"][for_h] = s["k_cache"][from_page, h, src % ps]
    s["v_cache"][for_h] = s["v_cache"][from_page, h, src % ps]
    weight = s["dst_weight"].masked_fill(live[:, None], 0.0)
    weight[b, h, n] = s["weight_acc"][b, h, src]
    s["dst_weight"].copy_(weight)
    return {"kept": kept.to(torch.int32), "new_lens": new_lens.to(torch.int32), "weight": s["dst_weight"],
            "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


PLAIN = {"linear_prefill": plain_linear_prefill, "linear_decode": plain_linear_decode,
         "attn_decode": plain_attn_decode, "cache_evict": plain_cache_evict}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def exact_linear_prefill(s):
    """Token by token."""
    cu, H = s["cu_seqlens"].tolist(), s["heads"]
    T, dev = s["q"].shape[0], s["q"].device
    first = torch.tensor(cu[:-1], device=dev)
    lens = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device=dev)
    g = s["log_decay"].double().expand(T, H)
    state = torch.zeros(s["seqs"], H, D, D, dtype=torch.float64, device=dev)
    if s["init_state"] is not None:
        state += s["init_state"].double()
    out = torch.zeros(T, H, D, dtype=torch.float64, device=dev)
    shortest = int(lens.min())
    for t in range(int(lens.max())):
        n = slice(None) if t < shortest else (lens > t).nonzero()[:, 0]
        at = (first + t)[n]
        new = state[n] * torch.exp(g[at])[..., None, None]
        new += s["k"][at].double()[..., :, None] * s["v"][at].double()[..., None, :]
        out[at] = (s["q"][at].double()[..., None, :] @ new)[..., 0, :] * SCALE
        if t < shortest:
            state = new
        else:
            state[n] = new
    return {"out": out, "final_state": state}


def exact_linear_decode(s):
    pool = s["pool"].double()
    decay = torch.exp(s["log_decay"].double().expand(s["rows"], s["heads"]))
    out = torch.empty(s["rows"], s["heads"], D, dtype=torch.float64, device=pool.device)
    for h in range(s["heads"]):
        k, v, q = (s[x][:, h].double() for x in "kvq")
        new = torch.einsum("r,rij->rij", decay[:, h], pool[s["slot_idx"].long(), h]) + torch.einsum("ri,rj->rij", k, v)
        out[:, h] = torch.einsum("ri,rij->rj", q, new) * SCALE
        pool[s["slot_idx"].long(), h] = new
    return {"out": out, "pool": pool}


def exact_attn_decode(s):
    Hq, Hkv = s["q_heads"], s["kv_heads"]
    out = torch.zeros(s["seqs"], Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["seqs"], Hq, dtype=torch.float64, device=s["q"].device)
    weight = None if s["weight_acc"] is None else s["weight_acc"].double()
    for b, n in enumerate(s["seq_lens"].tolist()):
        pages = s["block_table"][b, :-(-n // s["page"])].long()
        for h in range(Hkv):
            k = s["k_cache"][pages, h].reshape(-1, D)[:n].double()
            v = s["v_cache"][pages, h].reshape(-1, D)[:n].double()
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = torch.einsum("gd,nd->gn", s["q"][b, heads].double(), k) * SCALE
            lse[b, heads] = torch.logsumexp(x, -1)
            p = torch.softmax(x, -1)
            out[b, heads] = torch.einsum("gn,nd->gd", p, v)
            if weight is not None:
                weight[b, h, :n] += p.sum(0)
    return {"out": out, "lse": lse, "weight": weight}


def exact_cache_evict(s):
    ps, budget = s["page"], s["budget"]
    kept = torch.full_like(s["kept"], -1)
    new_lens = torch.zeros_like(s["new_lens"])
    weight, k, v = (s[x].double() for x in ("dst_weight", "k_cache", "v_cache"))
    for b, n in enumerate(s["seq_lens"].tolist()):
        m = min(n, budget)
        new_lens[b] = m
        for h in range(s["kv_heads"]):
            w = s["weight_acc"][b, h, :n].double()
            ids = torch.arange(n, device=w.device)
            if n > budget:
                free = ids[s["sink"]:n - s["recent"]]
                best = free[torch.sort(-w[free], stable=True).indices[:budget - s["sink"] - s["recent"]]]
                ids = torch.cat([ids[:s["sink"]], best.sort().values, ids[n - s["recent"]:]])
            kept[b, h, :m] = ids.to(torch.int32)
            weight[b, h, :n] = 0
            weight[b, h, :m] = w[ids]
            i = torch.arange(m, device=w.device)
            src, dst = s["block_table"][b, ids // ps].long(), s["dst_table"][b, i // ps].long()
            k[dst, h, i % ps] = s["k_cache"][src, h, ids % ps].double()
            v[dst, h, i % ps] = s["v_cache"][src, h, ids % ps].double()
    return {"kept": kept, "new_lens": new_lens, "weight": weight, "k_cache": k, "v_cache": v}


EXACT = {"linear_prefill": exact_linear_prefill, "linear_decode": exact_linear_decode,
         "attn_decode": exact_attn_decode, "cache_evict": exact_cache_evict}
