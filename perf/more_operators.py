"""Cases of the operators around the attention layer of a served model: pages of the key-value cache handed out as
requests grow and shrink, queries and keys normed, rotated and written into those pages, and attention of one new
token for rows that share a long prefix.

``own`` selects the side: False computes each operator in its plain form (elementary torch operations in 32 bits,
angles in 64, rounded once at the end), True calls the library.

    pages         a row of n tokens holds ceil(n / page size) pages; rows grow by pages from a ring of free ones and
                  give pages back to its end; token t of the packed new tokens goes to cache slot
                  page * page size + position % page size
    norm, rotary  y = x (mean x^2 + eps)^-1/2 w for each head, then the pairs of its first channels turn by
                  position * inv_freq; keys and values go to the cache's slots
    attention     o = sum_j p_j v_j, p = softmax_j(scale q . k_j), where the rows of a group hold the same first
                  tokens in the same pages
"""
import math

import torch

own = False

D = 128
SCALE = 1.0 / math.sqrt(D)
EPS = 1e-6


def listed():
    return [
        # one step of a small batch: every row's next token; a call's latency
        dict(name="pages_64rows_step", op="page_resize", rows=64, lo=256, hi=4096, page=16, kind="step", lens_seed=11),
        # a step of a busy server: some requests begin, some end, the others take a token
        dict(name="pages_1000rows_mixed", op="page_resize", rows=1000, lo=1, hi=4096, page=16, kind="mixed", lens_seed=12),
        # long prompts begin: slots for 131072 tokens
        dict(name="pages_8_prompts_16384", op="page_resize", rows=8, lo=16384, hi=16384, page=64, kind="begin",
             lens_seed=13),
        # one user's next token: latency
        dict(name="rope_1token_h8", op="qk_norm_rope", tokens=1, q_heads=8, kv_heads=8, rot=128, interleaved=False,
             norm="bf16", page=64, packed=True, far=8192, scaled=False, lens_seed=21),
        # an odd batch far into long contexts, part of the head rotated in interleaved pairs, no norm
        dict(name="rope_333tokens_h32_kv8", op="qk_norm_rope", tokens=333, q_heads=32, kv_heads=8, rot=64,
             interleaved=True, norm="none", page=16, packed=False, far=1000000, scaled=True, lens_seed=22),
        # packed ragged prompts of a fused projection
        dict(name="rope_33001tokens_h32_kv8", op="qk_norm_rope", tokens=33001, q_heads=32, kv_heads=8, rot=128,
             interleaved=False, norm="f32", page=16, packed=True, far=4096, scaled=False, lens_seed=23),
        # a large prompt batch: bandwidth
        dict(name="rope_131072tokens_h64_kv8", op="qk_norm_rope", tokens=131072, q_heads=64, kv_heads=8, rot=128,
             interleaved=False, norm="bf16", page=64, packed=False, far=16384, scaled=True, lens_seed=24),
        # four samples of one short prompt: latency
        dict(name="prefix_4rows_512_h8", op="attn_prefix", groups=1, rows=4, prefix_lo=512, prefix_hi=512, tail_lo=1,
             tail_hi=64, q_heads=8, kv_heads=8, page=64, lens_seed=31),
        # a few shared documents of odd lengths, small pages
        dict(name="prefix_32rows_4groups_h32_kv8", op="attn_prefix", groups=4, rows=32, prefix_lo=2048, prefix_hi=8192,
             tail_lo=1, tail_hi=512, q_heads=32, kv_heads=8, page=16, lens_seed=32),
        # many groups with a common instruction each, own histories of some length
        dict(name="prefix_512rows_16groups_h64_kv8", op="attn_prefix", groups=16, rows=512, prefix_lo=2048,
             prefix_hi=4096, tail_lo=1, tail_hi=1024, q_heads=64, kv_heads=8, page=64, lens_seed=33),
        # one long document asked by a large batch: products
        dict(name="prefix_128rows_32768_h64_kv8", op="attn_prefix", groups=1, rows=128, prefix_lo=32768,
             prefix_hi=32768, tail_lo=16, tail_hi=1024, q_heads=64, kv_heads=8, page=64, lens_seed=34),
    ]


def draw(rng):
    """One more case of these ranges, no dearer than the largest listed one of its kind."""
    def span(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["page_resize", "qk_norm_rope", "attn_prefix"])
    seed = rng.randrange(1 << 20)
    if op == "page_resize":
        hi = span(1, 16384)
        return dict(op=op, rows=max(1, min(span(1, 4096), (1 << 20) // hi)), lo=max(1, hi // rng.choice([1, 2, 16, 1024])),
                    hi=hi, page=rng.choice([8, 16, 32, 64, 128]), kind=rng.choice(["step", "mixed", "begin"]), lens_seed=seed)
    kv_heads, group = span(1, 16), rng.choice([1, 2, 3, 4, 6, 8])
    if op == "qk_norm_rope":
        tokens = max(1, min(span(1, 131072), (131072 * 72) // (kv_heads * (group + 2))))
        return dict(op=op, tokens=tokens, q_heads=kv_heads * group, kv_heads=kv_heads,
                    rot=rng.choice([128, 128, 96, 64, 32, 16]), interleaved=rng.random() < 0.5,
                    norm=rng.choice(["none", "bf16", "f32"]), page=rng.choice([8, 16, 32, 64, 128]),
                    packed=rng.random() < 0.5, far=span(1024, 4000000), scaled=rng.random() < 0.5, lens_seed=seed)
    prefix, rows = span(16, 32768), span(2, 256)
    rows = max(2, min(rows, (1 << 28) // (kv_heads * group * prefix)))
    groups = max(1, min(span(1, 16), rows // 2))
    tail = max(1, min(span(1, 4096), (1 << 22) // (rows * kv_heads)))
    return dict(op=op, groups=groups, rows=rows, prefix_lo=max(1, prefix // rng.choice([1, 2, 4])), prefix_hi=prefix,
                tail_lo=max(1, tail // rng.choice([1, 4, 64])), tail_hi=tail, q_heads=kv_heads * group,
                kv_heads=kv_heads, page=rng.choice([8, 16, 32, 64, 128, 256]), lens_seed=seed)


def _rand(case):
    return torch.Generator(device="cpu").manual_seed(case["lens_seed"])


def _ints(gen, lo, hi, n):
    return [int(x) for x in torch.randint(lo, hi + 1, (n,), generator=gen)]


def lengths(case):
    """Part of the case, the same for every seed. Pages: (tokens before, tokens after) of each row; attention:
    (first row of each group and the end, prefix of each group, tokens of each row)."""
    gen = _rand(case)
    n = case["rows"]
    if case["op"] == "page_resize":
        before = _ints(gen, case["lo"], case["hi"], n)
        if case["kind"] == "begin":
            return [0] * n, before
        after = [x + 1 for x in before]
        if case["kind"] == "mixed":  # of eight rows one begins, one ends, one drops what was drafted in vain
            for i, what in enumerate(_ints(gen, 0, 7, n)):
                if what == 0:
                    before[i], after[i] = 0, before[i]
                elif what == 1:
                    after[i] = 0
                elif what == 2:
                    after[i] = max(0, before[i] - 1 - i % 4)
        return before, after
    cuts = sorted(_ints(gen, 0, n - 2 * case["groups"], case["groups"] - 1))  # every group has two rows or more
    first = [0] + [c + 2 * (i + 1) for i, c in enumerate(cuts)] + [n]
    prefix = _ints(gen, case["prefix_lo"], case["prefix_hi"], case["groups"])
    tails = _ints(gen, case["tail_lo"], case["tail_hi"], n)
    lens = []
    for g in range(case["groups"]):
        lens += [prefix[g] + t for t in tails[first[g]:first[g + 1]]]
    return first, prefix, lens


def work(case):
    op = case["op"]
    if op == "page_resize":
        before, after = lengths(case)
        ps = case["page"]
        grown = sum(max(0, b - a) for a, b in zip(before, after))
        moved = sum(abs(-(-b // ps) - -(-a // ps)) for a, b in zip(before, after))
        return {"bytes": case["rows"] * 16 + moved * 8 + grown * (8 + 4 + 4), "flops": grown}
    if op == "qk_norm_rope":
        T, Hq, Hkv = case["tokens"], case["q_heads"], case["kv_heads"]
        return {"bytes": T * ((Hq + 2 * Hkv) * 2 * D * 2 + 12),
                "flops": T * (Hq + Hkv) * (3 * case["rot"] + (4 * D if case["norm"] != "none" else 0))}
    first, prefix, lens = lengths(case)
    shared = sum(prefix)
    tails = sum(lens) - sum(prefix[g] * (first[g + 1] - first[g]) for g in range(case["groups"]))
    return {"bytes": (shared + tails) * case["kv_heads"] * 2 * D * 2 + case["rows"] * case["q_heads"] * (2 * D * 2 + 4),
            "flops": 4 * D * sum(lens) * case["q_heads"]}


# ---------------------------------------------------------------- inputs


def frequencies(case, dev):
    """inv_freq FP32 and the factor on cos and sin. Scaled: waves longer than a quarter of the old context of 8192
    slow down by eight, those shorter than a sixteenth of that stay, a ramp between."""
    rot = case["rot"]
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if not case["scaled"]:
        return f.float().to(dev), 1.0
    turns = 8192 * f / (2 * math.pi)  # in the old context
    keep = ((turns - 4.0) / (64.0 - 4.0)).clamp(0, 1)
    return (f * keep + f / 8 * (1 - keep)).float().to(dev), 0.1 * math.log(8.0) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def order(n):
        return torch.randperm(n, generator=gen, device=dev).to(torch.int32)

    def ints(x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=dev)

    s = dict(case)
    if case["op"] == "page_resize":
        before, after = lengths(case)
        ps, B = case["page"], case["rows"]
        held = [-(-n // ps) for n in before]
        need = [max(0, -(-n // ps) - h) for n, h in zip(after, held)]
        P = max(max(held), max(h + n for h, n in zip(held, need)), 1)
        pages = sum(held) + sum(need) + 37
        ids = order(pages)
        at = torch.arange(P, device=dev)
        held_t = ints(held)
        table = torch.full((B, P), -1, dtype=torch.int32, device=dev)
        table[at < held_t[:, None]] = ids[:sum(held)]  # (row by row)
        free = ids[sum(held):]
        ring = torch.full((pages,), -1, dtype=torch.int32, device=dev)
        start = (seed * 7919) % pages
        ring[(start + torch.arange(free.numel(), device=dev)) % pages] = free
        s["block_table"], s["seq_lens"], s["new_lens"] = table, ints(before), ints(after)
        s["free_pages"], s["free_state"] = ring, ints([start, free.numel()])
        T = sum(max(0, b - a) for a, b in zip(before, after))
        s["max_tokens"] = T + 5  # (a step captured for a few more)
        s["out_lens"], s["out_state"] = torch.empty_like(s["seq_lens"]), torch.empty_like(s["free_state"])
        s["cu_tokens"] = torch.empty(B + 1, dtype=torch.int32, device=dev)
        s["slots"] = torch.empty(T + 5, dtype=torch.int64, device=dev)
        s["positions"], s["token_rows"] = (torch.empty(T + 5, dtype=torch.int32, device=dev) for _ in range(2))
        return s
    if case["op"] == "qk_norm_rope":
        T, Hq, Hkv, ps = case["tokens"], case["q_heads"], case["kv_heads"], case["page"]
        if case["packed"]:  # views of one projection's output
            x = randn(T, Hq + 2 * Hkv, D).to(torch.bfloat16)
            s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (randn(T, h, D).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
        # runs of positions, as prompts have them
        run_len = max(1, min(T, 4096))
        t = torch.arange(T, device=dev)
        base = torch.randint(0, max(1, case["far"] - run_len), (-(-T // run_len),), generator=gen, device=dev)
        s["positions"] = (base[t // run_len] + t % run_len).to(torch.int32)
        pages = -(-T // ps) + 3
        s["slots"] = order(pages).long()[t // ps] * ps + t % ps
        s["inv_freq"], s["magnitude"] = frequencies(case, dev)
        kind = {"none": None, "bf16": torch.bfloat16, "f32": torch.float32}[case["norm"]]
        s["q_weight"], s["k_weight"] = (None if kind is None else (1 + 0.1 * randn(D)).to(kind) for _ in range(2))
        s["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=dev)
        s["k_cache"], s["v_cache"] = (torch.zeros(pages, Hkv, ps, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return s
    first, prefix, lens = lengths(case)
    B, Hkv, ps = case["rows"], case["kv_heads"], case["page"]
    P = max(-(-n // ps) for n in lens)
    group_of = [g for g in range(case["groups"]) for _ in range(first[g], first[g + 1])]
    shared = [p // ps for p in prefix]  # whole pages that a group's rows hold together
    own_pages = [-(-n // ps) - shared[g] for n, g in zip(lens, group_of)]
    total = sum(shared) + sum(own_pages)
    ids = order(total)
    table, at = torch.full((B, P), -1, dtype=torch.int32, device=dev), 0
    for g in range(case["groups"]):
        table[first[g]:first[g + 1], :shared[g]] = ids[at:at + shared[g]]
        at += shared[g]
    for b in range(B):
        table[b, shared[group_of[b]]:shared[group_of[b]] + own_pages[b]] = ids[at:at + own_pages[b]]
        at += own_pages[b]
    k, v = (randn(total, Hkv, ps, D).to(torch.bfloat16) for _ in range(2))
    for g in range(case["groups"]):  # a prefix that ends inside a page: every row has its copy of that page's part
        n = prefix[g] % ps
        if n:
            pages = table[first[g]:first[g + 1], shared[g]].long()
            for cache in (k, v):
                cache[pages, :, :n] = cache[pages[0], :, :n].clone()
    s["q"] = (randn(B, case["q_heads"], D) * 1.5).to(torch.bfloat16)
    s["k_cache"], s["v_cache"], s["block_table"] = k, v, table
    s["seq_lens"], s["cu_groups"], s["prefix_lens"] = ints(lens), ints(first), ints(prefix)
    s["first"], s["prefix"] = first, prefix  # (what the host knows as it made them)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(B, case["q_heads"], device=dev)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    if own:
        return OWN[s["op"]](s)
    return PLAIN[s["op"]](s)


def own_page_resize(s):
    import kda_recurrent_gb300 as K
    K.kda_page_resize(s["block_table"], s["seq_lens"], s["new_lens"], s["free_pages"], s["free_state"], s["page"],
                      s["out_lens"], s["out_state"], cu_tokens=s["cu_tokens"], slots=s["slots"],
                      positions=s["positions"], rows=s["token_rows"])
    return {n: s[n] for n in ("block_table", "out_lens", "free_pages", "out_state", "cu_tokens", "slots", "positions",
                              "token_rows")}


def own_qk_norm_rope(s):
    import kda_recurrent_gb300 as K
    K.kda_qk_norm_rope(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], None, EPS, q_weight=s["q_weight"],
                       k_weight=s["k_weight"], magnitude=s["magnitude"], interleaved=s["interleaved"], v=s["v"],
                       k_cache=s["k_cache"], v_cache=s["v_cache"], slots=s["slots"])
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def own_attn_prefix(s):
    import kda_recurrent_gb300 as K
    if "workspace" not in s:  # kept for the state's later passes
        s["workspace"] = K.attn_prefix_decode_workspace(s["rows"], s["q_heads"], s["kv_heads"], s["block_table"].shape[1],
                                                        s["page"], s["groups"], s["q"].device)
    K.kda_attn_prefix_decode(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["cu_groups"],
                             s["prefix_lens"], s["out"], SCALE, s["workspace"], lse=s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


OWN = {"page_resize": own_page_resize, "qk_norm_rope": own_qk_norm_rope, "attn_prefix": own_attn_prefix}


def plain_page_resize(s):
    ps, table, ring = s["page"], s["block_table"], s["free_pages"]
    dev = table.device
    old, new = s["seq_lens"].long(), s["new_lens"].long()
    B, P = table.shape
    first, count = s["free_state"].long()
    held, want = -(-old // ps), -(-new // ps)
    take = (want - held).clamp_min(0)
    before = take.cumsum(0) - take
    served = before + take <= count  # in order: the first row that does not fit, and all later takers, get none
    served |= take == 0
    out_lens = torch.where(served, new, old)
    at = torch.arange(P, device=dev)
    taken = (at >= held[:, None]) & (at < want[:, None]) & served[:, None]
    source = (first + before[:, None] + at - held[:, None]) % ring.numel()
    given = (at < held[:, None]) & (at >= want[:, None])
    pages = table[given]  # row by row
    pages = pages[pages >= 0]
    grown = torch.where(taken, ring[source], table)
    ring[(first + count + torch.arange(pages.numel(), device=dev)) % ring.numel()] = pages
    table.copy_(grown)
    used = (take * served).sum()
    s["out_state"].copy_(torch.stack([(first + used) % ring.numel(), count - used + pages.numel()]))
    s["out_lens"].copy_(out_lens)
    n = (new - old).clamp_min(0)
    cu = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    s["cu_tokens"].copy_(cu)
    t = torch.arange(s["max_tokens"], device=dev)
    row = torch.searchsorted(cu, t, right=True) - 1
    live = row < B
    row = row.clamp_max(B - 1)
    position = old[row] + t - cu[row]
    page = table[row, (position // ps).clamp_max(P - 1)].long()
    s["slots"].copy_(torch.where(live & served[row] & (page >= 0), page * ps + position % ps, -1))
    s["positions"].copy_(torch.where(live, position, 0))
    s["token_rows"].copy_(torch.where(live, row, -1))
    return {n: s[n] for n in ("block_table", "out_lens", "free_pages", "out_state", "cu_tokens", "slots", "positions",
                              "token_rows")}


def plain_qk_norm_rope(s):
    half = s["rot"] // 2
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos = (torch.cos(angle) * s["magnitude"]).float()[:, None]
    sin = (torch.sin(angle) * s["magnitude"]).float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight.float()
        y = x.clone()
        if s["interleaved"]:
            a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
            y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
        else:
            a, b = x[..., :half], x[..., half:2 * half]
            y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
        return y.to(torch.bfloat16)

    s["q_out"].copy_(turned(s["q"], s["q_weight"]))
    page, at = s["slots"] // s["page"], s["slots"] % s["page"]
    s["k_cache"][page, :, at] = turned(s["k"], s["k_weight"])
    s["v_cache"][page, :, at] = s["v"]
    return {"q": s["q_out"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def plain_attn_prefix(s):
    """Group by group: the scores with the prefix once for all of its rows, those with the rows' own tokens, one
    softmax over both."""
    Hq, Hkv, ps = s["q_heads"], s["kv_heads"], s["page"]
    G, P = Hq // Hkv, s["block_table"].shape[1]
    out, lse = s["out"], s["lse"]
    for a, b, n in zip(s["first"], s["first"][1:], s["prefix"]):
        R = b - a
        pages = s["block_table"][a, :-(-n // ps)].long()
        k, v = (s[c][pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :n].float() for c in ("k_cache", "v_cache"))
        q = s["q"][a:b].float().view(R, Hkv, G, D)
        x = (q.transpose(0, 1).reshape(Hkv, R * G, D) @ k.transpose(-1, -2)).view(Hkv, R, G, n).transpose(0, 1) * SCALE
        from_page = n // ps
        pages = s["block_table"][a:b, from_page:].clamp_min(0).long()
        tk, tv = (s[c][pages].transpose(1, 2).reshape(R, Hkv, -1, D).float() for c in ("k_cache", "v_cache"))
        j = torch.arange(from_page * ps, P * ps, device=q.device)
        live = (j >= n) & (j < s["seq_lens"][a:b, None])
        y = (q @ tk.transpose(-1, -2) * SCALE).masked_fill(~live[:, None, None], -math.inf)
        tv = tv.masked_fill(~live[:, None, :, None], 0)
        top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
        x, y = torch.exp(x - top), torch.exp(y - top)
        norm = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
        o = (x.transpose(0, 1).reshape(Hkv, R * G, n) @ v).view(Hkv, R, G, D).transpose(0, 1) + y @ tv
        out[a:b] = (o / norm).reshape(R, Hq, D).to(torch.bfloat16)
        lse[a:b] = (top + torch.log(norm)).view(R, Hq)
    return {"out": out, "lse": lse}


PLAIN = {"page_resize": plain_page_resize, "qk_norm_rope": plain_qk_norm_rope, "attn_prefix": plain_attn_prefix}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def exact_page_resize(s):
    """Row by row on the host."""
    ps, dev = s["page"], s["block_table"].device
    table, ring = s["block_table"].tolist(), s["free_pages"].tolist()
    first, count = s["free_state"].tolist()
    old, new = s["seq_lens"].tolist(), s["new_lens"].tolist()
    tail, used, short = first + count, 0, False
    lens, cu, slots, positions, rows, back = [], [0], [], [], [], []
    for b, (n, m) in enumerate(zip(old, new)):
        held, want = (n + ps - 1) // ps, (m + ps - 1) // ps
        ok = True
        if want > held:
            short = short or used + want - held > count
            ok = not short
            if ok:
                for i in range(held, want):
                    table[b][i] = ring[(first + used) % len(ring)]
                    used += 1
        back += [p for p in table[b][want:held] if p >= 0]
        lens.append(m if ok else n)
        for j in range(n, m):
            page = table[b][j // ps] if ok else -1
            slots.append(page * ps + j % ps if page >= 0 else -1)
            positions.append(j)
            rows.append(b)
        cu.append(cu[-1] + max(0, m - n))
    for i, p in enumerate(back):
        ring[(tail + i) % len(ring)] = p
    pad = s["max_tokens"] - len(slots)

    def made(x, like):
        return torch.tensor(x, dtype=like.dtype, device=dev)

    return {"block_table": made(table, s["block_table"]), "out_lens": made(lens, s["seq_lens"]),
            "free_pages": made(ring, s["free_pages"]),
            "out_state": made([(first + used) % len(ring), count - used + len(back)], s["free_state"]),
            "cu_tokens": made(cu, s["cu_tokens"]), "slots": made(slots + [-1] * pad, s["slots"]),
            "positions": made(positions + [0] * pad, s["positions"]), "token_rows": made(rows + [-1] * pad, s["token_rows"])}


def exact_qk_norm_rope(s):
    """Each pair as a complex number."""
    half, T = s["rot"] // 2, s["tokens"]
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    q_out = torch.empty(T, s["q_heads"], D, dtype=torch.float64, device=k_cache.device)
    for lo in range(0, T, 8192):
        at = slice(lo, min(T, lo + 8192))
        turn = torch.polar(torch.full((1,), s["magnitude"], dtype=torch.float64, device=k_cache.device),
                           s["positions"][at].double()[:, None] * s["inv_freq"].double())[:, None]

        def turned(x, weight):
            x = x.double()
            if weight is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + EPS) * weight.double()
            pairs = x[..., :2 * half]
            pairs = pairs.unflatten(-1, (half, 2)) if s["interleaved"] else pairs.unflatten(-1, (2, half)).transpose(-1, -2)
            pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            pairs = pairs if s["interleaved"] else pairs.transpose(-1, -2)
            return torch.cat([pairs.flatten(-2), x[..., 2 * half:]], -1)

        q_out[at] = turned(s["q"][at], s["q_weight"])
        page, off = s["slots"][at] // s["page"], s["slots"][at] % s["page"]
        k_cache[page, :, off] = turned(s["k"][at], s["k_weight"])
        v_cache[page, :, off] = s["v"][at].double()
    return {"q": q_out, "k_cache": k_cache, "v_cache": v_cache}


def exact_attn_prefix(s):
    """Row by row over the row's own table."""
    Hq, Hkv, ps = s["q_heads"], s["kv_heads"], s["page"]
    lens = s["seq_lens"].tolist()
    if sum(lens) * Hq > 1 << 29:
        return None
    out = torch.zeros(s["rows"], Hq, D, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["rows"], Hq, dtype=torch.float64, device=s["q"].device)
    for b, n in enumerate(lens):
        pages = s["block_table"][b, :-(-n // ps)].long()
        k, v = (s[c][pages].permute(1, 0, 2, 3).flatten(1, 2)[:, :n].double() for c in ("k_cache", "v_cache"))
        q = s["q"][b].double().unflatten(0, (Hkv, -1))
        x = torch.einsum("hgd,hnd->hgn", q, k) * SCALE
        lse[b] = torch.logsumexp(x, -1).flatten()
        out[b] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), v).flatten(0, 1)
    return {"out": out, "lse": lse}


EXACT = {"page_resize": exact_page_resize, "qk_norm_rope": exact_qk_norm_rope, "attn_prefix": exact_attn_prefix}
