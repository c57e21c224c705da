"""Plain forms (CPU, 64 bits) of the operators around the attention layer of a served model, and their inputs."""
from __future__ import annotations

import math

import torch

D = 128


def page_resize(table, old, new, ring, state, page_size, max_tokens):
    """(table, lens, ring, state, cu_tokens, slots, positions, rows) after the call, from lists; lengths in range."""
    table, ring = [list(r) for r in table], list(ring)
    F = len(ring)
    first, count = state
    used, short, back = 0, False, []
    lens, cu, slots, positions, rows = [], [0], [], [], []
    for b, (n, m) in enumerate(zip(old, new)):
        held, want = -(-n // page_size), -(-m // page_size)
        if want > held and (short or used + want - held > count):
            short = True
        fits = want <= held or not short
        if fits:
            for i in range(held, want):
                table[b][i] = ring[(first + used) % F]
                used += 1
        back += [x for x in table[b][want:held] if x >= 0]
        lens.append(m if fits else n)
        for j in range(n, m):
            page = table[b][j // page_size] if fits else -1
            slots.append(page * page_size + j % page_size if page >= 0 else -1)
            positions.append(j)
            rows.append(b)
        cu.append(len(slots))
    for i, x in enumerate(back):
        ring[(first + count + i) % F] = x
    pad = max_tokens - len(slots)
    return (table, lens, ring, [(first + used) % F, count - used + len(back)], cu, slots + [-1] * pad, positions + [0] * pad,
            rows + [-1] * pad)


def page_inputs(old, new, page_size, *, seed, spare=5, max_pages=None, start=None):
    """Lists: rows of the lengths `old` in shuffled pages, and `spare` free pages more than `new` takes."""
    gen = torch.Generator().manual_seed(seed)
    held, want = [-(-n // page_size) for n in old], [-(-n // page_size) for n in new]
    need = sum(max(0, w - h) for h, w in zip(held, want))
    F = max(1, sum(held) + need + spare)
    ids = torch.randperm(F, generator=gen).tolist()
    P = max_pages or max(1, *held, *want)
    table, at = [], 0
    for h in held:
        table.append(ids[at:at + h] + [-7] * (P - h))
        at += h
    free = ids[at:at + need + spare]
    first = seed * 31 % F if start is None else start
    ring = [-3] * F
    for i, x in enumerate(free):
        ring[(first + i) % F] = x
    return table, ring, [first, len(free)]


def qk_rope(x, weight, positions, inv_freq, eps, magnitude, interleaved):
    """Normed and rotated heads [T, H, 128] in FP64."""
    x = x.cpu().double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.cpu().double()
    if inv_freq is None or inv_freq.numel() == 0:
        return x
    half = inv_freq.numel()
    angle = (positions.cpu().double()[:, None] * inv_freq.cpu().double())[:, None]
    y = x.clone()
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    y[..., a] = magnitude * (x[..., a] * angle.cos() - x[..., b] * angle.sin())
    y[..., b] = magnitude * (x[..., b] * angle.cos() + x[..., a] * angle.sin())
    return y


def prefix_inputs(first, prefix, lens, Hkv, page_size, *, seed, extra_pages=3, max_pages=None, combined=False, copies=False,
                  device="cuda"):
    """A paged cache whose rows first[g] .. first[g + 1] - 1 hold the same first prefix[g] tokens: in the same pages as
    far as those are whole (all of them copies where `copies`), then each row's own; NaN in every slot that no row owns."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-n // page_size) for n in lens]
    P = max(1, *need) if max_pages is None else max_pages
    order = torch.randperm(sum(need) + extra_pages, generator=gen).to(torch.int32)
    table = torch.full((len(lens), P), -1, dtype=torch.int32)
    kv = torch.full((sum(need) + extra_pages, 2, Hkv, page_size, D), math.nan, dtype=torch.bfloat16)
    at = 0
    for g in range(len(prefix)):
        leader = None
        for b in range(first[g], first[g + 1]):
            n, p = lens[b], prefix[g]
            data = torch.randn(2, Hkv, n, D, generator=gen).to(torch.bfloat16)
            # rows that hold the whole prefix share it; a shorter row has tokens of its own
            same = p if leader is not None and n >= p else 0
            for i in range(need[b]):
                lo, hi = i * page_size, min(n, (i + 1) * page_size)
                if same >= (i + 1) * page_size and not copies:
                    table[b, i] = table[leader, i]
                    continue
                page = order[at]
                at += 1
                table[b, i] = page
                kv[page, :, :, :hi - lo] = data[:, :, lo:hi]
                m = min(same, hi) - lo
                if m > 0:
                    kv[page, :, :, :m] = kv[table[leader, i].long(), :, :, :m]
            if leader is None and n >= p:
                leader = b
    kv = kv.to(device)
    k, v = kv[:, 0], kv[:, 1]
    if not combined:
        k, v = k.contiguous(), v.contiguous()
    i32 = dict(dtype=torch.int32, device=device)
    return dict(k_cache=k, v_cache=v, block_table=table.to(device), seq_lens=torch.tensor(lens, **i32),
                cu_groups=torch.tensor(first, **i32), prefix_lens=torch.tensor(prefix, **i32))
