"""A hybrid model served with the library: a KDA layer, a linear-attention layer with one decay a head, and a
full-attention layer over a paged key-value cache whose rows are cut to a budget as they grow, or share the pages of
a common beginning of their prompts.

    python examples/hybrid_serving.py [--batch 4] [--tokens 40] [--budget 96] [--prefix 0] [--check]

The cache's pages come from one ring of free ones as rows grow and go back to it as they are cut; queries and keys are
normed and rotated on their way, and keys and values written into the pages, by one call. Random weights; it prints the sampled tokens' shapes and checks, when --check is given, every step of the three
layers against a plain forward pass over the whole history in FP32 (no eviction happens before the check's end).
The attention layer is the last one, so that a prompt needs its output at the last position only: the prompt's
keys and values are written to the cache, and the last token attends by the same call as every later token.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import kda_recurrent_gb300 as K  # noqa: E402

D = 128
SCALE = 1.0 / math.sqrt(D)


def unit(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().sum(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Hybrid:
    """Three layers of `heads` heads over a residual stream of `width` channels."""

    def __init__(self, width, heads, kv_heads, vocab, batch, prompt, new_tokens, page, budget, device, seed=0, prefix=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device=device) / math.sqrt(shape[0])).to(torch.bfloat16)

        self.H, self.Hkv, self.dev, self.page, self.budget = heads, kv_heads, device, page, budget
        self.embed = weight(vocab, width) * math.sqrt(vocab)
        self.kda = {n: weight(width, heads * D) for n in ("q", "k", "v", "g")} | {"b": weight(width, heads), "o": weight(heads * D, width)}
        self.lin = {n: weight(width, heads * D) for n in ("q", "k", "v")} | {"g": weight(width, heads), "o": weight(heads * D, width)}
        self.att = {"q": weight(width, heads * D), "k": weight(width, kv_heads * D), "v": weight(width, kv_heads * D),
                    "o": weight(heads * D, width)}
        self.q_norm, self.k_norm = ((1 + 0.1 * torch.randn(D, generator=gen, device=device)).to(torch.bfloat16) for _ in range(2))
        self.inv_freq, self.magnitude = K.rope_frequencies(D, device=device)
        # one slot a row in each state pool; pages for the longest row
        i32 = dict(dtype=torch.int32, device=device)
        self.slots = torch.arange(batch, **i32)
        pages = -(-(prompt + new_tokens) // page)
        self.cache = torch.zeros(batch * pages, 2, kv_heads, page, D, dtype=torch.bfloat16, device=device)
        self.free = torch.randperm(batch * pages, generator=gen, device=device).to(torch.int32)
        self.free_state = torch.tensor([0, batch * pages], **i32)
        self.table = torch.full((batch, pages), -1, **i32)
        self.lens = torch.zeros(batch, **i32)
        self.positions = torch.zeros(batch, **i32)  # of the rows' next tokens (rows that are cut are shorter than that)
        self.shared = prefix // page  # whole pages that all rows begin with
        self.groups = torch.tensor([0, batch], **i32)
        self.prefix_lens = torch.tensor([self.shared * page], **i32)
        self.weight = torch.zeros(batch, kv_heads, pages * page, device=device)
        self.attn_ws = K.attn_decode_workspace(batch, heads, kv_heads, pages, page, True, device)
        self.evictions = 0

    def split(self, x, w):
        return (x @ w).view(*x.shape[:-1], -1, D)

    def resize(self, new_lens, max_tokens):
        """Pages for rows of `new_lens` tokens (or back from them); the new tokens' cache slots, positions and rows."""
        _, slots, positions, rows = K.page_resize(self.table, self.lens, new_lens, self.free, self.free_state, self.page,
                                                  max_tokens=max_tokens)
        return slots, positions, rows

    def append(self, x, positions, slots):
        """Normed and rotated queries of tokens x; their keys and values go to the cache's slots."""
        w = self.att
        return K.qk_norm_rope(self.split(x, w["q"]), self.split(x, w["k"]), positions, self.inv_freq, q_weight=self.q_norm,
                              k_weight=self.k_norm, magnitude=self.magnitude, v=self.split(x, w["v"]), k_cache=self.cache[:, 0],
                              v_cache=self.cache[:, 1], slots=slots)

    def attend(self, q):
        cache = self.cache[:, 0], self.cache[:, 1], self.table, self.lens
        if self.shared:
            return K.attn_prefix_decode(q, *cache, self.groups, self.prefix_lens, scale=SCALE)
        return K.attn_decode(q, *cache, scale=SCALE, weight=self.weight, workspace=self.attn_ws)

    def prefill(self, tokens, cu_seqlens):
        """Packed prompts [T]; returns the logits of each row's last token."""
        T, N = tokens.shape[0], cu_seqlens.shape[0] - 1
        x = self.embed[tokens]
        w = self.kda
        ws = K.prefill_workspace(N, T, self.H, self.dev)
        o, self.kda_state = K.prefill(unit(self.split(x, w["q"])), unit(self.split(x, w["k"])), self.split(x, w["v"]),
                                      self.split(x, w["g"]), torch.sigmoid((x @ w["b"]).float()), cu_seqlens, scale=SCALE,
                                      lower_bound=-5.0, workspace=ws)
        x = x + o.flatten(1) @ w["o"]
        w = self.lin
        ws = K.linear_prefill_workspace(N, T, self.H, self.dev)
        o, self.lin_state = K.linear_prefill(unit(self.split(x, w["q"])), unit(self.split(x, w["k"])),
                                             self.split(x, w["v"]), self.decay(x), cu_seqlens, scale=SCALE, workspace=ws)
        x = x + o.flatten(1) @ w["o"]
        lens = cu_seqlens[1:] - cu_seqlens[:-1]
        position = torch.arange(T, dtype=torch.int32, device=self.dev) - torch.repeat_interleave(cu_seqlens[:-1], lens)
        slot = torch.full((T,), -1, dtype=torch.int64, device=self.dev)

        def place(new_lens):
            slots, at, rows = self.resize(new_lens, T)
            new = rows >= 0
            slot[(cu_seqlens[rows[new].long()] + at[new]).long()] = slots[new]

        if self.shared:  # the first row's pages, which the others begin with
            place(torch.where(torch.arange(N, device=self.dev) == 0, lens, 0))
            self.table[1:, :self.shared] = self.table[0, :self.shared]
            self.lens[1:] = self.shared * self.page
        place(lens)
        self.positions.copy_(lens)
        last = (cu_seqlens[1:] - 1).long()
        return self.logits(x[last], self.attend(self.append(x, position, slot)[last]))

    def decay(self, x):
        return -torch.nn.functional.softplus((x @ self.lin["g"]).float()) / 16

    def logits(self, x, o):
        return ((x + o.flatten(1) @ self.att["o"]) @ self.embed.T).float()

    def step(self, tokens):
        """One token a row; returns its logits."""
        x = self.embed[tokens]
        w = self.kda
        o = K.decode(unit(self.split(x, w["q"])), unit(self.split(x, w["k"])), self.split(x, w["v"]),
                     self.split(x, w["g"]), torch.sigmoid((x @ w["b"]).float()), self.slots, self.kda_state, scale=SCALE,
                     lower_bound=-5.0)
        x = x + o.flatten(1) @ w["o"]
        w = self.lin
        o = K.linear_decode(unit(self.split(x, w["q"])), unit(self.split(x, w["k"])), self.split(x, w["v"]), self.decay(x),
                            self.slots, self.lin_state, scale=SCALE)
        x = x + o.flatten(1) @ w["o"]
        slots, _, _ = self.resize(self.lens + 1, x.shape[0])
        q = self.append(x, self.positions, slots)
        self.positions += 1
        out = self.logits(x, self.attend(q))
        if self.budget and int(self.lens.max()) > self.budget + self.budget // 4:
            # the heaviest tokens, the first four and the last quarter stay
            new_lens, _ = K.cache_evict(self.cache[:, 0], self.cache[:, 1], self.table, self.lens, self.weight,
                                        budget=self.budget, sink=4, recent=self.budget // 4)
            self.resize(new_lens, 0)  # the pages behind the kept tokens go back
            self.evictions += 1
        return out

    def turned(self, x, weight):
        """Heads [T, H, 128] of positions 0 .. T - 1, normed and rotated."""
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
        angle = (torch.arange(x.shape[0], dtype=torch.float64, device=self.dev)[:, None] * self.inv_freq.double())[:, None]
        a, b, cos, sin = *x.chunk(2, -1), angle.cos().float(), angle.sin().float()
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16).float()

    def plain(self, tokens):
        """The same model over one row's whole history [T], in FP32 and token by token: logits of the last."""
        x = self.embed[tokens]
        for w, kind in ((self.kda, "kda"), (self.lin, "lin")):
            q, k, v = unit(self.split(x, w["q"])).float(), unit(self.split(x, w["k"])).float(), self.split(x, w["v"]).float()
            S = torch.zeros(self.H, D, D, device=self.dev)
            o = torch.empty_like(q)
            for t in range(x.shape[0]):
                if kind == "kda":
                    S = S * torch.exp(-5.0 * torch.sigmoid(self.split(x, w["g"])[t].float()))[..., None]
                    beta = torch.sigmoid((x @ w["b"])[t].float())[:, None, None]
                    S = S + beta * k[t][..., None] * (v[t] - torch.einsum("hi,hij->hj", k[t], S))[:, None]
                else:
                    S = S * torch.exp(self.decay(x)[t])[:, None, None] + k[t][..., None] * v[t][:, None]
                o[t] = SCALE * torch.einsum("hi,hij->hj", q[t], S)
            x = x + o.to(torch.bfloat16).flatten(1) @ w["o"]
        q = self.turned(self.split(x, self.att["q"]), self.q_norm)[-1].view(self.Hkv, -1, D)
        k = self.turned(self.split(x, self.att["k"]), self.k_norm).transpose(0, 1)
        v = self.split(x, self.att["v"]).float().transpose(0, 1)
        o = torch.softmax(SCALE * q @ k.transpose(-1, -2), -1) @ v
        return self.logits(x[-1:], o.view(1, self.H, D).to(torch.bfloat16))


def serve(batch=4, heads=8, kv_heads=2, width=256, vocab=512, new_tokens=40, budget=96, page=16, check=False, device="cuda",
          prefix=0):
    if prefix and budget:
        raise ValueError("rows that share pages are not cut to a budget")
    gen = torch.Generator().manual_seed(1)
    lens = [prefix + n for n in torch.randint(20, 150, (batch,), generator=gen).tolist()]
    model = Hybrid(width, heads, kv_heads, vocab, batch, max(lens), new_tokens + 1, page, budget, device, prefix=prefix)
    prompts = [torch.randint(0, vocab, (n,), generator=gen).to(device) for n in lens]
    for p in prompts:
        p[:prefix] = prompts[0][:prefix]
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32).to(device)
    logits = model.prefill(torch.cat(prompts), cu)
    worst, history = 0.0, prompts
    for _ in range(new_tokens):
        if check and not model.evictions:
            for b in range(batch):
                ref = model.plain(history[b])[0]
                worst = max(worst, float((logits[b] - ref).norm() / ref.norm()))
        token = logits.argmax(-1)
        history = [torch.cat([h, token[b:b + 1]]) for b, h in enumerate(history)]
        logits = model.step(token)
    status = K.kda_device_status()
    assert status[0] == K.KDA_OK, status
    return dict(history=history, logits=logits, lens=model.lens.tolist(), evictions=model.evictions, worst=worst,
                free=int(model.free_state[1]), table=model.table.cpu())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--prefix", type=int, default=0, help="tokens that all prompts begin with (then without a budget)")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    r = serve(batch=a.batch, new_tokens=a.tokens, budget=0 if a.prefix else a.budget, check=a.check, prefix=a.prefix)
    for b, h in enumerate(r["history"]):
        print(f"row {b}: {h.numel()} tokens, {r['lens'][b]} cached, last five {h[-5:].tolist()}")
    print(f"evictions: {r['evictions']}" + (f", largest logits error before them {r['worst']:.2e}" if a.check else ""))


if __name__ == "__main__":
    main()
