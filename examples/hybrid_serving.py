"""A hybrid model served with the library: a KDA layer, a linear-attention layer with one decay a head, and a
full-attention layer over a paged key-value cache whose rows are cut to a budget as they grow.

    python examples/hybrid_serving.py [--batch 4] [--tokens 40] [--budget 96] [--check]

Random weights; it prints the sampled tokens' shapes and checks, when --check is given, every step of the three
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

    def __init__(self, width, heads, kv_heads, vocab, batch, prompt, new_tokens, page, budget, device, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=gen, device=device) / math.sqrt(shape[0])).to(torch.bfloat16)

        self.H, self.Hkv, self.dev, self.page, self.budget = heads, kv_heads, device, page, budget
        self.embed = weight(vocab, width) * math.sqrt(vocab)
        self.kda = {n: weight(width, heads * D) for n in ("q", "k", "v", "g")} | {"b": weight(width, heads), "o": weight(heads * D, width)}
        self.lin = {n: weight(width, heads * D) for n in ("q", "k", "v")} | {"g": weight(width, heads), "o": weight(heads * D, width)}
        self.att = {"q": weight(width, heads * D), "k": weight(width, kv_heads * D), "v": weight(width, kv_heads * D),
                    "o": weight(heads * D, width)}
        # one slot a row in each state pool; pages for the longest row
        self.slots = torch.arange(batch, dtype=torch.int32, device=device)
        pages = -(-(prompt + new_tokens) // page)
        self.cache = torch.zeros(batch * pages, 2, kv_heads, page, D, dtype=torch.bfloat16, device=device)
        self.table = torch.randperm(batch * pages, generator=gen, device=device).to(torch.int32).view(batch, pages)
        self.lens = torch.zeros(batch, dtype=torch.int32, device=device)
        self.weight = torch.zeros(batch, kv_heads, pages * page, device=device)
        self.attn_ws = K.attn_decode_workspace(batch, heads, kv_heads, pages, page, True, device)
        self.evictions = 0

    def split(self, x, w):
        return (x @ w).view(*x.shape[:-1], -1, D)

    def append(self, rows, k, v, at):
        """Writes keys and values [n, Hkv, 128] of batch rows `rows` at positions `at`."""
        page = self.table[rows, at // self.page].long()
        self.cache[page, 0, :, at % self.page] = k
        self.cache[page, 1, :, at % self.page] = v

    def attend(self, x):
        q = self.split(x, self.att["q"])
        return K.attn_decode(q, self.cache[:, 0], self.cache[:, 1], self.table, self.lens, scale=SCALE,
                             weight=self.weight, workspace=self.attn_ws)

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
        rows = torch.repeat_interleave(torch.arange(N, device=self.dev), lens.long())
        self.append(rows, self.split(x, self.att["k"]), self.split(x, self.att["v"]),
                    torch.arange(T, device=self.dev) - cu_seqlens[:-1][rows])
        self.lens.copy_(lens)
        last = x[(cu_seqlens[1:] - 1).long()]
        return self.logits(last, self.attend(last))

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
        self.append(self.slots.long(), self.split(x, self.att["k"]), self.split(x, self.att["v"]), self.lens.long())
        self.lens += 1
        out = self.logits(x, self.attend(x))
        if self.budget and int(self.lens.max()) > self.budget + self.budget // 4:
            # the heaviest tokens, the first four and the last quarter stay
            new_lens, _ = K.cache_evict(self.cache[:, 0], self.cache[:, 1], self.table, self.lens, self.weight,
                                        budget=self.budget, sink=4, recent=self.budget // 4)
            self.lens.copy_(new_lens)
            self.evictions += 1
        return out

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
        q = self.split(x[-1:], self.att["q"]).float().view(self.Hkv, -1, D)
        k, v = (self.split(x, self.att[n]).float().transpose(0, 1) for n in "kv")
        o = torch.softmax(SCALE * q @ k.transpose(-1, -2), -1) @ v
        return self.logits(x[-1:], o.view(1, self.H, D).to(torch.bfloat16))


def serve(batch=4, heads=8, kv_heads=2, width=256, vocab=512, new_tokens=40, budget=96, page=16, check=False, device="cuda"):
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(20, 150, (batch,), generator=gen).tolist()
    model = Hybrid(width, heads, kv_heads, vocab, batch, max(lens), new_tokens + 1, page, budget, device)
    prompts = [torch.randint(0, vocab, (n,), generator=gen).to(device) for n in lens]
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
    return dict(history=history, logits=logits, lens=model.lens.tolist(), evictions=model.evictions, worst=worst)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=40)
    ap.add_argument("--budget", type=int, default=96)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    r = serve(batch=a.batch, new_tokens=a.tokens, budget=a.budget, check=a.check)
    for b, h in enumerate(r["history"]):
        print(f"row {b}: {h.numel()} tokens, {r['lens'][b]} cached, last five {h[-5:].tolist()}")
    print(f"evictions: {r['evictions']}" + (f", largest logits error before them {r['worst']:.2e}" if a.check else ""))


if __name__ == "__main__":
    main()
