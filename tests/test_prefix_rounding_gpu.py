"""How far the rounded probabilities of a shared prefix may move an output, element by element, against 64 bits.

A probability is rounded to BF16 once (2^-8 of it at most); a score is an FP32 sum of 128 products, off by at most 128 x 2^-24 x
sum |q_i k_i| scale < 1.2e-4 for these inputs (that sum is below 15), which is the relative error of a probability and, once more,
of the sum that it is divided by; at most 200 additions a part and the join's add 200 x 2^-23. So before its own rounding an
output is off by at most (2^-8 + 2 x 1.2e-4 + 2.4e-5) sum_j p_j |v_j| < (2^-8 + 3e-4) sum_j p_j |v_j|, and the rounding adds 2^-8 of
what it rounds."""
import math

import pytest
import torch

import hybrid_reference as H
import kda_recurrent_gb300 as K
import serving_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)


@pytest.mark.parametrize("rows", [4, 40])  # 128 query rows of a key head at most, and more
@pytest.mark.parametrize("kind", ["independent", "far from zero", "cancelling", "equal keys", "one key", "one key in the rest"])
def test_each_output(kind, rows):
    page, prefix, Hq = 64, 1500, 8
    c = R.prefix_inputs([0, rows], [prefix], [prefix + 3 + i % 30 for i in range(rows)], 1, page, seed=rows, device=DEV)
    gen = torch.Generator().manual_seed(rows)
    q = torch.randn(1, Hq, 128, generator=gen).to(torch.bfloat16).expand(rows, Hq, 128).contiguous().to(DEV)
    k, v = c["k_cache"], c["v_cache"]
    shared = c["block_table"][0, :prefix // page].long()
    if kind == "far from zero":
        v.add_(100)
    elif kind == "cancelling":
        v[shared, :, 1::2] = -v[shared, :, 0::2]
    elif kind == "equal keys":  # after the first tile: the same probability, above the maximum that was fixed there
        k[shared[2:]] = (0.25 * q[0, 0]).to(torch.bfloat16)
    elif kind == "one key":
        k[shared[7], 0, 5] = (0.6 * q[0, 0].float()).to(torch.bfloat16)
    elif kind == "one key in the rest":
        k[c["block_table"][rows - 1, prefix // page].long(), 0, prefix % page] = (0.6 * q[0, 0].float()).to(torch.bfloat16)
    width = (48 << 20) // (512 * page * rows) + 1
    table = torch.full((rows, width), -1, dtype=torch.int32, device=DEV)
    table[:, :c["block_table"].shape[1]] = c["block_table"]
    out = K.attn_prefix_decode(q, k, v, table, c["seq_lens"], c["cu_groups"], c["prefix_lens"], scale=SCALE)
    plain = K.attn_decode(q, k, v, table, c["seq_lens"], scale=SCALE)
    ref, _, _ = H.attn_decode(q, c, SCALE)
    size, _, _ = H.attn_decode(q, dict(c, v_cache=v.abs()), SCALE)  # sum p |v|
    before = (2.0 ** -8 + 3e-4) * size
    err = (out.cpu().double() - ref).abs()
    assert (err <= before + 2.0 ** -8 * (ref.abs() + before)).all(), (err / size).max()
    before = 3e-4 * size + 2.0 ** -16 * size  # both terms of the probabilities
    err = (plain.cpu().double() - ref).abs()
    assert (err <= before + 2.0 ** -8 * (ref.abs() + before)).all(), (err / size).max()
    assert K.kda_device_status()[0] == K.KDA_OK
