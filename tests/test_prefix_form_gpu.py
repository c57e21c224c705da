"""Which of its two forms attention behind a prefix takes: that of kda_attn_decode, bit by bit, where the tables hold at most 48
MiB of keys and values (512 bytes a token, for each row, key head and 16 query heads of it), and whole tiles of shared
tokens computed together above. The latter rounds its probabilities to BF16 once where the former has two terms of them, so
that of the thousands of outputs of a call some differ in their last bit; both are within test_prefix_gpu.py's bounds of the 64-bit form."""
import math

import pytest
import torch

import hybrid_reference as H
import kda_recurrent_gb300 as K
import serving_reference as R
from helpers import assert_out_close

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1.0 / math.sqrt(128)
LIMIT = (48 << 20) // 512  # tokens of all tables


def both(rows, Hq, Hkv, prefix, page, table_tokens, seed):
    """Outputs of the call behind a prefix and of the plain one on the same tables, checked against 64 bits."""
    c = R.prefix_inputs([0, rows], [prefix], [prefix + 3 + i % 5 for i in range(rows)], Hkv, page, seed=seed, device=DEV)
    narrow = c["block_table"]
    table = torch.full((rows, table_tokens // page), -1, dtype=torch.int32, device=DEV)
    table[:, :narrow.shape[1]] = narrow
    q = torch.randn(rows, Hq, 128, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).to(DEV)
    cache = c["k_cache"], c["v_cache"], table, c["seq_lens"]
    out, lse = K.attn_prefix_decode(q, *cache, c["cu_groups"], c["prefix_lens"], scale=SCALE, want_lse=True)
    plain, plain_lse = K.attn_decode(q, *cache, scale=SCALE, want_lse=True)
    ref, ref_lse, _ = H.attn_decode(q, c, SCALE)
    for x, y in ((out, lse), (plain, plain_lse)):
        assert_out_close(x, ref)
        assert (y.cpu().double() - ref_lse).abs().max() <= 1.2e-4
    return torch.equal(out, plain), torch.equal(lse, plain_lse)


@pytest.mark.parametrize("rows,Hq,Hkv,page", [(3, 2, 2, 8), (7, 8, 8, 16), (5, 40, 2, 8), (2, 33, 1, 8), (16, 64, 8, 64), (12, 16, 1, 1024)])
def test_limit_of_few_tokens(rows, Hq, Hkv, page):
    items = rows * Hkv * -(-Hq // Hkv // 16)
    fits = LIMIT // items // page * page  # tokens of a table, whole pages
    assert items * fits <= LIMIT < items * (fits + page)
    assert both(rows, Hq, Hkv, 700, page, fits, rows) == (True, True)
    assert both(rows, Hq, Hkv, 700, page, fits + page, rows)[0] is False


@pytest.mark.parametrize("rows,Hq,Hkv,prefix,page", [(2, 1, 1, 2000, 64), (3, 4, 2, 256, 8), (9, 48, 1, 300, 16), (33, 8, 1, 700, 32), (40, 32, 8, 768, 16)])
def test_wide_tables_take_the_shared_form(rows, Hq, Hkv, prefix, page):
    # the shapes of test_prefix_gpu.py, and of the steps in test_serving_together_gpu.py, with the tables that those give them
    items = rows * Hkv * -(-Hq // Hkv // 16)
    tokens = -(-max((72 << 20) // 512 // items, prefix + 8) // page) * page
    assert items * tokens > LIMIT
    assert both(rows, Hq, Hkv, prefix, page, tokens, rows)[0] is False

