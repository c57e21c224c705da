"""Refusals of the page call for rows that share pages, on the host; pointers are integers that are never dereferenced."""
import pytest
import torch

import kda_recurrent_gb300 as K
from kda_recurrent_gb300 import build as kbuild

A = 0x10000
INVALID, UNSUPPORTED, MISALIGNED = K.KDA_ERR_INVALID_ARG, K.KDA_ERR_UNSUPPORTED, K.KDA_ERR_MISALIGNED


@pytest.mark.parametrize("over,want", [
    (dict(shared=A + 2), MISALIGNED), (dict(shared=None, bt=A + 2), MISALIGNED), (dict(bt=None), INVALID), (dict(nl=None), INVALID),
    (dict(ring=None), INVALID), (dict(F=0), INVALID), (dict(T=-1), INVALID), (dict(ps=24), UNSUPPORTED), (dict(F=1 << 30), UNSUPPORTED)])
def test_arguments(over, want):
    kbuild.build()
    a = dict(bt=A, sl=A, nl=A, shared=A, ol=A, ring=A, st=A, os=A, F=10, ps=16, B=2, P=4, cu=A, slots=A, pos=A, rows=A, T=5)
    a.update(over)
    assert K.load().kda_page_resize_ex(a["bt"], a["sl"], a["nl"], a["shared"], a["ol"], a["ring"], a["st"], a["os"], a["F"], a["ps"],
                                       a["B"], a["P"], a["cu"], a["slots"], a["pos"], a["rows"], a["T"], None) == want


def test_binding():
    i32 = dict(dtype=torch.int32)
    t, l, r, s = torch.zeros(2, 3, **i32), torch.zeros(2, **i32), torch.zeros(5, **i32), torch.zeros(2, **i32)
    for shared, error in ((l.long(), TypeError), (torch.zeros(3, **i32), ValueError), (torch.zeros(4, **i32)[::2], ValueError), (3, TypeError),
                          (l, ValueError)):  # (the last: not on a GPU)
        with pytest.raises(error):
            K.kda_page_resize(t, l, l, r, s, 8, l, s, shared_pages=shared)
