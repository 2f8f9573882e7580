"""Query rows of a decode over a 4-bit pool do not depend on the magnitude of
the rows beside them: rows of ordinary size with a peaked softmax next to rows
of 1e12 to 1e30, which share a unit of eight rows in the own pass and, on pages
of few query rows, in the prefix pass.  Every row is held to the float64 oracle
within the bound that test_gpu_i4_decode derives (it grows with the row's own
norm, not with its neighbours')."""
import numpy as np
import pytest

from oracle import tree_attention as ta
from tree_structured_shared_gb300 import workloads as wl

from test_gpu_i4_decode import cached, check, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def harness(padoc_lib):
    from tree_structured_shared_gb300 import harness as h
    return h


def page(P, own, q):
    return wl.DecodePage(P, [P] * len(own), own, q, [[-1] + list(range(n - 1)) for n in q])


# the own pass alone; a page of 8 rows a kv head; one of many; a long prefix of few rows, its results merged apart
PAGES = {"own": page(0, [300, 17], [4, 4]), "few": page(333, [40, 5], [2, 2]), "many": page(333, [40, 5, 0], [4, 7, 16]),
         "merged": page(3000, [20, 0], [2, 2])}


@pytest.mark.parametrize("big", [1e12, 1e15, 1e30])
@pytest.mark.parametrize("name", sorted(PAGES))
@pytest.mark.parametrize("by", ["head", "token"])
def test_a_huge_row_beside_others(harness, big, name, by):
    w = wl.DecodeWorkload("f", [PAGES[name]], 4, 2, 128, 1.0)
    vals = wl.decode_values(w, 3)
    tok, head = np.arange(w.n_queries)[:, None, None], np.arange(4)[None, :, None]
    vals.q = wl.round_bf16(vals.q * np.where((head if by == "head" else tok) % 2 == 0, big, 4.0).astype(np.float32))
    o, lse, _ = run(harness, w, vals)
    c = cached(vals)
    O, L = ta.branch_decode(w, c)
    check(o, lse, O, L, c, what=f"{name} {big} {by}")
