"""A query row with an infinity over a 4-bit pool: every score of it is infinite
or NaN, so the softmax is NaN (of scores that are all -inf too, as where each
visible key is negative in that dim), and the rows beside it do not change."""
import copy

import numpy as np
import pytest

from test_gpu_i4_decode import harness, page, run  # noqa: F401
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

PAGES = {"query block alone": page(0, [0, 0], [0, 0], [3, 1]), "own": page(0, [0], [40], [2]),
         "few rows": page(70, [70, 1], [17, 0], [1, 2]), "many rows": page(300, [300, 128, 0], [9, 70, 0], [16, 5, 7]),
         "merged": page(3000, [3000, 2999], [5, 0], [2, 1])}


@pytest.mark.parametrize("inf", [np.inf, -np.inf])
@pytest.mark.parametrize("sign", [-1.0, 1.0, 0.0])
@pytest.mark.parametrize("name", sorted(PAGES))
def test_infinite_query(harness, name, sign, inf):  # noqa: F811
    w = wl.DecodeWorkload("q", [PAGES[name]], 4, 2, 128, 1.0)
    clean = wl.decode_values(w, 9)
    for ks in (clean.prefix_k, clean.own_k, [clean.k_new]):
        for k in ks:
            k[:, :, 5] = sign * (1.0 + (np.arange(len(k)) % 3)[:, None])
    o0, l0, _ = run(harness, w, clean)
    assert np.isfinite(o0).all() and np.isfinite(l0).all()
    vals = copy.deepcopy(clean)
    row, head = w.n_queries - 1, 2
    vals.q[row, head, 5] = inf
    o, lse, _ = run(harness, w, vals)
    hit = np.zeros((w.n_queries, 4), bool)
    hit[row, head] = True
    assert np.isnan(o[hit]).all() and np.isnan(lse[hit]).all()
    assert np.array_equal(o[~hit], o0[~hit]) and np.array_equal(lse[~hit], l0[~hit])
