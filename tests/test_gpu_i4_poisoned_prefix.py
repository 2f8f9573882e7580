"""A prefix of a 4-bit pool of which a row sees poisoned tokens only, or sees
only poisoned ones among the keys that one unit or one tile of the kernels
takes: the rows that see such a token get NaN in O and LSE for the heads that
read its kv head, at few query rows a page and at many, and no other result
changes by a bit."""
import copy

import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def harness(padoc_lib):
    from tree_structured_shared_gb300 import harness as h
    return h


def run(harness, w, vals):
    import torch
    d = harness.Decode(w, vals, tree=False, dtype=padoc.I4)
    o, lse = d.run()
    torch.cuda.synchronize()
    padoc.device_status()
    n = w.n_queries
    return o.float().cpu().numpy()[:n], lse.cpu().numpy()[:n]


# branches of a page, query tokens of each: 8 and 80 query rows a kv head
ROWS = {8: (2, 2), 80: (10, 4)}
CASES = {
    # prefix length, poisoned tokens, forks (taken in turn by the branches)
    "one token": (1, [0], [1, 0]),
    "all of two tiles": (200, range(200), [200, 130, 128, 1, 0]),
    "the first tile": (200, range(128), [200, 128, 60]),
    "the first of four tiles": (500, range(128), [500, 128]),
    "the second tile": (256, range(128, 256), [256, 129, 128]),
    "last of many pieces": (3000, [2999], [3000, 2999]),
    "all of many pieces": (3000, range(3000), [3000, 1]),
}
CASES.update({f"at {k}": (2049, [k], [2049, k + 1, k]) for k in (128, 512, 1024, 1536, 2048)})


@pytest.mark.parametrize("rows", sorted(ROWS))
@pytest.mark.parametrize("case", sorted(CASES))
def test_poisoned_prefix(harness, rows, case):
    P, bad, forks = CASES[case]
    n, ql = ROWS[rows]
    forks = [forks[i % len(forks)] for i in range(n)]
    w = wl.DecodeWorkload("p", [wl.DecodePage(P, forks, [3 * i for i in range(n)], [ql] * n,
                                              [[-1] + list(range(ql - 1))] * n)], 4, 2, 128, 1.0)
    clean = wl.decode_values(w, P)
    o0, l0 = run(harness, w, clean)
    assert np.isfinite(o0).all() and np.isfinite(l0).all()
    vals = copy.deepcopy(clean)
    vals.prefix_k[0][list(bad), 1, 7] = np.nan
    o, lse = run(harness, w, vals)
    sees = np.repeat([any(t < f for t in bad) for f in forks], ql)
    hit = sees[:, None] & (np.arange(4) >= 2)[None]  # heads 2 and 3 read kv head 1
    assert np.isnan(lse[hit]).all() and np.isnan(o[hit]).all()
    assert np.array_equal(o[~hit], o0[~hit]) and np.array_equal(lse[~hit], l0[~hit])
