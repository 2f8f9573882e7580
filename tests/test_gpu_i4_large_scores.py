"""Scores of any finite size over a 4-bit pool.

Keys are whole numbers in [-7, 7] with a 7 in every group, which the pool holds
exactly, and a query is a vector of signs times 2^e, so every score is an exact
f32 number.  Each query token has one key of seven times its own signs, whose
score, 896 * 2^e, is at least 560 * 2^e ahead of the others': with the softmax
scale 2^-3.5, 71 log2 units at e = 0, so what 3000 other keys add is below
2^-59 of a value, 2^-56 at most.  The output is then that key's value, as the
pool holds it (its own rounding to 16 bits is far finer than a bf16 step), and
the LSE the key's score.  The LSE goes through a handful of f32 roundings (scale, log2 e,
their product, the score, the reference, ln 2 and the products with it): 2^-20
of it covers sixteen."""
import numpy as np
import pytest

import i4ref
from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def harness(padoc_lib):
    from tree_structured_shared_gb300 import harness as h
    return h


# prefix, own keys and query tokens of each branch
PAGES = {"few rows": (333, [70, 200], [2, 2]), "many rows": (333, [70, 0, 200, 33], [5, 16, 3, 7]),
         "merged": (3000, [40], [4])}


@pytest.mark.parametrize("e", [0, 6, 12] + list(range(16, 34)) + [40, 60, 90, 110])
@pytest.mark.parametrize("name", sorted(PAGES))
def test_large_scores(harness, name, e):
    import torch
    P, own, ql = PAGES[name]
    w = wl.DecodeWorkload("l", [wl.DecodePage(P, [P] * len(own), own, ql, [[-1] + list(range(n - 1)) for n in ql])], 4, 2,
                          128, 1.0)
    vals = wl.decode_values(w, e)
    rng = np.random.default_rng(1000 + e)

    def keys(n):
        k = rng.integers(-2, 3, size=(n, 2, 128)).astype(np.float32)
        k[:, :, ::16] = 7.0 * rng.choice([-1, 1], size=(n, 2, 8))
        return k

    vals.prefix_k, vals.own_k, vals.k_new = [keys(P)], [keys(n) for n in own], keys(w.n_queries)
    signs = rng.choice([-1.0, 1.0], size=(w.n_queries, 2, 128)).astype(np.float32)
    vals.q = np.repeat(signs, 2, axis=1) * np.float32(2.0 ** e)
    want = np.zeros((w.n_queries, 4, 128))
    stored = [i4ref.stored(k, v)[1] for k, v in ((vals.prefix_k[0], vals.prefix_v[0]), *zip(vals.own_k, vals.own_v))]
    row = 0
    for b, n in enumerate(ql):
        for t in range(n):
            # where the token's key lies: in turn the prefix, the branch's own keys, the query block
            place = (b + t) % 3
            if place == 1 and own[b]:
                at = (7 * t + 3) % own[b]
                vals.own_k[b][at] = 7 * signs[row]
                v = stored[1 + b][at]
            elif place == 2:
                vals.k_new[row] = 7 * signs[row]
                v = vals.v_new[row]
            else:
                at = (41 * row + 5) % P
                vals.prefix_k[0][at] = 7 * signs[row]
                v = stored[0][at]
            want[row] = np.repeat(v, 2, axis=0)
            row += 1
    for b, r in enumerate(np.split(np.arange(w.n_queries), np.cumsum(ql)[:-1])):
        for i in r:
            others = np.concatenate([vals.prefix_k[0], vals.own_k[b], vals.k_new[r[0]: i + 1]])
            top = np.sort(np.einsum("khd,hd->hk", others, signs[i]), axis=1)
            assert (top[:, -1] == 896).all() and (top[:, -2] <= 336).all()
    d = harness.Decode(w, vals, tree=False, dtype=padoc.I4)
    o, lse = d.run()
    torch.cuda.synchronize()
    padoc.device_status()
    n = w.n_queries
    L = 896 * 2.0 ** e / 128 ** 0.5
    assert np.abs(o.double().cpu().numpy()[:n] - want).max() <= 2.0 ** -56
    assert np.abs(lse.double().cpu().numpy()[:n] - L).max() <= 2.0 ** -20 * L
