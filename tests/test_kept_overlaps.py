"""The kept backward refuses outputs and workspaces that lie on what it reads, or on each other.
No GPU: made-up addresses, and every refusal comes before any launch."""
import pytest

from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300.workloads import Page

HQ, HKV, D = 4, 2, 128


@pytest.fixture
def call(padoc_lib):
    desc = padoc.TreeDesc([Page(20, [3], [5])])
    T = desc.info()["n_tokens"]
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(desc, HQ, HKV, D)
    names = ("q", "k", "v", "o", "lse", "d_o", "dq", "dk", "dv", "ws")
    good = {name: (i + 1) << 40 for i, name in enumerate(names)}
    q, k = T * HQ * D, T * HKV * D
    sizes = dict(q=q + q // 32, k=k + k // 32, v=k + k // 32, o=q + q // 32, lse=4 * T * HQ, d_o=2 * q, dq=2 * q, dk=2 * k, dv=2 * k, ws=size)

    def run(**kw):
        a = dict(good, **kw)
        return padoc_lib.padoc_tree_attn_varlen_bwd_kept(desc.handle, *(a[n] for n in names[:9]), HQ, HKV, D, 0.0, a["ws"], size, None)

    run.good, run.sizes = good, sizes
    return run


OUT = ("dq", "dk", "dv", "ws")


@pytest.mark.parametrize("out,other", [(a, b) for a in OUT for b in ("q", "k", "v", "o", "lse", "d_o") + OUT if a != b])
def test_overlaps(call, out, other):
    step = 256 if "ws" in (out, other) else 16
    at = call.good[other]
    ends = [at, at + (call.sizes[other] - 1) // step * step, at - (call.sizes[out] - 1) // step * step]
    for place in ends:  # the same place, the other's last bytes, the other's first
        assert call(**{out: place}) == padoc.ERR_INVALID
        assert b"overlaps" in padoc.lib().padoc_last_error()
