"""Rows that lie in a wider tensor, turned without a stride being given."""
import pytest

from tree_structured_shared_gb300 import padoc

from test_gpu_rope import table

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_projection_s_own_strides(padoc_lib, dtype):
    import torch
    n, Hq, Hkv, d = 57, 4, 2, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn(n, (Hq + 2 * Hkv) * d, generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    kind = padoc.BF16 if dtype == "bf16" else padoc.F32
    q, k = x[:, : Hq * d], x[:, Hq * d: (Hq + Hkv) * d]
    rope = padoc.Rope(table(n, d), d)
    dense, seen = ([torch.empty(n, H * d, dtype=x.dtype, device="cuda") for H in (Hq, Hkv)] for _ in range(2))
    padoc.rope_apply(rope, n, d, q.contiguous(), dense[0], Hq, k.contiguous(), dense[1], Hkv, dtype=kind)
    padoc.rope_apply(rope, n, d, q, seen[0], Hq, k, seen[1], Hkv, dtype=kind)
    assert torch.equal(dense[0], seen[0]) and torch.equal(dense[1], seen[1])
    rest = x[:, (Hq + Hkv) * d:].clone()
    padoc.rope_apply(rope, n, d, q, q, Hq, k, k, Hkv, dtype=kind)  # in place
    assert torch.equal(dense[0], q) and torch.equal(dense[1], k) and torch.equal(x[:, (Hq + Hkv) * d:], rest)
    padoc.rope_apply(rope, n, d, x, seen[0], Hq, dtype=kind)  # the head of each row
    padoc.rope_apply(rope, n, d, q, dense[0], Hq, dtype=kind)
    assert torch.equal(dense[0], seen[0])
