"""A page moved to another pool: its rows gathered and appended there.

A bf16 pool gives back what it was given, so a 4-bit pool filled from it holds
the bytes that the rows themselves would have left.  What a 4-bit pool gives
back quantises to itself: a group's largest code is 7 (its scale is a seventh of
the largest magnitude, to within 1 part in 16, so that magnitude rounds to
code 7), hence the same scale and the same codes."""
import pytest

from tree_structured_shared_gb300 import padoc

from test_gpu_kv_rows import make_pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("src,dst", [(padoc.BF16, padoc.I4), (padoc.I4, padoc.I4), (padoc.I4, padoc.BF16)])
@pytest.mark.parametrize("n", [1, 333])
def test_move(padoc_lib, src, dst, n):
    import torch
    Hkv = 2
    torch.manual_seed(n)
    k, v = (torch.randn(n, Hkv, 128, device="cuda").to(torch.bfloat16) for _ in range(2))

    def filled(dtype, k, v):
        """A pool's storage with the rows appended, and the rows read back."""
        pool, kp, vp = make_pool(torch, 40, Hkv, dtype)
        s = pool.alloc(0)
        pool.append(s, k, v, n)
        rows = padoc.KVRows(pool, [s], [0], [0, n])
        rows.upload()
        back = [torch.empty_like(k), torch.empty_like(v)]
        rows.gather(*back)
        torch.cuda.synchronize()
        return (kp, vp), back

    _, first = filled(src, k, v)
    storage, second = filled(dst, *first)
    direct, want = filled(dst, k, v)
    if src == padoc.BF16:
        assert torch.equal(first[0], k) and torch.equal(first[1], v)
    if dst == padoc.I4:
        assert all(torch.equal(a, b) for a, b in zip(storage, direct))
    else:
        want = first
    assert torch.equal(second[0], want[0]) and torch.equal(second[1], want[1])
