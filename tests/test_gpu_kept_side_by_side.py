"""The kept backward on tensors that follow one another in one allocation, none refused and none
written outside its own."""
import pytest

from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


def test_side_by_side(padoc_lib):
    import torch
    desc = padoc.TreeDesc([wl.Page(200, [5, 6], [30, 21]), wl.Page(50, [], [])])
    T, Hq, Hkv, d = desc.info()["n_tokens"], 4, 2, 128
    assert T * Hkv * d // 32 % 16 == 0
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = [torch.randn(T, H * d, generator=g, device="cuda").bfloat16() for H in (Hq, Hkv, Hkv, Hq, Hq)]
    lse = torch.full((Hq, T), 4.0, device="cuda")
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(desc, Hq, Hkv, d)
    sizes = [padoc.act_bytes(T, H * d) for H in (Hq, Hkv, Hkv, Hq)] + [4 * T * Hq] + [2 * T * H * d for H in (Hq, Hq, Hkv, Hkv)]
    sizes.append(size + -sum(sizes) % 256)  # ws last: its start has to be 256-byte aligned
    buf = torch.full((sum(sizes) + 256,), 0x3C, dtype=torch.uint8, device="cuda")
    assert buf.data_ptr() % 256 == 0
    parts = list(buf.split(sizes + [256]))
    ws = parts[9][-sum(sizes[:9]) % 256:]
    apart = [torch.empty_like(p) for p in parts[:4]]
    padoc.act_keep(x[:4], parts[:4])
    padoc.act_keep(x[:4], apart)
    parts[4].view(torch.float32).copy_(lse.flatten())
    parts[5].view(torch.bfloat16).copy_(x[4].flatten())
    want = [torch.empty(T, H, d, dtype=torch.bfloat16, device="cuda") for H in (Hq, Hkv, Hkv)]
    ws2 = torch.empty(size, dtype=torch.uint8, device="cuda")
    padoc.tree_attn_varlen_bwd_kept(desc, *apart, lse, x[4], *want, Hq, Hkv, d, ws2, size)
    padoc.tree_attn_varlen_bwd_kept(desc, *parts[:9], Hq, Hkv, d, ws, size)
    torch.cuda.synchronize()
    padoc.device_status()
    for a, b in zip(parts[6:9], want):
        assert torch.equal(a, b.view(torch.uint8).flatten())
    for a, b in zip(parts[:4], apart):
        assert torch.equal(a, b)
    assert bool((parts[10] == 0x3C).all())
