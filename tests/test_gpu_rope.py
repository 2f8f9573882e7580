"""Rotation of packed rows, its gradient and its tables on the GPU, against 64 bits.

A turned value is two products and a sum in f32, each off by half a step: within
1.5 * 2^-23 of |a c| + |b s|, and half a step of its own type when it is stored.  A
cosine or sine of a table is within 4 * 2^-24 of an amplitude: the remainder of the
angle rounded to f32 (pi 2^-25 at most), sincospif (two steps) and the amplitude."""
import math

import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc

pytestmark = pytest.mark.gpu


def table(n_pos, rot, seed=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    a = torch.rand(n_pos, rot // 2, generator=g, device="cuda") * 6.28
    return torch.cat([a.cos(), a.sin()], -1).contiguous()


def turned(x, w, rot, inter, back):
    """x [n, H, d] turned in 64 bits by rows w [n, rot], and the bound of the f32 steps."""
    import torch
    x, w = x.double(), w.double()[:, None]
    c, s = w[..., : rot // 2], w[..., rot // 2:]
    s = -s if back else s
    y, e = x.clone(), torch.zeros_like(x)
    sl = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., sl[0]], x[..., sl[1]]
    y[..., sl[0]], y[..., sl[1]] = a * c - b * s, b * c + a * s
    e[..., sl[0]] = 1.5 * 2.0 ** -23 * ((a * c).abs() + (b * s).abs())
    e[..., sl[1]] = 1.5 * 2.0 ** -23 * ((b * c).abs() + (a * s).abs())
    return y, e


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (128, 32), (128, 96), (64, 64), (64, 32), (128, 0)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("back", [False, True])
def test_rows(padoc_lib, dtype, d, rot, inter, back):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for n, Hq, Hkv in ((1, 1, 1), (7, 16, 8), (513, 5, 3), (97, 33, 0)):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        q = torch.randn(n, Hq, d, generator=g, device="cuda").to(dt)
        k = torch.randn(n, Hkv, d, generator=g, device="cuda").to(dt) if Hkv else None
        w = table(600, max(rot, 32))[:, :rot].contiguous() if rot else table(600, 32)
        pos = torch.randint(600, (n,), generator=g, device="cuda").to(torch.int32)
        qo = torch.full_like(q, 9.0)
        ko = torch.full_like(k, 9.0) if Hkv else None
        padoc.rope_apply(padoc.Rope(w, rot, inter), n, d, q, qo, Hq, k, ko, Hkv, positions=pos,
                         dtype=padoc.BF16 if dtype == "bf16" else padoc.F32, backward=back)
        for x, y in ((q, qo), (k, ko)):
            if x is None:
                continue
            ref, e = turned(x, w[pos.long()], rot, inter, back) if rot else (x.double(), 0.0)
            off = (y.double() - ref).abs()
            assert bool((off <= e + torch.finfo(dt).eps / 2 * (ref.abs() + e)).all()), (n, float(off.max()))


def test_in_place_in_a_fused_projection(padoc_lib):
    import torch
    n, Hq, Hkv, d = 301, 8, 2, 128
    x = torch.randn(n, (Hq + 2 * Hkv) * d, device="cuda").to(torch.bfloat16)
    was = x.clone()
    w = table(400, d)
    rope = padoc.Rope(w, d)
    q, k = x[:, : Hq * d], x[:, Hq * d: (Hq + Hkv) * d]
    s = x.stride(0)
    apart = torch.empty(n, Hq * d, dtype=x.dtype, device="cuda"), torch.empty(n, Hkv * d, dtype=x.dtype, device="cuda")
    padoc.rope_apply(rope, n, d, q, apart[0], Hq, k, apart[1], Hkv, q_stride=s, k_stride=s)
    padoc.rope_apply(rope, n, d, q, q, Hq, k, k, Hkv, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s)
    assert torch.equal(q, apart[0]) and torch.equal(k, apart[1])
    assert torch.equal(x[:, (Hq + Hkv) * d:], was[:, (Hq + Hkv) * d:])
    # and back: the rotation's transpose undoes it to the roundings of bf16, twice half a step of each pair's size
    padoc.rope_apply(rope, n, d, q, q, Hq, k, k, Hkv, q_stride=s, k_stride=s, q_out_stride=s, k_out_stride=s, backward=True)
    size = was.double().unflatten(-1, (-1, 2, d // 2)).norm(dim=-2, keepdim=True).expand(-1, -1, 2, -1).reshape(n, -1)
    assert bool(((x.double() - was.double()).abs() <= 3 * 2.0 ** -8 * size).all())


def test_positions_outside_the_table(padoc_lib):
    import torch
    n, d = 9, 128
    q = torch.randn(n, 2, d, device="cuda")
    pos = torch.tensor([0, -1, 49, 50, 2 ** 31 - 1, -2 ** 31, 3, 3, 4], dtype=torch.int32, device="cuda")
    out = torch.zeros_like(q)
    padoc.rope_apply(padoc.Rope(table(50, 64), 64), n, d, q, out, 2, positions=pos, dtype=padoc.F32)
    bad = torch.tensor([False, True, False, True, True, True, False, False, False], device="cuda")
    assert bool(out[bad][..., :64].isnan().all()) and torch.equal(out[bad][..., 64:], q[bad][..., 64:])
    assert bool(out[~bad].isfinite().all())


def test_same_bits_as_the_cache_write(padoc_lib):
    """Rows turned here and on their way into the cache."""
    import torch
    n, Hq, Hkv, d = 200, 4, 2, 128
    q, k, v = (torch.randn(n, H, d, device="cuda").to(torch.bfloat16) for H in (Hq, Hkv, Hkv))
    rope = padoc.Rope(table(300, d), d)
    pool_k, pool_v = (torch.zeros(20 * Hkv * 16 * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pool = padoc.KVPool(pool_k, pool_v, 20, Hkv, d, max_seqs=2, max_blocks_per_seq=20)
    pool.sync()
    a = pool.alloc(n)
    rows = padoc.KVRows(pool, [a], [0], [0, n])
    ws = torch.empty(max(rows.ws_size(), 16), dtype=torch.uint8, device="cuda")
    rows.upload(ws, ws.numel())
    q1, k1, q2, k2 = (torch.empty_like(x) for x in (q, k, q, k))
    rows.write(k, v, ws, rope=rope, q=q, Hq=Hq, q_rot=q1, k_rot=k1)
    padoc.rope_apply(rope, n, d, q, q2, Hq, k, k2, Hkv)
    assert torch.equal(q1, q2) and torch.equal(k1, k2)


def test_gradient_against_differences(padoc_lib):
    """<g, R(x + e u) - R(x - e u)> / 2e = <R'(g), u>: the map is linear, so e = 1 is as good as a small one."""
    import torch
    n, d = 50, 64
    rope = padoc.Rope(table(64, 32) * 1.3, 32, True)
    x, u, g = (torch.randn(n, 3, d, device="cuda") for _ in range(3))
    f = lambda y, back: (lambda o: (padoc.rope_apply(rope, n, d, y, o, 3, dtype=padoc.F32, backward=back), o)[1])(  # noqa: E731
        torch.empty_like(y))
    left = ((f(x + u, False).double() - f(x - u, False).double()) / 2 * g.double()).sum()
    right = (f(g, True).double() * u.double()).sum()
    size = float((g.double().abs() * (x.abs() + u.abs()).double() * 4).sum())
    assert abs(float(left - right)) <= 4 * 2.0 ** -23 * size


def frequencies(kind, base, rot, factor, context, lo_turns, hi_turns):
    """The definition, pair by pair."""
    out = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if kind == padoc.ROPE_BASE else base
        f = b ** (-2 * i / rot)
        if kind == padoc.ROPE_LINEAR:
            f /= factor
        if kind == padoc.ROPE_BANDS:
            w = min(1.0, max(0.0, (context * f / (2 * math.pi) - lo_turns) / (hi_turns - lo_turns)))
            f *= w + (1 - w) / factor
        if kind == padoc.ROPE_RAMP:
            at = lambda r: rot * math.log(context / (r * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
            a, z = max(math.floor(at(hi_turns)), 0), min(math.ceil(at(lo_turns)), rot - 1)
            w = 1 - min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            f *= w + (1 - w) / factor
        out.append(f)
    return np.array(out)


@pytest.mark.parametrize("kind", range(5))
@pytest.mark.parametrize("rot", [32, 64, 96, 128])
@pytest.mark.parametrize("n,first", [(1, 0), (1001, 0), (700, 2 ** 31 - 701), (5000, 131072)])
def test_tables(padoc_lib, kind, rot, n, first):
    import torch
    f = frequencies(kind, 5.0e5, rot, 8.0, 8192.0, 1.0, 32.0)
    out = torch.full((n + 2, rot), 9.0, device="cuda")
    padoc.rope_table(out, n, rot, 5.0e5, kind=kind, factor=8.0, context=8192.0, amplitude=1.25, first=first)
    assert bool((out[n:] == 9).all())
    # np.longdouble keeps the angles of far positions
    turns = np.arange(first, first + n, dtype=np.longdouble)[:, None] * (f.astype(np.longdouble) / (2 * np.longdouble(math.pi)))[None]
    ang = ((turns - np.rint(turns)) * 2 * np.longdouble(math.pi)).astype(np.float64)
    ref = 1.25 * np.concatenate([np.cos(ang), np.sin(ang)], -1)
    # a step's own rounding in 64 bits (pow, divisions: 8 half steps at most), times the position, is an angle
    drift = 8 * 2.0 ** -53 * (first + n) * np.concatenate([f, f])[None]
    off = np.abs(out[:n].double().cpu().numpy() - ref)
    assert (off <= 1.25 * (4 * 2.0 ** -24 + drift)).all(), off.max()


def test_captured(padoc_lib):
    import torch
    n, d = 40, 128
    q, out = torch.randn(n, 2, d, device="cuda"), torch.empty(n, 2, d, device="cuda")
    w = torch.empty(64, d, device="cuda")
    rope = padoc.Rope(w, d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        padoc.rope_table(w, 64, d, 1.0e4)
        padoc.rope_apply(rope, n, d, q, out, 2, dtype=padoc.F32)
    w.zero_()
    for seed in (1, 2):
        q.normal_()
        g.replay()
        ref, e = turned(q, w[:n], d, False, False)
        assert bool(((out.double() - ref).abs() <= e + 2.0 ** -24 * (ref.abs() + e)).all())


def test_many_rows(padoc_lib):
    """More rows than the launch has warps."""
    import torch
    n, d = 100003, 64
    q = torch.randn(n, 1, d, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    w = table(n, 64)
    padoc.rope_apply(padoc.Rope(w, 64), n, d, q, out, 1)
    ref, e = turned(q, w, 64, False, False)
    assert bool(((out.double() - ref).abs() <= e + 2.0 ** -8 * (ref.abs() + e)).all())
