"""8-bit checkpoints on the GPU, and the attention's gradients from them, against 64 bits."""
import numpy as np
import pytest

from oracle import tree_backward as tb
from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

from parity import check_grad

pytestmark = pytest.mark.gpu


def kept_ref(x):
    """Codes [n, width] and scale bytes [n, width / 32] of bf16 values given in float64."""
    g = x.reshape(x.shape[0], x.shape[1] // 32, 32)
    a = np.abs(g).max(-1)
    bad = ~np.isfinite(a)
    e = np.ones(a.shape, np.int64)
    for b in range(1, 255):  # the first scale of which 127 reach a
        e = np.where((127.0 * 2.0 ** (b - 1 - 127) < a) & (e == b - 1 if b > 1 else True), b, e)
    e = np.minimum(e, 248)  # 64 steps of the next scale are no bf16 number
    s = 2.0 ** (e - 127.0)
    with np.errstate(invalid="ignore"):
        code = np.rint(g / s[..., None])  # ties to even
    code = np.where(bad[..., None], 0, np.clip(code, -127, 127)).astype(np.int8)
    return code.reshape(x.shape), np.where(bad, 255, e).astype(np.uint8)


def value_ref(code, e):
    s = np.where(e == 255, np.nan, 2.0 ** (e.astype(np.float64) - 127))
    return (code.reshape(code.shape[0], code.shape[1] // 32, 32) * s[..., None]).reshape(code.shape)


def rows(n, width, seed, pad=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(n, width + pad, generator=g, device="cuda")
    x = x * torch.exp2(torch.randint(-20, 20, (n, 1), generator=g, device="cuda").float())
    return x.to(torch.bfloat16)[:, :width]


def buf(x):
    import torch
    return torch.full((padoc.act_bytes(*x.shape) + 64,), 0xA5, dtype=torch.uint8, device="cuda")


def check_one(x, kept, back):
    n, width = x.shape
    by = kept.cpu().numpy()
    code, e = kept_ref(x.double().cpu().numpy())
    assert np.array_equal(by[: n * width].view(np.int8).reshape(n, width), code)
    assert np.array_equal(by[n * width: n * width + e.size].reshape(e.shape), e)
    assert (by[n * width + e.size:] == 0xA5).all()
    want = value_ref(code, e)
    assert np.array_equal(back.double().cpu().numpy(), want, equal_nan=True)
    fine = np.isfinite(want)
    half = np.repeat(2.0 ** (e.astype(np.float64) - 128), 32, -1)  # the largest bf16 is half a step above 127 of its scale
    assert (np.abs(want - x.double().cpu().numpy())[fine] <= half[fine]).all()


@pytest.mark.parametrize("n,width", [(1, 32), (3, 96), (17, 64), (462, 512), (1000, 160), (5, 2048), (513, 32)])
@pytest.mark.parametrize("pad", [0, 40])
def test_there_and_back(padoc_lib, n, width, pad):
    import torch
    x = rows(n, width, n, pad)
    kept = buf(x)
    back = torch.full((n, width + pad), 3.0, dtype=torch.bfloat16, device="cuda")
    padoc.act_keep([x], [kept])
    padoc.act_restore([kept], [back[:, :width]])
    check_one(x, kept, back[:, :width])
    assert bool((back[:, width:] == 3).all())


def test_long_tensors(padoc_lib):
    """More than the GPU takes in one round of CTAs, and a short one behind."""
    import torch
    x = [rows(10007, 2080, 1, 16), rows(11, 64, 2)]
    kept, back = [buf(v) for v in x], [torch.empty(v.shape, dtype=v.dtype, device="cuda") for v in x]
    padoc.act_keep(x, kept)
    padoc.act_restore(kept, back)
    for v, b, r in zip(x, kept, back):
        check_one(v, b, r)


def test_special_values(padoc_lib):
    import torch
    x = torch.zeros(64, 64, dtype=torch.bfloat16, device="cuda")
    bits = torch.arange(64 * 64, device="cuda").view(64, 64) * 16 + 5   # values of every size, signs by halves
    x[:] = (bits % 65536).to(torch.int32).to(torch.int16).view(torch.bfloat16)
    x[0] = 0
    x[1, 3] = float("inf")
    x[2, 40] = float("nan")
    x[3] = 2.0 ** -133           # below the smallest scale
    x[4, :32] = torch.finfo(torch.bfloat16).max
    x[5, :32] = 127.0            # exactly 127 steps of 1
    x[6, :32] = 127.5            # a step above
    x[7, :32] = -0.0
    x[8, :16], x[8, 16:32] = 2.5, 127.0   # ties
    kept, back = buf(x), torch.empty_like(x)
    padoc.act_keep([x], [kept])
    padoc.act_restore([kept], [back])
    check_one(x, kept, back)
    assert bool(back[1, :32].isnan().all()) and bool((back[1, 32:] == back[1, 32:]).all())


def test_eight_tensors_and_empty_ones(padoc_lib):
    import torch
    shapes = [(0, 64), (37, 64), (1, 32), (0, 32), (900, 128), (2, 4096), (64, 96), (0, 64)]
    x = [rows(*s, i) for i, s in enumerate(shapes)]
    kept, back = [buf(v) for v in x], [torch.empty(v.shape, dtype=v.dtype, device="cuda") for v in x]
    padoc.act_keep(x, kept)
    padoc.act_restore(kept, back)
    for v, b, r in zip(x, kept, back):
        check_one(v, b, r)
    padoc.act_keep([], [])


def test_slices_of_one_projection(padoc_lib):
    import torch
    x = rows(300, 512, 1)
    parts = list(x.split([256, 128, 128], -1))
    kept = [buf(p) for p in parts]
    out = torch.zeros_like(x)
    padoc.act_keep(parts, kept)
    padoc.act_restore(kept, list(out.split([256, 128, 128], -1)))
    for p, b, r in zip(parts, kept, out.split([256, 128, 128], -1)):
        check_one(p, b, r)


def test_captured_on_another_stream(padoc_lib):
    import torch
    x = rows(100, 256, 1)
    kept, back = buf(x), torch.empty(100, 256, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        padoc.act_keep([x], [kept])
        padoc.act_restore([kept], [back])
    for seed in (2, 3):
        x.copy_(rows(100, 256, seed))
        g.replay()
        check_one(x, kept, back)


# ------------------------------------------------------------------ the attention's gradients


def kept_workload(w, seed, order=padoc.PACK_CANONICAL):
    """Checkpoints of a workload's q, k, v and of the o and lse that the forward
    gives for what they stand for, with those values in 64 bits."""
    import torch
    from tree_structured_shared_gb300 import harness
    T = w.n_tokens
    vals = wl.tree_qkv(w, seed)
    dev = [torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16).flatten(1) for x in vals]
    kept = [buf(x) for x in dev]
    padoc.act_keep(dev, kept)
    padoc.act_restore(kept, dev)
    q, k, v = (x.view(T, -1, w.d).float().cpu().numpy() for x in dev)
    return q, k, v, kept


def gradients(w, kept, o, lse, d_o, order):
    import torch
    T = w.n_tokens
    desc = padoc.TreeDesc(w.pages, order)
    grads = [torch.full((T, H, w.d), float("nan"), dtype=torch.bfloat16, device="cuda") for H in (w.Hq, w.Hkv, w.Hkv)]
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(desc, w.Hq, w.Hkv, w.d)
    ws = torch.full((size + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    o_kept = buf(o)
    padoc.act_keep([o], [o_kept])
    padoc.tree_attn_varlen_bwd_kept(desc, *kept, o_kept, lse, d_o, *grads, w.Hq, w.Hkv, w.d, ws, size)
    torch.cuda.synchronize()
    padoc.device_status()
    assert bool((ws[size:] == 0x5A).all())
    back = torch.empty_like(o)
    padoc.act_restore([o_kept], [back])
    return grads, back


@pytest.mark.parametrize("order", [padoc.PACK_CANONICAL, padoc.PACK_DOCUMENT])
@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_gradients_are_those_of_the_values(padoc_lib, G, order):
    """The backward of the values that the checkpoints stand for, up to the order of
    additions (row sums; dk and dv where a key tile's queries are cut into parts); and
    dv, which o does not enter, near the oracle's."""
    import torch
    from tree_structured_shared_gb300 import harness
    w = wl.random_pages(80 + G, n_pages=3, max_prefix=300, max_regions=5, max_layout=20, max_content=150,
                        Hq=2 * G, Hkv=2, d=128, dtype="bf16")
    T = w.n_tokens
    q, k, v, kept = kept_workload(w, G, order)
    f = harness.Forward(w, q, k, v, order)
    f.run()
    d_o = wl.round_bf16(wl.normal_f32(G + 5, (T, w.Hq, w.d), w.value_scale))
    b = harness.Backward(f, d_o)
    o = f.o.flatten(1)[:T]
    grads, o_back = gradients(w, kept, o, f.lse, b.d_o, order)
    f.o[:T] = o_back.view(T, w.Hq, w.d)  # the plain backward on the same values
    want = b.run()
    torch.cuda.synchronize()
    for g, r, name in zip(grads, want, ("dq", "dk", "dv")):
        check_grad(g.float().cpu().numpy(), r[:T].float().cpu().numpy(), "bf16", name)
    ref = tb.tree_backward(q, k, v, d_o, w.pages, order)
    check_grad(grads[2].float().cpu().numpy(), ref[2], "bf16", "dv")


@pytest.mark.parametrize("prefix", [900, 2700])
def test_many_key_tiles(padoc_lib, prefix):
    """Enough of them that no key tile's queries are cut: dv, which the row sums do not
    enter, is bit for bit that of the plain backward."""
    import torch
    from tree_structured_shared_gb300 import harness
    w = wl.TreeWorkload("pages", [wl.Page(prefix, [12] * 5, [130, 7, 64, 200, 1]), wl.Page(640, [], []), wl.Page(0, [3], [90])],
                        16, 8, 128, "bf16", 1.0, [0, 0, 0])
    T = w.n_tokens
    assert -(-T // 128) * 8 > 76
    q, k, v, kept = kept_workload(w, 2)
    f = harness.Forward(w, q, k, v)
    f.run()
    b = harness.Backward(f, wl.round_bf16(wl.normal_f32(5, (T, 16, 128), 1.0)))
    o = f.o.flatten(1)[:T]
    grads, o_back = gradients(w, kept, o, f.lse, b.d_o, padoc.PACK_CANONICAL)
    f.o[:T] = o_back.view(T, 16, 128)
    want = b.run()
    torch.cuda.synchronize()
    assert torch.equal(grads[2], want[2][:T])
    for g, r, name in zip(grads, want, ("dq", "dk", "dv")):
        check_grad(g.float().cpu().numpy(), r[:T].float().cpu().numpy(), "bf16", name)


def test_parts_repeat_bit_for_bit_and_in_a_graph(padoc_lib):
    import torch
    from tree_structured_shared_gb300 import harness
    w = wl.random_pages(5, n_pages=2, max_prefix=500, max_regions=5, max_layout=20, max_content=150, Hq=4, Hkv=1,
                        d=128, dtype="bf16")
    T = w.n_tokens
    q, k, v, kept = kept_workload(w, 1)
    f = harness.Forward(w, q, k, v)
    f.run()
    o_kept = buf(f.o.flatten(1)[:T])
    padoc.act_keep([f.o.flatten(1)[:T]], [o_kept])
    d_o = torch.randn(T, 4, 128, device="cuda").to(torch.bfloat16)
    grads = [torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda") for H in (4, 1, 1)]
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(f.desc, 4, 1, 128)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    run = lambda: padoc.tree_attn_varlen_bwd_kept(f.desc, *kept, o_kept, f.lse, d_o, *grads, 4, 1, 128, ws, size)  # noqa: E731
    run()
    torch.cuda.synchronize()
    first = [g.clone() for g in grads]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(4):
        for x in grads:
            x.fill_(7)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        padoc.device_status()
        for x, y in zip(grads, first):
            assert torch.equal(x, y)


def dense_gradients(w, q, k, v, o, lse, d_o):
    """The formula in 64 bits: P = exp(s q.k - lse), dS = P (dO.v - dO.o)."""
    from oracle import tree_attention as ta
    import torch
    T, G = w.n_tokens, w.Hq // w.Hkv
    desc = padoc.TreeDesc(w.pages, padoc.PACK_CANONICAL)
    qs, kv = desc.segments()
    seen = np.zeros((T, T), bool)
    for q0, n, first, count in qs:
        for s in range(first, first + count):
            a, m, causal = kv[s]
            for t in range(q0, q0 + n):
                seen[t, a: min(a + m, t + 1) if causal else a + m] = True
    dq, dk, dv = np.zeros((T, w.Hq, w.d)), np.zeros((T, w.Hkv, w.d)), np.zeros((T, w.Hkv, w.d))
    sc = 1 / np.sqrt(w.d)
    for h in range(w.Hq):
        g = h // G
        p = np.where(seen, np.exp(np.minimum(q[:, h] @ k[:, g].T * sc - lse[h][:, None], 50)), 0)
        ds = p * (d_o[:, h] @ v[:, g].T - (d_o[:, h] * o[:, h]).sum(-1, keepdims=True))
        dq[:, h] = sc * ds @ k[:, g]
        dk[:, g] += sc * ds.T @ q[:, h]
        dv[:, g] += p.T @ d_o[:, h]
    return dq, dk, dv


@pytest.mark.parametrize("d,G", [(128, 2), (64, 4), (64, 1)])
def test_gradients_against_the_formula(padoc_lib, d, G):
    """Everything as the checkpoints hold it, o included."""
    import torch
    w = wl.random_pages(90 + G, n_pages=2, max_prefix=150, max_regions=4, max_layout=9, max_content=60, Hq=2 * G,
                        Hkv=2, d=d, dtype="bf16")
    T = w.n_tokens
    q, k, v, kept = kept_workload(w, 3)
    from oracle import tree_attention as ta
    O, L = ta.tree_forward(q, k, v, w.pages)
    lse = torch.from_numpy(np.ascontiguousarray(L, np.float32)).cuda()
    o = torch.from_numpy(np.ascontiguousarray(O, np.float32)).cuda().to(torch.bfloat16).flatten(1)
    d_o = torch.randn(T, w.Hq, d, device="cuda").to(torch.bfloat16)
    grads, back = gradients(w, kept, o, lse, d_o, padoc.PACK_CANONICAL)
    ref = dense_gradients(w, *(x.astype(np.float64) for x in (q, k, v)), back.double().cpu().numpy().reshape(T, w.Hq, d),
                          lse.double().cpu().numpy(), d_o.double().cpu().numpy())
    for g, r, name in zip(grads, ref, ("dq", "dk", "dv")):
        check_grad(g.float().cpu().numpy(), r, "bf16", name)


def test_a_training_step(padoc_lib):
    """Rotation, attention, checkpoints, loss, and all gradients back to the projected
    rows, as they follow one another; against the same step in torch with autograd in
    64 bits at the values that the checkpoints hold."""
    import torch
    w = wl.random_pages(123, n_pages=2, max_prefix=120, max_regions=4, max_layout=9, max_content=60, Hq=4, Hkv=2,
                        d=128, dtype="bf16")
    T, Hq, Hkv, d, V = w.n_tokens, 4, 2, 128, 1501
    desc = padoc.TreeDesc(w.pages)
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    qkv, wv = rand(T, (Hq + 2 * Hkv) * d), (rand(V, Hq * d) * 0.05)
    t = torch.randint(V, (T,), generator=g, device="cuda").to(torch.int32)
    t[: T // 2] = -100
    pos = (torch.arange(T, device="cuda") % 300).to(torch.int32)
    cs = torch.empty(512, d, device="cuda")
    padoc.rope_table(cs, 512, d, 1.0e6, kind=padoc.ROPE_RAMP, factor=4.0, context=128.0)
    rope = padoc.Rope(cs, d)
    q, k, v = (x.contiguous().view(T, -1, d) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], -1))
    s = qkv.stride(0)
    padoc.rope_apply(rope, T, d, qkv, q, Hq, qkv[:, Hq * d:], k, Hkv, positions=pos, q_stride=s, k_stride=s)
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device="cuda")
    # the step computes from what it keeps
    kept = [buf(x.flatten(1)) for x in (q, k, v, o)]
    padoc.act_keep([x.flatten(1) for x in (q, k, v)], kept[:3])
    padoc.act_restore(kept[:3], [x.flatten(1) for x in (q, k, v)])
    padoc.tree_attn_varlen(desc, q, k, v, o, lse, padoc.BF16, Hq, Hkv, d)
    padoc.act_keep([o.flatten(1)], kept[3:])
    head = padoc.LmLoss(o.flatten(1), wv, t)
    ws = torch.empty(head.ws_size(True), dtype=torch.uint8, device="cuda")
    loss, l2 = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    d_loss = torch.full((T,), 1.0 / (T - T // 2), device="cuda")
    head.forward(loss, l2, ws, ws.numel())
    d_o, dw = torch.empty_like(o), torch.empty_like(wv)
    head.backward(l2, d_loss, d_o, dw, ws, ws.numel())
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    ws2 = torch.empty(padoc.tree_attn_varlen_bwd_kept_ws_size(desc, Hq, Hkv, d), dtype=torch.uint8, device="cuda")
    padoc.tree_attn_varlen_bwd_kept(desc, *kept, lse, d_o, dq, dk, dv, Hq, Hkv, d, ws2, ws2.numel())
    padoc.rope_apply(rope, T, d, dq, dq, Hq, dk, dk, Hkv, positions=pos, backward=True)
    torch.cuda.synchronize()
    padoc.device_status()
    # 64 bits
    seen = torch.zeros(T, T, dtype=torch.bool)
    qs, kv = desc.segments()
    for q0, n, first, count in qs:
        for a, m, causal in kv[first: first + count]:
            for i in range(q0, q0 + n):
                seen[i, a: min(a + m, i + 1) if causal else a + m] = True
    Q, K, Vv = (x.double().cpu().requires_grad_() for x in (q, k, v))
    W = wv.double().cpu().requires_grad_()
    x = torch.einsum("thd,jhd->htj", Q, K.repeat_interleave(2, 1)) / d ** 0.5
    p = torch.softmax(x.masked_fill(~seen, -float("inf")), -1)
    O = torch.einsum("htj,jhd->thd", p, Vv.repeat_interleave(2, 1))
    rows = torch.arange(T // 2, T)
    ls = torch.nn.functional.cross_entropy(O.flatten(1)[rows] @ W.T, t.cpu().long()[rows], reduction="sum") / len(rows)
    ls.backward()
    # the loss: o in bf16 moves a logit by at most 2^-8 of sum |o||w|
    move = 2.0 ** -8 * float((O.flatten(1)[rows].abs() @ W.abs().T).detach().max())
    assert abs(float((loss.double().cpu() * d_loss.double().cpu()).sum() - ls.detach())) <= 2 * move
    assert float((dw.double().cpu() - W.grad).norm()) <= 0.02 * float(W.grad.norm())
    c, sn = (cs[pos.long()].double().cpu()[:, None, i * 64: (i + 1) * 64] for i in range(2))
    turn = lambda z: torch.cat([z[..., :64] * c + z[..., 64:] * sn, z[..., 64:] * c - z[..., :64] * sn], -1)  # noqa: E731
    # o's 8 bits reach dq and dk through the row sums: an error of |dO.o| 2^-7 in a row that sums to zero; each of
    # the bf16 steps (d_o, P, dS, the gradients, the rotation) adds 2^-8 at most
    for name, a, b in (("dq", dq, turn(Q.grad)), ("dk", dk, turn(K.grad)), ("dv", dv, Vv.grad)):
        assert float((a.double().cpu() - b).norm()) <= 0.04 * float(b.norm()), name
