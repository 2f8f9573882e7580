"""Cross entropy of a large vocabulary and its gradient on the GPU, against the
definition in 64 bits.

Tolerances.  A logit is a sum of D products in f32, taken 16 at a time: at most
D / 16 + 2 additions that are each off by a step, 2^-23 of the running sum, which
is below S = max_v sum_k |h_k w_vk|.  lse is a weighted mean of such errors, and
its exponentials and sums add less than 2^-17.  G carries the relative error of its
exponential (that of the logit and of lse) and one rounding to bf16, 2^-8 (half of finfo.eps, 2^-7),
or, with 128 rows at most, the rounding of a second part, 2^-16; dh and dw one more of their own, and f32 sums.  Element by element these are bounds; by the
norm, where roundings do not all add up, each rounding counts 2^-8 at most."""
import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc

pytestmark = pytest.mark.gpu


def make(n, D, V, seed=0, masked=0.0, h_pad=0, w_pad=0):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = (torch.randn(V, D + w_pad, generator=g, device="cuda") * (2.0 / D ** 0.5)).to(torch.bfloat16)[:, :D]
    t = torch.randint(V, (n,), generator=g, device="cuda")
    h = torch.randn(n, D + h_pad, generator=g, device="cuda")
    h[:, :D] += w[t].float()
    h = h.to(torch.bfloat16)[:, :D]
    t[torch.rand(n, generator=g, device="cuda") < masked] = -1
    d = torch.rand(n, generator=g, device="cuda") + 0.1
    return h, w, t.to(torch.int32), d


def reference(h, w, t, d):
    """loss, lse, dh, dw in 64 bits, and the bounds of their errors."""
    import torch
    n, V = h.shape[0], w.shape[0]
    rows = torch.nonzero((t >= 0) & (t < V))[:, 0]
    D = h.shape[1]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")  # noqa: E731
    loss, lse, dh, dw = z(n), z(n), z(n, D), z(V, D)
    e_loss, e_dh, e_dw = z(n), z(n, D), z(V, D)
    W = w.double()
    for r in rows.split(4096):
        x = h[r].double()
        logits = x @ W.T
        ls = torch.logsumexp(logits, -1)
        tt = t[r].long()[:, None]
        lse[r], loss[r] = ls, ls - logits.gather(1, tt)[:, 0]
        e_logit = (D / 16 + 2) * 2.0 ** -23 * (x.abs() @ W.abs().T).amax(-1)
        e_loss[r] = 2 * e_logit + 2.0 ** -17 + 2.0 ** -22 * (ls.abs() + loss[r].abs())
        p = torch.exp(logits - ls[:, None])
        G = p.scatter_add(1, tt, -torch.ones_like(tt, dtype=torch.float64)) * d[r].double()[:, None]
        # the exponential's error is relative to p, the rounding's to G
        eG = G.abs() * 2.0 ** (-8 if len(rows) > 128 else -16) * 1.01 + p * d[r].double()[:, None] * (2 * e_logit + 2.0 ** -17)[:, None]
        dh[r] = G @ W
        dw += G.T @ x
        e_dh[r] = eG @ W.abs() + 2.0 ** -8 * dh[r].abs() + 2.0 ** -14 * (G.abs() @ W.abs())
        e_dw += eG.T @ x.abs() + 2.0 ** -14 * (G.abs().T @ x.abs())
    e_dw += 2.0 ** -8 * dw.abs()
    return (loss, lse, dh, dw), (e_loss, e_loss, e_dh + 1e-30, e_dw + 1e-30)


def launch(h, w, t, d, dh=True, dw=True, stream=None, reuse=None):
    import torch
    n, D, V = h.shape[0], h.shape[1], w.shape[0]
    nan = float("nan")
    head = padoc.LmLoss(h, w, t)
    ws = torch.full((head.ws_size(True),), 0xFF, dtype=torch.uint8, device="cuda") if reuse is None else reuse
    loss, lse = (torch.full((n,), nan, device="cuda") for _ in range(2))
    gh = torch.full((n, D), nan, dtype=torch.bfloat16, device="cuda") if dh else None
    gw = torch.full((V, D), nan, dtype=torch.bfloat16, device="cuda") if dw else None
    head.forward(loss, lse, ws, ws.numel(), stream)
    head.backward(lse, d, gh, gw, ws, ws.numel(), stream)
    return loss, lse, gh, gw


def check(got, ref, bound):
    import torch
    torch.cuda.synchronize()
    padoc.device_status()
    for name, g, r, e in zip(("loss", "lse", "dh", "dw"), got, ref, bound):
        if g is None:
            continue
        off = (g.double() - r).abs()
        assert bool((off <= e).all()), f"{name}: {float((off - e).max())} over, {float(off.max())} off"
        if name in ("dh", "dw") and float(r.norm()) > 0:
            assert float(off.norm()) <= 2 * 2.0 ** -8 * float(r.norm()), f"{name}: norm"


CASES = [(1, 64, 256), (1, 1024, 1000), (2, 8, 7), (3, 72, 1), (255, 64, 255), (256, 128, 256), (257, 200, 257),
         (128, 200, 900), (129, 200, 900), (65, 64, 300), (300, 64, 5000), (1, 64, 70001), (3, 72, 151936), (100, 4104, 300), (611, 896, 3001), (1000, 256, 513), (130, 1024, 32003), (700, 1032, 777)]


@pytest.mark.parametrize("n,D,V", CASES)
def test_against_definition(padoc_lib, n, D, V):
    h, w, t, d = make(n, D, V, seed=n + D)
    check(launch(h, w, t, d), *reference(h, w, t, d))


@pytest.mark.parametrize("masked", [0.3, 0.95])
@pytest.mark.parametrize("n,D,V", [(5, 64, 300), (611, 72, 1001), (1500, 320, 2000)])
def test_rows_without_target(padoc_lib, n, D, V, masked):
    h, w, t, d = make(n, D, V, seed=3, masked=masked)
    # what the other rows hold is not looked at
    h[t < 0] = float("nan")
    d[t < 0] = float("inf")
    got = launch(h, w, t, d)
    hz = h.clone()
    hz[t < 0] = 0
    ref, bound = reference(hz, w, t, d)
    check(got, ref, bound)
    out = t < 0
    for x in got[:3]:
        assert bool((x[out] == 0).all())


def test_no_target_at_all(padoc_lib):
    h, w, t, d = make(300, 64, 1000)
    t.fill_(-100)
    for x in launch(h, w, t, d):
        assert bool((x == 0).all())
    padoc.device_status()


def test_targets_past_the_vocabulary(padoc_lib):
    import torch
    h, w, t, d = make(270, 64, 600)
    bad = torch.tensor([0, 13, 269], device="cuda")
    t[bad] = torch.tensor([600, 2 ** 31 - 1, 601], dtype=torch.int32, device="cuda")
    loss, lse, dh, dw = launch(h, w, t, d)
    assert bool(loss[bad].isnan().all()) and bool((lse[bad] == 0).all()) and bool((dh[bad] == 0).all())
    ref, bound = reference(h, w, t, d)
    loss[bad] = 0
    check((loss, lse, dh, dw), ref, bound)


def test_strided_rows(padoc_lib):
    h, w, t, d = make(300, 136, 700, h_pad=24, w_pad=8)
    assert h.stride(0) == 160 and w.stride(0) == 144
    check(launch(h, w, t, d), *reference(h, w, t, d))


@pytest.mark.parametrize("which", ["dh", "dw"])
def test_one_gradient(padoc_lib, which):
    import torch
    h, w, t, d = make(400, 64, 3000)
    both = launch(h, w, t, d)
    one = launch(h, w, t, d, dh=which == "dh", dw=which == "dw")
    i = 2 if which == "dh" else 3
    assert torch.equal(both[i], one[i])


@pytest.mark.parametrize("n,V", [(20001, 17000), (40000, 17001)])
def test_several_pieces(padoc_lib, n, V):
    h, w, t, d = make(n, 64, V, seed=9, masked=0.2)
    check(launch(h, w, t, d), *reference(h, w, t, d))


def test_rows_on_their_own_or_among_others(padoc_lib):
    """A row's loss does not depend on which others have a target, nor does its dh while
    there are enough of them."""
    import torch
    h, w, t, d = make(700, 136, 2100, seed=21)
    whole = launch(h, w, t, d)
    few = t.clone()
    few[torch.arange(700, device="cuda") % 7 == 3] = -1
    part = launch(h, w, few, d)
    on = few >= 0
    for i in (0, 1, 2):
        assert torch.equal(whole[i][on], part[i][on])


def test_the_same_row_twice(padoc_lib):
    import torch
    h, w, t, d = make(520, 64, 700, seed=22)
    h[400], t[400], d[400] = h[3], t[3], d[3]
    loss, lse, dh, dw = launch(h, w, t, d)
    assert torch.equal(loss[400], loss[3]) and torch.equal(lse[400], lse[3]) and torch.equal(dh[400], dh[3])
    check((loss, lse, dh, dw), *reference(h, w, t, d))


def test_large_logits(padoc_lib):
    """A confident model: logits of hundreds, and rows all alike."""
    h, w, t, d = make(300, 64, 900, seed=4)
    h[:100] *= 200
    h[100:150] = 0
    check(launch(h, w, t, d), *reference(h, w, t, d))


def test_a_sure_row(padoc_lib):
    """A target far above all other words: the loss is small, and right to a few steps of
    the sum of exponentials, 1 + something, whatever the logits' size."""
    import torch
    n, D, V = 200, 64, 500
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    w = torch.randn(V, D, generator=g, device="cuda").sign().to(torch.bfloat16)  # products of halves and ones are exact
    t = torch.randint(V, (n,), generator=g, device="cuda").to(torch.int32)
    h = (w[t.long()].float() * 0.5).to(torch.bfloat16)
    x = h.double() @ w.double().T
    want = torch.logsumexp(x, -1) - x.gather(1, t.long()[:, None])[:, 0]
    head = padoc.LmLoss(h, w, t)
    ws = torch.empty(head.ws_size(), dtype=torch.uint8, device="cuda")
    loss, lse = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    head.forward(loss, lse, ws, ws.numel())
    assert float(want.max()) < 0.1
    # 500 exponentials, each within 2^-21 of itself, added in f32 to a sum of some 1
    assert float((loss.double() - want).abs().max()) <= 8 * 2.0 ** -23


def test_a_bad_row_stays_alone(padoc_lib):
    """A NaN or an infinity in a row with a target: that row's loss and gradient are
    NaN, every other row's are what they were; dw holds the NaN, as its formula does."""
    import torch
    h, w, t, d = make(300, 64, 900, seed=5)
    good = launch(h, w, t, d)
    h[7, 3] = float("nan")
    h[290, 0] = float("inf")
    bad = launch(h, w, t, d)
    rest = torch.ones(300, dtype=torch.bool, device="cuda")
    rest[[7, 290]] = False
    for a, b in zip(good[:3], bad[:3]):
        assert torch.equal(a[rest], b[rest])
    assert bool(bad[0][~rest].isnan().all()) and bool(bad[2][7].isnan().all())
    assert bool(bad[3].isnan().any())


def test_repeats_bit_for_bit(padoc_lib):
    import torch
    h, w, t, d = make(3000, 256, 9000, seed=6, masked=0.1)
    first = launch(h, w, t, d)
    for _ in range(3):
        for a, b in zip(first, launch(h, w, t, d)):
            assert torch.equal(a, b)


def test_captured_and_replayed(padoc_lib):
    """The number of rows with a target is read at replay."""
    import torch
    h, w, t, d = make(600, 64, 2000, seed=7)
    n, D, V = 600, 64, 2000
    head = padoc.LmLoss(h, w, t)
    ws = torch.empty(head.ws_size(True), dtype=torch.uint8, device="cuda")
    loss, lse = (torch.zeros(n, device="cuda") for _ in range(2))
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        head.forward(loss, lse, ws, ws.numel())
        head.backward(lse, d, dh, dw, ws, ws.numel())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        head.forward(loss, lse, ws, ws.numel())
        head.backward(lse, d, dh, dw, ws, ws.numel())
    for seed, masked in ((8, 0.6), (9, 0.0), (10, 1.0)):
        h2, w2, t2, d2 = make(n, D, V, seed=seed, masked=masked)
        for a, b in ((h, h2), (w, w2), (t, t2), (d, d2)):
            a.copy_(b)
        graph.replay()
        check((loss, lse, dh, dw), *reference(h2, w2, t2, d2))


def test_other_stream_and_two_at_once(padoc_lib):
    import torch
    a, b = make(700, 128, 4000, seed=11), make(900, 64, 3000, seed=12)
    want = [launch(*a), launch(*b)]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for st, x in zip(s, (a, b)):
        with torch.cuda.stream(st):
            got.append(launch(*x))
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        for p, q in zip(x, y):
            assert torch.equal(p, q)


def test_gradient_against_differences(padoc_lib):
    """Of sum(d_loss * loss), by central differences of the 64-bit loss along directions."""
    import torch
    h, w, t, d = make(40, 64, 200, seed=13, masked=0.2)
    _, _, dh, dw = launch(h, w, t, d)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    f = lambda hh, ww: sum(  # noqa: E731
        float(d[i]) * float(torch.logsumexp(hh[i] @ ww.T, -1) - hh[i] @ ww[int(t[i])]) for i in range(40) if int(t[i]) >= 0)
    for _ in range(3):
        uh = torch.randn(h.shape, generator=g, device="cuda", dtype=torch.float64)
        uw = torch.randn(w.shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-5
        num_h = (f(h.double() + e * uh, w.double()) - f(h.double() - e * uh, w.double())) / (2 * e)
        num_w = (f(h.double(), w.double() + e * uw) - f(h.double(), w.double() - e * uw)) / (2 * e)
        # two roundings of 2^-8 relative to the summands' sizes
        tol_h = 2 * 2.0 ** -8 * float((dh.double().abs() * uh.abs()).sum())
        tol_w = 2 * 2.0 ** -8 * float((dw.double().abs() * uw.abs()).sum())
        assert abs(float((dh.double() * uh).sum()) - num_h) <= tol_h
        assert abs(float((dw.double() * uw).sum()) - num_w) <= tol_w


def test_zero_rows(padoc_lib):
    import torch
    h, w, t, d = make(4, 64, 500)
    head = padoc.LmLoss(h[:0], w, t[:0])
    assert head.ws_size(True) == 0
    loss = torch.empty(0, device="cuda")
    dw = torch.full_like(w, 3.0)
    head.forward(loss, loss, None, 0)
    head.backward(loss, loss, None, dw, None, 0)
    assert bool((dw == 0).all())


def test_guards_around_outputs(padoc_lib):
    """Nothing is written outside the outputs."""
    import torch
    n, D, V = 333, 72, 517
    h, w, t, d = make(n, D, V, seed=15, masked=0.3)
    head = padoc.LmLoss(h, w, t)
    size = head.ws_size(True)
    ws = torch.full((size + 4096,), 7, dtype=torch.uint8, device="cuda")
    buf = {k: torch.full((m + 1024,), 5.0, dtype=dt, device="cuda")
           for k, m, dt in (("loss", n, torch.float32), ("lse", n, torch.float32), ("dh", n * D, torch.bfloat16),
                            ("dw", V * D, torch.bfloat16))}
    v = {k: b[512: 512 + m] for (k, b), m in zip(buf.items(), (n, n, n * D, V * D))}
    head.forward(v["loss"], v["lse"], ws, size)
    head.backward(v["lse"], d, v["dh"], v["dw"], ws, size)
    torch.cuda.synchronize()
    assert bool((ws[size:] == 7).all())
    for k, b in buf.items():
        m = v[k].numel()
        assert bool((b[:512] == 5).all()) and bool((b[512 + m:] == 5).all()), k
    ref, bound = reference(h, w, t, d)
    check((v["loss"], v["lse"], v["dh"].view(n, D), v["dw"].view(V, D)), ref, bound)
