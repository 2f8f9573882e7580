"""Small losses at any size of the logits, and sums that run through many tiles, on the GPU
against 64 bits.

All logits here are exact in f32: products of halves and whole numbers with ones.  What is
left are the sums of exp(x - m), m the row's maximum.
  - A term e^-y: y is exact or off by 2^-24 of itself, its product with log2(e) by 2^-24 and
    the constant's 2^-26, the exponential by 2^-22 of its value: (y + 1) 2^-22 of the term.
  - The maximum's own term is 1, so the loss, the logarithm of the sum plus how far the target
    lies below the maximum, is never negative.
  - An addition to a sum that holds the 1 is off by half a step, 2^-24 of the sum, but by the
    addend at most (the sum without it is a number of f32).  A row's 1 meets 19 additions in
    its tile, 15 in its unit's other tiles and 29 in the join at most (1188 partial results
    on 128 threads, or 76 on 32): 64.  So do the other terms among themselves, each addition
    off by 2^-24 of their sum."""
import pytest

from tree_structured_shared_gb300 import padoc

pytestmark = pytest.mark.gpu


def forward(h, w, t):
    import torch
    head = padoc.LmLoss(h, w, t)
    ws = torch.empty(head.ws_size(), dtype=torch.uint8, device="cuda")
    loss, lse = (torch.full((h.shape[0],), float("nan"), device="cuda") for _ in range(2))
    head.forward(loss, lse, ws, ws.numel())
    torch.cuda.synchronize()
    padoc.device_status()
    return loss, lse


def signs(n, D, V, words, seed):
    """Words of ones and minus ones, and a target a row among the first of them."""
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    w = torch.randn(V, D, generator=g, device="cuda").sign().to(torch.bfloat16)
    return w, torch.randint(words, (n,), generator=g, device="cuda").to(torch.int32)


def check_sure(h, w, t):
    import torch
    loss, lse = forward(h, w, t)
    W = w.double()
    for r in torch.arange(h.shape[0], device="cuda").split(512):
        x = h[r].double() @ W.T
        at = t[r].long()[:, None]
        top = x.gather(1, at)
        y = top - x
        e = torch.exp(-y).scatter_(1, at, 0.0)
        assert float(y.min()) >= 0.0  # the target is the largest
        rest = e.sum(-1)
        want = torch.log1p(rest)
        assert float(want.max()) < 0.1
        bound = 2.0 ** -22 * (e * (y + 1)).sum(-1) + 2.0 ** -17 * rest + 1.1 * rest.clamp(max=64 * 2.0 ** -24) + 1e-30
        off = (loss[r].double() - want).abs()
        assert bool((off <= bound).all()), (float((off - bound).max()), float(off.max()))
        # of lse also its own rounding
        full = top[:, 0] + want
        assert bool(((lse[r].double() - full).abs() <= bound + 2.0 ** -24 * full).all())
    assert float(loss.min()) >= 0.0


@pytest.mark.parametrize("times", [0.5, 1.0, 3.0])
@pytest.mark.parametrize("D", [56, 72, 136, 200, 1000])
def test_sure_rows(padoc_lib, D, times):
    """Target logits from 28 to 3000, of which log2(e) times is rounded in f32."""
    w, t = signs(200, D, 500, 500, D)
    check_sure((w[t.long()].float() * times).bfloat16(), w, t)


@pytest.mark.parametrize("n,V", [(1, 151936), (4300, 152001)])
def test_sure_rows_of_a_large_vocabulary(padoc_lib, n, V):
    """A unit of many rows goes through 16 tiles of words: the maximum is in the first, and by
    fifteen more nothing may drift."""
    w, t = signs(n, 72, V, 256, 1)
    check_sure((w[t.long()].float() * 0.5).bfloat16(), w, t)


def test_maxima_that_rise(padoc_lib):
    """Logits c v / 256 of word v: each tile's maximum lies above the one before it, or below,
    slowly or fast, and most rows' maxima are far from zero.  Terms below e^-17 of the maximum are
    e^-17 of a sum; the others are off by 18 2^-22 of themselves, by 15 rescalings (2^-22
    each) and 64 additions (2^-24): 2^-16 together; the logarithm of up to 152001 by 2^-23 of
    itself, 2^-19.  So 2^-15, and half a step of the result."""
    import torch
    n, V = 4300, 152001
    v = torch.arange(V, device="cuda")
    w = torch.zeros(V, 8, device="cuda")
    w[:, 0], w[:, 1], w[:, 2] = v // 1024 * 4, v // 256 % 4, v % 256 / 256  # 8 bits each
    w = w.bfloat16()
    c = torch.arange(n, device="cuda") % 127 / 8.0 - 7.875
    h = torch.zeros(n, 8, device="cuda")
    h[:, :3] = c[:, None]
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    t = torch.randint(V, (n,), generator=g, device="cuda")
    loss, lse = forward(h.bfloat16(), w, t.to(torch.int32))
    for i in range(127):
        r = torch.arange(i, n, 127, device="cuda")
        x = c[i].double() * v.double() / 256
        want = torch.logsumexp(x, 0)
        own = want - x[t[r]]
        assert bool(((lse[r].double() - want).abs() <= 2.0 ** -15 + 2.0 ** -24 * want.abs()).all()), float(c[i])
        assert bool(((loss[r].double() - own).abs() <= 2.0 ** -15 + 2.0 ** -24 * own).all()), float(c[i])
    assert float(loss.min()) >= 0.0
