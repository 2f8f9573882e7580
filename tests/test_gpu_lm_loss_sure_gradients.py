"""Gradients of rows whose target is far above all other words, at any size of the logits, on
the GPU against 64 bits.  Logits are exact in f32, as in test_gpu_lm_loss_sure, where the
errors of terms are derived too."""
import pytest

from tree_structured_shared_gb300 import padoc

from test_gpu_lm_loss_sure import forward, signs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [100, 300])
@pytest.mark.parametrize("D,times", [(72, 0.5), (200, 0.5), (200, 3.0)])
def test_gradients_of_sure_rows(padoc_lib, D, times, n):
    """G = d_loss (exp(x - lse) - onehot), first at the lse that the forward gave: a term p is
    off by (y + 1) 2^-22 of itself, y = lse - x, and for the target, where y is exact,
    by 2^-22 (by nothing where y is 0).  G is then rounded to bf16 (2^-8 of it; with 128 rows
    at most 2^-16), the products' sums of up to 512 terms take 16 at a time with two steps of
    2^-23 each (2^-17 of the sum of magnitudes), and the result is rounded once more.
    Then the gradient itself: lse is off by half a step of its own and by the loss's error
    (2^-18, as derived there), but by three times the loss at most: a loss below half a step of
    lse is lost in it, and the target's p is 1."""
    import torch
    V = 500
    w, t = signs(n, D, V, V, D)
    h = (w[t.long()].float() * times).bfloat16()
    _, lse = forward(h, w, t)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    d = torch.rand(n, generator=g, device="cuda") + 0.5
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    head = padoc.LmLoss(h, w, t)
    ws = torch.empty(head.ws_size(True), dtype=torch.uint8, device="cuda")
    head.backward(lse, d, dh, dw, ws, ws.numel())
    torch.cuda.synchronize()
    padoc.device_status()
    W, H, at = w.double(), h.double(), (torch.arange(n, device="cuda"), t.long())
    x = H @ W.T
    rest = torch.exp(x - x[at][:, None])
    rest[at] = 0.0
    true_loss = torch.log1p(rest.sum(-1))
    for true in (False, True):
        y = (x[at] + true_loss if true else lse.double())[:, None] - x
        if true:
            y[at] = true_loss
        p = torch.exp(-y)
        G = p.clone()
        G[at] = torch.expm1(-y[at])
        e = p * (y + 1) * 2.0 ** -22
        if true:
            e += p * torch.minimum(3 * true_loss, 2.0 ** -24 * lse.double() + 2.0 ** -18)[:, None]
            e[at] = torch.minimum(3 * true_loss, 2.0 ** -24 * lse.double() + 2.0 ** -18) + torch.clamp(true_loss, max=2.0 ** -22)
        else:
            e[at] = 2.0 ** -22 * (y[at] != 0).double()
        G, e = G * d.double()[:, None], e * d.double()[:, None]
        e = e + 1.01 * 2.0 ** (-16 if n <= 128 else -8) * (G.abs() + e)
        for name, got, want, bound in (("dh", dh, G @ W, e @ W.abs() + 2.0 ** -17 * (G.abs() @ W.abs())),
                                       ("dw", dw, G.T @ H, e.T @ H.abs() + 2.0 ** -17 * (G.abs().T @ H.abs()))):
            off = (got.double() - want).abs() - (bound + 2.0 ** -8 * (want.abs() + bound) + 1e-30)
            assert float(off.max()) <= 0, (name, true, float(off.max()), float((got.double() - want).abs().max()))
