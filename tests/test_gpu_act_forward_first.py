"""The kept backward in a training step's usual order: the forward runs on bf16 q, k and v,
its o and lse are those of these values, and only then are q, k, v and o kept.

What it computes then: P = exp(scale q.k - lse) with q and k as the checkpoints hold them and
the forward's lse, so a score is moved by what the codes leave of its q and k, and P's rows sum
to 1 only as far as that goes.  Against that formula the tolerances are those of every backward.

Against the gradients of the forward that ran: a code is off by a uniform part of its group's
step.  With r the root mean square of the scores' moves (measured here, over the pairs that
see one another), P is off by r relative, independently from pair to pair, and so is dv by the
norm; where strong channels make the scores, those of large P move more than the others, up to
twice as much.  dq and dk take about as much again from the codes of k and q and from o's
through the row sums.  Bound: 4 r, and 2^-7 for the roundings to bf16."""
import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

from parity import check_grad

pytestmark = pytest.mark.gpu

PAGES = [wl.Page(700, [9] * 5, [130, 7, 64, 200, 1]), wl.Page(300, [], []), wl.Page(0, [3, 4], [90, 40])]


def inputs(kind, T, H, d, g):
    import torch
    x = torch.randn(T, H, d, generator=g, device="cuda")
    if kind == "twice":
        x *= 2.0
    if kind == "channels":  # a few of them four times as strong as the others
        x *= 1.0 + 3.0 * (torch.arange(d, device="cuda") % 31 == 5)
    return x.bfloat16()


def seen_of(desc, T):
    import torch
    seen = torch.zeros(T, T, dtype=torch.bool)
    qs, kv = desc.segments()
    for q0, n, first, count in qs:
        for a, m, causal in kv[first: first + count]:
            for i in range(q0, q0 + n):
                seen[i, a: min(a + m, i + 1) if causal else a + m] = True
    return seen.cuda()


def gradients(q, k, v, o, lse, d_o, seen):
    """The backward's formula in 64 bits; lse and o None: of the forward on these values."""
    import torch
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    q, k, v, d_o = (x.double() for x in (q, k, v, d_o))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for h in range(Hq):
        s = (q[:, h] @ k[:, h // G].T / d ** 0.5).masked_fill(~seen, -float("inf"))
        p = torch.exp(s - lse[h, :, None].double()) if lse is not None else torch.softmax(s, -1)
        oh = o[:, h].double() if o is not None else p @ v[:, h // G]
        ds = p * (d_o[:, h] @ v[:, h // G].T - (d_o[:, h] * oh).sum(-1, keepdim=True)) / d ** 0.5
        dq[:, h] = ds @ k[:, h // G]
        dk[:, h // G] += ds.T @ q[:, h]
        dv[:, h // G] += p.T @ d_o[:, h]
    return dq, dk, dv


@pytest.mark.parametrize("kind", ["normal", "twice", "channels"])
@pytest.mark.parametrize("Hq,Hkv", [(4, 2), (8, 8)])
def test_forward_then_keep(padoc_lib, kind, Hq, Hkv):
    import torch
    desc = padoc.TreeDesc(PAGES)
    T, d = desc.info()["n_tokens"], 128
    g = torch.Generator(device="cuda")
    g.manual_seed(Hq)
    q, k = inputs(kind, T, Hq, d, g), inputs(kind, T, Hkv, d, g)
    v, d_o = inputs("normal", T, Hkv, d, g), inputs("normal", T, Hq, d, g)
    o, lse = torch.empty_like(q), torch.empty(Hq, T, device="cuda")
    padoc.tree_attn_varlen(desc, q, k, v, o, lse, padoc.BF16, Hq, Hkv, d)
    kept = [torch.empty(padoc.act_bytes(T, x.shape[1] * d), dtype=torch.uint8, device="cuda") for x in (q, k, v, o)]
    padoc.act_keep([x.flatten(1) for x in (q, k, v, o)], kept)
    back = [torch.empty_like(x) for x in (q, k, v, o)]
    padoc.act_restore(kept, [x.flatten(1) for x in back])
    grads = [torch.full_like(x, float("nan")) for x in (q, k, v)]
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(desc, Hq, Hkv, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    padoc.tree_attn_varlen_bwd_kept(desc, *kept, lse, d_o, *grads, Hq, Hkv, d, ws, size)
    torch.cuda.synchronize()
    padoc.device_status()
    seen = seen_of(desc, T)
    for x, r, name in zip(grads, gradients(*back, lse, d_o, seen), ("dq", "dk", "dv")):
        check_grad(x.double().cpu().numpy(), r.cpu().numpy(), "bf16", name)
    moves = []
    for h in range(Hq):
        s = [(a[:, h].double() @ b[:, h * Hkv // Hq].double().T / d ** 0.5)[seen] for a, b in ((q, k), back[:2])]
        moves.append((s[0] - s[1]).pow(2).mean())
    r = float(torch.stack(moves).mean().sqrt())
    off = {}
    for x, ref, name in zip(grads, gradients(q, k, v, None, None, d_o, seen), ("dq", "dk", "dv")):
        off[name] = float((x.double() - ref).norm() / ref.norm())
    print(f"{kind} {Hq}/{Hkv}: scores moved by {r:.4f}, gradients off by", {n: round(e, 4) for n, e in off.items()})
    for name, e in off.items():
        assert e <= 4 * r + 2.0 ** -7, (name, e, r)
