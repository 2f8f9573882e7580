"""Measured cases of the operators around the tree attention of a training step:
the rotation of packed rows and its gradient, rotation tables for long contexts,
the cross entropy of a large vocabulary with its gradient, and 8-bit checkpoints
of activations with the attention's backward pass that starts from them.

`run` computes a case with elementary torch operations, or, with `own` set,
through the library.  Both work on the same inputs.

A checkpoint of bf16 rows [n, width] is n * width codes (int8), row by row, and
behind them n * width / 32 scale bytes, one for 32 neighbours of a row: the byte e
stands for 2^(e - 127), the smallest power of two (at least 2^-126) of which 127
reach the group's largest magnitude; a value is code * scale.  Byte 255: the group
held an infinity or a NaN, and all of it reads back as NaN.
"""
import functools
import math

import numpy as np
import torch

own = False

GROUP = 32  # values that share a scale

# ------------------------------------------------------------------ the cases


def listed():
    return [
        # the loss of one token, as a scorer that goes along with decoding asks for it: latency, and one read of the weights
        dict(name="loss_one_token", op="loss", n=1, D=1024, V=151936, masked=0.0, train=False, lens=1),
        # a short document on a small vocabulary, odd sizes, a third of the rows without a target
        dict(name="loss_train_short", op="loss", n=611, D=896, V=32003, masked=0.35, train=True, lens=2),
        # evaluation of a page whose prefix (image and prompt) has no targets
        dict(name="loss_eval_page", op="loss", n=6561, D=1024, V=151936, masked=0.7, train=False, lens=3),
        # one packed sequence of the benchmark's training workload
        dict(name="loss_train_16k", op="loss", n=16384, D=1024, V=151936, masked=0.1, train=True, lens=4),
        # the next tokens of 16 pages with 24 branches each: latency
        dict(name="rope_tokens", op="rope", n=384, Hq=16, Hkv=8, d=128, rot=128, interleaved=False, dtype="bf16", fused=True,
             grad=False, lens=5),
        # queries and keys of the benchmark's packed forward, out of one projection
        dict(name="rope_8x16k", op="rope", n=131072, Hq=16, Hkv=8, d=128, rot=128, interleaved=False, dtype="bf16", fused=True,
             grad=False, lens=6),
        # gradients of queries and keys of half heads that turn in part, 32 bits
        dict(name="rope_grad_f32", op="rope", n=50003, Hq=4, Hkv=2, d=64, rot=32, interleaved=True, dtype="f32", fused=False,
             grad=True, lens=7),
        # the table of a context stretched to 131072 positions
        dict(name="rope_table_long", op="table", n=131072, rot=128, kind="ramp", factor=4.0, context=32768, base=1.0e6, first=0, lens=8),
        # q, k, v and o of a small page into a checkpoint and back
        dict(name="keep_page", op="keep", n=462, widths="512 256 256 512", fused=False, lens=9),
        # q, k, v and o of the benchmark's packed forward, into a checkpoint and back
        dict(name="keep_8x16k", op="keep", n=131072, widths="2048 1024 1024 2048", fused=False, lens=10),
        # one page, four query heads a kv head: the attention's gradients from the checkpoint
        dict(name="grad_kept_page", op="attn", pages=1, prefix_lo=420, prefix_hi=420, br_lo=7, br_hi=7, layout=12, content=40,
             Hq=8, Hkv=2, d=128, lens=11),
        # uneven pages, about the tokens of one packed sequence
        dict(name="grad_kept_pages", op="attn", pages=3, prefix_lo=2048, prefix_hi=4809, br_lo=8, br_hi=24, layout=12, content=100,
             Hq=16, Hkv=8, d=128, lens=12),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    lens = rng.randrange(1 << 20)
    op = rng.choice(["loss", "loss", "loss", "rope", "rope", "table", "keep", "attn", "attn"])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    if op == "loss":
        D, V, train = 8 * spread(8, 256), spread(40, 151936), rng.random() < 0.6
        top = int(2.0e12 / (D * V * (4 if train else 1)))
        return dict(op=op, n=spread(1, max(1, min(16384, top))), D=D, V=V, masked=rng.choice([0.0, 0.1, 0.2, 0.7, 0.9]),
                    train=train, lens=lens)
    if op == "rope":
        d = rng.choice([64, 128, 128])
        return dict(op=op, n=spread(1, 65536), Hq=G * Hkv, Hkv=Hkv, d=d, rot=rng.choice([32, 64, d]), interleaved=rng.random() < 0.4,
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fused=rng.random() < 0.5, grad=rng.random() < 0.5, lens=lens)
    if op == "table":
        return dict(op=op, n=spread(100, 131072), rot=rng.choice([32, 64, 96, 128]), kind=rng.choice(["plain", "linear", "base", "bands", "ramp"]),
                    factor=rng.choice([1.5, 2.0, 8.0, 32.0]), context=rng.choice([2048, 8192, 32768]), base=rng.choice([1.0e4, 5.0e5, 1.0e6]),
                    first=rng.choice([0, 0, 100001]), lens=lens)
    if op == "keep":
        return dict(op=op, n=spread(1, 32768), widths=" ".join(str(32 * spread(2, 64)) for _ in range(rng.randint(1, 4))),
                    fused=rng.random() < 0.5, lens=lens)
    prefix = spread(16, 4000)
    return dict(op=op, pages=rng.randint(1, 3), prefix_lo=max(1, prefix // 2), prefix_hi=prefix, br_lo=0, br_hi=rng.randint(1, 16),
                layout=rng.randint(1, 12), content=spread(5, 100), Hq=G * Hkv, Hkv=Hkv, d=128, lens=lens)


# ------------------------------------------------------------------ pages (from the case alone)


def _pages(case):
    """(prefix, layout lengths, content lengths) of each page."""
    r = np.random.default_rng(case["lens"])
    out = []
    for _ in range(case["pages"]):
        P, N = int(r.integers(case["prefix_lo"], case["prefix_hi"] + 1)), int(r.integers(case["br_lo"], case["br_hi"] + 1))
        y = np.clip(np.rint(r.lognormal(math.log(case["content"]), 0.8, N)), 1, 1024).astype(np.int64)
        out.append((P, [case["layout"]] * N, [int(c) for c in y]))
    return out


def _regions(page):
    """Region (-1: prefix) and whether it is content, of each token of a page packed [X | B_1 .. B_N | Y_1 .. Y_N]."""
    P, lay, con = page
    N = len(lay)
    region = np.concatenate([np.full(P, -1), np.repeat(np.arange(N), lay), np.repeat(np.arange(N), con)])
    return region, np.arange(len(region)) >= P + sum(lay)


def _seen(page, dev):
    """[L, L] truth values: token i sees token j."""
    region, content = (torch.from_numpy(a).to(dev) for a in _regions(page))
    at = torch.arange(len(region), device=dev)
    before = at[:, None] >= at[None, :]
    mine = content[:, None] & (region[:, None] >= region[None, :])
    return torch.where(content[None, :], content[:, None] & (region[:, None] == region[None, :]) & before,
                       torch.where(content[:, None], mine, before))


def _pairs(case):
    n = 0
    for P, lay, con in _pages(case):
        s = P + sum(lay)
        n += s * (s + 1) // 2
        for k, y in enumerate(con):
            n += y * (P + sum(lay[: k + 1])) + y * (y + 1) // 2
    return n


def _widths(case):
    return [int(c) for c in case["widths"].split()]


def _with_target(case):
    return max(1, case["n"] - int(round(case["n"] * case["masked"])))


# ------------------------------------------------------------------ checkpoints in torch


@functools.lru_cache
def _powers(dtype, dev):
    """2^(e - 127) for a scale byte e, and NaN for 255: from the host, whose powers of two are exact."""
    return torch.tensor([2.0 ** (e - 127) for e in range(255)] + [math.nan], dtype=torch.float64).to(dtype).to(dev)


def _keep(x):
    """Rows [n, width] f32 -> the bytes of their checkpoint."""
    g = x.unflatten(-1, (-1, GROUP))
    a = g.abs().amax(-1)
    m, e = torch.frexp(a)                           # a = m 2^e, m in [0.5, 1)
    e = e - 7 + (m > 127.0 / 128.0).to(e.dtype)     # 127 2^e reaches a
    e = torch.where(a > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    fine = torch.isfinite(a)
    code = torch.round(g / _powers(x.dtype, x.device)[(e + 127).clamp(max=254).long()][..., None])
    code = torch.where(fine[..., None], code, torch.zeros_like(code)).to(torch.int8)
    scale = torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)
    return torch.cat([code.flatten().view(torch.uint8), scale.flatten()])


def _kept(by, n, width, dtype=torch.float32):
    """The values [n, width] that a checkpoint's bytes stand for."""
    code = by[: n * width].view(torch.int8).to(dtype).unflatten(0, (n, width // GROUP, GROUP))
    scale = _powers(dtype, by.device)[by[n * width:].long()].unflatten(0, (n, width // GROUP))
    return (code * scale[..., None]).flatten(1)


# ------------------------------------------------------------------ inputs


def _table(n_pos, rot, base, dev):
    inv = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, generator=g, device=dev)  # noqa: E731
    empty = lambda *shape, dtype=torch.bfloat16: torch.empty(*shape, dtype=dtype, device=dev)  # noqa: E731
    s = dict(case=case)
    n = case.get("n")
    if case["op"] == "loss":
        D, V = case["D"], case["V"]
        w = (rand(V, D) * (2.5 / math.sqrt(D))).to(torch.bfloat16)
        t = torch.randint(V, (n,), generator=g, device=dev)
        # states of a model that has learnt something: they lean to their target
        s["h"] = (rand(n, D) + w[t].float()).to(torch.bfloat16)
        hidden = torch.argsort(torch.rand(n, generator=g, device=dev))[: n - _with_target(case)]
        t[hidden] = -100
        s["w"], s["t"] = w, t.to(torch.int32)
        s["d_loss"] = (0.5 + torch.rand(n, generator=g, device=dev)) / _with_target(case)
        s["loss"], s["lse"] = empty(n, dtype=torch.float32), empty(n, dtype=torch.float32)
        if case["train"]:
            s["dh"], s["dw"] = empty(n, D), empty(V, D)
    elif case["op"] == "rope":
        Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        wide = (Hq + 2 * Hkv) * d if case["fused"] else (Hq + Hkv) * d
        x = rand(n, wide).to(dt)
        s["q"], s["k"] = x[:, : Hq * d], x[:, Hq * d: (Hq + Hkv) * d]
        if not case["fused"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["table"] = _table(40960, case["rot"], 1.0e6, dev)
        s["pos"] = torch.randint(40960, (1,), generator=g, device=dev) + torch.arange(n, device=dev)
        s["pos"] = (s["pos"] % 40960).to(torch.int32)
        s["q_out"], s["k_out"] = empty(n, Hq * d, dtype=dt), empty(n, Hkv * d, dtype=dt)
    elif case["op"] == "table":
        # another seed, another base: models differ in it
        s["base"] = case["base"] * (1.0 + (seed % 9973) * 1.0e-3)
        s["out"] = empty(n, case["rot"], dtype=torch.float32)
    elif case["op"] == "keep":
        wide = sum(_widths(case))
        x = rand(n, wide) * (1.0 + 4.0 * (torch.rand(1, wide, generator=g, device=dev) < 0.05))  # a few strong channels
        s["x"] = list(x.to(torch.bfloat16).split(_widths(case), -1))
        if not case["fused"]:
            s["x"] = [c.contiguous() for c in s["x"]]
        s["kept"] = [empty(n * c + n * c // GROUP, dtype=torch.uint8) for c in _widths(case)]
        s["out"] = [empty(n, c) for c in _widths(case)]
    else:
        Hq, Hkv, d, pages = case["Hq"], case["Hkv"], case["d"], _pages(case)
        T = sum(len(_regions(p)[0]) for p in pages)
        s["pages"], s["T"] = pages, T
        s["kept"] = [_keep(rand(T, H * d).to(torch.bfloat16).float()) for H in (Hq, Hkv, Hkv)]
        q, k, v = (_kept(b, T, H * d).unflatten(-1, (H, d)) for b, H in zip(s["kept"], (Hq, Hkv, Hkv)))
        o, lse, t0 = torch.empty_like(q), torch.empty(Hq, T, device=dev), 0
        for page in pages:
            c = slice(t0, t0 + len(_regions(page)[0]))
            t0 = c.stop
            x = torch.einsum("thd,jhd->htj", q[c], k[c].repeat_interleave(Hq // Hkv, 1)) / math.sqrt(d)
            x = x.masked_fill(~_seen(page, dev), -math.inf)
            lse[:, c] = torch.logsumexp(x, -1)
            o[c] = torch.einsum("htj,jhd->thd", torch.exp(x - lse[:, c, None]), v[c].repeat_interleave(Hq // Hkv, 1))
        s["kept"].append(_keep(o.flatten(1).to(torch.bfloat16).float()))
        s["lse"] = lse
        s["d_o"] = rand(T, Hq, d).to(torch.bfloat16)
        s["dq"], s["dk"], s["dv"] = empty(T, Hq, d), empty(T, Hkv, d), empty(T, Hkv, d)
    if own:
        from tree_structured_shared_gb300 import padoc
        s["padoc"] = padoc
        if case["op"] == "loss":
            s["head"] = padoc.LmLoss(s["h"], s["w"], s["t"])
            size = s["head"].ws_size(backward=case["train"])
            s["ws"] = empty(size, dtype=torch.uint8)
        elif case["op"] == "rope":
            s["rope"] = padoc.Rope(s["table"], case["rot"], case["interleaved"])
        elif case["op"] == "attn":
            from tree_structured_shared_gb300.workloads import Page
            s["desc"] = padoc.TreeDesc([Page(*p) for p in pages])
            s["desc"].upload(Hq // Hkv)
            s["ws"] = empty(padoc.tree_attn_varlen_bwd_kept_ws_size(s["desc"], Hq, Hkv, d), dtype=torch.uint8)
    return s


# ------------------------------------------------------------------ plain forms


def _plain_loss(s):
    case = s["case"]
    rows = torch.nonzero(s["t"] >= 0)[:, 0]
    t = s["t"][rows].long()
    h, w = s["h"][rows].float(), s["w"].float()
    at = torch.arange(len(rows), device=h.device)
    x = h @ w.T
    m = x.amax(-1, keepdim=True)
    picked = x[at, t]
    e = torch.exp(x.sub_(m))
    total = e.sum(-1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    s["loss"].zero_()[rows] = lse - picked
    s["lse"].zero_()[rows] = lse
    out = dict(loss=s["loss"], lse=s["lse"])
    if case["train"]:
        g = e.div_(total)
        g[at, t] -= 1.0
        g *= s["d_loss"][rows, None]
        dh = torch.zeros_like(s["h"])
        dh[rows] = (g @ w).to(torch.bfloat16)
        out = dict(out, dh=dh, dw=(g.T @ h).to(torch.bfloat16))
    return out


def _plain_rope(s):
    case = s["case"]
    rot, d = case["rot"], case["d"]
    w = s["table"][s["pos"].long()][:, None]
    c, sn = w[..., : rot // 2], w[..., rot // 2:]
    if case["grad"]:
        sn = -sn

    def turn(x):
        y = x.float().unflatten(-1, (-1, d)).clone()
        a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if case["interleaved"] else (y[..., : rot // 2], y[..., rot // 2: rot])
        a2, b2 = a * c - b * sn, b * c + a * sn
        a.copy_(a2)
        b.copy_(b2)
        return y.flatten(1).to(x.dtype)

    return dict(q=turn(s["q"]), k=turn(s["k"]))


def _frequencies(case, base, dev):
    """Angles a position of the pairs, in 64 bits."""
    rot, f = case["rot"], case["factor"]
    i = torch.arange(rot // 2, dtype=torch.float64, device=dev)
    if case["kind"] == "base":
        base = base * f ** (rot / (rot - 2))
    inv = base ** (-2.0 * i / rot)
    if case["kind"] == "linear":
        return inv / f
    turns = case["context"] * inv / (2 * math.pi)
    if case["kind"] == "bands":
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        return inv * (keep + (1 - keep) / f)
    if case["kind"] == "ramp":
        pair = lambda r: rot * math.log(case["context"] / (2 * math.pi * r)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(pair(32.0)), 0), min(math.ceil(pair(1.0)), rot - 1)
        keep = 1 - ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        return inv * (keep + (1 - keep) / f)
    return inv


def _amplitude(case):
    return 0.1 * math.log(case["factor"]) + 1.0 if case["kind"] == "ramp" else 1.0


def _plain_table(s):
    case = s["case"]
    inv = _frequencies(case, s["base"], s["out"].device)
    pos = torch.arange(case["n"], dtype=torch.float64, device=inv.device) + case["first"]
    ang = pos[:, None] * inv
    return (torch.cat([ang.cos(), ang.sin()], -1) * _amplitude(case)).float()


def _plain_keep(s):
    return [_kept(_keep(x.float()), x.shape[0], x.shape[1]).to(torch.bfloat16) for x in s["x"]]


def _plain_attn(s):
    case = s["case"]
    Hq, Hkv, d, T = case["Hq"], case["Hkv"], case["d"], s["T"]
    G, scale = Hq // Hkv, 1 / math.sqrt(d)
    q, k, v, o = (_kept(b, T, H * d).unflatten(-1, (H, d)) for b, H in zip(s["kept"], (Hq, Hkv, Hkv, Hq)))
    d_o = s["d_o"].float()
    row = (d_o * o).sum(-1).T[..., None]
    t0 = 0
    for page in s["pages"]:
        c = slice(t0, t0 + len(_regions(page)[0]))
        t0 = c.stop
        qh, kh, vh, gh = (x[c].transpose(0, 1) for x in (q, k.repeat_interleave(G, 1), v.repeat_interleave(G, 1), d_o))
        p = torch.exp((qh @ kh.transpose(1, 2)) * scale - s["lse"][:, c, None]) * _seen(page, q.device)
        ds = p * (gh @ vh.transpose(1, 2) - row[:, c])
        s["dq"][c] = ((ds @ kh) * scale).transpose(0, 1).to(torch.bfloat16)
        s["dk"][c] = ((ds.transpose(1, 2) @ qh) * scale).unflatten(0, (Hkv, G)).sum(1).transpose(0, 1).to(torch.bfloat16)
        s["dv"][c] = (p.transpose(1, 2) @ gh).unflatten(0, (Hkv, G)).sum(1).transpose(0, 1).to(torch.bfloat16)
    return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])


_PLAIN = dict(loss=_plain_loss, rope=_plain_rope, table=_plain_table, keep=_plain_keep, attn=_plain_attn)


def run(s):
    case = s["case"]
    if not own:
        return _PLAIN[case["op"]](s)
    padoc = s["padoc"]
    if case["op"] == "loss":
        s["head"].forward(s["loss"], s["lse"], s["ws"], s["ws"].numel())
        out = dict(loss=s["loss"], lse=s["lse"])
        if case["train"]:
            s["head"].backward(s["lse"], s["d_loss"], s["dh"], s["dw"], s["ws"], s["ws"].numel())
            out = dict(out, dh=s["dh"], dw=s["dw"])
        return out
    if case["op"] == "rope":
        padoc.rope_apply(s["rope"], case["n"], case["d"], s["q"], s["q_out"], case["Hq"], s["k"], s["k_out"], case["Hkv"],
                         positions=s["pos"], dtype=padoc.BF16 if case["dtype"] == "bf16" else padoc.F32, backward=case["grad"],
                         q_stride=s["q"].stride(0), k_stride=s["k"].stride(0))
        return dict(q=s["q_out"], k=s["k_out"])
    if case["op"] == "table":
        kind = dict(plain=padoc.ROPE_PLAIN, linear=padoc.ROPE_LINEAR, base=padoc.ROPE_BASE, bands=padoc.ROPE_BANDS, ramp=padoc.ROPE_RAMP)
        padoc.rope_table(s["out"], case["n"], case["rot"], s["base"], kind=kind[case["kind"]], factor=case["factor"],
                         context=case["context"], turns_lo=1.0, turns_hi=32.0, amplitude=_amplitude(case), first=case["first"])
        return s["out"]
    if case["op"] == "keep":
        padoc.act_keep(s["x"], s["kept"])
        padoc.act_restore(s["kept"], s["out"])
        return s["out"]
    padoc.tree_attn_varlen_bwd_kept(s["desc"], *s["kept"], s["lse"], s["d_o"], s["dq"], s["dk"], s["dv"], case["Hq"], case["Hkv"],
                                    case["d"], s["ws"], s["ws"].numel())
    return dict(dq=s["dq"], dk=s["dk"], dv=s["dv"])


# ------------------------------------------------------------------ the work of a pass


def work(case):
    if case["op"] == "loss":
        D, V, n = case["D"], case["V"], _with_target(case)
        if case["train"]:  # the logits a second time, and a product for each gradient
            return dict(bytes=2 * V * D * 2 + n * D * 2 + case["n"] * (D * 2 + 16), flops=8.0 * n * D * V + 8.0 * n * V)
        return dict(bytes=V * D * 2 + n * D * 2 + case["n"] * 12, flops=2.0 * n * D * V + 4.0 * n * V)
    if case["op"] == "rope":
        n, H = case["n"], case["Hq"] + case["Hkv"]
        return dict(bytes=2 * n * H * case["d"] * (2 if case["dtype"] == "bf16" else 4) + min(n, 40960) * case["rot"] * 4 + 4 * n,
                    flops=3 * n * H * case["rot"])
    if case["op"] == "table":
        return dict(bytes=case["n"] * case["rot"] * 4, flops=10 * case["n"] * case["rot"])
    if case["op"] == "keep":
        n = case["n"] * sum(_widths(case))
        return dict(bytes=2 * (2 * n + n + n // GROUP), flops=6 * n)
    T, Hq, Hkv, d = sum(len(_regions(p)[0]) for p in _pages(case)), case["Hq"], case["Hkv"], case["d"]
    kept = T * (2 * Hq + 2 * Hkv) * d
    return dict(bytes=kept + kept // GROUP + T * (2 * Hq + 2 * Hkv) * d * 2 + 4 * T * Hq, flops=10.0 * d * Hq * _pairs(case))


# ------------------------------------------------------------------ in 64 bits, from the definitions


def exact(case, seed):
    s = prepare(case, seed)
    dev, n = "cuda", case.get("n")
    if case["op"] == "loss":
        D, V = case["D"], case["V"]
        if 2.0 * _with_target(case) * D * V * (4 if case["train"] else 1) > 4e12:
            return None
        w = s["w"].double()
        loss, lse = (torch.zeros(n, dtype=torch.float64, device=dev) for _ in range(2))
        dh, dw = torch.zeros(n, D, dtype=torch.float64, device=dev), torch.zeros(V, D, dtype=torch.float64, device=dev)
        for i in range(0, n, 2048):
            rows = torch.arange(i, min(n, i + 2048), device=dev)
            rows = rows[s["t"][rows] >= 0]
            if not len(rows):
                continue
            t, h = s["t"][rows].long()[:, None], s["h"][rows].double()
            logp = torch.log_softmax(h @ w.T, -1)
            loss[rows] = -logp.gather(1, t)[:, 0]
            lse[rows] = (h * w[t[:, 0]]).sum(-1) + loss[rows]
            if case["train"]:
                d = s["d_loss"][rows].double()[:, None]
                g = (logp.exp() * d).scatter_add(1, t, -d)
                dh[rows] = g @ w
                dw += g.T @ h
        return dict(loss=loss, lse=lse, dh=dh, dw=dw) if case["train"] else dict(loss=loss, lse=lse)
    if case["op"] == "rope":
        rot, d = case["rot"], case["d"]
        w = s["table"][s["pos"].long()].double()
        z = torch.complex(w[:, : rot // 2].contiguous(), w[:, rot // 2:].contiguous())[:, None]
        z = z.conj() if case["grad"] else z  # the transposed map

        def turn(x):
            x = x.double().reshape(n, -1, d)
            y = x.clone()
            if case["interleaved"]:
                u = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * z
                y[..., :rot] = torch.stack([u.real, u.imag], -1).flatten(-2)
            else:
                u = torch.complex(x[..., : rot // 2].contiguous(), x[..., rot // 2: rot].contiguous()) * z
                y[..., :rot] = torch.cat([u.real, u.imag], -1)
            return y.reshape(n, -1)

        return dict(q=turn(s["q"]), k=turn(s["k"]))
    if case["op"] == "table":
        rot, f, base = case["rot"], case["factor"], s["base"]
        inv = np.array([base ** (-2 * j / rot) for j in range(rot // 2)])
        if case["kind"] == "linear":
            inv = inv / f
        elif case["kind"] == "base":
            inv = np.array([(base * f ** (rot / (rot - 2))) ** (-2 * j / rot) for j in range(rot // 2)])
        elif case["kind"] in ("bands", "ramp"):
            turns = case["context"] * inv / (2 * math.pi)  # over the context
            if case["kind"] == "bands":
                part = np.clip((32.0 - turns) / 31.0, 0, 1)
            else:
                place = lambda r: math.log(case["context"] / (r * 2 * math.pi), base) * rot / 2  # noqa: E731
                lo, hi = max(math.floor(place(32.0)), 0), min(math.ceil(place(1.0)), rot - 1)
                part = np.clip((np.arange(rot // 2) - lo) / max(hi - lo, 0.001), 0, 1)
            inv = inv * ((1 - part) + part / f)
        ang = np.arange(case["first"], case["first"] + n, dtype=np.float64)[:, None] * inv[None]
        z = torch.polar(torch.full((), _amplitude(case), dtype=torch.float64).expand(ang.shape).contiguous(), torch.from_numpy(ang))
        return torch.cat([z.real, z.imag], -1).to(dev)
    if case["op"] == "keep":
        out = []
        for x in s["x"]:
            g = x.double().reshape(-1, GROUP)
            a = g.abs().amax(-1, keepdim=True)
            steps = torch.tensor([2.0 ** e for e in range(-126, 128)], dtype=torch.float64, device=dev)
            step = steps[torch.searchsorted(127 * steps, a)]  # the first of which 127 reach a
            out.append((torch.round(g / step) * step).reshape(x.shape).float())  # whole steps of a power of two: exact in 32 bits
        return out
    Hq, Hkv, d, T = case["Hq"], case["Hkv"], case["d"], s["T"]
    G = Hq // Hkv
    q, k, v, o = (_kept(b, T, H * d, torch.float64).unflatten(-1, (H, d)) for b, H in zip(s["kept"], (Hq, Hkv, Hkv, Hq)))
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    t0 = 0
    for page in s["pages"]:
        region, content = _regions(page)
        c = slice(t0, t0 + len(region))
        t0 = c.stop
        # row by row: what a token sees is the layout stream up to its region (up to itself, in the stream), and its own content before it
        L, stream = len(region), int((~content).sum())
        seen = torch.zeros(L, L, dtype=torch.bool, device=dev)
        seen[:stream, :stream] = torch.ones(stream, stream, dtype=torch.bool, device=dev).tril()
        a = stream
        for b, y in enumerate(page[2]):
            seen[a: a + y, : page[0] + sum(page[1][: b + 1])] = True
            seen[a: a + y, a: a + y] = torch.ones(y, y, dtype=torch.bool, device=dev).tril()
            a += y
        for h in range(Hq):
            kv = h // G
            x = (q[c, h] @ k[c, kv].T) / math.sqrt(d) - s["lse"][h, c, None].double()
            p = torch.where(seen, x.exp(), 0.0)
            gv = s["d_o"][c, h].double()
            ds = p * (gv @ v[c, kv].T - (gv * o[c, h]).sum(-1, keepdim=True)) / math.sqrt(d)
            dq[c, h] = ds @ k[c, kv]
            dk[c, kv] += ds.T @ q[c, h]
            dv[c, kv] += p.T @ gv
    return dict(dq=dq, dk=dk, dv=dv)
