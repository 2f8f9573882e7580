"""Refusals and host arithmetic of the operators around the attention of a training
step.  No GPU: every refusal comes before any launch, and what would launch is not called."""
import ctypes as C

import pytest

from tree_structured_shared_gb300 import padoc

A = 1 << 40  # an aligned address that nothing here reads
INV, UNS = padoc.ERR_INVALID, padoc.ERR_UNSUPPORTED


def refused(rc, code=INV):
    assert rc == code, (rc, padoc.lib().padoc_last_error())


@pytest.fixture
def L(padoc_lib):
    return padoc_lib


def scaling(**kw):
    d = dict(base=1e4, rot_dim=128, kind=padoc.ROPE_RAMP, factor=4.0, context=4096.0, turns_lo=1.0, turns_hi=32.0, amplitude=1.0)
    d.update(kw)
    return padoc.RopeScaling(**d)


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(rot_dim=0), dict(rot_dim=48),
                                dict(rot_dim=160), dict(kind=-1), dict(kind=5), dict(factor=0.5), dict(factor=float("nan")),
                                dict(context=0.0), dict(turns_lo=0.0), dict(turns_lo=33.0), dict(amplitude=-1.0),
                                dict(amplitude=float("inf")), dict(amplitude=1e39), dict(kind=padoc.ROPE_BASE, base=1e300, factor=1e300)])
def test_table(L, kw):
    refused(L.padoc_rope_table(C.byref(scaling(**kw)), 0, 16, A, None))


def test_table_places(L):
    sc = scaling()
    refused(L.padoc_rope_table(None, 0, 16, A, None))
    refused(L.padoc_rope_table(C.byref(sc), -1, 16, A, None))
    refused(L.padoc_rope_table(C.byref(sc), 0, -1, A, None))
    refused(L.padoc_rope_table(C.byref(sc), 2 ** 31 - 10, 11, A, None))
    refused(L.padoc_rope_table(C.byref(sc), 0, 16, A + 4, None))
    refused(L.padoc_rope_table(C.byref(sc), 0, 16, None, None))
    assert L.padoc_rope_table(C.byref(sc), 0, 0, None, None) == 0


def apply(L, parts, rot=64, n_pos=100, dtype=padoc.BF16, d=128, n=10, pos=None, table=A):
    rope = padoc.RopeSpec(table, n_pos, rot, 0)
    p = (padoc.RopePart * max(len(parts), 1))(*[padoc.RopePart(*x) for x in parts])
    return L.padoc_rope_apply(C.byref(rope), len(parts), p, dtype, d, n, pos, 0, None)


def test_apply(L):
    q = (A + (1 << 30), 256, A + (2 << 30), 256, 2)
    refused(apply(L, []))
    refused(apply(L, [q] * 5))
    refused(apply(L, [q], dtype=padoc.I4))
    refused(apply(L, [q], d=96), UNS)
    refused(apply(L, [q], rot=48))
    refused(apply(L, [q], rot=160))
    refused(apply(L, [q], n=-1))
    refused(apply(L, [q], pos=A + 2))
    refused(apply(L, [q], n=101))                       # no positions, and a shorter table
    refused(apply(L, [q], table=None))
    refused(apply(L, [q], table=A + 4))
    refused(apply(L, [(None,) + q[1:]]))
    refused(apply(L, [q[:2] + (None, 256, 2)]))
    refused(apply(L, [(q[0] + 2,) + q[1:]]))
    refused(apply(L, [q[:1] + (248,) + q[2:]]))         # rows shorter than the heads
    refused(apply(L, [q[:1] + (260,) + q[2:]]))         # rows that lose their alignment
    refused(apply(L, [q[:4] + (-1,)]))
    refused(apply(L, [(q[0], 1 << 21, q[2], 1 << 21, 1 << 13)] * 0 + [(q[0], 1 << 28, q[2], 1 << 28, (1 << 20) + 1)], n=1), UNS)
    rope = padoc.RopeSpec(A, 100, 64, 0)
    assert L.padoc_rope_apply(None, 1, None, 0, 128, 1, None, 0, None) == INV
    assert apply(L, [q], n=0) == 0
    assert apply(L, [(None, 0, None, 0, 0)], n=5) == 0
    assert rope.n_pos == 100


def test_apply_overlaps(L):
    x, y = A + (1 << 30), A + (2 << 30)
    refused(apply(L, [(x, 256, x + 512, 256, 2)]))                    # rows shifted by one
    refused(apply(L, [(x, 512, x, 256, 2)]))                          # on itself, closer together
    refused(apply(L, [(x, 256, y, 256, 2), (x + (1 << 20), 256, y + 512, 256, 2)]))   # two outputs
    refused(apply(L, [(x, 256, y, 256, 2), (y + 512 * 9, 256, x + (1 << 20), 256, 2)]))  # an output on another's rows
    refused(apply(L, [(x, 256, A + 64, 256, 2)]))                     # on the table
    refused(apply(L, [(x, 256, y, 256, 2)], pos=y + 16))              # on the positions
    refused(apply(L, [(x, 768, x + 512, 768, 2), (x + 512, 768, x, 768, 2)]))  # two parts that trade places


def act(L, fn, ts):
    a = (padoc.Act * max(len(ts), 1))(*[padoc.Act(*t) for t in ts])
    return getattr(L, fn)(len(ts), a, None)


@pytest.mark.parametrize("fn", ["padoc_act_keep", "padoc_act_restore"])
def test_act(L, fn):
    x, y = A, A + (1 << 30)
    refused(act(L, fn, [(x, 64, 4, 48, y)]))
    refused(act(L, fn, [(x, 64, 4, 0, y)]))
    refused(act(L, fn, [(x, 64, -1, 64, y)]))
    refused(act(L, fn, [(x, 56, 4, 64, y)]))
    refused(act(L, fn, [(x, 68, 4, 64, y)]))
    refused(act(L, fn, [(None, 64, 4, 64, y)]))
    refused(act(L, fn, [(x, 64, 4, 64, None)]))
    refused(act(L, fn, [(x + 2, 64, 4, 64, y)]))
    refused(act(L, fn, [(x, 64, 4, 64, y + 8)]))
    refused(act(L, fn, [(x, 64, 1 << 40, 64, y)]), UNS)
    refused(act(L, fn, [(x, 64, 4, 64, x)]))                          # in place
    refused(act(L, fn, [(x, 64, 4, 64, x + 496)]))
    out = [(x, 64, 4, 64, y), (x + (1 << 20), 64, 4, 64, y + 256)] if fn.endswith("keep") else \
        [(x, 64, 4, 64, y), (x + 496, 64, 4, 64, y + (1 << 20))]
    refused(act(L, fn, out))                                          # two outputs
    refused(act(L, fn, [(x, 64, 4, 64, y)] * 9))
    refused(getattr(L, fn)(-1, None, None))
    refused(getattr(L, fn)(1, None, None))
    assert act(L, fn, []) == 0
    assert act(L, fn, [(None, 64, 0, 64, None)]) == 0


def test_act_bytes(L):
    assert padoc.act_bytes(3, 64) == 3 * 64 + 6
    assert padoc.act_bytes(0, 64) == 0
    for n, w in ((-1, 64), (3, 0), (3, 33), (3, -32)):
        with pytest.raises(padoc.PadocError):
            padoc.act_bytes(n, w)


def head(**kw):
    d = dict(h=A, h_stride=64, w=A + (1 << 32), w_stride=64, targets=A + (2 << 32), n=10, D=64, V=100)
    d.update(kw)
    return padoc.LmHead(**d)


LOSS, LSE, WS = A + (3 << 32), A + (4 << 32), A + (5 << 32)


@pytest.mark.parametrize("kw,code", [(dict(n=-1), INV), (dict(D=0), INV), (dict(D=60), INV), (dict(V=0), INV), (dict(h=None), INV),
                                     (dict(w=None), INV), (dict(targets=None), INV), (dict(h=A + 2), INV), (dict(w=A + 8), INV),
                                     (dict(h_stride=56), INV), (dict(h_stride=68), INV), (dict(w_stride=56), INV),
                                     (dict(n=(1 << 25) + 1), UNS), (dict(targets=A + 1), INV), (dict(V=1 << 29), UNS), (dict(n=1 << 28, V=1 << 28), UNS)])
def test_loss(L, kw, code):
    h = head(**kw)
    refused(L.padoc_lm_loss(C.byref(h), LOSS, LSE, WS, 1 << 32, None), code)
    refused(L.padoc_lm_loss_bwd(C.byref(h), LSE, LOSS, None, None, WS, 1 << 32, None), code)


def test_loss_places(L):
    h = head()
    size, both = C.c_size_t(), C.c_size_t()
    assert L.padoc_lm_loss_ws_size(10, 64, 100, 0, C.byref(size)) == 0 and size.value > 0
    assert L.padoc_lm_loss_ws_size(10, 64, 100, 1, C.byref(both)) == 0 and both.value >= size.value
    refused(L.padoc_lm_loss_ws_size(10, 64, 100, 1, None))
    refused(L.padoc_lm_loss(None, LOSS, LSE, WS, 1 << 32, None))
    for args in ((None, LSE, WS, 1 << 32), (LOSS, None, WS, 1 << 32), (LOSS, LSE, None, 1 << 32), (LOSS, LSE, WS + 16, 1 << 32),
                 (LOSS, LSE, WS, size.value - 1), (LOSS, LOSS, WS, 1 << 32), (LOSS, LOSS + 36, WS, 1 << 32),
                 (h.h + 64, LSE, WS, 1 << 32), (h.targets, LSE, WS, 1 << 32), (LOSS, WS + 64, WS, 1 << 32),
                 (LOSS, LSE, h.w - 256, 1 << 32), (LOSS + 2, LSE, WS, 1 << 32), (LOSS, LSE + 1, WS, 1 << 32)):
        refused(L.padoc_lm_loss(C.byref(h), *args, None))
    dh, dw = A + (6 << 32), A + (7 << 32)
    for args in ((None, LOSS, dh, dw, WS), (LSE, None, dh, dw, WS), (LSE, LOSS, dh + 2, dw, WS), (LSE, LOSS, dh, dw + 8, WS),
                 (LSE, LOSS, dh, dh + 128, WS), (LSE, LOSS, h.h, dw, WS), (LSE, LOSS, dh, h.w, WS), (LSE, LOSS, LSE, dw, WS),
                 (LSE, LOSS, dh, dw, None), (LSE, LOSS, WS + 256, dw, WS), (LSE + 2, LOSS, dh, dw, WS),
                 (LSE, LOSS + 3, dh, dw, WS)):
        refused(L.padoc_lm_loss_bwd(C.byref(h), *args, 1 << 32, None))
    refused(L.padoc_lm_loss_bwd(C.byref(h), LSE, LOSS, dh, dw, WS, both.value - 1, None))
    assert L.padoc_lm_loss_bwd(C.byref(h), LSE, LOSS, None, None, WS, 1 << 32, None) == 0  # nothing is wanted
    empty = head(n=0, h=None, targets=None)
    assert L.padoc_lm_loss(C.byref(empty), None, None, None, 0, None) == 0


def test_loss_binding():
    torch = pytest.importorskip("torch")
    h, w, t = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for a in ((h[:3], w, t), (h, w[:, :32], t), (h.float(), w, t), (h, w, t.long()), (h.T.contiguous().T, w, t), (h, w, torch.zeros(8, dtype=torch.int32)[::2])):
        with pytest.raises(padoc.PadocError):
            padoc.LmLoss(*a)
    with pytest.raises(padoc.PadocError):
        padoc.act_keep([h], [torch.zeros(4 * 64 + 7, dtype=torch.uint8)])
    with pytest.raises(padoc.PadocError):
        padoc.act_keep([h], [])
    with pytest.raises(padoc.PadocError):
        padoc.act_keep([h.float()], [torch.zeros(4 * 64 + 8, dtype=torch.uint8)])


def test_kept_backward(L):
    from tree_structured_shared_gb300.workloads import Page
    desc = padoc.TreeDesc([Page(20, [3], [5])])
    size = padoc.tree_attn_varlen_bwd_kept_ws_size(desc, 4, 2, 128)
    good = dict(q=A, k=A, v=A, o=A, lse=A, d_o=A, dq=A, dk=A, dv=A, Hq=4, Hkv=2, d=128, ws=A, size=size)

    def call(**kw):
        a = dict(good, **kw)
        return L.padoc_tree_attn_varlen_bwd_kept(desc.handle, a["q"], a["k"], a["v"], a["o"], a["lse"], a["d_o"], a["dq"], a["dk"],
                                                 a["dv"], a["Hq"], a["Hkv"], a["d"], 0.0, a["ws"], a["size"], None)

    for k in ("q", "k", "v", "o", "lse", "d_o", "dq", "dk", "dv"):
        refused(call(**{k: None}))
        refused(call(**{k: A + 4}))
    refused(call(Hq=3))
    refused(call(Hkv=0))
    refused(call(Hq=6), UNS)
    refused(call(d=96), UNS)
    refused(call(ws=None))
    refused(call(ws=A + 16))
    refused(call(size=size - 1))
    empty = padoc.TreeDesc([])
    assert L.padoc_tree_attn_varlen_bwd_kept(empty.handle, *[None] * 9, 4, 2, 128, 0.0, None, 0, None) == 0
    with pytest.raises(padoc.PadocError):
        padoc.tree_attn_varlen_bwd_kept_ws_size(desc, 0, 2, 128)
