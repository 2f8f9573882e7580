"""Rows written to and read from bf16 and 4-bit pools on the GPU, against the
NumPy references of the rotation and of the 4-bit format.

The kernel turns a pair with f32 products and sums that are rounded one by one,
which NumPy's float32 arithmetic does too: what a 4-bit pool holds, and every
bf16 row, is compared bit for bit.  The float32 rotation itself is held to the
float64 one within its three roundings (3 * 2^-24 of |a| + |b|)."""
import numpy as np
import pytest

import i4ref
from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch(padoc_lib):
    import torch
    return torch


def rotate32(x, cs, rot, interleaved):
    y = np.asarray(x, np.float32).copy()
    c, s = cs[:, None, : rot // 2], cs[:, None, rot // 2: rot]
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y


def make_pool(torch, nb, Hkv, dtype, max_seqs=64, max_bps=64, fill=None):
    n = padoc.kv_storage_bytes(nb, Hkv, dtype=dtype)
    kp, vp = (torch.empty(n, dtype=torch.uint8, device="cuda") for _ in range(2))
    pool = padoc.KVPool(kp, vp, nb, Hkv, max_seqs=max_seqs, max_blocks_per_seq=max_bps, dtype=dtype)
    pool.sync()
    if fill is not None:
        kp.fill_(fill)
        vp.fill_(fill)
    torch.cuda.synchronize()
    return pool, kp, vp


def rows_on_host(torch, st, nb, Hkv, dtype, is_k):
    """Every slot of a pool's storage [nb, 16, Hkv, 128] float64."""
    if dtype == padoc.BF16:
        return st.view(torch.bfloat16).view(nb, Hkv, 16, 128).double().cpu().numpy().transpose(0, 2, 1, 3)
    u = st.view(nb, Hkv, 1152).cpu().numpy()
    return np.stack([np.stack([i4ref.unpack(u[b, h], is_k) for h in range(Hkv)], 1) for b in range(nb)])


def bf16(x):
    return wl.round_bf16(np.asarray(x, np.float32)).astype(np.float64)


CASES = [
    # Hq, Hkv, rot, interleaved, rows of each sequence, tokens before them
    (16, 8, 128, False, [1, 1, 1], [0, 5, 31]),
    (3, 1, 64, False, [2, 7, 40], [15, 0, 3]),
    (8, 2, 128, True, [17, 1, 3, 0, 16], [16, 0, 9, 4, 0]),
    (0, 3, 32, True, [33], [1]),
    (4, 4, 32, False, [19], [2]),
    (5, 5, 96, False, [4, 2], [0, 14]),
    (2, 2, 0, False, [5, 20], [11, 0]),
]


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("given", [False, True])
def test_write(torch, dtype, case, given):
    """Strided q, k, v of a fused projection; other slots keep their bytes; both position forms."""
    Hq, Hkv, rot, il, ns, prior = CASES[case]
    rng = np.random.default_rng(10 * case + given)
    n, nb = sum(ns), 24
    pool, kp, vp = make_pool(torch, nb, Hkv, dtype, fill=0x51)
    before = [rows_on_host(torch, s, nb, Hkv, dtype, k) for s, k in ((kp, True), (vp, False))]
    off = np.concatenate([[0], np.cumsum(ns)])
    seqs = []
    for m, p in zip(ns, prior):
        seqs.append(pool.alloc(p))
        pool.advance(seqs[-1], p)
        pool.reserve(seqs[-1], m)
    place = np.concatenate([np.arange(p, p + m) for m, p in zip(ns, prior)])
    pos = rng.integers(0, 300, n) if given else place
    W = Hq + 2 * Hkv
    x = wl.round_bf16(rng.normal(size=(n, W + 1, 128)).astype(np.float32) * 2.0 ** rng.integers(-6, 7, size=(n, W + 1, 1)))
    dev = torch.from_numpy(x.reshape(n, -1)).to(torch.bfloat16).cuda()
    tab = i4ref.rope_table(301, rot or 16)
    rows = padoc.KVRows(pool, seqs, None, off, positions=pos if given else None)
    ws = torch.empty(rows.ws_size() + 16, dtype=torch.uint8, device="cuda")
    rows.upload(ws, ws.numel())
    k_rot = torch.full((n + 1, Hkv, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    kw = {}
    if Hq:
        kw = dict(q=dev, Hq=Hq, q_stride=dev.stride(0),
                  q_rot=torch.full((n + 1, Hq, 128), 9.0, dtype=torch.bfloat16, device="cuda"))
    rows.write(dev[:, Hq * 128:], dev[:, (Hq + Hkv) * 128:], ws, k_stride=dev.stride(0), v_stride=dev.stride(0),
               rope=padoc.Rope(torch.from_numpy(tab).cuda(), rot) if not il else
               padoc.Rope(torch.from_numpy(tab).cuda(), rot, True), k_rot=k_rot, **kw)
    torch.cuda.synchronize()
    q, k, v = x[:, :Hq], x[:, Hq: Hq + Hkv], x[:, Hq + Hkv: W]
    k32 = rotate32(k, tab[pos], rot, il)
    k64 = i4ref.rotate(k, tab[pos], rot, il)
    mag = 2 * np.abs(k.astype(np.float64)).max(-1, keepdims=True)
    assert np.all(np.abs(k32 - k64) <= 3 * 2.0 ** -24 * mag)
    assert np.array_equal(k_rot[:n].double().cpu().numpy(), bf16(k32)) and bool((k_rot[n] == 9).all())
    if Hq:
        assert np.array_equal(kw["q_rot"][:n].double().cpu().numpy(), bf16(rotate32(q, tab[pos], rot, il)))
        assert bool((kw["q_rot"][n] == 9).all())
    want = (bf16(k32), bf16(v)) if dtype == padoc.BF16 else i4ref.stored(k32, v)
    for st, exp, was, is_k in ((kp, want[0], before[0], True), (vp, want[1], before[1], False)):
        got = rows_on_host(torch, st, nb, Hkv, dtype, is_k)
        for i, s in enumerate(seqs):
            blk = pool.seq_blocks(s)
            for j in range(ns[i]):
                t = prior[i] + j
                was[blk[t // 16], t % 16] = exp[off[i] + j]
        assert np.array_equal(got, was)


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
def test_many_records_and_gather(torch, dtype):
    """Enough blocks for the record list to live in the workspace; rows read back in another order, twice, and through
    a fork whose shared part ends inside a block."""
    Hkv, rng = 2, np.random.default_rng(3)
    ns = [700, 1, 901, 350, 2500]
    pool, kp, vp = make_pool(torch, 340, Hkv, dtype, max_bps=200)
    seqs = [pool.alloc(0) for _ in ns]
    off = np.concatenate([[0], np.cumsum(ns)])
    n = int(off[-1])
    x = wl.round_bf16(rng.normal(size=(2, n, Hkv, 128)).astype(np.float32))
    k, v = (torch.from_numpy(t).to(torch.bfloat16).cuda() for t in x)
    ws = torch.empty(16 * 400, dtype=torch.uint8, device="cuda")
    pool.append_rope(seqs, off, k, v, ws, ws.numel())
    assert [pool.seq_info(s)["length"] for s in seqs] == ns
    want = i4ref.stored(*x) if dtype == padoc.I4 else tuple(t.astype(np.float64) for t in x)
    child = pool.fork(seqs[2], 41)
    y = wl.round_bf16(rng.normal(size=(2, 20, Hkv, 128)).astype(np.float32))
    ky, vy = (torch.from_numpy(t).to(torch.bfloat16).cuda() for t in y)
    pool.append(child, ky, vy, 20)
    wy = i4ref.stored(*y) if dtype == padoc.I4 else tuple(t.astype(np.float64) for t in y)
    sel = [(seqs[4], 13, 2480), (child, 30, 31), (seqs[0], 0, 700), (seqs[1], 0, 1), (seqs[0], 699, 1), (seqs[3], 7, 0)]
    rows = padoc.KVRows(pool, [s[0] for s in sel], [s[1] for s in sel], np.concatenate([[0], np.cumsum([s[2] for s in sel])]))
    ws2 = torch.empty(rows.ws_size() + 16, dtype=torch.uint8, device="cuda")
    rows.upload(ws2, ws2.numel())
    ko, vo = (torch.full((rows.n + 1, Hkv, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows.gather(ko, vo, ws2)
    torch.cuda.synchronize()
    for got, w, wyy in ((ko, want[0], wy[0]), (vo, want[1], wy[1])):
        exp = np.concatenate([w[off[4] + 13: off[4] + 2493], w[off[2] + 30: off[2] + 41], wyy, w[:700], w[700:701], w[699:700]])
        assert np.array_equal(got[:-1].double().cpu().numpy(), exp) and bool((got[-1] == 5).all())


def test_extreme_values(torch):
    """Magnitudes from below a scale's smallest step to beyond its largest, zeros, NaN and infinities, next to ordinary
    heads in the same warp, rotated on the way (a rotation of large values may overflow, which poisons the token too)."""
    Hkv, n, rng = 8, 61, np.random.default_rng(17)
    e = rng.integers(-140, 128, size=(2, n, Hkv, 1)) * (rng.random((2, n, Hkv, 1)) < 0.4)
    x = wl.round_bf16((rng.normal(size=(2, n, Hkv, 128)) * 2.0 ** e).astype(np.float32))
    x[rng.random((2, n, Hkv)) < 0.1] = 0
    for value in (np.nan, np.inf, -np.inf):
        for which in (0, 1):
            x[which, rng.integers(n), rng.integers(Hkv), rng.integers(128)] = value
    x[0, 5, 3, 16:32] = -0.0
    tab = i4ref.rope_table(80, 128)
    pool, kp, vp = make_pool(torch, 8, Hkv, padoc.I4)
    s = pool.alloc(0)
    k, v = (torch.from_numpy(t).to(torch.bfloat16).cuda() for t in x)
    pool.append_rope([s], [0, n], k, v, rope=padoc.Rope(torch.from_numpy(tab).cuda(), 128))
    rows = padoc.KVRows(pool, [s], [0], [0, n])
    rows.upload()
    ko, vo = (torch.zeros(n, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows.gather(ko, vo)
    with np.errstate(all="ignore"):
        want = i4ref.stored(rotate32(x[0], tab[:n], 128, False), x[1])
    assert np.isnan(want[0]).any(-1).sum() >= 6
    assert np.array_equal(ko.double().cpu().numpy(), want[0], equal_nan=True)
    assert np.array_equal(vo.double().cpu().numpy(), want[1])


def test_commit_and_append_quantise(torch):
    """padoc_kv_append and padoc_kv_commit on a 4-bit pool hold the same values as the rows written one call each."""
    Hkv, rng = 3, np.random.default_rng(5)
    x = wl.round_bf16(rng.normal(size=(2, 50, Hkv, 128)).astype(np.float32))
    x[0, 4, 1, 9], x[1, 7, 0, 100], x[0, 20, 2] = np.inf, np.nan, 0
    k, v = (torch.from_numpy(t).to(torch.bfloat16).cuda() for t in x)
    pool, kp, vp = make_pool(torch, 20, Hkv, padoc.I4)
    a, b = pool.alloc(0), pool.alloc(0)
    pool.append(a, k, v, 9)
    pool.append(a, k[9:], v[9:], 30)
    idx = [3, 4, 49, 7, 7, 20]
    ws = torch.empty(16 * len(idx), dtype=torch.uint8, device="cuda")
    pool.commit([b, a], [0, 4, 6], idx, 50, k, v, ws, ws.numel())
    rows = padoc.KVRows(pool, [a, b], [0, 0], [0, 41, 45])
    rows.upload()
    ko, vo = (torch.zeros(45, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows.gather(ko, vo)
    order = list(range(39)) + [7, 20] + [3, 4, 49, 7]
    want = i4ref.stored(x[0][order], x[1][order])
    assert np.array_equal(ko.double().cpu().numpy(), want[0], equal_nan=True)
    assert np.array_equal(vo.double().cpu().numpy(), want[1])


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
def test_captured_on_a_side_stream(torch, dtype):
    """A write and a gather captured into a graph on another stream, replayed over new inputs in place."""
    Hkv, rng = 2, np.random.default_rng(7)
    pool, kp, vp = make_pool(torch, 12, Hkv, dtype)
    s = pool.alloc(60)
    rows = padoc.KVRows(pool, [s], [0], [0, 45], positions=rng.integers(0, 50, 45))
    ws = torch.empty(rows.ws_size(), dtype=torch.uint8, device="cuda")
    rows.upload(ws, ws.numel())
    pool.advance(s, 45)
    tab = i4ref.rope_table(50, 128)
    rope = padoc.Rope(torch.from_numpy(tab).cuda(), 128)
    k, v, ko, vo = (torch.zeros(45, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4))
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        rows.write(k, v, ws, rope=rope)
        rows.gather(ko, vo, ws)
    rng2 = np.random.default_rng(7)
    pos = rng2.integers(0, 50, 45)
    for seed in range(2):
        x = wl.round_bf16(np.random.default_rng(seed).normal(size=(2, 45, Hkv, 128)).astype(np.float32))
        k.copy_(torch.from_numpy(x[0]))
        v.copy_(torch.from_numpy(x[1]))
        g.replay()
        torch.cuda.synchronize()
        k32 = rotate32(x[0], tab[pos], 128, False)
        want = i4ref.stored(k32, x[1]) if dtype == padoc.I4 else (bf16(k32), bf16(x[1]))
        assert np.array_equal(ko.double().cpu().numpy(), want[0]) and np.array_equal(vo.double().cpu().numpy(), want[1])


def test_in_place_rotation(torch):
    """q_rot = q and k_rot = k when they are dense."""
    rng = np.random.default_rng(9)
    pool, _, _ = make_pool(torch, 4, 2, padoc.BF16)
    s = pool.alloc(20)
    x, y = (wl.round_bf16(rng.normal(size=(20, h, 128)).astype(np.float32)) for h in (3, 2))
    q, k = torch.from_numpy(x).to(torch.bfloat16).cuda(), torch.from_numpy(y).to(torch.bfloat16).cuda()
    rows = padoc.KVRows(pool, [s], [0], [0, 20])
    rows.upload()
    tab = i4ref.rope_table(20, 128)
    rows.write(k, k.clone(), rope=padoc.Rope(torch.from_numpy(tab).cuda(), 128), q=q, Hq=3, q_rot=q, k_rot=k)
    assert np.array_equal(q.double().cpu().numpy(), bf16(rotate32(x, tab, 128, False)))
    assert np.array_equal(k.double().cpu().numpy(), bf16(rotate32(y, tab, 128, False)))


def test_refusals_after_upload(torch):
    """Slots that another sequence can see, sequences named twice, uncounted tokens, released and trimmed sequences."""
    pool, kp, vp = make_pool(torch, 16, 2, padoc.I4)
    t = torch.zeros(40, 2, 128, dtype=torch.bfloat16, device="cuda")
    a = pool.alloc(0)
    pool.append(a, t, t, 20)
    child = pool.fork(a, 18)
    pool.append(child, t, t, 3)

    def code(fn, seqs, first, ns, *args):
        rows = padoc.KVRows(pool, seqs, first, np.concatenate([[0], np.cumsum(ns)]))
        rows.upload()
        try:
            getattr(rows, fn)(t, t, *args)
        except padoc.PadocError as e:
            return e.code
        return 0

    I = padoc.ERR_INVALID
    assert code("write", [child], [17], [2]) == I            # token 17 belongs to the parent
    assert code("write", [a], [19], [1]) == I                # counted, and its block is held by the child
    assert code("write", [child], [18], [3]) == 0            # its own, unshared
    assert code("write", [a], [20], [4]) == 0                # slots nobody has counted
    assert code("gather", [a], [0], [21]) == I               # token 20 is not counted
    assert code("gather", [a, a, child], [0, 3, 0], [20, 5, 15]) == 0
    assert code("write", [child, child], [18, 19], [1, 1]) == I
    b = pool.alloc(32)
    rows = padoc.KVRows(pool, [b], [0], [0, 32])
    rows.upload()
    pool.trim(b)
    for what in ("trimmed", "released"):
        with pytest.raises(padoc.PadocError) as e:
            rows.write(t, t)
        assert e.value.code == I, what
        if what == "trimmed":
            pool.release(b)
            pool.alloc(32)  # the slot lives again, as another sequence
    c = pool.alloc(32)
    rows = padoc.KVRows(pool, [c], [0], [0, 32])
    rows.upload()
    pool.advance(c, 16)
    pool.trim(c)                                             # its second block goes ...
    d = pool.alloc(16)                                       # ... to another sequence,
    pool.reserve(c, 16)                                      # and a different one comes
    assert code_of(lambda: rows.write(t, t)) == I
    kept = padoc.KVRows(pool, [c], [0], [0, 16])
    kept.upload()
    pool.release(d)
    pool.trim(c)
    assert code_of(lambda: kept.write(t, t)) == 0            # the block it names was kept
    dev = pool.device()
    pool.debug_rehome(dev + 1)
    assert code_of(lambda: padoc.KVRows(pool, [a], [0], [0, 2]).upload()) == I
    pool.debug_rehome(dev)
    torch.cuda.synchronize()


def code_of(f):
    try:
        f()
    except padoc.PadocError as e:
        return e.code
    return 0
