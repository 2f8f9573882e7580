"""Branch decode / verify over a 4-bit pool against the float64 oracle run on
the values the pool holds.

Tolerances.  O is rounded to bf16 once (2^-8 of the value).  Before that its
error is that of the weights: P is rounded to fp16 (2^-11 of each weight, or for
weights below 2^-24 of the row's largest an absolute 2^-25 * 2^-10 of it, nothing
next to the rest), exp2 is good to 2^-22, and a score is a 128-term f32 sum of
exact products, off by at most 128 * 2^-24 * sum|q_i k_i| * scale; a weight's
relative error e moves O by at most 2 e max|v| (the numerator and the sum).  So
|dO| <= 2^-8 |O| + 2 (2^-11 + 2^-20 + 2 ds) max|v|, and |dLSE| <= ds + 2^-18
(its sum runs over f32 in a fixed tree) + 2^-23 |LSE|."""
import copy

import numpy as np
import pytest

import i4ref
from oracle import tree_attention as ta
from tree_structured_shared_gb300 import padoc
from tree_structured_shared_gb300 import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def harness(padoc_lib):
    from tree_structured_shared_gb300 import harness as h
    return h


def cached(vals):
    """vals with the cached K/V replaced by what a 4-bit pool holds of them."""
    c = copy.copy(vals)
    for a, b in (("prefix_k", "prefix_v"), ("own_k", "own_v")):
        pairs = [i4ref.stored(k, v) for k, v in zip(getattr(vals, a), getattr(vals, b))]
        setattr(c, a, [p[0] for p in pairs])
        setattr(c, b, [p[1] for p in pairs])
    return c


def check(o, lse, O, L, vals, d=128, scale=None, what=""):
    o, lse = o.astype(np.float64), lse.astype(np.float64)
    ks = [x for x in vals.prefix_k + vals.own_k + [vals.k_new] if len(x)]
    vs = [x for x in vals.prefix_v + vals.own_v + [vals.v_new] if len(x)]
    kn = max(np.sqrt((np.asarray(k, np.float64) ** 2).sum(-1)).max() for k in ks)
    qn = np.sqrt((np.asarray(vals.q, np.float64) ** 2).sum(-1))[..., None]
    vmax = max(np.abs(v).max() for v in vs)
    ds = 128 * 2.0 ** -24 * qn * kn * (scale or d ** -0.5)
    tol = 2.0 ** -8 * np.abs(O) + 2 * (2.0 ** -11 + 2.0 ** -20 + 2 * ds) * vmax
    assert np.all(np.isfinite(o)), what
    assert np.all(np.abs(o - O) <= tol), f"{what}: {(np.abs(o - O) / tol).max():.3f} of the bound"
    tl = ds[..., 0] + 2.0 ** -18 + 2.0 ** -23 * np.abs(L)
    assert np.all(np.abs(lse - L) <= tl), f"{what}: LSE {(np.abs(lse - L) / tl).max():.3f} of the bound"


def run(harness, w, vals, tree=True, **kw):
    import torch
    d = harness.Decode(w, vals, tree=tree, dtype=padoc.I4, **kw)
    o, lse = d.run()
    torch.cuda.synchronize()
    padoc.device_status()
    n = w.n_queries
    return o.float().cpu().numpy()[:n], lse.cpu().numpy()[:n], d


def both(harness, w, seed, tree=True, what="", **kw):
    vals = wl.decode_values(w, seed)
    o, lse, d = run(harness, w, vals, tree, **kw)
    c = cached(vals)
    O, L = ta.branch_decode(w, c, tree=tree)
    check(o, lse, O, L, c, what=what)
    return d


@pytest.mark.parametrize("seed", range(4))
def test_verify_ragged(harness, seed):
    w = wl.small_decode(seed, n_pages=4, max_prefix=700, max_branches=6, max_own=300, Hq=4, Hkv=2)
    both(harness, w, seed, what=f"seed {seed}")


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("verify", [False, True])
def test_groups(harness, G, verify):
    """From one row a unit to 128 (16 query tokens of 8 heads), odd groups among them."""
    w = wl.small_decode(20 + G, n_pages=3, max_prefix=400, max_branches=5, max_own=100, verify=verify, Hq=2 * G, Hkv=2)
    both(harness, w, G, tree=verify, what=f"G {G}")


def page(P, fork, own, q, parents=None):
    parents = parents or [[-1] + list(range(n - 1)) for n in q]
    return wl.DecodePage(P, fork, own, q, parents)


@pytest.mark.parametrize("lens", [(0, 0), (0, 1), (1, 0), (15, 16), (16, 17), (17, 15), (64, 65), (127, 129)])
def test_block_borders(harness, lens):
    """Prefixes and suffixes that are empty, one token, or end on, before and after a block border."""
    P, own = lens
    w = wl.DecodeWorkload("b", [page(P, [P, P, max(0, P - 1)], [own, 0, own + 1], [1, 2, 16])], 4, 2, 128, 1.0)
    both(harness, w, P + own, what=str(lens))


def test_many_branches_and_chunks(harness):
    """A page whose rows fill several row tiles, and a long prefix cut into more chunks than the own pass joins."""
    pages = [page(3000, [3000 - 3 * i for i in range(45)], [i * 7 % 40 for i in range(45)], [1 + i % 3 for i in range(45)]),
             page(9000, [9000], [2100], [3]), page(0, [0, 0], [5000, 0], [2, 1])]
    w = wl.DecodeWorkload("m", pages, 8, 4, 128, 0.5)
    d = both(harness, w, 5, what="chunks")
    both(harness, w, 6, what="fragmented", fragment=True)
    # the same bits from a second run, from noalloc and from the passes of a plan
    import torch
    first = (d.o.clone(), d.lse.clone())
    d.o.zero_()
    d.run()
    assert torch.equal(d.o, first[0]) and torch.equal(d.lse, first[1])
    d.o.zero_()
    padoc.branch_decode_noalloc(d.pool, d.batch, w.Hq, d.q, d.k_new, d.v_new, d.tree_bits, d.o, d.lse)
    assert torch.equal(d.o, first[0]) and torch.equal(d.lse, first[1])


@pytest.mark.parametrize("prefixes", [(100, 100), (1, 128), (120, 300), (257, 640)])
def test_many_pages_of_few_tiles(harness, prefixes):
    """Several units of one to five key tiles for each SM, with 20 to 150 query rows: short units one after another."""
    rng = np.random.default_rng(prefixes[1])
    pages = []
    for _ in range(230):
        P, N = int(rng.integers(prefixes[0], prefixes[1] + 1)), int(rng.integers(5, 9))
        q = [int(x) for x in rng.integers(1, 6, N)]
        pages.append(page(P, [max(0, P - int(x)) for x in rng.integers(0, 9, N)], [int(x) for x in rng.integers(0, 20, N)], q))
    w = wl.DecodeWorkload("p", pages, 8, 2, 128, 0.7)
    both(harness, w, prefixes[0], what=str(prefixes))


def test_row_tiles_cut_differently(harness):
    """Pages of several row tiles and uneven lengths: a page's row tiles are cut into different numbers of pieces."""
    rng = np.random.default_rng(41)
    pages = []
    for P, N in ((1812, 6), (795, 19), (2825, 11), (300, 16)):
        q = [int(x) for x in rng.integers(1, 17, N)]
        pages.append(page(P, [max(0, P - int(x)) for x in rng.integers(0, 900, N)], [int(x) for x in rng.integers(0, 40, N)], q))
    w = wl.DecodeWorkload("p", pages, 16, 4, 128, 0.7)
    both(harness, w, 41, what="uneven")


def test_captured_passes(harness):
    """A plan's two passes captured on another stream and replayed over new queries."""
    import torch
    w = wl.small_decode(3, n_pages=3, max_prefix=900, max_branches=6, max_own=600, Hq=8, Hkv=2)
    vals = wl.decode_values(w, 3)
    _, _, d = run(harness, w, vals)
    d.plan()
    torch.cuda.synchronize()
    g, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=st):
        d.prefix_pass()
        d.own_pass()
    for seed in (11, 12):
        new = wl.decode_values(w, seed)
        c = cached(vals)
        c.q, c.k_new, c.v_new = new.q, new.k_new, new.v_new
        for t, x in ((d.q, new.q), (d.k_new, new.k_new), (d.v_new, new.v_new)):
            t.copy_(torch.from_numpy(x))
        d.o.zero_()
        g.replay()
        torch.cuda.synchronize()
        O, L = ta.branch_decode(w, c)
        check(d.o.float().cpu().numpy()[: w.n_queries], d.lse.cpu().numpy()[: w.n_queries], O, L, c, what="replay")


@pytest.mark.parametrize("mag", [1e-30, 1e-4, 1.0, 300.0])
def test_magnitudes(harness, mag):
    """Queries from far below to far above fp16's range next to each other, strong keys, peaked and flat softmaxes."""
    w = wl.small_decode(8, n_pages=2, max_prefix=500, max_branches=5, max_own=200, Hq=8, Hkv=2)
    vals = wl.decode_values(w, 8)
    rows = np.arange(w.n_queries)[:, None, None] % 3
    vals.q = wl.round_bf16(vals.q * np.where(rows == 0, mag, np.where(rows == 1, 1.0, 1e-3)).astype(np.float32))
    o, lse, _ = run(harness, w, vals)
    c = cached(vals)
    O, L = ta.branch_decode(w, c)
    check(o, lse, O, L, c, what=f"mag {mag}")


def test_rising_scores(harness):
    """Scores that grow along the keys move the running maximum again and again."""
    w = wl.DecodeWorkload("r", [page(1500, [1500, 1400], [700, 20], [4, 1])], 4, 2, 128, 1.0)
    vals = wl.decode_values(w, 1)
    for ks in (vals.prefix_k, vals.own_k):
        for k in ks:
            k *= np.linspace(0.05, 4.0, len(k), dtype=np.float32)[:, None, None]
            k[:] = wl.round_bf16(k)
    o, lse, _ = run(harness, w, vals)
    c = cached(vals)
    O, L = ta.branch_decode(w, c)
    check(o, lse, O, L, c, what="rising")


def test_nan_stays_with_the_rows_that_see_it(harness):
    """NaN and infinities in cached rows, in hidden draft tokens, in one query row and in freed blocks."""
    w = wl.DecodeWorkload("n", [page(200, [200, 150, 150], [30, 0, 21], [3, 3, 2],
                                     [[-1, 0, 0], [-1, 0, 1], [-1, 0]])], 4, 2, 128, 1.0)
    clean = wl.decode_values(w, 2)
    O, L = ta.branch_decode(w, cached(clean))
    # rows: branch 0 -> 0..2, branch 1 -> 3..5, branch 2 -> 6, 7
    def rows_hit(vals):
        o, lse, _ = run(harness, w, vals)
        hit = np.isnan(o).any(-1) | np.isnan(lse)
        ok = ~hit
        # the rows that are not hit: as without the change
        assert np.abs(o.astype(np.float64) - O)[ok].max() <= 2.0 ** -8 * np.abs(O).max() + 2.0 ** -9 * 5
        return sorted({int(r) for r in np.nonzero(hit)[0]})

    def change(field, i, idx, value):
        vals = copy.deepcopy(clean)
        x = getattr(vals, field) if i is None else getattr(vals, field)[i]
        x[idx] = value
        return rows_hit(vals)

    assert change("prefix_v", 0, (180, 0, 5), np.nan) == [0, 1, 2]     # branches 1 and 2 end at 150
    assert change("prefix_k", 0, (180, 1, 5), np.inf) == [0, 1, 2]
    assert change("own_v", 2, (20, 0, 127), np.inf) == [6, 7]
    assert change("v_new", None, (1, 0, 3), np.nan) == [1]             # a leaf of branch 0's tree
    assert change("k_new", None, (7, 1, 3), np.nan) == [7]
    assert change("q", None, (5, 2, 3), np.nan) == [5]


def test_nan_on_wide_pages(harness):
    """The same where a page has 80 query rows: a poisoned token of the prefix, infinite and NaN queries."""
    forks = [400] * 5 + [250] * 5
    w = wl.DecodeWorkload("n", [page(400, forks, [20] * 10, [4] * 10)], 4, 2, 128, 1.0)
    clean = wl.decode_values(w, 5)
    base, lse0, _ = run(harness, w, clean, tree=False)

    def rows_hit(vals):
        o, lse, _ = run(harness, w, vals, tree=False)
        hit = np.isnan(o).any(-1) | np.isnan(lse)
        ok = ~hit
        # the others see nothing of it: not a bit changes
        assert np.array_equal(o[ok], base[ok]) and np.array_equal(lse[ok], lse0[ok])
        return sorted({int(r) for r in np.nonzero(hit)[0]})

    def change(field, i, idx, value):
        vals = copy.deepcopy(clean)
        x = getattr(vals, field) if i is None else getattr(vals, field)[i]
        x[idx] = value
        return rows_hit(vals)

    assert change("prefix_k", 0, (399, 1, 5), np.nan) == list(range(20))  # branches 5 .. 9 end at 250
    assert change("prefix_v", 0, (250, 0, 77), np.inf) == list(range(20))
    assert change("prefix_v", 0, (0, 0, 0), -np.inf) == list(range(40))
    # 8 rows share a factor in the own pass, the row alone has one in the prefix pass
    assert change("q", None, (21, 3, 9), np.nan) == [21]


def test_noalloc_and_plan_agree(harness):
    """The workspace call, the plan's two passes and the call without allocation give the same bits."""
    import torch
    w = wl.small_decode(21, n_pages=3, max_prefix=700, max_branches=8, max_own=300, Hq=8, Hkv=2)
    vals = wl.decode_values(w, 21)
    o, lse, d = run(harness, w, vals)
    d.o.zero_()
    padoc.branch_decode_noalloc(d.pool, d.batch, 8, d.q, d.k_new, d.v_new, d.tree_bits, d.o, d.lse)
    torch.cuda.synchronize()
    n = w.n_queries
    assert np.array_equal(d.o.float().cpu().numpy()[:n], o) and np.array_equal(d.lse.cpu().numpy()[:n], lse)
    d.plan()
    d.o.zero_()
    d.prefix_pass()
    d.own_pass()
    torch.cuda.synchronize()
    assert np.array_equal(d.o.float().cpu().numpy()[:n], o) and np.array_equal(d.lse.cpu().numpy()[:n], lse)


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
def test_blocks_far_into_a_large_pool(harness, dtype):
    """Blocks whose bytes start past 2^32: rows written, decoded (few and many query rows) and read back as in a small pool."""
    import torch
    Hkv, Hq, rng = 8, 16, np.random.default_rng(9)
    far = (2 ** 32 // (Hkv * (1152 if dtype == padoc.I4 else 4096))) + 100
    dev = lambda *s: torch.from_numpy(rng.normal(size=s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731
    pk, pv, ok, ov = dev(333, Hkv, 128), dev(333, Hkv, 128), dev(70, Hkv, 128), dev(70, Hkv, 128)
    q, kn, vn = dev(14, Hq, 128), dev(14, Hkv, 128), dev(14, Hkv, 128)
    tab = torch.from_numpy(i4ref.rope_table(400, 128)).cuda()
    got = []
    for skip in (0, far):
        nb = skip + 64
        size = padoc.kv_storage_bytes(nb, Hkv, dtype=dtype)
        kp, vp = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
        pool = padoc.KVPool(kp, vp, nb, Hkv, max_seqs=8, max_blocks_per_seq=max(skip, 32), dtype=dtype)
        if skip:
            pool.alloc(16 * skip)
        p = pool.alloc(0)
        pool.append_rope([p], [0, 333], pk, pv, rope=padoc.Rope(tab, 128))
        assert min(pool.seq_blocks(p)) >= skip
        br = [pool.fork(p, 333), pool.fork(p, 200)]
        for b in br:
            pool.append(b, ok, ov, 70)
        out = []
        for off in ([0, 1, 2], [0, 7, 14]):  # 4 and 28 query rows a kv head
            batch = padoc.Batch([p], [0, 2], br, off)
            n = padoc.branch_decode_ws_size(pool, batch, Hq)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            o = torch.zeros(14, Hq, 128, dtype=torch.bfloat16, device="cuda")
            lse = torch.zeros(14, Hq, device="cuda")
            padoc.branch_decode(pool, batch, Hq, q, kn, vn, None, o, lse, ws, n)
            out += [o, lse]
        back = padoc.KVRows(pool, br, [0, 0], [0, 403, 673])
        back.upload()
        k, v = (torch.empty(673, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        back.gather(k, v)
        torch.cuda.synchronize()
        padoc.device_status()
        got.append([x.cpu() for x in out + [k, v]])
        del kp, vp, pool
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][0].abs().sum() > 0 and got[0][-1].abs().sum() > 0


def test_stale_blocks(harness):
    """Slots past a sequence's end keep what an earlier, poisoned sequence left there."""
    import torch
    w = wl.DecodeWorkload("s", [page(37, [37, 20], [5, 9], [1, 4])], 4, 2, 128, 1.0)
    vals = wl.decode_values(w, 4)
    nb = 12
    size = padoc.kv_storage_bytes(nb, 2, dtype=padoc.I4)
    kp, vp = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    pool = padoc.KVPool(kp, vp, nb, 2, max_seqs=8, max_blocks_per_seq=12, dtype=padoc.I4)
    bad = torch.full((16 * nb, 2, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    s = pool.alloc(0)
    pool.append(s, bad, bad, 16 * nb)
    pool.release(s)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).cuda()  # noqa: E731
    p = pool.alloc(0)
    pool.append(p, dev(vals.prefix_k[0]), dev(vals.prefix_v[0]), 37)
    br = [pool.fork(p, 37), pool.fork(p, 20)]
    for b, k, v in zip(br, vals.own_k, vals.own_v):
        pool.append(b, dev(k), dev(v), len(k))
    batch = padoc.Batch([p], [0, 2], br, [0, 1, 5])
    n = padoc.branch_decode_ws_size(pool, batch, 4)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o = torch.empty(5, 4, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(5, 4, device="cuda")
    padoc.branch_decode(pool, batch, 4, dev(vals.q), dev(vals.k_new), dev(vals.v_new), None, o, lse, ws, n)
    c = cached(vals)
    O, L = ta.branch_decode(w, c, tree=False)
    check(o.float().cpu().numpy(), lse.cpu().numpy(), O, L, c, what="stale")


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale(harness, scale):
    import torch
    w = wl.small_decode(6, n_pages=2, max_prefix=300, max_branches=4, max_own=150, Hq=4, Hkv=2)
    vals = wl.decode_values(w, 6)
    d = harness.Decode(w, vals, dtype=padoc.I4)
    padoc.branch_decode(d.pool, d.batch, 4, d.q, d.k_new, d.v_new, d.tree_bits, d.o, d.lse, d.ws, d.ws_bytes, scale)
    torch.cuda.synchronize()
    c = cached(vals)
    O, L = ta.branch_decode(w, c, scale=scale)
    check(d.o.float().cpu().numpy()[: w.n_queries], d.lse.cpu().numpy()[: w.n_queries], O, L, c, scale=scale, what="scale")


@pytest.mark.parametrize("dtype", [padoc.BF16, padoc.I4])
def test_a_step_end_to_end(harness, dtype):
    """Prefill rows appended with their rotation, branches forked, a step's rows rotated into reserved slots, the step
    decoded from q_rot / k_rot, accepted rows counted, and the cache read back."""
    import torch
    rng = np.random.default_rng(0)
    Hq, Hkv, P, nbr = 8, 2, 83, 3
    size = padoc.kv_storage_bytes(64, Hkv, dtype=dtype)
    kp, vp = (torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    pool = padoc.KVPool(kp, vp, 64, Hkv, max_seqs=8, max_blocks_per_seq=32, dtype=dtype)
    tab = i4ref.rope_table(200, 128)
    rope = padoc.Rope(torch.from_numpy(tab).cuda(), 128)
    mk = lambda *s: wl.round_bf16(rng.normal(size=s).astype(np.float32))  # noqa: E731
    dev = lambda x: torch.from_numpy(x).to(torch.bfloat16).cuda()  # noqa: E731
    held = (lambda k, v: i4ref.stored(k, v)) if dtype == padoc.I4 else \
        (lambda k, v: (wl.round_bf16(k.astype(np.float32)).astype(np.float64), v.astype(np.float64)))

    def rot32(x, pos):
        c, s = tab[pos][:, None, :64], tab[pos][:, None, 64:]
        a, b = x[..., :64], x[..., 64:]
        return np.concatenate([a * c - b * s, b * c + a * s], -1)

    pk, pv = mk(P, Hkv, 128), mk(P, Hkv, 128)
    page_seq = pool.alloc(0)
    pool.append_rope([page_seq], [0, P], dev(pk), dev(pv), rope=rope)
    br = [pool.fork(page_seq, P - 5 * i) for i in range(nbr)]
    own = [[np.zeros((0, Hkv, 128))] * 2 for _ in br]
    for step in range(3):
        off = [0, 2, 3, 7]
        n = off[-1]
        q, k, v = mk(n, Hq, 128), mk(n, Hkv, 128), mk(n, Hkv, 128)
        first = [pool.seq_info(b)["length"] for b in br]
        pos = np.concatenate([np.arange(f, f + m) for f, m in zip(first, np.diff(off))])
        for b, m in zip(br, np.diff(off)):
            pool.reserve(b, int(m))
        rows = padoc.KVRows(pool, br, None, off)
        rows.upload()
        q_rot = torch.empty(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
        k_rot = torch.empty(n, Hkv, 128, dtype=torch.bfloat16, device="cuda")
        dv = dev(v)
        rows.write(dev(k), dv, rope=rope, q=dev(q), Hq=Hq, q_rot=q_rot, k_rot=k_rot)
        batch = padoc.Batch([page_seq], [0, nbr], br, off)
        nb = padoc.branch_decode_ws_size(pool, batch, Hq)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        o = torch.empty(n, Hq, 128, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(n, Hq, device="cuda")
        padoc.branch_decode(pool, batch, Hq, q_rot, k_rot, dv, None, o, lse, ws, nb)
        torch.cuda.synchronize()
        kr = rot32(k, pos)
        PK, PV = held(rot32(pk, np.arange(P)), pv)
        for i in range(nbr):
            r = slice(off[i], off[i + 1])
            for t in range(off[i + 1] - off[i]):
                m = slice(off[i], off[i] + t + 1)
                f = P - 5 * i
                K = np.concatenate([PK[:f], own[i][0], wl.round_bf16(kr[m]).astype(np.float64)])
                V = np.concatenate([PV[:f], own[i][1], v[m].astype(np.float64)])
                O, L = ta._attend(q_rot[off[i] + t].double().cpu().numpy(), K, V, 128 ** -0.5)
                got = o[off[i] + t].double().cpu().numpy()
                assert np.abs(got - O).max() <= 2.0 ** -8 * np.abs(O).max() + 2.0 ** -7 * 0.5 * np.abs(V).max()
                assert np.abs(lse[off[i] + t].cpu().numpy() - L).max() <= 1e-3 * np.abs(L).max()
            # all of the block's rows count from here on
            pool.advance(br[i], off[i + 1] - off[i])
            hk, hv = held(kr[r], v[r])
            own[i] = [np.concatenate([own[i][0], hk]), np.concatenate([own[i][1], hv])]
    back = padoc.KVRows(pool, br, [0] * nbr, np.concatenate([[0], np.cumsum([pool.seq_info(b)["length"] for b in br])]))
    back.upload()
    ko, vo = (torch.empty(back.n, Hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    back.gather(ko, vo)
    wk = np.concatenate([np.concatenate([PK[: P - 5 * i], own[i][0]]) for i in range(nbr)])
    wv = np.concatenate([np.concatenate([PV[: P - 5 * i], own[i][1]]) for i in range(nbr)])
    assert np.array_equal(ko.double().cpu().numpy(), wk) and np.array_equal(vo.double().cpu().numpy(), wv)
