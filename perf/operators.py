"""Measured cases of the paged-cache operators: rows written with the position
rotation on the way (bf16 and 4-bit pools), rows read back as dense K/V, and
branch decode / verify over a 4-bit pool.

`run` computes a case with elementary torch operations, or, with `own` set,
through the library.  Both work on the same inputs: tensors of one layer, the
pool's storage and the block tables of its sequences.

The 4-bit storage of one (block, kv head), 1152 bytes, 16 token slots:
  K: codes [4 chunks of 32 dims][16 slots][16 bytes], scales [16 slots][8 groups]
  V: codes [8 groups of 16 dims][16 slots][8 bytes], scales [8 groups][16 slots]
A 32-bit word holds 8 consecutive dims: nibble j the dim 2j, nibble 4 + j the
dim 2j + 1, each as n + 8 with n in [-7, 7].  A group's scale is a byte, bits
14..7 of an fp16 number; a value is n * scale.
"""
import math

import numpy as np
import torch

own = False

D = 128            # head dimension
BS = 16            # tokens of a block
UNIT = 1152        # bytes of one (block, kv head) of a 4-bit pool
MAX_SCALE = 896.0
ROPE_BASE = 1.0e6

# ------------------------------------------------------------------ the cases


def listed():
    return [
        # one decode step's new tokens of 16 pages with 24 live branches each: latency
        dict(name="write_step_bf16", op="write", dtype="bf16", seqs=384, rows_lo=1, rows_hi=1, prior_hi=48, Hq=16, Hkv=8,
             rot=128, interleaved=False, far=True, lens=1),
        # prefill of 16 pages of 4809 tokens into a bf16 cache
        dict(name="write_prefill_bf16", op="write", dtype="bf16", seqs=16, rows_lo=4809, rows_hi=4809, prior_hi=0, Hq=16,
             Hkv=8, rot=128, interleaved=False, far=False, lens=2),
        # draft blocks of a verify step of 64 pages, written to a 4-bit cache and read back
        dict(name="write_drafts_i4", op="write", dtype="i4", seqs=1490, rows_lo=1, rows_hi=16, prior_hi=33, Hq=16, Hkv=8,
             rot=128, interleaved=False, far=True, lens=3),
        # prefill of 64 pages into a 4-bit cache, read back for the next chunk's attention
        dict(name="write_prefill_i4", op="write", dtype="i4", seqs=64, rows_lo=4809, rows_hi=4809, prior_hi=0, Hq=16, Hkv=8,
             rot=128, interleaved=False, far=False, lens=4),
        # one page's cached prefix expanded for the rows that follow it
        dict(name="gather_page_i4", op="gather", dtype="i4", seqs=1, len_lo=2048, len_hi=2048, first_hi=5, Hkv=8, lens=5),
        # the prefixes of 64 pages of uneven lengths
        dict(name="gather_pages_i4", op="gather", dtype="i4", seqs=64, len_lo=4000, len_hi=6144, first_hi=40, Hkv=8, lens=6),
        # one page, a token a branch: latency
        dict(name="decode_page", op="decode", pages=1, prefix_lo=2048, prefix_hi=2048, br_lo=24, br_hi=24, own_hi=1024, q_hi=1,
             Hq=16, Hkv=8, ragged=True, lens=7),
        # the branch-decode workload of the benchmark, from a 4-bit cache
        dict(name="decode_16_pages", op="decode", pages=16, prefix_lo=4809, prefix_hi=4809, br_lo=8, br_hi=40, own_hi=512,
             q_hi=1, Hq=16, Hkv=8, ragged=False, lens=8),
        # a quarter of the serving workload of the benchmark
        dict(name="decode_serving", op="decode", pages=128, prefix_lo=4000, prefix_hi=6144, br_lo=8, br_hi=60, own_hi=1024,
             q_hi=1, Hq=16, Hkv=8, ragged=False, lens=9),
        # the verify workload of the benchmark: draft trees of up to 16 tokens
        dict(name="verify_64_pages", op="decode", pages=64, prefix_lo=4809, prefix_hi=4809, br_lo=8, br_hi=40, own_hi=512,
             q_hi=16, Hq=16, Hkv=8, ragged=False, lens=10),
        # one long document, one stream, eight query heads a kv head
        dict(name="decode_long", op="decode", pages=1, prefix_lo=131072, prefix_hi=131072, br_lo=1, br_hi=1, own_hi=1500,
             q_hi=1, Hq=32, Hkv=4, ragged=False, lens=11),
        # uneven pages and draft trees, four query heads a kv head
        dict(name="verify_uneven", op="decode", pages=7, prefix_lo=90, prefix_hi=2900, br_lo=1, br_hi=19, own_hi=333, q_hi=16,
             Hq=32, Hkv=8, ragged=True, lens=12),
    ]


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 8])
    lens = rng.randrange(1 << 20)
    op = rng.choice(["write", "write", "gather", "decode", "decode", "decode"])
    if op == "write":
        seqs = spread(1, 1500)
        rows = spread(1, max(1, min(5000, 120000 // seqs)))
        return dict(op=op, dtype=rng.choice(["bf16", "i4", "i4"]), seqs=seqs, rows_lo=max(1, rows // 2), rows_hi=rows,
                    prior_hi=rng.choice([0, 17, 48]), Hq=G * Hkv, Hkv=Hkv, rot=rng.choice([128, 128, 64, 32]),
                    interleaved=rng.random() < 0.3, far=rng.random() < 0.5, lens=lens)
    if op == "gather":
        hi = spread(1, 6144)
        return dict(op=op, dtype=rng.choice(["bf16", "i4", "i4"]), seqs=spread(1, 64), len_lo=max(1, hi // 2), len_hi=hi,
                    first_hi=rng.choice([0, 7, 40]), Hkv=Hkv, lens=lens)
    pages = spread(1, 64)
    prefix = spread(1, max(64, min(20000, 200000 // pages)))
    br = rng.randint(1, 40)
    return dict(op=op, pages=pages, prefix_lo=max(1, prefix // 2), prefix_hi=prefix, br_lo=1, br_hi=br,
                own_hi=rng.choice([0, 100, 512, 1024]), q_hi=rng.choice([1, 1, 7, 16]), Hq=G * Hkv, Hkv=Hkv,
                ragged=rng.random() < 0.5, lens=lens)


# ------------------------------------------------------------------ lengths (from the case alone)


def _write_lens(case):
    r = np.random.default_rng(case["lens"])
    rows = r.integers(case["rows_lo"], case["rows_hi"] + 1, size=case["seqs"])
    prior = r.integers(0, case["prior_hi"] + 1, size=case["seqs"])
    start = r.integers(4000, 6600, size=case["seqs"]) if case["far"] else prior
    return rows, prior, start


def _gather_lens(case):
    r = np.random.default_rng(case["lens"])
    lens = r.integers(case["len_lo"], case["len_hi"] + 1, size=case["seqs"])
    first = np.minimum(r.integers(0, case["first_hi"] + 1, size=case["seqs"]), lens - 1)
    return lens, first


def _decode_lens(case):
    r = np.random.default_rng(case["lens"])
    P = r.integers(case["prefix_lo"], case["prefix_hi"] + 1, size=case["pages"])
    nbr = r.integers(case["br_lo"], case["br_hi"] + 1, size=case["pages"])
    B = int(nbr.sum())
    page = np.repeat(np.arange(case["pages"]), nbr)
    back = r.integers(0, 201, size=B) if case["ragged"] else np.zeros(B, np.int64)
    fork = np.maximum(P[page] - back, 0)
    ownl = r.integers(0, case["own_hi"] + 1, size=B)
    ql = r.integers(1, case["q_hi"] + 1, size=B)
    # draft trees: node i > 0 hangs on an earlier node; reach[b, i, j]: j is i or an ancestor of i
    u = r.random((B, 16))
    parent = np.minimum((u * np.arange(16)).astype(np.int64), np.maximum(np.arange(16) - 1, 0))
    m = np.zeros((B, 16, 16), np.int64)
    m[np.arange(B)[:, None], np.arange(16)[None, :], parent] = 1
    m[:, 0, 0] = 0
    reach = (m + np.eye(16, dtype=np.int64)) > 0
    reach = (reach.astype(np.int64) @ reach) > 0
    reach = (reach.astype(np.int64) @ reach) > 0
    reach = (reach.astype(np.int64) @ reach) > 0
    reach = (reach.astype(np.int64) @ reach) > 0
    return P, nbr, page, fork, ownl, ql, reach


def _runs(n):
    """Segment number and place within the segment of each of sum(n) rows."""
    n = np.asarray(n)
    seg = np.repeat(np.arange(len(n)), n)
    return seg, np.arange(int(n.sum())) - np.repeat(np.cumsum(n) - n, n)


# ------------------------------------------------------------------ the 4-bit format in torch

_UNPERM = [0, 4, 1, 5, 2, 6, 3, 7]  # dim k of a word is its nibble _UNPERM[k]


def _quant(x):
    """Codes n [..., 128] and scales [..., 8] (f32) of x [..., 128] f32."""
    g = x.unflatten(-1, (8, 16))
    a = g.abs().amax(-1)
    a = a / torch.full_like(a, 7.0)  # a true division: borders between scales are hit exactly
    _, e = torch.frexp(a)
    quantum = torch.ldexp(torch.ones_like(a), (e - 1).clamp(min=-14) - 3)
    s = (torch.round(a / quantum) * quantum).clamp(max=MAX_SCALE)
    n = torch.where(s[..., None] > 0, torch.round(g / torch.where(s > 0, s, 1.0)[..., None]), 0.0).clamp(-7, 7)
    return n.flatten(-2), s


def _pack(x, is_k):
    """x [nb, Hkv, 16, 128] f32 -> storage [nb, Hkv, 1152] uint8."""
    n, s = _quant(x)
    w = (n + 8).to(torch.uint8).unflatten(-1, (16, 8))
    w = torch.cat([w[..., 0::2], w[..., 1::2]], -1)         # nibble order
    by = (w[..., 0::2] | (w[..., 1::2] << 4)).flatten(-2)   # [nb, Hkv, 16, 64]
    sb = (s.half().view(torch.int16) >> 7).to(torch.uint8)  # [nb, Hkv, 16, 8]
    if is_k:
        by = by.unflatten(-1, (4, 16)).transpose(2, 3)
    else:
        by = by.unflatten(-1, (8, 8)).transpose(2, 3)
        sb = sb.transpose(2, 3)
    return torch.cat([by.flatten(2), sb.flatten(2)], -1).contiguous()


def _unpack(st, is_k):
    """Storage [nb, Hkv, 1152] uint8 -> values [nb, Hkv, 16, 128] f32."""
    by, sb = st[..., :1024], st[..., 1024:]
    if is_k:
        by = by.unflatten(-1, (4, 16, 16)).transpose(2, 3).flatten(3)
        sb = sb.unflatten(-1, (16, 8))
    else:
        by = by.unflatten(-1, (8, 16, 8)).transpose(2, 3).flatten(3)
        sb = sb.unflatten(-1, (8, 16)).transpose(2, 3)
    nib = torch.stack([by & 15, by >> 4], -1).unflatten(3, (16, 4)).flatten(-2)  # [nb, Hkv, 16, 16 words, 8]
    n = nib[..., _UNPERM].flatten(-2).float() - 8.0
    s = (sb.to(torch.int16) << 7).view(torch.half).float()
    return n * s.repeat_interleave(16, -1)


# ------------------------------------------------------------------ inputs


def _rope_table(n_pos, rot, dev):
    inv = ROPE_BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()


def _cached(g, nb, Hkv, dev):
    """Keys or values of a filled pool, with a few strong channels."""
    x = torch.randn(nb, Hkv, BS, D, generator=g, device=dev) * 0.5
    return x * (1.0 + 3.0 * (torch.rand(Hkv, 1, D, generator=g, device=dev) < 0.06))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case=case)
    dt = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
    Hkv = case["Hkv"]
    if case["op"] == "write":
        rows, prior, start = _write_lens(case)
        Hq, n = case["Hq"], int(rows.sum())
        nblk = -(-(prior + rows) // BS)
        base = np.cumsum(nblk) - nblk
        nb = int(nblk.sum())
        seg, at = _runs(rows)
        slot = prior[seg] + at
        pos = start[seg] + at
        s["qkv"] = torch.randn(n, (Hq + 2 * Hkv) * D, generator=g, device=dev).to(torch.bfloat16)
        s["table"] = _rope_table(int(pos.max()) + 1, case["rot"], dev)
        s["blk"], s["slot"], s["pos"] = dt(base[seg] + slot // BS), dt(slot % BS), dt(pos)
        s["q_rot"] = torch.zeros(n, Hq, D, dtype=torch.bfloat16, device=dev)
        s["k_rot"] = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=dev)
        if case["dtype"] == "bf16":
            s["k_pool"] = torch.zeros(nb, Hkv, BS, D, dtype=torch.bfloat16, device=dev)
            s["v_pool"] = torch.zeros_like(s["k_pool"])
        else:
            s["k_pool"] = torch.zeros(nb, Hkv, UNIT, dtype=torch.uint8, device=dev)
            s["v_pool"] = torch.zeros_like(s["k_pool"])
            s["k_out"] = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=dev)
            s["v_out"] = torch.zeros_like(s["k_out"])
        if own:
            from tree_structured_shared_gb300 import padoc
            i4 = case["dtype"] == "i4"
            pool = padoc.KVPool(s["k_pool"], s["v_pool"], nb, Hkv, D, max_seqs=len(rows), max_blocks_per_seq=int(nblk.max()),
                                dtype=padoc.I4 if i4 else padoc.BF16)
            seqs = []
            for r, p in zip(rows, prior):
                q = pool.alloc(int(p))
                pool.advance(q, int(p))
                pool.reserve(q, int(r))
                seqs.append(q)
            off = np.concatenate([[0], np.cumsum(rows)])
            s["rows"] = padoc.KVRows(pool, seqs, prior, off, positions=pos if case["far"] else None)
            s["ws"] = torch.empty(s["rows"].ws_size() + 256, dtype=torch.uint8, device=dev)
            s["rows"].upload(s["ws"], s["ws"].numel())
            if i4:
                for q, r in zip(seqs, rows):
                    pool.advance(q, int(r))
                s["back"] = padoc.KVRows(pool, seqs, prior, off)
                s["ws2"] = torch.empty(s["back"].ws_size() + 256, dtype=torch.uint8, device=dev)
                s["back"].upload(s["ws2"], s["ws2"].numel())
            s["rope"] = padoc.Rope(s["table"], case["rot"], case["interleaved"])
            s["pool"], s["padoc"] = pool, padoc
    elif case["op"] == "gather":
        lens, first = _gather_lens(case)
        nblk = -(-lens // BS)
        base = np.cumsum(nblk) - nblk
        nb, n = int(nblk.sum()), int((lens - first).sum())
        seg, at = _runs(lens - first)
        slot = first[seg] + at
        s["blk"], s["slot"] = dt(base[seg] + slot // BS), dt(slot % BS)
        k, v = _cached(g, nb, Hkv, dev), _cached(g, nb, Hkv, dev)
        bf = case["dtype"] == "bf16"
        k, v = (k.to(torch.bfloat16), v.to(torch.bfloat16)) if bf else (_pack(k, True), _pack(v, False))
        s["k_pool"], s["v_pool"] = k, v
        s["k_out"] = torch.zeros(n, Hkv, D, dtype=torch.bfloat16, device=dev)
        s["v_out"] = torch.zeros_like(s["k_out"])
        if own:
            from tree_structured_shared_gb300 import padoc
            s["k_pool"], s["v_pool"] = torch.empty_like(k), torch.empty_like(v)
            pool = padoc.KVPool(s["k_pool"], s["v_pool"], nb, Hkv, D, max_seqs=len(lens), max_blocks_per_seq=int(nblk.max()),
                                dtype=padoc.BF16 if bf else padoc.I4)
            pool.sync()
            s["k_pool"].copy_(k)
            s["v_pool"].copy_(v)
            seqs = []
            for L in lens:
                seqs.append(pool.alloc(int(L)))
                pool.advance(seqs[-1], int(L))
            s["back"] = padoc.KVRows(pool, seqs, first, np.concatenate([[0], np.cumsum(lens - first)]))
            s["ws2"] = torch.empty(s["back"].ws_size() + 256, dtype=torch.uint8, device=dev)
            s["back"].upload(s["ws2"], s["ws2"].numel())
            s["pool"], s["padoc"] = pool, padoc
    else:
        P, nbr, page, fork, ownl, ql, reach = _decode_lens(case)
        Hq, B, nq = case["Hq"], len(page), int(ql.sum())
        pblk, oblk = -(-P // BS), -(-ownl // BS)
        # blocks in the order of creation: a page's prefix, then its branches' own blocks
        order = np.argsort(np.concatenate([np.arange(len(P)) * 2, page * 2 + 1]), kind="stable")
        size = np.concatenate([pblk, oblk])
        base = np.zeros(len(size), np.int64)
        base[order] = np.cumsum(size[order]) - size[order]
        nb = int(size.sum())
        k, v = _pack(_cached(g, nb, Hkv, dev), True), _pack(_cached(g, nb, Hkv, dev), False)
        s["k_pool"], s["v_pool"] = k, v
        s["q"] = torch.randn(nq, Hq, D, generator=g, device=dev).to(torch.bfloat16)
        s["k_new"] = torch.randn(nq, Hkv, D, generator=g, device=dev).mul_(0.7).to(torch.bfloat16)
        s["v_new"] = torch.randn(nq, Hkv, D, generator=g, device=dev).mul_(0.7).to(torch.bfloat16)
        br, at = _runs(ql)
        first_of_page = np.cumsum(np.bincount(page, ql, len(P)).astype(np.int64)) - np.bincount(page, ql, len(P)).astype(np.int64)
        s["base_p"], s["base_o"] = dt(base[: len(P)]), dt(base[len(P):])
        s["P"], s["fork"], s["ownl"], s["ql"] = dt(P), dt(fork), dt(ownl), dt(ql)
        s["row_br"], s["row_at"] = dt(br), dt(at)
        s["row_page"], s["row_in_page"] = dt(page[br]), dt(np.arange(nq) - first_of_page[page[br]])
        s["reach"] = dt(reach)
        s["sizes"] = (int(P.max()), max(1, int(ownl.max())), int(ql.max()), int(np.bincount(page, ql, len(P)).max()))
        bits = (reach[br, at].astype(np.int64) << np.arange(16)).sum(-1)
        bits &= (1 << ql[br]) - 1
        s["bits"] = dt(bits.astype(np.uint16).view(np.int16))
        if own:
            from tree_structured_shared_gb300 import padoc
            s["k_pool"], s["v_pool"] = torch.empty_like(k), torch.empty_like(v)
            pool = padoc.KVPool(s["k_pool"], s["v_pool"], nb, Hkv, D, max_seqs=len(P) + B,
                                max_blocks_per_seq=int(pblk.max() + oblk.max()) + 1, dtype=padoc.I4)
            pool.sync()
            s["k_pool"].copy_(k)
            s["v_pool"].copy_(v)
            ps, bs, b = [], [], 0
            for p in range(len(P)):
                ps.append(pool.alloc(int(P[p])))
                pool.advance(ps[-1], int(P[p]))
                for _ in range(nbr[p]):
                    c = pool.fork(ps[-1], int(fork[b]))
                    pool.reserve(c, int(ownl[b]))
                    pool.advance(c, int(ownl[b]))
                    bs.append(c)
                    b += 1
            batch = padoc.Batch(ps, np.concatenate([[0], np.cumsum(nbr)]), bs, np.concatenate([[0], np.cumsum(ql)]))
            s["plan"] = padoc.DecodePlan(pool, batch, Hq)
            s["ws"] = torch.empty(s["plan"].ws_size() + 256, dtype=torch.uint8, device=dev)
            s["plan"].upload(s["ws"], s["ws"].numel())
            s["o"] = torch.zeros(nq, Hq, D, dtype=torch.bfloat16, device=dev)
            s["lse"] = torch.zeros(nq, Hq, dtype=torch.float32, device=dev)
            s["pool"], s["padoc"] = pool, padoc
    return s


# ------------------------------------------------------------------ the plain forms


def _rotate(x, cs, rot, interleaved):
    """x [n, H, 128] f32, cs [n, rot] (cosines, then sines): the first rot dims turned pairwise."""
    c, sn = cs[:, None, : rot // 2], cs[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_write(s):
    case = s["case"]
    Hq, Hkv, rot = case["Hq"], case["Hkv"], case["rot"]
    x = s["qkv"].unflatten(-1, (Hq + 2 * Hkv, D))
    cs = s["table"][s["pos"]]
    q = _rotate(x[:, :Hq].float(), cs, rot, case["interleaved"])
    k = _rotate(x[:, Hq: Hq + Hkv].float(), cs, rot, case["interleaved"])
    v = x[:, Hq + Hkv:].float()
    out = dict(q_rot=q.to(torch.bfloat16), k_rot=k.to(torch.bfloat16))
    if case["dtype"] == "bf16":
        s["k_pool"][s["blk"], :, s["slot"]] = out["k_rot"]
        s["v_pool"][s["blk"], :, s["slot"]] = v.to(torch.bfloat16)
        return dict(out, k_pool=s["k_pool"], v_pool=s["v_pool"])
    (nk, sk), (nv, sv) = _quant(k), _quant(v)
    return dict(out, k_out=(nk * sk.repeat_interleave(16, -1)).to(torch.bfloat16),
                v_out=(nv * sv.repeat_interleave(16, -1)).to(torch.bfloat16))


def _plain_gather(s):
    k, v = s["k_pool"], s["v_pool"]
    if s["case"]["dtype"] == "i4":
        k, v = _unpack(k, True).to(torch.bfloat16), _unpack(v, False).to(torch.bfloat16)
    return dict(k_out=k[s["blk"], :, s["slot"]], v_out=v[s["blk"], :, s["slot"]])


def _plain_decode(s):
    case = s["case"]
    Hq, Hkv = case["Hq"], case["Hkv"]
    G = Hq // Hkv
    Pm, Om, Qm, Rm = s["sizes"]
    dev = s["q"].device
    n_p, n_b, nq = len(s["P"]), len(s["fork"]), s["q"].shape[0]
    k, v = _unpack(s["k_pool"], True), _unpack(s["v_pool"], False)  # [nb, Hkv, 16, 128]
    t_p, t_o, t_q = torch.arange(Pm, device=dev), torch.arange(Om, device=dev), torch.arange(Qm, device=dev)
    ar = lambda n: torch.arange(n, device=dev)  # noqa: E731
    last = k.shape[0] - 1
    bp = (s["base_p"][:, None] + t_p // BS).clamp(max=last)
    bo = (s["base_o"][:, None] + t_o // BS).clamp(max=last)
    kp, vp = k[bp, :, t_p % BS].transpose(1, 2), v[bp, :, t_p % BS].transpose(1, 2)  # [pages, Hkv, Pm, 128]
    ko, vo = k[bo, :, t_o % BS].transpose(1, 2), v[bo, :, t_o % BS].transpose(1, 2)  # [branches, Hkv, Om, 128]
    q = s["q"].float() * (1.0 / math.sqrt(D))
    # rows laid out by page and by branch
    qp = torch.zeros(n_p, Rm, Hq, D, device=dev)
    qp[s["row_page"], s["row_in_page"]] = q
    qb = torch.zeros(n_b, Qm, Hq, D, device=dev)
    qb[s["row_br"], s["row_at"]] = q
    kn = torch.zeros(n_b, Qm, Hkv, D, device=dev)
    vn = torch.zeros(n_b, Qm, Hkv, D, device=dev)
    kn[s["row_br"], s["row_at"]] = s["k_new"].float()
    vn[s["row_br"], s["row_at"]] = s["v_new"].float()
    heads = lambda x: x.unflatten(2, (Hkv, G)).transpose(1, 2).flatten(2, 3)  # noqa: E731  [., Hkv, rows * G, D]
    back = lambda x, rows: x.unflatten(2, (rows, G)).transpose(1, 2).flatten(2, 3)  # noqa: E731
    limit = torch.zeros(n_p, Rm, dtype=torch.int64, device=dev)
    limit[s["row_page"], s["row_in_page"]] = s["fork"][s["row_br"]]
    sp = heads(qp) @ kp.transpose(2, 3)
    sp = sp.masked_fill(t_p >= limit.repeat_interleave(G, 1)[:, None, :, None], -math.inf)
    so = heads(qb) @ ko.transpose(2, 3)
    so = so.masked_fill(t_o >= s["ownl"][:, None, None, None], -math.inf)
    sn = heads(qb) @ kn.permute(0, 2, 3, 1)
    see = s["reach"][:, :Qm, :Qm] & (t_q < s["ql"][:, None])[:, None, :]
    sn = sn.masked_fill(~see.repeat_interleave(G, 1)[:, None], -math.inf)
    # the largest score of each row over its three parts
    at_p, at_b = (s["row_page"], s["row_in_page"]), (s["row_br"], s["row_at"])
    m = torch.maximum(back(sp.amax(-1, keepdim=True), Rm)[at_p],
                      back(torch.maximum(so.amax(-1, keepdim=True), sn.amax(-1, keepdim=True)), Qm)[at_b])  # [nq, Hq, 1]
    mp = torch.zeros(n_p, Rm, Hq, 1, device=dev)
    mp[at_p] = m
    mb = torch.zeros(n_b, Qm, Hq, 1, device=dev)
    mb[at_b] = m
    ep = sp.sub_(heads(mp)).exp_()
    eo = so.sub_(heads(mb)).exp_()
    en = sn.sub_(heads(mb)).exp_()
    tot = back(ep.sum(-1, keepdim=True), Rm)[at_p] + back(eo.sum(-1, keepdim=True) + en.sum(-1, keepdim=True), Qm)[at_b]
    o = back(ep @ vp, Rm)[at_p] + back(eo @ vo + en @ vn.transpose(1, 2), Qm)[at_b]
    return dict(o=(o / tot).to(torch.bfloat16), lse=(m + tot.log())[..., 0])


def run(s):
    case = s["case"]
    if not own:
        return (_plain_write if case["op"] == "write" else _plain_gather if case["op"] == "gather" else _plain_decode)(s)
    if case["op"] == "decode":
        s["plan"].prefix_pass(s["q"], s["ws"])
        s["plan"].own_pass(s["q"], s["k_new"], s["v_new"], s["bits"], s["o"], s["lse"], s["ws"])
        return dict(o=s["o"], lse=s["lse"])
    if case["op"] == "gather":
        s["back"].gather(s["k_out"], s["v_out"], s["ws2"])
        return dict(k_out=s["k_out"], v_out=s["v_out"])
    Hq, Hkv = case["Hq"], case["Hkv"]
    x = s["qkv"]
    s["rows"].write(x[:, Hq * D:], x[:, (Hq + Hkv) * D:], s["ws"], rope=s["rope"], q=x, Hq=Hq, q_rot=s["q_rot"],
                    k_rot=s["k_rot"], q_stride=x.stride(0), k_stride=x.stride(0), v_stride=x.stride(0))
    out = dict(q_rot=s["q_rot"], k_rot=s["k_rot"])
    if case["dtype"] == "bf16":
        return dict(out, k_pool=s["k_pool"], v_pool=s["v_pool"])
    s["back"].gather(s["k_out"], s["v_out"], s["ws2"])
    return dict(out, k_out=s["k_out"], v_out=s["v_out"])


# ------------------------------------------------------------------ the work of a pass


def work(case):
    Hkv = case["Hkv"]
    if case["op"] == "write":
        rows, prior, start = _write_lens(case)
        n, Hq = int(rows.sum()), case["Hq"]
        cache = Hkv * 2 * (D * 2 if case["dtype"] == "bf16" else 72)
        span = len(np.unique(np.concatenate([np.arange(a, a + r) for a, r in zip(start, rows)])))
        b = n * (2 * Hq * D * 2 + 2 * Hkv * D * 2 + Hkv * D * 2 + cache) + span * case["rot"] * 4
        if case["dtype"] == "i4":
            b += n * (cache + Hkv * 2 * D * 2)  # and read back
        return dict(bytes=b, flops=n * (Hq + Hkv) * case["rot"] * 3)
    if case["op"] == "gather":
        lens, first = _gather_lens(case)
        n = int((lens - first).sum())
        return dict(bytes=n * Hkv * 2 * (D * 2 + (D * 2 if case["dtype"] == "bf16" else 72)), flops=n * Hkv * 2 * D)
    P, nbr, page, fork, ownl, ql, reach = _decode_lens(case)
    Hq, nq = case["Hq"], int(ql.sum())
    seen = np.zeros(len(P), np.int64)
    np.maximum.at(seen, page, fork)
    keys = int(seen.sum() + ownl.sum())
    block = sum(int(reach[b, :n, :n].sum()) for b, n in enumerate(ql))
    pairs = int((ql * (fork + ownl)).sum()) + block
    return dict(bytes=keys * Hkv * 144 + nq * (2 * Hq * D * 2 + 2 * Hkv * D * 2 + Hq * 4), flops=4.0 * D * Hq * pairs)


# ------------------------------------------------------------------ in 64 bits, from the definitions


def _scale64(dev):
    """The 256 scale bytes: exponent b >> 3 (bias 15), mantissa b & 7."""
    b = torch.arange(256, device=dev)
    e, m = (b >> 3).double(), (b & 7).double()
    return torch.where(b < 8, m * 2.0 ** -17, (1 + m / 8) * torch.pow(2.0, e - 15))


def _values64(st, is_k, toks):
    """Values [len(toks), Hkv, 128] in 64 bits of consecutive tokens `toks` (block * 16 + slot) of a storage."""
    dim = torch.arange(D, device=st.device)
    word, k = dim // 8, dim % 8
    nib = torch.where(k % 2 == 0, k // 2, 4 + k // 2)
    blk, slot = (toks // BS)[:, None], (toks % BS)[:, None]
    if is_k:
        at = (dim // 32) * 256 + slot * 16 + (word % 4) * 4 + nib // 2
        sc = 1024 + slot * 8 + dim // 16
    else:
        at = (dim // 16) * 128 + slot * 8 + (word % 2) * 4 + nib // 2
        sc = 1024 + (dim // 16) * 16 + slot
    h = torch.arange(st.shape[1], device=st.device)[None, :, None]
    code = (st[blk[:, :, None], h, at[:, None, :]].long() >> (4 * (nib % 2))) & 15
    return (code - 8).double() * _scale64(st.device)[st[blk[:, :, None], h, sc[:, None, :]].long()]


def _quant64(x):
    """Values that x [n, H, 128] (64 bits) stands for in the 4-bit format."""
    steps = _scale64(x.device)
    steps = steps[steps <= MAX_SCALE]
    g = x.reshape(x.shape[0], x.shape[1], 8, 16)
    a = g.abs().amax(-1)
    a = a / torch.full_like(a, 7)
    hi = torch.searchsorted(steps, a).clamp(max=len(steps) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - steps[lo], steps[hi] - a
    pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    s = steps[pick][..., None]
    n = torch.where(s > 0, torch.round(g / s.clamp(min=2.0 ** -20)), 0).clamp(-7, 7)
    return (n * s).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    dev, Hkv = "cuda", case["Hkv"]
    if case["op"] == "gather":
        t = s["blk"] * BS + s["slot"]
        if case["dtype"] == "bf16":
            pick = lambda p: p.double()[s["blk"], :, s["slot"]]  # noqa: E731
            return dict(k_out=pick(s["k_pool"]), v_out=pick(s["v_pool"]))
        cut = lambda p, f: torch.cat([_values64(p, f, c).float() for c in t.split(65536)])  # noqa: E731  (exact in 32 bits)
        return dict(k_out=cut(s["k_pool"], True), v_out=cut(s["v_pool"], False))
    if case["op"] == "write":
        Hq, rot = case["Hq"], case["rot"]
        n = s["qkv"].shape[0]
        out = dict(q_rot=torch.empty(n, Hq, D, device=dev), k_rot=torch.empty(n, Hkv, D, device=dev))
        kq, vq = torch.empty(n, Hkv, D, device=dev), torch.empty(n, Hkv, D, device=dev)
        for i in range(0, n, 32768):
            c = slice(i, min(n, i + 32768))
            x = s["qkv"][c].double().reshape(-1, Hq + 2 * Hkv, D)
            w = s["table"][s["pos"][c]].double()
            z = torch.complex(w[:, : rot // 2], w[:, rot // 2:])[:, None]
            qk, y = x[:, : Hq + Hkv], x[:, : Hq + Hkv].clone()
            if case["interleaved"]:
                turned = torch.complex(qk[..., 0:rot:2].contiguous(), qk[..., 1:rot:2].contiguous()) * z
                y[..., 0:rot:2], y[..., 1:rot:2] = turned.real, turned.imag
            else:
                turned = torch.complex(qk[..., : rot // 2].contiguous(), qk[..., rot // 2: rot].contiguous()) * z
                y[..., : rot // 2], y[..., rot // 2: rot] = turned.real, turned.imag
            out["q_rot"][c], out["k_rot"][c] = y[:, :Hq].float(), y[:, Hq:].float()
            if case["dtype"] == "i4":
                kq[c], vq[c] = _quant64(y[:, Hq:]).float(), _quant64(x[:, Hq + Hkv:]).float()
        if case["dtype"] == "i4":
            return dict(out, k_out=kq, v_out=vq)
        kp, vp = torch.zeros_like(s["k_pool"], dtype=torch.float32), torch.zeros_like(s["v_pool"], dtype=torch.float32)
        kp[s["blk"], :, s["slot"]] = out["k_rot"]
        vp[s["blk"], :, s["slot"]] = s["qkv"].float().reshape(n, -1, D)[:, Hq + Hkv:]
        return dict(out, k_pool=kp, v_pool=vp)
    P, nbr, page, fork, ownl, ql, reach = _decode_lens(case)
    Hq = case["Hq"]
    G = Hq // Hkv
    base_p, base_o = s["base_p"].tolist(), s["base_o"].tolist()
    o = torch.empty(len(s["q"]), Hq, D, dtype=torch.float64, device=dev)
    lse = torch.empty(len(s["q"]), Hq, dtype=torch.float64, device=dev)
    row, b = 0, 0
    tokens = lambda base, n: torch.arange(base * BS, base * BS + n, device=dev)  # noqa: E731
    for p in range(len(P)):
        kp, vp = (_values64(s[x], x[0] == "k", tokens(base_p[p], int(P[p]))) for x in ("k_pool", "v_pool"))
        kp, vp = kp.transpose(0, 1).contiguous(), vp.transpose(0, 1).contiguous()
        for _ in range(int(nbr[p])):
            n, f, L = int(ql[b]), int(fork[b]), int(ownl[b])
            r = slice(row, row + n)
            ko, vo = (_values64(s[x], x[0] == "k", tokens(base_o[b], L)).transpose(0, 1) for x in ("k_pool", "v_pool"))
            keys = torch.cat([kp[:, :f], ko, s["k_new"][r].double().transpose(0, 1)], 1)
            vals = torch.cat([vp[:, :f], vo, s["v_new"][r].double().transpose(0, 1)], 1)
            q = s["q"][r].double().reshape(n, Hkv, G, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
            sc = torch.einsum("hgnd,htd->hgnt", q, keys) / math.sqrt(D)
            hid = ~torch.from_numpy(reach[b, :n, :n]).to(dev)
            sc[..., f + L:] = sc[..., f + L:].masked_fill(hid, -math.inf)
            o[r] = torch.einsum("hgnt,htd->nhgd", torch.softmax(sc, -1), vals).reshape(n, Hq, D)
            lse[r] = torch.logsumexp(sc, -1).permute(2, 0, 1).reshape(n, Hq)
            row, b = row + n, b + 1
    return dict(o=o, lse=lse)
