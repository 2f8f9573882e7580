"""Plain references of the paged-cache operators, in NumPy float64 on the host:
the 4-bit format (encode, decode, storage layout) and the position rotation.
Written from the format's description; shares no code with the library."""
import numpy as np

MAX_SCALE = 896.0
UNIT = 1152


def scale_values():
    """The value of each scale byte below the poisoned one: bits 14..7 of an fp16 number."""
    with np.errstate(invalid="ignore"):
        return (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)


def quantise(x):
    """x [..., 128] -> integer codes n in [-7, 7] [..., 128] and scale bytes [..., 8]; groups with a
    non-finite value are the caller's to handle."""
    x = np.asarray(x, np.float64)
    g = x.reshape(x.shape[:-1] + (8, 16))
    a = np.minimum(np.abs(g).max(-1) / 7.0, MAX_SCALE)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -14)))
    q = 2.0 ** (e - 3)
    s = np.rint(a / q) * q  # half to even
    n = np.clip(np.rint(g / np.where(s > 0, s, 1.0)[..., None]), -7, 7) * (s > 0)[..., None]
    return n.reshape(x.shape).astype(np.int64), (s.astype(np.float16).view(np.uint16) >> 7).astype(np.uint8)


def stored(k, v):
    """What the rows k, v [n, Hkv, 128] read back as: (k', v') float64.  A token with a non-finite value in its K or V
    of a head has NaN in K's first group and zeros everywhere else."""
    sv = scale_values()
    bad = ~(np.isfinite(k).all(-1) & np.isfinite(v).all(-1))  # [n, Hkv]
    out = []
    for x in (k, v):
        n, b = quantise(np.where(bad[..., None], 0.0, x))
        out.append(n * np.repeat(sv[b], 16, axis=-1))
    out[0][bad, :16] = np.nan
    return out[0], out[1]


def unpack(unit, is_k):
    """The 16 x 128 values of one (block, kv head): unit [1152] uint8 -> [16, 128] float64."""
    sv = scale_values()
    out = np.zeros((16, 128))
    for t in range(16):
        for d in range(128):
            w, k = d // 8, d % 8
            nib = k // 2 if k % 2 == 0 else 4 + k // 2
            at = (256 * (d // 32) + 16 * t + 4 * (w % 4) if is_k else 128 * (d // 16) + 8 * t + 4 * (w % 2)) + nib // 2
            code = (int(unit[at]) >> (4 * (nib % 2))) & 15
            s = unit[1024 + 8 * t + d // 16] if is_k else unit[1024 + 16 * (d // 16) + t]
            out[t, d] = (code - 8) * sv[s]
    return out


def rope_table(n_pos, rot, base=1.0e4):
    ang = np.arange(n_pos)[:, None] * base ** (-np.arange(0, rot, 2) / rot)
    return np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rotate(x, cs, rot, interleaved):
    """x [n, H, 128], cs [n, rot] -> float64, the first rot dims turned pairwise."""
    y = np.asarray(x, np.float64).copy()
    c, s = (np.asarray(t, np.float64)[:, None] for t in (cs[:, : rot // 2], cs[:, rot // 2: rot]))
    ia = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia].copy(), y[..., ib].copy()
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    return y
