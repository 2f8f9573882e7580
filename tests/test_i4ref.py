"""The 4-bit format's reference, pinned by hand-worked values and by its own
definition searched exhaustively (CPU only)."""
import numpy as np
import pytest

import i4ref


def test_scale_bytes_are_the_upper_bits_of_fp16():
    sv = i4ref.scale_values()
    assert sv[0] == 0 and sv[1] == 2.0 ** -17 and sv[7] == 7 * 2.0 ** -17 and sv[8] == 2.0 ** -14
    assert sv[0xC6] == 896.0 and np.isnan(sv[0xFF])
    assert np.all(np.diff(sv[:0xF8]) > 0)


@pytest.mark.parametrize("seed", range(3))
def test_quantise_is_nearest(seed):
    """Every scale is the nearest of all scales to max / 7 and every code the nearest integer to x / s."""
    rng = np.random.default_rng(seed)
    x = rng.normal(size=(40, 128)) * 2.0 ** rng.integers(-22, 14, size=(40, 1))
    n, b = i4ref.quantise(x)
    sv = i4ref.scale_values()[:0xC7]
    a = np.abs(x.reshape(40, 8, 16)).max(-1) / 7
    d = np.abs(sv - a[..., None])
    assert np.array_equal(sv[b], np.where(a > 896, 896, sv[d.argmin(-1)]))
    s = np.repeat(sv[b], 16, axis=-1)
    ok = s > 0
    assert np.all(np.abs(x - n * s)[ok] <= (s / 2 + np.maximum(np.abs(x) - 7.5 * s, 0) + 1e-12 * s)[ok])
    assert np.all(n[~ok] == 0) and np.abs(n).max() <= 7


def test_ties_and_limits():
    x = np.zeros((4, 128))
    x[0, 0], x[0, 1], x[0, 2] = 7.0, 0.5, 1.5       # s = 1: ties go to even codes
    x[1, 16:32] = 1e5                                # saturates at 7 * 896
    x[2, 0] = 7 * 2.0 ** -18                         # a tie between scale 0 and 2^-17: to even, zero
    x[3, 0] = 7 * 1.0625                             # a tie between 1.0 and 1.125: to even mantissa, 1.0
    k, v = i4ref.stored(x[:, None], x[:, None])
    k = k[:, 0]
    assert list(k[0, :3]) == [7.0, 0.0, 2.0]
    assert np.all(k[1, 16:32] == 6272.0) and np.all(k[2] == 0)
    n, b = i4ref.quantise(x)
    assert i4ref.scale_values()[b[3, 0]] == 1.0 and n[3, 0] == 7


def test_poisoned_tokens():
    k, v = np.ones((3, 2, 128)), np.ones((3, 2, 128))
    k[0, 1, 70], v[2, 0, 5] = np.inf, np.nan
    ks, vs = i4ref.stored(k, v)
    for t, h in ((0, 1), (2, 0)):
        assert np.isnan(ks[t, h, :16]).all() and (ks[t, h, 16:] == 0).all() and (vs[t, h] == 0).all()
    assert np.isfinite(ks[1]).all() and np.isfinite(vs).all()


def test_rotation_is_a_rotation():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(5, 3, 128))
    for rot in (16, 48, 128):
        cs = i4ref.rope_table(9, rot)[[0, 3, 8, 1, 1]]
        for il in (False, True):
            y = i4ref.rotate(x, cs, rot, il)
            assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-6)
            assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., rot:], x[..., rot:])
    # one pair by hand: position 1, pair 0 turns by one radian
    cs = i4ref.rope_table(2, 16)[[1]]
    e = np.zeros((1, 1, 128))
    e[0, 0, 0] = 1
    y = i4ref.rotate(e, cs, 16, False)[0, 0]
    assert abs(y[0] - np.cos(1)) < 1e-7 and abs(y[8] - np.sin(1)) < 1e-7
    y = i4ref.rotate(e, cs, 16, True)[0, 0]
    assert abs(y[0] - np.cos(1)) < 1e-7 and abs(y[1] - np.sin(1)) < 1e-7
