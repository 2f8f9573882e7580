"""The last positions of a rotation table, 2^31 - 1 among them.  Against long doubles; a value is
off by 4 2^-24 of the amplitude (three half steps of the remaining angle, the polynomial's sums,
the product), the angle by what is cut off of it, 2^-32 of a turn, and of
its step, 2^-64 of a turn times the position, and by the step's own
roundings as a double (a power and a division by 2 pi: 8 half steps at most) times the position."""
import math

import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 10, 300])
def test_last_positions(padoc_lib, n):
    import torch
    rot, base = 64, 1.0e6
    first = 2 ** 31 - n
    out = torch.full((n + 1, rot), 9.0, device="cuda")
    padoc.rope_table(out, n, rot, base, first=first)
    assert bool((out[n:] == 9).all())
    f = np.array([base ** (-2 * i / rot) for i in range(rot // 2)])
    turns = np.arange(first, first + n, dtype=np.longdouble)[:, None] * (f.astype(np.longdouble) / (2 * np.longdouble(math.pi)))[None]
    ang = ((turns - np.rint(turns)) * 2 * np.longdouble(math.pi)).astype(np.float64)
    ref = np.concatenate([np.cos(ang), np.sin(ang)], -1)
    bound = 4 * 2.0 ** -24 + 2 * math.pi * 1.5 * 2.0 ** -32 + 8 * 2.0 ** -53 * 2.0 ** 31 * np.concatenate([f, f])[None]
    assert (np.abs(out[:n].double().cpu().numpy() - ref) <= bound).all()


def test_past_the_last_one(padoc_lib):
    import torch
    out = torch.empty(4, 64, device="cuda")
    with pytest.raises(padoc.PadocError):
        padoc.rope_table(out, 2, 64, 1.0e4, first=2 ** 31 - 1)
