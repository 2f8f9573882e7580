"""Outputs of a row write that lie on rows the call reads: only an output on
its own dense input is taken.  Host checks; a call that passes them stops at
the next one (the rows were not uploaded), so no address is touched."""
import itertools

import pytest

from tree_structured_shared_gb300 import padoc

A = 1 << 20
HKV, HQ, D, N = 2, 4, 128, 5
ROW, QROW = HKV * D, HQ * D          # elements
W = QROW + 2 * ROW                   # of a fused projection's row


@pytest.fixture
def pool(padoc_lib):
    return padoc.KVPool(None, None, 32, HKV, max_seqs=8, max_blocks_per_seq=6)


def refused(pool, n=N, **step):
    """Whether the step is refused for an overlap, by the write and by append_rope."""
    s = pool.alloc(n)
    rows = padoc.KVRows(pool, [s], [0], [0, n])
    out = []
    for call in (lambda k, v, **kw: rows.write(k, v, **kw), lambda k, v, **kw: pool.append_rope([s], [0, n], k, v, **kw)):
        kw = dict(step)
        with pytest.raises(padoc.PadocError) as e:
            call(kw.pop("k"), kw.pop("v"), **kw)
        assert e.value.code == padoc.ERR_INVALID
        out.append("overlap" in str(e.value))
    rows.free()
    pool.release(s)
    assert out[0] == out[1]
    return out[0]


def fused(**more):
    """q, k, v as slices of one projection at A."""
    s = dict(q=A, Hq=HQ, q_stride=W, k=A + 2 * QROW, v=A + 2 * (QROW + ROW), k_stride=W, v_stride=W, q_rot=A + (1 << 18))
    s.update(more)
    return s


def dense(**more):
    s = dict(q=A, Hq=HQ, k=A + (1 << 16), v=A + (1 << 17), q_rot=A + (1 << 18))
    s.update(more)
    return s


def test_in_place_on_strided_rows(pool):
    assert refused(pool, **fused(q_rot=A))
    assert refused(pool, **fused(k_rot=A + 2 * QROW))
    # one row has no next one to lie on; its outputs end where the next slice starts
    assert not refused(pool, n=1, **fused(q_rot=A, k_rot=A + 2 * QROW))


def test_in_place_on_dense_rows(pool):
    assert not refused(pool, **dense(q_rot=A, k_rot=A + (1 << 16)))
    assert refused(pool, **dense(q_rot=A + 16))
    assert refused(pool, **dense(q_rot=A - 16))
    assert refused(pool, **dense(k_rot=A + (1 << 16) + 2 * ROW))


def test_outputs_on_other_rows(pool):
    assert not refused(pool, **dense()) and not refused(pool, **fused(k_rot=A + (1 << 19)))
    assert refused(pool, **dense(k_rot=A)) and refused(pool, **dense(k_rot=A + (1 << 17)))
    assert refused(pool, **dense(q_rot=A + (1 << 16))) and refused(pool, **dense(q_rot=A + (1 << 17)))
    assert refused(pool, **dense(k_rot=A + (1 << 18)))  # on each other
    assert not refused(pool, **dense(k_rot=A + (1 << 18) + 2 * N * QROW))


def test_against_every_byte(pool):
    """Outputs around strided rows with room for one output row between them, byte by byte."""
    stride = 3 * ROW
    base = dict(k=A, v=A + (1 << 19), k_stride=stride)
    for n, off in itertools.product((1, 2, 3), range(-4 * 2 * ROW, (3 * 3 + 1) * 2 * ROW, ROW // 2)):
        out = range(A + off, A + off + n * 2 * ROW)
        hit = any(max(out.start, A + i * 2 * stride) < min(out.stop, A + i * 2 * stride + 2 * ROW) for i in range(n))
        want = hit and not (off == 0 and n == 1)
        assert refused(pool, n=n, **base, k_rot=A + off) == want, (n, off)
