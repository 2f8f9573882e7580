"""Rows handles, 4-bit pools and append_rope: host bookkeeping and refusals
that need no GPU."""
import numpy as np
import pytest

from tree_structured_shared_gb300 import padoc

PTR = 1 << 20  # an aligned address that no refused call touches


@pytest.fixture
def pool(padoc_lib):
    return padoc.KVPool(None, None, 32, 2, max_seqs=8, max_blocks_per_seq=6)


def code(fn, *a, **k):
    with pytest.raises(padoc.PadocError) as e:
        fn(*a, **k)
    return e.value.code


def test_storage_bytes(padoc_lib):
    assert padoc.kv_storage_bytes(3, 5) == 3 * 5 * 16 * 128 * 2
    assert padoc.kv_storage_bytes(3, 5, dtype=padoc.I4) == 3 * 5 * 1152
    assert code(padoc.kv_storage_bytes, 3, 5, 64) == padoc.ERR_UNSUPPORTED
    assert code(padoc.kv_storage_bytes, 3, 5, 128, padoc.F32) == padoc.ERR_UNSUPPORTED
    assert code(padoc.kv_storage_bytes, 0, 5) == padoc.ERR_INVALID
    assert code(padoc.KVPool, None, None, 4, 2, dtype=padoc.F32) == padoc.ERR_UNSUPPORTED
    padoc.KVPool(None, None, 4, 2, dtype=padoc.I4).destroy()


def test_rows_ranges(pool):
    s = pool.alloc(40)
    pool.advance(s, 40)
    rows = padoc.KVRows(pool, [s], [3], [0, 37])
    assert rows.n == 37 and rows.ws_size() == 0  # a short list rides in the launch
    assert padoc.KVRows(pool, [s], [3], [0, 37], positions=np.arange(37)).ws_size() == 4 * 37
    assert padoc.KVRows(pool, [s], None, [0, 8]).n == 8  # the reserved slots after token 40
    assert code(padoc.KVRows, pool, [s], None, [0, 9]) == padoc.ERR_INVALID
    assert code(padoc.KVRows, pool, [s], [-1], [0, 2]) == padoc.ERR_INVALID
    assert code(padoc.KVRows, pool, [s + 1], [0], [0, 2]) == padoc.ERR_INVALID
    assert code(padoc.KVRows, pool, [s], [0], [0, -1]) == padoc.ERR_INVALID
    assert code(padoc.KVRows, pool, [s], [0], [1, 2]) == padoc.ERR_INVALID
    assert code(padoc.KVRows, pool, [s], [0], [0, 2], positions=[0, -1]) == padoc.ERR_INVALID
    assert padoc.KVRows(pool, [], [], [0]).ws_size() == 0


def test_long_lists_want_a_workspace(padoc_lib):
    pool = padoc.KVPool(None, None, 400, 1, max_seqs=2, max_blocks_per_seq=400)
    s = pool.alloc(16 * 224)
    assert padoc.KVRows(pool, [s], [0], [0, 16 * 224]).ws_size() == 0
    pool.reserve(s, 16 * 225)
    rows = padoc.KVRows(pool, [s], [0], [0, 16 * 225])
    assert rows.ws_size() == 16 * 225
    assert code(rows.upload, None, 1 << 20) == padoc.ERR_INVALID
    assert code(rows.upload, PTR + 8, 1 << 20) == padoc.ERR_INVALID
    assert code(rows.upload, PTR, 16) == padoc.ERR_INVALID


def test_write_and_gather_refusals(pool):
    s = pool.alloc(16)
    rows = padoc.KVRows(pool, [s], [0], [0, 16])
    assert code(rows.write, PTR, PTR) == padoc.ERR_INVALID          # not uploaded
    assert code(rows.upload) == padoc.ERR_INVALID                   # no storage
    assert code(rows.gather, PTR, PTR) == padoc.ERR_INVALID
    w = lambda *a, **k: code(rows.write, *a, **k)  # noqa: E731
    I = padoc.ERR_INVALID
    assert w(None, PTR) == I and w(PTR, None) == I and w(PTR + 2, PTR) == I and w(PTR, PTR, k_rot=PTR + 4) == I
    assert w(PTR, PTR, k_stride=255) == I and w(PTR, PTR, v_stride=260) == I
    assert w(PTR, PTR, q=PTR, Hq=4) == I and w(PTR, PTR, q_rot=PTR, Hq=4) == I and w(PTR, PTR, q=PTR, q_rot=PTR, Hq=0) == I
    assert w(PTR, PTR, q=PTR, q_rot=PTR, Hq=4, q_stride=504) == I
    for rot, n_pos, tab in ((24, 99, PTR), (48, 99, PTR), (144, 99, PTR), (-16, 99, PTR), (128, 15, PTR), (128, 99, None), (128, 99, PTR + 4)):
        assert w(PTR, PTR, rope=padoc.Rope(tab, rot, n_pos=n_pos)) == I
    assert code(rows.gather, None, PTR) == I and code(rows.gather, PTR, PTR + 8) == I
    empty = padoc.KVRows(pool, [s], [0], [0, 0])
    empty.upload()
    empty.write(PTR, PTR)  # nothing to do
    empty.gather(None, None)


def test_append_rope_refuses_before_it_changes_anything(pool):
    a, b = pool.alloc(0), pool.alloc(0)
    before = pool.stats()
    f = lambda *x, **k: code(pool.append_rope, *x, **k)  # noqa: E731
    I = padoc.ERR_INVALID
    assert f([a, a], [0, 1, 2], PTR, PTR) == I
    assert f([a, 7], [0, 1, 2], PTR, PTR) == I
    assert f([a, b], [0, 5, 2], PTR, PTR) == I
    assert f([a], [0, 16 * 6 + 1], PTR, PTR) == I                 # above max_blocks_per_seq
    assert f([a], [0, 4], PTR, PTR) == I                          # no storage
    assert f([a], [0, 4], None, PTR) == I
    assert f([a], [0, 4], PTR, PTR, positions=[0, 1, 2, -3]) == I
    assert f([a], [0, 4], PTR, PTR, positions=[0, 1, 2, 9], rope=padoc.Rope(PTR, 128, n_pos=9)) == I
    pool.append_rope([a, b], [0, 0, 0], PTR, PTR)                  # no rows: nothing to do
    pool.append_rope([], [0], PTR, PTR)
    assert pool.stats() == before and pool.seq_info(a)["length"] == 0


def test_append_rope_out_of_blocks(padoc_lib):
    pool = padoc.KVPool(PTR, PTR, 3, 2, max_seqs=4, max_blocks_per_seq=6)
    a, b = pool.alloc(16), pool.alloc(0)
    before = pool.stats()
    assert code(pool.append_rope, [a, b], [0, 17, 50], PTR, PTR) == padoc.ERR_OOM
    assert pool.stats() == before and pool.seq_info(a) == {"length": 0, "fork_len": 0, "n_blocks": 1}
    assert code(pool.append_rope, [a], [0, 17], PTR, PTR, positions=np.zeros(17)) == padoc.ERR_INVALID  # ws too small
    assert pool.stats() == before


def test_i4_plan_workspace(padoc_lib):
    """Plans over a 4-bit pool: validated like bf16 ones; the workspace holds the partial rows."""
    pool = padoc.KVPool(None, None, 4000, 2, max_seqs=40, max_blocks_per_seq=2000, dtype=padoc.I4)
    page = pool.alloc(20000)
    pool.advance(page, 20000)
    br = [pool.fork(page, 20000) for _ in range(3)]
    batch = padoc.Batch([page], [0, 3], br, [0, 1, 2, 3])
    plan = padoc.DecodePlan(pool, batch, 4)
    assert not plan.fused()
    n = plan.ws_size()
    assert n >= 3 * 4 * 128 * 4 and n == padoc.branch_decode_ws_size(pool, batch, 4)
    assert code(padoc.DecodePlan, pool, batch, 5) == padoc.ERR_INVALID
    assert code(padoc.DecodePlan, pool, batch, 32) == padoc.ERR_UNSUPPORTED
    assert code(padoc.DecodePlan, pool, padoc.Batch([page], [0, 3], br, [0, 1, 18, 19]), 4) == padoc.ERR_INVALID
    assert padoc.DecodePlan(pool, padoc.Batch([], [0], [], [0]), 4).ws_size() == 0
