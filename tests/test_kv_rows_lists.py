"""Row lists shorter than what the library reads of them are refused by the
binding, before the library sees them."""
import pytest

from tree_structured_shared_gb300 import padoc

PTR = 1 << 20


@pytest.fixture
def pool(padoc_lib):
    return padoc.KVPool(PTR, PTR, 32, 2, max_seqs=8, max_blocks_per_seq=6)


@pytest.mark.parametrize("first,offsets,positions", [
    ([0], [0, 3, 6], None), ([0, 0], [0, 3], None), (None, [0, 3], None), ([0, 0], [], None),
    ([0, 0], [0, 3, 6], [1, 2, 3, 4, 5]), ([0, 0], [0, 3, 6], []),
])
def test_short_lists(pool, first, offsets, positions):
    a, b = pool.alloc(8), pool.alloc(8)
    before = pool.stats()
    with pytest.raises(padoc.PadocError) as e:
        padoc.KVRows(pool, [a, b], first, offsets, positions=positions)
    assert e.value.code == padoc.ERR_INVALID
    if first is None or len(first) == 2:
        with pytest.raises(padoc.PadocError) as e:
            pool.append_rope([a, b], offsets, PTR, PTR, PTR, 1 << 20, positions=positions)
        assert e.value.code == padoc.ERR_INVALID
    assert pool.stats() == before and pool.seq_info(a)["length"] == 0


def test_lists_that_suffice(pool):
    a, b = pool.alloc(8), pool.alloc(8)
    rows = padoc.KVRows(pool, [a, b], [0, 2], [0, 3, 6], positions=range(7))
    assert rows.n == 6 and rows.ws_size() == 24
    assert padoc.KVRows(pool, [a, b], [0, 2, 5], [0, 3, 6, 9]).n == 6
    assert padoc.KVRows(pool, [], None, [0], positions=[]).n == 0
