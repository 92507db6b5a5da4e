"""The oracle's block-table build and slot-mapped cache write, pinned: a
hand-worked step, the walk of a sequence page by page against a flat list of
its pages, exhausted and bad metadata, and the slot-mapped write against the
block-table write."""
import numpy as np
import pytest

from oracle import oracle as orc


def test_hand_worked_step():
    # block size 4; request 0: 6 positions, 3 new (held 1 page, needs 1); request 1: 4 positions,
    # none new; request 2: 9 positions, all new (needs 3)
    table = np.array([[5, -1, -1], [7, -1, -1], [-1, -1, -1]])
    t, slots, pos, end, st = orc.block_tables([6, 4, 9], [0, 3, 3, 12], table, 4, 10, 13,
                                              free_pages=[9, 0, 1, 2, 3], free_start=1)
    assert st == 0 and end == 5
    assert t.tolist() == [[5, 0, -1], [7, -1, -1], [1, 2, 3]]
    assert pos.tolist() == [3, 4, 5] + list(range(9)) + [0]
    assert slots.tolist() == [23, 0, 1, 4, 5, 6, 7, 8, 9, 10, 11, 12, -1]


def test_steps_of_a_sequence_use_its_pages_in_order():
    rng = np.random.default_rng(3)
    pages = rng.permutation(40)
    table, start, length = np.full((1, 40), -1), 0, 0
    for q in (1, 7, 16, 1, 1, 15, 33, 1):
        length += q
        table, slots, pos, start, st = orc.block_tables([length], [0, q], table, 16, 40, q,
                                                        free_pages=pages, free_start=start)
        want = [int(pages[p // 16]) * 16 + p % 16 for p in range(length - q, length)]
        assert st == 0 and slots.tolist() == want and start == -(-length // 16)


def test_free_pages_run_out_in_request_order():
    table = np.full((4, 3), -1)
    # needs 1, 2, 1, 0 (its token fits a page it holds)
    table[3, 0] = 6
    t, slots, _, end, st = orc.block_tables([4, 8, 2, 3], [0, 4, 12, 14, 15], table, 4, 8, 15,
                                            free_pages=[1, 2], free_start=0)
    assert st == orc.DEV_NO_PAGES and end == 1
    assert t[0, 0] == 1 and (t[1:3] == -1).all()
    assert slots.tolist() == [4, 5, 6, 7] + [-1] * 10 + [26]


@pytest.mark.parametrize("lens,qsl,status", [
    ([4, 4], [0, 5, 4], orc.DEV_BAD_QSL), ([4, 4], [1, 2, 4], orc.DEV_BAD_QSL),
    ([4, 4], [0, 4, 9], orc.DEV_BAD_QSL), ([2, 4], [0, 4, 8], orc.DEV_BAD_QLEN),
    ([13, 4], [0, 4, 8], orc.DEV_BAD_SEQLEN), ([-1, 4], [0, 0, 4], orc.DEV_BAD_SEQLEN),
])
def test_bad_metadata(lens, qsl, status):
    table = np.array([[0, 1, 2], [3, 4, 5]])
    _, slots, _, _, st = orc.block_tables(lens, qsl, table, 4, 8, 8)
    assert st == status
    if status == orc.DEV_BAD_QSL:
        assert (slots == -1).all()
    else:
        assert slots[:qsl[1]].tolist() == [-1] * qsl[1]
        assert slots[qsl[1]:qsl[2]].tolist() == [12 + i for i in range(4 - (qsl[2] - qsl[1]), 4)]


@pytest.mark.parametrize("layout", ["nhd", "hnd"])
def test_slot_write_is_the_block_table_write(layout):
    rng = np.random.default_rng(5)
    lens, qsl, bs, nb = [20, 3, 9], [0, 5, 5, 14], 8, 9
    table = rng.permutation(nb)[:9].reshape(3, 3)
    k, v = rng.standard_normal((2, 14, 2, 4)).astype(np.float32)
    shape = (nb, bs, 2, 4) if layout == "nhd" else (nb, 2, bs, 4)
    kc, vc = rng.standard_normal((2, *shape)).astype(np.float32)
    _, slots, _, _, st = orc.block_tables(lens, qsl, table, bs, nb, 14)
    assert st == 0
    got = orc.cache_write_slots(k, v, kc, vc, slots, bs, layout)
    want = orc.cache_write(k, v, kc, vc, table, lens, qsl, bs, layout)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and got[2] == 0
    slots[3], slots[4] = -7, nb * bs
    got = orc.cache_write_slots(k, v, kc, vc, slots, bs, layout)
    assert got[2] == orc.DEV_BAD_BLOCK
    keep = orc.nhd_view(kc, layout)[table[0, 18 // bs], 18 % bs]
    assert np.array_equal(orc.nhd_view(got[0], layout)[table[0, 18 // bs], 18 % bs], keep)
