"""The block-table oracle by hand-computed steps and by what every step keeps:
no page is held twice, none is lost."""
import numpy as np
import pytest

from oracle import tables as T


def test_a_step_by_hand():
    table = np.full((3, 4), -1, np.int32)
    table[0, :2] = [7, 5]
    table[2, 0] = 3
    # request 0: 17 -> 20 tokens (no page), 1: 0 -> 33 (three pages), 2: 16 -> 17 (one)
    lens, count, out, slots, pos, off, bits = T.extend(
        [17, 0, 16], [3, 33, 1], table, [9, 8, 2, 1, 0], 5, 10, 40)
    assert lens.tolist() == [20, 33, 17] and count == 1 and bits == 0
    assert out[0].tolist() == [7, 5, -1, -1]
    assert out[1].tolist() == [0, 1, 2, -1]
    assert out[2].tolist() == [3, 8, -1, -1]
    assert off.tolist() == [0, 3, 36, 37]
    assert slots[:3].tolist() == [81, 82, 83] and pos[:3].tolist() == [17, 18, 19]
    assert slots[3] == 0 and slots[3 + 16] == 16 and slots[3 + 32] == 32
    assert slots[36] == 128 and pos[36] == 16
    assert slots[37:].tolist() == [-1] * 3 and pos[37:].tolist() == [-1] * 3


def test_the_stack_runs_out_in_order():
    table = np.full((4, 4), -1, np.int32)
    table[3, 0] = 6
    # request 1 finds one page of two: neither it nor request 2 gets any, 3 needs none
    lens, count, out, slots, pos, off, bits = T.extend(
        [0, 0, 0, 5], [16, 20, 1, 2], table, [2, 1], 2, 8, 39)
    assert lens.tolist() == [16, 0, 0, 7] and count == 1 and bits == T.SLOT_RANGE
    assert out[0, 0] == 1 and (out[1:3] == -1).all()
    assert (slots[16:37] == -1).all() and slots[37:].tolist() == [101, 102]


def test_truncate_by_hand():
    table = np.arange(12, dtype=np.int32).reshape(3, 4)
    lens, count, stack, bits = T.truncate([50, 33, 64], [32, 33, 0], table,
                                          np.full(8, -1, np.int32), 1, [0, 0, 2])
    assert lens.tolist() == [32, 33, 0] and bits == 0
    assert count == 5 and stack[:5].tolist() == [-1, 2, 3, 10, 11]


@pytest.mark.parametrize("seed", range(4))
def test_pages_are_neither_lost_nor_held_twice(seed):
    rng = np.random.default_rng(seed)
    B, W, N = 9, 8, 40
    table = np.full((B, W), -1, np.int32)
    lens, stack, count = np.zeros(B, np.int32), rng.permutation(N).astype(np.int32), N
    for _ in range(30):
        new = rng.integers(0, 40, B)
        lens, count, table, *_ = T.extend(lens, new, table, stack, count, N, 400)
        lens, count, stack, bits = T.truncate(lens, rng.integers(0, lens + 1), table, stack, count)
        assert bits == 0
        held = [int(table[s, j]) for s in range(B) for j in range(-(-int(lens[s]) // 16))]
        assert sorted(held + stack[:count].tolist()) == list(range(N))


def test_truncate_reports_pages_below_zero_where_it_pushes_them():
    table = np.array([[5, -1, 6]], np.int32)
    stack = np.zeros(4, np.int32)
    assert T.truncate([48], [10], table, stack, 0)[1] == 2
    assert T.truncate([48], [10], table, stack, 0)[3] == T.PAGE_RANGE
    assert T.truncate([48], [20], table, stack, 0)[3] == 0            # page 1 is kept
    assert T.truncate([48], [10], table, stack, 0, [2])[3] == 0       # page 1 is another's
