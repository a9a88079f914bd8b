"""The order in which block ids leave the list and come back to it: the list's last id is taken first, and of the blocks
given back the last one is put on the list first, so that a release undoes a grow and the next grow hands the same ids
out in the same places.

The lists of test_gpu_block_tables.py put them in another order; its tests run here with lists in this one."""
import numpy as np
import pytest

import test_gpu_block_tables as tables
from test_gpu_block_tables import (i32, m, test_captured_steps_and_another_stream, test_grow_then_release,  # noqa: F401
                                   test_grow_unaligned_and_unwanted_arrays, test_ids_outside_the_pool,
                                   test_release_any_ranges, test_release_of_everything, up)

pytestmark = pytest.mark.gpu


class Stack(tables.Lists):
    def grow(self, new, nt):
        taken = sum(up(p + n, self.block) - up(p, self.block) for p, n in zip(self.past, new))
        part = slice(self.n_free - taken, self.n_free)
        self.free[part] = self.free[part][::-1].copy()
        out = super().grow(new, nt)
        self.free[part] = self.free[part][::-1].copy()
        return out

    def release(self, lo, hi):
        first = self.n_free
        bad = super().release(lo, hi)
        self.free[first:self.n_free] = self.free[first:self.n_free][::-1].copy()
        return bad


@pytest.fixture(autouse=True)
def in_this_order(monkeypatch):
    monkeypatch.setattr(tables, "Lists", Stack)


def test_ids_by_hand(m):
    """Two sequences, the first with a block of 16 rows nearly full, the second without one."""
    table = i32([[7, -1, -1, -1], [-1, -1, -1, -1]])
    free, n_free, err = i32([3, 0, 5, 1, 6, 2]), i32([6]), i32([0])
    off, pos, slot = i32([0] * 3), i32([0] * 40), i32([0] * 40)
    m.minf_block_table_grow(table, 16, 128, i32([15, 0]), i32([18, 17]), free, n_free, n_free, off, pos, slot, err)
    assert int(err) == 0 and int(n_free) == 2 and off.tolist() == [0, 18, 35]
    assert table.tolist() == [[7, 2, 6, -1], [1, 5, -1, -1]]
    rows = [7 * 16 + 15] + [2 * 16 + i for i in range(16)] + [6 * 16] + [16 + i for i in range(16)] + [5 * 16]
    assert slot.tolist() == rows + [-1] * 5
    assert pos.tolist() == list(range(15, 33)) + list(range(17)) + [-1] * 5
    # two of the first's blocks and one of the second's go back
    m.minf_block_table_release(table, 16, 128, i32([16, 16]), i32([64, 64]), free, n_free, n_free, err)
    assert int(err) == 0 and int(n_free) == 5 and free[:5].tolist() == [3, 0, 5, 6, 2]
    assert table.tolist() == [[7, -1, -1, -1], [1, -1, -1, -1]]


@pytest.mark.parametrize("n,mb", [(3, 5), (700, 30), (16384, 3)])
def test_a_release_is_undone_by_the_next_grow(m, n, mb):
    """Tables and list after a step is taken back and made again are those after it was made first."""
    r = np.random.default_rng(n)
    past = [int(x) for x in r.integers(0, mb * 8, n)]
    new = [int(x) for x in r.integers(0, mb * 8, n)]
    l = Stack(past, 16, mb, sum(up(p + c, 16) - up(p, 16) for p, c in zip(past, new)) + 3, seed=n)
    d = tables.Device(l)
    d.grow(m, new, sum(new))
    first = [x.clone() for x in (d.table, d.slot, d.n_free)]
    d.release(m, [up(p, 16) * 16 for p in past], [mb * 16] * n)
    d.grow(m, new, sum(new))
    assert int(d.err) == 0
    assert all(bool((a == b).all()) for a, b in zip(first, (d.table, d.slot, d.n_free)))


@pytest.mark.parametrize("pos", [False, True])
@pytest.mark.parametrize("slot", [False, True])
def test_ids_are_checked_whatever_arrays_are_wanted(m, pos, slot):
    """An id of the list, or the held one of a partly filled block that gets tokens, outside the pool: an error bit."""
    def grow(held=2, new=(4, 0), listed=1):
        d = tables.Device(Stack([20, 16], 16, 4, 6, seed=1))
        d.table[0, 1] = held        # rows 16 .. 19 of the first sequence
        d.free[5] = listed          # the id that is taken first
        d.table[0, 0] = d.table[1, 0] = -9  # full blocks: nobody's new rows
        d.grow(m, list(new), sum(new), pos=pos, slot=slot)
        return int(d.err)

    ok = [dict(), dict(new=(12, 0)), dict(new=(13, 0)), dict(new=(0, 3)), dict(new=(0, 3), held=-1), dict(new=(4, 0), listed=-1),
          dict(new=(0, 0), held=99, listed=99)]
    bad = [dict(held=-1), dict(held=9), dict(held=1 << 30), dict(new=(13, 0), listed=-1), dict(new=(0, 1), listed=9),
           dict(new=(0, 1), listed=-(1 << 31)), dict(new=(1, 40), held=-1)]
    assert [grow(**a) for a in ok] == [0] * len(ok)
    assert [grow(**a) for a in bad] == [m.ERRBIT_BLOCK] * len(bad)


@pytest.mark.parametrize("n", [1, 1023, 1025, 16384])
def test_the_last_sequences_held_id_is_checked(m, n):
    d = tables.Device(Stack([3] * n, 16, 1, 2, seed=n))
    for at in {0, n // 2, n - 1}:
        d.err.zero_()
        first = int(d.table[at, 0])
        d.table[at, 0] = -1
        d.grow(m, [1] * n, n, pos=False, slot=False)
        assert int(d.err) == m.ERRBIT_BLOCK
        d.table[at, 0] = first
    d.err.zero_()
    d.grow(m, [1] * n, n, pos=False, slot=False)
    assert int(d.err) == 0
