"""Counts that do not cover the table entries which name their pages: reported, and what is concerned is left out, so that no
page gets two owners unseen."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
from persistent_megakernel_streaming_gb300 import cp
from test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("refs,growing", [(1, 2), (1, 3), (2, 3), (2, 4), (3, 5)])
@pytest.mark.parametrize("others", [0, 3, 3000])
def test_more_sequences_grow_into_a_page_than_its_count(refs, growing, others):
    """All of them are left out; the others of the call grow, and so does a page's rightful number."""
    n = growing + 2 + others
    counts = np.zeros(2 * n + 16, np.int64)
    table, length = np.full((n, 3), -1), np.zeros(n, np.int64)
    g = np.random.default_rng(n)
    place = g.permutation(n)
    for i in place[:growing]:
        table[i, 0], length[i] = 7, g.integers(1, 16)
    for i in place[growing:growing + 2]:                       # a page whose two holders grow
        table[i, 0], length[i] = 9, 5
    counts[7], counts[9] = refs, 2
    b = Both(counts, table, length, 16)
    add = g.integers(1, 30, n)
    moves = b.grow(add)
    assert b.plain.bad and len(moves) == 1 and moves[0][0] == 9
    assert (b.plain.length[place[:growing]] == length[place[:growing]]).all() and b.plain.refs[7] == refs
    b.pool.clear_status()
    b.plain.bad = False
    b.grow(np.where(np.isin(np.arange(n), place[:growing]), 0, 1))     # the page was nobody's to take
    assert not b.plain.bad
    assert not (b.plain.table[place[growing:]] == 7).any()
    only = np.zeros(n, int)
    only[place[:refs]] = 1                                     # as many as it counts may grow
    b.grow(only)
    assert not b.plain.bad and (b.plain.refs[7] == 1)


def test_a_short_count_in_a_full_pool():
    """What is left out needs no pages."""
    b = Both([2, 1], [[0, -1], [0, -1], [0, -1], [1, -1]], [3, 3, 3, 16], 16)
    b.grow([20, 20, 20, 0])
    assert b.plain.bad and int(b.count) == 0


@pytest.mark.parametrize("count", [0, -1, -2 ** 31])
@pytest.mark.parametrize("place", [0, 1, 299])
def test_a_forked_page_that_nobody_holds(count, place):
    """Those that copy its sequence are left out, however many; another pair of the call stands."""
    refs, table = np.zeros(700, np.int64), np.full((8, 300), -1)
    table[0], table[1], table[2, :2] = np.arange(300), np.arange(300, 600), [600, 601]
    refs[:602] = 1
    refs[table[0, place]] = count
    b = Both(refs, table, [4800, 4799, 17, 0, 0, 0, 0, 0], 16)
    b.fork([0, 1, 0, 2], [3, 5, 4, 7])
    assert b.plain.bad and b.plain.length.tolist() == [4800, 4799, 17, 0, 0, 4799, 0, 17]
    assert b.plain.refs[table[0, place]] == count


@pytest.mark.parametrize("pages,sequences,width", [(40, 3, 8), (5000, 900, 30), (33000, 400, 30)])
@pytest.mark.parametrize("above", [False, True])
def test_a_compaction_over_pages_that_nobody_holds(pages, sequences, width, above):
    """Entries that name them, below the number held or above, stay as they are; all others follow their pages."""
    g = np.random.default_rng(pages)
    table, length, refs = np.full((sequences, width), -1), np.zeros(sequences, np.int64), np.zeros(pages, np.int64)
    order, at = g.permutation(pages), 0
    for i in range(sequences):
        k = int(g.integers(1, width + 1))
        if at + k > pages * 2 // 3:
            break
        table[i, :k], length[i] = order[at:at + k], 16 * k
        at += k
    refs[order[:at]] = 1
    short = max(2, at // 50)
    named = order[:at]
    named = (named[named >= at - short] if above else named[named < at - short])[:short]
    refs[named] = 0
    b = Both(refs, table, length, 16)
    moves = b.compact()
    assert b.plain.bad and moves and len(named) == short
    b.pool.clear_status()
    b.plain.bad = False
    stays = np.isin(table, named)
    np.testing.assert_array_equal(b.plain.table[stays], table[stays])
