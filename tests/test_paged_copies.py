"""How the paged attention divides a tile's blocks into copies (on the host, by
the functions the kernel calls): every block that is there is copied once, from
its own place, and the copies' bytes are those the tile waits for."""
import itertools

import pytest

from test_abi import _lib


def copied(at):
    """For each block of the tile the place its bytes come from, None where no copy lands."""
    _lib()
    from ternary_weight_decode_b200 import tern
    got = [None] * 8
    for j, size in enumerate(tern.tern_debug_paged_copies(at)):
        if size < 0:
            continue
        assert size <= 3 and j % (1 << size) == 0
        for i in range(1 << size):
            assert got[j + i] is None, (at, "two copies of one block")
            got[j + i] = at[j] + i
    return got


def check(at):
    assert copied(at) == [a if a >= 0 else None for a in at], at


def test_missing_blocks_before_the_cache_s_first():
    for at in ([-1, 0], [-1, 0, 7, 9], [-1, 0, 1, 2, 3, 4, 5, 6], [5, 6, 7, -1, 0, 1, 2, 3], [8, -1, -1, 0, 1, -1, 0, 1],
               [3, 4, 5, 6, -1, 0, 1, 2]):
        check(at + [-1] * (8 - len(at)))


def test_every_pattern_of_missing_following_and_jumping_blocks():
    """Each block is missing, behind its predecessor (of a missing one: place 0), or elsewhere."""
    for steps in itertools.product("mfj", repeat=8):
        for start in (0, 41):
            at, last = [], start - 1
            for i, s in enumerate(steps):
                last = -1 if s == "m" else last + 1 if s == "f" else 100 * (i + 1)
                at.append(last)
            check(at)


def test_runs_are_copied_together():
    _lib()
    from ternary_weight_decode_b200 import tern
    for at, want in (([0, 1, 2, 3, 4, 5, 6, 7], [3] + [-1] * 7), ([9, 4, 5, 6, 20, 21, 22, 23], [0, 0, 1, -1, 2, -1, -1, -1]),
                     ([4, 5, 6, 7, -1, -1, -1, -1], [2] + [-1] * 7), ([7, 6, 5, 4, 3, 2, 1, 0], [0] * 8)):
        assert tern.tern_debug_paged_copies(at) == want


@pytest.mark.parametrize("at,size", [(None, 4096), (4096, None)])
def test_null_pointers_are_refused(at, size):
    assert _lib().tern_debug_paged_copies(at, size) == 1


@pytest.mark.parametrize("cycles", [-1, 10 ** 9 + 1])
def test_wait_budgets_out_of_range_are_refused(cycles):
    assert _lib().tern_debug_paged_wait_budget(cycles) == 1
