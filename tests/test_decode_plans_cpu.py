"""CPU checks of the host-side arithmetic behind the decode step's operators
(no GPU): where the merge looks for the states of a list."""

import ctypes
import os
import random

import pytest

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

I32 = 1 << 31


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mattn.LIB_PATH):
        from block_sparse_attention_masked_gb300 import build

        build.build()
    return mattn.lib()


def _pieces(L, start, tiles, per, warps):
    f = L.mattn_internal_list_pieces
    f.argtypes, f.restype = [ctypes.c_int] * 4 + [ctypes.POINTER(ctypes.c_int)] * 2, None
    w0, n = ctypes.c_int(-1), ctypes.c_int(-1)
    f(start, tiles, per, warps, ctypes.byref(w0), ctypes.byref(n))
    return w0.value, n.value


def test_merge_finds_every_piece_of_a_list(L):
    """Lists laid end to end and dealt in equal shares, worker w taking tiles
    w * per ..: a list's pieces are the workers whose shares meet it."""
    rng = random.Random(5)
    for _ in range(200):
        warps = rng.choice((1, 6, 152, 912, 1824))
        lists = [rng.choice((1, 2, 40, rng.randint(1, 5000))) for _ in range(rng.randint(1, 40))]
        per = (sum(lists) - 1) // warps + 1
        start = 0
        for tiles in lists:
            workers = {t // per for t in (start, start + tiles - 1)} | {t // per for t in range(start, start + tiles, per)}
            assert _pieces(L, start, tiles, per, warps) == (min(workers), len(workers))
            start += tiles
    # the last list of as many tiles as 32 bits number
    assert _pieces(L, I32 - 1 - 5, 5, (I32 - 2) // 1824 + 1, 1824) == (1823, 1)


def test_merge_stays_among_the_workers_whatever_the_table_holds(L):
    """A worker that gives up a wait leaves its lists' entries unwritten: the
    merge must not read past the states then."""
    rng = random.Random(6)
    wild = [0, 1, -1, I32 - 1, -I32, 0x7F7F7F7F, -0x5A5A5A5B, 1823, 1824, 1 << 20]
    for _ in range(20000):
        start, per = (rng.choice(wild + [rng.randint(-I32, I32 - 1)]) for _ in range(2))
        tiles, warps = rng.choice((0, 1, 3, 70000, I32 - 1)), rng.choice((1, 912, 1824))
        w0, n = _pieces(L, start, tiles, per, warps)
        assert n == 0 or (0 <= w0 and 1 <= n and w0 + n <= warps), (start, tiles, per, warps)
