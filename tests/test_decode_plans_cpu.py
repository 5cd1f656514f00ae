"""CPU checks of the host-side arithmetic behind the decode step's operators
(no GPU): where the merge looks for the states of a list, how a call over a
shared prefix is split between the prefix and the sequences' own keys, and how
block lists are dealt."""

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


SMS = 152


def _shared_plan(L, B, H, Hkv, P, own, d):
    out = (ctypes.c_int * 7)()
    assert L.mattn_internal_shared_plan(B, H, Hkv, P, own, d, out) == 0
    return dict(zip(("sub", "seqs", "row_tiles", "n_split", "tiles", "per_split", "own_ctas"), out))


def _prices(plan, B, Hkv, P, own, d):
    """Microseconds of a call by the rates that the plan is made with (decode_shared.cu):
    as planned, and with a CTA of own keys on every SM behind the prefix's."""
    ctas = plan["row_tiles"] * plan["n_split"] * Hkv
    waves = -(-ctas // SMS)
    steps = waves * (plan["per_split"] * plan["sub"] + 6) + 0.02 * plan["n_split"]
    prefix = max(0.95 * steps, 4 * d * Hkv * P / 6.5e6)
    keys = 2 * d * Hkv * B * own  # bytes, the sequences half full
    after = prefix + 8 + keys / 4.5e6
    n = plan["own_ctas"]
    return (after if n >= SMS else max(prefix, 6 + keys / (n * 60e3))), after


@pytest.mark.parametrize("B,H,Hkv", [(1, 8, 1), (4, 16, 4), (16, 32, 8), (64, 32, 8), (128, 8, 8), (300, 8, 2)])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_own_keys_get_their_share_of_the_machine(L, B, H, Hkv, d):
    """Own keys are kept to SMs of their own only where that is no slower than a
    CTA of them on every SM, by the plan's own rates; a long prefix and few own
    keys still run beside each other."""
    beside = 0
    for P in (1, 100, 512, 1024, 2048, 2304, 2560, 4096, 8192, 16384, 131071):
        for own in (1, 64, 512, 4096, 16384, 100000):
            if 4 * d * Hkv * B * own > 1e11:
                continue
            plan = _shared_plan(L, B, H, Hkv, P, own, d)
            assert 8 <= plan["own_ctas"] <= SMS
            ctas = plan["row_tiles"] * plan["n_split"] * Hkv
            planned, after = _prices(plan, B, Hkv, P, own, d)
            assert planned <= after * (1 + 1e-6), (P, own, plan)
            if plan["own_ctas"] < SMS:
                assert ctas + plan["own_ctas"] <= SMS, (P, own, plan)
                beside += 1
    assert beside


@pytest.mark.parametrize("P", [512, 1024, 2048, 2304, 2560, 4096])
def test_long_own_keys_behind_a_short_prefix_take_most_of_the_machine(L, P):
    """64 sequences of 16,384 own keys hold more than 99% of the bytes."""
    assert _shared_plan(L, 64, 32, 8, P, 16384, 128)["own_ctas"] >= SMS // 2


@pytest.mark.parametrize("d,block,top_k", [(64, 64, 32), (128, 64, 16), (128, 64, 64), (256, 16, 64), (256, 64, 128)])
def test_block_lists_do_not_wait_for_a_wave_of_a_few(L, d, block, top_k):
    """More groups than places of one wave (two CTAs an SM): clusters only where
    the groups fill five sevenths of the waves' places."""
    out = (ctypes.c_int * 2)()
    seen = set()
    for groups in [*range(1, 1300), 5000, 65535]:
        assert L.mattn_internal_list_plan(groups, 4, 1, top_k, block, d, out) == 0
        cluster, warps = out
        assert cluster in (0, 1, 2, 4, 8) and warps >= 1
        seen.add(cluster)
        places = -(-groups // (2 * SMS)) * 2 * SMS
        if groups > 2 * SMS:
            assert (cluster == 0) == (places * 5 > groups * 7), groups
        elif groups > SMS:
            assert cluster == 1
    assert {0, 1} <= seen
