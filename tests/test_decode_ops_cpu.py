"""CPU checks of the decode step's operators: what they refuse on the host
before any launch, and the host-side plans behind the workspace queries.
The pointers passed here are never read: every call is refused first."""

import ctypes
import os

import pytest

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

P16, P256 = 1 << 20, 1 << 21  # stand-ins for aligned device addresses


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mattn.LIB_PATH):
        from block_sparse_attention_masked_gb300 import build

        build.build()
    return mattn.lib()


def _rope_desc(**kw):
    d = mattn.RopeDesc()
    d.n_axes = 2
    d.sections[0], d.sections[1] = 32, 32
    d.eps = 1e-6
    d.inv_freq = P16
    for i in range(3):
        d.token_stride[i], d.batch_stride[i] = 1024, 65536
    for k, v in kw.items():
        if isinstance(v, tuple):
            for i, x in enumerate(v):
                getattr(d, k)[i] = x
        else:
            setattr(d, k, v)
    return d


ROPE = dict(q=P16, k=P16, v=P16, q_out=P16, k_out=P16, v_out=P16, positions=None, starts=None, lens=None, B=2, H=8,
            H_kv=2, N=64, L=64, d=128, dtype=0)


@pytest.mark.parametrize("why,args,desc,code", [
    ("no queries", {"q": None}, {}, -1),
    ("values without their output", {"v_out": None}, {}, -1),
    ("output without values", {"v": None}, {}, -1),
    ("no tokens", {"N": 0}, {}, -1),
    ("no cache rows", {"L": 0}, {}, -1),
    ("head dim 48", {"d": 48}, {}, -2),
    ("unknown type", {"dtype": 2}, {}, -2),
    ("rows off a 16-byte boundary", {"q": P16 + 8}, {}, -2),
    ("positions off a 4-byte boundary", {"positions": P16 + 2}, {}, -1),
    ("four axes", {}, {"n_axes": 4}, -1),
    ("no axis", {}, {"n_axes": 0}, -1),
    ("a negative section", {}, {"sections": (-8, 32, 0)}, -1),
    ("more pairs than d / 2", {}, {"sections": (40, 32, 0)}, -1),
    ("pairs no multiple of 8", {}, {"sections": (20, 20, 0), "n_axes": 1}, -2),
    ("no frequencies", {}, {"inv_freq": None}, -1),
    ("eps < 0", {}, {"eps": -1.0}, -1),
    ("eps NaN", {}, {"eps": float("nan")}, -1),
    ("stride < 0", {}, {"token_stride": (-1024, 1024, 1024)}, -1),
    ("stride off 16 bytes", {}, {"token_stride": (1024, 1020, 1024)}, -2),
    ("more than 2^30 tokens", {"B": 1 << 16, "N": 1 << 15}, {}, -2),
])
def test_qk_rope_refuses(L, why, args, desc, code):
    a = dict(ROPE, **args)
    rc = L.mattn_qk_rope(a["q"], a["k"], a["v"], a["q_out"], a["k_out"], a["v_out"], a["positions"], a["starts"],
                         a["lens"], a["B"], a["H"], a["H_kv"], a["N"], a["L"], a["d"], a["dtype"],
                         ctypes.byref(_rope_desc(**desc)), None)
    assert rc == code, why
    assert L.mattn_last_error()


# q [2][64][8][128] bf16 with token stride 1024 and batch stride 65536: 256 KB; k and v 64 KB each
APART = dict(ROPE, q=1 << 24, k=2 << 24, v=3 << 24, q_out=4 << 24, k_out=5 << 24, v_out=6 << 24)


@pytest.mark.parametrize("why,args", [
    ("queries in place", {"q_out": 1 << 24}),
    ("an output that begins in the last row of q", {"k_out": (1 << 24) + 262144 - 256}),
    ("an output that ends in the first row of v", {"k_out": (3 << 24) - 65536 + 256}),
    ("one cache for keys and values", {"v_out": 5 << 24}),
    ("a value cache that ends in the queries' output", {"v_out": (4 << 24) - 65536 + 256}),
    ("a long cache that reaches the next one", {"L": 1 << 20}),
])
def test_qk_rope_refuses_overlaps(L, why, args):
    """Rows are read and written in no order: an output over an input would be read half written."""
    a = dict(APART, **args)
    rc = L.mattn_qk_rope(a["q"], a["k"], a["v"], a["q_out"], a["k_out"], a["v_out"], None, None, None, a["B"], a["H"],
                         a["H_kv"], a["N"], a["L"], a["d"], 0, ctypes.byref(_rope_desc()), None)
    assert rc == mattn.ERR_INVALID_ARG, why
    assert b"overlaps" in L.mattn_last_error()


def test_qk_rope_refuses_a_null_descriptor(L):
    a = ROPE
    rc = L.mattn_qk_rope(a["q"], a["k"], a["v"], a["q_out"], a["k_out"], a["v_out"], None, None, None, 2, 8, 2, 64, 64,
                         128, 0, None, None)
    assert rc == mattn.ERR_INVALID_ARG


HEADS = [
    ("H no multiple of H_kv", {"H": 9}, -1),
    ("no head", {"H": 0}, -1),
    ("no sequence", {"B": 0}, -1),
    ("17 query heads per key/value head", {"H": 34}, -2),
    ("head dim 96", {"d": 96}, -2),
    ("fp32", {"dtype": 1}, -2),
    ("B * H_kv past the grid", {"B": 40000}, -2),
]


def _shared(lib, **kw):
    a = dict(q=P16, kp=P16, vp=P16, k=P16, v=P16, o=P16, lse=P16, lens=None, B=2, H=8, H_kv=2, P=100, P_cap=128, L=64,
             d=128, dtype=0, sink=None, scale=0.0, ws=P256, ws_bytes=1 << 40)
    a.update(kw)
    return lib.mattn_decode_shared(a["q"], a["kp"], a["vp"], a["k"], a["v"], a["o"], a["lse"], a["lens"], a["B"], a["H"],
                                 a["H_kv"], a["P"], a["P_cap"], a["L"], a["d"], a["dtype"], a["sink"], a["scale"],
                                 a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("why,args,code", HEADS + [
    ("no output", {"o": None}, -1),
    ("no prefix keys", {"kp": None}, -1),
    ("no own values", {"v": None}, -1),
    ("P < 0", {"P": -1}, -1),
    ("P past its capacity", {"P": 129}, -1),
    ("L < 0", {"L": -1}, -1),
    ("own keys past 2^31 tiles", {"B": 64, "L": 1 << 30}, -2),
    ("unaligned prefix", {"kp": P16 + 8}, -2),
    ("scale < 0", {"scale": -1.0}, -1),
    ("scale infinite", {"scale": float("inf")}, -1),
    ("no workspace", {"ws": None}, -6),
    ("a small workspace", {"ws_bytes": 1000}, -6),
    ("an unaligned workspace", {"ws": P256 + 16}, -1),
    ("unaligned lengths", {"lens": P16 + 2}, -1),
])
def test_decode_shared_refuses(L, why, args, code):
    assert _shared(L, **args) == code, why


def _select(lib, **kw):
    a = dict(q=P16, m=P16, lens=None, ids=P16, B=2, H=8, H_kv=2, n=100, d=128, dtype=0, block=64, k=8, first=1,
             recent=1, ws=P256, ws_bytes=1 << 40)
    a.update(kw)
    return lib.mattn_decode_select(a["q"], a["m"], a["lens"], a["ids"], a["B"], a["H"], a["H_kv"], a["n"], a["d"],
                                 a["dtype"], a["block"], a["k"], a["first"], a["recent"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("why,args,code", HEADS + [
    ("no blocks", {"n": 0}, -1),
    ("more blocks than supported", {"n": 32769}, -2),
    ("top_k 0", {"k": 0, "first": 0, "recent": 0}, -1),
    ("more kept than chosen", {"k": 4, "first": 3, "recent": 2}, -1),
    ("kept counts that overflow", {"k": 4, "first": 2147483647, "recent": 2147483647}, -1),
    ("negative keep", {"first": -1}, -1),
    ("block 0", {"block": 0}, -1),
    ("unaligned means", {"m": P16 + 8}, -2),
    ("a small workspace", {"ws_bytes": 16}, -6),
])
def test_decode_select_refuses(L, why, args, code):
    assert _select(L, **args) == code, why


def _blocks(lib, **kw):
    a = dict(q=P16, k=P16, v=P16, o=P16, lse=None, lens=None, ids=P16, B=2, H=8, H_kv=2, L=512, d=128, dtype=0,
             block=64, top_k=8, sink=None, scale=0.0, ws=P256, ws_bytes=1 << 40)
    a.update(kw)
    return lib.mattn_decode_blocks(a["q"], a["k"], a["v"], a["o"], a["lse"], a["lens"], a["ids"], a["B"], a["H"],
                                 a["H_kv"], a["L"], a["d"], a["dtype"], a["block"], a["top_k"], a["sink"], a["scale"],
                                 a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("why,args,code", HEADS + [
    ("no list", {"ids": None}, -1),
    ("an empty list", {"top_k": 0}, -1),
    ("block 24", {"block": 24}, -2),
    ("block 8", {"block": 8}, -2),
    ("no cache", {"L": 0}, -1),
    ("a list past 2^30 keys", {"top_k": 1 << 20, "block": 2048}, -2),
    ("a block past 2^20 keys", {"block": (1 << 20) + 16, "top_k": 1}, -2),
    ("a small workspace", {"top_k": 2000, "ws_bytes": 16}, -6),
])
def test_decode_blocks_refuses(L, why, args, code):
    assert _blocks(L, **args) == code, why


@pytest.mark.parametrize("why,args,code", [
    ("no means", {"m": None}, -1),
    ("block 8", {"block": 8}, -2),
    ("no new key", {"new": 0}, -1),
    ("head dim 80", {"d": 80}, -2),
    ("fp32", {"dtype": 1}, -2),
    ("no cache", {"L": 0}, -1),
])
def test_block_means_refuses(L, why, args, code):
    a = dict(k=P16, m=P16, lens=None, first=None, B=2, H_kv=2, L=512, d=128, dtype=0, block=64, new=1)
    a.update(args)
    rc = L.mattn_block_means(a["k"], a["m"], a["lens"], a["first"], a["B"], a["H_kv"], a["L"], a["d"], a["dtype"],
                             a["block"], a["new"], None)
    assert rc == code, why


def test_workspace_queries(L):
    """Sizes of every kind have a workspace, with room for at least one state
    per query row where there is one, and bad sizes are refused."""
    n = ctypes.c_size_t(0)
    for B, H, H_kv in ((1, 1, 1), (3, 6, 2), (64, 32, 8), (300, 16, 1)):
        for d in (64, 128, 256):
            for P, own in ((0, 0), (0, 5), (1, 0), (129, 1), (32768, 512), (1 << 20, 70000)):
                assert L.mattn_decode_shared_workspace(B, H, H_kv, P, own, d, ctypes.byref(n)) == 0
                states = (P > 0) + (own > 0)
                assert states * B * H * (d + 2) * 4 <= n.value < (600 * B * H + 2000 * H // H_kv) * (d + 64) * 4 + 8192
            for top_k, block in ((1, 16), (64, 64), (1000, 48)):
                assert L.mattn_decode_blocks_workspace(B, H, H_kv, top_k, block, d, ctypes.byref(n)) == 0
            for blocks in (1, 33, 32768):
                assert L.mattn_decode_select_workspace(B, H, H_kv, blocks, d, ctypes.byref(n)) == 0
                assert n.value >= 16 * B * H_kv * blocks
    assert L.mattn_decode_shared_workspace(1, 8, 3, 10, 10, 128, ctypes.byref(n)) == mattn.ERR_INVALID_ARG
    assert L.mattn_decode_shared_workspace(1, 8, 2, 10, 10, 128, None) == mattn.ERR_INVALID_ARG
    assert L.mattn_decode_select_workspace(1, 8, 2, 40000, 128, ctypes.byref(n)) == mattn.ERR_UNSUPPORTED


def test_descriptor_layout_matches_the_header():
    # 4 + 12 + 4 + 4, three pointers, six 64-bit strides
    assert ctypes.sizeof(mattn.RopeDesc) == 24 + 3 * 8 + 6 * 8
    assert mattn.RopeDesc.eps.offset == 20
    assert mattn.RopeDesc.token_stride.offset == 48


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    q, c = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mattn.decode_shared(q, c[0], c[0], c, c)
    with pytest.raises(ValueError):
        mattn.decode_select(q, c, 16, 1)
    with pytest.raises(ValueError):
        mattn.decode_blocks(q, c, c, torch.zeros(1, 1, 1, dtype=torch.int32), 16)
    with pytest.raises(ValueError):
        mattn.block_means(c, 16)
    with pytest.raises(ValueError):
        mattn.RopePlan(torch.zeros(32))
