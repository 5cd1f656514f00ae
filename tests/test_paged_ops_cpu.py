"""CPU checks of the operators around a paged cache: what they refuse on the host
before any launch.  The pointers passed here are never read: every call is refused
first, or reaches the check of the device (there is none here)."""

import ctypes
import os

import pytest

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

MB = 1 << 20
BF16, F32, E4M3 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(mattn.LIB_PATH):
        from block_sparse_attention_masked_gb300 import build

        build.build()
    return mattn.lib()


def _cache(e4m3=False, n_pages=10, H_kv=2, page=16, d=128, **kw):
    """Dense pages of k at 256 MB and v at 512 MB, their exponents at 768 and 800 MB."""
    c = mattn.PagedCache()
    c.k, c.v = 256 * MB, 512 * MB
    if e4m3:
        c.k_exponents, c.v_exponents = 768 * MB, 800 * MB
    for i in range(2):
        c.page_stride[i], c.head_stride[i], c.row_stride[i] = H_kv * page * d, page * d, d
        c.exp_page_stride[i], c.exp_head_stride[i], c.exp_row_stride[i] = H_kv * page, page, 1
    c.page_table, c.table_pages, c.n_pages, c.page, c.dtype = 900 * MB, 4, n_pages, page, E4M3 if e4m3 else BF16
    for k, v in kw.items():
        if isinstance(v, tuple):
            for i, x in enumerate(v):
                getattr(c, k)[i] = x
        else:
            setattr(c, k, v)
    return c


def _two(a, b):
    return (ctypes.c_int64 * 2)(a, b)


CACHE = [
    ("no keys", {"k": None}, -1),
    ("no values", {"v": None}, -1),
    ("no page table", {"page_table": None}, -1),
    ("an unknown type", {"dtype": F32}, -2),
    ("codes without exponents", {"dtype": E4M3}, -1),
    ("bf16 with exponents", {"k_exponents": MB, "v_exponents": MB}, -1),
    ("pages of 8 rows", {"page": 8}, -2),
    ("pages of 24 rows", {"page": 24}, -2),
    ("an empty table", {"table_pages": 0}, -1),
    ("no pages", {"n_pages": 0}, -1),
    ("a table of more than 2^30 positions", {"table_pages": (1 << 26) + 1}, -2),
    ("keys off a 16-byte boundary", {"k": 256 * MB + 8}, -2),
    ("a table off a 4-byte boundary", {"page_table": 900 * MB + 2}, -2),
    ("a stride off 16 bytes", {"row_stride": (132, 128)}, -2),
    ("a stride of zero", {"head_stride": (0, 2048)}, -2),
    ("a negative stride", {"page_stride": (4096, -4096)}, -2),
    ("a stride of 2^40 bytes", {"page_stride": (4096, 1 << 39)}, -2),
    ("rows that overlap", {"row_stride": (64, 128)}, -1),
    ("heads that overlap", {"head_stride": (1920, 2048)}, -1),
    ("pages that overlap", {"page_stride": (4096, 3968)}, -1),
]


def _write(L, cache, k=MB, v=100 * MB, token=(256, 256), head=(128, 128), cu=None, starts=None, B=3, T=3, H_kv=2, d=128,
           dtype=BF16, read=False):
    fn = L.mattn_cache_read if read else L.mattn_cache_write
    return fn(k, v, _two(*token), _two(*head), ctypes.byref(cache) if cache else None, cu, starts, B, T, H_kv, d, dtype, None)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("why,kw,code", CACHE)
def test_cache_rows_refuse_the_cache(L, why, kw, code, read):
    assert _write(L, _cache(**kw), read=read) == code, why
    assert L.mattn_last_error()


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("why,kw,code", [
    ("no rows", {"k": None}, -1),
    ("fp32 rows", {"dtype": F32}, -2),
    ("head dim 96", {"d": 96}, -2),
    ("no sequence", {"B": 0, "T": 0}, -1),
    ("no head", {"H_kv": 0}, -1),
    ("a negative count", {"T": -1, "cu": MB}, -1),
    ("more rows than sequences and no cu_seqlens", {"T": 4}, -1),
    ("2^31 rows", {"T": 1 << 30, "cu": MB}, -2),
    ("rows off a 16-byte boundary", {"v": 100 * MB + 8}, -2),
    ("a token stride off 16 bytes", {"token": (260, 256)}, -2),
    ("a negative stride", {"head": (128, -128)}, -1),
    ("cu_seqlens off a 4-byte boundary", {"cu": MB + 2}, -1),
    ("starts off a 4-byte boundary", {"starts": MB + 1}, -1),
    ("rows in the cache", {"k": 256 * MB + 4096}, -1),
    ("rows that end in the cache", {"v": 512 * MB - 256}, -1),
    ("a NULL cache", {"cache": None}, -1),
])
def test_cache_rows_refuse(L, why, kw, code, read):
    kw = dict(kw)
    cache = kw.pop("cache", _cache())
    assert _write(L, cache, read=read, **kw) == code, why
    assert L.mattn_last_error()


def test_cache_rows_that_would_be_written_twice(L):
    """k and v in one place; outputs whose rows overlap; inputs may (a broadcast row)."""
    assert _write(L, _cache(v=256 * MB)) == -1
    assert _write(L, _cache(True, v_exponents=768 * MB)) == -1
    assert _write(L, _cache(), v=MB, read=True) == -1
    assert _write(L, _cache(), token=(0, 256), read=True) == -1
    assert _write(L, _cache(), token=(128, 256), read=True) == -1
    for kw in (dict(token=(0, 0)), dict(head=(0, 0)), dict(k=MB, v=MB)):
        assert _write(L, _cache(), **kw) in (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)  # (nothing but the device is missing)


def test_cache_layouts_that_are_accepted(L):
    """Rows before heads, k and v of a page side by side, rows with room behind them, one page or head of any stride."""
    ok = (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)
    for e in (False, True):
        assert _write(L, _cache(e)) in ok
        assert _write(L, _cache(e, head_stride=(128, 128), row_stride=(256, 256), exp_head_stride=(1, 1),
                                exp_row_stride=(2, 2))) in ok
        assert _write(L, _cache(e, page_stride=(8192, 8192), v=256 * MB + 8192)) in ok
        assert _write(L, _cache(e, row_stride=(144, 160), head_stride=(2304, 2560), page_stride=(4608, 5120))) in ok
        assert _write(L, _cache(e, n_pages=1, page_stride=(16, 16))) in ok
    assert _write(L, _cache(True, exp_row_stride=(1, 3))) == -1  # (the rows' bytes reach into the next head's)


def _paged(L, cache, q=MB, o=2 * MB, lse=3 * MB, lens=None, B=3, H=8, H_kv=2, d=128, dtype=BF16, window=0, first=0,
           sink=None, scale=0.0, ws=200 * MB, ws_bytes=1 << 30):
    return L.mattn_decode_paged(q, ctypes.byref(cache) if cache else None, o, lse, lens, B, H, H_kv, d, dtype, window, first,
                                sink, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("why,kw,code", CACHE)
def test_decode_paged_refuses_the_cache(L, why, kw, code):
    assert _paged(L, _cache(**kw)) == code, why


@pytest.mark.parametrize("why,kw,code", [
    ("a NULL cache", {"cache": None}, -1),
    ("no queries", {"q": None}, -1),
    ("no output", {"o": None}, -1),
    ("H no multiple of H_kv", {"H": 9}, -1),
    ("17 query heads per key/value head", {"H": 34}, -2),
    ("head dim 96", {"d": 96}, -2),
    ("fp32", {"dtype": F32}, -2),
    ("65536 groups", {"B": 32768}, -2),
    ("queries off a 16-byte boundary", {"q": MB + 8}, -2),
    ("lse off a 4-byte boundary", {"lse": MB + 2}, -1),
    ("a negative window", {"window": -1}, -1),
    ("negative first tokens", {"window": 5, "first": -1}, -1),
    ("first tokens without a window", {"first": 4}, -1),
    ("a negative scale", {"scale": -1.0}, -1),
    ("an infinite scale", {"scale": float("inf")}, -1),
    ("no workspace", {"ws": None}, -6),
    ("a small workspace", {"ws_bytes": 1000}, -6),
    ("a workspace off a 256-byte boundary", {"ws": MB + 16}, -1),
    ("an output over the queries", {"q": 5 * MB, "o": 5 * MB + 512}, -1),
    ("an output over the keys", {"o": 256 * MB + 4096}, -1),
    ("an output that ends in the values", {"o": 512 * MB - 256}, -1),
    ("an lse over the keys", {"lse": 256 * MB + 4096}, -1),
    ("an lse over the output", {"o": 5 * MB, "lse": 5 * MB + 64}, -1),
])
def test_decode_paged_refuses(L, why, kw, code):
    kw = dict(kw)
    cache = kw.pop("cache", _cache())
    assert _paged(L, cache, **kw) == code, why
    assert L.mattn_last_error()


def test_decode_paged_workspace(L):
    n = ctypes.c_size_t(0)
    f = L.mattn_decode_paged_workspace
    assert f(3, 8, 2, 4, 16, 128, BF16, ctypes.byref(n)) == 0 and n.value > 0
    assert _paged(L, _cache(), ws_bytes=n.value - 1) == mattn.ERR_CAPACITY
    assert _paged(L, _cache(), ws_bytes=n.value) in (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)
    assert f(3, 8, 2, 4, 16, 128, BF16, None) == -1
    assert f(3, 8, 2, 4, 16, 128, F32, ctypes.byref(n)) == -2
    assert f(3, 8, 2, 0, 16, 128, BF16, ctypes.byref(n)) == -1
    assert f(3, 8, 2, 1 << 27, 16, 128, BF16, ctypes.byref(n)) == -2
    assert f(4096, 8, 8, 1 << 24, 64, 128, E4M3, ctypes.byref(n)) == -2  # 2^35 tiles


def _plan(L, B, H, Hkv, pages, page=64, d=128, dtype=E4M3, window=0, first=0):
    out = (ctypes.c_int * 3)()
    assert L.mattn_internal_paged_plan(B, H, Hkv, pages, page, d, dtype, window, first, out) == 0
    return tuple(out)


def test_decode_paged_plan(L):
    """Clusters for few groups with short lists, equal shares for the others; the tile by type, head dim and group."""
    assert _plan(L, 4, 16, 4, 63, 16, dtype=BF16) == (4, 6, 16)  # 1,008 keys
    assert _plan(L, 1, 32, 8, 128)[0] == 8  # 8,192 keys of eight groups
    assert _plan(L, 1, 32, 8, 512)[0] == 0  # 32,768: eleven rounds against four and a half
    assert _plan(L, 2, 32, 8, 128)[0] == 0  # sixteen groups: four CTAs each, six rounds
    assert _plan(L, 16, 32, 8, 64)[0] == 1 and _plan(L, 16, 32, 8, 256)[0] == 0
    assert _plan(L, 20, 32, 8, 1)[0] == 0  # 160 groups
    assert _plan(L, 64, 32, 8, 128) == (0, 12, 32)
    assert _plan(L, 1, 32, 8, 512, window=1024)[0] == 4 and _plan(L, 1, 32, 8, 512, window=1024, first=20000)[0] == 0
    for d, group, dtype, tile in ((64, 4, E4M3, 64), (128, 16, E4M3, 32), (256, 8, E4M3, 32), (256, 9, E4M3, 16), (64, 1, BF16, 32),
                                  (128, 1, BF16, 16), (256, 16, BF16, 16)):
        assert _plan(L, 200, group, 1, 10, d=d, dtype=dtype)[2] == tile


def test_a_null_size_and_the_binding(L):
    import torch

    for bad in (0, -3):
        with pytest.raises(ValueError):
            mattn.decode_paged(None, None, None, None, window=bad)
    x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # a CPU tensor
        mattn.decode_paged(x, x, x, x)
    with pytest.raises(ValueError):
        mattn.cache_write(x, x, x, x, x)
    with pytest.raises(ValueError):
        mattn.cache_read(x, x, x, x)


PACKED = dict(q=MB, k=2 * MB, v=3 * MB, token=(1024, 256, 256), head=(128, 128, 128), o=4 * MB, lse=None, cu=5 * MB, cu_k=None, B=3,
              T=100, T_k=100, H=8, H_kv=2, d=128, dtype=BF16, causal=1, window=0, sink=None, scale=0.0, ws=256 * MB,
              ws_bytes=1 << 20)


def _packed(L, **kw):
    a = dict(PACKED, **kw)
    three = ctypes.c_int64 * 3
    return L.mattn_attention_packed(a["q"], a["k"], a["v"], three(*a["token"]), three(*a["head"]), a["o"], a["lse"], a["cu"],
                                    a["cu_k"], a["B"], a["T"], a["T_k"], a["H"], a["H_kv"], a["d"], a["dtype"], a["causal"],
                                    a["window"], a["sink"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("why,kw,code", [
    ("no queries", {"q": None}, -1),
    ("no keys", {"k": None}, -1),
    ("no output", {"o": None}, -1),
    ("no cu_seqlens", {"cu": None}, -1),
    ("no sequence", {"B": 0}, -1),
    ("no head", {"H": 0}, -1),
    ("H no multiple of H_kv", {"H_kv": 3}, -1),
    ("a negative count", {"T": -1}, -1),
    ("a negative count of keys", {"T_k": -1, "cu_k": MB}, -1),
    ("other keys than queries and no cu_seqlens_k", {"T_k": 99}, -1),
    ("more than 2^30 rows", {"T": (1 << 30) + 1, "T_k": (1 << 30) + 1}, -2),
    ("2^31 items", {"T": 1 << 30, "T_k": 1 << 30, "H": 512}, -2),
    ("head dim 112", {"d": 112}, -2),
    ("head dim 72", {"d": 72}, -2),
    ("fp32", {"dtype": F32}, -2),
    ("a negative window", {"window": -4}, -1),
    ("a window without causality", {"window": 4, "causal": 0}, -1),
    ("queries off a 16-byte boundary", {"q": MB + 8}, -2),
    ("cu_seqlens off a 4-byte boundary", {"cu": MB + 2}, -1),
    ("lse off a 4-byte boundary", {"lse": MB + 2}, -1),
    ("a stride off 16 bytes", {"token": (1024, 252, 256)}, -2),
    ("a stride of zero", {"head": (128, 0, 128)}, -2),
    ("a negative stride", {"token": (-1024, 256, 256)}, -2),
    ("a stride of 2^40 bytes", {"token": (1 << 39, 256, 256)}, -2),
    ("an infinite scale", {"scale": float("inf")}, -1),
    ("a scale that is NaN", {"scale": float("nan")}, -1),
    ("no workspace", {"ws": None}, -6),
    ("a small workspace", {"ws_bytes": 64}, -6),
    ("a workspace off a 256-byte boundary", {"ws": MB + 16}, -1),
    ("an output over the queries", {"o": MB}, -1),
    ("an output that ends in the keys", {"o": 2 * MB - 512}, -1),
    ("an output over the values' last row", {"o": 3 * MB + 99 * 512}, -1),
    ("an lse over the queries", {"lse": MB + 4096}, -1),
    ("an lse over the output", {"lse": 4 * MB + 4096}, -1),
])
def test_attention_packed_refuses(L, why, kw, code):
    assert _packed(L, **kw) == code, why
    assert L.mattn_last_error()


def test_attention_packed_accepts(L):
    """Only the device is missing: strides of single entries, no keys at all, the least workspace."""
    ok = (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)
    n = ctypes.c_size_t(0)
    f = L.mattn_attention_packed_workspace
    assert f(3, 100, 8, ctypes.byref(n)) == 0
    assert _packed(L, ws_bytes=n.value) in ok and _packed(L, ws_bytes=n.value - 1) == mattn.ERR_CAPACITY
    assert _packed(L, H_kv=1, head=(128, 0, -5)) in ok
    assert _packed(L, d=256, token=(2048, 512, 512), head=(256, 256, 256)) in ok
    assert _packed(L, o=MB + 99 * 2048 + 2048, lse=2 * MB - 3200) in ok  # behind the queries, before the keys
    assert _packed(L, T=1, T_k=1, token=(0, 0, 0)) in ok
    assert _packed(L, T_k=0, k=None, v=None, cu_k=MB) in ok
    assert f(0, 100, 8, ctypes.byref(n)) == -1 and f(3, -1, 8, ctypes.byref(n)) == -1 and f(3, 100, 8, None) == -1
    assert f(1, 1 << 30, 1024, ctypes.byref(n)) == -2


@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_tensors_that_overlap(L, e4m3):
    """What a call writes overlaps neither itself nor what it reads: k and v a few bytes or a row apart, codes and
    exponents, tables and offsets, outputs a row apart.  Interleaved ones share an extent and no byte."""
    ok = (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)
    es = 1 if e4m3 else 2
    k, page = 256 * MB, 2 * 16 * 128 * es  # bytes of a page
    for off in (16, 128 * es, 16 * 128 * es, page // 2, page + 16, 3 * page - 128 * es, 9 * page + 16, -16, -page - 16):
        assert _write(L, _cache(e4m3, v=k + off)) == -1, off
        assert L.mattn_last_error()
    assert _write(L, _cache(e4m3, v=k + 10 * page)) in ok and _write(L, _cache(e4m3, v=k - 10 * page)) in ok
    # one pool: its even pages k's, v's a page behind, by the table; k and v of a page, a head or a row side by side
    assert _write(L, _cache(e4m3, v=k + page)) in ok
    wide = dict(page_stride=(8192, 8192))
    assert _write(L, _cache(e4m3, v=k + page, **wide)) in ok and _write(L, _cache(e4m3, v=k + 3 * page, **wide)) in ok
    assert _write(L, _cache(e4m3, v=k + page - 16, **wide)) == -1 and _write(L, _cache(e4m3, v=k + page + 16, **wide)) == -1
    assert _write(L, _cache(e4m3, v=k + 16 * 128 * es, head_stride=(4096, 4096), **wide)) in ok
    rows = dict(row_stride=(256, 256), head_stride=(4096, 4096), **wide)
    assert _write(L, _cache(e4m3, v=k + 128 * es, **rows)) in ok and _write(L, _cache(e4m3, v=k + 64 * es, **rows)) == -1
    # heads apart by more than their pages: a page's v a head of k's behind
    apart = dict(page_stride=(2048, 2048), head_stride=(20480, 20480))
    assert _write(L, _cache(e4m3, v=k + 20480 * es, **apart)) == -1 and _write(L, _cache(e4m3, v=k + 2048 * es, **apart)) in ok
    # different layouts in one place
    assert _write(L, _cache(e4m3, v=k + 32, head_stride=(2048, 128), row_stride=(128, 256))) == -1
    table, size = 900 * MB, 3 * 4 * 4
    for kw in (dict(page_table=k + 64), dict(page_table=k - size + 4), dict(page_table=512 * MB + 10 * page - 4)):
        assert _write(L, _cache(e4m3, **kw)) == -1 and _write(L, _cache(e4m3, **kw), read=True) in ok, kw
    for kw in (dict(cu=k + 4), dict(starts=512 * MB), dict(cu=k - 12)):
        assert _write(L, _cache(e4m3), **kw) == -1 and _write(L, _cache(e4m3), read=True, **kw) in ok, kw
    assert _write(L, _cache(e4m3, page_table=k - size), cu=k + 10 * page, starts=512 * MB - 12) in ok
    # outputs of a read: 3 tokens of 2 heads of 128, 512 bytes each
    for off in (16, 256, 512, 1024, 1280, -16, -512):
        assert _write(L, _cache(e4m3), k=MB, v=MB + off, read=True) == -1, off
    assert _write(L, _cache(e4m3), k=MB, v=MB + 3 * 512, read=True) in ok
    assert _write(L, _cache(e4m3), k=MB, v=MB + 512, token=(512, 512), read=True) in ok
    assert _write(L, _cache(e4m3), k=MB, v=MB + 256, token=(512, 512), head=(256, 256), read=True) in ok
    assert _write(L, _cache(e4m3), k=MB, v=MB + 128, token=(512, 512), head=(256, 256), read=True) == -1
    for kw in (dict(cu=MB + 4), dict(cu=MB - 12), dict(starts=100 * MB + 1532)):
        assert _write(L, _cache(e4m3), read=True, **kw) == -1 and _write(L, _cache(e4m3), **kw) in ok, kw
    assert _write(L, _cache(e4m3, page_table=100 * MB), read=True) == -1
    if not e4m3:
        return
    # exponents: over the rows, the codes, each other; in one pool with the codes, page by page or row by row
    for kw in (dict(k_exponents=MB), dict(v_exponents=100 * MB + 1500), dict(k_exponents=k + 100), dict(v_exponents=k + 100),
               dict(k_exponents=512 * MB - 100), dict(v_exponents=768 * MB + 8), dict(v_exponents=768 * MB + 16),
               dict(v_exponents=768 * MB + 31), dict(page_table=768 * MB + 8)):
        assert _write(L, _cache(True, **kw)) == -1, kw
    assert _write(L, _cache(True, k_exponents=MB), read=True) == -1 and _write(L, _cache(True, page_table=768 * MB + 8), read=True) in ok
    assert _write(L, _cache(True, v_exponents=768 * MB + 32)) in ok  # (a whole page)
    pool = dict(page_stride=(12288, 12288), exp_page_stride=(12288, 12288), v=k + 4096)
    assert _write(L, _cache(True, k_exponents=k + 8192, v_exponents=k + 8224, **pool)) in ok
    assert _write(L, _cache(True, k_exponents=k + 8191, v_exponents=k + 8224, **pool)) == -1
    assert _write(L, _cache(True, k_exponents=k + 8192, v_exponents=k + 12288 - 31, **pool)) == -1
    beside = dict(row_stride=(144, 144), head_stride=(2304, 2304), page_stride=(4608, 4608), exp_row_stride=(144, 144),
                  exp_head_stride=(2304, 2304), exp_page_stride=(4608, 4608), v=512 * MB)
    assert _write(L, _cache(True, k_exponents=k + 128, v_exponents=512 * MB + 143, **beside)) in ok
    assert _write(L, _cache(True, k_exponents=k + 127, v_exponents=512 * MB + 143, **beside)) == -1


def test_cache_tensors_that_overlap_by_enumeration(L):
    """k's and v's pages at offsets and strides of many kinds: refused exactly where rows of theirs share bytes, but for
    pools a whole number of pages apart, whose pages of one number are apart."""
    import random

    r = random.Random(1)
    seen = {True: 0, False: 0}
    for _ in range(1500):
        n, H, page, d = r.choice((1, 2, 3)), r.choice((1, 2, 3)), 16, 64
        size, order = (n, H, page), r.sample(range(3), 3)
        stride, end = [0, 0, 0], d
        for i in order:  # (each dimension steps over those below it, and some room)
            stride[i] = end + 8 * r.choice((0, 0, 8, 64, end // 8))
            end = stride[i] * (size[i] - 1) + end
        off = r.choice((8 * r.randint(-end // 8 - 8, end // 8 + 8), r.choice((-1, 1)) * r.choice(stride), d, -d, 2 * stride[0],
                        stride[0] + stride[1]))
        row = lambda p, h, x: p * stride[0] + h * stride[1] + x * stride[2]  # noqa: E731
        spots = [[(p, row(p, h, x)) for p in range(n) for h in range(H) for x in range(page)] for _ in range(2)]
        hit = [(p, q) for p, a in spots[0] for q, b in spots[1] if abs(a - b - off) < d]
        bad = any(p == q for p, q in hit) or (bool(hit) and off % stride[0] != 0)
        c = _cache(n_pages=n, H_kv=H, d=d, v=256 * MB + 2 * off, page_stride=(stride[0],) * 2, head_stride=(stride[1],) * 2,
                   row_stride=(stride[2],) * 2)
        got = _write(L, c, H_kv=H, d=d, token=(H * d,) * 2, head=(d, d))
        assert (got == -1) == bad and (bad or got in (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)), (size, stride, off, got, hit[:3])
        seen[bad] += 1
    assert min(seen.values()) > 300


@pytest.mark.parametrize("why,kw", [
    ("an output over the key exponents", {"o": 768 * MB}),
    ("an output that ends in the value exponents", {"o": 800 * MB - 64}),
    ("an lse over the page table", {"lse": 900 * MB + 44}),
    ("an output over seq_lens", {"lens": 2 * MB + 6140}),
    ("an lse over seq_lens", {"lens": 3 * MB}),
    ("an output over the sink logits", {"sink": 2 * MB + 64}),
    ("a workspace over the output", {"ws": 2 * MB}),
    ("a workspace over the lse", {"ws": 3 * MB - 4096}),
    ("a workspace over the queries", {"ws": MB}),
    ("a workspace that ends in the keys", {"ws": 256 * MB - 65536}),
    ("a workspace over the exponents", {"ws": 768 * MB}),
    ("a workspace over the page table", {"ws": 900 * MB}),
    ("a workspace over seq_lens", {"lens": 200 * MB + 1024}),
])
def test_decode_paged_refuses_what_overlaps(L, why, kw):
    assert _paged(L, _cache(True), **kw) == -1, why
    assert L.mattn_last_error()


@pytest.mark.parametrize("why,kw", [
    ("an output over cu_seqlens", {"cu": 4 * MB + 8}),
    ("an output over cu_seqlens_k", {"cu_k": 4 * MB + 100 * 2048 - 4}),
    ("an lse over cu_seqlens", {"lse": 5 * MB - 3196}),
    ("an output over the sink logits", {"sink": 4 * MB + 64}),
    ("an lse over the sink logits", {"lse": 6 * MB, "sink": 6 * MB + 3196}),
    ("a workspace over the queries", {"ws": MB}),
    ("a workspace over the values", {"ws": 3 * MB + 256}),
    ("a workspace over the output", {"ws": 4 * MB + 4096}),
    ("a workspace over the lse", {"lse": 256 * MB + 64}),
    ("a workspace over cu_seqlens", {"cu": 256 * MB}),
    ("a workspace over the sink logits", {"sink": 256 * MB + 4}),
])
def test_attention_packed_refuses_what_overlaps(L, why, kw):
    assert _packed(L, **kw) == -1, why
    assert L.mattn_last_error()


def test_attention_packed_refuses_2_30_items_of_256(L):
    """At d = 256 an item is half as many rows."""
    big = dict(T=1 << 29, T_k=1 << 29, H=512, H_kv=512, o=1 << 60, ws=1 << 62, ws_bytes=1 << 50, k=1 << 58, v=1 << 59)
    strides = dict(token=(512 * 256,) * 3, head=(256,) * 3)
    ok = (mattn.ERR_NO_DEVICE, mattn.ERR_CUDA)
    assert _packed(L, d=256, **strides, **big) == -2
    assert _packed(L, d=256, **strides, **dict(big, T=1 << 28, T_k=1 << 28)) in ok
    assert _packed(L, d=128, **strides, **big) in ok


def test_attention_packed_plan(L):
    """No plan kernel for up to four items an SM, unless there are hundreds of sequences to look through."""
    f = L.mattn_internal_packed_direct
    assert f(8, 700, 16, 128) and f(1, 2048, 32, 64) and f(1, 1, 1, 80) and f(384, 64, 4, 128) and f(2, 128, 304, 128)
    assert not f(385, 64, 4, 128) and not f(100000, 1, 1, 64)
    assert not f(2, 128, 305, 128) and not f(8, 16384, 32, 128) and not f(8, 700, 16, 256)
