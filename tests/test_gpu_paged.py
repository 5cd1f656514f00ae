"""GPU tests of the operators around a paged cache (cache_write, cache_read,
decode_paged) against plain implementations in 64 bits written here.

Tolerances, derived before the first run; u = 2^-8 is bf16's half step relative
to the value, e = 2^-24 fp32's.
  write, read  none: a power of two is exact, a code's rounding is one to nearest
               even of an exact product, and a code times its power is a bf16.
  decode       o = sum p v / sum p, A = sum p |v| / sum p: the output rounded once
               (u |o|), a weight off by h (2^-16 for two bf16 parts, 2^-11 for one
               f16 value) and by the score's error t twice (weight and sum), 2^-13
               for exponentials and sums over keys: |do| <= u |o| + (h + 2 t + 2^-13) A.
               In e4m3 a weight with its value's power w = p 2^e is off by 2^-39 of
               the largest one where it is small: n 2^-39 max(w) 448 / sum p.
  scores       t = d e sum |q k| scale, in e4m3 and 2^-39 max|q| sum |k| scale for
               queries in f16.
  lse          t + 2^-19 (1 + |lse|).
"""

import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

U, E = 2.0 ** -8, 2.0 ** -24
NAN, INF = float("nan"), float("inf")
CODES = torch.float8_e4m3fn
GRID = None  # the values of e4m3, ascending


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(mattn.LIB_PATH):
        from block_sparse_attention_masked_gb300 import build

        build.build()
    mattn.lib()


@pytest.fixture(autouse=True)
def _clean_error_word():
    yield
    rc, word = mattn.device_status()
    assert rc == 0, f"device error word {word:#x}"


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the cache, plainly
def ref_codes(row):
    """One row (64 bits, CPU) -> (values of its codes, exponent byte), from the definition."""
    top = float(row.abs().max())
    if not math.isfinite(top):
        return torch.full_like(row, NAN), 255
    e = 0
    while 448.0 * 2.0 ** (e - 127) < top:
        e += 1
    x = row * 2.0 ** (127 - e)
    step = torch.full_like(x, 2.0 ** -9)
    for k in range(-5, 9):
        step = torch.where(x.abs() >= 2.0 ** k, torch.full_like(x, 2.0 ** (k - 3)), step)
    return torch.round(x / step) * step, e


class Cache:
    """A paged cache of random rows with its copy in 64 bits on the CPU; `layout`: how
    the pages lie in memory."""

    def __init__(self, B, Hkv, d, page, slots, e4m3, seed=0, layout="dense", spread=0, spare=2):
        g = _gen(seed)
        n = B * slots + spare
        self.shape = n, Hkv, page, d
        self.e4m3, self.page = e4m3, page
        self.table = torch.randperm(n, generator=g, device="cuda")[: B * slots].view(B, slots).to(torch.int32)
        self.k, self.v = (self._laid(_randn(g, n, Hkv, page, d, scale=64 if e4m3 else 1), layout) for _ in range(2))
        if layout == "pool":  # k and v of a page side by side
            pool = torch.stack((self.k, self.v), dim=1)
            self.k, self.v = pool[:, 0], pool[:, 1]
        self.ke = self.ve = None
        if e4m3:
            self.ke, self.ve = (torch.randint(121 - spread, 124 + spread, (n, Hkv, page), generator=g, device="cuda",
                                              dtype=torch.uint8) for _ in range(2))
            if layout == "rows":
                self.ke, self.ve = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (self.ke, self.ve))

    def _laid(self, x, layout):
        if self.e4m3:
            x = x.to(CODES)
        if layout == "rows":  # [n, page, Hkv, d] in memory
            x = self._bytes(x).transpose(1, 2).contiguous().transpose(1, 2).view(x.dtype)
        if layout == "padded":
            y = torch.zeros((*x.shape[:3], x.shape[3] + 16), dtype=torch.uint8 if self.e4m3 else x.dtype, device="cuda")
            y[..., : x.shape[3]] = self._bytes(x)
            x = y[..., : x.shape[3]].view(x.dtype)
        return x

    @staticmethod
    def _bytes(x):
        return x.view(torch.uint8) if x.dtype == CODES else x

    def kw(self):
        return dict(k_exponents=self.ke, v_exponents=self.ve)

    def held(self, which):
        """[n_pages, Hkv, page, d] in 64 bits on the CPU."""
        x, e = (self.k, self.ke) if which == "k" else (self.v, self.ve)
        x = x.float().double().cpu()
        if e is None:
            return x
        e = e.cpu()
        f = torch.where(e == 255, torch.full(e.shape, NAN, dtype=torch.float64), torch.pow(2.0, e.double() - 127))
        return x * f[..., None]

    def rows(self, b, h, positions):
        """Keys and values [n, d] of these positions of sequence b; positions without a page dropped."""
        table = self.table.cpu()
        at = [(int(table[b, j // self.page]), j % self.page) for j in positions]
        at = [(p, r) for p, r in at if 0 <= p < self.shape[0]]
        p, r = [x[0] for x in at], [x[1] for x in at]
        return self._k64[p, h, r], self._v64[p, h, r]

    def freeze(self):
        self._k64, self._v64 = self.held("k"), self.held("v")
        return self

    def hide(self, seen):
        """What no query sees, NaN: rows of `seen`'s complement ([n, page] bool) and their powers."""
        for x in (self.k, self.v):
            y = self._bytes(x)
            hidden = (~seen)[:, None, :, None].expand(x.shape)
            y[hidden] = 0x7F if self.e4m3 else NAN
        if self.e4m3:
            for e in (self.ke, self.ve):
                e[(~seen)[:, None, :].expand(e.shape)] = 255


def ref_decode(q, keys, values, sink, scale, e4m3):
    """One head -> (o, lse, tolerance of o, tolerance of lse)."""
    d, n = q.shape[0], keys.shape[0]
    s = keys @ q * scale
    x = s if sink is None else torch.cat((s, s.new_tensor([sink])))
    if x.numel() == 0:
        return torch.zeros_like(q), -INF, torch.zeros_like(q), 0.0
    m = x.max()
    p = torch.exp(x - m)
    z = p.sum()
    w = p[:n] / z
    o, a = w @ values, w @ values.abs()
    lse = float(m + torch.log(z))
    t = float((keys.abs() @ q.abs()).max()) * scale * d * E if n else 0.0
    h, floor = 2.0 ** -16, 0.0
    if e4m3 and n:
        t += 2.0 ** -39 * float(q.abs().max()) * float(keys.abs().sum(dim=1).max()) * scale
        h = 2.0 ** -11
        # a value row's power is at most its largest |value| / 224 (or as planted, / 2^-9)
        floor = n * 2.0 ** -39 * float((w * values.abs().amax(dim=1)).max()) * 2.0 ** 18
    return o, lse, U * o.abs() + (h + 2 * t + 2.0 ** -13) * a + floor, t + 2.0 ** -19 * (1 + abs(lse))


def check_decode(o, lse, q, cache, positions, sink, scale, tag=""):
    """positions[b]: the key positions that sequence b's query sees."""
    B, H, d = q.shape
    Hkv = cache.shape[1]
    qd, got, gl = q.double().cpu(), o.double().cpu(), lse.double().cpu()
    for b in range(B):
        for h in range(H):
            keys, values = cache.rows(b, h // (H // Hkv), positions[b])
            r, l, tol, tl = ref_decode(qd[b, h], keys, values, None if sink is None else float(sink[h]), scale, cache.e4m3)
            err = (got[b, h] - r).abs()
            assert bool((err <= tol + 1e-30).all()), f"{tag} b{b} h{h}: o off by {(err - tol).max():.3e} over its bound"
            if math.isinf(l):
                assert float(gl[b, h]) == l, f"{tag} b{b} h{h}: lse {float(gl[b, h])}"
            else:
                assert abs(float(gl[b, h]) - l) <= tl, f"{tag} b{b} h{h}: lse off by {abs(float(gl[b, h]) - l):.3e} ({tl:.1e})"


def visible(n, window, first):
    if not window or n <= window:
        return list(range(n))
    return list(range(min(first, n - window))) + list(range(n - window, n))


def decode_case(B, H, Hkv, d, page, slots, lens, e4m3, window=None, first=0, sink=False, scale=None, seed=0, layout="dense",
                holes=(), spread=0, q_scale=1.0):
    c = Cache(B, Hkv, d, page, slots, e4m3, seed, layout, spread)
    for b, j, to in holes:
        c.table[b, j] = to
    c.freeze()
    L = page * slots
    n = [min(max(x, 0), L) for x in lens]
    seen = torch.zeros((c.shape[0], page), dtype=torch.bool, device="cuda")
    positions = [visible(x, window, first) for x in n]
    table = c.table.tolist()
    for b, ps in enumerate(positions):
        for j in ps:
            if 0 <= table[b][j // page] < c.shape[0]:
                seen[table[b][j // page], j % page] = True
    c.hide(seen)
    q = _randn(_gen(seed + 100), B, H, d, scale=q_scale)
    sk = torch.linspace(-2, 3, H, device="cuda") if sink else None
    o, lse = mattn.decode_paged(q, c.k, c.v, c.table, _i32(lens), window=window, sink_tokens=first, sink=sk, scale=scale,
                                **c.kw())
    torch.cuda.synchronize()
    check_decode(o, lse, q, c, positions, sk, d ** -0.5 if scale is None else scale)
    return o, lse


HEADS = [(1, 1), (8, 2), (3, 1), (8, 1), (12, 1), (32, 2)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads", HEADS)
def test_decode_paged_heads(heads, d, e4m3):
    decode_case(3, *heads, d, 16, 9, [100, 1, 37], e4m3, seed=d + heads[0])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 144])
@pytest.mark.parametrize("lens", [[0, 1, 15, 16], [17, 31, 32, 33], [144, 143, 500, -3], [63, 64, 65, 0]])
def test_decode_paged_lengths_and_pages(page, lens, e4m3):
    """Lengths of zero and one, around a tile and a page, past the table (clamped) and negative."""
    decode_case(4, 4, 2, 128, page, -(-144 // page), lens, e4m3, seed=page + lens[0], sink=lens[0] == 17)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,first", [(1, 0), (5, 1), (32, 4), (33, 40), (100, 100), (1000, 7), (64, 0)])
def test_decode_paged_windows(d, window, first, e4m3):
    decode_case(5, 8, 2, d, 32, 7, [224, 0, 1, 101, 170], e4m3, window=window, first=first, seed=window + first,
                sink=first == 4)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("layout", ["rows", "pool", "padded"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_paged_layouts(d, layout, e4m3):
    decode_case(2, 8, 2, d, 16, 5, [80, 33], e4m3, seed=3, layout=layout, sink=True, scale=0.3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_paged_positions_without_pages(e4m3):
    """Table entries outside the pages: no keys, wherever they lie; a sequence with none at all."""
    decode_case(3, 4, 2, 128, 16, 6, [96, 90, 60], e4m3,
                holes=[(0, 0, -1), (0, 3, 1 << 30), (1, 5, -5), (1, 2, 20)] + [(2, j, -1) for j in range(6)])
    decode_case(3, 4, 2, 64, 16, 6, [96, 90, 60], e4m3, window=40, first=3, sink=True,
                holes=[(0, 0, -1), (0, 5, 1 << 30), (1, 5, -5)] + [(2, j, -1) for j in range(6)])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_paged_long(d, e4m3):
    """Many tiles a warp, states of many warps."""
    decode_case(2, 4, 1, d, 64, 400, [25600, 12345], e4m3, seed=5)


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_paged_many_sequences(e4m3):
    g = _gen(9)
    B = 700
    lens = torch.randint(0, 49, (B,), generator=g, device="cuda").tolist()
    decode_case(B, 2, 1, 64, 16, 3, lens, e4m3, seed=9)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("what", ["plain", "window", "holes", "rows", "group"])
def test_decode_paged_in_equal_shares(d, what, e4m3):
    """More groups than SMs: warps' shares end anywhere in the lists."""
    B, Hkv, slots = 80, 2, 9
    lens = [(37 * b) % 150 for b in range(B)]
    kw = {"plain": dict(), "window": dict(window=50, first=5, sink=True), "rows": dict(layout="rows", scale=0.2),
          "holes": dict(holes=[(b, (3 * b) % slots, -1) for b in range(0, B, 2)] + [(7, j, 1 << 20) for j in range(slots)]),
          "group": dict(sink=True)}[what]
    decode_case(B, 24 if what == "group" else 4, Hkv, d, 16, slots, lens, e4m3, seed=12, **kw)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,slots,lens", [(1, 40, [640]), (2, 40, [600, 333]), (9, 8, [128] * 9), (1, 3, [1]), (30, 4, [0] * 15 + [64] * 15)])
def test_decode_paged_in_clusters(B, slots, lens, e4m3):
    """Clusters of 8, 4, 2 and 1 CTAs; more warps than tiles, and CTAs without any."""
    decode_case(B, 8, 4, 128, 16, slots, lens, e4m3, seed=B, sink=B == 2)


def test_decode_paged_powers_far_apart():
    """Rows whose powers lie 2^80 apart, queries from 2^-60 on: weights and their powers meet in range."""
    for q_scale in (2.0 ** -60, 1.0):
        decode_case(2, 8, 2, 128, 16, 9, [144, 77], True, spread=40, q_scale=q_scale, seed=11, scale=2.0 ** -44)
    c = Cache(1, 1, 128, 16, 8, True, seed=2)
    c.ve[:] = 127
    c.ke[:] = 127 - 8
    far = c.table[0, 3]
    c.ve[far, 0, 5] = 230  # one value row 2^103 above the others, its weight far below
    q = _randn(_gen(3), 1, 4, 128)
    kq = c.k[far, 0, 5].float() * 2.0 ** -8
    scale = -70.0 / float((q[0].float() @ kq).abs().min())  # ..
    q = q * torch.sign(q[0].float() @ kq)[None, :, None].to(q.dtype) * -1
    c.freeze()
    o, lse = mattn.decode_paged(q, c.k, c.v, c.table, None, scale=abs(scale), **c.kw())
    check_decode(o, lse, q, c, [list(range(128))], None, abs(scale))


@pytest.mark.parametrize("e4m3", [False, True])
def test_decode_paged_nan_and_infinite_rows(e4m3):
    """A visible NaN reaches its own sequence and head group alone, an infinite value its columns."""
    B, H, Hkv, d = 3, 8, 2, 128
    c = Cache(B, Hkv, d, 16, 4, e4m3, seed=4)
    q = _randn(_gen(5), B, H, d)
    run = lambda: mattn.decode_paged(q, c.k, c.v, c.table, _i32([64, 64, 50]), **c.kw())  # noqa: E731
    want = [x.clone() for x in run()]
    p = int(c.table[1, 2])
    if e4m3:
        c.ve[p, 1, 7] = 255
        o, lse = run()
        assert torch.isnan(o[1, 4:]).all() and torch.equal(lse, want[1])
    else:
        c.v[p, 1, 7, 3] = INF
        c.v[p, 1, 7, 4] = NAN
        o, lse = run()
        assert bool((o[1, 4:, 3] == INF).all()) and torch.isnan(o[1, 4:, 4]).all() and torch.equal(lse, want[1])
        o[1, 4:, 3:5] = want[0][1, 4:, 3:5]
        assert torch.equal(o, want[0])
    keep = torch.ones((B, H), dtype=torch.bool, device="cuda")
    keep[1, 4:] = False
    assert torch.equal(o[keep], want[0][keep])
    if e4m3:
        c.ke[p, 0, 7] = 255
    else:
        c.k[p, 0, 7, 9] = NAN
    o, lse = run()
    assert torch.isnan(o[1, :4]).all() and torch.isnan(lse[1, :4]).all()
    keep[1, :4] = False
    assert torch.equal(o[keep], want[0][keep]) and torch.equal(lse[keep], want[1][keep])


# ------------------------------------------------------------------ write and read
def _lens_to_cu(n):
    return _i32([0] + torch.tensor(n).cumsum(0).tolist())


def ref_places(c, n, starts, T):
    """(t, page, row) of each row that has a place; t of those in a sequence without one."""
    table = c.table.cpu()
    placed, lost, t = [], [], 0
    for b, k in enumerate(n):
        for i in range(k):
            j = starts[b] + i
            p = int(table[b, j // c.page]) if 0 <= j < c.page * table.shape[1] else -1
            if 0 <= p < c.shape[0]:
                placed.append((t + i, p, j % c.page))
            else:
                lost.append(t + i)
        t += k
    return placed, lost


def rows_of(seed, T, Hkv, d, layout="dense"):
    g = _gen(seed)
    if layout == "fused":  # one projection's output
        x = _randn(g, T, 3 * Hkv, d)
        return x[:, Hkv : 2 * Hkv], x[:, 2 * Hkv :]
    if layout == "heads":  # [Hkv, T, d] in memory
        return tuple(_randn(g, Hkv, T, d).transpose(0, 1) for _ in range(2))
    return tuple(_randn(g, T, Hkv, d) for _ in range(2))


CACHE_CASES = [
    # n, starts, padding rows behind the last sequence
    ([1], [0], 0), ([5, 0, 33, 1, 0], [0, 7, 30, 95, 3], 0), ([17, 40], [79, 0], 9), ([0, 0], [0, 5], 4),
    ([3, 70, 2], [-2, 90, 200], 1),
]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("case", CACHE_CASES)
@pytest.mark.parametrize("layout", ["dense", "rows", "pool", "padded"])
def test_cache_write_and_read(case, d, layout, e4m3):
    """Every written row and its power bit for bit, every other byte as it was; back as bf16."""
    n, starts, pad = case
    Hkv, page, slots = (1, 48, 2) if layout == "padded" else (3, 32, 3)
    T = sum(n) + pad
    c = Cache(len(n), Hkv, d, page, slots, e4m3, seed=T + d, layout=layout)
    c.table[0, 1] = -1
    k, v = rows_of(T, T, Hkv, d, {"rows": "heads", "pool": "fused"}.get(layout, "dense"))
    k, v = k * torch.exp2(torch.arange(T, device="cuda") % 40 - 20).to(k.dtype)[:, None, None], v
    before = {x: (c.held(x), None if not e4m3 else (c.ke if x == "k" else c.ve).cpu().clone()) for x in "kv"}
    cu = _lens_to_cu(n)
    got = mattn.cache_write(k, v, c.k, c.v, c.table, cu, _i32(starts), **c.kw())
    torch.cuda.synchronize()
    assert got[0] is c.k and got[1] is c.v
    placed, lost = ref_places(c, n, starts, T)
    for name, rows, pages, exps in (("k", k, c.k, c.ke), ("v", v, c.v, c.ve)):
        want, e_want = before[name]
        x = rows.double().cpu()
        after = c.held(name)
        for t, p, r in placed:
            for h in range(Hkv):
                if e4m3:
                    codes, e = ref_codes(x[t, h])
                    want[p, h, r], e_want[p, h, r] = codes * 2.0 ** (e - 127), e
                else:
                    want[p, h, r] = x[t, h]
        assert torch.equal(after, want)
        if e4m3:
            assert torch.equal(exps.cpu(), e_want)
    outs = [torch.full((T, Hkv, d), 7.0, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    outs[1] = outs[1].transpose(0, 1).contiguous().transpose(0, 1)
    ko, vo = mattn.cache_read(c.k, c.v, c.table, cu, starts=_i32(starts), k_out=outs[0], v_out=outs[1], **c.kw())
    made = mattn.cache_read(c.k, c.v, c.table, cu, T, _i32(starts), **c.kw())
    torch.cuda.synchronize()
    for name, y, z in (("k", ko, made[0]), ("v", vo, made[1])):
        want = torch.full((T, Hkv, d), 7.0, dtype=torch.float64)
        want[lost] = 0
        h64 = c.held(name)
        for t, p, r in placed:
            want[t] = h64[p, :, r]
        assert torch.equal(y.double().cpu(), want)
        want[sum(n):] = 0
        assert torch.equal(z.double().cpu(), want)


def test_cache_rows_of_every_size():
    """Powers from the least bf16 to the largest, the borders of 448 2^e, zeros, infinities, NaN."""
    T, d = 700, 64
    x = torch.zeros((T, 1, d), device="cuda")
    top = torch.tensor([2.0 ** (i - 133) if i < 250 else 1.0 for i in range(T)])
    g = torch.Generator().manual_seed(1)
    base = torch.randn((T, d), generator=g).clamp(-3, 3) / 3
    rows = base * top[:, None]
    for i, m in enumerate((448.0, 450.0, 446.0, 224.0, 226.0, 222.0)):
        rows[300 + i] = base[300 + i] * m * 0.9
        rows[300 + i, i] = -m
    rows[310] = 0
    rows[311, 5], rows[312, 6], rows[313, 63], rows[314, 0] = INF, NAN, -INF, 3.3e38
    rows[315] = 3.3895e38
    x[:, 0] = rows.cuda()
    k = x.to(torch.bfloat16)
    c = Cache(1, 1, d, 16, 44, True, seed=1)
    mattn.cache_write(k, k.flip(0), c.k, c.v, c.table, _i32([0, T]), **c.kw())
    out = mattn.cache_read(c.k, c.v, c.table, _i32([0, T]), T, **c.kw())
    for y, src in ((out[0], k), (out[1], k.flip(0))):
        src, y = src[:, 0].double().cpu(), y[:, 0].double().cpu()
        for t in range(T):
            codes, e = ref_codes(src[t])
            want = (codes * 2.0 ** (e - 127)) if e < 255 else codes
            want = want.to(torch.bfloat16).double()  # (below bf16's least: none, or rounded once)
            assert torch.equal(torch.nan_to_num(y[t], nan=12.5), torch.nan_to_num(want, nan=12.5)), (t, y[t], want)


@pytest.mark.parametrize("T,Hkv,d", [(20000, 8, 128), (30000, 1, 64), (9000, 5, 256)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_write_and_read_large(T, Hkv, d, e4m3):
    """Rows of several groups a warp, sequences that begin anywhere."""
    n = [T // 3, 1, 0, T // 2, 7]
    n.append(T - sum(n) - 5)
    starts = [0, 100, 3, 17, 0, 5]
    slots = -(-max(a + b for a, b in zip(n, starts)) // 64)
    c = Cache(len(n), Hkv, d, 64, slots, e4m3, seed=8)
    k, v = rows_of(4, T, Hkv, d, "fused")
    cu = _lens_to_cu(n)
    mattn.cache_write(k, v, c.k, c.v, c.table, cu, _i32(starts), **c.kw())
    ko, vo = mattn.cache_read(c.k, c.v, c.table, cu, T, _i32(starts), **c.kw())
    for x, y in ((k, ko), (v, vo)):
        assert not y[T - 5:].any()
        x, y = x[: T - 5].double(), y[: T - 5].double()
        if e4m3:  # half a step of e4m3, 2^-4 of a value, or of its smallest numbers, 2^-10 of the power (<= 2^-7 of the top)
            tol = torch.maximum(x.abs() / 16, x.abs().amax(dim=-1, keepdim=True) * 2.0 ** -17)
            assert bool(((x - y).abs() <= tol).all())
        else:
            assert torch.equal(x, y)


def test_cache_write_of_one_token_each():
    B, Hkv, d = 37, 4, 128
    for e4m3 in (False, True):
        c = Cache(B, Hkv, d, 16, 4, e4m3, seed=6)
        k, v = rows_of(5, B, Hkv, d)
        at = [(7 * b) % 64 for b in range(B)]
        mattn.cache_write(k, v, c.k, c.v, c.table, starts=_i32(at), **c.kw())
        a = mattn.cache_read(c.k, c.v, c.table, _i32(list(range(B + 1))), B, _i32(at), **c.kw())
        b = mattn.cache_read(*[x.clone() for x in (c.k, c.v)], c.table, _i32(list(range(B + 1))), B, _i32(at), **c.kw())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        if not e4m3:
            assert torch.equal(a[0], k) and torch.equal(a[1], v)


def test_cache_calls_without_rows():
    """A step with nothing to write or read back."""
    c = Cache(2, 2, 64, 16, 3, True)
    before = c.held("k")
    none = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    mattn.cache_write(none, none, c.k, c.v, c.table, _i32([0, 0, 0]), **c.kw())
    k, v = mattn.cache_read(c.k, c.v, c.table, _i32([0, 0, 0]), 0, **c.kw())
    assert k.shape == v.shape == (0, 2, 64) and torch.equal(c.held("k"), before)


@pytest.mark.parametrize("bad", [[5, 3, 40], [-7, 2000000000, 3], [2147483647, -2147483648, 0], [40, 40, 40]])
def test_cache_calls_with_sequences_that_are_none(bad):
    """Ends that do not ascend or lie outside the rows: every row stays inside its tensors."""
    c = Cache(2, 2, 64, 16, 3, True, spare=0)
    k, v = rows_of(1, 40, 2, 64)
    mattn.cache_write(k, v, c.k, c.v, c.table, _i32(bad), _i32([2147483647, -5]), **c.kw())
    mattn.cache_read(c.k, c.v, c.table, _i32(bad), 40, _i32([-2147483648, 7]), **c.kw())
    torch.cuda.synchronize()


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [3, 90])
def test_decode_paged_waits_run_out(d, e4m3, B):
    """In clusters (3 sequences) and in equal shares with the merge (90)."""
    H, Hkv = 8, 2
    c = Cache(B, Hkv, d, 16, 12, e4m3, seed=1)
    q = _randn(_gen(2), B, H, d)
    lens = _i32(([190, 3, 100] * B)[:B])
    ws = mattn.decode_paged_workspace(B, H, Hkv, 12, 16, d, e4m3)
    run = lambda: mattn.decode_paged(q, c.k, c.v, c.table, lens, workspace=ws, **c.kw())  # noqa: E731
    want = [x.clone() for x in run()]
    hook = mattn.lib().mattn_internal_paged_wait_selftest
    torch.cuda.synchronize()
    assert mattn.device_status()[0] == 0
    for fill in (0x7F, 0xFF):
        ws.fill_(fill)
        mattn.set_wait_timeout_ns(50_000_000)  # 50 ms
        assert hook(1) == 0
        try:
            run()
            torch.cuda.synchronize()
            rc, word = mattn.device_status()
        finally:
            hook(0)
            mattn.set_wait_timeout_ns(0)
        assert rc == mattn.ERR_TIMEOUT, hex(word)
        ws.fill_(fill)
        for a, b in zip(run(), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H", [4, 12])
def test_decode_paged_large_queries_small_keys(H, d):
    """Powers whose product is ordinary, the query's alone near the end of fp32's range."""
    c = Cache(2, 1, d, 16, 9, True, seed=21)
    c.ke[:] = torch.randint(1, 4, c.ke.shape, generator=_gen(1), device="cuda", dtype=torch.uint8)
    q = _randn(_gen(2), 2, H, d, scale=2.0 ** 121)
    c.freeze()
    o, lse = mattn.decode_paged(q, c.k, c.v, c.table, _i32([144, 77]), **c.kw())
    check_decode(o, lse, q, c, [list(range(144)), list(range(77))], None, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [2, 90])
def test_decode_paged_small_values(B, d):
    """Values down to fp32's least powers, in clusters (2 sequences) and in equal shares: none is flushed on the way."""
    H, Hkv = 12, 2
    c = Cache(B, Hkv, d, 16, 9, True, seed=22)
    c.ve[:] = torch.randint(8, 12, c.ve.shape, generator=_gen(1), device="cuda", dtype=torch.uint8)
    q = _randn(_gen(2), B, H, d)
    lens = [144 - b for b in range(B)]
    c.freeze()
    o, lse = mattn.decode_paged(q, c.k, c.v, c.table, _i32(lens), **c.kw())
    qd, got = q.double().cpu(), o.double().cpu()
    for b in (0, B - 1):
        for h in range(H):
            keys, values = c.rows(b, h // (H // Hkv), range(lens[b]))
            r, _, tol, _ = ref_decode(qd[b, h], keys, values, None, d ** -0.5, True)
            assert bool((r.abs().max() > 2.0 ** -119) and ((got[b, h] - r).abs() <= tol).all()), (b, h)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_write_of_one_token_each_by_value(e4m3, d):
    """A decode step's write: each token's codes and powers against the definition, every other byte as it was."""
    B, Hkv, page, slots = 37, 3, 16, 4
    c = Cache(B, Hkv, d, page, slots, e4m3, seed=6)
    k, v = rows_of(5, B, Hkv, d, "fused")
    k = k * torch.exp2(torch.arange(B, device="cuda") % 40 - 20).to(k.dtype)[:, None, None]
    at = [(7 * b) % (page * slots) for b in range(B)]
    at[3], at[9] = page * slots, -1  # past the table, before it: left out
    c.table[5] = -1
    before = {x: (c.held(x), None if not e4m3 else (c.ke if x == "k" else c.ve).cpu().clone()) for x in "kv"}
    mattn.cache_write(k, v, c.k, c.v, c.table, starts=_i32(at), **c.kw())
    placed, _ = ref_places(c, [1] * B, at, B)
    assert len(placed) == B - 3
    for name, rows, exps in (("k", k, c.ke), ("v", v, c.ve)):
        want, e_want = before[name]
        for t, p, r in placed:
            for h in range(Hkv):
                x = rows[t, h].double().cpu()
                if e4m3:
                    codes, e = ref_codes(x)
                    want[p, h, r], e_want[p, h, r] = codes * 2.0 ** (e - 127), e
                else:
                    want[p, h, r] = x
        assert torch.equal(c.held(name), want)
        if e4m3:
            assert torch.equal(exps.cpu(), e_want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("bad", [[5, 3, 40], [-7, 2000000000, 3], [2147483647, -2147483648, 0], [40, 40, 40], [0, 20, 40]])
def test_cache_calls_with_sequences_that_are_none_stay_inside(bad, e4m3):
    """What such calls write lies in their tensors: bytes around the pages, the powers and the outputs stay."""
    T, n, Hkv, page, d = 40, 6, 2, 16, 64
    guards = []

    def guarded(shape, dtype):
        size = math.prod(shape) * torch.empty((), dtype=dtype).element_size()
        x = torch.full((size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
        guards.append((x[:4096], x[4096 + size :]))
        return x[4096 : 4096 + size].view(dtype).view(shape)

    kp, vp = (guarded((n, Hkv, page, d), CODES if e4m3 else torch.bfloat16) for _ in range(2))
    ke, ve = (guarded((n, Hkv, page), torch.uint8) if e4m3 else None for _ in range(2))
    ko, vo = (guarded((T, Hkv, d), torch.bfloat16) for _ in range(2))
    table = _i32([[0, n - 1, 1 << 30], [n, 2, -1]])
    k, v = rows_of(1, T, Hkv, d)
    for starts in ([2147483647, -5], [-2147483648, 7], [40, 15], [0, 16]):
        mattn.cache_write(k, v, kp, vp, table, _i32(bad), _i32(starts), k_exponents=ke, v_exponents=ve)
        mattn.cache_read(kp, vp, table, _i32(bad), T, _i32(starts), k_exponents=ke, v_exponents=ve, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    for a, b in guards:
        assert bool((a == 0x5A).all()) and bool((b == 0x5A).all())


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("pool", ["shifted", "page", "row"])
def test_cache_pools(pool, e4m3):
    """k and v in one pool, the odd pages v's; codes and exponents of a page or of a row side by side: as apart."""
    if pool == "row" and not e4m3:
        pytest.skip("bf16 rows have no exponents")
    B, H, Hkv, d, page, slots = 3, 4, 2, 64, 16, 4
    n, T, es = 2 * B * slots, 90, 1 if e4m3 else 2
    dtype = CODES if e4m3 else torch.bfloat16
    ke = ve = None
    if pool == "shifted":
        both = torch.zeros((n, Hkv, page, d * es), dtype=torch.uint8, device="cuda").view(dtype)
        k, v = both[:-1], both[1:]
        if e4m3:
            exps = torch.zeros((n, Hkv, page), dtype=torch.uint8, device="cuda")
            ke, ve = exps[:-1], exps[1:]
        table = _i32([[2 * (b * slots + j) for j in range(slots)] for b in range(B)])
    else:
        table = _i32([[n - 1 - b * slots - j for j in range(slots)] for b in range(B)])
        if pool == "page":
            rows = Hkv * page * d * es
            both = torch.zeros((n, 2 * rows + 2 * Hkv * page), dtype=torch.uint8, device="cuda")
            k, v = (both[:, i * rows : (i + 1) * rows].view(dtype).view(n, Hkv, page, d) for i in range(2))
            if e4m3:
                ke, ve = (both[:, 2 * rows + i * Hkv * page : 2 * rows + (i + 1) * Hkv * page].view(n, Hkv, page) for i in range(2))
        else:
            both = torch.zeros((n, Hkv, page, 2 * d + 16), dtype=torch.uint8, device="cuda")
            k, v = both[..., :d].view(dtype), both[..., d : 2 * d].view(dtype)
            ke, ve = both[..., 2 * d], both[..., 2 * d + 1]
    c = Cache(B, Hkv, d, page, slots, e4m3)
    lens = [50, 7, 33]
    x, y = rows_of(7, T, Hkv, d)
    cu, q = _lens_to_cu(lens), _randn(_gen(8), B, H, d)
    got = []
    for kp, vp, t, kw in ((c.k, c.v, c.table, c.kw()), (k, v, table, dict(k_exponents=ke, v_exponents=ve))):
        mattn.cache_write(x, y, kp, vp, t, cu, **kw)
        got.append([*mattn.cache_read(kp, vp, t, cu, T, **kw), *mattn.decode_paged(q, kp, vp, t, _i32(lens), **kw)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [2, 90])
def test_decode_paged_large_values(B, d):
    """Values up to 2^117, rows of zeros (the least power) among them; keys of 2^110 under queries of 2^-117."""
    H, Hkv = 12, 2
    c = Cache(B, Hkv, d, 16, 9, True, seed=23)
    c.ve[:] = torch.randint(233, 236, c.ve.shape, generator=_gen(1), device="cuda", dtype=torch.uint8)
    c.ke[:] = 231
    zero = torch.rand(c.ve.shape, generator=_gen(3), device="cuda") < 0.2
    c.ve[zero], Cache._bytes(c.v)[zero] = 0, 0
    q = _randn(_gen(2), B, H, d, scale=2.0 ** -117)
    lens = [144 - b for b in range(B)]
    c.freeze()
    o, lse = mattn.decode_paged(q, c.k, c.v, c.table, _i32(lens), scale=2.0 ** -4, **c.kw())
    rows = [0, B - 1]
    part = Cache.__new__(Cache)
    part.__dict__.update(c.__dict__, table=c.table[rows])
    check_decode(o[rows], lse[rows], q[rows], part, [range(lens[b]) for b in rows], None, 2.0 ** -4)
