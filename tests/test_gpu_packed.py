"""GPU tests of attention over packed sequences (attention_packed) against a plain
implementation in 64 bits written here, and of a serving step's operators together.

Tolerances, derived before the first run; u = 2^-8 is bf16's half step relative to
the value, e = 2^-24 fp32's.  o = sum p v / sum p: weights rounded to bf16 (u each),
the output rounded once (u): |do| <= u |o| + (u + 2 t + 2^-13) A with A = sum p |v| /
sum p.  Where the sum of the rounded weights p (1 + c_j), |c_j| <= u, divides (rows of few
keys), o is off by sum p c_j (v_j - o) / sum p, and sum p |v_j - o| / sum p <= A + |o|: u |o|
more, and u^2 (A + |o|), which 2^-13 A holds.
t = d e max_j sum_c |q_c k_jc| scale is the error of a score, which moves a weight and the
sum by as much; 2^-13 for exponentials and sums.  lse: t + 2^-19 (1 + |lse|).
"""

import math
import os

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

U, E = 2.0 ** -8, 2.0 ** -24
NAN, INF = float("nan"), float("inf")


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


def _cu(n, at=0):
    c = [at]
    for x in n:
        c.append(c[-1] + x)
    return c


def ref_sequence(q, k, v, causal, window, sink, scale):
    """One sequence and head: q [n, d], k, v [m, d] in 64 bits -> (o, lse, tolerances)."""
    n, m, d = q.shape[0], k.shape[0], q.shape[1]
    s = q @ k.T * scale
    if causal:
        age = torch.arange(m - n, m, device=q.device)[:, None] - torch.arange(m, device=q.device)
        s = s.masked_fill((age < 0) | (age >= (window or 1 << 40)), -INF)
    top = s.amax(dim=1) if m else torch.full((n,), -INF, dtype=q.dtype, device=q.device)
    if sink is not None:
        top = top.clamp(min=sink)
    ref = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp(s - ref[:, None])
    z = p.sum(dim=1) + (math.e ** (sink - ref) if sink is not None else 0)
    w = p / torch.where(z > 0, z, torch.ones_like(z))[:, None]
    o, a = w @ v, w @ v.abs()
    lse = torch.where(z > 0, ref + torch.log(z), torch.full_like(z, -INF))
    t = (q.abs() @ k.abs().T).amax(dim=1) * scale * d * E if m else torch.zeros_like(z)
    return o, lse, 2 * U * o.abs() + (U + 2 * t + 2.0 ** -13)[:, None] * a, t + 2.0 ** -19 * (1 + lse.abs().nan_to_num(posinf=0))


def check(o, lse, q, k, v, cq, ck, causal, window, sink, scale, tag=""):
    H, Hkv = q.shape[1], k.shape[1]
    for b in range(len(cq) - 1):
        i, j = slice(cq[b], cq[b + 1]), slice(ck[b], ck[b + 1])
        if cq[b] == cq[b + 1]:
            continue
        for h in range(H):
            r, l, tol, tl = ref_sequence(q[i, h].double(), k[j, h // (H // Hkv)].double(), v[j, h // (H // Hkv)].double(), causal,
                                         window, None if sink is None else float(sink[h]), scale)
            err = (o[i, h].double() - r).abs() - tol
            assert bool((err <= 1e-30).all()), f"{tag} b{b} h{h}: o off by {float(err.max()):.3e} over its bound, row {int(err.amax(dim=1).argmax())}"
            got, none = lse[h, i].double(), torch.isinf(l)
            assert torch.equal(got[none], l[none]), f"{tag} b{b} h{h}: lse of rows without keys"
            err = (got - l)[~none].abs() - tl[~none]
            assert bool((err <= 0).all()), f"{tag} b{b} h{h}: lse off by {float(err.max()):.3e} over its bound"


def inputs(T, Tk, H, Hkv, d, seed=0, layout="dense", q_scale=1.0):
    g = _gen(seed)
    if layout == "fused":  # one projection's output
        x = _randn(g, max(T, Tk), H + 2 * Hkv, d)
        return x[:T, :H] * q_scale if q_scale != 1 else x[:T, :H], x[:Tk, H : H + Hkv], x[:Tk, H + Hkv :]
    if layout == "heads":  # [heads, T, d] in memory
        return tuple(_randn(g, h, n, d).transpose(0, 1) for h, n in ((H, T), (Hkv, Tk), (Hkv, Tk)))
    return _randn(g, T, H, d, scale=q_scale), _randn(g, Tk, Hkv, d), _randn(g, Tk, Hkv, d)


def packed_case(nq, H, Hkv, d, nk=None, causal=True, window=None, sink=False, scale=None, seed=0, layout="dense", pad=(0, 0),
                q_scale=1.0):
    """pad: rows of no sequence before the first and behind the last one, NaN in q, k and v."""
    cq = _cu(nq, pad[0])
    ck = cq if nk is None else _cu(nk, pad[0])
    T, Tk = cq[-1] + pad[1], ck[-1] + pad[1]
    q, k, v = inputs(T, Tk, H, Hkv, d, seed, layout, q_scale)
    for x, c in ((q, cq), (k, ck), (v, ck)):
        x[: c[0]], x[c[-1]:] = NAN, NAN
    sk = torch.linspace(-2, 3, H, device="cuda") if sink else None
    out = torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((H, T), 7.0, device="cuda")
    r = mattn.attention_packed(q, k, v, _i32(cq), None if nk is None else _i32(ck), causal=causal, window=window, sink=sk,
                               scale=scale, out=out, lse=lse)
    torch.cuda.synchronize()
    assert r[0] is not None and r[0].data_ptr() == out.data_ptr() and r[1].data_ptr() == lse.data_ptr()
    for x in (out[: cq[0]], out[cq[-1]:], lse[:, : cq[0]], lse[:, cq[-1]:]):
        assert bool((x == 7).all())
    check(out, lse, q, k, v, cq, ck, causal, window, sk, d ** -0.5 if scale is None else scale)
    return out, lse


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads", [(1, 1), (4, 4), (8, 2), (6, 1)])
def test_packed_heads(heads, causal, d):
    packed_case([5, 130, 300, 1], *heads, d, causal=causal, seed=d + heads[0])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq", [[1], [2], [127, 128, 129], [255, 256, 257], [0, 3, 0, 0, 511, 0], [1] * 70, [1025], [640, 1, 640]])
def test_packed_lengths(nq, causal):
    packed_case(nq, 4, 2, 128, causal=causal, seed=len(nq) + nq[0], sink=nq[0] == 127)


@pytest.mark.parametrize("d", [80, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 100, 128, 129, 500, 100000])
def test_packed_windows(window, d):
    packed_case([700, 33, 260], 4, 1, d, window=window, seed=window, sink=window == 100)
    packed_case([70, 33, 260], 4, 2, d, nk=[900, 33, 100], window=window, seed=window)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
def test_packed_with_cached_rows(d, causal):
    """More keys than queries, none, fewer (rows that see nothing under causality)."""
    nq, nk = [100, 1, 64, 300, 7, 140], [612, 900, 0, 120, 0, 139]
    packed_case(nq, 4, 2, d, nk=nk, causal=causal, seed=d)
    packed_case(nq, 4, 2, d, nk=nk, causal=causal, seed=d, sink=True, scale=0.4)
    packed_case([200, 3], 2, 1, d, nk=[0, 0], causal=causal, sink=True)


@pytest.mark.parametrize("layout", ["fused", "heads"])
@pytest.mark.parametrize("d", [64, 80, 128, 256])
def test_packed_layouts(d, layout):
    packed_case([100, 300, 29], 6, 2, d, layout=layout, seed=1)
    packed_case([100, 300], 4, 1, d, nk=[150, 300], layout=layout, seed=2, causal=False)


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
def test_packed_padding(d):
    """Rows of no sequence, NaN: unused, and left as they are."""
    packed_case([100, 0, 257], 4, 2, d, pad=(3, 40), seed=3)
    packed_case([130, 200], 4, 2, d, nk=[131, 333], pad=(9, 200), causal=False, seed=4)


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -20, 40.0, 400.0])
def test_packed_score_ranges(q_scale):
    """Equal scores; scores whose exponentials leave the range of fp32 in either direction."""
    packed_case([300, 20, 515], 4, 2, 128, q_scale=q_scale, seed=5, scale=0.1)
    packed_case([300, 20, 515], 4, 2, 80, q_scale=q_scale, seed=6, causal=False, sink=True, scale=0.1)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("nq", [[1], [63, 64, 65], [127, 128, 129], [255, 256, 257], [0, 3, 0, 0, 511, 0], [1] * 70, [1025], [640, 1, 640]])
def test_packed_256_lengths(nq, causal):
    packed_case(nq, 4, 2, 256, causal=causal, seed=len(nq) + nq[0], sink=nq[0] == 127)
    packed_case(nq, 12, 1, 256, nk=[2 * n + 1 for n in nq], causal=causal, seed=len(nq))


@pytest.mark.parametrize("q_scale", [0.0, 2.0 ** -20, 40.0, 400.0])
def test_packed_256_score_ranges(q_scale):
    packed_case([300, 20, 515], 4, 2, 256, q_scale=q_scale, seed=5, scale=0.1)
    packed_case([300, 20, 515], 4, 2, 256, q_scale=q_scale, seed=6, causal=False, sink=True, scale=0.1)


@pytest.mark.parametrize("d", [64, 256])
def test_packed_many_sequences_without_keys(d):
    """A few with keys, hundreds without behind them: zeros, or the sink's part."""
    nq = [300] + [3] * 400 + [200, 64]
    nk = [300] + [0] * 400 + [500, 64]
    packed_case(nq, 8, 2, d, nk=nk, seed=13)
    packed_case(nq, 8, 8, d, nk=nk, seed=14, sink=True, causal=False)


def test_packed_256_more_items_than_sms():
    """Items behind one another in a CTA, marked ones among them."""
    nq = [2000, 5, 700, 1300, 64, 900]
    packed_case(nq, 16, 4, 256, seed=11)
    cq = _cu(nq)
    q, k, v = inputs(cq[-1], cq[-1], 16, 4, 256, 12)
    want, lse = mattn.attention_packed(q, k, v, _i32(cq))
    for b in (0, 2, 3, 5):
        v[cq[b + 1] - 1] = NAN  # the last query's alone
    for _ in range(3):
        o, l = mattn.attention_packed(q, k, v, _i32(cq))
        hit = torch.zeros(cq[-1], dtype=torch.bool, device="cuda")
        hit[[cq[b + 1] - 1 for b in (0, 2, 3, 5)]] = True
        assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], want[~hit]) and torch.equal(l, lse)


def test_packed_many_sequences():
    """More sequences than the plan takes at a time."""
    g = torch.Generator().manual_seed(1)
    nq = torch.randint(0, 9, (2500,), generator=g).tolist()
    nq[1700] = 600
    packed_case(nq, 2, 1, 64, seed=7)


def test_packed_long():
    packed_case([5000, 300, 9000, 1], 2, 1, 128, seed=8)
    packed_case([40, 9], 2, 2, 64, nk=[70000, 20], seed=9)
    packed_case([3000, 200, 40, 1], 2, 1, 256, nk=[3000, 9000, 70000, 2], seed=10)


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_values_that_are_not_finite(d, causal):
    """Infinite and NaN values reach the rows that see them, in their columns, and no other;
    NaN keys and queries likewise."""
    nq, H, Hkv = [200, 150, 90], 4, 2
    cq = _cu(nq)
    q, k, v = inputs(cq[-1], cq[-1], H, Hkv, d, 3)
    call = lambda: mattn.attention_packed(q, k, v, _i32(cq), causal=causal)  # noqa: E731
    want, lse = [x.clone() for x in call()]
    planted = [(0, 70, 0, 3, INF), (0, 199, 1, 5, NAN), (1, 0, 0, 6, -INF), (1, 149, 0, 7, INF), (1, 130, 0, 7, -INF), (2, 40, 1, d - 1, NAN),
               (2, 64, 0, d - 17, INF)]
    for b, j, h, c, x in planted:
        v[cq[b] + j, h, c] = x
    o, l = call()
    assert torch.equal(l, lse)
    expect = want.double()
    for b, j, h, c, x in planted:
        rows = slice(cq[b] + (j if causal else 0), cq[b + 1])
        expect[rows, 2 * h : 2 * h + 2, c] += x
    # (what is not finite: exactly so; the rest to the bit but for the sums' finite part, which is the same)
    o = o.double()
    assert torch.equal(torch.isnan(o), torch.isnan(expect)) and torch.equal(torch.isinf(o), torch.isinf(expect))
    assert torch.equal(o[torch.isinf(o)], expect[torch.isinf(expect)])
    fine = torch.isfinite(expect)
    assert torch.equal(o[fine], expect[fine])
    q, k, v = inputs(cq[-1], cq[-1], H, Hkv, d, 3)
    k[cq[1] + 60, 1, 2] = NAN
    q[cq[2] + 33, 0, 1] = NAN
    o, l = call()
    hit = torch.zeros((cq[-1], H), dtype=torch.bool, device="cuda")
    hit[cq[1] + (60 if causal else 0) : cq[2], 2:] = True
    hit[cq[2] + 33, 0] = True
    assert torch.isnan(o[hit]).all() and torch.isnan(l.t()[hit]).all()
    assert torch.equal(o[~hit], want[~hit]) and torch.equal(l.t()[~hit], lse.t()[~hit])


def test_packed_order_of_sequences_does_not_matter():
    """A sequence's rows bit for bit, wherever in the batch it lies."""
    nq = [300, 77, 513, 1]
    q, k, v = inputs(sum(nq), sum(nq), 4, 2, 128, 5)
    cq = _cu(nq)
    a, la = mattn.attention_packed(q, k, v, _i32(cq))
    order = [2, 0, 3, 1]
    rows = torch.cat([torch.arange(cq[b], cq[b + 1]) for b in order]).cuda()
    b, lb = mattn.attention_packed(q[rows], k[rows], v[rows], _i32(_cu([nq[i] for i in order])))
    assert torch.equal(a[rows], b) and torch.equal(la[:, rows], lb)


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
def test_packed_one_key(d):
    """A row that sees one key: its value, bit for bit."""
    n = [1, 300, 2, 129]
    cq = _cu(n)
    q, k, v = inputs(cq[-1], cq[-1], 4, 2, d, 8, q_scale=3.0)
    o, _ = mattn.attention_packed(q, k, v, _i32(cq), window=1)
    assert torch.equal(o, v.repeat_interleave(2, dim=1))
    o, _ = mattn.attention_packed(q, k, v, _i32(cq))
    for c in cq[:-1]:
        assert torch.equal(o[c], v[c].repeat_interleave(2, dim=0))


def test_packed_agrees_with_attention():
    """One sequence: the causal forward of the package, within the two calls' roundings."""
    from workloads import MaskSpec

    n, H, d = 900, 4, 128
    q, k, v = inputs(n, n, H, H, d, 6)
    o, lse = mattn.attention_packed(q, k, v, _i32([0, n]))
    mask = mattn.prepare(MaskSpec("causal_window", [n] * H), H, n)
    r, l = mattn.attention(*(x.transpose(0, 1)[None].contiguous() for x in (q, k, v)), mask)
    r, l = r[0].transpose(0, 1).double(), l[0]
    assert bool(((o.double() - r).abs() <= 2 * U * (r.abs() + 4)).all()) and bool(((lse - l).abs() < 1e-5 * (1 + l.abs())).all())


def test_packed_outputs_made_by_the_call():
    q, k, v = inputs(50, 50, 4, 2, 64, 7)
    want, lse = mattn.attention_packed(q, k, v, _i32([4, 30, 45]))
    junk = [torch.full_like(want, NAN) for _ in range(3)]
    del junk
    o, none = mattn.attention_packed(q, k, v, _i32([4, 30, 45]), want_lse=False)
    assert none is None and torch.equal(o, want)
    assert not o[:4].any() and not o[45:].any() and not lse[:, :4].any() and not lse[:, 45:].any()
    empty = mattn.attention_packed(q[:0], k[:0], v[:0], _i32([0, 0]))
    assert empty[0].shape == (0, 4, 64) and empty[1].shape == (4, 0)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("T,B", [(300, 3), (9000, 3), (9000, 2000)])
def test_packed_sequences_that_are_none(T, B, d):
    """Ends that do not ascend, overlap or lie outside the rows: clamped, nothing outside the outputs
    is written, and the next call is right."""
    q, k, v = inputs(T, T, 4, 2, d, 9)
    g = torch.Generator().manual_seed(3)
    for low, high in ((-50, T + 50), (-(1 << 31), (1 << 31) - 1)):
        cu = torch.randint(low, high, (B + 1,), generator=g).to(torch.int32).cuda()
        guard = torch.full((T + 64, 4, d), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((4, T), 7.0, device="cuda")
        mattn.attention_packed(q, k, v, cu, cu.flip(0), out=guard[32 : 32 + T], lse=lse)
        torch.cuda.synchronize()
        assert bool((guard[:32] == 7).all()) and bool((guard[32 + T:] == 7).all())
    c = _cu([100, 77, T - 177])
    o, lse = mattn.attention_packed(q, k, v, _i32(c))
    check(o, lse, q, k, v, c, c, True, None, None, d ** -0.5)


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
def test_packed_waits_run_out(d):
    q, k, v = inputs(700, 700, 4, 2, d, 7)
    cu = _i32([0, 300, 700])
    ws = mattn.attention_packed_workspace(700, 2, 4)
    run = lambda: mattn.attention_packed(q, k, v, cu, workspace=ws)  # noqa: E731
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


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("window", [None, 20, 64, 100, 128, 200])
def test_packed_row_of_a_prompt_in_chunks(window, d):
    """A row's bits come from its own keys alone: a prompt whole, and its rows from any one on as a chunk."""
    n = 400
    q, k, v = inputs(n, n, 4, 2, d, 15)
    o, lse = mattn.attention_packed(q, k, v, _i32([0, n]), window=window)
    for at, end in ((1, n), (37, n), (100, n), (127, 300), (128, n), (200, 201), (255, 390), (300, n)):
        a, l = mattn.attention_packed(q[at:end], k[:end], v[:end], _i32([0, end - at]), _i32([0, end]), window=window)
        assert torch.equal(a, o[at:end]) and torch.equal(l, lse[:, at:end]), at


@pytest.mark.parametrize("d", [64, 80, 96, 128, 256])
@pytest.mark.parametrize("causal,window", [(True, None), (False, None), (True, 65), (True, 300)])
def test_packed_rounding_of_rows_of_many_keys(causal, window, d):
    """A row whose last key lies behind its sequence's first 128 divides by the sum of the weights as they were: one u |o|
    less than the bound of the other rows."""
    nq, nk = [700, 129, 260, 40], [700, 300, 260, 41]
    cq, ck = _cu(nq), _cu(nk)
    q, k, v = inputs(cq[-1], ck[-1], 4, 2, d, 17)
    o, lse = mattn.attention_packed(q, k, v, _i32(cq), _i32(ck), causal=causal, window=window)
    check(o, lse, q, k, v, cq, ck, causal, window, None, d ** -0.5)
    for b, (n, m) in enumerate(zip(nq, nk)):
        first = max(0, 128 - (m - n)) if causal else (0 if m > 128 else n)  # the first row that sees key 128 or later
        i, j = slice(cq[b] + first, cq[b + 1]), slice(ck[b], ck[b + 1])
        for h in range(4):
            r, _, tol, _ = ref_sequence(q[cq[b] : cq[b + 1], h].double(), k[j, h // 2].double(), v[j, h // 2].double(), causal, window,
                                        None, d ** -0.5)
            assert bool(((o[i, h].double() - r[first:]).abs() <= (tol - U * r.abs())[first:]).all()), (b, h)


def test_packed_256_items_longer_than_the_wait_limit():
    """The limit is one for a wait without progress: items of thousands of key tiles, several a CTA, run through."""
    n, m, H = 2560, 1 << 20, 32
    q, k, v = inputs(n, m, H, 1, 256, 16)
    call = lambda: mattn.attention_packed(q, k, v, _i32([0, n]), _i32([0, m]), causal=False)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    mattn.set_wait_timeout_ns(4_000_000)  # 4 ms; an item takes about 13
    try:
        got = call()
        torch.cuda.synchronize()
        rc, word = mattn.device_status()
    finally:
        mattn.set_wait_timeout_ns(0)
    assert rc == 0, hex(word)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_packed_hundreds_of_sequences_without_rows():
    """Few rows among many empty sequences, on both sides of the border between dealing items and planning them."""
    for B in (384, 385, 3000):
        nq = [0] * B
        nq[0], nq[B // 2], nq[B - 1] = 40, 7, 17
        packed_case(nq, 4, 2, 64, seed=B)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
def test_packed_items_longer_than_the_wait_limit(causal, d):
    """The same where an item is a pair of query tiles: the second one without rows, or both, several items a CTA."""
    m = 1 << 20
    for nq, H in (([100], 2), ([100] * 3, 200), ([300], 2)):
        T = sum(nq)
        q, k, v = inputs(T, m, H, 1, d, 18)
        cu, cu_k = _i32(_cu(nq)), _i32([0] * len(nq) + [m])
        call = lambda: mattn.attention_packed(q, k, v, cu, cu_k, causal=causal)  # noqa: E731
        want = call()
        torch.cuda.synchronize()
        mattn.set_wait_timeout_ns(3_000_000)  # 3 ms; an item takes about 8
        try:
            got = call()
            torch.cuda.synchronize()
            rc, word = mattn.device_status()
        finally:
            mattn.set_wait_timeout_ns(0)
        assert rc == 0, hex(word)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
