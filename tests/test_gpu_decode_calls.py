"""GPU tests of the decode step's operators: what a call reads and returns when
the tensors of a plan move, outputs are left to the call, and rows start off
the widest alignment.  Tolerances as in test_gpu_decode_ops.py, whose 64-bit
forms are used."""

import math
import os
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")
import test_gpu_decode_ops as ops  # noqa: E402  (the 64-bit forms)


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


# ------------------------------------------------------------------ a plan's tensors
def _rope_inputs(seed=1, B=2, N=3, H=4, Hkv=2, d=128):
    g = _gen(seed)
    return tuple(_randn(g, B, N, h, d) for h in (H, Hkv, Hkv))


def _freq(n=64, base=1e4):
    return (base ** (-torch.arange(n, device="cuda") / n)).float()


@pytest.mark.parametrize("which", ["inv_freq", "q_weight", "k_weight"])
@pytest.mark.parametrize("how", ["values", "storage", "attribute"])
def test_rope_plan_reads_its_tensors_at_each_call(which, how):
    """New values, new storage behind the same tensor (the old one kept alive here
    and overwritten) and another tensor on the plan: the next call uses them."""
    x = _rope_inputs()
    g = _gen(2)
    old = {"inv_freq": _freq(), "q_weight": 1 + 0.2 * torch.randn(128, generator=g, device="cuda"),
           "k_weight": 1 + 0.2 * torch.randn(128, generator=g, device="cuda")}
    new = dict(old, **{which: _freq(base=50.0) if which == "inv_freq" else 2 + torch.rand(128, generator=g, device="cuda")})
    kw = lambda t: dict(inv_freq=t["inv_freq"].clone(), q_weight=t["q_weight"].clone(), k_weight=t["k_weight"].clone())  # noqa: E731
    starts = _i32([5, 90])
    caches = lambda: dict(k_out=torch.zeros((2, 2, 100, 128), dtype=torch.bfloat16, device="cuda"),  # noqa: E731
                          v_out=torch.zeros((2, 2, 100, 128), dtype=torch.bfloat16, device="cuda"), starts=starts)
    want = mattn.qk_rope(*x, mattn.RopePlan(**kw(new)), **caches())
    plan = mattn.RopePlan(**kw(old))
    before = mattn.qk_rope(*x, plan, **caches())
    assert not all(torch.equal(a, b) for a, b in zip(before, want))
    t = getattr(plan, which)
    if how == "values":
        t.copy_(new[which])
    elif how == "storage":
        keep = t.data
        t.data = new[which].clone()
        keep.fill_(-3.0)
    else:
        setattr(plan, which, new[which].clone())
        t.fill_(-3.0)
    got = mattn.qk_rope(*x, plan, **caches())
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_rope_plan_checks_its_tensors_at_each_call():
    x = _rope_inputs()
    for name, bad in (("q_weight", torch.ones(128)), ("k_weight", torch.ones(128, device="cuda", dtype=torch.bfloat16)),
                      ("q_weight", torch.ones(64, device="cuda")), ("k_weight", torch.ones(256, device="cuda")[::2]),
                      ("inv_freq", torch.ones(64)), ("inv_freq", torch.ones(56, device="cuda")),
                      ("inv_freq", torch.ones((8, 8), device="cuda")), ("inv_freq", None)):
        plan = mattn.RopePlan(_freq(), q_weight=torch.ones(128, device="cuda"), k_weight=torch.ones(128, device="cuda"))
        setattr(plan, name, bad)
        with pytest.raises(ValueError):
            mattn.qk_rope(*x, plan)
    plan = mattn.RopePlan(_freq(), [16, 24, 24])
    assert plan.sections == [16, 24, 24] and plan.eps == 1e-6 and plan.interleaved is False
    for name, value in (("sections", [64]), ("eps", 1.0), ("interleaved", True)):
        with pytest.raises(AttributeError):
            setattr(plan, name, value)
    plan.q_weight = torch.ones(128, device="cuda")  # (one norm alone)
    assert torch.isfinite(mattn.qk_rope(*x, plan)[0].float()).all()


# ------------------------------------------------------------------ outputs that the call makes
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_outputs_made_by_the_call_hold_nothing_else(dtype):
    """Padding rows of outputs that the call makes are zeros, the others as in given outputs."""
    g = _gen(3)
    B, N, H, Hkv, d = 3, 50, 4, 2, 64
    x = tuple(_randn(g, B, N, h, d, dtype=dtype) for h in (H, Hkv, Hkv))
    plan = mattn.RopePlan(_freq(32), q_weight=torch.ones(d, device="cuda"))
    lens = _i32([50, 0, 17])
    given = [torch.zeros((B, h, N, d), dtype=dtype, device="cuda") for h in (H, Hkv, Hkv)]
    mattn.qk_rope(*x, plan, *given, lens=lens)
    for _ in range(4):
        junk = [torch.full_like(t, float("nan")) for t in given]  # what the allocator hands out next
        del junk
        for a, b in zip(mattn.qk_rope(*x, plan, lens=lens), given):
            assert torch.equal(a, b)
    q, k, v = mattn.qk_rope(x[0], x[1], None, plan, lens=lens)
    assert v is None and torch.equal(q, given[0]) and torch.equal(k, given[1])
    got = mattn.qk_rope(*x, plan, lens=lens, v_out=given[2].clone())  # one of them given
    for a, b in zip(got, given):
        assert torch.equal(a, b)


def test_rope_refuses_starts_without_caches():
    x = _rope_inputs()
    plan = mattn.RopePlan(_freq())
    starts = _i32([0, 1])
    cache = torch.zeros((2, 2, 9, 128), dtype=torch.bfloat16, device="cuda")
    for kw in (dict(starts=starts), dict(starts=starts, k_out=cache), dict(k_out=cache),
               dict(starts=starts, v_out=torch.zeros((2, 2, 3, 128), dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(ValueError):
            mattn.qk_rope(*x, plan, **kw)
    with pytest.raises(ValueError):
        mattn.qk_rope(x[0], x[1], None, plan, starts=starts)
    mattn.qk_rope(x[0], x[1], None, plan, starts=starts, k_out=cache)
    mattn.qk_rope(*x, plan, starts=starts, k_out=cache, v_out=cache.clone())


# ------------------------------------------------------------------ first calls
FIRST_UNDER_CAPTURE = """
import torch
import block_sparse_attention_masked_gb300 as mattn
torch.manual_seed(1)
def randn(*s):
    return torch.randn(s, device="cuda").to(torch.bfloat16)
q, k, v, qd, cache = randn(2, 3, 8, 128), randn(2, 3, 2, 128), randn(2, 3, 2, 128), randn(2, 8, 128), randn(2, 2, 640, 128)
plan = mattn.RopePlan(torch.ones(64, device="cuda"))
calls = {"rope": lambda: mattn.qk_rope(q, k, v, plan),
         "means": lambda: (mattn.block_means(cache, 16),),
         "select": lambda: (mattn.decode_select(qd, cache, 16, 7),),
         "refused": lambda: mattn.decode_shared(qd, cache[0], cache[1], cache, cache)}
call = calls[WHICH]
torch.cuda.synchronize()
if WHICH == "refused":
    graph = torch.cuda.CUDAGraph()
    try:
        with torch.cuda.graph(graph):
            call()
        raise SystemExit("captured an allocation")
    except mattn.MattnError as e:
        assert e.code == mattn.ERR_UNSUPPORTED, e
else:
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, call()):
        assert torch.equal(a, b)
print("fine")
"""


@pytest.mark.parametrize("which", ["rope", "means", "select", "refused"])
def test_first_call_of_a_process_under_capture(which):
    """qk_rope, block_means and decode_select need nothing of the device before their
    first launch; decode_shared makes the error word, and says so."""
    env = dict(os.environ, PYTHONPATH=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    r = subprocess.run([sys.executable, "-c", f"WHICH = {which!r}\n" + FIRST_UNDER_CAPTURE], env=env, timeout=240,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr


# ------------------------------------------------------------------ errors of calls that allocate
def test_out_of_memory_is_torchs_own_error():
    """Outputs and workspaces that torch's allocator has no room for raise its
    OutOfMemoryError, and the next call runs."""
    g = _gen(6)
    cache, q = _randn(g, 8, 8, 16384, 128), _randn(g, 8, 8, 128)
    want = mattn.block_means(cache[:, :, :64].contiguous(), 16)
    small = cache[:, :, :64].contiguous()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (4 << 20)) / total)
    try:
        hold = []
        with pytest.raises(torch.OutOfMemoryError):
            for _ in range(64):
                hold.append(mattn.block_means(cache, 16))
        with pytest.raises(torch.OutOfMemoryError):
            for _ in range(100000):
                hold.append(mattn.decode_shared(q, cache[0], cache[0], cache, cache))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(mattn.block_means(small, 16), want)


def test_want_lse_must_be_a_truth_value():
    g = _gen(7)
    q, c = _randn(g, 1, 2, 64), _randn(g, 1, 2, 16, 64)
    with pytest.raises(ValueError):
        mattn.decode_shared(q, c[0], c[0], c, c, want_lse=torch.ones(2, device="cuda"))
    assert mattn.decode_shared(q, c[0], c[0], c, c, want_lse=False)[1] is None


# ------------------------------------------------------------------ angles
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_rope_angles_next_to_quarter_turns(inter, sign):
    """Rows (1, 0) in fp32 come out as the cosine and sine of their angle: each within
    four half steps of its own value (one step of sincospi, half a step of the
    reduced angle), next to its zeros too, and 2^-51 of the whole angle (the 64-bit
    fraction's two roundings, and the formula's)."""
    n, R = 20000, 32
    f = _freq(R)
    x = torch.zeros((1, n, 1, 2 * R), device="cuda")
    x[..., (slice(0, None, 2) if inter else slice(0, R))] = 1.0
    # positions whose angle at pair 0 (1 radian a position) comes near quarter turns, among others
    near = [round(j * math.pi / 2) for j in range(1, n // 2)] + [355 * j for j in range(1, 200)] + [103993, 104348, 208341, 312689]
    pos = torch.cat((torch.tensor(near), torch.arange(n - len(near)))).to(torch.int32).cuda() * sign
    q, _, _ = mattn.qk_rope(x, x, None, mattn.RopePlan(f, interleaved=inter), positions=pos.view(1, 1, n).contiguous())
    got = q[0, 0].double()
    t = pos.double()[:, None] * f.double()
    c, s = (got[:, 0::2], got[:, 1::2]) if inter else (got[:, :R], got[:, R:])
    for value, ref in ((c, t.cos()), (s, t.sin())):
        bound = 4 * 2.0 ** -24 * ref.abs() + 2.0 ** -51 * t.abs()
        assert bool(((value - ref).abs() <= bound).all()), float(((value - ref).abs() - bound).max())


@pytest.mark.parametrize("sign", [1, -1])
def test_rope_angles_of_small_frequencies_at_far_positions(sign):
    """Frequencies of either sign down to 10^-9 at positions of any size: within four
    half steps of each value, 2^-51 of the whole angle and 2^-30 (the fraction's last bit, 2^-64 of
    a turn, at 2^31 positions is 2^-30.3)."""
    n, R = 4000, 32
    f = sign * _freq(R, base=1e9)
    x = torch.zeros((1, n, 1, 2 * R), device="cuda")
    x[..., :R] = 1.0
    pos = torch.randint(-(1 << 31), 1 << 31, (n,), generator=_gen(9), device="cuda", dtype=torch.int64).to(torch.int32)
    pos[:4] = _i32([(1 << 31) - 1, -(1 << 31), 0, 1])
    q, _, _ = mattn.qk_rope(x, x, None, mattn.RopePlan(f), positions=pos.view(1, 1, n))
    got = q[0, 0].double()
    t = pos.double()[:, None] * f.double()
    for value, ref in ((got[:, :R], t.cos()), (got[:, R:], t.sin())):
        bound = 4 * 2.0 ** -24 * ref.abs() + 2.0 ** -51 * t.abs() + 2.0 ** -30
        assert bool(((value - ref).abs() <= bound).all()), float(((value - ref).abs() - bound).max())


# ------------------------------------------------------------------ rows off the widest alignment
def _off(t, by, row_pad=0):
    """A copy of t, `by` elements off the start of its allocation, tokens row_pad elements further apart."""
    B, N, h, d = t.shape
    row = h * d + row_pad
    buf = torch.full((B * N * row + by + 64,), float("nan"), dtype=t.dtype, device="cuda")
    v = buf[by:].as_strided((B, N, h, d), (N * row, row, d, 1), by)
    v.copy_(t)
    return v


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [32, 64, 80, 96, 128, 256])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_rows_on_16_byte_boundaries(dtype, d, inter):
    """Inputs, outputs or token strides 16 but not 32 bytes aligned, each alone and together:
    the result of aligned rows."""
    g = _gen(d)
    B, N, H, Hkv = 2, 5, 3, 2
    e = 16 // torch.empty((), dtype=dtype).element_size()
    x = [_randn(g, B, N, h, d, dtype=dtype) for h in (H, Hkv, Hkv)]
    plan = mattn.RopePlan(_freq(d // 2 // 8 * 8), q_weight=1 + 0.1 * torch.randn(d, generator=g, device="cuda"), interleaved=inter)
    want = mattn.qk_rope(*x, plan)
    ref, mag = ops.ref_rope(x[0], plan.q_weight, torch.arange(N, device="cuda").expand(1, B, N), plan.inv_freq,
                            [plan.inv_freq.numel()], 1e-6, inter)
    h = torch.finfo(dtype).eps / 2
    assert bool(((want[0].transpose(1, 2).double().cpu() - ref).abs() <= h * ref.abs() + 2.0 ** -19 * mag).all())

    def outs(off):
        made = []
        for w in want:
            buf = torch.zeros(w.numel() + 64, dtype=dtype, device="cuda")
            made.append(buf[off:off + w.numel()].view(w.shape))
        return made

    for moved in ((0,), (1,), (2,), (0, 1, 2)):
        for off, pad in ((e, 0), (0, e), (e, e)):
            y = [_off(t, off if i in moved else 0, pad if i in moved else 0) for i, t in enumerate(x)]
            for o in (0, e):
                for a, b in zip(mattn.qk_rope(*y, plan, *outs(o)), want):
                    assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_batch_and_token_strides(dtype):
    """Expanded batches and tokens (stride 0), sequences further apart than their tokens, and one token of a longer run."""
    g = _gen(4)
    d, H, Hkv, N = 64, 4, 2, 6
    plan = mattn.RopePlan(_freq(32), k_weight=1 + 0.1 * torch.randn(d, generator=g, device="cuda"))
    one = [_randn(g, 1, N, h, d, dtype=dtype) for h in (H, Hkv, Hkv)]
    token = [t[:, :1] for t in one]
    long = [_randn(g, 3, 4 * N, h, d, dtype=dtype) for h in (H, Hkv, Hkv)]
    for x in ([t.expand(3, N, *t.shape[2:]) for t in one], [t.expand(3, N, *t.shape[2:]) for t in token],
              [t[:, 3:3 + N] for t in long], [t[:, ::4] for t in long], [t[:, 7:8] for t in long], [t[1:2, ::2] for t in long]):
        for a, b in zip(mattn.qk_rope(*x, plan), mattn.qk_rope(*(t.contiguous() for t in x), plan)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ near-equal scores past what shared memory keeps
@pytest.mark.parametrize("n", [6144 + 2, 9000, 32768])
@pytest.mark.parametrize("kind", ["few near the border", "many near the border", "ties", "extremes"])
def test_select_near_border_of_many_blocks(n, kind):
    """More competing blocks than the 6,144 whose scores fit in shared memory."""
    g = _gen(n)
    q = _randn(g, 1, 4, 64, scale=8.0)
    means = _randn(g, 1, 1, n, 64, scale=0.25)
    top_k = n // 3
    if kind == "few near the border":
        # a dozen copies of the border's block that differ by one step in one value
        s = (means[0, 0].double() @ q[0].double().T).amax(1)
        at = int(s.argsort(descending=True)[top_k - 6])
        to = torch.randperm(n, generator=g, device="cuda")[:12]
        means[0, 0, to] = means[0, 0, at].clone()
        c = torch.arange(12, device="cuda") * 5
        means[0, 0, to, c] = (means[0, 0, to, c].float() * (1 + 2.0 ** -7)).to(torch.bfloat16)
    elif kind == "many near the border":
        means = means[:, :, :1].expand(1, 1, n, 64).clone()
        c = torch.randint(0, 64, (n,), generator=g, device="cuda")
        i = torch.arange(n, device="cuda")
        means[0, 0, i, c] = (means[0, 0, i, c].float() * (1 + 2.0 ** -7)).to(torch.bfloat16)
    elif kind == "ties":
        means = means[:, :, torch.randint(0, 7, (n,), generator=g, device="cuda")].contiguous()
    else:
        means[0, 0, 17] *= 1e30
        means[0, 0, 300, 5], means[0, 0, 301, 6], means[0, 0, 302, 7] = float("nan"), math.inf, -math.inf
        means[0, 0, 400:900] = 0
    ops.select_case(q, means, 64, top_k, [n * 64])
    ops.select_case(q, means, 64, 64, [n * 64], first=2, recent=3)


# ------------------------------------------------------------------ weights in two parts
def _cancelling(g, n, d):
    """Keys, values and a query such that the output is almost 0 while the weighted
    values are not: the output's own rounding is small then, and what is left is
    the weights'.  -> q, k, v, the 64-bit output, sum of weights times |values|."""
    q, k, v = _randn(g, d, scale=0.5), _randn(g, n, d), _randn(g, n, d)
    p = torch.softmax(k.double() @ q.double() * d ** -0.5, 0)
    for j in (n - 3, n - 2, n - 1):  # each takes off what is left, to the half step of its own type
        left = (p[:, None] * v.double()).sum(0) - p[j] * v[j].double()
        v[j] = (-left / p[j]).to(torch.bfloat16)
    return q, k, v, p @ v.double(), p @ v.double().abs()


def _runs(q, k, v, n):
    """The same list of n keys by every path that sends weights in two parts, as 8 query heads of one key/value head."""
    d = q.shape[0]
    qs = q.expand(1, 8, d).contiguous()
    cache = [torch.full((1, 1, -(-n // 16) * 16, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for c, x in zip(cache, (k, v)):
        c[0, 0, :n] = x
    lens, none = _i32([n]), k.new_zeros((1, 1, 0, d))
    ids = torch.arange(-(-n // 16), dtype=torch.int32, device="cuda").view(1, 1, -1)
    many = torch.cat((ids, ids.new_full((1, 1, 1100), -1)), -1)
    yield "block lists in a cluster", mattn.decode_blocks(qs, *cache, ids, 16, seq_lens=lens)[0]
    yield "block lists in shares", mattn.decode_blocks(qs, *cache, many, 16, seq_lens=lens)[0]
    yield "own keys", mattn.decode_shared(qs, none[0], none[0], *cache, seq_lens=lens)[0]
    yield "prefix of one row tile", mattn.decode_shared(qs, k[None], v[None], none, none)[0]
    m = n // 2
    own = [torch.cat((c[:, :, m:], c[:, :, :m]), 2) for c in cache]
    yield "prefix and own keys", mattn.decode_shared(qs, k[None, :m].contiguous(), v[None, :m].contiguous(),
                                                     own[0], own[1], seq_lens=_i32([n - m]))[0]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [8, 50, 300])
def test_weights_keep_sixteen_bits(d, n):
    """|do| <= u |o| + (2^-15 + 2 t + 2^-13) A where weights go to the tensor cores
    as two bf16 parts (2^-16 of a weight off at most, and twice that after the division by
    their sum); one part alone is off by up to 2^-8 of a weight, and at 8 keys about
    2^-10 A.  t and 2^-13: see test_gpu_decode_ops.py."""
    q, k, v, ref, a = _cancelling(_gen(d + n), n, d)
    t = float((k.double().abs() @ q.double().abs()).max()) * d ** -0.5 * d * 2.0 ** -24
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -15 + 2 * t + 2.0 ** -13) * a
    if n <= 50:  # (one part alone, by the formula: over the bound in many of the dims)
        w = torch.exp(k.double() @ q.double() * d ** -0.5)
        one = w.to(torch.bfloat16).double() @ v.double() / w.sum()
        assert float(((one - ref).abs() > tol).double().mean()) > 0.1
    for name, o in _runs(q, k, v, n):
        over = (o.double() - ref).abs() - tol
        assert bool((over <= 0).all()), f"{name}: {float(over.max()):.3e} over its bound"


@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_key_gives_its_value(d):
    """A single visible key: its value row, bit for bit (2^-16 of a value is far below
    its half step); with more than 128 query rows a key/value head, where weights have
    one part, one step off at most."""
    g = _gen(d)
    for seed in range(6):
        q, k, v = _randn(g, d, scale=1 + seed), _randn(g, 1, d), _randn(g, 1, d)
        for name, o in _runs(q, k, v, 1):
            if name != "prefix and own keys":  # (0 and 1 keys: the same as own keys)
                assert torch.equal(o, v[0].expand(1, 8, d)), name
        none = k.new_zeros((40, 1, 0, d))
        o = mattn.decode_shared(_randn(g, 40, 8, d), k[None], v[None], none, none)[0].double()
        assert bool(((o - v[0].double()).abs() <= 2 * 2.0 ** -8 * v[0].double().abs()).all())


# ------------------------------------------------------------------ block lists of a few more groups than a wave holds
@pytest.mark.parametrize("d,block,B", [(64, 32, 39), (128, 16, 40), (256, 16, 39), (128, 16, 80)])
def test_blocks_of_more_groups_than_a_wave(d, block, B):
    """Long lists of 312 to 640 groups, read in equal shares: entries unused, repeated
    and past the end; sequences without a key."""
    Hkv, L = 8, 70 * block
    rng = torch.Generator().manual_seed(d + B)
    ids = torch.randint(-5, 72, (B, Hkv, 64), generator=rng)
    ids[1], ids[2, 3] = -1, 0
    lens = torch.randint(0, L + 9, (B,), generator=rng)
    lens[0], lens[3] = L, 0
    ops.blocks_case(B, 2 * Hkv, Hkv, d, L, block, ids.tolist(), lens.tolist(), sink=bool(B % 2), seed=d)


@pytest.mark.parametrize("d", [64, 256])
def test_select_products_below_the_least_normal_number(d):
    """Scores that are sums of many products below 2^-126 against one product of
    nearly their sum: the larger sum is chosen, however small."""
    n = 40
    q = torch.full((1, 2, d), 2.0 ** -70, dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 2.0 ** -60
    means = torch.zeros((1, 1, n, d), dtype=torch.bfloat16, device="cuda")
    means[0, 0, 7, 1:] = 1.9921875 * 2.0 ** -57  # d - 1 products of almost 2^-126
    for share in (0.96875, 1.0078125):  # of their sum, as one product
        means[0, 0, 20] = 0
        means[0, 0, 20, 0] = share * float((means[0, 0, 7].double() @ q[0, 0].double())) / 2.0 ** -60
        for top_k in (1, 2, 5):
            ops.select_case(q, means, 16, top_k, [n * 16], first=0, recent=0)
