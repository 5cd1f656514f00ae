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
