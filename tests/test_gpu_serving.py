"""GPU tests of the operators around a paged cache as a serving loop uses them: a run of
them together, captured and replayed, on streams and threads of their own, and past
32-bit offsets.  Tolerances as in test_gpu_paged.py and test_gpu_packed.py, whose 64-bit
forms are used."""

import math
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")
import test_gpu_packed as packed  # noqa: E402  (the 64-bit forms)
import test_gpu_paged as paged  # noqa: E402

CODES = torch.float8_e4m3fn


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


# ------------------------------------------------------------------ a request's life
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_prefill_chunk_and_decode(d, e4m3):
    """Two chunks of packed prompts and three single tokens: norms and rotation, rows into the
    cache, attention over the chunk with the cached rows in front of it, attention over the
    pages.  Each attention is compared on the rows that the cache holds."""
    B, H, Hkv, page, slots = 3, 8, 2, 16, 12
    g = _gen(5)
    c = paged.Cache(B, Hkv, d, page, slots, e4m3, seed=7)
    plan = mattn.RopePlan((1e4 ** (-torch.arange(d // 2, device="cuda") / (d // 2))).float(),
                          q_weight=torch.ones(d, device="cuda"), k_weight=torch.ones(d, device="cuda"))
    done = [0] * B
    for chunk in ([40, 1, 77], [50, 63, 3]):
        T = sum(chunk)
        cu = paged._lens_to_cu(chunk)
        x = _randn(g, 1, T, H + 2 * Hkv, d)
        pos = torch.cat([torch.arange(a, a + n) for a, n in zip(done, chunk)]).to(torch.int32).cuda()[None, None]
        q, k, v = mattn.qk_rope(x[:, :, :H], x[:, :, H : H + Hkv], x[:, :, H + Hkv :], plan, positions=pos)
        q, k, v = (y[0].transpose(0, 1) for y in (q, k, v))  # [T, heads, d], heads apart
        mattn.cache_write(k, v, c.k, c.v, c.table, cu, _i32(done), **c.kw())
        done = [a + n for a, n in zip(done, chunk)]
        cu_k = paged._lens_to_cu(done)
        kk, vv = mattn.cache_read(c.k, c.v, c.table, cu_k, sum(done), **c.kw())
        if not e4m3 and done == chunk:
            assert torch.equal(kk, k) and torch.equal(vv, v)
        o, lse = mattn.attention_packed(q, kk, vv, cu, cu_k)
        packed.check(o, lse, q, kk, vv, cu.tolist(), cu_k.tolist(), True, None, None, d ** -0.5)
    for _ in range(3):
        x = _randn(g, B, 1, H + 2 * Hkv, d)
        pos = _i32(done)[None, :, None]
        q, k, v = mattn.qk_rope(x[:, :, :H], x[:, :, H : H + Hkv], x[:, :, H + Hkv :], plan, positions=pos)
        mattn.cache_write(k[:, :, 0], v[:, :, 0], c.k, c.v, c.table, starts=_i32(done), **c.kw())
        done = [a + 1 for a in done]
        o, lse = mattn.decode_paged(q[:, :, 0], c.k, c.v, c.table, _i32(done), **c.kw())
        torch.cuda.synchronize()
        c.freeze()
        paged.check_decode(o, lse, q[:, :, 0], c, [list(range(n)) for n in done], None, d ** -0.5)


# ------------------------------------------------------------------ captured and replayed
class Calls:
    """One call of each operator on tensors that stay, of `seed`'s values."""

    def __init__(self, seed, e4m3=True, B=3, d=128):
        g = _gen(seed)
        self.B = B
        self.c = paged.Cache(B, 2, d, 32, 5, e4m3, seed=seed)
        n = ([50, 0, 31] * B)[:B]
        self.cu, self.starts, self.lens = paged._lens_to_cu(n), _i32([3] * B), _i32(([160, 3, 77] * B)[:B])
        T = sum(n)
        self.q, self.k, self.v = _randn(g, T, 8, d), _randn(g, T, 2, d), _randn(g, T, 2, d)
        self.qd = _randn(g, B, 8, d)
        self.ko, self.vo = torch.zeros_like(self.k), torch.zeros_like(self.v)
        self.od, self.ld = torch.zeros_like(self.qd), torch.zeros((B, 8), device="cuda")
        self.op, self.lp = torch.zeros_like(self.q), torch.zeros((8, T), device="cuda")
        self.wd = mattn.decode_paged_workspace(B, 8, 2, 5, 32, d, e4m3)
        self.wp = mattn.attention_packed_workspace(T, B, 8)

    def inputs(self):
        return [self.q, self.k, self.v, self.qd]

    def outputs(self):
        return [paged.Cache._bytes(self.c.k), paged.Cache._bytes(self.c.v), self.ko, self.vo, self.od, self.ld, self.op, self.lp]

    def run(self, stream=None):
        c, kw = self.c, dict(self.c.kw(), stream=stream)
        mattn.cache_write(self.k, self.v, c.k, c.v, c.table, self.cu, self.starts, **kw)
        mattn.cache_read(c.k, c.v, c.table, self.cu, None, self.starts, k_out=self.ko, v_out=self.vo, **kw)
        mattn.decode_paged(self.qd, c.k, c.v, c.table, self.lens, out=self.od, lse=self.ld, workspace=self.wd, **kw)
        mattn.attention_packed(self.q, self.ko, self.vo, self.cu, out=self.op, lse=self.lp, workspace=self.wp, stream=stream)


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("B", [3, 90])
@pytest.mark.parametrize("e4m3", [False, True])
def test_captured_chain_replays_on_new_values(e4m3, B, d):
    """A graph of the four, replayed twice on other inputs, between eager calls of other tensors."""
    x, other = Calls(1, e4m3, B, d), Calls(2, e4m3, B, d)
    x.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for seed in (3, 4):
        want = Calls(seed, e4m3, B, d)
        for a, b in zip((paged.Cache._bytes(x.c.k), paged.Cache._bytes(x.c.v), x.c.table), (paged.Cache._bytes(want.c.k), paged.Cache._bytes(want.c.v), want.c.table)):
            a.copy_(b)
        if e4m3:
            x.c.ke.copy_(want.c.ke)
            x.c.ve.copy_(want.c.ve)
        for a, b in zip(x.inputs(), want.inputs()):
            a.copy_(b)
        other.run()
        graph.replay()
        other.run()
        want.run()
        torch.cuda.synchronize()
        for a, b in zip(x.outputs(), want.outputs()):
            assert torch.equal(a, b)


def test_two_graphs_replayed_side_by_side():
    """Graphs with workspaces of their own, replayed on two streams at once."""
    xs = [Calls(s, B=b, d=d) for s, b, d in ((1, 3, 128), (2, 40, 128), (3, 40, 256))]
    graphs, want = [], []
    for x in xs:
        x.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in x.outputs()])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x.run()
        graphs.append(graph)
        for t in x.outputs()[2:]:
            t.fill_(3)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for x, w in zip(xs, want):
        for a, b in zip(x.outputs(), w):
            assert torch.equal(a, b)


def test_calls_wait_for_their_stream_alone():
    """On another stream, by context and by handle: after the work before it there, its results for the work behind it."""
    for by_handle in (False, True):
        x, want = Calls(1), Calls(1)
        want.run()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        late = [t.clone() for t in x.inputs()]
        for t in x.inputs():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            for a, b in zip(x.inputs(), late):
                a.copy_(b, non_blocking=True)
            if not by_handle:
                x.run()
        if by_handle:
            x.run(stream=s.cuda_stream)
        with torch.cuda.stream(s):
            got = [t.clone() for t in x.outputs()]
        s.synchronize()
        for a, b in zip(got, want.outputs()):
            assert torch.equal(a, b)


def test_calls_from_threads_on_streams_of_their_own():
    xs = [Calls(s, B=b) for s, b in ((1, 3), (2, 90), (3, 5), (4, 33))]
    want = []
    for x in xs:
        x.run()
        torch.cuda.synchronize()
        want.append([t.clone() for t in x.outputs()])
        for t in x.outputs()[2:]:
            t.zero_()
    torch.cuda.synchronize()
    errors = []

    def work(x):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    x.run()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(x,)) for x in xs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for x, w in zip(xs, want):
        for a, b in zip(x.outputs(), w):
            assert torch.equal(a, b)


FIRST_UNDER_CAPTURE = """
import torch
import block_sparse_attention_masked_gb300 as mattn
x = torch.randn(20, 2, 64, device="cuda").to(torch.bfloat16)
pages = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
table, cu = torch.tensor([[2, 1]], dtype=torch.int32, device="cuda"), torch.tensor([0, 20], dtype=torch.int32, device="cuda")
other, out = pages.clone(), torch.zeros_like(x)
calls = {"write": lambda: mattn.cache_write(x, x, pages, other, table, cu),
         "read": lambda: mattn.cache_read(pages, other, table, cu, k_out=out, v_out=out.clone()),
         "decode": lambda: mattn.decode_paged(x[:1], pages, other, table),
         "packed": lambda: mattn.attention_packed(x, x, x, cu)}
call = calls[WHICH]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
try:
    with torch.cuda.graph(graph):
        call()
    assert WHICH in ("write", "read"), "captured an allocation"
    graph.replay()
    torch.cuda.synchronize()
    if WHICH == "write":
        assert torch.equal(pages[2].transpose(0, 1), x[:16])
except mattn.MattnError as e:
    assert WHICH in ("decode", "packed") and e.code == mattn.ERR_UNSUPPORTED, e
print("fine")
"""


@pytest.mark.parametrize("which", ["write", "read", "decode", "packed"])
def test_first_call_of_a_process_under_capture(which):
    env = dict(os.environ, PYTHONPATH=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    r = subprocess.run([sys.executable, "-c", f"WHICH = {which!r}\n" + FIRST_UNDER_CAPTURE], env=env, timeout=240,
                       capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("fine"), r.stdout + r.stderr


# ------------------------------------------------------------------ past 32 bits
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_past_four_gigabytes(e4m3):
    """Pages whose rows lie past 2^32 bytes of each pool: written, read back and attended."""
    B, H, Hkv, d, page = 2, 8, 2, 128, 64
    n = (1 << 32) // (Hkv * page * d * (1 if e4m3 else 2)) + 40
    dtype = CODES if e4m3 else torch.bfloat16
    k, v = (torch.zeros((n, Hkv, page, d), dtype=torch.uint8 if e4m3 else dtype, device="cuda").view(dtype) for _ in range(2))
    exps = [torch.zeros((n, Hkv, page), dtype=torch.uint8, device="cuda") if e4m3 else None for _ in range(2)]
    kw = dict(k_exponents=exps[0], v_exponents=exps[1])
    table = _i32([[n - 1, n - 30], [n - 2, n - 3]])
    lens = [100, 77]
    g = _gen(3)
    kr, vr, q = _randn(g, 177, Hkv, d), _randn(g, 177, Hkv, d), _randn(g, B, H, d)
    cu = paged._lens_to_cu(lens)
    mattn.cache_write(kr, vr, k, v, table, cu, **kw)
    ko, vo = mattn.cache_read(k, v, table, cu, 177, **kw)
    for a, b in ((ko, kr), (vo, vr)):
        if e4m3:
            tol = torch.maximum(b.abs().double() / 16, b.abs().amax(dim=-1, keepdim=True).double() * 2.0 ** -17)
            assert bool(((a.double() - b.double()).abs() <= tol).all())
        else:
            assert torch.equal(a, b)
    o, lse = mattn.decode_paged(q, k, v, table, _i32(lens), **kw)
    small = torch.cat([k[n - 40 :].view(torch.uint8 if e4m3 else dtype), ]), torch.cat([v[n - 40 :].view(torch.uint8 if e4m3 else dtype)])
    same = mattn.decode_paged(q, small[0].view(dtype), small[1].view(dtype), table - (n - 40), _i32(lens),
                              **{a: (b if b is None else b[n - 40 :].contiguous()) for a, b in kw.items()})
    assert torch.equal(o, same[0]) and torch.equal(lse, same[1])
    cu_list = cu.tolist()
    for b in range(B):
        i = slice(cu_list[b], cu_list[b + 1])
        for h in range(H):
            r, l, tol, tl = paged.ref_decode(q[b, h].double().cpu(), ko[i, h // 4].double().cpu(), vo[i, h // 4].double().cpu(), None,
                                             d ** -0.5, e4m3)
            assert bool(((o[b, h].double().cpu() - r).abs() <= tol).all()) and abs(float(lse[b, h]) - l) <= tl


def test_packed_rows_past_four_gigabytes():
    """2.4 G elements of q and o: sequences at the far end as the same ones alone."""
    T, H, Hkv, d = 600_000, 32, 1, 128
    q, k, v = (torch.zeros((T, h, d), dtype=torch.bfloat16, device="cuda") for h in (H, Hkv, Hkv))
    n = [300] * 2000
    cu = paged._lens_to_cu(n)
    g = _gen(1)
    at = cu.tolist()[-4]
    for x in (q, k, v):
        x[at:] = _randn(g, *x[at:].shape)
    o, lse = mattn.attention_packed(q, k, v, cu)
    same = mattn.attention_packed(q[at:].clone(), k[at:].clone(), v[at:].clone(), _i32([0, 300, 600, 900]))
    assert torch.equal(o[at:], same[0]) and torch.equal(lse[:, at:], same[1])
    c = [0, 300, 600, 900]
    packed.check(o[at:, :4], lse[:4, at:], q[at:, :4], k[at:], v[at:], c, c, True, None, None, d ** -0.5)
    assert not o[:at].any() and math.isfinite(float(lse[:, :at].sum()))


# ------------------------------------------------------------------ the debug library
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B", [3, 90])
@pytest.mark.parametrize("d", [128, 256])
def test_debug_library_gives_the_same(e4m3, B, d):
    """Bounds checks before every copy: none fails, and the results are the product library's bit for bit."""
    want, got = Calls(1, e4m3, B, d), Calls(1, e4m3, B, d)
    want.run()
    torch.cuda.synchronize()
    mattn.use_debug_library(True)
    try:
        if not os.path.exists(mattn.DEBUG_LIB_PATH):
            pytest.skip("the debug library is not built")
        got.run()
        torch.cuda.synchronize()
        rc, word = mattn.device_status()
        assert mattn.lib().mattn_debug_checks() == 1 and rc == 0, hex(word)
    finally:
        mattn.use_debug_library(False)
    for a, b in zip(got.outputs(), want.outputs()):
        assert torch.equal(a, b)
