"""GPU tests of the decode step's operators against plain implementations in
64 bits written here: head norms with the position rotation, attention over
a shared prefix, block means, block selection, attention over selected blocks,
and a run of them together.

Tolerances, derived before the first run.  u = 2^-8 is bf16's half step relative
to the value, e = 2^-24 fp32's.
  attention  o = sum p v / sum p: weights rounded to bf16 (u each) and the
             output rounded once (u): |do| <= u |o| + (u + 2 t + 2^-13) A with
             A = sum p |v| / sum p, t the largest error of a score (below),
             which moves a weight and the sum by as much, and 2^-13 for the
             exponentials and the sums over keys.
  lse        a score is a sum of d exact products: t = d e max_j sum_c |q_c k_jc|
             scale; the exponentials' and logarithm's approximations add
             2^-19 (1 + |lse|).
  rotation   |dy| <= h |y| + 2^-19 (|a| + |b|), h the type's half step: the
             norm's sum of up to 256 squares is off by at most 20 e, halved by
             the root, the sine and cosine by 4 e, three products by 3 e; 2^-19
             is 32 e.
  means      u |m| + n e mean|k| for n keys.
"""

import math
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

mattn = pytest.importorskip("block_sparse_attention_masked_gb300")

U, E = 2.0 ** -8, 2.0 ** -24
NAN = float("nan")


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


# ------------------------------------------------------------------ attention
def ref_rows(q, keys, values, sink, scale):
    """One head: q [d], keys, values [n, d] (64 bits), sink float or None ->
    (o, lse, tolerance of o, tolerance of lse)."""
    d = q.shape[0]
    s = keys @ q * scale
    x = s if sink is None else torch.cat((s, s.new_tensor([sink])))
    if x.numel() == 0:
        return torch.zeros_like(q), -math.inf, torch.zeros_like(q), 0.0
    m = x.max()
    p = torch.exp(x - m)
    z = p.sum()
    w = p[:s.numel()] / z
    o, a = w @ values, w @ values.abs()
    lse = float(m + torch.log(z))
    tol_s = float((keys.abs() @ q.abs()).max()) * scale * d * E if s.numel() else 0.0
    return o, lse, U * o.abs() + (U + 2 * tol_s + 2.0 ** -13) * a, tol_s + 2.0 ** -19 * (1 + abs(lse))


def check_attention(o, lse, q, lists, sink, scale, tag=""):
    """lists[b][kv head] = (keys [n, d], values [n, d]) on the CPU in 64 bits."""
    B, H, d = q.shape
    qd, got, gl = q.double().cpu(), o.double().cpu(), lse.double().cpu()
    for b in range(B):
        G = H // len(lists[b])
        for h in range(H):
            keys, values = lists[b][h // G]
            r, l, tol, tl = ref_rows(qd[b, h], keys, values, None if sink is None else float(sink[h]), scale)
            err = (got[b, h] - r).abs()
            assert bool((err <= tol + 1e-30).all()), f"{tag} b{b} h{h}: o off by {(err - tol).max():.3e} over its bound"
            if math.isinf(l):
                assert float(gl[b, h]) == l, f"{tag} b{b} h{h}: lse {float(gl[b, h])}"
            else:
                assert abs(float(gl[b, h]) - l) <= tl, f"{tag} b{b} h{h}: lse off by {abs(float(gl[b, h]) - l):.3e} ({tl:.1e})"


HEADS = [(1, 1), (8, 2), (3, 1), (8, 1), (12, 1), (32, 2)]


def shared_case(B, H, Hkv, d, P, L, lens, sink=False, scale=None, q_scale=1.0, cap=None, seed=0):
    g = _gen(seed)
    cap = P if cap is None else cap
    q = _randn(g, B, H, d, scale=q_scale)
    kp, vp = _randn(g, Hkv, cap, d), _randn(g, Hkv, cap, d)
    k, v = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    kp[:, P:], vp[:, P:] = NAN, NAN  # what lies behind the prefix is nobody's business
    for b, n in enumerate(lens):
        k[b, :, min(max(n, 0), L):], v[b, :, min(max(n, 0), L):] = NAN, NAN
    sk = torch.linspace(-2, 3, H, device="cuda") if sink else None
    o, lse = mattn.decode_shared(q, kp, vp, k, v, seq_lens=_i32(lens), prefix_len=P, sink=sk, scale=scale)
    torch.cuda.synchronize()
    lists = []
    for b, n in enumerate(lens):
        n = min(max(n, 0), L)
        lists.append([(torch.cat((kp[h, :P], k[b, h, :n])).double().cpu(), torch.cat((vp[h, :P], v[b, h, :n])).double().cpu())
                      for h in range(Hkv)])
    check_attention(o, lse, q, lists, sk, scale or d ** -0.5, f"B{B} H{H}/{Hkv} d{d} P{P} L{L}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_shared_heads(d, H, Hkv):
    """Head layouts incl. more than eight query heads per key/value head; own
    lengths 0, 1, full, past the capacity (clamped) and negative (0)."""
    shared_case(5, H, Hkv, d, 300, 77, [0, 1, 77, 1000, -5], sink=True, seed=d + H)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("P", [0, 1, 63, 64, 65, 127, 128, 129, 1000, 20011])
def test_shared_prefix_lengths(d, P):
    """Prefix lengths around the key tile, with rows behind it in the buffer."""
    shared_case(3, 4, 2, d, P, 40, [40, 0, 33], cap=P + 70, seed=P + d)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B,H,Hkv", [(31, 4, 1), (32, 4, 1), (33, 4, 1), (70, 12, 3), (130, 4, 2)])
def test_shared_row_tiles(d, B, H, Hkv):
    """Query rows per key/value head below, at and past 128 and 256."""
    shared_case(B, H, Hkv, d, 500, 9, [b % 10 for b in range(B)], sink=True, seed=B)


@pytest.mark.parametrize("L", [0, 1, 15, 16, 17, 31, 32, 33, 500, 5003])
def test_shared_own_lengths(L):
    shared_case(2, 8, 2, 128, 130, L, [L, L // 2], seed=L)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q_scale", [0.0, 30.0, 1000.0])
def test_shared_extreme_scores(d, q_scale):
    """Uniform weights, and scores far enough apart that a later key tile's
    scores dwarf the earlier ones (the running reference moves)."""
    shared_case(2, 4, 1, d, 700, 70, [70, 35], q_scale=q_scale, seed=3)
    shared_case(2, 4, 1, d, 700, 70, [70, 35], q_scale=q_scale, sink=True, scale=0.25, seed=4)


def test_shared_rising_scores():
    """Key tiles whose scores rise by more than the running reference allows, and
    a first tile far below 0, for more than 128 rows (two query tiles)."""
    for d, B in ((128, 2), (128, 80), (64, 80), (256, 40)):
        g = _gen(d + B)
        q = torch.ones((B, 4, d), device="cuda", dtype=torch.bfloat16)
        ramp = torch.linspace(-40, 40, 1500, device="cuda")[None, :, None].expand(1, 1500, d) / math.sqrt(d) * 2
        kp, vp = ramp.to(torch.bfloat16).contiguous(), _randn(g, 1, 1500, d)
        k = v = torch.zeros((B, 1, 0, d), device="cuda", dtype=torch.bfloat16)
        o, lse = mattn.decode_shared(q, kp, vp, k, v)
        one = (kp[0].double().cpu(), vp[0].double().cpu())
        check_attention(o, lse, q, [[one]] * B, None, d ** -0.5, f"ramp d{d} B{B}")


def test_shared_equals_decode_on_the_joined_cache():
    B, H, Hkv, d, P, L = 3, 8, 2, 128, 600, 100
    g = _gen(1)
    q, kp, vp = _randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, Hkv, P, d)
    k, v, lens = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d), [100, 1, 50]
    o, lse = mattn.decode_shared(q, kp, vp, k, v, seq_lens=_i32(lens))
    from workloads import MaskSpec

    joined = [torch.cat((p[None].expand(B, Hkv, P, d), c), dim=2).contiguous() for p, c in ((kp, k), (vp, v))]
    o2, lse2 = mattn.decode(q, *joined, mattn.prepare(MaskSpec("full", [0] * H), H, P + L),
                            seq_lens=_i32([P + n for n in lens]))
    # two results within their bounds of the same value: |o| and A are below max|v|
    assert float((o.float() - o2.float()).abs().max()) <= 2 * (2 * U + 2.0 ** -13) * float(vp.float().abs().max())
    assert float((lse - lse2).abs().max()) <= 1e-4


def blocks_case(B, H, Hkv, d, L, block, ids, lens, sink=False, seed=0):
    """ids[b][kv head] lists; everything a list does not name is poisoned."""
    g = _gen(seed)
    q, k, v = _randn(g, B, H, d), _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    sk = torch.linspace(-1, 2, H, device="cuda") if sink else None
    lists = []
    for b in range(B):
        n = min(max(lens[b], 0), L)
        row = []
        for h in range(Hkv):
            seen = torch.zeros(L, dtype=torch.bool)
            spans = [(i * block, min(i * block + block, n)) for i in ids[b][h] if i >= 0 and i * block < n]
            for x, y in spans:
                seen[x:y] = True
            bad = ~seen.cuda()
            k[b, h][bad], v[b, h][bad] = NAN, NAN
            empty = torch.zeros((0, d), dtype=torch.float64)
            row.append((torch.cat([empty] + [k[b, h, x:y].double().cpu() for x, y in spans]),
                        torch.cat([empty] + [v[b, h, x:y].double().cpu() for x, y in spans])))
        lists.append(row)
    o, lse = mattn.decode_blocks(q, k, v, _i32(ids), block, seq_lens=_i32(lens), sink=sk)
    torch.cuda.synchronize()
    check_attention(o, lse, q, lists, sk, d ** -0.5, f"B{B} H{H}/{Hkv} d{d} L{L} block{block}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("block", [16, 32, 48, 64, 128])
def test_blocks_sizes(d, block):
    """Lists with unused entries anywhere, blocks past the sequence's end, the
    partly filled newest block, a block listed twice, and nothing at all."""
    L, Hkv = 7 * block + 5, 2
    ids = [[[0, 3, 7, -1, -1], [1, 2, 3, 4, 5]], [[6, -1, 2, 2, 99], [-1, -1, -1, -1, -1]],
           [[0, 1, 2, 3, 4], [0, 7, 7, 1 << 30, -(1 << 31)]]]
    blocks_case(3, 4, Hkv, d, L, block, ids, [L, 6 * block + 1, 1], sink=False, seed=block + d)
    blocks_case(3, 4, Hkv, d, L, block, ids, [0, -3, 1000000], sink=True, seed=block + d + 1)


@pytest.mark.parametrize("H,Hkv", HEADS)
def test_blocks_heads(H, Hkv):
    ids = [[list(range(k, k + 6)) for k in range(Hkv)] for _ in range(2)]
    blocks_case(2, H, Hkv, 128, 600, 64, ids, [600, 390], sink=True, seed=H)


@pytest.mark.parametrize("top_k", [1, 33, 300])
def test_blocks_long_lists(top_k):
    """One split and many; top_k past the number of blocks."""
    n = 200
    ids = [[sorted(np.random.default_rng(top_k + h).permutation(n)[:min(top_k, n)].tolist()) + [-1] * max(0, top_k - n)
            for h in range(2)]]
    blocks_case(1, 8, 2, 128, n * 32, 32, ids, [n * 32 - 7], seed=top_k)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_blocks_more_groups_than_sms(d):
    """More groups than one wave of CTAs, with lists of none, one and every block."""
    B, Hkv = 20, 8
    ids = [[[(b + h + j) % 5 if j < (b + h) % 6 else -1 for j in range(6)] for h in range(Hkv)] for b in range(B)]
    blocks_case(B, 16, Hkv, d, 5 * 32, 32, ids, [160 - 7 * b for b in range(B)], sink=True, seed=d)


@pytest.mark.parametrize("d,top_k", [(64, 1025), (128, 1100), (256, 1025), (256, 200)])
def test_blocks_in_equal_shares(d, top_k):
    """Lists past the clusters' table, and one long list of one group, read in equal shares."""
    rng = np.random.default_rng(d + top_k)
    ids = [[rng.integers(-3, 40, size=top_k).tolist()]]
    blocks_case(1, 4, 1, d, 40 * 16, 16, ids, [40 * 16 - 3], sink=True, seed=top_k)


@pytest.mark.parametrize("B,Hkv,d,L", [(2, 1, 128, 150000), (1, 1, 256, 147001), (1, 2, 64, 300001)])
def test_shared_long_own_lists(B, Hkv, d, L):
    """Own keys alone, long enough for whole CTAs of row workers."""
    shared_case(B, 2 * Hkv, Hkv, d, 0, L, [L - 9 * b for b in range(B)], seed=d)


def test_blocks_everything_equals_decode():
    """All blocks listed: the plain decode step's result."""
    from workloads import MaskSpec

    B, H, Hkv, d, L, block = 2, 8, 2, 256, 1000, 64
    g = _gen(2)
    q, k, v = _randn(g, B, H, d), _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    lens = _i32([1000, 130])
    ids = torch.arange(16, dtype=torch.int32, device="cuda").expand(B, Hkv, 16).contiguous()
    o, lse = mattn.decode_blocks(q, k, v, ids, block, seq_lens=lens)
    o2, lse2 = mattn.decode(q, k, v, mattn.prepare(MaskSpec("full", [0] * H), H, L), seq_lens=lens)
    assert float((o.float() - o2.float()).abs().max()) <= 2 * (2 * U + 2.0 ** -13) * float(v.float().abs().max())
    assert float((lse - lse2).abs().max()) <= 1e-4


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("B", [2, 40])
def test_infinite_values(d, B):
    """An infinite value of an attended key makes its dim infinite, and no other dim or sequence."""
    g = _gen(d + B)
    H, Hkv, P, L = 8, 2, 200, 64
    q, kp, vp = _randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, Hkv, P, d)
    k, v = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    vp[0, 131, 7], v[1, 1, 20, 9], v[0, 0, 63, 5] = math.inf, -math.inf, math.inf
    lens = _i32([63] + [L] * (B - 1))  # (sequence 0's one is past its end)
    want = torch.zeros((B, H, d), device="cuda")
    want[1, 4:, 9] = -math.inf
    ids = torch.arange(4, dtype=torch.int32, device="cuda").expand(B, Hkv, 4).contiguous()
    many = torch.cat([ids, ids.new_full((B, Hkv, 1100), -1)], dim=-1)
    outs = [mattn.decode_blocks(q, k, v, x, 16, seq_lens=lens)[0] for x in (ids, many)]
    for o in outs:
        assert torch.equal(torch.where(o.isfinite(), 0.0, o.float()), want)
    o = mattn.decode_shared(q, kp, vp, k, v, seq_lens=lens)[0]
    want[:, :4, 7] = math.inf
    assert torch.equal(torch.where(o.isfinite(), 0.0, o.float()), want)


@pytest.mark.parametrize("B,H,Hkv,d", [(3000, 2, 1, 64), (5001, 4, 4, 128), (700, 16, 16, 256), (65535, 1, 1, 64)])
def test_large_batches(B, H, Hkv, d):
    """Thousands of sequences of 0 to 40 own keys: shared prefix and block lists."""
    g = _gen(B)
    P, L, G, scale = 70, 40, H // Hkv, d ** -0.5
    q, kp, vp = _randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, Hkv, P, d)
    k, v = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    lens = torch.randint(0, L + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    ids = torch.tensor([2, 0, -1], dtype=torch.int32, device="cuda").expand(B, Hkv, 3).contiguous()
    o, lse = mattn.decode_shared(q, kp, vp, k, v, seq_lens=lens)
    o2, lse2 = mattn.decode_blocks(q, k, v, ids, 16, seq_lens=lens)
    pos = torch.arange(L, device="cuda")
    live = pos < lens[:, None]
    listed = live & ((pos < 16) | (pos >= 32))
    for b0 in range(0, B, 2000):
        sl = slice(b0, b0 + 2000)
        n = q[sl].shape[0]
        qd = q[sl].double().view(n, Hkv, G, d)
        own = (qd @ k[sl].double().transpose(-1, -2)) * scale
        pre = torch.einsum("bhgd,hpd->bhgp", qd, kp.double()) * scale
        vo, vpd = v[sl].double(), vp.double()
        # the scores' error: d e max sum |q k| scale, with |q| |k| as a bound of the sum
        tol = float(qd.norm(dim=-1).max() * torch.maximum(k.float().norm(dim=-1).max(), kp.float().norm(dim=-1).max())) * scale * d * E
        for got, gl, mask, prefix in ((o, lse, live, True), (o2, lse2, listed, False)):
            x = own.masked_fill(~mask[sl][:, None, None, :], -math.inf)
            if prefix:
                x = torch.cat((pre, x), dim=-1)
            m = x.amax(-1, keepdim=True).clamp_min(-1e300)
            w = torch.exp(x - m)
            z = w.sum(-1, keepdim=True)
            p = torch.where(z > 0, w / z, 0.0)
            wo = p[..., P:] if prefix else p
            r, a = wo @ vo, wo @ vo.abs()
            if prefix:
                r, a = (y + torch.einsum("bhgp,hpd->bhgd", p[..., :P], u) for y, u in ((r, vpd), (a, vpd.abs())))
            err = (got[sl].double().view_as(r) - r).abs() - (U * r.abs() + (U + 2 * tol + 2.0 ** -13) * a)
            assert float(err.max()) <= 1e-30
            l = (m + torch.log(z)).squeeze(-1)
            gld = gl[sl].double().view_as(l)
            none = z.squeeze(-1) == 0
            assert bool((gld[none] == -math.inf).all())
            assert bool(((gld - l).abs()[~none] <= tol + 2.0 ** -19 * (1 + l.abs()[~none])).all())


def test_offsets_past_32_bits():
    """Caches of more than 2^32 bytes: the last sequence's rows and its means."""
    B, Hkv, L, d, block = 9, 8, 131072, 256, 64
    g = _gen(6)
    k = torch.zeros((B, Hkv, L, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    k[-1, -1, -block:], v[-1, -1, -block:] = _randn(g, block, d), _randn(g, block, d)
    q = _randn(g, B, Hkv, d)
    ids = torch.full((B, Hkv, 1), L // block - 1, dtype=torch.int32, device="cuda")
    o, lse = mattn.decode_blocks(q, k, v, ids, block)
    zero = torch.zeros((block, d), dtype=torch.float64)
    lists = [[(zero, zero)] * Hkv for _ in range(B)]
    lists[-1][-1] = (k[-1, -1, -block:].double().cpu(), v[-1, -1, -block:].double().cpu())
    check_attention(o, lse, q, lists, None, d ** -0.5, "long cache")
    means = mattn.block_means(k, block)
    assert torch.equal(means[-1, -1, -1], k[-1, -1, -block:].float().mean(0).to(torch.bfloat16)) or float(
        (means[-1, -1, -1].float() - k[-1, -1, -block:].float().mean(0)).abs().max()) <= U
    assert float(means[:, :, :-1].float().abs().max()) == 0.0
    plan = mattn.RopePlan(torch.ones(8, device="cuda"), interleaved=True)
    x = _randn(g, B, 1, Hkv, d)
    starts = _i32([L - 1] * B)
    mattn.qk_rope(x, x, x, plan, k_out=k, v_out=v, starts=starts)
    assert torch.equal(v[-1, -1, -1], x[-1, 0, -1])


# ------------------------------------------------------------------ means
def ref_means(k, block, lens, first, max_new, old):
    B, Hkv, L, d = k.shape
    out, tol = old.double().cpu(), torch.zeros(old.shape, dtype=torch.float64)
    kd = k.double().cpu()
    for b in range(B):
        n = min(max(lens[b], 0), L)
        f = max(first[b], 0)
        end = min(n, f + max_new)
        if f >= end:
            continue
        for blk in range(f // block, (end - 1) // block + 1):
            rows = kd[b, :, blk * block:min(n, (blk + 1) * block)]
            out[b, :, blk] = rows.mean(dim=1)
            tol[b, :, blk] = U * out[b, :, blk].abs() + rows.shape[1] * E * rows.abs().mean(dim=1)
    return out, tol


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("block", [16, 48, 64, 512])
@pytest.mark.parametrize("L,lens,first,max_new", [
    (700, [700, 1, 0, 333], None, None),
    (700, [700, 1, 0, 333], [699, 0, 0, 300], 1),
    (700, [700, 65, 64, 900], [600, 64, 63, -7], 100),
    (700, [16, 17, 500, 700], [16, 15, 480, 690], 20),
    (1, [1, 1, 0, 5], [0, 0, 0, 0], 3),
    (129, [129, 128, 127, 1], [1000, 127, 126, 0], 1 << 30),
])
def test_block_means(d, block, L, lens, first, max_new):
    """Whole caches and updates; what holds no new key stays, what is not
    cached is not read (it is NaN)."""
    Hkv = 2
    g = _gen(d + block + L)
    k = _randn(g, 4, Hkv, L, d)
    for b, n in enumerate(lens):
        k[b, :, min(max(n, 0), L):] = NAN
    old = _randn(g, 4, Hkv, -(-L // block), d)
    got = mattn.block_means(k, block, seq_lens=_i32(lens), first=None if first is None else _i32(first),
                            max_new=max_new, out=old.clone())
    ref, tol = ref_means(k, block, lens, first or [0] * 4, max_new or L, old)
    assert bool(((got.double().cpu() - ref).abs() <= tol).all())


# ------------------------------------------------------------------ selection
def ref_select(q, means, block, top_k, lens, first, recent):
    B, H, d = q.shape
    Hkv, n_all = means.shape[1], means.shape[2]
    G = H // Hkv
    out = torch.full((B, Hkv, top_k), -1, dtype=torch.int32)
    qd, md = q.double().cpu(), means.double().cpu()
    for b in range(B):
        n = min(n_all, -(-max(lens[b], 0) // block))
        for h in range(Hkv):
            x = torch.nan_to_num(md[b, h, :n] @ qd[b, h * G:(h + 1) * G].T, nan=-math.inf, posinf=math.inf, neginf=-math.inf)
            bad = torch.isnan(md[b, h, :n] @ qd[b, h * G:(h + 1) * G].T).any(dim=1)
            x = x.max(dim=1).values if n else x.new_zeros(0)
            x = torch.where(bad, torch.full_like(x, -math.inf), x).tolist()
            order = sorted(range(n), key=lambda i: (not (i < first or i >= n - recent), -x[i], i))
            take = sorted(order[:top_k])
            out[b, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
    return out


def select_case(q, means, block, top_k, lens, first=1, recent=1):
    got = mattn.decode_select(q, means, block, top_k, seq_lens=_i32(lens), keep_first=first, keep_recent=recent)
    ref = ref_select(q, means, block, top_k, lens, first, recent)
    assert torch.equal(got.cpu(), ref)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("H,Hkv", HEADS)
def test_select_heads(d, H, Hkv):
    g = _gen(d + H)
    q, means = _randn(g, 3, H, d), _randn(g, 3, Hkv, 130, d, scale=0.25)
    select_case(q, means, 64, 16, [130 * 64, 64 * 64 - 63, 5])


@pytest.mark.parametrize("n,top_k,first,recent", [
    (1, 1, 0, 0), (1, 3, 1, 1), (31, 32, 1, 1), (32, 31, 0, 0), (33, 2, 1, 1), (500, 499, 5, 7), (2048, 64, 1, 1),
    (2048, 1, 0, 0), (5000, 300, 100, 200), (32768, 700, 1, 3),
])
def test_select_sizes(n, top_k, first, recent):
    g = _gen(n + top_k)
    q, means = _randn(g, 2, 4, 128), _randn(g, 2, 1, n, 128, scale=0.25)
    select_case(q, means, 16, top_k, [n * 16, max(1, n * 8 - 3)], first, recent)


def test_select_empty_and_clamped():
    g = _gen(9)
    q, means = _randn(g, 3, 2, 64), _randn(g, 3, 2, 40, 64)
    select_case(q, means, 32, 8, [0, -9, 10 ** 9])
    got = mattn.decode_select(q, means, 32, 8)  # without lengths: every block
    assert torch.equal(got.cpu(), ref_select(q, means, 32, 8, [40 * 32] * 3, 1, 1))


@pytest.mark.parametrize("n", [100, 300, 3000])
def test_select_ties(n):
    """Equal scores: all zero, a few distinct values, repeated rows (few and
    many blocks next to the border), negative zero against zero."""
    g = _gen(n)
    q = _randn(g, 2, 4, 128)
    zero = torch.zeros((2, 2, n, 128), dtype=torch.bfloat16, device="cuda")
    select_case(q, zero, 64, 20, [n * 64] * 2)
    rows = _randn(g, 2, 2, 7, 128)
    pick = torch.randint(0, 7, (n,), generator=g, device="cuda")
    select_case(q, rows[:, :, pick].contiguous(), 64, 33, [n * 64, n * 32])
    zero[:, :, ::2] = -0.0
    select_case(q, zero, 64, 20, [n * 64] * 2, first=0, recent=0)


@pytest.mark.parametrize("n", [200, 1500])
def test_select_near_border(n):
    """Rows that differ from one another in one value by one bf16 step, so that
    scores differ by less than a 32-bit sum's error: exact arithmetic decides."""
    g = _gen(n + 1)
    q = _randn(g, 1, 4, 128, scale=8.0)
    row = _randn(g, 1, 1, 1, 128, scale=16.0).expand(1, 1, n, 128).clone()
    i = torch.arange(n, device="cuda")
    c = torch.randint(0, 128, (n,), generator=g, device="cuda")
    row[0, 0, i, c] = (row[0, 0, i, c].float() * (1 + 2.0 ** -7)).to(torch.bfloat16)
    tiny = torch.randint(0, 3, (n,), generator=g, device="cuda").float() * 1e-6
    row[0, 0, i, (c + 1) % 128] = (row[0, 0, i, (c + 1) % 128].float() * (1 + tiny)).to(torch.bfloat16)
    select_case(q, row, 64, n // 3, [n * 64])
    small = (torch.randint(0, 5, (1, 1, n, 128), generator=g, device="cuda").float() * 2.0 ** -20)
    big = torch.zeros_like(small)
    big[..., 0], big[..., 1] = 256.0, -256.0
    q2 = torch.ones((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    select_case(q2, (small + big).to(torch.bfloat16), 64, n // 4, [n * 64])


def test_select_outliers_and_extremes():
    """Rows with huge norms, infinities and NaN next to ordinary ones, and
    values whose squares underflow."""
    g = _gen(77)
    n = 600
    q = _randn(g, 1, 4, 128)
    means = _randn(g, 1, 1, n, 128, scale=0.25)
    means[0, 0, 17] *= 1e4
    means[0, 0, 300] *= 1e30
    means[0, 0, 301, 5] = NAN
    means[0, 0, 302, 6] = math.inf
    means[0, 0, 303, 6] = -math.inf
    means[0, 0, 304] = 3e38
    select_case(q, means, 64, 50, [n * 64])
    select_case(q, means, 64, 595, [n * 64])
    select_case(q, _randn(g, 1, 1, n, 128, scale=1e-25), 64, 50, [n * 64])
    select_case(_randn(g, 1, 4, 128, scale=1e-30), _randn(g, 1, 1, n, 128, scale=1e-8), 64, 50, [n * 64])
    q[0, 1, 3] = NAN  # one head's scores all NaN: every block counts as -inf
    select_case(q, means, 64, 50, [n * 64])


# ------------------------------------------------------------------ rope
def ref_rope(x, w, pos, inv_freq, sections, eps, inter):
    """x [B, N, heads, d], pos [axes, B, N] -> (y, |a| + |b| per value) in 64 bits."""
    x = x.double().cpu()
    d = x.shape[-1]
    if w is not None:
        x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w.double().cpu()
    R = sum(sections)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    y, mag = x.clone(), x.abs()
    f = inv_freq.double().cpu()
    for p in range(R):
        i, j = (2 * p, 2 * p + 1) if inter else (p, p + R)
        t = (pos[axis[p]].double().cpu() * f[p])[..., None]
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()
        mag[..., i] = mag[..., j] = a.abs() + b.abs()
    return y, mag


def rope_case(B, N, H, Hkv, d, sections, norm, inter, dtype, far=0, L=None, lens=None, starts=None, positions=True,
              with_v=True, seed=0):
    g = _gen(seed)
    R = sum(sections)
    L = N if L is None else L
    qkv = _randn(g, B, N, (H + 2 * Hkv) * d, dtype=dtype)
    q, k, v = (t.unflatten(-1, (-1, d)) for t in qkv.split([H * d, Hkv * d, Hkv * d], dim=-1))
    f = (10000.0 ** (-torch.arange(max(R, 1), device="cuda", dtype=torch.float64)[:R] / max(R, 1))).float()
    wq, wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)) if norm else (None, None)
    st = [0] * B if starts is None else starts
    if positions:
        pos = torch.randint(-far, far + 1, (len(sections), B, N), generator=g, device="cuda", dtype=torch.int32)
    else:
        pos = (torch.tensor(st)[None, :, None] + torch.arange(N)[None, None]).expand(len(sections), B, N)
    plan = mattn.RopePlan(f, sections, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter)
    outs = [torch.full((B, H, N, d), 7.0, dtype=dtype, device="cuda")]
    outs += [torch.full((B, Hkv, L, d), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
    mattn.qk_rope(q, k, v if with_v else None, plan, outs[0], outs[1], outs[2] if with_v else None,
                  positions=pos if positions else None, starts=None if starts is None else _i32(starts),
                  lens=None if lens is None else _i32(lens))
    torch.cuda.synchronize()
    h = torch.finfo(dtype).eps / 2
    rq, mq = ref_rope(q, wq, pos, f, sections, 1e-5, inter)
    rk, mk = ref_rope(k, wk, pos, f, sections, 1e-5, inter)
    n_of = [N] * B if lens is None else [min(max(n, 0), N) for n in lens]
    for b in range(B):
        n = n_of[b]
        got = outs[0][b, :, :n].transpose(0, 1).double().cpu()
        assert bool(((got - rq[b, :n]).abs() <= h * rq[b, :n].abs() + 2.0 ** -19 * mq[b, :n]).all()), "q"
        assert bool((outs[0][b, :, n:] == 7).all()), "padding of q written"
        written = torch.zeros(L, dtype=torch.bool)
        for i in range(n):
            r = st[b] + i
            if not 0 <= r < L:
                continue
            written[r] = True
            got = outs[1][b, :, r].double().cpu()
            assert bool(((got - rk[b, i]).abs() <= h * rk[b, i].abs() + 2.0 ** -19 * mk[b, i]).all()), f"k row {r}"
            assert torch.equal(outs[2][b, :, r], v[b, i]) or not with_v, f"v row {r}"
        for t in outs[1:]:
            assert bool((t[b][:, ~written.cuda()] == 7).all()), "a row nobody asked for was written"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d", [32, 64, 80, 96, 128, 256])
def test_rope_head_dims(d, inter, dtype):
    """Every head dim, type and pairing: full rotation on two axes with norms,
    and a partial one on three without."""
    rope_case(2, 5, 6, 3, d, [d // 2 - d // 4, d // 4], True, inter, dtype, far=2000, seed=d)
    r = 8 * max(1, d // 32)
    rope_case(1, 3, 3, 1, d, [1, r - 3, 2], False, inter, dtype, far=100, seed=d + 1)


@pytest.mark.parametrize("far", [1, 1 << 20, (1 << 31) - 1])
def test_rope_far_positions(far):
    """Angles of far (and negative) positions keep their precision."""
    rope_case(2, 9, 2, 1, 128, [64], True, False, torch.float32, far=far, seed=far % 1000)


@pytest.mark.parametrize("B,N,H,Hkv", [(1, 1, 1, 1), (64, 1, 32, 8), (3, 2, 12, 1), (1, 700, 4, 4), (2, 33, 33, 11)])
def test_rope_append(B, N, H, Hkv):
    """Rows of a cache: starts before, inside and past it, padded batches."""
    rng = np.random.default_rng(B * 100 + N)
    L = N + 9
    starts = rng.integers(0, 10, B).tolist()
    starts[0] = -1 if B > 1 else 3
    starts[-1] = 8 + N if B > 2 else starts[-1]
    lens = rng.integers(0, N + 2, B).tolist()
    rope_case(B, N, H, Hkv, 128, [16, 24, 24], True, False, torch.bfloat16, far=5000, L=L, lens=lens, starts=starts,
              seed=B + N)
    rope_case(B, N, H, Hkv, 64, [32], False, True, torch.bfloat16, L=L, starts=starts, positions=False, with_v=False,
              seed=B + N + 1)


def test_rope_norm_only_and_zero_rows():
    rope_case(2, 4, 4, 2, 80, [0], True, False, torch.bfloat16)
    plan = mattn.RopePlan(torch.ones(32, device="cuda"), q_weight=torch.ones(64, device="cuda"))
    x = torch.zeros((1, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, k, v = mattn.qk_rope(x, x, None, plan)
    assert v is None and float(q.abs().max()) == 0.0 and float(k.abs().max()) == 0.0


# ------------------------------------------------------------------ together, streams, graphs
def _step_inputs(seed, B=3, H=8, Hkv=2, d=128, L=3000, n0=(2950, 64, 1500)):
    g = _gen(seed)
    s = {"plan": mattn.RopePlan((1e6 ** (-torch.arange(64, device="cuda") / 64.0)).float(), [16, 24, 24],
                                q_weight=1 + 0.1 * torch.randn(d, generator=g, device="cuda"),
                                k_weight=1 + 0.1 * torch.randn(d, generator=g, device="cuda"))}
    s["kc"], s["vc"] = _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)
    s["starts"] = _i32(list(n0))
    s["lens"] = s["starts"] + 1
    s["qkv"] = _randn(g, B, 1, (H + 2 * Hkv) * d)
    s["pos"] = s["starts"][None, :, None].expand(3, B, 1).contiguous()
    s["q"] = torch.empty((B, H, 1, d), dtype=torch.bfloat16, device="cuda")
    s["means"] = mattn.block_means(s["kc"], 64, seq_lens=s["starts"])
    s["ids"] = torch.empty((B, Hkv, 12), dtype=torch.int32, device="cuda")
    s["o"] = torch.empty((B, H, d), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty((B, H), dtype=torch.float32, device="cuda")
    s["ws1"] = mattn.decode_select_workspace(B, H, Hkv, 47, d)
    s["ws2"] = mattn.decode_blocks_workspace(B, H, Hkv, 12, 64, d)
    return s


def _step(s):
    """One decode step: projection output -> cache -> means -> blocks -> attention."""
    B, H, Hkv, d = s["o"].shape[0], s["o"].shape[1], s["kc"].shape[1], s["o"].shape[2]
    q, k, v = (t.unflatten(-1, (-1, d)) for t in s["qkv"].split([H * d, Hkv * d, Hkv * d], dim=-1))
    mattn.qk_rope(q, k, v, s["plan"], s["q"], s["kc"], s["vc"], positions=s["pos"], starts=s["starts"])
    mattn.block_means(s["kc"], 64, seq_lens=s["lens"], first=s["starts"], max_new=1, out=s["means"])
    q1 = s["q"].view(B, H, d)
    mattn.decode_select(q1, s["means"], 64, 12, seq_lens=s["lens"], out=s["ids"], workspace=s["ws1"])
    mattn.decode_blocks(q1, s["kc"], s["vc"], s["ids"], 64, seq_lens=s["lens"], out=s["o"], lse=s["lse"],
                        workspace=s["ws2"])


def test_a_step_of_them_together():
    """Each operator's output against the 64-bit form of what it was given."""
    s = _step_inputs(5)
    old = s["means"].clone()
    B, Hkv, d, starts = 3, 2, 128, s["starts"].tolist()
    _step(s)
    torch.cuda.synchronize()
    qkv = s["qkv"].unflatten(-1, (-1, d))
    for got, x, w in ((s["q"], qkv[:, :, :8], s["plan"].q_weight),
                      (torch.stack([s["kc"][b, :, n] for b, n in enumerate(starts)])[:, :, None], qkv[:, :, 8:10],
                       s["plan"].k_weight)):
        y, mag = ref_rope(x, w, s["pos"], s["plan"].inv_freq, [16, 24, 24], 1e-6, False)
        assert bool(((got.transpose(1, 2).double().cpu() - y).abs() <= U * y.abs() + 2.0 ** -19 * mag).all())
    ref, tol = ref_means(s["kc"], 64, s["lens"].tolist(), starts, 1, old)
    assert bool(((s["means"].double().cpu() - ref).abs() <= tol).all())
    q1 = s["q"].view(B, 8, d)
    assert torch.equal(s["ids"].cpu(), ref_select(q1, s["means"], 64, 12, s["lens"].tolist(), 1, 1))
    lists = []
    for b, n in enumerate(s["lens"].tolist()):
        row = []
        for h in range(Hkv):
            spans = [(i * 64, min(i * 64 + 64, n)) for i in s["ids"][b, h].tolist() if i >= 0]
            row.append(tuple(torch.cat([t[b, h, x:y] for x, y in spans]).double().cpu() for t in (s["kc"], s["vc"])))
        lists.append(row)
    check_attention(s["o"], s["lse"], q1, lists, None, d ** -0.5, "step")


def _outs(s):
    return [s[x].clone() for x in ("q", "kc", "vc", "means", "ids", "o", "lse")]


def test_two_captured_steps_replayed_together():
    """Two graphs with workspaces of their own, replayed on two streams at once,
    give the eager results bit for bit, on new inputs."""
    states, graphs = [_step_inputs(21), _step_inputs(22)], []
    for s in states:
        _step(s)  # (outside a capture once)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(s)
        graphs.append(graph)
    for rounds in range(3):
        g = _gen(100 + rounds)
        for s in states:
            s["qkv"].copy_(_randn(g, *s["qkv"].shape))
        want = []
        for s in states:
            _step(s)
            torch.cuda.synchronize()
            want.append(_outs(s))
        streams = [torch.cuda.Stream() for _ in graphs]
        for s in states:
            for x in ("o", "lse", "ids"):
                s[x].zero_()
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for s, w in zip(states, want):
            for x, y in zip(_outs(s), w):
                assert torch.equal(x, y)


def _guarded(shape, dtype, fill):
    """A tensor inside a buffer of `fill`, with 4 KB of it on either side."""
    n = int(np.prod(shape))
    pad = 4096 // torch.empty((), dtype=dtype).element_size()
    whole = torch.full((n + 2 * pad,), fill, dtype=dtype, device="cuda")
    return whole[pad:pad + n].view(shape), (whole[:pad], whole[pad + n:])


@pytest.mark.parametrize("B,H,Hkv,d,P,L", [(1, 4, 1, 64, 130, 0), (5, 12, 1, 128, 1000, 45), (37, 8, 2, 128, 257, 33),
                                           (70, 6, 2, 64, 300, 17), (33, 4, 1, 256, 129, 50), (3, 8, 2, 256, 0, 700)])
def test_writes_stay_in_their_buffers(B, H, Hkv, d, P, L):
    """Outputs and workspaces of exactly the bytes asked for, between guards."""
    g = _gen(B + d)
    q, kp, k = _randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, B, Hkv, L, d)
    guards = []

    def buf(shape, dtype, fill):
        t, around = _guarded(shape, dtype, fill)
        guards.append((around, fill))
        return t

    def workspace(made):
        return buf((made.numel() * made.element_size(),), torch.uint8, 165)

    o, lse = buf((B, H, d), torch.bfloat16, 7.0), buf((B, H), torch.float32, 7.0)
    mattn.decode_shared(q, kp, kp, k, k, out=o, lse=lse, workspace=workspace(mattn.decode_shared_workspace(B, H, Hkv, P, L, d)))
    if L:
        n = -(-L // 16)
        means, ids = buf((B, Hkv, n, d), torch.bfloat16, 7.0), buf((B, Hkv, 2), torch.int32, 7)
        mattn.block_means(k, 16, out=means)
        mattn.decode_select(q, means, 16, 2, out=ids, workspace=workspace(mattn.decode_select_workspace(B, H, Hkv, n, d)))
        o, lse = buf((B, H, d), torch.bfloat16, 7.0), buf((B, H), torch.float32, 7.0)
        mattn.decode_blocks(q, k, k, ids, 16, out=o, lse=lse,
                            workspace=workspace(mattn.decode_blocks_workspace(B, H, Hkv, 2, 16, d)))
        many = torch.zeros((B, Hkv, 1100), dtype=torch.int32, device="cuda")
        mattn.decode_blocks(q, k, k, many, 16, out=o, lse=lse,
                            workspace=workspace(mattn.decode_blocks_workspace(B, H, Hkv, 1100, 16, d)))
        x = _randn(g, B, 3, H + 2 * Hkv, d)
        plan = mattn.RopePlan(torch.ones(16, device="cuda"))
        qo, kc, vc = (buf((B, h, r, d), torch.bfloat16, 7.0) for h, r in ((H, 3), (Hkv, L), (Hkv, L)))
        starts = _i32([(-2, L - 1, L, 5, (1 << 31) - 1, -(1 << 31))[b % 6] for b in range(B)])
        mattn.qk_rope(x[:, :, :H], x[:, :, H:H + Hkv], x[:, :, H + Hkv:], plan, qo, kc, vc, starts=starts)
        for b, n0 in enumerate(starts.tolist()):
            for c, at in ((kc, H), (vc, H + Hkv)):
                there = [n0 + i for i in range(3) if 0 <= n0 + i < L]
                rest = torch.ones(L, dtype=torch.bool)
                rest[there] = False
                assert bool((c[b][:, rest.cuda()] == 7.0).all()), "a cache row that no token has"
                if c is vc and there:
                    assert torch.equal(c[b][:, there], x[b, [r - n0 for r in there], at:].transpose(0, 1))
    torch.cuda.synchronize()
    for around, fill in guards:
        for t in around:
            assert bool((t == fill).all()), "a write outside the buffer"


def test_lengths_of_any_32_bit_value():
    """Lengths past the cache count as its own, negative ones as 0, to the ends of int32."""
    g = _gen(77)
    B, H, Hkv, d, L = 4, 8, 2, 128, 100
    q, k, v, kp = _randn(g, B, H, d), _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d), _randn(g, Hkv, 70, d)
    wild, tame = _i32([-(1 << 31), (1 << 31) - 1, 37, -1]), _i32([0, L, 37, 0])
    ids = torch.tensor([0, 3, 6, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32, device="cuda").expand(B, Hkv, 5).contiguous()
    means = mattn.block_means(k, 16)
    for run in (lambda n: mattn.decode_shared(q, kp, kp, k, v, seq_lens=n),
                lambda n: mattn.decode_blocks(q, k, v, ids, 16, seq_lens=n),
                lambda n: (mattn.block_means(k, 16, seq_lens=n),),
                lambda n: (mattn.block_means(k, 16, seq_lens=n, first=n, max_new=(1 << 31) - 1, out=means.clone()),),
                lambda n: (mattn.decode_select(q, means, 16, 3, seq_lens=n),)):
        for x, y in zip(run(wild), run(tame)):
            assert torch.equal(x, y)


def test_calls_on_other_streams_overlap_safely():
    """Shared-prefix calls without a given workspace on two streams, one named by
    its handle, repeated: bit-identical results."""
    g = _gen(8)
    B, H, Hkv, d, P, L = 40, 8, 2, 128, 2000, 60
    a = [(_randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, Hkv, P, d), _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d))
         for _ in range(2)]
    want = [mattn.decode_shared(*x) for x in a]
    torch.cuda.synchronize()
    s0, s1 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s0):
            got.append((0, mattn.decode_shared(*a[0])))
        got.append((1, mattn.decode_shared(*a[1], stream=s1.cuda_stream)))
    torch.cuda.synchronize()
    for i, (o, lse) in got:
        assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_calls_from_threads():
    """Four threads on streams of their own: every result as if alone."""
    import threading

    cases, wrong = [], []
    for i in range(4):
        g = _gen(60 + i)
        B = 3 + 7 * i
        x = (_randn(g, B, 8, 128), _randn(g, 2, 900, 128), _randn(g, 2, 900, 128), _randn(g, B, 2, 200, 128),
             _randn(g, B, 2, 200, 128))
        cases.append(x)

    def run(x):
        means = mattn.block_means(x[3], 16)
        ids = mattn.decode_select(x[0], means, 16, 5)
        return [*mattn.decode_shared(*x), means, ids, *mattn.decode_blocks(x[0], x[3], x[4], ids, 16)]

    want = [run(x) for x in cases]
    torch.cuda.synchronize()

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(60):
                    got = run(cases[i])
                st.synchronize()
            if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                wrong.append(i)
        except Exception as e:  # (an exception in a thread would pass unseen)
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_shared_replays_in_a_graph():
    g = _gen(12)
    B, H, Hkv, d, P, L = 33, 8, 2, 64, 700, 40
    x = [_randn(g, B, H, d), _randn(g, Hkv, P, d), _randn(g, Hkv, P, d), _randn(g, B, Hkv, L, d), _randn(g, B, Hkv, L, d)]
    lens = _i32([b % 41 for b in range(B)])
    mattn.decode_shared(*x, seq_lens=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = mattn.decode_shared(*x, seq_lens=lens)  # the workspace is the graph's
    for seed in (1, 2):
        for t in x:
            t.copy_(_randn(_gen(seed), *t.shape))
        lens.add_(1)
        graph.replay()
        o2, lse2 = mattn.decode_shared(*x, seq_lens=lens)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_chained_calls_see_what_came_before():
    """Long runs of calls without a wait between them, on buffers that torch's
    own kernels and copies rewrite before each: every call begins only after
    what came before it on the stream, and what follows begins after it."""
    s = _step_inputs(41)
    g = _gen(42)
    rows = [_randn(g, *s["qkv"].shape) for _ in range(8)]
    host = [r.cpu().pin_memory() for r in rows]
    want = []
    for i in range(24):  # one at a time
        s["qkv"].copy_(rows[i % 8])
        _step(s)
        torch.cuda.synchronize()
        want.append(_outs(s))
    got = []
    for i in range(24):
        if i % 3 == 0:
            s["qkv"].zero_()
            s["qkv"].add_(rows[i % 8])
        else:
            s["qkv"].copy_(rows[i % 8] if i % 3 == 1 else host[i % 8], non_blocking=True)
        for x in ("q", "o", "lse", "ids"):
            s[x].zero_()
        _step(s)
        got.append(_outs(s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_capture_among_other_work():
    """A captured step behind memory sets, copies and work joined from another
    stream, followed by torch's kernels: the replay equals the eager run."""
    s = _step_inputs(51)
    src = torch.empty_like(s["qkv"])
    side = torch.cuda.Stream()
    total = torch.zeros((), device="cuda")

    def run():
        here = torch.cuda.current_stream()
        s["qkv"].zero_()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            half = src * 0.5
        here.wait_stream(side)
        s["qkv"].copy_(half)
        s["qkv"].add_(half)
        s["o"].zero_()
        _step(s)
        total.copy_(s["o"].float().sum())
        mattn.decode_shared(s["q"].view(3, 8, 128), s["kc"][0, :, :500].contiguous(), s["vc"][0, :, :500].contiguous(),
                            s["kc"], s["vc"], seq_lens=s["lens"], out=s["o2"], lse=s["lse"])
        half.record_stream(here)

    s["o2"] = torch.empty_like(s["o"])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for seed in (1, 2, 3):
        src.copy_(_randn(_gen(seed), *src.shape))
        run()
        torch.cuda.synchronize()
        want = _outs(s) + [s["o2"].clone(), total.clone()]
        for x in ("q", "o", "o2", "lse"):
            s[x].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(_outs(s) + [s["o2"], total], want):
            assert torch.equal(x, y)


def test_binding_refusals():
    g = _gen(0)
    q, kp, c = _randn(g, 2, 4, 128), _randn(g, 2, 64, 128), _randn(g, 2, 2, 32, 128)
    with pytest.raises(ValueError):
        mattn.decode_shared(q, kp[:1], kp[:1], c, c)
    with pytest.raises(ValueError):
        mattn.decode_shared(q, kp, kp, c, c, seq_lens=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        mattn.decode_shared(q, kp, kp, c.transpose(1, 2), c.transpose(1, 2))
    with pytest.raises(mattn.MattnError):
        mattn.decode_shared(q, kp, kp, c, c, prefix_len=65)
    with pytest.raises(mattn.MattnError):
        mattn.decode_shared(q, kp, kp, c, c, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mattn.decode_blocks(q, c, c, torch.zeros((2, 1, 4), dtype=torch.int32, device="cuda"), 16)
    with pytest.raises(ValueError):
        mattn.block_means(c, 16, first=_i32([0, 0]))
    with pytest.raises(mattn.MattnError):
        mattn.decode_select(q, c, 16, 2, keep_first=2, keep_recent=1)
    x = _randn(g, 2, 3, 4, 128)
    plan = mattn.RopePlan(torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        mattn.qk_rope(x.transpose(1, 2), x, None, plan)
    with pytest.raises(ValueError):
        mattn.qk_rope(x, x, None, plan, positions=torch.zeros((2, 2, 3), dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        mattn.RopePlan(torch.ones(64, device="cuda"), [30, 30])


def test_debug_library_agrees():
    """The library with device bounds checks gives the same bits and finds nothing."""
    s = _step_inputs(31)
    _step(s)
    a = [_randn(_gen(3), 20, 8, 128), _randn(_gen(4), 1, 300, 128), _randn(_gen(5), 1, 300, 128),
         _randn(_gen(6), 20, 1, 50, 128), _randn(_gen(7), 20, 1, 50, 128)]
    want = _outs(s) + list(mattn.decode_shared(*a, seq_lens=_i32([n + 7 for n in range(20)])))
    torch.cuda.synchronize()
    mattn.use_debug_library(True)
    try:
        _step(s)
        got = _outs(s) + list(mattn.decode_shared(*a, seq_lens=_i32([n + 7 for n in range(20)])))
        torch.cuda.synchronize()
        rc, word = mattn.device_status()
        assert rc == 0, f"device error word {word:#x}"
    finally:
        mattn.use_debug_library(False)
    for x, y in zip(got, want):
        assert torch.equal(x, y)
