"""Operators of a decode step and of the pass that feeds it, as measured cases.

    rope    norms of queries and keys per head with the position rotation (one
            to three position axes) in the same pass, from the projection's
            layout into the attention's layouts, keys and values into the cache
    shared  decode attention of a batch whose sequences share one long prefix
    means   the mean key of every block of a key cache, whole or kept up to date
    select  per sequence and key/value head, the blocks its queries score highest
    blocks  decode attention over the selected blocks of the cache

`own` chooses between the plain form (elementary torch operations in 32 bits,
64 for far angles and for scores next to a border) and this package's calls.
Sizes come from the package's workloads: 16,384-token ViT layers of 16 heads of
80, 32,768-token prefill with 32 query and 8 key/value heads of 128, and the
131,072-token decode step with 16 query and 4 key/value heads of 256.
"""

import math

import torch

own = False
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # prefill of a 32,768-token image-and-text prompt: 3 position axes, normed heads
        {"name": "rope_prefill32k", "op": "rope", "B": 1, "N": 32768, "H": 32, "Hkv": 8, "d": 128, "L": 32768,
         "axes": 3, "rot": 64, "norm": True, "interleaved": False, "base": 1e6, "far": 0, "dtype": "bf16"},
        # a ViT layer over a 128 x 128 patch grid, 2 axes, pairs side by side, 32-bit activations
        {"name": "rope_vit16384_f32", "op": "rope", "B": 1, "N": 16384, "H": 16, "Hkv": 16, "d": 80, "L": 16384,
         "axes": 2, "rot": 40, "norm": False, "interleaved": True, "base": 1e4, "far": 0, "dtype": "f32"},
        # one new token for each of 64 requests, appended to their caches at far positions (latency)
        {"name": "rope_step", "op": "rope", "B": 64, "N": 1, "H": 32, "Hkv": 8, "d": 128, "L": 1024,
         "axes": 1, "rot": 64, "norm": True, "interleaved": False, "base": 1e6, "far": 1 << 20, "dtype": "bf16"},
        # four requests behind a short system prompt (latency)
        {"name": "shared_small", "op": "shared", "B": 4, "H": 16, "Hkv": 4, "d": 128, "P": 1024, "L": 64,
         "sink": False},
        # 64 requests over one 32K-token document, some hundred own tokens each
        {"name": "shared_64x32k", "op": "shared", "B": 64, "H": 32, "Hkv": 8, "d": 128, "P": 32768, "L": 512,
         "sink": False},
        # 16 samples of one 128K-token prompt, heads of 256, sink logits; an odd prefix length
        {"name": "shared_16x128k_d256", "op": "shared", "B": 16, "H": 16, "Hkv": 4, "d": 256, "P": 131071, "L": 1000,
         "sink": True},
        # block means of freshly prefilled caches
        {"name": "means_8x32k", "op": "means", "B": 8, "Hkv": 8, "d": 128, "L": 32768, "block": 64, "new": 0},
        # the same kept up to date after one new token per request (latency)
        {"name": "means_step", "op": "means", "B": 64, "Hkv": 8, "d": 128, "L": 4096, "block": 64, "new": 1},
        # 64 of 2,048 blocks for each of 16 x 8 key/value heads
        {"name": "select_16x128k", "op": "select", "B": 16, "H": 32, "Hkv": 8, "d": 128, "n_blocks": 2048,
         "block": 64, "top_k": 64},
        # one request at 128K tokens, heads of 256 (latency)
        {"name": "select_1x128k_d256", "op": "select", "B": 1, "H": 16, "Hkv": 4, "d": 256, "n_blocks": 2048,
         "block": 64, "top_k": 32},
        # the selected 4,096 tokens of 16 requests' 32K caches
        {"name": "blocks_16x32k", "op": "blocks", "B": 16, "H": 32, "Hkv": 8, "d": 128, "L": 32768, "block": 64,
         "top_k": 64, "sink": False},
        # one request's 2,048 selected tokens of 128K, heads of 256, sink logits (latency)
        {"name": "blocks_1x128k_d256", "op": "blocks", "B": 1, "H": 16, "Hkv": 4, "d": 256, "L": 131072, "block": 64,
         "top_k": 32, "sink": True},
    ]


HEADS = ((4, 4), (8, 2), (16, 4), (32, 8), (8, 1), (6, 2), (32, 4), (5, 1), (12, 1))


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "shared", "means", "select", "blocks"))
    H, Hkv = rng.choice(HEADS)
    if op == "rope":
        d = rng.choice((64, 80, 96, 128, 256))
        step = rng.random() < 0.4  # one or a few new tokens of many requests, or a prefill
        B, N = (_log(rng, 1, 128), rng.randint(1, 4)) if step else (rng.randint(1, 4), _log(rng, 5, 16384))
        while B * N * (H + 2 * Hkv) * d > 48 * 128 * 32768:
            N //= 2
        rot = d // 2 if rng.random() < 0.7 else 8 * rng.randint(1, d // 16)
        return {"op": op, "B": B, "N": N, "H": H, "Hkv": Hkv, "d": d, "L": N + _log(rng, 1, 600), "axes": rng.randint(1, 3),
                "rot": rot, "norm": rng.random() < 0.6, "interleaved": rng.random() < 0.3,
                "base": rng.choice((1e4, 5e5, 1e6)), "far": rng.choice((0, 1000, 1 << 20)),
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
    if op == "shared":
        d = rng.choice((64, 128, 256))
        B, P, L = _log(rng, 1, 128), _log(rng, 1, 131072), _log(rng, 1, 2048)
        while B * H * P * d > 64 * 32 * 32768 * 128:  # no more work than the largest listed case
            P = P // 2 + 1
        while B * Hkv * L * d > 64 * 8 * 512 * 128:
            L = L // 2 + 1
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "P": P, "L": L, "sink": rng.random() < 0.4}
    if op == "means":
        d, L, B = rng.choice((64, 128, 256)), _log(rng, 1, 65536), _log(rng, 1, 64)
        while B * Hkv * L * d > 8 * 8 * 32768 * 128:
            L = L // 2 + 1
        return {"op": op, "B": B, "Hkv": Hkv, "d": d, "L": L, "block": rng.choice((16, 32, 64, 128)),
                "new": rng.choice((0, 0, 1, rng.randint(2, 300)))}
    if op == "select":
        d, n, B = rng.choice((64, 128, 256)), _log(rng, 1, 8192), _log(rng, 1, 64)
        while B * Hkv * n * d > 16 * 8 * 2048 * 128:
            n = n // 2 + 1
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "n_blocks": n, "block": rng.choice((16, 32, 64, 128)),
                "top_k": rng.choice((2, 7, 16, 64, _log(rng, 2, 512)))}
    d, block = rng.choice((64, 128, 256)), rng.choice((16, 32, 64, 128))
    L, B, k = _log(rng, 1, 65536), _log(rng, 1, 32), _log(rng, 2, 128)
    while B * Hkv * L * d > 16 * 8 * 32768 * 128:
        L = L // 2 + 1
    while B * Hkv * k * block * d > 16 * 8 * 4096 * 128:
        k = k // 2 + 1
    return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "L": L, "block": block, "top_k": k, "sink": rng.random() < 0.4}


# ------------------------------------------------------------------ the inputs
def _ceil(a, b):
    return -(-a // b)


def _sections(c):
    """Rotated pairs of each axis: 1/4, 3/8, 3/8 of them for three axes, else even shares."""
    r, n = c["rot"], c["axes"]
    if n == 1:
        return [r]
    if n == 2:
        return [r - r // 2, r // 2]
    a = max(1, r // 4)
    b = (r - a) // 2
    return [a, r - a - b, b]


def _inv_freq(c):
    p = torch.arange(c["rot"], dtype=torch.float64, device=DEVICE)
    return torch.pow(torch.tensor(c["base"], dtype=torch.float64, device=DEVICE), -p / c["rot"]).to(torch.float32)


def _lens(g, B, low, high):
    """Lengths of [low, high], the first one full."""
    n = torch.randint(low, high + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32)
    n[0] = high
    return n


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(int(seed) * 7919 + 11)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)

    s = {"c": c}
    if c["op"] == "rope":
        B, N, H, Hkv, d, L = (c[x] for x in ("B", "N", "H", "Hkv", "d", "L"))
        t = TYPES[c["dtype"]]
        qkv = normal(B, N, (H + 2 * Hkv) * d, dtype=t)  # the projection's output, heads side by side
        s["q"] = qkv[..., : H * d].view(B, N, H, d)
        s["k"] = qkv[..., H * d : (H + Hkv) * d].view(B, N, Hkv, d)
        s["v"] = qkv[..., (H + Hkv) * d :].view(B, N, Hkv, d)
        s["starts"] = torch.randint(0, L - N + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32)
        s["lens"] = _lens(g, B, 1, N) if B > 1 else None  # a padded batch
        n = torch.arange(N, device=DEVICE, dtype=torch.int32)
        if c["axes"] == 1:
            pos = n[None, None] + s["starts"][None, :, None]
        else:  # (time,) row, column of a patch grid
            side = max(1, math.isqrt(N))
            pos = torch.stack([n // (side * side), n // side % side, n % side][3 - c["axes"] :])[:, None]
            pos = pos + 0 * s["starts"][None, :, None]
        if c["far"]:
            pos = pos + torch.randint(0, c["far"], (1, B, 1), generator=g, device=DEVICE, dtype=torch.int32)
        s["pos"] = pos.to(torch.int32).contiguous()
        s["inv_freq"], s["sections"] = _inv_freq(c), _sections(c)
        s["wq"] = 1 + 0.1 * normal(d, dtype=torch.float32) if c["norm"] else None
        s["wk"] = 1 + 0.1 * normal(d, dtype=torch.float32) if c["norm"] else None
        s["q_out"] = torch.zeros((B, H, N, d), device=DEVICE, dtype=t)
        s["k_cache"], s["v_cache"] = normal(B, Hkv, L, d, dtype=t), normal(B, Hkv, L, d, dtype=t)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["plan"] = mattn.RopePlan(s["inv_freq"], s["sections"], q_weight=s["wq"], k_weight=s["wk"], eps=EPS,
                                       interleaved=c["interleaved"])
    elif c["op"] == "shared":
        B, H, Hkv, d, P, L = (c[x] for x in ("B", "H", "Hkv", "d", "P", "L"))
        s["q"] = normal(B, H, d)
        s["kp"], s["vp"] = normal(Hkv, P, d), normal(Hkv, P, d)
        s["k"], s["v"] = normal(B, Hkv, L, d), normal(B, Hkv, L, d)
        s["lens"] = _lens(g, B, 0, L)
        s["sink"] = normal(H, dtype=torch.float32) if c["sink"] else None
        _outputs(s, B, H, d)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["work"] = mattn.decode_shared_workspace(B, H, Hkv, P, L, d, device=DEVICE)
    elif c["op"] == "means":
        B, Hkv, d, L, bs = (c[x] for x in ("B", "Hkv", "d", "L", "block"))
        s["k"] = normal(B, Hkv, L, d)
        s["lens"] = _lens(g, B, max(1, L // 2), L)
        s["new"] = c["new"] or L
        s["first"] = (s["lens"] - c["new"]).clamp(min=0) if c["new"] else torch.zeros_like(s["lens"])
        s["means"] = normal(B, Hkv, _ceil(L, bs), d)
    elif c["op"] == "select":
        B, H, Hkv, d, n = (c[x] for x in ("B", "H", "Hkv", "d", "n_blocks"))
        s["q"] = normal(B, H, d)
        s["means"] = normal(B, Hkv, n, d) * 0.25
        s["lens"] = _lens(g, B, max(1, n * c["block"] // 2), n * c["block"])
        s["ids"] = torch.empty((B, Hkv, c["top_k"]), device=DEVICE, dtype=torch.int32)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["work"] = mattn.decode_select_workspace(B, H, Hkv, n, d, device=DEVICE)
    else:
        B, H, Hkv, d, L, bs, k = (c[x] for x in ("B", "H", "Hkv", "d", "L", "block", "top_k"))
        s["q"] = normal(B, H, d)
        s["k"], s["v"] = normal(B, Hkv, L, d), normal(B, Hkv, L, d)
        s["lens"] = _lens(g, B, max(1, L // 2), L)
        n = (s["lens"].long() + bs - 1) // bs  # blocks of each sequence
        at = torch.rand((B, Hkv, max(k, _ceil(L, bs))), generator=g, device=DEVICE)
        i = torch.arange(at.shape[2], device=DEVICE)
        at = torch.where(i < n[:, None, None], at, torch.full_like(at, 2.0))
        at[torch.arange(B, device=DEVICE), :, n - 1] = -1.0  # the newest block is always kept
        order = at.argsort(dim=2)[..., :k]
        order = torch.where(order < n[:, None, None], order, torch.full_like(order, 1 << 30)).sort(dim=2).values
        s["ids"] = torch.where(order < (1 << 30), order, torch.full_like(order, -1)).to(torch.int32)
        s["sink"] = normal(H, dtype=torch.float32) if c["sink"] else None
        _outputs(s, B, H, d)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["work"] = mattn.decode_blocks_workspace(B, H, Hkv, k, bs, d, device=DEVICE)
    return s


def _outputs(s, B, H, d):
    s["o"] = torch.empty((B, H, d), device=DEVICE, dtype=torch.bfloat16)
    s["lse"] = torch.empty((B, H), device=DEVICE, dtype=torch.float32)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"rope": _rope, "shared": _shared, "means": _means, "select": _select, "blocks": _blocks}[s["c"]["op"]](s)


def _own(s):
    import block_sparse_attention_masked_gb300 as mattn

    c = s["c"]
    if c["op"] == "rope":
        mattn.qk_rope(s["q"], s["k"], s["v"], s["plan"], s["q_out"], s["k_cache"], s["v_cache"], positions=s["pos"],
                      starts=s["starts"], lens=s["lens"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if c["op"] == "shared":
        return mattn.decode_shared(s["q"], s["kp"], s["vp"], s["k"], s["v"], seq_lens=s["lens"], sink=s["sink"],
                                   out=s["o"], lse=s["lse"], workspace=s["work"])
    if c["op"] == "means":
        return mattn.block_means(s["k"], c["block"], seq_lens=s["lens"], first=s["first"], max_new=s["new"],
                                 out=s["means"])
    if c["op"] == "select":
        return mattn.decode_select(s["q"], s["means"], c["block"], c["top_k"], seq_lens=s["lens"], keep_first=1,
                                   keep_recent=1, out=s["ids"], workspace=s["work"])
    return mattn.decode_blocks(s["q"], s["k"], s["v"], s["ids"], c["block"], seq_lens=s["lens"], sink=s["sink"],
                               out=s["o"], lse=s["lse"], workspace=s["work"])


def _rotate(x, cos, sin, rot, interleaved):
    """x [..., heads, d] with its first 2 rot dims turned by the angles [..., 1, rot]."""
    if interleaved:
        a, b = x[..., 0 : 2 * rot : 2], x[..., 1 : 2 * rot : 2]
    else:
        a, b = x[..., :rot], x[..., rot : 2 * rot]
    ra, rb = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((ra, rb), dim=-1).flatten(-2) if interleaved else torch.cat((ra, rb), dim=-1)
    return torch.cat((turned, x[..., 2 * rot :]), dim=-1)


def _normed(x, w):
    if w is None:
        return x
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS) * w


def _rope(s):
    c = s["c"]
    B, N, L = c["B"], c["N"], c["L"]
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=s["pos"].device),
                                   torch.tensor(s["sections"], device=s["pos"].device), output_size=c["rot"])
    angle = s["pos"].double()[axis].permute(1, 2, 0) * s["inv_freq"].double()  # [B, N, rot], far positions in 64 bits
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    q = _rotate(_normed(s["q"].float(), s["wq"]), cos, sin, c["rot"], c["interleaved"]).to(s["q"].dtype)
    k = _rotate(_normed(s["k"].float(), s["wk"]), cos, sin, c["rot"], c["interleaved"]).to(s["k"].dtype)
    n = torch.arange(N, device=q.device)
    lens = s["lens"] if s["lens"] is not None else torch.full((B,), N, device=q.device)
    there = n[None] < lens[:, None]  # [B, N]: tokens of the batch, not its padding
    at = (s["starts"][:, None].long() + n[None]).clamp(max=L - 1)
    b = torch.arange(B, device=q.device)[:, None]
    s["q_out"].copy_(torch.where(there[:, None, :, None], q.transpose(1, 2), s["q_out"]))
    kt, vt = s["k_cache"].transpose(1, 2), s["v_cache"].transpose(1, 2)  # [B, L, heads, d] views
    kt[b, at] = torch.where(there[..., None, None], k, kt[b, at])
    vt[b, at] = torch.where(there[..., None, None], s["v"], vt[b, at])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _softmax_sum(x, values, sink):
    """sum_j softmax(x)_j values_j and the log of the normaliser, which `sink` joins; x [..., G, J], values [..., J, d]."""
    m = x.amax(dim=-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(x - m)
    z = e.sum(dim=-1, keepdim=True)
    if sink is not None:
        z = z + torch.exp(sink - m)
    o = torch.matmul(e, values) / torch.where(z > 0, z, torch.ones_like(z))
    return o, (m + torch.log(z)).squeeze(-1)


def _shared(s):
    c = s["c"]
    B, H, Hkv, d, P, L = (c[x] for x in ("B", "H", "Hkv", "d", "P", "L"))
    G = H // Hkv
    q = s["q"].float().view(B, Hkv, G, d) / math.sqrt(d)
    # the prefix's scores as one product per key/value head over all sequences' queries
    rows = q.transpose(0, 1).reshape(Hkv, B * G, d)
    x = torch.matmul(rows, s["kp"].float().transpose(1, 2))  # [Hkv, B G, P]
    y = torch.matmul(q, s["k"].float().transpose(2, 3))  # [B, Hkv, G, L]
    j = torch.arange(L, device=q.device)
    y = torch.where(j < s["lens"][:, None, None, None], y, torch.full_like(y, -math.inf))
    y = y.transpose(0, 1).reshape(Hkv, B * G, L)
    m = torch.maximum(x.amax(dim=-1), y.amax(dim=-1))[..., None]
    if s["sink"] is not None:
        sink = s["sink"].view(Hkv, 1, G).expand(Hkv, B, G).reshape(Hkv, B * G, 1)
        m = torch.maximum(m, sink)
    x, y = torch.exp(x - m), torch.exp(y - m)
    z = x.sum(dim=-1, keepdim=True) + y.sum(dim=-1, keepdim=True)
    if s["sink"] is not None:
        z = z + torch.exp(sink - m)
    own_part = torch.matmul(y.view(Hkv, B, G, L).transpose(0, 1), s["v"].float())  # [B, Hkv, G, d]
    o = torch.matmul(x, s["vp"].float()) + own_part.transpose(0, 1).reshape(Hkv, B * G, d)
    o = (o / z).view(Hkv, B, G, d).transpose(0, 1).reshape(B, H, d)
    lse = (m + torch.log(z)).view(Hkv, B, G).transpose(0, 1).reshape(B, H)
    return o.to(torch.bfloat16), lse


def _means(s):
    c = s["c"]
    B, Hkv, d, L, bs = (c[x] for x in ("B", "Hkv", "d", "L", "block"))
    blocks = s["means"].shape[2]
    n = min(blocks, (s["new"] - 1) // bs + 2)  # blocks that `new` keys can lie in
    dev = s["k"].device
    first, lens = s["first"].long()[:, None], s["lens"].long()[:, None]
    end = torch.minimum(lens, first + s["new"])
    blk = torch.minimum(first // bs, torch.full_like(first, blocks - n)) + torch.arange(n, device=dev)  # [B, n]
    there = (blk >= first // bs) & (blk * bs < end) & (first < end)  # the block holds a new key
    at = blk[..., None] * bs + torch.arange(bs, device=dev)  # [B, n, bs] positions
    seen = at < lens[..., None]
    b = torch.arange(B, device=dev)[:, None]
    if n == blocks and L == n * bs:  # the whole cache, in order
        rows = s["k"].view(B, Hkv, n, bs, d).transpose(1, 2).transpose(2, 3).float()  # [B, n, bs, Hkv, d]
    else:
        rows = s["k"].transpose(1, 2)[b[..., None], at.clamp(max=L - 1)].float()
    sums = (rows * seen[..., None, None]).sum(dim=2)
    mean = (sums / seen.sum(dim=-1).clamp(min=1)[..., None, None]).to(torch.bfloat16)
    old = s["means"].transpose(1, 2)  # [B, blocks, Hkv, d] view
    old[b, blk] = torch.where(there[..., None, None], mean, old[b, blk])
    return s["means"]


def _select(s):
    c = s["c"]
    B, H, Hkv, d, n, k = (c[x] for x in ("B", "H", "Hkv", "d", "n_blocks", "top_k"))
    # scores next to the border decide: 64 bits
    x = torch.matmul(s["means"].double(), s["q"].double().view(B, Hkv, H // Hkv, d).transpose(2, 3)).amax(dim=-1)
    i = torch.arange(n, device=x.device)
    have = ((s["lens"].long() + c["block"] - 1) // c["block"]).clamp(max=n)[:, None, None]
    x = torch.where((i < 1) | (i >= have - 1), torch.full_like(x, math.inf), x)  # the first and the newest block
    x = torch.where(i < have, x, torch.full_like(x, -math.inf))
    order = torch.sort(x, dim=-1, descending=True, stable=True).indices[..., :k]
    order = torch.where(order < have, order, torch.full_like(order, n)).sort(dim=-1).values
    order = torch.where(order < n, order, torch.full_like(order, -1)).to(torch.int32)
    s["ids"].fill_(-1)
    s["ids"][..., : order.shape[-1]] = order
    return s["ids"]


def _blocks(s):
    c = s["c"]
    B, H, Hkv, d, L, bs, k = (c[x] for x in ("B", "H", "Hkv", "d", "L", "block", "top_k"))
    dev = s["k"].device
    at = s["ids"].long()[..., None] * bs + torch.arange(bs, device=dev)  # [B, Hkv, k, bs]
    seen = ((s["ids"][..., None] >= 0) & (at < s["lens"].long()[:, None, None, None])).view(B, Hkv, 1, k * bs)
    at = at.clamp(0, L - 1).view(B, Hkv, k * bs, 1).expand(B, Hkv, k * bs, d)
    keys, values = s["k"].gather(2, at).float(), s["v"].gather(2, at).float()
    x = torch.matmul(s["q"].float().view(B, Hkv, H // Hkv, d) / math.sqrt(d), keys.transpose(2, 3))
    x = torch.where(seen, x, torch.full_like(x, -math.inf))
    sink = s["sink"].view(1, Hkv, H // Hkv, 1) if s["sink"] is not None else None
    o, lse = _softmax_sum(x, values, sink)
    return o.reshape(B, H, d).to(torch.bfloat16), lse.reshape(B, H)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "rope":
        e = 4 if c["dtype"] == "f32" else 2
        T, h = c["B"] * c["N"], c["H"] + 2 * c["Hkv"]
        return {"bytes": 2 * T * h * c["d"] * e + 4 * T * c["axes"], "flops": 10 * T * h * c["d"]}
    if c["op"] == "shared":
        keys = c["Hkv"] * (c["P"] + c["B"] * c["L"] // 2)  # own tokens: half the capacity on average
        return {"bytes": 4 * c["d"] * keys + 4 * c["B"] * c["H"] * (c["d"] + 1),
                "flops": 4 * c["d"] * c["B"] * c["H"] * (c["P"] + c["L"] // 2)}
    if c["op"] == "means":
        rows = c["B"] * c["Hkv"]
        keys = min(3 * c["L"] // 4, c["new"] + c["block"] // 2) if c["new"] else 3 * c["L"] // 4
        return {"bytes": 2 * rows * c["d"] * (keys + _ceil(keys, c["block"])), "flops": rows * c["d"] * max(1, keys)}
    if c["op"] == "select":
        n = _ceil(3 * c["n_blocks"], 4)
        return {"bytes": 2 * c["d"] * (c["B"] * c["Hkv"] * n + c["B"] * c["H"]) + 4 * c["B"] * c["Hkv"] * c["top_k"],
                "flops": 2 * c["d"] * c["B"] * c["H"] * n}
    keys = min(c["top_k"] * c["block"], _ceil(3 * c["L"], 4))
    return {"bytes": 4 * c["d"] * c["B"] * c["Hkv"] * keys + 4 * c["B"] * c["H"] * (c["d"] + 1),
            "flops": 4 * c["d"] * c["B"] * c["H"] * keys}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions, sequence by sequence in 64 bits."""
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rope":
        return _exact_rope(s)
    if c["op"] == "means":
        return _exact_means(s)
    B, H, Hkv, d = (c[x] for x in ("B", "H", "Hkv", "d"))
    G = H // Hkv
    if c["op"] == "select":
        out = torch.full((B, Hkv, c["top_k"]), -1, dtype=torch.int32)
        lens, q = s["lens"].tolist(), s["q"].double().cpu()
        for b in range(B):
            n = min(c["n_blocks"], _ceil(lens[b], c["block"]))
            if not n:
                continue
            mean = s["means"][b, :, :n].double().cpu()
            for h in range(Hkv):
                score = (mean[h] @ q[b, h * G : (h + 1) * G].T).max(dim=1).values.tolist()
                rank = sorted(range(n), key=lambda i: (i != 0 and i != n - 1, -score[i], i))[: c["top_k"]]
                out[b, h, : len(rank)] = torch.tensor(sorted(rank), dtype=torch.int32)
        return out
    o = torch.zeros((B, H, d), dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((B, H), dtype=torch.float64, device=DEVICE)
    lens = s["lens"].tolist()
    if c["op"] == "shared":
        prefix = s["kp"].double(), s["vp"].double()
    else:
        ids = s["ids"].tolist()
    for b in range(B):
        for h in range(Hkv):
            if c["op"] == "shared":
                keys = torch.cat((prefix[0][h], s["k"][b, h, : lens[b]].double()))
                values = torch.cat((prefix[1][h], s["v"][b, h, : lens[b]].double()))
            else:
                bs = c["block"]
                spans = [(i * bs, min(i * bs + bs, lens[b])) for i in ids[b][h] if 0 <= i * bs < lens[b]]
                keys = torch.cat([s["k"][b, h, x:y] for x, y in spans]).double()
                values = torch.cat([s["v"][b, h, x:y] for x, y in spans]).double()
            x = s["q"][b, h * G : (h + 1) * G].double() @ keys.T * d**-0.5
            if s["sink"] is not None:  # one more logit without a value row
                x = torch.cat((x, s["sink"][h * G : (h + 1) * G].double()[:, None]), dim=1)
                values = torch.cat((values, torch.zeros_like(values[:1])))
            lse[b, h * G : (h + 1) * G] = torch.logsumexp(x, dim=1)
            o[b, h * G : (h + 1) * G] = torch.softmax(x, dim=1) @ values
    return o, lse


def _exact_rope(s):
    c = s["c"]
    B, N, R = c["B"], c["N"], c["rot"]
    q_out, k_out, v_out = s["q_out"].double(), s["k_cache"].double(), s["v_cache"].double()
    owner = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    lens = s["lens"].tolist() if s["lens"] is not None else [N] * B
    for b, start in enumerate(s["starts"].tolist()):
        n = lens[b]
        angle = s["pos"][owner, b, :n].double().T * s["inv_freq"].double()[None]
        turn = torch.complex(angle.cos(), angle.sin())  # [n, R]
        for src, w, dst, to in ((s["q"], s["wq"], q_out, 0), (s["k"], s["wk"], k_out, start)):
            x = src[b, :n].double()
            if w is not None:
                x = w.double() * x / ((x * x).sum(dim=-1, keepdim=True) / c["d"] + EPS).sqrt()
            if c["interleaved"]:
                z = torch.complex(x[..., 0 : 2 * R : 2].contiguous(), x[..., 1 : 2 * R : 2].contiguous())
            else:
                z = torch.complex(x[..., :R].contiguous(), x[..., R : 2 * R].contiguous())
            z = z * turn[:, None]
            y = x.clone()
            if c["interleaved"]:
                y[..., 0 : 2 * R : 2], y[..., 1 : 2 * R : 2] = z.real, z.imag
            else:
                y[..., :R], y[..., R : 2 * R] = z.real, z.imag
            dst[b, :, to : to + n] = y.transpose(0, 1)
        v_out[b, :, start : start + n] = s["v"][b, :n].double().transpose(0, 1)
    return q_out, k_out, v_out


def _exact_means(s):
    c = s["c"]
    bs, out = c["block"], s["means"].double()
    for b, (n, first) in enumerate(zip(s["lens"].tolist(), s["first"].tolist())):
        end = min(n, first + s["new"])
        lo = first // bs
        hi = _ceil(end, bs)  # blocks [lo, hi) hold the new keys
        if end <= first:
            continue
        keys = s["k"][b, :, lo * bs : min(n, hi * bs)].double()
        full = keys.shape[1] // bs
        if full:
            out[b, :, lo : lo + full] = keys[:, : full * bs].unflatten(1, (full, bs)).mean(dim=2)
        if keys.shape[1] > full * bs:
            out[b, :, lo + full] = keys[:, full * bs :].mean(dim=1)
    return out
