"""Operators of serving from a paged cache, as measured cases.

    write   new keys and values of packed prompts or of one token per request into
            the pages of a cache, as bf16 or in eight bits (e4m3) with a power of
            two for each token and head
    read    cached rows back as packed bf16 rows, in front of a prompt's own
    paged   attention of one new token per request over its pages
    packed  attention over a batch of prompts laid end to end, causal or not, with
            cached rows in front of them or without

`own` chooses between the plain form (elementary torch operations in 32 bits) and
this package's calls.  Sizes come from the package's workloads: layers of 32 query
and 8 key/value heads of 128, the 131,072-token decode step with 16 and 4 heads of
256, and 16,384 patches of ViT layers of 16 heads of 80.
"""

import math
import random

import torch

own = False
DEVICE = "cuda"
CODES = torch.float8_e4m3fn


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one new token for each of 64 requests (latency)
        {"name": "write_step", "op": "write", "B": 64, "T": 64, "Hkv": 8, "d": 128, "page": 64, "e4m3": True, "far": 4096},
        # the keys and values of 16 prompts, 32,768 tokens in all
        {"name": "write_prefill32k", "op": "write", "B": 16, "T": 32768, "Hkv": 8, "d": 128, "page": 64, "e4m3": True,
         "far": 0},
        # two short requests' rows back from small pages (latency)
        {"name": "read_small", "op": "read", "B": 2, "T": 601, "Hkv": 4, "d": 128, "page": 16, "e4m3": False, "far": 0},
        # what 16 requests have cached, in front of the next chunk of their prompts
        {"name": "read_32k", "op": "read", "B": 16, "T": 32768, "Hkv": 8, "d": 128, "page": 64, "e4m3": True, "far": 0},
        # four requests of up to 1,000 tokens (latency)
        {"name": "paged_small", "op": "paged", "B": 4, "H": 16, "Hkv": 4, "d": 128, "L": 1000, "page": 16, "e4m3": False,
         "sink": False, "window": 0, "first": 0},
        # a full batch of 64 requests of 4K to 8K tokens, in eight bits
        {"name": "paged_64x8k_e4m3", "op": "paged", "B": 64, "H": 32, "Hkv": 8, "d": 128, "L": 8192, "page": 64, "e4m3": True,
         "sink": False, "window": 0, "first": 0},
        # 16 long requests in bf16
        {"name": "paged_16x32k", "op": "paged", "B": 16, "H": 32, "Hkv": 8, "d": 128, "L": 32768, "page": 32, "e4m3": False,
         "sink": False, "window": 0, "first": 0},
        # one request at 128K tokens, heads of 256, sink logits; an odd length
        {"name": "paged_1x128k_d256", "op": "paged", "B": 1, "H": 16, "Hkv": 4, "d": 256, "L": 131071, "page": 128, "e4m3": True,
         "sink": True, "window": 0, "first": 0},
        # the first pass over a few short questions (latency)
        {"name": "packed_small", "op": "packed", "B": 8, "T": 700, "ctx": 0, "H": 16, "Hkv": 4, "d": 128, "causal": True,
         "window": 0, "sink": False, "spread": 0.8},
        # a prefill batch of eight prompts, 16,384 tokens in all
        {"name": "packed_16k", "op": "packed", "B": 8, "T": 16384, "ctx": 0, "H": 32, "Hkv": 8, "d": 128, "causal": True,
         "window": 0, "sink": False, "spread": 0.8},
        # images of different sizes through one ViT layer, each patch over its own image
        {"name": "packed_vit16384", "op": "packed", "B": 12, "T": 16384, "ctx": 0, "H": 16, "Hkv": 16, "d": 80, "causal": False,
         "window": 0, "sink": False, "spread": 0.8},
        # the next 512 tokens or so of eight prompts behind what they have cached, sink logits
        {"name": "packed_chunk", "op": "packed", "B": 8, "T": 4096, "ctx": 32768, "H": 32, "Hkv": 8, "d": 128, "causal": True,
         "window": 0, "sink": True, "spread": 0.3},
    ]


HEADS = ((4, 4), (8, 2), (16, 4), (32, 8), (8, 1), (6, 2), (32, 4), (5, 1), (12, 1), (16, 1))


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "read", "paged", "paged", "packed", "packed"))
    H, Hkv = rng.choice(HEADS)
    d, page, e4m3 = rng.choice((64, 128, 256)), rng.choice((16, 32, 48, 64, 128)), rng.random() < 0.6
    if op in ("write", "read"):
        B = _log(rng, 1, 128)
        T = B if op == "write" and rng.random() < 0.4 else _log(rng, B, 32768)
        while T * Hkv * d > 32768 * 8 * 128:
            T = T // 2 + 1
        return {"op": op, "B": min(B, T), "T": T, "Hkv": Hkv, "d": d, "page": page, "e4m3": e4m3,
                "far": rng.choice((0, 1, 1000, 4096))}
    if op == "paged":
        B, L = _log(rng, 1, 128), _log(rng, 1, 131072)
        while B * Hkv * L * d > 16 * 8 * 32768 * 128:
            L = L // 2 + 1
        window = _log(rng, 1, 8192) if rng.random() < 0.3 else 0
        return {"op": op, "B": B, "H": H, "Hkv": Hkv, "d": d, "L": L, "page": page, "e4m3": e4m3, "sink": rng.random() < 0.4,
                "window": window, "first": rng.choice((0, 4, 100)) if window else 0}
    causal = rng.random() < 0.7
    B, T, spread = _log(rng, 1, 48), _log(rng, 1, 16384), rng.choice((0.0, 0.5, 0.9))
    c = {"op": op, "B": min(B, T), "T": T, "ctx": 0, "H": H, "Hkv": Hkv, "d": rng.choice((64, 80, 96, 128)), "causal": causal,
         "window": _log(rng, 1, 4096) if causal and rng.random() < 0.4 else 0, "sink": rng.random() < 0.4, "spread": spread}
    if rng.random() < 0.4:
        c["ctx"] = _log(rng, 1, 32768)
    top = _padded(listed()[9])
    while _padded(c) > top:  # no more work than the largest listed case, padded out as the plain form has it
        c["T"], c["ctx"] = c["T"] // 2 + 1, c["ctx"] // 2
        c["B"] = min(c["B"], c["T"])
    return c


def _lengths(B, T, spread, salt):
    """B lengths of T tokens in all: T / B each, give or take `spread` of it; from four on, one of them is of one token."""
    r = random.Random(1000003 * B + 101 * T + salt)
    w = [1 + spread * r.uniform(-1, 1) for _ in range(B)]
    if B >= 4:
        w[1] = 0.0
    n = [int(T * x / sum(w)) for x in w]
    if B >= 4:
        n[1] = 1
    n[0] += T - sum(n)
    return n if n[0] >= 0 else [T] + [0] * (B - 1)


def _packed_lengths(c):
    """Query rows and keys of each sequence."""
    nq = _lengths(c["B"], c["T"], c["spread"], 1)
    ctx = _lengths(c["B"], c["ctx"], c["spread"], 2) if c["ctx"] else [0] * c["B"]
    return nq, [a + b for a, b in zip(nq, ctx)]


def _padded(c):
    nq, nk = _packed_lengths(c)
    return c["B"] * c["H"] * max(nq) * max(nk) * c["d"]


# ------------------------------------------------------------------ the inputs
def _ceil(a, b):
    return -(-a // b)


def _ends(n, dev):
    return torch.nn.functional.pad(n.cumsum(0), (1, 0)).to(torch.int32).to(dev)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEVICE).manual_seed(int(seed) * 7919 + 17)
    r = random.Random(int(seed))

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(shape, generator=g, device=DEVICE, dtype=dtype)

    s = {"c": c}
    if c["op"] == "packed":
        B, T, H, Hkv, d = (c[x] for x in ("B", "T", "H", "Hkv", "d"))
        order = r.sample(range(B), B)
        nq, nk = _packed_lengths(c)
        s["nq"], s["nk"] = [nq[i] for i in order], [nk[i] for i in order]
        s["cu"] = _ends(torch.tensor(s["nq"]), DEVICE)
        s["cu_k"] = _ends(torch.tensor(s["nk"]), DEVICE) if c["ctx"] else None
        if c["ctx"]:
            s["q"], s["k"], s["v"] = normal(T, H, d), normal(sum(nk), Hkv, d), normal(sum(nk), Hkv, d)
        else:  # the projection's output, heads side by side
            qkv = normal(T, H + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H : H + Hkv], qkv[:, H + Hkv :]
        s["sink"] = normal(H, dtype=torch.float32) if c["sink"] else None
        s["o"] = torch.empty((T, H, d), device=DEVICE, dtype=torch.bfloat16)
        s["lse"] = torch.empty((H, T), device=DEVICE, dtype=torch.float32)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["work"] = mattn.attention_packed_workspace(T, B, H, device=DEVICE)
        return s
    B, Hkv, d, page = (c[x] for x in ("B", "Hkv", "d", "page"))
    if c["op"] == "paged":
        s["lens"] = torch.randint(c["L"] // 2, c["L"] + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32)
        s["lens"][0] = c["L"]
        slots = _ceil(c["L"], page)
    else:
        n = _lengths(B, c["T"], 0.8, 3) if c["T"] > B else [1] * B
        s["n"] = r.sample(n, B)
        s["cu"] = _ends(torch.tensor(s["n"]), DEVICE)
        s["starts"] = torch.randint(0, c["far"] + 1, (B,), generator=g, device=DEVICE, dtype=torch.int32)
        slots = _ceil(max(n) + c["far"], page)
    # pages in no order, some of them another request's
    pages = B * slots + 3
    s["table"] = torch.randperm(pages, generator=g, device=DEVICE)[: B * slots].view(B, slots).to(torch.int32)
    s["k_pages"], s["v_pages"] = normal(pages, Hkv, page, d), normal(pages, Hkv, page, d)
    s["k_exp"] = s["v_exp"] = None
    if c["e4m3"]:
        s["k_pages"], s["v_pages"] = (64 * s["k_pages"]).to(CODES), (64 * s["v_pages"]).to(CODES)
        s["k_exp"], s["v_exp"] = (torch.randint(120, 123, (pages, Hkv, page), generator=g, device=DEVICE, dtype=torch.uint8)
                                  for _ in range(2))
    if c["op"] == "write":
        rows = normal(c["T"], 2 * Hkv, d) * torch.exp2(2 * normal(c["T"], 2 * Hkv, 1))  # rows of different size
        s["k"], s["v"] = rows[:, :Hkv], rows[:, Hkv:]
    elif c["op"] == "read":
        s["k"], s["v"] = (torch.empty((c["T"], Hkv, d), device=DEVICE, dtype=torch.bfloat16) for _ in range(2))
    else:
        H = c["H"]
        s["q"] = normal(B, H, d)
        s["sink"] = normal(H, dtype=torch.float32) if c["sink"] else None
        s["o"] = torch.empty((B, H, d), device=DEVICE, dtype=torch.bfloat16)
        s["lse"] = torch.empty((B, H), device=DEVICE, dtype=torch.float32)
        if own:
            import block_sparse_attention_masked_gb300 as mattn

            s["work"] = mattn.decode_paged_workspace(B, H, Hkv, slots, page, d, e4m3=c["e4m3"], device=DEVICE)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        return _own(s)
    return {"write": _write, "read": _read, "paged": _paged, "packed": _packed}[s["c"]["op"]](s)


def _own(s):
    import block_sparse_attention_masked_gb300 as mattn

    c = s["c"]
    if c["op"] == "write":
        mattn.cache_write(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], cu_seqlens=s["cu"], starts=s["starts"],
                          k_exponents=s["k_exp"], v_exponents=s["v_exp"])
        return s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"]
    if c["op"] == "read":
        return mattn.cache_read(s["k_pages"], s["v_pages"], s["table"], s["cu"], starts=s["starts"], k_exponents=s["k_exp"],
                                v_exponents=s["v_exp"], k_out=s["k"], v_out=s["v"])
    if c["op"] == "paged":
        return mattn.decode_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], k_exponents=s["k_exp"],
                                  v_exponents=s["v_exp"], window=c["window"] or None, sink_tokens=c["first"], sink=s["sink"],
                                  out=s["o"], lse=s["lse"], workspace=s["work"])
    return mattn.attention_packed(s["q"], s["k"], s["v"], s["cu"], cu_seqlens_k=s["cu_k"], causal=c["causal"],
                                  window=c["window"] or None, sink=s["sink"], out=s["o"], lse=s["lse"], workspace=s["work"])


def _two_to(e):
    """2^(e - 127) in 32 bits, by its bits (e: 0 .. 254)."""
    return torch.where(e == 0, torch.full_like(e, 1 << 22), e << 23).view(torch.float32)


def _codes(x):
    """Rows x [.., d] in 32 bits as codes and exponents: the least power of two that leaves no value above e4m3's 448."""
    top = x.abs().amax(dim=-1, keepdim=True)
    m, e = torch.frexp(top)  # top = m 2^e, 1/2 <= m < 1
    e = torch.where(top > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, -127)).clamp(min=-127)
    return (x * _two_to(127 - e)).to(CODES), (e + 127)[..., 0].to(torch.uint8)


def _places(s):
    """Sequence, position, page and place in it of every packed row."""
    c = s["c"]
    t = torch.arange(c["T"], device=s["cu"].device)
    b = torch.searchsorted(s["cu"][1:].contiguous(), t, right=True)
    pos = s["starts"].long()[b] + t - s["cu"].long()[b]
    return s["table"].long()[b, pos // c["page"]], pos % c["page"]


def _bytes(x):
    return x.view(torch.uint8) if x.dtype == CODES else x


def _write(s):
    page, at = _places(s)
    if s["c"]["e4m3"]:
        (k, ek), (v, ev) = _codes(s["k"].float()), _codes(s["v"].float())
        s["k_exp"][page, :, at], s["v_exp"][page, :, at] = ek, ev
    else:
        k, v = s["k"], s["v"]
    _bytes(s["k_pages"])[page, :, at], _bytes(s["v_pages"])[page, :, at] = _bytes(k), _bytes(v)
    return s["k_pages"], s["v_pages"], s["k_exp"], s["v_exp"]


def _values(pages, exponents, at):
    """Rows `at` of a cache in 32 bits."""
    x = _bytes(pages)[at]
    if exponents is None:
        return x.float()
    return x.view(CODES).float() * _two_to(exponents[at].int())[..., None]


def _read(s):
    page, at = _places(s)
    index = (page, slice(None), at)
    s["k"].copy_(_values(s["k_pages"], s["k_exp"], index))
    s["v"].copy_(_values(s["v_pages"], s["v_exp"], index))
    return s["k"], s["v"]


def _softmax_sum(x, values, sink):
    """sum_j softmax(x)_j values_j and the log of the normaliser, which `sink` joins; x [.., J] is used up, values [.., J, d]."""
    m = x.amax(dim=-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    x.sub_(m).exp_()
    z = x.sum(dim=-1, keepdim=True)
    if sink is not None:
        z = z + torch.exp(sink - m)
    o = torch.matmul(x, values) / torch.where(z > 0, z, torch.ones_like(z))
    return o, (m + torch.log(z)).squeeze(-1)


def _paged(s):
    c = s["c"]
    B, H, Hkv, d, page = (c[x] for x in ("B", "H", "Hkv", "d", "page"))
    G, slots = H // Hkv, s["table"].shape[1]
    keys, values = (_values(p, e, s["table"].long()).transpose(1, 2).reshape(B, Hkv, slots * page, d)
                    for p, e in ((s["k_pages"], s["k_exp"]), (s["v_pages"], s["v_exp"])))
    x = torch.matmul(s["q"].float().view(B, Hkv, G, d) / math.sqrt(d), keys.transpose(2, 3))
    j, n = torch.arange(slots * page, device=x.device), s["lens"].long()[:, None]
    seen = j < n
    if c["window"]:
        seen = seen & ((j >= n - c["window"]) | (j < c["first"]))
    x = torch.where(seen[:, None, None], x, torch.full_like(x, -math.inf))
    o, lse = _softmax_sum(x, values, s["sink"].view(1, Hkv, G, 1) if c["sink"] else None)
    return o.reshape(B, H, d).to(torch.bfloat16), lse.reshape(B, H)


def _packed(s):
    c = s["c"]
    B, T, H, Hkv, d = (c[x] for x in ("B", "T", "H", "Hkv", "d"))
    dev, G, mq, mk = s["q"].device, H // Hkv, max(s["nq"]), max(s["nk"])
    cq = s["cu"].long()
    ck = s["cu_k"].long() if c["ctx"] else cq
    nq, nk = cq.diff()[:, None, None], ck.diff()[:, None, None]
    i, j = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    q = s["q"][(cq[:-1, None] + i).clamp(max=T - 1)].float() / math.sqrt(d)  # [B, mq, H, d]
    at = (ck[:-1, None] + j).clamp(max=s["k"].shape[0] - 1)
    k, v = s["k"][at].float().transpose(1, 2), s["v"][at].float().transpose(1, 2)  # [B, Hkv, mk, d]
    q = q.view(B, mq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * mq, d)
    x = torch.matmul(q, k.transpose(2, 3)).view(B, Hkv, G, mq, mk)
    hidden = j >= nk
    if c["causal"]:  # the last query sees the last key
        last = i[:, None] + nk - nq
        hidden = hidden | (j > last)
        if c["window"]:
            hidden = hidden | (j <= last - c["window"])
    x.masked_fill_(hidden.expand(B, mq, mk)[:, None, None], -math.inf)
    sink = s["sink"].view(1, Hkv, G, 1, 1) if c["sink"] else None
    o, lse = _softmax_sum(x, v[:, :, None], sink)  # [B, Hkv, G, mq, d]
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(cq[1:].contiguous(), t, right=True)
    t = t - cq[b]
    s["o"].copy_(o.permute(0, 3, 1, 2, 4).reshape(B, mq, H, d)[b, t])
    s["lse"].copy_(lse.reshape(B, H, mq).transpose(1, 2)[b, t].t())
    return s["o"], s["lse"]


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["op"] == "packed":
        nq, nk = _packed_lengths(c)
        pairs = 0
        for a, b in zip(nq, nk):
            if not c["causal"]:
                pairs += a * b
            else:
                w = c["window"] or b
                pairs += sum(min(w, b - a + i + 1) for i in range(a))
        return {"bytes": 4 * c["d"] * (c["T"] * c["H"] + sum(nk) * c["Hkv"]) + 4 * c["T"] * c["H"],
                "flops": 4 * c["d"] * c["H"] * max(1, pairs)}
    cell = c["d"] + 1 if c["e4m3"] else 2 * c["d"]  # bytes of a cached row
    if c["op"] == "paged":
        n = 3 * c["L"] / 4
        if c["window"]:
            n = min(n, c["window"] + c["first"])
        return {"bytes": int(2 * c["B"] * c["Hkv"] * n * cell) + 4 * c["B"] * c["H"] * (c["d"] + 1),
                "flops": int(4 * c["d"] * c["B"] * c["H"] * max(1, n))}
    return {"bytes": 2 * c["T"] * c["Hkv"] * (2 * c["d"] + cell), "flops": 4 * c["T"] * c["Hkv"] * c["d"]}


# ------------------------------------------------------------------ the same in 64 bits
def exact(case, seed):
    """What run() returns for these inputs, from the definitions, sequence by sequence in 64 bits."""
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "packed":
        return _exact_packed(s)
    held = [_held(s["k_pages"], s["k_exp"]), _held(s["v_pages"], s["v_exp"])]
    if c["op"] == "paged":
        return _exact_paged(s, held)
    pages = [s["k_pages"].double(), s["v_pages"].double()]
    out = [torch.zeros(s["k"].shape, dtype=torch.float64, device=DEVICE) for _ in range(2)]
    t = 0
    for b, (n, start) in enumerate(zip(s["n"], s["starts"].tolist())):
        pos = torch.arange(start, start + n, device=DEVICE)
        page, at = s["table"][b].long()[pos // c["page"]], pos % c["page"]
        for i, name in enumerate("kv"):
            if c["op"] == "read":
                out[i][t : t + n] = held[i][page, :, at]
            else:
                x = s[name][t : t + n].double()
                if c["e4m3"]:
                    top = x.abs().amax(dim=-1, keepdim=True)
                    e = torch.round(torch.log2(top / 448))
                    x = x / _power(e + (448 * _power(e) < top).double() - (224 * _power(e) >= top).double())
                    step = _power(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6)) + 1e-9) - 3)  # of e4m3 at x
                    x = torch.round(x / step) * step
                pages[i][page, :, at] = x
        t += n
    return tuple(out) if c["op"] == "read" else (pages[0], pages[1], None, None)


def _power(e):
    """2^e in 64 bits: the library's exp2 and log2 may be a bit off, which would move whole rows."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _held(pages, exponents):
    return pages.double() if exponents is None else pages.double() * _power(exponents.double() - 127)[..., None]


def _attend(q, keys, values, sink, hidden):
    x = q @ keys.T * q.shape[-1] ** -0.5
    if hidden is not None:
        x[hidden] = -math.inf
    if sink is not None:  # one more logit without a value row
        x = torch.cat((x, sink.double().expand(x.shape[0], 1)), dim=1)
        values = torch.cat((values, torch.zeros_like(values[:1])))
    lse = torch.logsumexp(x, dim=1)
    return torch.exp(x - lse.clamp(min=-1e300)[:, None]) @ values, lse


def _exact_paged(s, held):
    c = s["c"]
    B, H, Hkv, d = (c[x] for x in ("B", "H", "Hkv", "d"))
    o = torch.zeros((B, H, d), dtype=torch.float64, device=DEVICE)
    lse = torch.zeros((B, H), dtype=torch.float64, device=DEVICE)
    for b, n in enumerate(s["lens"].tolist()):
        at = list(range(n))
        if c["window"]:
            w = max(0, n - c["window"])
            at = at[: min(c["first"], w)] + at[w:]
        at = torch.tensor(at, dtype=torch.int64, device=DEVICE)
        page, at = s["table"][b].long()[at // c["page"]], at % c["page"]
        for h in range(H):
            keys, values = (x[page, h // (H // Hkv), at] for x in held)
            sink = s["sink"][h] if c["sink"] else None
            o[b, h], lse[b, h] = (x[0] for x in _attend(s["q"][b, h : h + 1].double(), keys, values, sink, None))
    return o, lse


def _exact_packed(s):
    c = s["c"]
    H, G = c["H"], c["H"] // c["Hkv"]
    o = torch.zeros(s["o"].shape, dtype=torch.float64, device=DEVICE)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEVICE)
    i0 = j0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        hidden = None
        if c["causal"]:
            past = torch.arange(nk - nq, nk, device=DEVICE)[:, None] - torch.arange(nk, device=DEVICE)  # a key's age
            hidden = (past < 0) | (past >= (c["window"] or 1 << 40))
        for h in range(H):
            keys, values = (s[x][j0 : j0 + nk, h // G].double() for x in "kv")
            sink = s["sink"][h] if c["sink"] else None
            o[i0 : i0 + nq, h], lse[h, i0 : i0 + nq] = _attend(s["q"][i0 : i0 + nq, h].double(), keys, values, sink, hidden)
        i0, j0 = i0 + nq, j0 + nk
    return o, lse
