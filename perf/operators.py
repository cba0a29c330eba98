"""Cases of the operators around the paged caches, and what each computes in elementary torch operations.

The operators are those that feed and read a paged key/value cache: the FP32 RoPE tables, the norms of query and
key heads with the rotation, the publication of new rows into 128-row pages, and the attention of a chunk of new
tokens (or of single tokens) over such a cache.  With ``own`` set, the same inputs go through the library's calls.
"""

import math

import torch

own = False

PAGE = 128
EPS = 1e-6


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # a table for the smallest decode workload: capacity 4096, 64 rotated channels
        dict(name="rope_4k", op="rope_table", n_pos=4096, rope_dim=64, theta=10000.0, scaling="none", factor=1.0,
             orig_len=0),
        # the million-position workload's table, stretched from a 64k training context
        dict(name="rope_million", op="rope_table", n_pos=1048576, rope_dim=64, theta=10000.0, scaling="yarn",
             factor=16.0, orig_len=65536),
        # one decode step: 4 requests x 2 rows, 64 query heads of 512, their last 64 channels rotated
        dict(name="qk_decode", op="qk_norm_rope", rows=8, heads=64, kv_heads=1, dim=512, rope_dim=64,
             layout="adjacent", gamma=False, fused=False),
        # a prefill chunk of a grouped-query layer, q and k taken out of one QKV projection
        dict(name="qk_chunk", op="qk_norm_rope", rows=2047, heads=32, kv_heads=8, dim=128, rope_dim=128,
             layout="half", gamma=True, fused=True),
        # the largest prefill chunk, 64 heads of 512
        dict(name="qk_prefill", op="qk_norm_rope", rows=8192, heads=64, kv_heads=1, dim=512, rope_dim=64,
             layout="adjacent", gamma=True, fused=False),
        # a decode batch publishes one row per request
        dict(name="append_decode", op="kv_append", requests=64, rows=1, ctx=1500, kv_heads=8, dim=128,
             rope_dim=128, layout="half", fmt="bf16", norm=True),
        # a prefill chunk publishes its shared key/value rows in the low-bit window format
        dict(name="append_window", op="kv_append", requests=1, rows=8192, ctx=8192, kv_heads=1, dim=512,
             rope_dim=64, layout="adjacent", fmt="mxfp8", norm=True),
        # the first tokens of an answer: one request, one row, a short cache
        dict(name="attn_one", op="paged_attn", requests=1, rows=1, ctx=1001, heads=32, kv_heads=8, dim=128,
             window=0, sink=False, ragged=False),
        # a serving batch of single tokens with ragged contexts
        dict(name="attn_batch", op="paged_attn", requests=32, rows=1, ctx=16384, heads=64, kv_heads=8, dim=128,
             window=0, sink=True, ragged=True),
        # draft and verify rows over long contexts
        dict(name="attn_long", op="paged_attn", requests=4, rows=2, ctx=131072, heads=64, kv_heads=8, dim=128,
             window=0, sink=True, ragged=False),
        # chunks of different lengths in one batch over a longer cache, a sliding-window layer of narrow heads
        dict(name="attn_mixed", op="paged_attn", requests=5, rows=777, ctx=12345, heads=24, kv_heads=8, dim=64,
             window=4096, sink=True, ragged=True),
        # a whole prompt of 8192 tokens
        dict(name="attn_prefill", op="paged_attn", requests=1, rows=8192, ctx=8192, heads=32, kv_heads=8, dim=128,
             window=0, sink=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_once(rng):
    op = rng.choice(["rope_table", "qk_norm_rope", "kv_append", "paged_attn", "paged_attn"])
    if op == "rope_table":
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op=op, n_pos=_log(rng, 512, 1048576), rope_dim=rng.choice([32, 64, 128]),
                    theta=rng.choice([10000.0, 500000.0]), scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 16.0, 40.0]),
                    orig_len=rng.choice([4096, 8192, 65536]) if scaling == "yarn" else 0)
    if op == "qk_norm_rope":
        dim = rng.choice([64, 96, 128, 256, 512])
        return dict(op=op, rows=_log(rng, 1, 8192), heads=rng.choice([1, 7, 16, 24, 32, 64]),
                    kv_heads=rng.choice([0, 1, 4, 8]), dim=dim, rope_dim=rng.choice([r for r in (32, 64, dim) if r <= dim]),
                    layout=rng.choice(["adjacent", "half"]), gamma=rng.random() < 0.5, fused=rng.random() < 0.5)
    if op == "kv_append":
        fmt = rng.choice(["bf16", "mxfp8"])
        dim = rng.choice([64, 128, 256, 512])
        requests = _log(rng, 1, 64)
        rows = _log(rng, 1, max(1, 8192 // requests))
        return dict(op=op, requests=requests, rows=rows, ctx=rows + _log(rng, 1, 2000),
                    kv_heads=1 if dim == 512 else rng.choice([1, 2, 8]), dim=dim,
                    rope_dim=rng.choice([r for r in (32, 64, dim) if r <= dim]),
                    layout=rng.choice(["adjacent", "half"]), fmt=fmt, norm=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16])
    requests = _log(rng, 1, 32)
    rows = 1 if rng.random() < 0.35 else _log(rng, 1, 4096)
    return dict(op=op, requests=requests, rows=rows, ctx=rows + _log(rng, 1, 131072), heads=heads, kv_heads=kv_heads,
                dim=rng.choice([64, 128]), window=rng.choice([0, 0, 0, 128, 1000, 4096]), sink=rng.random() < 0.5,
                ragged=rng.random() < 0.5)


def draw(rng):
    top_bytes = max(work(c)["bytes"] for c in listed())
    top_flops = max(work(c)["flops"] for c in listed())
    while True:
        c = _draw_once(rng)
        if c["op"] == "paged_attn":
            req, pos, ctx = _rows(c)
            pad = c["requests"] * max(_row_counts(c))
            # the plain form holds every score, and the padded cache, in 32 bits
            if pad * c["heads"] * max(ctx) * 4 > 9e9 or c["requests"] * max(ctx) * c["kv_heads"] * c["dim"] > 6e8:
                continue
        if c["op"] == "kv_append" and c["requests"] * c["ctx"] * c["kv_heads"] * c["dim"] > 1.5e8:
            continue
        w = work(c)
        if w["bytes"] <= top_bytes and w["flops"] <= top_flops:
            return c


# ---------------------------------------------------------------- rows of a batch


def _row_counts(c):
    """New rows of each request; a ragged batch has chunks of 1 to ``rows``."""
    n, r = c["rows"], c["requests"]
    return [max(1, n * (r - i) // r - (i % 3)) if c.get("ragged") else n for i in range(r)]


def _contexts(c):
    """Cached positions of each request, its new rows included."""
    n, r = c["ctx"], c["requests"]
    rows = _row_counts(c)
    return [max(rows[i], n * (r + 3 * (r - i)) // (4 * r) - 5 * (i % 7) if c.get("ragged") else n) for i in range(r)]


def _rows(c):
    """(request, position) of every row, request after request, and each request's length."""
    ctx = _contexts(c)
    req, pos = [], []
    for b, n in enumerate(_row_counts(c)):
        req += [b] * n
        pos += range(ctx[b] - n, ctx[b])
    return req, pos, ctx


def work(c):
    if c["op"] == "rope_table":
        n = c["n_pos"] * c["rope_dim"] // 2
        return {"bytes": 8 * n, "flops": 4 * n}
    if c["op"] == "qk_norm_rope":
        n = c["rows"] * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 4 * n + c["rows"] * (4 * c["rope_dim"] + 4), "flops": 6 * n}
    if c["op"] == "kv_append":
        rows = c["requests"] * c["rows"]
        n = rows * c["kv_heads"] * c["dim"]
        parts = 1 if c["dim"] == 512 else 2
        out = 2 * n if c["fmt"] == "bf16" else n + n // 32
        return {"bytes": parts * (2 * n + out) + rows * (4 * c["rope_dim"] + 8), "flops": 8 * n}
    counts, ctx = _row_counts(c), _contexts(c)
    w = c["window"] or (1 << 30)
    pairs = keys = 0
    for n, L in zip(counts, ctx):
        p0 = L - n
        full = max(0, min(n, w - p0))  # rows that the window does not cut
        pairs += full * p0 + full * (full + 1) // 2 + (n - full) * w if full else n * min(w, L)
        keys += L - max(0, p0 - w + 1)
    rows = sum(counts)
    return {"bytes": 4 * rows * c["heads"] * c["dim"] + 4 * rows * c["heads"] + 4 * keys * c["kv_heads"] * c["dim"] + 8 * rows,
            "flops": 4 * c["dim"] * c["heads"] * pairs}


# ---------------------------------------------------------------- inputs


def _table(n_pos, rope_dim, device):
    """cos and sin of the positions 0 .. n_pos - 1, FP32 [n_pos, rope_dim / 2]."""
    f = 10000.0 ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64, device=device) / rope_dim)
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * f
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).bfloat16()

    s = {"c": c}
    if c["op"] == "rope_table":
        # the seed moves the base a little: another seed is another table
        c["theta"] = c["theta"] * (1.0 + (seed % 9973) * 1e-6)
        s["cos"] = torch.empty((c["n_pos"], c["rope_dim"] // 2), device=dev)
        s["sin"] = torch.empty_like(s["cos"])
    elif c["op"] == "qk_norm_rope":
        T, H, K, D = c["rows"], c["heads"], c["kv_heads"], c["dim"]
        if c["fused"]:  # views of one projection [rows, H + 2 K, D]
            qkv = normal(T, H + 2 * K, D, scale=2.0)
            s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + K]
        else:
            s["q"], s["k"] = normal(T, H, D, scale=2.0), normal(T, K, D, scale=2.0)
        s["q_gamma"] = (1.0 + 0.2 * normal(D).float()).bfloat16() if c["gamma"] else None
        s["k_gamma"] = (1.0 + 0.2 * normal(D).float()).bfloat16() if c["gamma"] else None
        s["cos"], s["sin"] = _table(16384, c["rope_dim"], dev)
        s["pos"] = (torch.arange(T, dtype=torch.int32, device=dev) + (seed % 7919)) % 16384
        s["q_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((T, K, D), dtype=torch.bfloat16, device=dev)
    else:
        req, pos, ctx = _rows(c)
        T, K, D = len(req), c["kv_heads"], c["dim"]
        s["req"] = torch.tensor(req, dtype=torch.int32).to(dev)
        s["pos"] = torch.tensor(pos, dtype=torch.int32).to(dev)
        pages = [-(-n // PAGE) for n in ctx]
        most, total = max(pages), sum(pages)
        order = torch.randperm(total, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu()
        table = torch.full((len(ctx), most), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table.to(dev)
        if c["op"] == "kv_append":
            shape = (total, PAGE, K, D)
            low = c["fmt"] == "mxfp8"
            s["k"] = normal(T, K, D, scale=2.0)
            s["gamma"] = (1.0 + 0.2 * normal(D).float()).bfloat16() if c["norm"] else None
            s["cos"], s["sin"] = _table(max(ctx), c["rope_dim"], dev)
            kind = torch.uint8 if low else torch.bfloat16
            names = ["k"] if D == 512 else ["k", "v"]  # rows of 512 are keys and values at once
            if "v" in names:
                s["v"] = normal(T, K, D)
            for n in names:
                s[n + "_pool"] = torch.zeros(shape, dtype=kind, device=dev)
                if low:
                    s[n + "_scale"] = torch.zeros((total, PAGE, K, D // 32), dtype=torch.uint8, device=dev)
        else:
            s["q"] = normal(T, c["heads"], D, scale=1.5)
            s["k_pool"] = torch.empty((total, PAGE, K, D), dtype=torch.bfloat16, device=dev).normal_(0, 1.5, generator=g)
            s["v_pool"] = torch.empty((total, PAGE, K, D), dtype=torch.bfloat16, device=dev).normal_(0, 1.0, generator=g)
            s["kv_len"] = torch.tensor(ctx, dtype=torch.int32).to(dev)
            # where each request's new rows begin: they end at its last position
            s["first"] = torch.tensor([n - r for n, r in zip(ctx, _row_counts(c))], dtype=torch.int32).to(dev)
            s["sink"] = torch.randn(c["heads"], generator=g, device=dev) if c["sink"] else None
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty((T, c["heads"]), device=dev)
    if own:
        s["call"] = _prepared(s)
    return s


# ---------------------------------------------------------------- the library's calls


def _prepared(s):
    """The library's prepared call: arguments checked and marshalled, workspace sized."""
    import prefill_csa_compress_gb300 as csa

    c = s["c"]
    if c["op"] == "rope_table":
        return csa.csa_rope_table(cos=s["cos"], sin=s["sin"], theta=c["theta"], scaling=c["scaling"], factor=c["factor"],
                                  orig_len=c["orig_len"], prepare=True)
    if c["op"] == "qk_norm_rope":
        return csa.csa_qk_norm_rope(
            q=s["q"], k=s["k"] if c["kv_heads"] else None, q_out=s["q_out"], k_out=s["k_out"] if c["kv_heads"] else None,
            row_pos=s["pos"], q_gamma=s["q_gamma"],
            k_gamma=s["k_gamma"] if c["kv_heads"] else None, eps=EPS, rope_cos=s["cos"], rope_sin=s["sin"],
            rope_layout=c["layout"], prepare=True)
    if c["op"] == "kv_append":
        return csa.csa_kv_append(
            k=s["k"], v=s.get("v"), row_req=s["req"], row_pos=s["pos"], block_table=s["table"], k_pool=s["k_pool"],
            v_pool=s.get("v_pool"), k_scale_pool=s.get("k_scale"), v_scale_pool=s.get("v_scale"), norm=c["norm"],
            k_gamma=s["gamma"], eps=EPS, rope_cos=s["cos"], rope_sin=s["sin"], rope_layout=c["layout"], prepare=True)
    return csa.csa_paged_attn(
        q=s["q"], row_req=s["req"], row_pos=s["pos"], k_pool=s["k_pool"], v_pool=s["v_pool"], block_table=s["table"],
        kv_len=s["kv_len"], out=s["out"], lse=s["lse"], sink=s["sink"], window=c["window"], prepare=True)


# ---------------------------------------------------------------- the plain forms


def _frequencies(c, device):
    """The rotation per position of each channel pair, in 64 bits."""
    d, s = c["rope_dim"], c["factor"]
    i = torch.arange(d // 2, dtype=torch.float64, device=device)
    theta = c["theta"] * s ** (d / (d - 2)) if c["scaling"] == "ntk" else c["theta"]
    f = theta ** (-2.0 * i / d)
    if c["scaling"] == "linear":
        f = f / s
    if c["scaling"] == "yarn":
        # pairs that turn more than 32 times over the original context keep their rotation, those that turn less
        # than once are stretched, a ramp between
        at = [d * math.log(c["orig_len"] / (2 * math.pi * t)) / (2 * math.log(theta)) for t in (32.0, 1.0)]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f * (1 - ramp) + f / s * ramp
    return f


def _rotate(x, cos, sin, layout):
    """The last 2 * cos.shape[-1] channels of x [rows, heads, D] turned; cos, sin [rows, pairs]."""
    n = cos.shape[-1]
    keep, r = x[..., :x.shape[-1] - 2 * n], x[..., x.shape[-1] - 2 * n:]
    cos, sin = cos[:, None], sin[:, None]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "adjacent" else (r[..., :n], r[..., n:])
    u, v = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack((u, v), -1).flatten(-2) if layout == "adjacent" else torch.cat((u, v), -1)
    return torch.cat((keep, turned), -1)


def _norm(x, gamma):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if gamma is None else y * gamma


def _mxfp8(y):
    """E4M3 codes and E8M0 scale bytes of y [..., D]: the smallest 2^e with 448 * 2^e >= amax for every 32."""
    g = y.unflatten(-1, (-1, 32))
    m, k = torch.frexp(g.abs().amax(-1))
    e = torch.where(m > 0, k - 9 + (2 * m > 1.75).int(), torch.full_like(k, -127)).clamp(-127, 127)
    codes = torch.ldexp(g, -e[..., None]).to(torch.float8_e4m3fn).flatten(-2)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def run(s):
    c = s["c"]
    if own:
        s["call"]()
    elif c["op"] == "rope_table":
        a = torch.arange(c["n_pos"], dtype=torch.float64, device=s["cos"].device)[:, None] * _frequencies(c, s["cos"].device)
        s["cos"].copy_(a.cos())
        s["sin"].copy_(a.sin())
    elif c["op"] == "qk_norm_rope":
        p = s["pos"].long()
        cos, sin = s["cos"][p], s["sin"][p]
        q = _norm(s["q"].float(), None if s["q_gamma"] is None else s["q_gamma"].float())
        s["q_out"].copy_(_rotate(q, cos, sin, c["layout"]))
        if c["kv_heads"]:
            k = _norm(s["k"].float(), None if s["k_gamma"] is None else s["k_gamma"].float())
            s["k_out"].copy_(_rotate(k, cos, sin, c["layout"]))
    elif c["op"] == "kv_append":
        p = s["pos"].long()
        phys, at = s["table"][s["req"].long(), p // PAGE].long(), p % PAGE
        k = s["k"].float()
        if c["norm"]:
            k = _norm(k, s["gamma"].float())
        k = _rotate(k, s["cos"][p], s["sin"][p], c["layout"])
        if c["fmt"] == "bf16":
            s["k_pool"][phys, at] = k.bfloat16()
            if "v" in s:
                s["v_pool"][phys, at] = s["v"]
        else:
            s["k_pool"][phys, at], s["k_scale"][phys, at] = _mxfp8(k)
            if "v" in s:
                s["v_pool"][phys, at], s["v_scale"][phys, at] = _mxfp8(s["v"].float())
    else:
        _attend(s)
    return _outputs(s)


def _outputs(s):
    c = s["c"]
    if c["op"] == "rope_table":
        return {"cos": s["cos"], "sin": s["sin"]}
    if c["op"] == "qk_norm_rope":
        return {"q": s["q_out"], "k": s["k_out"]} if c["kv_heads"] else {"q": s["q_out"]}
    if c["op"] == "kv_append":
        if c["fmt"] == "bf16":
            return {n: s[n] for n in ("k_pool", "v_pool") if n in s}
        return ({n: s[n].view(torch.float8_e4m3fn) for n in ("k_pool", "v_pool") if n in s}
                | {n: s[n].view(torch.float8_e8m0fnu) for n in ("k_scale", "v_scale") if n in s})
    return {"out": s["out"], "lse": s["lse"]}


def _attend(s):
    """Softmax attention of every row over the visible positions of its request, heads in groups."""
    c, dev = s["c"], s["q"].device
    K, D = c["kv_heads"], c["dim"]
    G, B = c["heads"] // K, c["requests"]
    req, pos = s["req"].long(), s["pos"].long()
    last = s["kv_len"].long()
    at = pos - s["first"].long()[req]
    n = max(_row_counts(c))
    L = s["table"].shape[1] * PAGE
    tab = s["table"].clamp(min=0).long()
    k = s["k_pool"][tab].view(B, L, K, D).float()
    q = torch.zeros((B, n, K, G, D), device=dev)
    q[req, at] = s["q"].view(-1, K, G, D).float()
    p = torch.full((B, n), -1, dtype=torch.int64, device=dev)
    p[req, at] = pos
    x = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(B, K, G * n, D), k.permute(0, 2, 3, 1)) * D ** -0.5
    del k
    x = x.view(B, K, G, n, L)
    j = torch.arange(L, device=dev)
    seen = (j <= p[..., None]) & (j < last[:, None, None])
    if c["window"]:
        seen &= j > p[..., None] - c["window"]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    if s["sink"] is not None:
        sink = s["sink"].view(1, K, G, 1, 1)
        m = torch.maximum(m, sink)
    m = m.clamp(min=-1e30)  # rows that see nothing
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if s["sink"] is not None:
        total = total + torch.exp(sink - m)
    v = s["v_pool"][tab].view(B, L, K, D).float().permute(0, 2, 1, 3)
    o = torch.matmul(x.view(B, K, G * n, L), v).view(B, K, G, n, D) / total
    lse = (m + total.log()).squeeze(-1)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[req, at].flatten(1, 2))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[req, at].flatten(1, 2))


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["c"]
    if c["op"] == "rope_table":
        d, cos, sin = c["rope_dim"], [], []
        p = torch.arange(c["n_pos"], dtype=torch.float64, device=s["cos"].device)
        for i in range(d // 2):
            f = _one_frequency(c, i)
            cos.append(torch.cos(p * f))
            sin.append(torch.sin(p * f))
        return {"cos": torch.stack(cos, 1), "sin": torch.stack(sin, 1)}
    if c["op"] == "qk_norm_rope":
        turn = s["cos"][s["pos"].long()].double(), s["sin"][s["pos"].long()].double()
        got = {"q": _turned64(_normed64(s["q"], s["q_gamma"]), turn, c["layout"])}
        if c["kv_heads"]:
            got["k"] = _turned64(_normed64(s["k"], s["k_gamma"]), turn, c["layout"])
        return got
    if c["op"] == "kv_append":
        if c["fmt"] != "bf16":
            return None  # codes and their scales: rounded, with no value in 64 bits
        p = s["pos"].long()
        x = _normed64(s["k"], s["gamma"]) if c["norm"] else s["k"].double()
        x = _turned64(x, (s["cos"][p].double(), s["sin"][p].double()), c["layout"])
        got = {}
        for name, y in (("k_pool", x), ("v_pool", s.get("v"))):
            if y is not None:
                pool = s[name].double()
                flat = pool.view(-1, *pool.shape[2:])
                where = s["table"].long()[s["req"].long(), torch.div(p, PAGE, rounding_mode="floor")] * PAGE + p.remainder(PAGE)
                flat[where] = y.double()
                got[name] = pool
        return got
    if work(case)["flops"] > 6e12:
        return None
    return _attended64(s)


def _one_frequency(c, i):
    d, s, kind = c["rope_dim"], c["factor"], c["scaling"]
    base = c["theta"] * (s ** (d / (d - 2.0)) if kind == "ntk" else 1.0)
    f = math.exp(-2.0 * i / d * math.log(base))
    if kind == "linear":
        return f / s
    if kind != "yarn":
        return f

    def pair_of(turns):  # the pair that turns so often over the original context
        return d / 2.0 * math.log(c["orig_len"] / (turns * 2.0 * math.pi)) / math.log(base)

    first, end = max(0, math.floor(pair_of(32.0))), min(d - 1, math.ceil(pair_of(1.0)))
    r = min(1.0, max(0.0, (i - first) / max(end - first, 0.001)))
    return r * (f / s) + (1.0 - r) * f


def _normed64(x, gamma):
    x = x.double()
    y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS)
    return y * gamma.double() if gamma is not None else y


def _turned64(x, turn, layout):
    """Each rotated pair as a complex number times e^(i angle)."""
    z = torch.complex(*turn)[:, None]
    n, D = z.shape[-1], x.shape[-1]
    y = x.clone()
    first = torch.arange(n, device=x.device) * (2 if layout == "adjacent" else 1) + D - 2 * n
    second = first + (1 if layout == "adjacent" else n)
    w = torch.complex(x[..., first], x[..., second]) * z
    y[..., first], y[..., second] = w.real, w.imag
    return y


def _attended64(s):
    c = s["c"]
    G = c["heads"] // c["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=s["q"].device)
    for b, (n, L) in enumerate(zip(_row_counts(c), _contexts(c))):
        t0 = sum(_row_counts(c)[:b])
        pages = s["table"][b, :-(-L // PAGE)].long()
        p = s["pos"][t0:t0 + n].long()[:, None]
        j = torch.arange(L, device=out.device)[None]
        hidden = (j > p) | ((p - j) >= (c["window"] or 1 << 40))
        for h in range(c["kv_heads"]):
            k = s["k_pool"][pages, :, h].reshape(-1, c["dim"])[:L].double()
            v = s["v_pool"][pages, :, h].reshape(-1, c["dim"])[:L].double()
            for i in range(h * G, h * G + G):
                x = (s["q"][t0:t0 + n, i].double() @ k.T) / math.sqrt(c["dim"])
                x = x.masked_fill(hidden, -math.inf)
                if s["sink"] is not None:  # the sink is one more logit, without a value
                    x = torch.cat((x, s["sink"][i].double().expand(n, 1)), 1)
                lse[t0:t0 + n, i] = torch.logsumexp(x, 1)
                out[t0:t0 + n, i] = torch.softmax(x, 1)[:, :L] @ v
    return {"out": out, "lse": lse}
