"""Cases of the latent-cache and eviction operators, and what each computes in elementary torch operations.

Latent attention keeps one vector of 512 channels and one rotated key of 64 a token instead of keys and values a head.
It is read in two forms: absorbed (queries and outputs in the latent space, over the latents themselves) and expanded
(keys of 128 + 64 and values of 128 a head, made of the latents by the up-projections, then attention over them).
Eviction shrinks a paged cache to the positions that attention has weighed most: the weights are summed a position
over the new rows and heads, and a cache is cut to a budget in place.  With ``own`` set, the same inputs go through
the library's calls.
"""

import math

import torch

own = False

PAGE = 128
LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128
SCALE = (NOPE + ROPE) ** -0.5


# ---------------------------------------------------------------- the cases


def listed():
    return [
        # the first tokens of an answer: one request, one row, all 128 heads, a short cache
        dict(name="latent_one", op="latent_attn", requests=1, rows=1, ctx=1001, heads=128, window=0, sink=False,
             ragged=False, joined=True),
        # a serving batch of single tokens with ragged contexts, an eighth of the heads
        dict(name="latent_batch", op="latent_attn", requests=32, rows=1, ctx=16384, heads=16, window=0, sink=False,
             ragged=True, joined=True),
        # draft and verify rows of all heads over long contexts
        dict(name="latent_long", op="latent_attn", requests=4, rows=2, ctx=131072, heads=128, window=0, sink=False,
             ragged=False, joined=True),
        # chunks of different lengths in one batch, a sliding-window layer with sinks, latents and keys apart
        dict(name="latent_mixed", op="latent_attn", requests=5, rows=333, ctx=12345, heads=32, window=4096, sink=True,
             ragged=True, joined=False),
        # two short ragged prompts made into keys and values of a quarter of the heads
        dict(name="expand_short", op="latent_expand", requests=2, ctx=1500, heads=32, ragged=True, joined=True),
        # a whole prompt of 8192 tokens, all heads
        dict(name="expand_prompt", op="latent_expand", requests=1, ctx=8192, heads=128, ragged=False, joined=True),
        # chunks of different lengths over the expanded caches, an odd number of heads
        dict(name="expanded_mixed", op="expanded_attn", requests=5, rows=511, ctx=2000, heads=20, ragged=True),
        # a whole prompt of 8192 tokens, half of the heads
        dict(name="expanded_prompt", op="expanded_attn", requests=1, rows=8192, ctx=8192, heads=64, ragged=False),
        # a decode step adds its weights: 32 requests, ragged contexts
        dict(name="mass_batch", op="attn_mass", requests=32, rows=1, ctx=16384, heads=64, kv_heads=8, dim=128,
             window=0, decay=1.0, ragged=True),
        # the weights of a prompt of 8192 tokens
        dict(name="mass_prompt", op="attn_mass", requests=1, rows=8192, ctx=8192, heads=32, kv_heads=8, dim=128,
             window=0, decay=0.0, ragged=False),
        # three short caches cut to about half
        dict(name="evict_short", op="kv_evict", requests=3, ctx=2049, budget=1024, first=4, recent=64, kv_heads=8,
             dim=128, latent=False, ragged=True),
        # eight long caches cut to half
        dict(name="evict_long", op="kv_evict", requests=8, ctx=32768, budget=16384, first=4, recent=512, kv_heads=8,
             dim=128, latent=False, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_once(rng):
    op = rng.choice(["latent_attn", "latent_attn", "latent_expand", "expanded_attn", "attn_mass", "kv_evict"])
    if op == "latent_attn":
        rows = 1 if rng.random() < 0.35 else _log(rng, 1, 1024)
        return dict(op=op, requests=_log(rng, 1, 32), rows=rows, ctx=rows + _log(rng, 1, 131072),
                    heads=rng.choice([1, 7, 8, 16, 20, 32, 64, 96, 128]), window=rng.choice([0, 0, 0, 1000, 4096]),
                    sink=rng.random() < 0.5, ragged=rng.random() < 0.5, joined=rng.random() < 0.5)
    if op == "latent_expand":
        return dict(op=op, requests=_log(rng, 1, 8), ctx=_log(rng, 1, 8192), heads=rng.choice([1, 7, 8, 20, 32, 64, 128]),
                    ragged=rng.random() < 0.5, joined=rng.random() < 0.5)
    if op == "expanded_attn":
        rows = _log(rng, 1, 8192)
        return dict(op=op, requests=_log(rng, 1, 8), rows=rows, ctx=rows + _log(rng, 1, 8192),
                    heads=rng.choice([1, 7, 8, 20, 32, 64, 128]), ragged=rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "attn_mass":
        rows = 1 if rng.random() < 0.35 else _log(rng, 1, 4096)
        return dict(op=op, requests=_log(rng, 1, 32), rows=rows, ctx=rows + _log(rng, 1, 65536),
                    heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16]), kv_heads=kv_heads, dim=rng.choice([64, 128]),
                    window=rng.choice([0, 0, 0, 1000, 4096]), decay=rng.choice([0.0, 0.9, 1.0]),
                    ragged=rng.random() < 0.5)
    ctx = _log(rng, 64, 131072)
    latent = rng.random() < 0.3
    budget = max(1, int(ctx * rng.uniform(0.1, 0.95)))
    return dict(op=op, requests=_log(rng, 1, 32), ctx=ctx, budget=budget, first=rng.choice([0, 1, 4]),
                recent=rng.choice([0, 1, budget // 8, budget // 2]), kv_heads=1 if latent else kv_heads,
                dim=LATENT if latent else rng.choice([64, 128]), latent=latent, ragged=rng.random() < 0.5)


def draw(rng):
    top_bytes = max(work(c)["bytes"] for c in listed())
    top_flops = max(work(c)["flops"] for c in listed())
    while True:
        c = _draw_once(rng)
        w = work(c)
        if w["bytes"] > top_bytes or w["flops"] > top_flops:
            continue
        if c["op"] == "kv_evict" and sum(_contexts(c)) * _row_bytes(c) > 2.2e9:
            continue
        if c["op"] in ("latent_attn", "expanded_attn", "attn_mass"):
            # the plain form computes every score, seen or not
            if sum(n * L for n, L in zip(_row_counts(c), _contexts(c))) * c["heads"] > 1.2e10:
                continue
        return c


# ---------------------------------------------------------------- rows of a batch


def _row_counts(c):
    """New rows of each request; a ragged batch has chunks of 1 to ``rows``."""
    n, r = c.get("rows", 1), c["requests"]
    return [max(1, n * (r - i) // r - (i % 3)) if c["ragged"] else n for i in range(r)]


def _contexts(c):
    """Cached positions of each request, its new rows included."""
    n, r = c["ctx"], c["requests"]
    rows = _row_counts(c)
    return [max(rows[i], n * (r + 3 * (r - i)) // (4 * r) - 5 * (i % 7) if c["ragged"] else n) for i in range(r)]


def _budgets(c):
    n, r = c["budget"], c["requests"]
    return [max(1, n - 3 * i) if c["ragged"] else n for i in range(r)]


def _row_bytes(c):
    """Bytes of a cached position, keys and values (or latent and key) together."""
    return 2 * (LATENT + ROPE) if c.get("latent") else 4 * c["kv_heads"] * c["dim"]


def _rows(c):
    """(request, position) of every row, request after request, and each request's length."""
    ctx = _contexts(c)
    req, pos = [], []
    for b, n in enumerate(_row_counts(c)):
        req += [b] * n
        pos += range(ctx[b] - n, ctx[b])
    return req, pos, ctx


def _pairs_keys(c):
    """Pairs of a row and a position that it sees, and positions that some row sees."""
    w = c.get("window") or (1 << 30)
    pairs = keys = 0
    for n, L in zip(_row_counts(c), _contexts(c)):
        p0 = L - n
        full = max(0, min(n, w - p0))  # rows that the window does not cut
        pairs += full * p0 + full * (full + 1) // 2 + (n - full) * w if full else n * min(w, L)
        keys += L - max(0, p0 - w + 1)
    return pairs, keys


def work(c):
    if c["op"] == "latent_expand":
        n, h = sum(_contexts(c)), c["heads"]
        return {"bytes": 2 * n * (LATENT + ROPE) + 2 * h * (NOPE + VALUE) * LATENT + 2 * n * h * (NOPE + ROPE + VALUE),
                "flops": 2 * n * h * (NOPE + VALUE) * LATENT}
    if c["op"] == "kv_evict":
        moved = kept = 0
        for L, k in zip(_contexts(c), _budgets(c)):
            if k < L:
                recent = min(c["recent"], k)  # all of them lie behind the cut, or as many as there is room for
                tail = min(recent, L - k)
                moved += tail + (L - k - tail) * (k - recent) // max(1, L - recent)
            kept += min(k, L)
        return {"bytes": 4 * sum(_contexts(c)) + 12 * kept + 2 * moved * _row_bytes(c), "flops": 4 * sum(_contexts(c))}
    rows, (pairs, keys) = sum(_row_counts(c)), _pairs_keys(c)
    h = c["heads"]
    if c["op"] == "latent_attn":
        return {"bytes": 2 * rows * h * (2 * LATENT + ROPE) + 4 * rows * h + 2 * keys * (LATENT + ROPE) + 8 * rows,
                "flops": 2 * (2 * LATENT + ROPE) * h * pairs}
    if c["op"] == "expanded_attn":
        d = NOPE + ROPE + VALUE
        return {"bytes": 2 * rows * h * d + 4 * rows * h + 2 * keys * h * d + 8 * rows, "flops": 2 * d * h * pairs}
    return {"bytes": 2 * rows * h * c["dim"] + 4 * rows * h + 2 * keys * c["kv_heads"] * c["dim"]
            + 4 * sum(_contexts(c)) * (2 if c["decay"] else 1) + 8 * rows,
            "flops": 2 * c["dim"] * h * pairs + 2 * h * pairs}


# ---------------------------------------------------------------- inputs


def _block_table(ctx, g, dev):
    """Pages in a random order; entries past a request's pages are -1."""
    pages = [-(-n // PAGE) for n in ctx]
    most, total = max(pages), sum(pages)
    order = torch.randperm(total, generator=g, device=dev, dtype=torch.int64).to(torch.int32).cpu()
    table = torch.full((len(ctx), most), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table.to(dev), total


def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.empty(shape, dtype=torch.bfloat16, device=dev).normal_(0, scale, generator=g)

    def empty(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=dev)

    s = {"c": c}
    ctx = _contexts(c)
    s["table"], total = _block_table(ctx, g, dev)
    s["kv_len"] = torch.tensor(ctx, dtype=torch.int32).to(dev)
    if c["op"] in ("latent_attn", "expanded_attn", "attn_mass"):
        req, pos, _ = _rows(c)
        T = len(req)
        s["req"] = torch.tensor(req, dtype=torch.int32).to(dev)
        s["pos"] = torch.tensor(pos, dtype=torch.int32).to(dev)
    if c["op"] in ("latent_attn", "latent_expand"):
        # normed latents beside the rotated key: one row of 576, or two pools
        if c["joined"]:
            pool = normal(total, PAGE, LATENT + ROPE)
            s["c_pool"], s["r_pool"] = pool[..., :LATENT], pool[..., LATENT:]
        else:
            s["c_pool"], s["r_pool"] = normal(total, PAGE, LATENT), normal(total, PAGE, ROPE)
    if c["op"] == "latent_attn":
        # logits of a standard deviation of about two
        s["q"], s["q_rope"] = normal(T, c["heads"], LATENT, scale=1.1), normal(T, c["heads"], ROPE, scale=1.5)
        s["sink"] = torch.randn(c["heads"], generator=g, device=dev) if c["sink"] else None
        s["out"], s["lse"] = empty(T, c["heads"], LATENT), empty(T, c["heads"], dtype=torch.float32)
    elif c["op"] == "latent_expand":
        H = c["heads"]
        # the up-projection as a checkpoint holds it: a head's key rows, then its value rows
        w = normal(H, NOPE + VALUE, LATENT, scale=LATENT ** -0.5)
        s["w_uk"], s["w_uv"] = w[:, :NOPE], w[:, NOPE:]
        s["k_pool"] = torch.zeros((total, PAGE, H, NOPE + ROPE), dtype=torch.bfloat16, device=dev)
        s["v_pool"] = torch.zeros((total, PAGE, H, VALUE), dtype=torch.bfloat16, device=dev)
    elif c["op"] == "expanded_attn":
        H = c["heads"]
        s["q"] = normal(T, H, NOPE + ROPE, scale=1.5)
        s["k_pool"] = normal(total, PAGE, H, NOPE + ROPE, scale=1.3)
        s["v_pool"] = normal(total, PAGE, H, VALUE)
        s["out"], s["lse"] = empty(T, H, VALUE), empty(T, H, dtype=torch.float32)
    elif c["op"] == "attn_mass":
        K, D = c["kv_heads"], c["dim"]
        s["q"] = normal(T, c["heads"], D, scale=1.5)
        s["k_pool"] = normal(total, PAGE, K, D, scale=1.5)
        s["lse"] = empty(T, c["heads"], dtype=torch.float32)
        cols = s["table"].shape[1] * PAGE
        # what earlier steps left
        s["mass"] = torch.empty((len(ctx), cols), device=dev).exponential_(1.0, generator=g)
        s["mass_out"] = torch.zeros((len(ctx), cols), device=dev)
        for b, t, n, h0, h1 in _blocks(c):
            x = _scores(s["q"][t:t + n, h0:h1], _cached(s, s["k_pool"], b), D ** -0.5)
            s["lse"][t:t + n, h0:h1] = _masked(x, s["pos"][t:t + n], c["window"]).logsumexp(-1).t()
    else:
        cols = s["table"].shape[1] * PAGE
        # a few positions hold most of the weight
        s["mass"] = torch.empty((len(ctx), cols), device=dev).normal_(0, 2.0, generator=g).exp_()
        s["budget"] = torch.tensor(_budgets(c), dtype=torch.int32).to(dev)
        if c["latent"]:
            pool = normal(total, PAGE, LATENT + ROPE)
            s["k_pool"], s["v_pool"] = pool[..., None, :LATENT], pool[..., None, LATENT:]
        else:
            s["k_pool"], s["v_pool"] = normal(total, PAGE, c["kv_heads"], c["dim"]), normal(total, PAGE, c["kv_heads"], c["dim"])
        s["kv_len_out"] = torch.zeros_like(s["kv_len"])
        s["mass_out"] = torch.zeros_like(s["mass"])
        s["slot_src"] = torch.full(s["mass"].shape, -1, dtype=torch.int32, device=dev)
    if own:
        s["call"] = _prepared(s)
    return s


# ---------------------------------------------------------------- the library's calls


def _prepared(s):
    """The library's prepared call: arguments checked and marshalled, workspace sized."""
    import prefill_csa_compress_gb300 as csa

    c = s["c"]
    if c["op"] == "latent_attn":
        return csa.csa_latent_attn(
            q=s["q"], q_rope=s["q_rope"], row_req=s["req"], row_pos=s["pos"], c_pool=s["c_pool"], r_pool=s["r_pool"],
            block_table=s["table"], kv_len=s["kv_len"], out=s["out"], lse=s["lse"], sink=s["sink"],
            softmax_scale=SCALE, window=c["window"], prepare=True)
    if c["op"] == "latent_expand":
        return csa.csa_latent_expand(
            c_pool=s["c_pool"], r_pool=s["r_pool"], block_table=s["table"], kv_len=s["kv_len"], w_uk=s["w_uk"],
            w_uv=s["w_uv"], k_pool=s["k_pool"], v_pool=s["v_pool"], out_table=s["table"], prepare=True)
    if c["op"] == "expanded_attn":
        return csa.csa_paged_attn(
            q=s["q"], row_req=s["req"], row_pos=s["pos"], k_pool=s["k_pool"], v_pool=s["v_pool"],
            block_table=s["table"], kv_len=s["kv_len"], out=s["out"], lse=s["lse"], prepare=True)
    if c["op"] == "attn_mass":
        return csa.csa_attn_mass(
            q=s["q"], lse=s["lse"], row_req=s["req"], row_pos=s["pos"], k_pool=s["k_pool"], block_table=s["table"],
            kv_len=s["kv_len"], mass=s["mass"], mass_out=s["mass_out"], decay=c["decay"], window=c["window"],
            prepare=True)
    return csa.csa_kv_evict(
        mass=s["mass"], kv_len=s["kv_len"], budget=s["budget"], kv_len_out=s["kv_len_out"], block_table=s["table"],
        k_pool=s["k_pool"], v_pool=s["v_pool"], first=c["first"], recent=c["recent"], mass_out=s["mass_out"],
        slot_src=s["slot_src"], prepare=True)


# ---------------------------------------------------------------- the plain forms


def _blocks(c):
    """(request, first row, rows, first head, end head): blocks of rows and heads with at most 2^29 scores."""
    t, K = 0, c.get("kv_heads") or c["heads"]
    unit = c["heads"] // K  # heads that share a key head stay together
    for b, (n, L) in enumerate(zip(_row_counts(c), _contexts(c))):
        step = unit * max(1, min(K, (1 << 29) // max(1, n * L * unit)))
        for h0 in range(0, c["heads"], step):
            yield b, t, n, h0, min(c["heads"], h0 + step)
        t += n


def _cached(s, pool, b):
    """Request b's rows of a pool, in order."""
    L = _contexts(s["c"])[b]
    pages = s["table"][b, :-(-L // PAGE)].long()
    return pool[pages].flatten(0, 1)[:L]


def _scores(q, k, scale):
    """q [rows, heads, D] against k [positions, kv_heads, D], heads in groups: [heads, rows, positions] in 32 bits."""
    n, h, d = q.shape
    K = k.shape[1]
    q = q.float().view(n, K, h // K, d).permute(1, 2, 0, 3).reshape(K, h // K * n, d)
    return (torch.matmul(q, k.float().permute(1, 2, 0)) * scale).view(h, n, k.shape[0])


def _masked(x, pos, window):
    p, j = pos.long()[:, None], torch.arange(x.shape[-1], device=x.device)
    seen = j <= p
    if window:
        seen &= j > p - window
    return x.masked_fill_(~seen, -math.inf)


def _softmax(x, sink):
    """Probabilities and the log of the sum [heads, rows, positions]; the sink is in the sum alone."""
    m = x.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink.view(-1, 1, 1))
    x.sub_(m).exp_()
    total = x.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink.view(-1, 1, 1) - m)
    return x.div_(total), (m + total.log()).squeeze(-1)


def _kv_heads_of(c, k, h0, h1):
    g = c["heads"] // c["kv_heads"]
    return k[:, h0 // g:h1 // g]


def run(s):
    c = s["c"]
    if own:
        s["call"]()
    elif c["op"] == "latent_attn":
        last = None
        for b, t, n, h0, h1 in _blocks(c):
            if b != last:
                lat, key = _cached(s, s["c_pool"], b).float(), _cached(s, s["r_pool"], b).float()
                k, last = torch.cat((lat, key), -1)[:, None], b
            q = torch.cat((s["q"][t:t + n, h0:h1], s["q_rope"][t:t + n, h0:h1]), -1)
            x = _masked(_scores(q, k, SCALE), s["pos"][t:t + n], c["window"])
            p, lse = _softmax(x, None if s["sink"] is None else s["sink"][h0:h1])
            s["out"][t:t + n, h0:h1] = torch.matmul(p, lat).transpose(0, 1)
            s["lse"][t:t + n, h0:h1] = lse.t()
    elif c["op"] == "latent_expand":
        w_uk, w_uv = s["w_uk"].float(), s["w_uv"].float()
        for b, L in enumerate(_contexts(c)):
            lat, key = _cached(s, s["c_pool"], b).float(), _cached(s, s["r_pool"], b)
            j = torch.arange(L, device=lat.device)
            page, at = s["table"][b].long()[j // PAGE], j % PAGE
            k = torch.matmul(lat, w_uk.flatten(0, 1).t()).view(L, c["heads"], NOPE).bfloat16()
            s["k_pool"][page, at] = torch.cat((k, key[:, None].expand(-1, c["heads"], -1)), -1)
            s["v_pool"][page, at] = torch.matmul(lat, w_uv.flatten(0, 1).t()).view(L, c["heads"], VALUE).bfloat16()
    elif c["op"] == "expanded_attn":
        last = None
        for b, t, n, h0, h1 in _blocks(c):
            if b != last:
                k, v, last = _cached(s, s["k_pool"], b), _cached(s, s["v_pool"], b), b
            x = _masked(_scores(s["q"][t:t + n, h0:h1], k[:, h0:h1], SCALE), s["pos"][t:t + n], 0)
            p, lse = _softmax(x, None)
            s["out"][t:t + n, h0:h1] = torch.matmul(p, v[:, h0:h1].float().transpose(0, 1)).transpose(0, 1)
            s["lse"][t:t + n, h0:h1] = lse.t()
    elif c["op"] == "attn_mass":
        total = {}
        for b, t, n, h0, h1 in _blocks(c):
            k = _kv_heads_of(c, _cached(s, s["k_pool"], b), h0, h1)
            x = _masked(_scores(s["q"][t:t + n, h0:h1], k, c["dim"] ** -0.5), s["pos"][t:t + n], c["window"])
            w = x.sub_(s["lse"][t:t + n, h0:h1].t()[..., None]).exp_().flatten(0, 1).sum(0)
            total[b] = total[b] + w if b in total else w
        for b, w in total.items():
            n = w.shape[0]
            s["mass_out"][b, :n] = w + c["decay"] * s["mass"][b, :n] if c["decay"] else w
    else:
        for b, (L, most) in enumerate(zip(_contexts(c), _budgets(c))):
            n = min(L, most)
            s["kv_len_out"][b] = n
            key = s["mass"][b, :L].clone()
            key[:c["first"]] = math.inf
            key[max(0, L - c["recent"]):] = math.inf
            kept = torch.zeros(L, dtype=torch.bool, device=key.device)
            kept[key.sort(descending=True, stable=True)[1][:n]] = True
            src = torch.arange(n, device=key.device)
            # kept positions behind the cut go, in order, where evicted ones before it were
            hole = torch.nonzero(~kept[:n])[:, 0]
            src[hole] = torch.nonzero(kept[n:])[:, 0] + n
            s["slot_src"][b, :n] = src.int()
            s["mass_out"][b, :n] = s["mass"][b, src]
            row = s["table"][b].long()
            for name in ("k_pool", "v_pool"):
                pool = s[name]
                pool[row[hole // PAGE], hole % PAGE] = pool[row[src[hole] // PAGE], src[hole] % PAGE]
    return _outputs(s)


def _outputs(s):
    c = s["c"]
    if c["op"] in ("latent_attn", "expanded_attn"):
        return {"out": s["out"], "lse": s["lse"]}
    if c["op"] == "latent_expand":
        return {"k_pool": s["k_pool"], "v_pool": s["v_pool"]}
    if c["op"] == "attn_mass":
        return {"mass": s["mass_out"]}
    return {n: s[n] for n in ("kv_len_out", "mass_out", "slot_src", "k_pool", "v_pool")}


# ---------------------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    global own
    if case["op"] == "kv_evict":
        return None  # a choice and its moves: nothing is computed
    if work(case)["flops"] > 3e12:
        return None  # over 20 seconds
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    c = s["c"]
    if c["op"] == "latent_expand":
        k, v = s["k_pool"].double(), s["v_pool"].double()
        for b, L in enumerate(_contexts(c)):
            for at in range(0, L, PAGE):
                page, n = int(s["table"][b, at // PAGE]), min(PAGE, L - at)
                lat = s["c_pool"][page, :n].double()
                k[page, :n, :, :NOPE] = torch.einsum("jc,hdc->jhd", lat, s["w_uk"].double())
                k[page, :n, :, NOPE:] = s["r_pool"][page, :n, None].double()
                v[page, :n] = torch.einsum("jc,hdc->jhd", lat, s["w_uv"].double())
        return {"k_pool": k, "v_pool": v}
    dev = s["q"].device
    if c["op"] == "attn_mass":
        got = s["mass_out"].double()
        first = 0
        for b, (n, L) in enumerate(zip(_row_counts(c), _contexts(c))):
            hidden = _hidden(s["pos"][first:first + n], L, c["window"])
            w = c["decay"] * s["mass"][b, :L].double()
            for h in range(c["heads"]):
                kh = h * c["kv_heads"] // c["heads"]
                k = _cached(s, s["k_pool"], b)[:, kh].double()
                x = s["q"][first:first + n, h].double() @ k.T / math.sqrt(c["dim"])
                w = w + torch.exp(x - s["lse"][first:first + n, h, None].double()).masked_fill(hidden, 0.0).sum(0)
            got[b, :L] = w
            first += n
        return {"mass": got}
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=dev)
    first = 0
    for b, (n, L) in enumerate(zip(_row_counts(c), _contexts(c))):
        hidden = _hidden(s["pos"][first:first + n], L, c.get("window") or 0)
        if c["op"] == "latent_attn":
            lat, key = _cached(s, s["c_pool"], b).double(), _cached(s, s["r_pool"], b).double()
        else:
            k, v = _cached(s, s["k_pool"], b), _cached(s, s["v_pool"], b)
        for h in range(c["heads"]):
            q = s["q"][first:first + n, h].double()
            if c["op"] == "latent_attn":
                x, val = q @ lat.T + s["q_rope"][first:first + n, h].double() @ key.T, lat
            else:
                x, val = q @ k[:, h].double().T, v[:, h].double()
            x = (x / math.sqrt(NOPE + ROPE)).masked_fill(hidden, -math.inf)
            if s.get("sink") is not None:  # the sink is one more logit, without a value
                x = torch.cat((x, s["sink"][h].double().expand(n, 1)), 1)
            lse[first:first + n, h] = torch.logsumexp(x, 1)
            out[first:first + n, h] = torch.softmax(x, 1)[:, :L] @ val
        first += n
    return {"out": out, "lse": lse}


def _hidden(pos, L, window):
    behind = pos.long()[:, None] - torch.arange(L, device=pos.device)
    return (behind < 0) | (behind >= (window or 1 << 40))
