"""Calls of the latent cache and eviction operators as programs make them: captured
and replayed, on other streams, with workspaces kept, over views of larger pools, with
rows in any order, and the same bits every time."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import prefill_csa_compress_gb300 as csa  # noqa: E402
from test_gpu_cache import DEV, NAN, SCALE, Latent, Mass, _bf, _i32, _np, chunk, compare, paged  # noqa: E402


# ---------------------------------------------------------------- shapes


@pytest.mark.parametrize("heads", [65, 128])
def test_latent_attention_many_rows_of_many_heads(heads):
    """Over 512 rows, two groups of heads, requests of one to seven rows."""
    rng = np.random.default_rng(heads)
    rows, lens = [], []
    while len(rows) < 515:
        n = int(rng.integers(1, 8))
        lens.append(n + int(rng.integers(0, 12)))
        rows += chunk(len(lens) - 1, lens[-1] - n, n)
    rows[17] = (-1, 0)
    rows[300] = (rows[300][0], -3)  # sees nothing
    Latent(rows, lens, heads, seed=heads, sink=heads == 65).check()


def test_latent_attention_single_heads_of_many_requests():
    """64 rows an item, each of another request."""
    lens = [1 + i % 37 for i in range(530)]
    Latent([(i, n - 1) for i, n in enumerate(lens)], lens, 1, seed=3).check()
    Latent([(i, n - 1) for i, n in enumerate(lens[:500])], lens[:500], 2, seed=4).check()


def test_latent_attention_rows_taken_whole():
    """More items than are cut into shares, and more rows."""
    Latent(chunk(0, 5, 2500) + chunk(1, 0, 3), [2505, 3], 33, window=3, seed=8).check()
    Latent(chunk(0, 5, 4200) + chunk(1, 0, 3), [4205, 3], 2, window=2, seed=9, sink=True).check()


def test_latent_attention_rows_in_any_order():
    rows = [(0, 205), (0, 3), (0, 205), (1, 9), (0, 130), (0, 64), (1, 400), (1, 0), (0, 63)]
    Latent(rows, [206, 401], 10, seed=5).check()
    Latent(rows, [206, 401], 10, seed=6, window=66, sink=True).check()


def test_latent_attention_over_a_layered_pool():
    """Pools that are views of one allocation of several layers, q in two buffers."""
    rng = np.random.default_rng(7)
    b = Latent(chunk(0, 150, 3) + [(1, 40)], [153, 41], 6, seed=7)
    pages = b.c.shape[0]
    whole = torch.full((3, pages, 128, 640), float("nan"), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    whole[:, 1, :, 64:576], whole[:, 1, :, 576:] = b.c, b.r
    got = b.call(c_pool=whole[:, 1, :, 64:576], r_pool=whole[:, 1, :, 576:])
    want = b.call()
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    q = torch.full((4, 9, 600), 3.0, dtype=torch.bfloat16, device=DEV)
    q[:, 1:7, 8:584] = torch.cat((b.q, b.qr), -1)
    got = b.call(q=q[:, 1:7, 8:520], q_rope=q[:, 1:7, 520:584])
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    del rng


@pytest.mark.parametrize("requests,rows_each,heads,kv_heads", [(40, 1, 6, 6), (21, 3, 8, 2), (3, 90, 4, 4), (70, 2, 64, 1)])
def test_expanded_attention_of_many_requests(requests, rows_each, heads, kv_heads):
    rng = np.random.default_rng(requests)
    lens = [rows_each + int(rng.integers(0, 300)) for _ in range(requests)]
    rows = [x for b in range(requests) for x in chunk(b, lens[b] - rows_each, rows_each)]
    rows.insert(5, (-1, 0))
    table, total = paged(rng, lens)
    k, v = _bf(rng, total, 128, kv_heads, 192), _bf(rng, total, 128, kv_heads, 128)
    q = _bf(rng, len(rows), heads, 192)
    out = torch.full((len(rows), heads, 128), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(rows), heads), 77.0, device=DEV)
    req, pos = (np.array([r[i] for r in rows]) for i in range(2))
    csa.csa_paged_attn(q=q, row_req=_i32(req), row_pos=_i32(pos), k_pool=k, v_pool=v, block_table=_i32(table),
                       kv_len=_i32(lens), out=out, lse=lse)
    torch.cuda.synchronize()
    o, ls, spread = PO.paged_attention(_np(q), req, pos, _np(k), _np(v), table, lens, SCALE)
    compare(_np(out), _np(lse), o, ls, spread, req < 0, np.abs(_np(q)).max() * np.abs(_np(k)).max(), 192, SCALE, max(lens))


@pytest.mark.parametrize("heads", [1, 3])
def test_latent_expand_of_long_requests(heads):
    """Pages that are written whole beside the first and last ones, odd page counts."""
    rng = np.random.default_rng(heads)
    lens, first = [128 * 3, 128 * 4 + 1, 256], [0, 128, 5]
    table, total = paged(rng, lens)
    pool = _bf(rng, total, 128, 576)
    w = _bf(rng, heads, 256, 512, scale=512 ** -0.5)
    k, v = (torch.full((total, 128, heads, d), 77.0, dtype=torch.bfloat16, device=DEV) for d in (192, 128))
    csa.csa_latent_expand(c_pool=pool[..., :512], r_pool=pool[..., 512:], block_table=_i32(table), kv_len=_i32(lens),
                          w_uk=w[:, :128], w_uv=w[:, 128:], k_pool=k, v_pool=v, out_table=_i32(table), first=_i32(first))
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        j = np.arange(first[b], n)
        at = torch.as_tensor(table[b, j // 128], device=DEV), torch.as_tensor(j % 128, device=DEV)
        c, r = pool[at][:, :512].double(), pool[at][:, 512:]
        assert torch.equal(k[at][..., 128:], r[:, None].expand(-1, heads, -1))
        for got, ww in ((k[at][..., :128], w[:, :128]), (v[at], w[:, 128:])):
            want = torch.einsum("jc,hdc->jhd", c, ww.double())
            slack = 512 * 2.0 ** -24 * 16 * float(c.abs().max() * ww.abs().max())
            assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + slack).all()
        assert (k[int(table[b, 0]), :first[b] % 128 if first[b] < 128 else 128] == 77).all()


# ---------------------------------------------------------------- graphs, streams, workspaces


def _decode_state(seed):
    """A cache that is read, weighed and cut: the calls' arguments."""
    rng = np.random.default_rng(seed)
    lens = [600, 333, 129]
    table, total = paged(rng, lens)
    s = dict(k=_bf(rng, total, 128, 2, 64), v=_bf(rng, total, 128, 2, 64), q=_bf(rng, 3, 8, 64),
             table=_i32(table), kv_len=_i32(lens), req=_i32([0, 1, 2]), pos=_i32([n - 1 for n in lens]),
             mass=torch.from_numpy(rng.random((3, table.shape[1] * 128)).astype(np.float32)).to(DEV))
    s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((3, 8), device=DEV)
    s["budget"] = _i32([300, 300, 64])
    s["src"] = torch.zeros(s["mass"].shape, dtype=torch.int32, device=DEV)
    return s


def _decode_calls(s, **kw):
    at = dict(row_req=s["req"], row_pos=s["pos"], block_table=s["table"], kv_len=s["kv_len"], **kw)
    return [csa.csa_paged_attn(q=s["q"], k_pool=s["k"], v_pool=s["v"], out=s["out"], lse=s["lse"], **at),
            csa.csa_attn_mass(q=s["q"], lse=s["lse"], k_pool=s["k"], mass=s["mass"], decay=0.9, **at),
            csa.csa_kv_evict(mass=s["mass"], kv_len=s["kv_len"], budget=s["budget"], block_table=s["table"],
                             k_pool=s["k"], v_pool=s["v"], first=2, recent=16, mass_out=s["mass"], slot_src=s["src"], **kw)]


def test_decode_run_captured():
    """Attention, weights and eviction in one graph, replayed: what the calls give one
    by one."""
    one, two = _decode_state(1), _decode_state(1)
    start = {n: t.clone() for n, t in two.items()}
    _decode_calls(one)
    calls = _decode_calls(two, prepare=True)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        for c in calls:
            c()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls:
            c()
    for _ in range(2):
        for n, t in two.items():
            t.copy_(start[n])
        g.replay()
        torch.cuda.synchronize()
        for n in ("k", "v", "kv_len", "mass", "src", "out", "lse"):
            assert torch.equal(one[n], two[n]), n
    assert one["kv_len"].tolist() == [300, 300, 64]


@pytest.mark.parametrize("heads,rows", [(16, [(0, 900), (1, 30)]), (128, [(0, 900), (1, 30)]), (8, chunk(0, 300, 601))])
def test_latent_attention_captured(heads, rows):
    """A prepared call captured and replayed on new queries; the workspace kept for a
    later call; the same bits every time."""
    b = Latent(rows, [901, 31], heads, seed=11)
    T = len(rows)
    out, lse = torch.empty((T, heads, 512), dtype=torch.bfloat16, device=DEV), torch.empty((T, heads), device=DEV)
    kw = dict(q=b.q, q_rope=b.qr, row_req=_i32(b.req), row_pos=_i32(b.pos), c_pool=b.c, r_pool=b.r,
              block_table=_i32(b.table), kv_len=_i32(b.lens), softmax_scale=SCALE)
    call = csa.csa_latent_attn(out=out, lse=lse, prepare=True, **kw)
    ws = call()
    first = out.clone(), lse.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    old = b.q.clone()
    b.q.copy_(old.flip(0))
    g.replay()
    torch.cuda.synchronize()
    changed = out.clone()
    b.q.copy_(old)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    assert not torch.equal(changed, first[0])
    ws.fill_(255)
    out.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert csa.csa_latent_attn(out=out, lse=lse, workspace=ws, stream=side, **kw) is ws
    side.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


def test_two_calls_at_once():
    """On two streams, each with a workspace of its own."""
    bs = [Latent(chunk(0, 2000, 2), [2002], 64, seed=20 + i) for i in range(2)]
    want = [b.call()[0] for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    outs, calls = [], []
    for b in bs:
        outs.append(torch.empty((2, 64, 512), dtype=torch.bfloat16, device=DEV))
        calls.append(csa.csa_latent_attn(
            q=b.q, q_rope=b.qr, row_req=_i32(b.req), row_pos=_i32(b.pos), c_pool=b.c, r_pool=b.r, block_table=_i32(b.table),
            kv_len=_i32(b.lens), out=outs[-1], softmax_scale=SCALE, prepare=True))
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert np.array_equal(_np(o), w)


@pytest.mark.parametrize("requests,step,window", [(400, 5, 0), (170, 12, 600)])
def test_attention_mass_of_many_requests(requests, step, window):
    """More pairs of pages than CTAs: several a CTA one after the other, with odd numbers
    of pages, and requests that no row has."""
    lens = [1 + step * b for b in range(requests)]
    rows = [(b, lens[b] - 1) for b in range(requests) if b % 7] + chunk(requests - 1, 0, 40)
    Mass(rows, lens, 4, 2, 64, seed=step, window=window).check(0.5)


@pytest.mark.parametrize("gone", [[0], [1], [2], [0, 1], [1, 2], [0, 1, 2], [4]])
@pytest.mark.parametrize("rows", [1, 80])
def test_attention_mass_unmapped_pages(gone, rows):
    """A page that is not there leaves the other page of its pair as it is."""
    b = Mass(chunk(0, 600 - rows, rows), [600], 8, 2, 128, seed=len(gone))
    b.table[0, gone] = -1
    b.check(0.5, status=1)


@pytest.mark.parametrize("rows,heads,kv_heads,dim", [(1, 8, 1, 128), (1, 8, 2, 64), (16, 8, 1, 128), (17, 8, 1, 64), (3, 21, 3, 64),
                                                     (130, 4, 4, 64)])
def test_attention_mass_infinite_keys(rows, heads, kv_heads, dim):
    """A key that is not finite has its weight by the definition (e^-inf = 0, e^inf,
    NaN), however the rows fill a tile; other positions keep their bits."""
    b = Mass(chunk(0, 400 - rows, rows), [400], heads, kv_heads, dim, seed=rows)
    b.q[..., 3] = -b.q[..., 3].abs() - 0.125  # against an infinite channel: all of one sign
    want, got = torch.zeros_like(b.mass), torch.zeros_like(b.mass)
    b.call(mass_out=want, decay=0.0)
    for j, value in ((5, np.inf), (150, np.inf), (77, -np.inf), (200, NAN)):  # (all rows see them)
        b.k[int(b.table[0, j // 128]), j % 128, :, 3] = value
    b.call(mass_out=got, decay=0.0)
    assert (got[0, [5, 150]] == 0).all() and torch.isposinf(got[0, 77]) and torch.isnan(got[0, 200])
    rest = [j for j in range(400) if j not in (5, 150, 77, 200)]
    assert torch.equal(got[0, rest], want[0, rest])


def test_attention_mass_captured_and_alike():
    b = Mass(chunk(0, 600, 300) + chunk(1, 40, 40), [900, 80], 16, 4, 128, seed=12)
    out = [torch.zeros_like(b.mass) for _ in range(2)]
    assert b.call(mass_out=out[0], decay=0.5) == 0
    call = csa.csa_attn_mass(q=b.q, lse=b.lse, row_req=_i32(b.req), row_pos=_i32(b.pos), k_pool=b.k,
                             block_table=_i32(b.table), kv_len=_i32(b.lens), mass=b.mass, mass_out=out[1], decay=0.5,
                             prepare=True)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for _ in range(3):
        out[1].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], out[1])


def test_attention_mass_in_a_strided_buffer():
    b = Mass(chunk(0, 100, 5) + [(1, 60)], [105, 61], 4, 2, 64, seed=13)
    wide = torch.full((2, 200), 5.0, device=DEV)
    view = wide[:, 20:20 + b.mass.shape[1]]
    want = torch.zeros_like(b.mass)
    b.call(mass_out=want, decay=0.25)
    view.copy_(b.mass)
    assert b.call(mass=view, decay=0.25) == 0
    for r, n in enumerate(b.lens):
        assert torch.equal(view[r, :n], want[r, :n]) and torch.equal(view[r, n:], b.mass[r, n:])
    assert (wide[:, :20] == 5).all() and (wide[:, 20 + b.mass.shape[1]:] == 5).all()


def test_latent_cache_cut():
    """Eviction from a latent cache: one pool of rows of 576, attention before and after."""
    rng = np.random.default_rng(14)
    b = Latent([(0, 499), (1, 199)], [500, 200], 4, seed=14)
    b.c[torch.isnan(b.c)] = 0
    b.r[torch.isnan(b.r)] = 0
    mass = torch.from_numpy(rng.random((2, b.table.shape[1] * 128)).astype(np.float32)).to(DEV)
    c0, r0, lens, budget = _np(b.c), _np(b.r), [500, 200], [130, 199]
    kv_len = _i32(lens)
    csa.csa_kv_evict(mass=mass, kv_len=kv_len, budget=_i32(budget), block_table=_i32(b.table), k_pool=b.c, v_pool=b.r,
                     recent=8)
    out = torch.empty((2, 4, 512), dtype=torch.bfloat16, device=DEV)
    csa.csa_latent_attn(q=b.q, q_rope=b.qr, row_req=_i32([0, 1]), row_pos=kv_len, c_pool=b.c, r_pool=b.r,
                        block_table=_i32(b.table), kv_len=kv_len, out=out, softmax_scale=SCALE)
    torch.cuda.synchronize()
    for r in range(2):
        kept = np.array(PO.evict(_np(mass[r]), lens[r], budget[r], 0, 8))
        at = b.table[r, kept // 128], kept % 128
        pad = -len(kept) % 128
        c, rr = (np.concatenate([p[at], np.zeros((pad, p.shape[-1]))]).reshape(-1, 128, p.shape[-1]) for p in (c0, r0))
        o, _, spread = PO.latent_attention(_np(b.q)[r:r + 1], _np(b.qr)[r:r + 1], [0], [len(kept)], c, rr,
                                           np.arange(len(c))[None], [len(kept)], SCALE)
        e = 576 * 2.0 ** -24 * np.abs(_np(b.q)).max() * np.abs(c0).max() * 576 * SCALE
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -8 + 2 * e + 2.0 ** -12) * spread
        assert (np.abs(_np(out)[r:r + 1] - o) <= tol).all()


def test_weights_through_two_cuts():
    """Attention, weights, eviction, publication, and again: every position's weight is its
    own through two cuts, where the entries behind a cut are cleared before new positions
    are published there."""
    rng = np.random.default_rng(31)
    heads, kvh, dim, decay = 8, 2, 64, 0.75
    lens, budget, new = [520, 300], [250, 200], 3
    table, total = paged(rng, lens)
    k, v = _bf(rng, total, 128, kvh, dim), _bf(rng, total, 128, kvh, dim)
    table_dev, kv_len, mass = _i32(table), _i32(lens), torch.zeros((2, table.shape[1] * 128), device=DEV)
    slots = torch.arange(mass.shape[1], device=DEV)
    want = [np.zeros(n) for n in lens]  # the weight of what each slot holds
    for turn in range(3):
        n = [int(x) for x in kv_len]
        rows = [(b, n[b] - new + i) for b in range(2) for i in range(new)]
        at = dict(row_req=_i32([r for r, _ in rows]), row_pos=_i32([p for _, p in rows]), block_table=table_dev, kv_len=kv_len)
        q = _bf(rng, len(rows), heads, dim)
        out, lse = torch.empty_like(q), torch.empty((len(rows), heads), device=DEV)
        csa.csa_paged_attn(q=q, k_pool=k, v_pool=v, out=out, lse=lse, **at)
        csa.csa_attn_mass(q=q, lse=lse, k_pool=k, mass=mass, decay=decay, **at)
        torch.cuda.synchronize()
        qn, kn, ln = _np(q), _np(k), _np(lse)
        add = PO.attention_mass(qn, ln, [r for r, _ in rows], [p for _, p in rows], kn, table, n, dim ** -0.5)
        # a logit is an FP32 sum of 64 products (64 2^-24 of the sum of their sizes, twice that
        # for sums that are cut off, not rounded), its exponent and the reference are rounded,
        # 24 weights and the decay added each turn
        sizes = max((np.abs(kn[..., h, :]) @ np.abs(qn[:, 4 * h:4 * h + 4].reshape(-1, dim)).T).max() for h in range(kvh))
        e = 2 * 64 * 2.0 ** -24 * sizes / 8 + 2.0 ** -20 * (1 + np.abs(ln).max()) + 32 * 2.0 ** -24
        want = [decay * w + a for w, a in zip(want, add)]
        for b in range(2):
            tol = (turn + 1) * e * want[b]
            assert (np.abs(_np(mass[b, :n[b]]) - want[b]) <= tol).all(), (turn, b)
            if turn:  # (what the entries held behind the cut would show)
                assert (decay * stale[b] > tol[n[b] - new:]).any()
        before = mass.clone()
        csa.csa_kv_evict(mass=mass, mass_out=mass, kv_len=kv_len, budget=_i32(budget), block_table=table_dev, k_pool=k, v_pool=v,
                         first=2, recent=new)
        left = [int(x) for x in kv_len]
        assert left == budget
        for b in range(2):
            assert torch.equal(mass[b, left[b]:], before[b, left[b]:])  # of positions that are gone
            want[b] = want[b][PO.evict(_np(before[b]), n[b], budget[b], 2, new)]
        stale = [_np(before[b, left[b]:left[b] + new]) for b in range(2)]
        mass.masked_fill_(slots >= kv_len[:, None], 0.0)
        # new tokens at the slots behind the cut
        pos = [(b, left[b] + i) for b in range(2) for i in range(new)]
        csa.csa_kv_append(k=_bf(rng, len(pos), kvh, dim), v=_bf(rng, len(pos), kvh, dim), k_pool=k, v_pool=v,
                          row_req=_i32([r for r, _ in pos]), row_pos=_i32([p for _, p in pos]), block_table=table_dev)
        kv_len += new
        want = [np.concatenate([w, np.zeros(new)]) for w in want]

def test_launches_are_counted_and_timed():
    from prefill_csa_compress_gb300 import prof_disable, prof_enable, prof_read

    s = _decode_state(3)
    before = csa.launch_count()
    _decode_calls(s)
    assert csa.launch_count() - before >= 5  # attention, weights, their join or not, choice, moves
    for name in ("attn_mass", "evict_plan", "evict_move"):
        prof_enable(name, 4)
        try:
            _decode_calls(s)
            ms, n = prof_read(name)
            assert n == 1 and ms > 0
        finally:
            prof_disable()
