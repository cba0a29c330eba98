"""Latent attention in both forms, accumulated attention weights and eviction on
the GPU against their float64 definitions (oracle/paged_oracle.py).

Tolerances count roundings, as in test_gpu_paged.py: half a BF16 step is 2^-8 of a
value, probabilities rounded to BF16 move an output by at most 2^-8 sum p |v|, and an
FP32 sum of n products is off by at most n 2^-24 of the sum of their sizes.
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import prefill_csa_compress_gb300 as csa  # noqa: E402

DEV = torch.device("cuda:0")
NAN = float("nan")
H8 = 2.0 ** -8  # half a BF16 step
SCALE = 192 ** -0.5


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16().to(DEV)


def chunk(b, first, n):
    return [(b, first + i) for i in range(n)]


def paged(rng, lens, spare=3):
    """Pages of requests of these lengths in a random order among a few unused
    ones, and how many there are; entries past a request's pages are -1."""
    pages = [-(-n // 128) for n in lens]
    total = sum(pages) + spare
    order = rng.permutation(total)
    table, at = np.full((len(lens), max(max(pages), 1)), -1), 0
    for b, n in enumerate(pages):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def blank_unseen(pools, table, seen):
    """NaN in every row of the pools but the positions `seen` (a set a request)."""
    keep = torch.zeros(pools[0].shape[:2], dtype=torch.bool)
    for b, js in enumerate(seen):
        for j in js:
            if 0 <= table[b, j // 128] < keep.shape[0]:
                keep[table[b, j // 128], j % 128] = True
    for p in pools:
        p[~keep.to(DEV)] = NAN


class Latent:
    def __init__(self, rows, lens, heads, *, causal=True, window=0, sink=False, joined=True,
                 by_head=False, seed=0, scale=1.0):
        rng = np.random.default_rng(seed)
        self.lens, self.kw = np.array(lens), dict(causal=causal, window=window)
        self.req, self.pos = (np.array([r[i] for r in rows]) for i in range(2))
        self.table, total = paged(rng, lens)
        T = len(rows)
        if joined:
            pool = _bf(rng, total, 128, 576)
            self.c, self.r = pool[..., :512], pool[..., 512:]
        else:
            self.c, self.r = _bf(rng, total, 128, 512), _bf(rng, total, 128, 64)
        if by_head:
            self.q, self.qr = (_bf(rng, heads, T, d, scale=scale).transpose(0, 1) for d in (512, 64))
        else:
            q = _bf(rng, T, heads, 576, scale=scale)
            self.q, self.qr = q[..., :512], q[..., 512:]
        self.sink = torch.from_numpy(rng.standard_normal(heads).astype(np.float32)).to(DEV) if sink else None
        seen = [set() for _ in lens]
        for b, p in rows:
            if 0 <= b < len(lens):
                lo, hi = PO.visible(p, min(lens[b], self.table.shape[1] * 128), causal, window)
                seen[b] |= set(range(lo, hi))
        blank_unseen([self.c, self.r], self.table, seen)

    def call(self, **kw):
        T, H, _ = self.q.shape
        out = torch.full((T, H, 512), 77.0, dtype=torch.bfloat16, device=DEV)
        lse = torch.full((T, H), 77.0, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        csa.csa_latent_attn(**{**dict(
            q=self.q, q_rope=self.qr, row_req=_i32(self.req), row_pos=_i32(self.pos), c_pool=self.c,
            r_pool=self.r, block_table=_i32(self.table), kv_len=_i32(self.lens), out=out, lse=lse,
            sink=self.sink, softmax_scale=SCALE, status=st), **self.kw, **kw})
        torch.cuda.synchronize()
        return _np(out), _np(lse), int(st.item())

    def check(self, status=0):
        got, gl, st = self.call()
        assert st == status
        sink = None if self.sink is None else _np(self.sink)
        q, qr, c, r = (_np(x) for x in (self.q, self.qr, self.c, self.r))
        o, ls, spread = PO.latent_attention(q, qr, self.req, self.pos, c, r, self.table, self.lens, SCALE,
                                            sink=sink, **self.kw)
        compare(got, gl, o, ls, spread, (self.req < 0) | (self.req >= len(self.lens)),
                np.abs(q).max() * np.nanmax(np.abs(c)) if np.isfinite(c).any() else 0.0, 576, SCALE,
                int(self.lens.max()))


def compare(got, gl, o, ls, spread, skip, qk, dim, scale, n):
    """out and lse against the definition; rows to skip keep their 77."""
    assert (got[skip] == 77).all() and (gl[skip] == 77).all()
    got, gl, o, ls, spread = (x[~skip] for x in (got, gl, o, ls, spread))
    e = dim * 2.0 ** -24 * qk * dim * scale  # a logit's FP32 sum
    assert np.isfinite(got).all()
    tol = H8 * np.abs(o) + (H8 + 2 * e + 2.0 ** -12) * spread + 1e-30
    assert (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
    none = np.isneginf(ls)
    assert np.array_equal(none, np.isneginf(gl))
    lt = e + (n + 64) * 2.0 ** -24 + 2.0 ** -21 * np.abs(ls[~none]) + 2.0 ** -20
    assert (np.abs(gl[~none] - ls[~none]) <= lt).all(), (np.abs(gl[~none] - ls[~none]) / lt).max()


# ---------------------------------------------------------------- absorbed


@pytest.mark.parametrize("rows,lens", [
    ([(0, 0)], [1]), ([(0, 300)], [301]), (chunk(0, 60, 10), [70]), (chunk(0, 0, 33), [33]),
    ([(0, 63)], [64]), ([(0, 64), (1, 127), (2, 128)], [65, 128, 129]),
    (chunk(0, 250, 7) + [(-1, 0)] + chunk(1, 3, 5) + [(5, 9)] + [(0, 2)], [257, 8]),
    ([(0, 5), (1, 5), (0, 4), (1, 4)], [600, 0])])
@pytest.mark.parametrize("heads", [1, 5, 16, 64, 128])
def test_latent_attention(rows, lens, heads):
    bad = 2 if any(b >= len(lens) for b, _ in rows) else 0
    Latent(rows, lens, heads, seed=heads).check(bad)


@pytest.mark.parametrize("heads", [3, 8, 20, 24, 32, 40, 48, 63, 65, 96, 127])
@pytest.mark.parametrize("joined,by_head", [(True, False), (False, True)])
def test_latent_attention_heads(heads, joined, by_head):
    Latent(chunk(0, 100, 5) + [(1, 200)], [105, 201], heads, joined=joined, by_head=by_head, sink=True,
           seed=heads).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 64, 100, 300])
@pytest.mark.parametrize("sink", [True, False])
def test_latent_attention_masks(causal, window, sink):
    # rows in front of the cache, behind it, and at negative positions
    rows = chunk(0, 200, 6) + [(0, 900), (0, -5), (1, 50), (2, 0), (0, 399), (0, 400)]
    Latent(rows, [400, 31, 0], 12, causal=causal, window=window, sink=sink, seed=window).check()


def test_latent_attention_many_rows():
    """More rows than one list holds: several requests, runs of odd lengths."""
    rows = chunk(0, 0, 301) + chunk(1, 20, 223) + [(-1, 0)] * 5 + chunk(2, 500, 50)
    Latent(rows, [301, 243, 550], 4, seed=4).check()
    Latent(rows, [301, 243, 550], 4, window=90, sink=True, seed=5).check()


def test_latent_attention_long():
    Latent([(0, 40000), (1, 500), (0, 39999), (2, 20000)], [40001, 501, 20001], 16, seed=6).check()
    Latent([(0, 17000)], [17001], 130 - 2, seed=7, window=9000).check()


def test_latent_attention_large_logits():
    """References move: logits of both signs up to some thousands."""
    for scale in (30.0, 300.0):
        b = Latent(chunk(0, 900, 3), [903], 8, seed=8, scale=scale)
        got, gl, st = b.call()
        q, qr, c, r = (_np(x) for x in (b.q, b.qr, b.c, b.r))
        o, ls, _ = PO.latent_attention(q, qr, b.req, b.pos, c, r, b.table, b.lens, SCALE)
        e = 576 * 2.0 ** -24 * np.abs(q).max() * np.nanmax(np.abs(c)) * 576 * SCALE
        assert np.isfinite(got).all() and (np.abs(gl - ls) <= e + 2.0 ** -20 * np.abs(ls)).all()
        if scale == 30.0:
            assert np.abs(got - o).max() <= 0.05 * np.abs(o).max()


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("heads", [8, 64])
def test_latent_attention_hidden_infinities(value, heads):
    rows = chunk(0, 180, 12) + chunk(1, 150, 3)
    b = Latent(rows, [192, 153], heads, seed=9)
    want, wl, _ = b.call()
    at = (int(b.table[0, 1]), 186 - 128)
    b.c[at][7] = value
    b.r[int(b.table[1, 1]), 151 - 128][3] = value
    got, gl, st = b.call()
    assert st == 0
    for t, (r, p) in enumerate(rows):
        if p < (186, 151)[r]:
            assert np.array_equal(got[t], want[t]) and np.array_equal(gl[t], wl[t])
        elif r == 0:
            assert not np.isfinite(got[t, :, 7]).any()


def test_latent_attention_unmapped():
    rows = chunk(0, 300, 4) + [(1, 10)]
    b = Latent(rows, [304, 11], 16, seed=10)
    for entry in (-1, 99999):
        b.table[0, 1] = entry
        b.check(status=1)
    b.table[0, :] = -1
    b.check(status=1)


# ---------------------------------------------------------------- expanded


def _expand_case(rng, lens, heads, joined=True, out_order=None):
    table, total = paged(rng, lens)
    pool = _bf(rng, total, 128, 576)
    c, r = (pool[..., :512], pool[..., 512:]) if joined else (pool[..., :512].contiguous(), pool[..., 512:].contiguous())
    w = _bf(rng, heads, 256, 512, scale=512 ** -0.5)
    return table, total, c, r, w[:, :128], w[:, 128:]


@pytest.mark.parametrize("lens,heads,joined,head_first", [
    ([1], 1, True, False), ([128], 2, True, False), ([129, 0, 127], 3, False, False),
    ([300, 77], 5, True, True), ([1000], 8, False, False), ([260], 20, True, False), ([130], 128, True, False)])
def test_latent_expand(lens, heads, joined, head_first):
    rng = np.random.default_rng(heads)
    table, total, c, r, uk, uv = _expand_case(rng, lens, heads, joined)
    out_table, n_out = paged(rng, lens, spare=2)
    out_table = np.concatenate([out_table, np.full((len(lens), 1), -1)], 1)
    shape = (n_out, heads, 128) if head_first else (n_out, 128, heads)
    k, v = (torch.full(shape + (d,), 77.0, dtype=torch.bfloat16, device=DEV) for d in (192, 128))
    if head_first:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    first = [n // 3 - (n == 1) for n in lens]  # (a negative one counts as 0)
    csa.csa_latent_expand(c_pool=c, r_pool=r, block_table=_i32(table), kv_len=_i32(lens), w_uk=uk, w_uv=uv,
                          k_pool=k, v_pool=v, out_table=_i32(out_table), first=_i32(first), status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    gk, gv, c, r, uk, uv = (_np(x) for x in (k, v, c, r, uk, uv))
    left = np.ones((n_out, 128), dtype=bool)
    for b, n in enumerate(lens):
        j = np.arange(max(0, first[b]), n)
        src, dst = table[b, j // 128], out_table[b, j // 128]
        left[dst, j % 128] = False
        ek, ev = PO.latent_expand(c[src, j % 128], r[src, j % 128], uk, uv)
        # 512 products of a standard deviation of 1 / sqrt(512) each, the sum rounded once
        slack = 512 * 2.0 ** -24 * np.abs(c).max() * np.abs(uk).max() * 16
        for got, want in ((gk[dst, j % 128], ek), (gv[dst, j % 128], ev)):
            assert (np.abs(got - want) <= H8 * np.abs(want) + slack).all()
        assert np.array_equal(gk[dst, j % 128][..., 128:], ek[..., 128:])
    assert (gk[left] == 77).all() and (gv[left] == 77).all()


def test_latent_expand_bad_pages_and_values():
    rng = np.random.default_rng(3)
    table, total, c, r, uk, uv = _expand_case(rng, [400, 300], 3)
    out_table, n_out = paged(rng, [400, 300])
    c[int(table[0, 0]), 5, 9] = NAN
    c[int(table[1, 2]), 300 - 256:] = NAN  # behind the last position
    good = [torch.zeros((n_out, 128, 3, d), dtype=torch.bfloat16, device=DEV) for d in (192, 128)]
    kw = dict(c_pool=c, r_pool=r, kv_len=_i32([400, 300]), w_uk=uk, w_uv=uv)
    csa.csa_latent_expand(block_table=_i32(table), out_table=_i32(out_table), k_pool=good[0], v_pool=good[1], **kw)
    for p in good:
        nan = torch.isnan(p.float()).flatten(2).any(-1)
        assert nan.sum() == 1 and nan[int(out_table[0, 0]), 5]
    for where in range(3):
        t, o = table.copy(), out_table.copy()
        if where == 0:
            t[0, 1] = total
        elif where == 1:
            o[0, 1] = -1
        else:
            o = o[:, :3]  # request 0 has a fourth page, of its last 16 positions
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = [torch.zeros_like(p) for p in good]
        csa.csa_latent_expand(block_table=_i32(t), out_table=_i32(np.ascontiguousarray(o)), k_pool=got[0], v_pool=got[1],
                              status=st, **kw)
        torch.cuda.synchronize()
        assert int(st.item()) == 1
        skipped = int(out_table[0, 3 if where == 2 else 1])
        for p, g in zip(got, good):
            same = torch.eq(p.view(torch.int16), g.view(torch.int16)).flatten(1).all(1)
            assert not same[skipped] and same.sum() == n_out - 1 and not p[skipped].any()


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (7, 7), (20, 20), (12, 4), (32, 1)])
@pytest.mark.parametrize("rows,lens", [
    ([(0, 0)], [1]), (chunk(0, 0, 200), [200]), (chunk(0, 300, 140) + chunk(1, 5, 3) + [(-1, 2), (4, 2)], [440, 8]),
    ([(b, 250 + b) for b in range(6)], [260] * 6), (chunk(0, 120, 9) + chunk(0, 128, 1), [129])])
@pytest.mark.parametrize("window,sink", [(0, False), (70, True)])
def test_expanded_attention(heads, kv_heads, rows, lens, window, sink):
    rng = np.random.default_rng(heads)
    table, total = paged(rng, lens)
    k, v = _bf(rng, total, 128, kv_heads, 192), _bf(rng, total, kv_heads, 128, 128).transpose(1, 2)
    q = _bf(rng, len(rows), heads, 192)
    seen = [set() for _ in lens]
    for b, p in rows:
        if 0 <= b < len(lens):
            seen[b] |= set(range(*PO.visible(p, lens[b], True, window)))
    blank_unseen([k, v], table, seen)
    s = torch.from_numpy(rng.standard_normal(heads).astype(np.float32)).to(DEV) if sink else None
    out = torch.full((len(rows), heads, 128), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(rows), heads), 77.0, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    req, pos = (np.array([r[i] for r in rows]) for i in range(2))
    csa.csa_paged_attn(q=q, row_req=_i32(req), row_pos=_i32(pos), k_pool=k, v_pool=v, block_table=_i32(table),
                       kv_len=_i32(lens), out=out, lse=lse, sink=s, window=window, status=st,
                       mode=csa.CSA_MODE_DECODE if heads == 7 else csa.CSA_MODE_AUTO)
    torch.cuda.synchronize()
    assert int(st.item()) == (2 if (req >= len(lens)).any() else 0)
    o, ls, spread = PO.paged_attention(_np(q), req, pos, _np(k), _np(v), table, lens, SCALE, window=window,
                                       sink=None if s is None else _np(s))
    compare(_np(out), _np(lse), o, ls, spread, (req < 0) | (req >= len(lens)),
            np.abs(_np(q)).max() * np.nanmax(np.abs(_np(k))), 192, SCALE, max(lens))


@pytest.mark.parametrize("value", [float("inf"), NAN])
def test_expanded_attention_hidden_infinities(value):
    rng = np.random.default_rng(1)
    rows, lens, heads = chunk(0, 100, 180), [280], 3
    table, total = paged(rng, lens)
    k, v, q = _bf(rng, total, 128, heads, 192), _bf(rng, total, 128, heads, 128), _bf(rng, 180, heads, 192)
    out = [torch.zeros((180, heads, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for o in out:
        csa.csa_paged_attn(q=q, row_req=_i32([0] * 180), row_pos=_i32(range(100, 280)), k_pool=k, v_pool=v,
                           block_table=_i32(table), kv_len=_i32(lens), out=o)
        v[int(table[0, 1]), 200 - 128] = value
    torch.cuda.synchronize()
    assert torch.equal(out[0][:100], out[1][:100]) and not torch.isfinite(out[1][100:]).any()


def test_both_forms_agree():
    """Publication of latents, then the absorbed form and the expanded one on the
    same cache, against the definition on the published rows."""
    rng = np.random.default_rng(12)
    n, H = 333, 6
    lat, key = _bf(rng, n, 1, 512, scale=3.0), _bf(rng, n, 1, 64)
    gamma = (1 + 0.2 * _bf(rng, 512).float()).bfloat16()
    cos, sin = torch.empty((512, 32), device=DEV), torch.empty((512, 32), device=DEV)
    csa.csa_rope_table(cos=cos, sin=sin)
    table, total = paged(rng, [n])
    pool = torch.full((total, 128, 576), NAN, dtype=torch.bfloat16, device=DEV)
    c, r = pool[..., :512], pool[..., 512:]
    at = dict(row_req=_i32([0] * n), row_pos=_i32(range(n)), block_table=_i32(table))
    csa.csa_kv_append(k=lat, k_pool=c, norm=True, k_gamma=gamma, **at)
    csa.csa_kv_append(k=key, k_pool=r, rope_cos=cos, rope_sin=sin, **at)
    w = _bf(rng, H, 256, 512, scale=512 ** -0.5)
    uk, uv = w[:, :128], w[:, 128:]
    q = _bf(rng, n, H, 192)
    csa.csa_qk_norm_rope(q=q, row_pos=at["row_pos"], norm=False, rope_cos=cos, rope_sin=sin)
    # absorbed
    qa = torch.bmm(q[..., :128].transpose(0, 1), uk).transpose(0, 1)
    lat_out = torch.empty((n, H, 512), dtype=torch.bfloat16, device=DEV)
    lse = [torch.empty((n, H), device=DEV) for _ in range(2)]
    csa.csa_latent_attn(q=qa, q_rope=q[..., 128:], c_pool=c, r_pool=r, kv_len=_i32([n]), out=lat_out, lse=lse[0],
                        softmax_scale=SCALE, **at)
    absorbed = torch.bmm(lat_out.transpose(0, 1), uv.transpose(1, 2)).transpose(0, 1)
    # expanded
    k = torch.empty((total, 128, H, 192), dtype=torch.bfloat16, device=DEV)
    v = torch.empty((total, 128, H, 128), dtype=torch.bfloat16, device=DEV)
    csa.csa_latent_expand(c_pool=c, r_pool=r, block_table=at["block_table"], kv_len=_i32([n]), w_uk=uk, w_uv=uv, k_pool=k,
                          v_pool=v, out_table=at["block_table"])
    out = torch.empty((n, H, 128), dtype=torch.bfloat16, device=DEV)
    csa.csa_paged_attn(q=q, k_pool=k, v_pool=v, kv_len=_i32([n]), out=out, lse=lse[1], **at)
    torch.cuda.synchronize()
    j = np.arange(n)
    ek, ev = PO.latent_expand(_np(c)[table[0, j // 128], j % 128], _np(r)[table[0, j // 128], j % 128], _np(uk), _np(uv))
    pk, pv = np.zeros((2, 384, H, 192))
    pv = np.zeros((384, H, 128))
    pk = np.zeros((384, H, 192))
    pk[:n], pv[:n] = ek, ev
    o, ls, spread = PO.paged_attention(_np(q), [0] * n, j, pk.reshape(3, 128, H, 192), pv.reshape(3, 128, H, 128),
                                       np.array([[0, 1, 2]]), [n], SCALE)
    # a logit is a sum of 192 products, one factor of each rounded to BF16 (absorbed: the query's 512)
    for got, gl, d, size in ((absorbed, lse[0], 512, np.abs(_np(qa)).max() * np.nanmax(np.abs(_np(c)))),
                             (out, lse[1], 128, np.abs(_np(q)).max() * np.abs(ek).max())):
        e = H8 * d ** 0.5 * size * SCALE
        assert (np.abs(_np(gl) - ls) <= e + 1e-4).all()
        tol = (3 * H8 + 2 * e) * spread + 2 * H8 * np.abs(o)
        if d == 512:  # W_uv on rounded latents: 512 products, each off by 2^-8
            tol = tol + 2 * H8 * np.einsum("nhc,hdc->nhd", np.abs(_np(lat_out)), np.abs(_np(uv)))
        assert (np.abs(_np(got) - o) <= tol).all()


# ---------------------------------------------------------------- weights and eviction


class Mass:
    def __init__(self, rows, lens, heads, kv_heads, dim, *, causal=True, window=0, seed=0, head_first=False, cols=0):
        rng = np.random.default_rng(seed)
        self.lens, self.kw = np.array(lens), dict(causal=causal, window=window)
        self.req, self.pos = (np.array([r[i] for r in rows], dtype=int) for i in range(2))
        self.table, total = paged(rng, lens)
        shape = (total, kv_heads, 128, dim) if head_first else (total, 128, kv_heads, dim)
        self.k = _bf(rng, *shape)
        self.k = self.k.transpose(1, 2) if head_first else self.k
        self.q = _bf(rng, len(rows), heads, dim)
        self.lse = torch.from_numpy(rng.normal(2.0, 1.0, (len(rows), heads)).astype(np.float32)).to(DEV)
        self.mass = torch.from_numpy(rng.random((len(lens), self.table.shape[1] * 128)).astype(np.float32)).to(DEV)
        seen = [set() for _ in lens]
        for b, p in rows:
            if 0 <= b < len(lens):
                seen[b] |= set(range(*PO.visible(p, min(lens[b], self.table.shape[1] * 128), causal, window)))
        blank_unseen([self.k], self.table, seen)

    def call(self, **kw):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        csa.csa_attn_mass(**{**dict(
            q=self.q, lse=self.lse, row_req=_i32(self.req), row_pos=_i32(self.pos), k_pool=self.k,
            block_table=_i32(self.table), kv_len=_i32(self.lens), mass=self.mass, status=st), **self.kw, **kw})
        torch.cuda.synchronize()
        return int(st.item())

    def check(self, decay, status=0):
        before = _np(self.mass)
        out = torch.full_like(self.mass, 77.0)
        assert self.call(mass_out=out, decay=decay, **(dict(mass=None) if decay == 0 else {})) == status
        d = self.q.shape[2]
        want = PO.attention_mass(_np(self.q), _np(self.lse), self.req, self.pos, _np(self.k), self.table, self.lens,
                                 d ** -0.5, mass=before, decay=decay, **self.kw)
        # a weight e^x, x a sum of d products less the reference: off by its sum's rounding
        qk = np.abs(_np(self.q)).max(initial=0) * (np.nanmax(np.abs(_np(self.k))) if np.isfinite(_np(self.k)).any() else 0)
        e = 2 * d * 2.0 ** -24 * qk * d ** 0.5 + 2.0 ** -20 * (1 + np.abs(_np(self.lse)).max(initial=0))
        n = self.q.shape[0] * self.q.shape[1]
        for b, w in enumerate(want):
            got = _np(out[b, :len(w)])
            assert (np.abs(got - w) <= (e + (n + 8) * 2.0 ** -24) * w + 1e-30).all(), b
            assert (out[b, len(w):] == 77).all()
        # in place: the same bits
        if decay:
            keep = self.mass.clone()
            assert self.call(decay=decay) == status
            for b, w in enumerate(want):
                assert torch.equal(self.mass[b, :len(w)], out[b, :len(w)])
                assert torch.equal(self.mass[b, len(w):], keep[b, len(w):])


MASS_ROWS = [
    ([(0, 0)], [1]), ([(0, 300)], [301]), (chunk(0, 0, 140), [140]),
    (chunk(0, 250, 7) + [(-1, 0)] + chunk(1, 3, 5) + [(5, 9)] + [(0, 2)], [257, 8]),
    ([(b, 100 + 31 * b) for b in range(9)], [400] * 9), ([(0, 5), (1, 5), (0, 4), (1, 4)], [600, 0])]


@pytest.mark.parametrize("rows,lens", MASS_ROWS)
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (8, 2, 128), (21, 3, 64), (128, 1, 128), (16, 16, 64)])
def test_attention_mass(rows, lens, heads, kv_heads, dim):
    bad = 2 if any(b >= len(lens) for b, _ in rows) else 0
    Mass(rows, lens, heads, kv_heads, dim, seed=heads, head_first=heads == 8).check(1.0, bad)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 100, 300])
@pytest.mark.parametrize("decay", [0.0, 0.5])
def test_attention_mass_masks(causal, window, decay):
    rows = chunk(0, 200, 6) + [(0, 900), (0, -5), (1, 50), (2, 0), (0, 399), (0, 400)]
    Mass(rows, [400, 31, 0], 12, 4, 128, causal=causal, window=window, seed=window).check(decay)


def test_attention_mass_many():
    Mass(chunk(0, 0, 501) + chunk(1, 40, 333), [501, 373], 8, 2, 64, seed=3).check(1.0)
    Mass([(0, 20000), (1, 300)], [20001, 301], 8, 4, 128, seed=4).check(0.25)


def test_attention_mass_special_references():
    """A reference of -inf adds nothing, one of +inf zero, NaN stays NaN; unmapped
    pages are not seen; an unread decay of NaN is left out."""
    b = Mass(chunk(0, 290, 4), [294], 4, 2, 64, seed=5)
    b.lse[1] = float("-inf")
    b.lse[2, 1] = float("inf")
    b.check(0.0)
    b.mass[:] = NAN
    out = torch.zeros_like(b.mass)
    assert b.call(mass_out=out, decay=0.0) == 0 and torch.isfinite(out).all()
    b.lse[0, 0] = NAN
    assert b.call(mass_out=out, decay=0.0) == 0
    assert torch.isnan(out[0, :291]).all() and torch.isfinite(out[0, 291:]).all()
    b = Mass(chunk(0, 290, 4), [294], 4, 2, 64, seed=6)
    b.table[0, 1] = -1
    b.check(0.5, status=1)


def test_attention_mass_without_rows():
    b = Mass([], [200, 3], 4, 2, 64, seed=7)
    b.check(0.5)


def test_attention_mass_sums_to_the_rows():
    """With the attention's own lse and no sink every row and head gives one."""
    b = Mass(chunk(0, 100, 150), [250], 8, 2, 128, seed=8)
    v = torch.randn_like(b.k)
    out = torch.empty_like(b.q)
    b.k[torch.isnan(b.k)] = 0
    csa.csa_paged_attn(q=b.q, row_req=_i32(b.req), row_pos=_i32(b.pos), k_pool=b.k, v_pool=v, block_table=_i32(b.table),
                       kv_len=_i32(b.lens), out=out, lse=b.lse)
    w = torch.zeros_like(b.mass)
    b.call(mass_out=w, decay=0.0)
    assert abs(float(w[0, :250].double().sum()) - 150 * 8) <= 150 * 8 * 2.0 ** -12


def _evict(mass, lens, budget, *, first=0, recent=0, heads=2, kd=64, vd=64, seed=0, in_place=False, layout="token"):
    rng = np.random.default_rng(seed)
    table, total = paged(rng, lens)
    cols = table.shape[1] * 128
    m = torch.full((len(lens), cols), NAN, device=DEV)
    for b, x in enumerate(mass):
        m[b, :lens[b]] = torch.tensor(np.asarray(x, dtype=np.float32)[:lens[b]])
    if layout == "latent":
        pool = _bf(rng, total, 128, kd + vd)
        k, v = pool[..., :kd], pool[..., kd:]
    else:
        k, v = _bf(rng, total, 128, heads, kd), _bf(rng, total, heads, 128, vd).transpose(1, 2)
    k0, v0, m0 = k.clone(), v.clone(), m.clone()
    kv_len = _i32(lens)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    src = torch.full((len(lens), cols), -7, dtype=torch.int32, device=DEV)
    new = kv_len if in_place else torch.full_like(kv_len, -7)
    mo = m if in_place else torch.full_like(m, 77.0)
    csa.csa_kv_evict(mass=m, kv_len=kv_len, budget=_i32(budget), block_table=_i32(table), k_pool=k, v_pool=v,
                     kv_len_out=None if in_place else new, first=first, recent=recent, mass_out=mo, slot_src=src,
                     status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    touched = torch.zeros((total, 128), dtype=torch.bool, device=DEV)
    for b, L in enumerate(lens):
        want = PO.evict(_np(m0[b]), L, budget[b], first, recent)
        n = len(want)
        assert int(new[b]) == n
        assert src[b, :n].tolist() == want and (src[b, n:] == -7).all()
        at, to = np.array(want, dtype=int), np.arange(n)
        rows = [torch.as_tensor(x, device=DEV, dtype=torch.long) for x in
                (table[b, to // 128], to % 128, table[b, at // 128], at % 128)]
        for p, p0 in ((k, k0), (v, v0)):
            assert torch.equal(p[rows[0], rows[1]], p0[rows[2], rows[3]])
        touched[rows[0], rows[1]] = True
        assert torch.equal(mo[b, :n].view(torch.int32), m0[b, rows[2].new_tensor(at)].view(torch.int32))
        rest = m0[b, n:] if in_place else torch.full_like(m0[b, n:], 77.0)
        assert torch.equal(mo[b, n:].view(torch.int32), rest.view(torch.int32))
    for p, p0 in ((k, k0), (v, v0)):
        assert torch.equal(p[~touched], p0[~touched])


@pytest.mark.parametrize("lens,budget", [
    ([1], [1]), ([1], [0]), ([2], [1]), ([300], [100]), ([300, 0, 128, 77], [299, 5, 128, 76]), ([257], [256]),
    ([2049, 1500, 700], [1024, 1021, 699]), ([500, 600], [-3, 10000])])
@pytest.mark.parametrize("first,recent", [(0, 0), (4, 64), (0, 5000), (3000, 7)])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(lens, budget, first, recent, in_place):
    rng = np.random.default_rng(len(lens))
    _evict([np.exp(2 * rng.standard_normal(n)) for n in lens], lens, budget, first=first, recent=recent, in_place=in_place)


def test_evict_ties_and_special_masses():
    n = 1111
    rng = np.random.default_rng(2)
    ties = rng.integers(0, 3, n).astype(float)
    odd = ties.copy()
    odd[rng.random(n) < 0.3] = NAN
    odd[rng.random(n) < 0.1] = float("inf")
    odd[rng.random(n) < 0.1] = -float("inf")
    odd[rng.random(n) < 0.1] = -0.0
    neg = -np.exp(rng.standard_normal(n))
    lens = [n] * 6
    _evict([np.zeros(n), ties, odd, odd, neg, np.full(n, NAN)], lens, [500, 700, 300, 1000, 555, 20])
    _evict([np.zeros(n), ties, odd, odd, neg, np.full(n, NAN)], lens, [500, 700, 300, 1000, 555, 20], first=2, recent=30)


@pytest.mark.parametrize("heads,kd,vd,layout", [(1, 512, 64, "latent"), (1, 8, 24, "token"), (5, 96, 128, "token"),
                                                 (8, 128, 128, "token"), (1, 64, 8, "latent")])
def test_evict_layouts(heads, kd, vd, layout):
    rng = np.random.default_rng(heads)
    lens = [900, 130, 500]
    _evict([rng.random(n) for n in lens], lens, [450, 64, 499], heads=heads, kd=kd, vd=vd, layout=layout, recent=16)


@pytest.mark.parametrize("n,budget", [(40000, 20000), (131072 + 77, 1000), (70001, 70000)])
def test_evict_long(n, budget):
    rng = np.random.default_rng(n)
    _evict([np.exp(2 * rng.standard_normal(n)), rng.random(n - 5)], [n, n - 5], [budget, budget], first=4, recent=512,
           heads=1, kd=8, vd=8)


def test_evict_bad_pages():
    """A move to or from a page outside the pool is not made; the rest is."""
    rng = np.random.default_rng(5)
    lens, n = [640], 300
    table, total = paged(rng, lens)
    mass = torch.from_numpy(rng.random((1, 640)).astype(np.float32)).to(DEV)
    k = _bf(rng, total, 128, 1, 64)
    want = np.array(PO.evict(_np(mass[0]), 640, n))
    for page in (0, 3):
        t = table.copy()
        t[0, page] = total
        got, st = k.clone(), torch.zeros(1, dtype=torch.int32, device=DEV)
        new = _i32([0])
        csa.csa_kv_evict(mass=mass, kv_len=_i32(lens), budget=_i32([n]), block_table=_i32(t), k_pool=got, kv_len_out=new,
                         status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 1 and int(new) == n
        ref = k.clone()
        for d, s in enumerate(want):
            if d != s and d // 128 != page and s // 128 != page:
                ref[table[0, d // 128], d % 128] = k[table[0, s // 128], s % 128]
        assert torch.equal(got, ref)


def test_attention_over_a_cut_cache():
    """A run as it is used: attention, its weights, eviction, attention over the
    kept positions alone."""
    rng = np.random.default_rng(21)
    heads, kvh, dim, lens = 8, 2, 64, [700, 300]
    budget = [256, 299]
    table, total = paged(rng, lens)
    k, v = _bf(rng, total, 128, kvh, dim), _bf(rng, total, 128, kvh, dim)
    k0, v0 = _np(k), _np(v)
    rows = chunk(0, 690, 10) + chunk(1, 299, 1)
    req, pos = (np.array([r[i] for r in rows]) for i in range(2))
    q = _bf(rng, len(rows), heads, dim)
    kv_len, mass = _i32(lens), torch.zeros((2, table.shape[1] * 128), device=DEV)
    out, lse = torch.empty_like(q), torch.empty((len(rows), heads), device=DEV)
    src = torch.zeros(mass.shape, dtype=torch.int32, device=DEV)
    kw = dict(row_req=_i32(req), block_table=_i32(table), kv_len=kv_len)
    csa.csa_paged_attn(q=q, row_pos=_i32(pos), k_pool=k, v_pool=v, out=out, lse=lse, **kw)
    csa.csa_attn_mass(q=q, lse=lse, row_pos=_i32(pos), k_pool=k, mass=mass, **kw)
    weights = mass.clone()
    csa.csa_kv_evict(mass=mass, kv_len=kv_len, budget=_i32(budget), block_table=kw["block_table"], k_pool=k, v_pool=v,
                     recent=32, slot_src=src, mass_out=mass)
    # the next token of each request sees all that was kept
    nxt = _bf(rng, 2, heads, dim)
    out2, lse2 = torch.empty_like(nxt), torch.empty((2, heads), device=DEV)
    csa.csa_paged_attn(q=nxt, row_req=_i32([0, 1]), row_pos=kv_len, k_pool=k, v_pool=v, block_table=kw["block_table"],
                       kv_len=kv_len, out=out2, lse=lse2)
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        kept = np.array(PO.evict(_np(weights[b]), n, budget[b], 0, 32))
        assert src[b, :len(kept)].tolist() == kept.tolist() and int(kv_len[b]) == len(kept)
        x = np.zeros((1, 1, -(-len(kept) // 128) * 128, kvh, dim))
        kk, vv = x[0, 0].copy(), x[0, 0].copy()
        kk[:len(kept)], vv[:len(kept)] = (p[table[b, kept // 128], kept % 128] for p in (k0, v0))
        pages = np.arange(len(kk) // 128)[None]
        o, ls, spread = PO.paged_attention(_np(nxt)[b:b + 1], [0], [len(kept)], kk.reshape(-1, 128, kvh, dim),
                                           vv.reshape(-1, 128, kvh, dim), pages, [len(kept)], dim ** -0.5)
        compare(_np(out2)[b:b + 1], _np(lse2)[b:b + 1], o, ls, spread, np.zeros(1, bool),
                np.abs(_np(nxt)).max() * np.abs(k0).max(), dim, dim ** -0.5, len(kept))
