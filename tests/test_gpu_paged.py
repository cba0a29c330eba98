"""The paged key/value cache operators on the GPU against their float64
definitions (oracle/paged_oracle.py).

Tolerances count roundings.  A BF16 result is off by at most 2^-8 of its value
(half a step) plus what the FP32 arithmetic before it leaves; the attention
also rounds its probabilities to BF16 before the product with the values, which
moves an output by at most 2^-8 sum p |v| (the oracle's ``spread``).
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
DECODE, PREFILL = csa.CSA_MODE_DECODE, csa.CSA_MODE_PREFILL
H8 = 2.0 ** -8  # half a BF16 step


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _bf(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).bfloat16().to(DEV)


def _status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- rope tables


@pytest.mark.parametrize("kw", [
    dict(), dict(theta=500000.0), dict(scaling="linear", factor=4.0),
    dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=40.0, orig_len=4096),
    dict(scaling="yarn", factor=16.0, orig_len=65536, beta_fast=16.0, beta_slow=2.0),
    dict(scaling="yarn", factor=2.0, orig_len=1)])
@pytest.mark.parametrize("n_pos,rope_dim,pos0", [(1, 2 + 2, 0), (333, 64, 0), (100, 6, 1 << 20),
                                                 (65, 512, 131071), (7, 128, 2 ** 31 - 7)])
def test_rope_table(kw, n_pos, rope_dim, pos0):
    cos = torch.full((n_pos + 1, rope_dim // 2), NAN, device=DEV)
    sin = cos.clone()
    amp = 1.25
    csa.csa_rope_table(cos=cos[:n_pos], sin=sin[:n_pos], pos0=pos0, attn_factor=amp, **kw)
    torch.cuda.synchronize()
    assert cos[n_pos:].isnan().all() and sin[n_pos:].isnan().all()
    c, s = PO.rope_table(n_pos, rope_dim, pos0=pos0, attn_factor=amp, **kw)
    # 2e-7: include/csa.h; the definition's own product p * f is off by p * 2^-52 radians
    tol = (2e-7 + (pos0 + n_pos) * 2.0 ** -51) * amp
    assert np.abs(_np(cos[:n_pos]) - c).max() <= tol
    assert np.abs(_np(sin[:n_pos]) - s).max() <= tol


def test_rope_table_unaligned_and_pieces():
    """Any 4-byte aligned destination; a table in pieces equals the whole."""
    whole = torch.empty((2, 301, 5), device=DEV)
    csa.csa_rope_table(cos=whole[0], sin=whole[1])
    flat = torch.full((2, 301 * 5 + 2), NAN, device=DEV)
    c, s = flat[0, 1:-1].view(301, 5), flat[1, 1:-1].view(301, 5)
    csa.csa_rope_table(cos=c[:100], sin=s[:100])
    csa.csa_rope_table(cos=c[100:], sin=s[100:], pos0=100)
    torch.cuda.synchronize()
    assert torch.equal(c, whole[0]) and torch.equal(s, whole[1])
    assert flat[:, 0].isnan().all() and flat[:, -1].isnan().all()


# ---------------------------------------------------------------- norms and rotation


def _close_vec(got, ref, extra=0.0):
    """BF16 vectors [..., D]: half a step of the value, and FP32 arithmetic
    bounded by 2^-16 of the vector's largest value (sums of up to 512 squares
    and five products: under 2^6 roundings of 2^-24, and a pair's rotation
    mixes two channels)."""
    tol = H8 * np.abs(ref) + 2.0 ** -16 * np.abs(ref).max(-1, keepdims=True) + extra
    assert np.isfinite(got).all()
    assert (np.abs(got - ref) <= tol).all(), (np.abs(got - ref) / tol).max()


QK = [  # rows, q heads, k heads, dim, rope_dim, start
    (1, 1, 0, 64, 64, None), (8, 64, 1, 512, 64, None), (3, 5, 2, 128, 128, None),
    (17, 7, 3, 96, 32, 0), (2, 3, 1, 8, 8, None), (5, 2, 2, 80, 16, 32), (9, 1, 1, 320, 320, None),
    (4, 3, 2, 512, 512, None), (6, 2, 1, 264, 208, 16), (700, 3, 1, 128, 64, 64), (3, 2, 1, 16, 16, 0),
    (2, 3, 2, 24, 16, 8), (2, 1, 1, 496, 0, None)]


@pytest.mark.parametrize("layout", ["adjacent", "half"])
@pytest.mark.parametrize("rows,hq,hk,dim,rd,start", QK)
@pytest.mark.parametrize("norm,gamma", [(True, True), (True, False), (False, False)])
def test_qk_norm_rope(layout, rows, hq, hk, dim, rd, start, norm, gamma):
    if layout == "half" and rd % 16:
        rd += 8 if rd + 8 <= dim else -8
        if rd <= 0:
            pytest.skip("no half layout of 8 channels")
    rng = np.random.default_rng(rows + dim)
    q, k = _bf(rng, rows, hq, dim, scale=2), _bf(rng, rows, max(hk, 1), dim, scale=0.5)
    k = k if hk else None
    gq = _bf(rng, dim) if gamma else None
    gk = _bf(rng, dim) if gamma and hk else None
    pos = rng.integers(-1, 200, rows)
    pos[0] = 199
    cos, sin = PO.rope_table(200, rd or 2)
    tabs = dict(rope_cos=torch.from_numpy(cos).float().to(DEV), rope_sin=torch.from_numpy(sin).float().to(DEV),
                rope_layout=layout, rope_start=start) if rd else {}
    qo = torch.full_like(q, NAN)
    ko = torch.full_like(k, NAN) if hk else None
    st = _status()
    csa.csa_qk_norm_rope(q=q, k=k, q_out=qo, k_out=ko, row_pos=_i32(pos), norm=norm, q_gamma=gq, k_gamma=gk,
                         eps=1e-5, status=st, **tabs)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, o, g in ((q, qo, gq), (k, ko, gk)):
        if x is None:
            continue
        ref = PO.norm_rotate(_np(x), pos, norm=norm, gamma=None if g is None else _np(g), eps=1e-5,
                             cos=_np(tabs["rope_cos"]) if rd else None, sin=_np(tabs["rope_sin"]) if rd else None,
                             layout=layout, start=start)
        _close_vec(_np(o), ref)


@pytest.mark.parametrize("layout", ["adjacent", "half"])
@pytest.mark.parametrize("dim", [64, 128, 512])
def test_qk_in_place_of_a_projection(layout, dim):
    """q and k as views of one projection, replaced in place: the same bits as
    into outputs of their own; the values between them stay; padded rows and
    rows past the tables."""
    rng = np.random.default_rng(3)
    T, hq, hk = 37, 4, 2
    qkv = _bf(rng, T, hq + 2 * hk, dim)
    keep = qkv.clone()
    pos = np.arange(T) + 90  # some past the tables' 100 rows
    req = np.where(np.arange(T) % 5 == 3, -1, 0)
    cos, sin = (torch.from_numpy(x).float().to(DEV) for x in PO.rope_table(100, 32))
    kw = dict(row_pos=_i32(pos), row_req=_i32(req), rope_cos=cos, rope_sin=sin, rope_layout=layout)
    qo = torch.full((T, hq, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((T, hk, dim), 5.0, dtype=torch.bfloat16, device=DEV)
    st = _status()
    csa.csa_qk_norm_rope(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], q_out=qo, k_out=ko, status=st, **kw)
    torch.cuda.synchronize()
    assert int(st.item()) == 0x8
    assert torch.equal(qkv, keep)
    csa.csa_qk_norm_rope(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], **kw)
    torch.cuda.synchronize()
    pad = torch.from_numpy(req < 0).to(DEV)
    assert torch.equal(qkv[:, hq + hk:], keep[:, hq + hk:])
    assert torch.equal(qkv[pad], keep[pad]) and (qo[pad] == 5).all() and (ko[pad] == 5).all()
    assert torch.equal(qkv[~pad][:, :hq], qo[~pad]) and torch.equal(qkv[~pad][:, hq:hq + hk], ko[~pad])
    ref = PO.norm_rotate(_np(keep[:, :hq]), pos, cos=_np(cos), sin=_np(sin), layout=layout)
    _close_vec(_np(qo[~pad]), ref[req >= 0])


def test_norm_of_zero_rows_and_large_values():
    q = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device=DEV)
    q[1] = 1e18  # squares up to 1e36 stay inside FP32
    csa.csa_qk_norm_rope(q=q, row_pos=_i32([0, 0]))
    torch.cuda.synchronize()
    assert (q[0] == 0).all() and torch.allclose(q[1].float(), torch.ones(64, device=DEV), rtol=2 * H8)


# ---------------------------------------------------------------- publication


def _pool(n, heads, dim, kind, fill=7.0, dtype=torch.bfloat16):
    """A pool [n, 128, heads, dim] in several memory layouts; also the whole
    allocation."""
    if kind == "dense":
        big = torch.full((n, 128, heads, dim), fill, dtype=dtype, device=DEV)
        return big, big
    if kind == "heads_first":  # [pages, heads, 128, dim]
        big = torch.full((n, heads, 128, dim), fill, dtype=dtype, device=DEV)
        return big.transpose(1, 2), big
    if kind == "beside":  # keys beside values in each row
        big = torch.full((n, 128, 2, heads, dim), fill, dtype=dtype, device=DEV)
        return big[:, :, 1], big
    assert kind == "layers"  # one layer of three, rows padded
    big = torch.full((n, 3, 128, heads, dim + 8), fill, dtype=dtype, device=DEV)
    return big[:, 1, :, :, :dim], big


TABLE = np.array([[3, 0, -1, 9], [1, 4, 2, -7]])  # of 5 blocks: 9, -1, -7 are bad pages
APPEND = [  # request, position: ends of pages, a bad page, past the table, padding, no position
    (0, 0), (0, 127), (0, 128), (0, 255), (0, 256), (0, 300), (0, 400), (0, 512), (-1, 5), (1, -3), (2, 0),
    (1, 0), (1, 383), (1, 130), (1, 129), (1, 128), (7, 9), (0, 60)]


@pytest.mark.parametrize("kind", ["dense", "heads_first", "beside", "layers"])
@pytest.mark.parametrize("heads,dim,with_v", [(2, 128, True), (1, 512, False), (3, 64, True), (1, 8, True),
                                              (2, 264, True)])
def test_append_bf16(kind, heads, dim, with_v):
    rng = np.random.default_rng(heads)
    T = len(APPEND)
    req, pos = np.array(APPEND).T
    src = _bf(rng, T, 2 * heads + 1, dim)  # k and v as views of one projection
    k, v = src[:, :heads], src[:, heads:2 * heads] if with_v else None
    g = _bf(rng, dim)
    rd = min(64, dim)
    cos, sin = (torch.from_numpy(x).float().to(DEV) for x in PO.rope_table(250, rd))
    kp, kbig = _pool(5, heads, dim, kind)
    vp, vbig = _pool(5, heads, dim, kind) if with_v else (None, None)
    k0, v0 = kbig.clone(), vbig.clone() if with_v else None
    st = _status()
    csa.csa_kv_append(k=k, v=v, row_req=_i32(req), row_pos=_i32(pos), block_table=_i32(TABLE), k_pool=kp, v_pool=vp,
                      norm=True, k_gamma=g, eps=1e-5, rope_cos=cos, rope_sin=sin, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0x1 | 0x2 | 0x8  # bad page, bad request, past the tables
    ref = PO.norm_rotate(_np(k), pos, gamma=_np(g), eps=1e-5, cos=_np(cos), sin=_np(sin))
    written = []
    for t, (b, p) in enumerate(APPEND):
        if b < 0 or b > 1 or p < 0 or p // 128 >= 4 or not 0 <= TABLE[b, p // 128] < 5:
            continue
        slot = (int(TABLE[b, p // 128]), p % 128)
        written.append(slot)
        _close_vec(_np(kp[slot]), ref[t])
        if with_v:
            assert torch.equal(vp[slot], v[t])
        kp[slot] = 7.0
        if with_v:
            vp[slot] = 7.0
    assert len(written) == 10
    assert torch.equal(kbig, k0) and (not with_v or torch.equal(vbig, v0))  # nothing else was touched


@pytest.mark.parametrize("heads,dim,with_v", [(1, 512, False), (2, 128, True), (3, 32, True), (1, 96, True)])
def test_append_mxfp8(heads, dim, with_v):
    rng = np.random.default_rng(dim)
    T = 200
    k, v = _bf(rng, T, heads, dim, scale=3), _bf(rng, T, heads, dim)
    k[3] = 0
    k[4, :, 5] = 2.0 ** 100
    v[5] *= 2.0 ** -126
    v = v if with_v else None
    cos, sin = (torch.from_numpy(x).float().to(DEV) for x in PO.rope_table(256, 32))
    shape = (3, 128, heads, dim)
    kp, ks = torch.full(shape, 9, dtype=torch.uint8, device=DEV), torch.full(shape[:3] + (dim // 32,), 9,
                                                                             dtype=torch.uint8, device=DEV)
    vp, vs = (kp.clone(), ks.clone()) if with_v else (None, None)
    csa.csa_kv_append(k=k, v=v, row_req=_i32([0] * T), row_pos=_i32(np.arange(T)), block_table=_i32([[2, 0]]),
                      k_pool=kp, v_pool=vp, k_scale_pool=ks, v_scale_pool=vs, rope_cos=cos, rope_sin=sin,
                      rope_layout="half")
    torch.cuda.synchronize()
    ref_k = PO.norm_rotate(_np(k), np.arange(T), norm=False, cos=_np(cos), sin=_np(sin), layout="half")
    for x, codes, scales in ((ref_k, kp, ks), (_np(v) if with_v else None, vp, vs)):
        if x is None:
            continue
        val = codes.view(torch.float8_e4m3fn).float().double().cpu().numpy()
        e = scales.cpu().numpy().astype(int) - 127
        for t in range(T):
            slot = ([2, 0][t // 128], t % 128)
            for h in range(heads):
                for g in range(dim // 32):
                    y = x[t, h, 32 * g:32 * g + 32]
                    lo, hi = (PO.mxfp8_exponent(y * f) for f in (1 - 2.0 ** -20, 1 + 2.0 ** -20))
                    assert lo <= e[slot][h, g] <= hi
                    s = 2.0 ** int(e[slot][h, g])
                    got = val[slot][h, 32 * g:32 * g + 32] * s
                    # half an E4M3 step (2^-4 of the value, 2^-10 of the scale below 2^-6), FP32 before it
                    tol = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * s + 2.0 ** -20 * np.abs(y).max()
                    assert (np.abs(got - y) <= tol).all()
        assert (codes[1] == 9).all() and (codes[0, 72:] == 9).all() and (scales[1] == 9).all()


def test_append_feeds_the_sparse_attention():
    """Window rows published here (BF16 and MXFP8) are what the decode
    attention reads: the same output as with the rows laid there by hand."""
    from oracle import dequant_mxfp8  # noqa: F401  (the format's definition)

    rng = np.random.default_rng(11)
    n, H = 130, 64
    raw = _bf(rng, n, 1, 512)
    cos, sin = (torch.from_numpy(x).float().to(DEV) for x in PO.rope_table(256, 64))
    table = _i32([[1, 0]])
    common = dict(k=raw, row_req=_i32([0] * n), row_pos=_i32(np.arange(n)), block_table=table, norm=True,
                  rope_cos=cos, rope_sin=sin)
    bf = torch.zeros((2, 128, 512), dtype=torch.bfloat16, device=DEV)
    csa.csa_kv_append(k_pool=bf, **common)
    fp8 = torch.zeros((2, 128, 512), dtype=torch.uint8, device=DEV)
    sc = torch.zeros((2, 128, 16), dtype=torch.uint8, device=DEV)
    csa.csa_kv_append(k_pool=fp8, k_scale_pool=sc, **common)
    deq = (fp8.view(torch.float8_e4m3fn).float().view(2, 128, 16, 32)
           * torch.exp2(sc.float() - 127)[..., None]).view(2, 128, 512).bfloat16()
    ref = PO.norm_rotate(_np(raw), np.arange(n), cos=_np(cos), sin=_np(sin))[:, 0]
    hand = torch.zeros_like(bf)
    hand[1], hand[0, :2] = torch.from_numpy(ref[:128]).to(DEV), torch.from_numpy(ref[128:]).to(DEV)
    assert ((hand.float() - bf.float()).abs() <= 2 * H8 * hand.float().abs() + 1e-4).all()
    assert ((deq.float() - bf.float()).abs() <= 0.08 * bf.float().abs() + 0.02).all()
    q = _bf(rng, 2, H, 512)
    outs = []
    for pool, scale in ((bf, None), (deq, None), (fp8, sc)):
        out = torch.zeros_like(q)
        csa.csa_sparse_attn_decode(
            q=q, row_req=_i32([0, 0]), row_pos=_i32([128, 129]), topk_idx=_i32([[-1] * 8] * 2), kv_pool=pool,
            kv_block_table=table, kv_len=_i32([n]), cmp_pool=bf, cmp_block_table=table, n_cmp=_i32([0]), ratio=4,
            out=out, kv_scale_pool=scale)
        outs.append(out)
    torch.cuda.synchronize()
    assert torch.equal(outs[1], outs[2])
    k64 = _np(bf).reshape(256, 512)[np.r_[128:256, 0:2]].reshape(1, n, 1, 512)
    for t, p in enumerate((128, 129)):
        win = np.arange(p - 127, p + 1)
        x = _np(q)[t] @ k64[0, win, 0].T / np.sqrt(512)
        w = np.exp(x - x.max(1, keepdims=True))
        o = w @ k64[0, win, 0] / w.sum(1, keepdims=True)
        assert np.abs(_np(outs[0])[t] - o).max() <= 2e-2


# ---------------------------------------------------------------- attention


class Batch:
    """A paged cache and the rows that read it.  Everything that no row may
    see holds NaN: pages outside the tables, positions past a request's
    length."""

    def __init__(self, rows, lens, heads, kv_heads, dim, seed=0, kind="dense", extra_pages=3, qk=1.5, table=None):
        rng = np.random.default_rng(seed)
        self.req, self.pos = (np.array(x, dtype=np.int32) for x in zip(*rows))
        self.lens = np.array(lens, dtype=np.int32)
        pages = [-(-max(n, 1) // 128) for n in lens]
        if table is None:
            order = rng.permutation(sum(pages) + extra_pages)
            table, at = np.full((len(lens), max(pages)), -1, dtype=np.int32), 0
            for b, n in enumerate(pages):
                table[b, :n] = order[at:at + n]
                at += n
        self.table = table
        nb = sum(pages) + extra_pages
        kp, vp = np.full((2, nb, 128, kv_heads, dim), np.nan)
        for b, n in enumerate(lens):
            for j in range(0, n, 128):
                ph, m = table[b, j // 128], min(128, n - j)
                if 0 <= ph < nb:
                    kp[ph, :m] = rng.standard_normal((m, kv_heads, dim)) * qk
                    vp[ph, :m] = rng.standard_normal((m, kv_heads, dim))
        self.k, self.kbig = _pool(nb, kv_heads, dim, kind, NAN)
        self.v, self.vbig = _pool(nb, kv_heads, dim, kind, NAN)
        self.k.copy_(torch.from_numpy(kp).to(DEV))
        self.v.copy_(torch.from_numpy(vp).to(DEV))
        self.q = _bf(rng, len(rows), heads, dim, scale=qk)
        self.sink = torch.from_numpy(rng.standard_normal(heads)).float().to(DEV)
        self.heads, self.dim = heads, dim

    def call(self, mode, causal=True, window=0, sink=True, out=None, lse=None, **kw):
        T = len(self.req)
        out = torch.full((T, self.heads, self.dim), 77.0, dtype=torch.bfloat16, device=DEV) if out is None else out
        lse = torch.full((T, self.heads), 77.0, device=DEV) if lse is None else lse
        st = _status()
        r = csa.csa_paged_attn(q=self.q, row_req=_i32(self.req), row_pos=_i32(self.pos), k_pool=self.k, v_pool=self.v,
                               block_table=_i32(self.table), kv_len=_i32(self.lens), out=out, lse=lse,
                               sink=self.sink if sink else None, causal=causal, window=window, mode=mode, status=st,
                               **kw)
        if kw.get("prepare"):
            return r, out, lse, st
        torch.cuda.synchronize()
        return out, lse, int(st.item())

    def oracle(self, causal=True, window=0, sink=True):
        return PO.paged_attention(_np(self.q), self.req, self.pos, _np(self.k), _np(self.v), self.table, self.lens,
                                  self.dim ** -0.5, causal=causal, window=window,
                                  sink=_np(self.sink) if sink else None)

    def check(self, mode, status=0, **kw):
        out, lse, st = self.call(mode, **kw)
        assert st == status
        self.compare(out, lse, **kw)
        return out, lse

    def compare(self, out, lse, **kw):
        o, ls, spread = self.oracle(**kw)
        got, gl = _np(out), _np(lse)
        skip = (self.req < 0) | (self.req >= len(self.lens))
        assert (got[skip] == 77).all() and (gl[skip] == 77).all()
        got, gl, o, ls, spread = (x[~skip] for x in (got, gl, o, ls, spread))
        # FP32 logits: dim products of |q||k| scale, each sum off by 2^-24 of it
        qn = np.abs(_np(self.q)).max() * np.nanmax(np.abs(_np(self.k))) if np.isfinite(_np(self.k)).any() else 0
        e = (self.dim * 2.0 ** -24) * qn * self.dim ** 0.5
        assert np.isfinite(got).all()
        tol = H8 * np.abs(o) + (H8 + 2 * e + 2.0 ** -12) * spread + 1e-30
        assert (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
        none = np.isneginf(ls)
        assert np.array_equal(none, np.isneginf(gl))
        n = int(self.lens.max()) if len(self.lens) else 0
        lt = e + (n + 64) * 2.0 ** -24 + 2.0 ** -21 * np.abs(ls[~none]) + 2.0 ** -20
        assert (np.abs(gl[~none] - ls[~none]) <= lt).all(), (np.abs(gl[~none] - ls[~none]) / lt).max()


def chunk(b, first, n):
    return [(b, first + i) for i in range(n)]


MODES = pytest.mark.parametrize("mode", [DECODE, PREFILL])


@MODES
@pytest.mark.parametrize("n", [1, 2, 16, 127, 128, 129, 255, 257, 1000])
@pytest.mark.parametrize("heads,kv_heads,dim", [(8, 2, 128), (4, 4, 64)])
def test_one_token(mode, n, heads, kv_heads, dim):
    Batch([(0, n - 1)], [n], heads, kv_heads, dim, seed=n).check(mode)


@MODES
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (2, 2), (8, 4), (9, 3), (7, 1), (16, 1), (17, 1), (40, 2),
                                            (64, 1), (100, 1), (128, 1), (24, 8)])
@pytest.mark.parametrize("dim", [64, 128])
def test_head_layouts(mode, heads, kv_heads, dim):
    rows = chunk(0, 130, 3) + chunk(1, 299, 1) + chunk(2, 0, 2)
    Batch(rows, [133, 300, 2], heads, kv_heads, dim, seed=heads).check(mode)


@MODES
@pytest.mark.parametrize("first,n,tail", [(0, 1, 0), (0, 5, 0), (0, 33, 0), (0, 130, 0), (0, 300, 0), (127, 2, 0),
                                          (500, 64, 0), (700, 257, 3), (250, 20, 200)])
@pytest.mark.parametrize("kw", [dict(), dict(window=1), dict(window=100), dict(window=129, sink=False),
                                dict(window=4096), dict(causal=False), dict(causal=False, window=50, sink=False)],
                         ids=lambda k: ",".join(f"{a}={b}" for a, b in k.items()) or "causal")
def test_chunks(mode, first, n, tail, kw):
    """Chunks at the start, across pages and inside a longer cache (``tail``
    positions after the last row)."""
    Batch(chunk(0, first, n), [first + n + tail], 4, 2, 64, seed=n).check(mode, **kw)


@MODES
@pytest.mark.parametrize("kw", [dict(), dict(window=70)])
def test_mixed_batch(mode, kw):
    """Chunks and single tokens of different requests, padding between them, a
    row without a position, a row past its cache, an empty cache."""
    rows = (chunk(0, 100, 70) + [(-1, 3)] + chunk(1, 0, 40) + [(2, 600)] + [(3, 0)] + [(2, 601)] + chunk(4, 5, 1)
            + [(-1, -1)] * 3 + [(0, -1)] + [(5, 300)] + [(1, 500)])
    Batch(rows, [170, 40, 602, 0, 6, 130], 8, 2, 128).check(mode, **kw)


@MODES
def test_rows_in_any_order(mode):
    rng = np.random.default_rng(5)
    rows = chunk(0, 0, 60) + chunk(1, 200, 60) + chunk(2, 3, 30)
    rows = [rows[i] for i in rng.permutation(len(rows))]
    Batch(rows, [60, 260, 33], 4, 1, 64).check(mode)


@MODES
@pytest.mark.parametrize("kind", ["dense", "heads_first", "beside", "layers"])
@pytest.mark.parametrize("dim", [64, 128])
def test_pool_layouts(mode, kind, dim):
    rows = chunk(0, 120, 20) + [(1, 256)]
    ref = Batch(rows, [140, 257], 6, 3, dim)
    b = Batch(rows, [140, 257], 6, 3, dim, kind=kind)
    assert torch.equal(b.q, ref.q)
    o, l = b.check(mode)
    r, rl, _ = ref.call(mode)
    assert torch.equal(o, r) and torch.equal(l, rl)


@MODES
def test_strided_queries(mode):
    b = Batch(chunk(0, 60, 50), [110], 4, 2, 128)
    want = b.call(mode)
    big = torch.full((50, 9, 128), NAN, dtype=torch.bfloat16, device=DEV)
    big[:, 2:6] = b.q
    b.q = big[:, 2:6]
    got = b.call(mode)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@MODES
def test_bad_pages_and_requests(mode):
    """Pages outside the pool hide their positions and raise the flag; a
    request outside the table skips its rows; a length past the table ends at
    the table."""
    table = np.array([[0, 7, 2], [3, -1, 5], [1, 4, 99]], dtype=np.int32)
    rows = chunk(0, 250, 30) + [(1, 300), (1, 100)] + [(3, 5), (9, 5)] + [(2, 255)]
    b = Batch(rows, [384, 384, 256], 4, 2, 64, table=table, extra_pages=0)
    assert b.k.shape[0] == 8
    b.lens[0] = 5000
    b.check(mode, status=0x1 | 0x2)


@MODES
def test_nothing_is_seen(mode):
    """Empty rows: out = 0 and lse = the sink, or -inf without one."""
    rows = [(0, 5), (1, -1), (1, -2147483648), (0, 2147483647)]
    b = Batch(rows, [0, 9], 4, 2, 128)
    for sink in (True, False):
        out, lse = b.check(mode, sink=sink)
        assert (out == 0).all()
        assert torch.equal(lse, b.sink.expand(4, 4)) if sink else torch.isneginf(lse).all()
    # far positions with a cache behind them
    b = Batch([(0, 2147483647), (0, 300)], [200], 4, 2, 128)
    b.check(mode)
    out, _ = b.check(mode, window=150)
    assert (out[0] == 0).all() and (out[1] != 0).any()
    b.check(mode, causal=False, window=2147483647)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,kv_heads", [(64, 1), (32, 8), (2, 2)])
def test_many_rows_that_see_nothing(heads, kv_heads, dim):
    """Whole tiles without a page, among tiles with pages: zeros where the
    queries were on their way, over and over."""
    n = 3000
    b = Batch([(t // 1000, t % 1000) for t in range(n)], [0, 40, 0], heads, kv_heads, dim)
    b.q.fill_(float("inf"))
    b.q[1000:2000] = 0.5
    for _ in range(10):
        out, lse, st = b.call(PREFILL)
        assert st == 0
        assert (out[:1000] == 0).all() and (out[2000:] == 0).all()
        assert torch.equal(lse[:1000], b.sink.expand(1000, heads)) and torch.equal(lse[2000:], lse[:1000])
        assert out[1000:2000].isfinite().all() and (out[1000:2000] != 0).any()


@MODES
def test_unbounded_sinks(mode):
    """A sink of +inf takes everything: out = 0, lse = inf; a row that sees
    nothing returns its sink's bits.  Whole rows and rows in parts."""
    for b in (Batch(chunk(0, 30, 6) + [(1, -1)], [36, 0], 8, 2, 128), Batch([(0, 4000), (1, 3)], [4001, 0], 8, 2, 64)):
        b.sink[::2] = float("inf")
        out, lse, st = b.call(mode)
        assert st == 0
        assert (out[:, ::2] == 0).all() and (lse[:, ::2] == float("inf")).all()
        assert torch.equal(lse[-1], b.sink) and (out[-1] == 0).all()
        b.sink[::2] = -float("inf")
        b.check(mode)


@MODES
def test_last_positions_of_a_table(mode):
    """A window over the last of 2^31 positions: the one past kv_len lies on
    the same page and holds NaN."""
    top, window, heads, kv_heads, dim = 2 ** 31 - 1, 200, 4, 2, 128
    rng = np.random.default_rng(5)
    k, v = _bf(rng, 3, 128, kv_heads, dim), _bf(rng, 3, 128, kv_heads, dim)
    k[2, 127], v[2, 127] = NAN, NAN
    table = torch.full((1, 1 << 24), -1, dtype=torch.int32, device=DEV)
    table[0, -3:] = _i32([0, 1, 2])
    pos = np.array([top - 2, top - 1, top - 130, top], dtype=np.int64)
    q, sink = _bf(rng, 4, heads, dim), torch.zeros(heads, device=DEV)
    out, lse, st = torch.empty_like(q), torch.empty((4, heads), device=DEV), _status()
    csa.csa_paged_attn(q=q, row_req=_i32([0] * 4), row_pos=torch.from_numpy(pos).int().to(DEV), k_pool=k, v_pool=v,
                       block_table=table, kv_len=_i32([top]), out=out, lse=lse, sink=sink, window=window, mode=mode,
                       status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # the same rows over the last three pages alone
    o, ls, spread = PO.paged_attention(_np(q), np.zeros(4, int), pos - (top + 1 - 384), _np(k), _np(v),
                                       np.array([[0, 1, 2]]), [383], dim ** -0.5, window=window, sink=np.zeros(heads))
    # as Batch.compare counts them
    e = dim * 2.0 ** -24 * np.abs(_np(q)).max() * np.nanmax(np.abs(_np(k))) * dim ** 0.5
    assert (np.abs(_np(out) - o) <= H8 * np.abs(o) + (H8 + 2 * e + 2.0 ** -12) * spread).all()
    assert (np.abs(_np(lse) - ls) <= e + 512 * 2.0 ** -24 + 2.0 ** -21 * np.abs(ls) + 2.0 ** -20).all()


@MODES
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), NAN])
@pytest.mark.parametrize("heads,kv_heads,dim,window", [(8, 1, 128, 0), (4, 4, 64, 0), (8, 2, 64, 40)])
def test_hidden_infinities(mode, value, heads, kv_heads, dim, window):
    """Keys and values that are not finite reach the rows that see them, and no
    other row of the chunk or of another request."""
    rows = chunk(0, 180, 40) + chunk(1, 150, 10)
    b = Batch(rows, [220, 160], heads, kv_heads, dim)
    want, wl, _ = b.call(mode, window=window)
    clean = b.v.clone(), b.k.clone()
    for where in (200, 130):  # a position in the chunk, one before it
        for pool in (b.v, b.k):
            at = (int(b.table[0, where // 128]), where % 128)
            pool[at[0], at[1], :, 3] = value
            out, lse, st = b.call(mode, window=window)
            assert st == 0
            sees = np.array([r == 0 and p >= where and not (window and p - where >= window) for r, p in rows])
            ok = torch.from_numpy(~sees).to(DEV)
            assert torch.equal(out[ok], want[ok]) and torch.equal(lse[ok], wl[ok])
            if pool is b.v:
                assert not torch.isfinite(out[~ok][..., 3]).any()
                rest = torch.ones(dim, dtype=torch.bool, device=DEV)
                rest[3] = False
                if sees.any():
                    d = (out[~ok][..., rest].float() - want[~ok][..., rest].float()).abs()
                    assert (d <= 2 * H8 * (want[~ok][..., rest].float().abs() + 1)).all()
            b.v.copy_(clean[0])
            b.k.copy_(clean[1])


@MODES
@pytest.mark.parametrize("value", [float("inf"), NAN])
def test_a_broken_query_stays_alone(mode, value):
    """A query row that is not finite leaves every other row's bits as they were."""
    b = Batch(chunk(0, 180, 40) + chunk(1, 100, 3), [220, 103], 8, 2, 128)
    want, wl, _ = b.call(mode)
    for t in (7, 41):
        keep = b.q.clone()
        b.q[t, 3, 5] = value
        out, lse, _ = b.call(mode)
        other = torch.ones(43, 8, dtype=torch.bool, device=DEV)
        other[t, 3] = False
        assert torch.equal(out[other], want[other]) and torch.equal(lse[other], wl[other])
        assert out[t, 3].isnan().any()
        b.q.copy_(keep)


@MODES
@pytest.mark.parametrize("n,heads,kv_heads", [(511, 4, 2), (512, 2, 2), (600, 4, 1)])
def test_many_single_rows(mode, n, heads, kv_heads):
    """Requests of one row around the decode kernel's most rows, some of them
    empty, some long enough for parts."""
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 40, n)
    lens[5], lens[300], lens[301] = 700, 0, 400
    Batch([(b, max(int(k) - 1, 0)) for b, k in enumerate(lens)], lens.tolist(), heads, kv_heads, 64).check(mode)


@pytest.mark.parametrize("n,heads,kv_heads", [(30, 40, 2), (48, 17, 1), (49, 17, 1), (330, 4, 2), (345, 4, 2)])
def test_single_rows_of_narrow_heads(n, heads, kv_heads):
    """Either side of the row counts up to which two CTAs share an SM; every
    third context ends inside a page that holds NaN from there on."""
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 700, n)
    lens[::7] = 128
    b = Batch([(i, int(lens[i]) - 1 + (i % 3 == 0)) for i in range(n)], lens, heads, kv_heads, 64, seed=n)
    b.check(DECODE)
    b.check(DECODE, window=200)


def test_chosen_kernel_agrees():
    """Sizes around the choice between the two kernels: the chosen one's result
    is one of the two."""
    for req, rows, heads, kv, dim in ((4, 16, 32, 8, 128), (24, 8, 64, 8, 64), (3, 8, 32, 1, 128), (2, 12, 16, 4, 64)):
        b = Batch([r for i in range(req) for r in chunk(i, 90 + 30 * i, rows)],
                  [90 + 30 * i + rows for i in range(req)], heads, kv, dim)
        got = b.check(csa.CSA_MODE_AUTO)
        both = [b.call(m) for m in (DECODE, PREFILL)]
        assert any(torch.equal(got[0], o) and torch.equal(got[1], l) for o, l, _ in both)


@MODES
def test_equal_positions_and_far_rows(mode):
    """Rows that repeat a position, and positions far past the cache."""
    rows = [(0, 50)] * 5 + [(0, 7)] * 3 + [(0, 10 ** 9)] * 2 + [(1, 3)] * 30
    b = Batch(rows, [300, 260], 4, 2, 64)
    out, lse = b.check(mode)
    b.q[1:5] = b.q[0]
    out, lse, _ = b.call(mode)
    assert all(torch.equal(out[0], out[i]) and torch.equal(lse[0], lse[i]) for i in range(1, 5))


@MODES
def test_large_logits(mode):
    """Logits to about +-1000, and their maximum in any page."""
    b = Batch(chunk(0, 300, 20), [320], 4, 2, 128, qk=9.0)
    b.check(mode, sink=False)
    b.sink.fill_(-3e38)
    b.check(mode)
    b.sink.fill_(500.0)
    b.check(mode)


@MODES
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_of_two_to_the_28(mode, sign):
    """Powers of two, so that the logits are exact: the positions with the
    largest share the row evenly, the others get nothing."""
    b = Batch([(0, 299), (0, 300), (1, 20), (1, 1)], [301, 30], 4, 2, 64)
    seen = ~b.k.isnan()
    b.q.zero_()
    b.q[..., 0] = 2.0 ** 16
    few = torch.arange(128, device=DEV)[None, :, None] % 16 == 3
    b.k[..., 0] = torch.where(few.expand(b.k.shape[:3]) == (sign > 0), 2.0 ** 15 * sign, 2.0 ** 14 * sign).bfloat16()
    b.k.masked_fill_(~seen, NAN)
    out, lse, st = b.call(mode, sink=False)
    assert st == 0
    for t, (r, p) in enumerate(zip(b.req, b.pos)):
        j = np.arange(p + 1)
        top = j[j % 16 == 3] if (j % 16 == 3).any() else j
        # sign < 0: the small ones (2^14) are the largest
        v = _np(b.v)[b.table[r][top // 128], top % 128]  # [n, kv_heads, dim]
        o, spread = np.repeat(v.mean(0), 2, 0), np.repeat(np.abs(v).mean(0), 2, 0)
        assert (np.abs(_np(out)[t] - o) <= H8 * np.abs(o) + (H8 + 2.0 ** -12) * spread).all()
        x = 2.0 ** 13 * _np(b.k)[b.table[r][top[0] // 128], top[0] % 128, :, 0]
        ref = np.repeat(x, 2) + np.log(len(top))
        assert (np.abs(_np(lse)[t] - ref) <= 2.0 ** -21 * np.abs(ref)).all()


@MODES
@pytest.mark.parametrize("n,heads,kv_heads", [(40000, 8, 1), (20001, 16, 2)])
def test_long_cache(mode, n, heads, kv_heads):
    b = Batch([(0, n - 2), (0, n - 1), (1, 500)], [n, 501], heads, kv_heads, 64, seed=2)
    b.check(mode)
    b.check(mode, window=9000)


def test_pools_past_four_gigabytes():
    """Byte offsets past 32 bits: pages at the end of pools of 5 GB."""
    nb = 20480
    big = [torch.empty((nb, 128, 8, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    small = Batch(chunk(0, 100, 60) + [(1, 300)], [160, 301], 16, 8, 128)
    top = nb - 1 - np.arange(small.k.shape[0])
    for p, s in zip(big, (small.k, small.v)):
        p[torch.from_numpy(top).to(DEV)] = s
    ok = small.table >= 0
    want = [small.call(m) for m in (DECODE, PREFILL)]
    small.k, small.v = big
    small.table = np.where(ok, top[np.where(ok, small.table, 0)], -1).astype(np.int32)
    for m, w in zip((DECODE, PREFILL), want):
        got = small.call(m)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    # rows published there
    k = _bf(np.random.default_rng(0), 3, 8, 128)
    csa.csa_kv_append(k=k, row_req=_i32([0] * 3), row_pos=_i32([1, 2, 128]), block_table=_i32([[nb - 30, nb - 40]]),
                      k_pool=big[0])
    torch.cuda.synchronize()
    assert torch.equal(big[0][nb - 30, 1:3], k[:2]) and torch.equal(big[0][nb - 40, 0], k[2])


@MODES
def test_same_bits_every_time(mode):
    b = Batch(chunk(0, 2000, 40) + [(1, 700)], [2040, 701], 16, 2, 128)
    ref = b.call(mode)
    for _ in range(5):
        got = b.call(mode)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@MODES
def test_workspace_is_scratch(mode):
    """A workspace with anything in it, used by calls of other sizes in between."""
    b = Batch(chunk(0, 3000, 3), [3003], 16, 2, 128)
    c = Batch(chunk(0, 100, 80) + [(1, 5000)], [180, 5001], 8, 4, 64)
    rb, rc = b.call(mode), c.call(mode)
    ws = torch.full((512 << 20,), 0xFF, dtype=torch.uint8, device=DEV)
    for x, r in ((b, rb), (c, rc), (b, rb)):
        got = x.call(mode, workspace=ws)
        assert torch.equal(got[0], r[0]) and torch.equal(got[1], r[1])
    ws.fill_(0x7F)
    got = c.call(mode, workspace=ws)
    assert torch.equal(got[0], rc[0])


@MODES
def test_streams_and_graphs(mode):
    """Prepared calls on a side stream and in captured graphs, two graphs that
    share nothing replayed at once, new inputs through the same tensors."""
    a = Batch(chunk(0, 400, 90), [490], 8, 2, 128, seed=1)
    b = Batch(chunk(0, 900, 4) + [(1, 300)], [904, 301], 8, 2, 64, seed=2)
    want = [x.call(mode) for x in (a, b)]
    side = torch.cuda.Stream()
    calls = [x.call(mode, prepare=True) for x in (a, b)]
    torch.cuda.synchronize()
    for _ in range(3):
        for (call, *_), s in zip(calls, (side, None)):
            call(s)
    torch.cuda.synchronize()
    for (_, out, lse, st), w in zip(calls, want):
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
        out.fill_(3), lse.fill_(3)
    graphs = []
    for call, *_ in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for (_, out, lse, st), w in zip(calls, want):
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1]) and int(st.item()) == 0
    a.q.copy_(a.q.flip(0))
    graphs[0].replay()
    torch.cuda.synchronize()
    new = a.call(mode)
    assert not torch.equal(new[0], want[0][0]) and torch.equal(calls[0][1], new[0])


@MODES
def test_graphs_that_share_a_workspace(mode):
    """Two graphs captured on one workspace and replayed in turn, the caller's
    own references gone."""
    a = Batch(chunk(0, 2000, 20), [2020], 8, 2, 128, seed=1)
    b = Batch([(0, 4000), (1, 77)], [4001, 78], 16, 4, 64, seed=2)
    want = [x.call(mode) for x in (a, b)]
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device=DEV)
    runs = []
    for x in (a, b):
        call, out, lse, _ = x.call(mode, prepare=True, workspace=ws)
        call()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        runs.append((g, out, lse, call))
    del a, b, x, ws
    junk = [torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(4)]
    for _ in range(3):
        for (g, out, lse, _), w in zip(runs, want):
            out.fill_(1)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
    del junk


def test_no_rows():
    """Calls with nothing to do launch nothing and touch nothing."""
    q, k = (torch.zeros((0, h, 64), dtype=torch.bfloat16, device=DEV) for h in (4, 2))
    none, tab = _i32([]), _i32([[0]])
    cos, sin = (torch.ones((16, 32), device=DEV) for _ in range(2))
    pool = torch.full((1, 128, 2, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    torch.cuda.synchronize()
    before = csa.launch_count()
    csa.csa_rope_table(cos=cos[:0], sin=sin[:0])
    csa.csa_qk_norm_rope(q=q, k=k, row_pos=none, rope_cos=cos, rope_sin=sin)
    csa.csa_kv_append(k=k, v=k, row_req=none, row_pos=none, block_table=tab, k_pool=pool, v_pool=pool.clone(), norm=True,
                      rope_cos=cos, rope_sin=sin)
    csa.csa_paged_attn(q=q, row_req=none, row_pos=none, k_pool=pool, v_pool=pool, block_table=tab, kv_len=_i32([5]),
                       out=q.clone())
    torch.cuda.synchronize()
    assert csa.launch_count() == before and (pool == 3).all()


def test_both_kernels_agree_with_auto():
    for rows, lens in ((chunk(0, 900, 1) + [(1, 44)], [901, 45]), (chunk(0, 0, 600), [600])):
        b = Batch(rows, lens, 8, 2, 128)
        got = b.check(csa.CSA_MODE_AUTO)
        assert any(torch.equal(got[0], b.call(m)[0]) for m in (DECODE, PREFILL))


# ---------------------------------------------------------------- the operators together


@pytest.mark.parametrize("dim,layout,window", [(128, "half", 0), (64, "adjacent", 100)])
def test_a_layer_from_prompt_to_tokens(dim, layout, window):
    """Tables, norms, publication and attention as a layer uses them: a prompt
    chunk, then single tokens, against the definitions from the same inputs."""
    rng = np.random.default_rng(7)
    hq, hk, first, steps = 8, 2, 150, 3
    n = first + steps
    qkv = _bf(rng, n, hq + 2 * hk, dim)
    gq, gk = _bf(rng, dim), _bf(rng, dim)
    cos, sin = torch.empty((256, dim // 2), device=DEV), torch.empty((256, dim // 2), device=DEV)
    scaling = dict(scaling="yarn", factor=4.0, orig_len=128)
    csa.csa_rope_table(cos=cos, sin=sin, **scaling)
    table = _i32([[2, 0]])
    kp, vp = (torch.full((3, 128, hk, dim), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros((n, hq, dim), dtype=torch.bfloat16, device=DEV)
    qo = torch.empty_like(out)
    st = _status()
    for t0, t1 in [(0, first)] + [(first + i, first + i + 1) for i in range(steps)]:
        x = qkv[t0:t1]
        req, pos, ln = _i32([0] * (t1 - t0)), _i32(np.arange(t0, t1)), _i32([t1])
        rope = dict(rope_cos=cos, rope_sin=sin, rope_layout=layout, status=st)
        csa.csa_qk_norm_rope(q=x[:, :hq], q_out=qo[t0:t1], row_pos=pos, q_gamma=gq, **rope)
        csa.csa_kv_append(k=x[:, hq:hq + hk], v=x[:, hq + hk:], row_req=req, row_pos=pos, block_table=table, k_pool=kp,
                          v_pool=vp, norm=True, k_gamma=gk, **rope)
        csa.csa_paged_attn(q=qo[t0:t1], row_req=req, row_pos=pos, k_pool=kp, v_pool=vp, block_table=table, kv_len=ln,
                           out=out[t0:t1], window=window, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    c64, s64 = PO.rope_table(256, dim, **scaling)
    turn = dict(cos=c64, sin=s64, layout=layout)
    x = _np(qkv)
    q64 = PO.norm_rotate(x[:, :hq], np.arange(n), gamma=_np(gq), **turn)
    k64, v64 = np.zeros((2, 3, 128, hk, dim))
    kk = PO.norm_rotate(x[:, hq:hq + hk], np.arange(n), gamma=_np(gk), **turn)
    for j in range(n):
        k64[[2, 0][j // 128], j % 128], v64[[2, 0][j // 128], j % 128] = kk[j], x[j, hq + hk:]
    o, _, spread = PO.paged_attention(q64, [0] * n, np.arange(n), k64, v64, _np(table).astype(int), [n], dim ** -0.5,
                                      window=window)
    # BF16 q and k move a logit by up to 2 * 2^-8 sum |q||k| scale
    logit = 2 * H8 * np.abs(q64).max() * np.abs(kk).max() * dim ** 0.5
    assert (np.abs(_np(out) - o) <= H8 * np.abs(o) + (H8 + 2 * logit) * spread + 1e-6).all()
    assert np.abs(_np(out) - o).mean() <= 2 * H8 * np.abs(o).mean() + 1e-3


@pytest.mark.parametrize("lowbit", [False, True])
def test_csa_step_publishes_its_window(lowbit):
    """A CSA step that publishes its own window rows: the same result as the
    step on a pool that already holds them, run eagerly, prepared and captured."""
    from prefill_csa_compress_gb300.pipeline import CsaStep
    from workloads import make_workload, spec_for

    spec = spec_for("lowbit_decode" if lowbit else "serving_decode", seed=77)
    t = make_workload(spec).to(DEV)
    n = t["row_req"].shape[0]
    t["win_raw"] = _bf(np.random.default_rng(1), n, 512)
    t["win_gamma"] = _bf(np.random.default_rng(2), 512)
    names = ["kv_pool", "kv_scale"] if lowbit else ["kv_pool"]
    before = {k: t[k].clone() for k in names}
    step = CsaStep(t, spec.ratio, spec.topk)
    step.publish_window()
    torch.cuda.synchronize()
    after = {k: t[k].clone() for k in names}
    changed = (after["kv_pool"] != before["kv_pool"]).flatten(2).any(-1)
    assert int(changed.sum()) == n and int(step.status.item()) == 0
    plain = CsaStep({k: v for k, v in t.items() if not k.startswith("win_")}, spec.ratio, spec.topk)
    plain.run()
    torch.cuda.synchronize()
    want = plain.out.clone(), plain.lse.clone()
    graph = []

    def captured():
        if not graph:
            step.capture()
            graph.append(1)
        step.replay()

    for run in (step.run, lambda: step.prepare().run(), captured):
        for k in names:
            t[k].copy_(before[k])
        step.out.zero_()
        run()
        torch.cuda.synchronize()
        assert int(step.status.item()) == 0
        assert all(torch.equal(t[k], after[k]) for k in names)
        assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])


def test_paged_attn_step():
    """The step object: a prompt eagerly, then tokens through one captured
    graph whose inputs change in place, against the calls one by one; and as
    a layer of a chain with another."""
    from prefill_csa_compress_gb300.pipeline import PagedAttnStep, StepChain

    rng = np.random.default_rng(9)
    hq, hk, dim, first = 8, 2, 128, 300
    cos, sin = torch.empty((512, 64), device=DEV), torch.empty((512, 64), device=DEV)
    csa.csa_rope_table(cos=cos, sin=sin)
    table = _i32([[1, 4, 0]])
    gq, gk = _bf(rng, dim), _bf(rng, dim)
    sink = torch.zeros(hq, device=DEV)

    def tensors(n, pos, pools):
        qkv = _bf(rng, n, hq + 2 * hk, dim)
        return dict(q=qkv[:, :hq], k=qkv[:, hq:hq + hk], v=qkv[:, hq + hk:], row_req=_i32([0] * n),
                    row_pos=_i32(np.arange(pos, pos + n)), kv_len=_i32([pos + n]), k_pool=pools[0], v_pool=pools[1],
                    kv_table=table, rope_cos=cos, rope_sin=sin, q_gamma=gq, k_gamma=gk, sink=sink, qkv=qkv)

    def by_hand(t, window):
        q = torch.empty(t["q"].shape, dtype=torch.bfloat16, device=DEV)
        out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device=DEV)
        rope = dict(rope_cos=cos, rope_sin=sin, rope_layout="half")
        csa.csa_qk_norm_rope(q=t["q"], q_out=q, row_pos=t["row_pos"], q_gamma=gq, **rope)
        csa.csa_kv_append(k=t["k"], v=t["v"], row_req=t["row_req"], row_pos=t["row_pos"], block_table=table,
                          k_pool=t["k_pool"], v_pool=t["v_pool"], norm=True, k_gamma=gk, **rope)
        csa.csa_paged_attn(q=q, row_req=t["row_req"], row_pos=t["row_pos"], k_pool=t["k_pool"], v_pool=t["v_pool"],
                           block_table=table, kv_len=t["kv_len"], out=out, lse=lse, sink=sink, window=window)
        torch.cuda.synchronize()
        return out, lse

    pools = [torch.full((5, 128, hk, dim), NAN, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    mine = [p.clone() for p in pools]
    t = tensors(first, 0, pools)
    step = PagedAttnStep(t, rope_layout="half")
    step.run()
    want = by_hand({**t, "k_pool": mine[0], "v_pool": mine[1]}, 0)
    assert torch.equal(step.out, want[0]) and torch.equal(step.lse, want[1])
    t = tensors(1, first, pools)
    other = [p.clone() for p in pools]
    chain = StepChain([PagedAttnStep(t, rope_layout="half"),
                       PagedAttnStep({**t, "k_pool": other[0], "v_pool": other[1]}, rope_layout="half", window=128)])
    chain.run()
    chain.capture()
    for i in range(3):
        t["qkv"].copy_(_bf(rng, 1, hq + 2 * hk, dim))
        t["row_pos"].fill_(first + i)
        t["kv_len"].fill_(first + i + 1)
        chain.replay()
        torch.cuda.synchronize()
        want = by_hand({**t, "k_pool": mine[0], "v_pool": mine[1]}, 0)
        assert torch.equal(chain.steps[0].out, want[0]) and torch.equal(chain.steps[0].lse, want[1])
        if i == 0:
            windowed = [p.clone() for p in other]
        want = by_hand({**t, "k_pool": windowed[0], "v_pool": windowed[1]}, 128)
        assert torch.equal(chain.out, want[0]) and torch.equal(chain.lse, want[1])
    for p, q in zip(pools, mine):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))
    assert int(chain.status.item()) == 0
