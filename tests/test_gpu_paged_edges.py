"""The paged key/value cache operators at the ends of their arguments' ranges:
far positions, large and small channels."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import prefill_csa_compress_gb300 as csa  # noqa: E402

from test_gpu_paged import DEV, MODES, Batch, _bf, _close_vec, _i32, _np, _pool, _status  # noqa: E402

LOWEST = -2 ** 31


# ---------------------------------------------------------------- rope tables

PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def _exact_angle(pos, f):
    """pos * f modulo a turn, from the exact product of the two numbers."""
    x = pos * Fraction(f) / (2 * PI)
    return float((x - round(x)) * 2 * PI)


@pytest.mark.parametrize("kw", [
    dict(), dict(theta=500000.0), dict(theta=1.5), dict(scaling="linear", factor=3.0),
    dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=40.0, orig_len=4096),
    dict(scaling="yarn", factor=7.0, orig_len=65536, theta=500000.0, beta_fast=16.0, beta_slow=2.0)])
@pytest.mark.parametrize("pos0", [0, 131071, 2 ** 24 + 12345, 2147308307, 2 ** 31 - 7])
@pytest.mark.parametrize("rope_dim,amp", [(128, 1.0), (64, 1.3688879454113936), (6, 0.5973347702152793)])
def test_rope_table_far_positions(kw, pos0, rope_dim, amp):
    """2e-7 of the FP64 rotation times the position, at any position (the
    definition's frequencies, and their product with the position exactly; the
    library's cosine of an FP64 angle adds 2^-52)."""
    n_pos, pairs = 7, rope_dim // 2
    cos, sin = torch.empty((n_pos, pairs), device=DEV), torch.empty((n_pos, pairs), device=DEV)
    csa.csa_rope_table(cos=cos, sin=sin, pos0=pos0, attn_factor=amp, **kw)
    torch.cuda.synchronize()
    f = PO.rope_frequencies(rope_dim, **kw)
    a = np.array([[_exact_angle(pos0 + j, float(f[i])) for i in range(pairs)] for j in range(n_pos)])
    assert np.abs(_np(cos) - amp * np.cos(a)).max() <= 2e-7 * amp
    assert np.abs(_np(sin) - amp * np.sin(a)).max() <= 2e-7 * amp


# ---------------------------------------------------------------- norms


def _extreme_heads(rng, rows, heads, dim):
    """Heads of one row at very different scales: the squares of the large ones
    leave FP32 (some only in the sum of 512), those of the small ones vanish."""
    x = rng.standard_normal((rows, heads, dim))
    scales = [1.0, 1e18, 3e-38, 1e30, 1e-30, 2.0 ** 125, 2.0 ** -100, 1e19, 3e17]
    for t in range(rows):
        for h in range(heads):
            x[t, h] *= scales[(3 * t + h) % len(scales)]
    x = torch.from_numpy(x).clamp(-3e38, 3e38).bfloat16()
    if rows > 1:
        x[1, 0] = torch.finfo(torch.bfloat16).max
        x[1, -1] = 2.0 ** -133  # the smallest BF16
        x[1, -1, 0] = -(2.0 ** -130)
    return x.to(DEV)


@pytest.mark.parametrize("layout", ["adjacent", "half"])
@pytest.mark.parametrize("heads,dim,rd", [(9, 512, 64), (2, 512, 512), (9, 128, 128), (5, 64, 32), (40, 8, 0), (3, 264, 208)])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-6])
def test_norm_of_extreme_heads(layout, heads, dim, rd, eps):
    """Finite channels of any size are normed as the formula says, in every head
    by itself; NaN and infinities stay in their head."""
    rng = np.random.default_rng(dim + heads)
    rows = 7
    x = _extreme_heads(rng, rows, heads, dim)
    gamma = _bf(rng, dim)
    pos = rng.integers(0, 50, rows)
    cos, sin = PO.rope_table(50, rd or 2)
    tabs = dict(rope_cos=torch.from_numpy(cos).float().to(DEV), rope_sin=torch.from_numpy(sin).float().to(DEV),
                rope_layout=layout) if rd else {}
    turn = dict(cos=_np(tabs["rope_cos"]), sin=_np(tabs["rope_sin"]), layout=layout) if rd else {}
    ref = PO.norm_rotate(_np(x), pos, gamma=_np(gamma), eps=eps, **turn)
    # below the normal range FP32 and BF16 resolve steps of 2^-149 and 2^-133 of the result
    out = torch.empty_like(x)
    csa.csa_qk_norm_rope(q=x, q_out=out, row_pos=_i32(pos), q_gamma=gamma, eps=eps, **tabs)
    _close_vec(_np(out), ref, extra=2.0 ** -133)
    pool, _ = _pool(2, heads, dim, "dense")
    csa.csa_kv_append(k=x, row_req=_i32([0] * rows), row_pos=_i32(np.arange(rows)), block_table=_i32([[1]]),
                      k_pool=pool, norm=True, k_gamma=gamma, eps=eps)
    _close_vec(_np(pool[1, :rows]), PO.norm_rotate(_np(x), pos, gamma=_np(gamma), eps=eps), extra=2.0 ** -133)
    for value in (math.nan, math.inf):
        y = x.clone()
        y[2, 0, dim // 2] = value
        broken = torch.empty_like(x)
        csa.csa_qk_norm_rope(q=y, q_out=broken, row_pos=_i32(pos), q_gamma=gamma, eps=eps, **tabs)
        torch.cuda.synchronize()
        assert broken[2, 0].isnan().any()
        same = torch.ones((rows, heads), dtype=torch.bool, device=DEV)
        same[2, 0] = False
        assert torch.equal(broken[same], out[same])


def test_publication_of_extreme_heads():
    """The same into an MXFP8 pool: codes of values between -gamma sqrt(512) and it."""
    rng = np.random.default_rng(8)
    rows, dim = 9, 512
    x = _extreme_heads(rng, rows, 1, dim)
    codes = torch.zeros((1, 128, 1, dim), dtype=torch.uint8, device=DEV)
    scales = torch.zeros((1, 128, 1, dim // 32), dtype=torch.uint8, device=DEV)
    csa.csa_kv_append(k=x, row_req=_i32([0] * rows), row_pos=_i32(np.arange(rows)), block_table=_i32([[0]]), k_pool=codes,
                      k_scale_pool=scales, norm=True, eps=0.0)
    torch.cuda.synchronize()
    ref = PO.norm_rotate(_np(x), np.zeros(rows), eps=0.0)[:, 0].reshape(rows, 16, 32)
    got = _np(codes[0, :rows, 0].view(torch.float8_e4m3fn).float()).reshape(rows, 16, 32)
    got = got * 2.0 ** (_np(scales[0, :rows, 0])[..., None] - 127)
    # half a step of E4M3, and below its normal range (2^-6) half of 2^-9, times the group's scale, at most
    # 2 amax / 448; FP32 as _close_vec counts it
    amax = np.abs(ref).max(-1, keepdims=True)
    assert (np.abs(got - ref) <= 2.0 ** -4 * np.abs(ref) + 2.0 ** -10 * amax / 224 + 2.0 ** -16 * amax).all()


# ---------------------------------------------------------------- attention


@MODES
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 128), (4, 2, 64), (34, 2, 64)])
def test_far_negative_positions(mode, heads, kv_heads, dim):
    """Rows whose position lies far below zero see nothing, also beside rows of
    their request that see several pages; so do requests of a negative length."""
    rows = [(0, LOWEST), (0, 299), (0, LOWEST + 130), (0, 700), (0, LOWEST + 600), (0, -1), (1, 5), (1, LOWEST), (0, 40)]
    b = Batch(rows, [701, 9], heads, kv_heads, dim)
    for kw in (dict(), dict(sink=False), dict(window=300), dict(window=2 ** 31 - 1)):
        out, lse = b.check(mode, **kw)
        none = [t for t, (_, p) in enumerate(rows) if p < 0]
        assert (out[none] == 0).all()
        want = b.sink.expand(len(none), heads) if kw.get("sink", True) else torch.full((), -math.inf, device=DEV)
        assert torch.equal(lse[none], want.expand(len(none), heads))
    b.check(mode, causal=False)
    b.check(mode, causal=False, window=200)
    b.lens[1] = LOWEST
    b.check(mode)
    b.check(mode, causal=False)
