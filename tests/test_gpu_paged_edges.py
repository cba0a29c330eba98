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
