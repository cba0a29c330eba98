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
