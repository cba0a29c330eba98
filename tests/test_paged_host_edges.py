"""Host checks of the paged key/value cache operators at sizes whose products
leave 64 bits (no GPU)."""

import ctypes

import pytest
import torch

from prefill_csa_compress_gb300 import _binding as B
from prefill_csa_compress_gb300 import _paged as P
from test_paged_host import APPEND, ATTN, L  # noqa: F401


def _status(name, args):
    a = P._CALLS[name]()
    a.struct_size = ctypes.sizeof(a)
    for k, v in args.items():
        setattr(a, k, v)
    return P._fn(name)(ctypes.byref(a), None)


TOP = 2 ** 31 - 1


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("page,token,head", [
    (1 << 33, 1 << 34, 1 << 39),              # pages reach 2^64, which wraps to a small number
    (1 << 39, (1 << 39) + 16, (1 << 39) + 32),  # to 2^70
    (1 << 33, 1 << 39, 1 << 34)])
def test_slots_that_overlap_past_64_bits(L, which, page, token, head):  # noqa: F811
    """Strides that fold the pool onto itself are refused, also where the bytes
    that its pages reach over leave 64 bits."""
    strides = {f"{which}_page_stride": page, f"{which}_token_stride": token, f"{which}_head_stride": head}
    assert _status("csa_kv_append", dict(APPEND, n_rows=0, n_blocks=TOP, **strides)) == B.CSA_ERR_INVALID_ARG
    assert _status("csa_paged_attn", dict(ATTN, n_rows=0, n_blocks=TOP, **strides)) == B.CSA_ERR_INVALID_ARG


def test_wide_strides_that_keep_slots_apart(L):  # noqa: F811
    """The largest strides of pools that do not overlap are taken."""
    strides = dict(k_page_stride=(1 << 40) - 16, k_token_stride=1 << 30, k_head_stride=1 << 20)
    assert _status("csa_kv_append", dict(APPEND, n_rows=0, n_blocks=TOP, **strides)) == B.CSA_OK
    assert _status("csa_paged_attn", dict(ATTN, n_rows=0, n_blocks=TOP, **strides)) == B.CSA_OK


def _meta(*shape, dtype=torch.int32):
    return torch.empty(shape, dtype=dtype, device="meta")


def _attn(**kw):
    bf = dict(dtype=torch.bfloat16)
    args = dict(q=_meta(1, 2, 64, **bf), row_req=_meta(1), row_pos=_meta(1), k_pool=_meta(1, 128, 1, 64, **bf),
                v_pool=_meta(1, 128, 1, 64, **bf), block_table=_meta(1, 1), kv_len=_meta(1), out=_meta(1, 2, 64, **bf))
    return P.csa_paged_attn(**{**args, **kw})


def _append(**kw):
    bf = dict(dtype=torch.bfloat16)
    args = dict(k=_meta(1, 1, 64, **bf), row_req=_meta(1), row_pos=_meta(1), block_table=_meta(1, 1),
                k_pool=_meta(1, 128, 1, 64, **bf))
    return P.csa_kv_append(**{**args, **kw})


MANY = 2 ** 32 + 1  # 1 in 32 bits


@pytest.mark.parametrize("call", [
    lambda: _attn(block_table=_meta(MANY, 1), kv_len=_meta(MANY)),
    lambda: _attn(block_table=_meta(1, MANY)),
    lambda: _attn(k_pool=_meta(MANY, 128, 1, 64, dtype=torch.bfloat16), v_pool=_meta(MANY, 128, 1, 64, dtype=torch.bfloat16)),
    lambda: _append(block_table=_meta(MANY, 1)),
    lambda: _append(block_table=_meta(1, MANY)),
    lambda: _append(k_pool=_meta(MANY, 128, 1, 64, dtype=torch.bfloat16)),
    lambda: P._rope(P.KvAppendArgs(), [], _meta(MANY, 32, dtype=torch.float32), _meta(MANY, 32, dtype=torch.float32),
                    "adjacent", None, 64),
    lambda: P.csa_qk_norm_rope(q=_meta(1, MANY, 64, dtype=torch.bfloat16), row_pos=_meta(1)),
    lambda: P.csa_qk_norm_rope(q=_meta(1, 1, 64, dtype=torch.bfloat16), k=_meta(1, MANY, 64, dtype=torch.bfloat16),
                               row_pos=_meta(1)),
    lambda: _append(k=_meta(1, MANY, 64, dtype=torch.bfloat16), k_pool=_meta(1, 128, MANY, 64, dtype=torch.bfloat16)),
])
def test_sizes_past_32_bits_are_refused(call):
    """A size that 32 bits would cut is named, not cut."""
    with pytest.raises(ValueError, match="32 bits"):
        call()
