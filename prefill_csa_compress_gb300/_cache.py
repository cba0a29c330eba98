"""ctypes binding of the latent cache and eviction calls: ``csa_latent_attn``,
``csa_latent_expand``, ``csa_attn_mass`` and ``csa_kv_evict`` of ``include/csa.h``
(argument marshalling only).

Checks, devices, streams and ``prepare`` are as in ``_paged``.
"""

from __future__ import annotations

import ctypes
from ctypes import c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p

import torch

from . import _paged as P
from ._paged import PAGE, _dense, _int32, _launch, _pool_strides, _ptr, _rows, _want

LATENT, ROPE, NOPE, VALUE = 512, 64, 128, 128


class LatentAttnArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_rows", c_int32), ("n_heads", c_int32), ("causal", c_int32),
        ("window", c_int32), ("softmax_scale", c_float), ("n_req", c_int32),
        ("max_blocks", c_int32), ("n_blocks", c_int32), ("q", c_void_p), ("q_rope", c_void_p),
        ("q_row_stride", c_int64), ("q_head_stride", c_int64), ("q_rope_row_stride", c_int64),
        ("q_rope_head_stride", c_int64), ("row_req", c_void_p), ("row_pos", c_void_p),
        ("kv_len", c_void_p), ("block_table", c_void_p), ("c_pool", c_void_p),
        ("r_pool", c_void_p), ("c_page_stride", c_int64), ("c_token_stride", c_int64),
        ("r_page_stride", c_int64), ("r_token_stride", c_int64), ("sink", c_void_p),
        ("out", c_void_p), ("lse", c_void_p), ("status_dev", c_void_p), ("workspace", c_void_p),
        ("workspace_bytes", c_size_t),
    ]


class LatentExpandArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_heads", c_int32), ("n_req", c_int32),
        ("max_blocks", c_int32), ("n_blocks", c_int32), ("out_max_blocks", c_int32),
        ("n_out_blocks", c_int32), ("kv_len", c_void_p), ("first", c_void_p),
        ("block_table", c_void_p), ("out_table", c_void_p), ("c_pool", c_void_p),
        ("r_pool", c_void_p), ("c_page_stride", c_int64), ("c_token_stride", c_int64),
        ("r_page_stride", c_int64), ("r_token_stride", c_int64), ("w_uk", c_void_p),
        ("w_uv", c_void_p), ("w_uk_head_stride", c_int64), ("w_uv_head_stride", c_int64),
        ("k_pool", c_void_p), ("v_pool", c_void_p), ("k_page_stride", c_int64),
        ("k_token_stride", c_int64), ("k_head_stride", c_int64), ("v_page_stride", c_int64),
        ("v_token_stride", c_int64), ("v_head_stride", c_int64), ("status_dev", c_void_p),
    ]


class AttnMassArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_rows", c_int32), ("n_heads", c_int32),
        ("n_kv_heads", c_int32), ("head_dim", c_int32), ("causal", c_int32),
        ("window", c_int32), ("softmax_scale", c_float), ("decay", c_float), ("n_req", c_int32),
        ("max_blocks", c_int32), ("n_blocks", c_int32), ("q", c_void_p),
        ("q_row_stride", c_int64), ("lse", c_void_p), ("row_req", c_void_p),
        ("row_pos", c_void_p), ("kv_len", c_void_p), ("block_table", c_void_p),
        ("k_pool", c_void_p), ("k_page_stride", c_int64), ("k_token_stride", c_int64),
        ("k_head_stride", c_int64), ("mass", c_void_p), ("mass_out", c_void_p),
        ("mass_row_stride", c_int64), ("mass_out_row_stride", c_int64),
        ("status_dev", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class KvEvictArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_req", c_int32), ("max_blocks", c_int32),
        ("n_blocks", c_int32), ("n_heads", c_int32), ("k_dim", c_int32), ("v_dim", c_int32),
        ("first", c_int32), ("recent", c_int32), ("mass", c_void_p),
        ("mass_row_stride", c_int64), ("kv_len", c_void_p), ("budget", c_void_p),
        ("block_table", c_void_p), ("k_pool", c_void_p), ("v_pool", c_void_p),
        ("k_page_stride", c_int64), ("k_token_stride", c_int64), ("k_head_stride", c_int64),
        ("v_page_stride", c_int64), ("v_token_stride", c_int64), ("v_head_stride", c_int64),
        ("kv_len_out", c_void_p), ("mass_out", c_void_p), ("mass_out_row_stride", c_int64),
        ("slot_src", c_void_p), ("status_dev", c_void_p), ("workspace", c_void_p),
        ("workspace_bytes", c_size_t),
    ]


P._CALLS.update(csa_latent_attn=LatentAttnArgs, csa_latent_expand=LatentExpandArgs,
                csa_attn_mass=AttnMassArgs, csa_kv_evict=KvEvictArgs)


# ---------------------------------------------------------------- checks


def _row_head_strides(t, name, shape):
    """Row and head strides in bytes of a BF16 [rows, heads, dim] tensor in
    either order (a head's channels contiguous)."""
    _want(t, name, torch.bfloat16, shape)
    n, h, d = t.shape
    if t.numel() == 0:  # (strides of an empty tensor say nothing)
        return h * d * 2, d * 2
    if d > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: a head's channels must be contiguous")
    head = t.stride(1) if h > 1 else d
    row = t.stride(0) if n > 1 else h * head
    if n > 1 and h > 1:
        apart = row >= head * (h - 1) + d if row >= head else head >= row * (n - 1) + d
    else:
        apart = True
    if min(row, head) < d or not apart:
        raise ValueError(f"{name}: rows must not overlap")
    return row * 2, head * 2


def _latent_pools(a, c_pool, r_pool):
    _want(c_pool, "c_pool", torch.bfloat16, (None, PAGE, LATENT))
    _want(r_pool, "r_pool", torch.bfloat16, (c_pool.shape[0], PAGE, ROPE))
    a.n_blocks = _int32(c_pool.shape[0], "pools")
    a.c_page_stride, a.c_token_stride, _ = _pool_strides(c_pool.unsqueeze(2), "c_pool")
    a.r_page_stride, a.r_token_stride, _ = _pool_strides(r_pool.unsqueeze(2), "r_pool")


def _kv_strides(a, prefix, t, name):
    for field, x in zip(("page", "token", "head"), _pool_strides(t, name)):
        setattr(a, f"{prefix}_{field}_stride", x)


def _table(a, block_table, kv_len):
    _dense(block_table, "block_table", torch.int32, (None, None))
    a.n_req, a.max_blocks = (_int32(x, "block_table") for x in block_table.shape)
    _dense(kv_len, "kv_len", torch.int32, (a.n_req,))


def _float_rows(t, name, shape):
    """Row stride in bytes of FP32 [requests, positions]."""
    _want(t, name, torch.float32, shape)
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: a request's entries must be contiguous")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}: rows must not overlap")
    return (t.stride(0) if t.shape[0] > 1 else t.shape[1]) * 4


def _optional(checks):
    for name, x, dtype, shape in checks:
        if x is not None:
            _dense(x, name, dtype, shape)


def _pointers(a, tensors, pairs):
    for name, x in pairs:
        setattr(a, name, _ptr(tensors, name, x))


# ---------------------------------------------------------------- calls


def csa_latent_attn(*, q, q_rope, row_req, row_pos, c_pool, r_pool, block_table, kv_len, out,
                    softmax_scale, lse=None, sink=None, causal=True, window=0, status=None,
                    workspace=None, stream=None, prepare=False):
    """Absorbed latent attention of the rows of ``q`` [rows, heads, 512] and
    ``q_rope`` [rows, heads, 64] over a paged latent cache, ``c_pool`` [pages, 128,
    512] and ``r_pool`` [pages, 128, 64], strided views included
    (``include/csa.h``: csa_latent_attn).  ``softmax_scale`` is that of the heads the
    latents stand for.  Returns the workspace, which a later call of the same sizes
    may be given; calls that overlap need one each."""
    a, tensors = LatentAttnArgs(), []
    a.struct_size = ctypes.sizeof(a)
    a.q_row_stride, a.q_head_stride = _row_head_strides(q, "q", (None, None, LATENT))
    n, h = int(q.shape[0]), int(q.shape[1])
    a.n_rows, a.n_heads = _int32(n, "q"), _int32(h, "q")
    a.q_rope_row_stride, a.q_rope_head_stride = _row_head_strides(q_rope, "q_rope", (n, h, ROPE))
    _latent_pools(a, c_pool, r_pool)
    _table(a, block_table, kv_len)
    _dense(row_req, "row_req", torch.int32, (n,))
    _dense(row_pos, "row_pos", torch.int32, (n,))
    _dense(out, "out", torch.bfloat16, (n, h, LATENT))
    _optional([("lse", lse, torch.float32, (n, h)), ("sink", sink, torch.float32, (h,)),
               ("status", status, torch.int32, (1,)), ("workspace", workspace, torch.uint8, (None,))])
    a.causal, a.window = 1 if causal else 0, _int32(window, "window")
    a.softmax_scale = float(softmax_scale)
    _pointers(a, tensors, [
        ("q", q), ("q_rope", q_rope), ("row_req", row_req), ("row_pos", row_pos),
        ("kv_len", kv_len), ("block_table", block_table), ("c_pool", c_pool), ("r_pool", r_pool),
        ("sink", sink), ("out", out), ("lse", lse)])
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_latent_attn", a, tensors, stream, prepare, workspace, sized=True)


def csa_latent_expand(*, c_pool, r_pool, block_table, kv_len, w_uk, w_uv, k_pool, v_pool,
                      out_table, first=None, status=None, stream=None, prepare=False):
    """Keys [pages, 128, heads, 192] and values [pages, 128, heads, 128] of every
    head from a paged latent cache and the up-projections ``w_uk``, ``w_uv`` [heads,
    128, 512] (``include/csa.h``: csa_latent_expand).  Position j of request b goes
    to slot j of ``out_table``; ``first`` (int32 [requests], default 0) skips the
    positions before it."""
    a, tensors = LatentExpandArgs(), []
    a.struct_size = ctypes.sizeof(a)
    _latent_pools(a, c_pool, r_pool)
    _table(a, block_table, kv_len)
    _dense(out_table, "out_table", torch.int32, (a.n_req, None))
    a.out_max_blocks = _int32(out_table.shape[1], "out_table")
    _optional([("first", first, torch.int32, (a.n_req,)), ("status", status, torch.int32, (1,))])
    h = None
    for name, w in (("w_uk", w_uk), ("w_uv", w_uv)):
        _want(w, name, torch.bfloat16, (h, NOPE if name == "w_uk" else VALUE, LATENT))
        h = int(w.shape[0])
        if w.stride(2) != 1 or w.stride(1) != LATENT:
            raise ValueError(f"{name}: a head's rows must be contiguous")
        if h > 1 and w.stride(0) < w.shape[1] * LATENT:
            raise ValueError(f"{name}: heads must not overlap")
        setattr(a, name + "_head_stride", (w.stride(0) if h > 1 else w.shape[1] * LATENT) * 2)
    a.n_heads = _int32(h, "w_uk")
    _want(k_pool, "k_pool", torch.bfloat16, (None, PAGE, h, NOPE + ROPE))
    _want(v_pool, "v_pool", torch.bfloat16, (k_pool.shape[0], PAGE, h, VALUE))
    a.n_out_blocks = _int32(k_pool.shape[0], "k_pool")
    _kv_strides(a, "k", k_pool, "k_pool")
    _kv_strides(a, "v", v_pool, "v_pool")
    _pointers(a, tensors, [
        ("kv_len", kv_len), ("first", first), ("block_table", block_table),
        ("out_table", out_table), ("c_pool", c_pool), ("r_pool", r_pool), ("w_uk", w_uk),
        ("w_uv", w_uv), ("k_pool", k_pool), ("v_pool", v_pool)])
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_latent_expand", a, tensors, stream, prepare)


def csa_attn_mass(*, q, lse, row_req, row_pos, k_pool, block_table, kv_len, mass=None,
                  mass_out=None, decay=1.0, softmax_scale=None, causal=True, window=0,
                  status=None, workspace=None, stream=None, prepare=False):
    """The attention weight that each cached position receives from the rows of
    ``q`` [rows, heads, dim] whose log-sums are ``lse`` [rows, heads], added to
    ``decay * mass`` [requests, 128 * pages a request] (``include/csa.h``:
    csa_attn_mass).  Without ``mass_out`` the sums replace ``mass``; ``decay`` 0 needs
    no ``mass``.  A position published since the last call starts from what its entry
    holds: 0 in a buffer that began as zeros, but not behind a cut (csa_kv_evict)."""
    a, tensors = AttnMassArgs(), []
    a.struct_size = ctypes.sizeof(a)
    a.q_row_stride = _rows(q, "q", (None, None, None))
    n, h, d = (int(x) for x in q.shape)
    a.n_rows, a.n_heads, a.head_dim = (_int32(x, "q") for x in (n, h, d))
    _want(k_pool, "k_pool", torch.bfloat16, (None, PAGE, None, d))
    a.n_blocks, a.n_kv_heads = _int32(k_pool.shape[0], "k_pool"), _int32(k_pool.shape[2], "k_pool")
    if a.n_kv_heads < 1 or h % a.n_kv_heads:
        raise ValueError(f"{h} query heads do not divide among {a.n_kv_heads} key heads")
    _kv_strides(a, "k", k_pool, "k_pool")
    _table(a, block_table, kv_len)
    _dense(lse, "lse", torch.float32, (n, h))
    _dense(row_req, "row_req", torch.int32, (n,))
    _dense(row_pos, "row_pos", torch.int32, (n,))
    mass_out = mass if mass_out is None else mass_out
    a.decay = float(decay)
    if mass_out is None or (mass is None and a.decay != 0.0):
        raise ValueError("mass is needed, or with decay 0 mass_out")
    shape = (a.n_req, a.max_blocks * PAGE)
    a.mass_out_row_stride = _float_rows(mass_out, "mass_out", shape)
    if mass is not None:
        a.mass_row_stride = _float_rows(mass, "mass", shape)
    _optional([("status", status, torch.int32, (1,)), ("workspace", workspace, torch.uint8, (None,))])
    a.causal, a.window = 1 if causal else 0, _int32(window, "window")
    a.softmax_scale = float(d ** -0.5 if softmax_scale is None else softmax_scale)
    _pointers(a, tensors, [
        ("q", q), ("lse", lse), ("row_req", row_req), ("row_pos", row_pos), ("kv_len", kv_len),
        ("block_table", block_table), ("k_pool", k_pool), ("mass", mass), ("mass_out", mass_out)])
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_attn_mass", a, tensors, stream, prepare, workspace, sized=True)


def csa_kv_evict(*, mass, kv_len, budget, block_table, k_pool, v_pool=None, kv_len_out=None,
                 first=0, recent=0, mass_out=None, slot_src=None, status=None, workspace=None,
                 stream=None, prepare=False):
    """Cuts every request's cache to its ``budget`` (int32 [requests]) heaviest
    positions by ``mass`` [requests, 128 * pages a request], in place
    (``include/csa.h``: csa_kv_evict).  The ``first`` and the last ``recent``
    positions stay as far as the budget goes.  ``kv_len_out`` (default: ``kv_len``
    itself) gets the new lengths, ``mass_out`` and ``slot_src`` each slot's mass and
    old position.  Entries of ``mass_out`` behind the new length keep what they held:
    set them to 0 before new positions are published there and weighed.  Pools are BF16 [pages, 128, heads, dim] (one head: [pages, 128,
    dim] too), keys and values of widths of their own."""
    a, tensors = KvEvictArgs(), []
    a.struct_size = ctypes.sizeof(a)

    def headed(t):
        return t.unsqueeze(2) if isinstance(t, torch.Tensor) and t.dim() == 3 else t

    k_pool, v_pool = headed(k_pool), headed(v_pool)
    _want(k_pool, "k_pool", torch.bfloat16, (None, PAGE, None, None))
    a.n_blocks, a.n_heads, a.k_dim = (_int32(k_pool.shape[i], "k_pool") for i in (0, 2, 3))
    _kv_strides(a, "k", k_pool, "k_pool")
    if v_pool is not None:
        _want(v_pool, "v_pool", torch.bfloat16, (k_pool.shape[0], PAGE, k_pool.shape[2], None))
        a.v_dim = _int32(v_pool.shape[3], "v_pool")
        _kv_strides(a, "v", v_pool, "v_pool")
    _table(a, block_table, kv_len)
    kv_len_out = kv_len if kv_len_out is None else kv_len_out
    shape = (a.n_req, a.max_blocks * PAGE)
    a.mass_row_stride = _float_rows(mass, "mass", shape)
    if mass_out is not None:
        a.mass_out_row_stride = _float_rows(mass_out, "mass_out", shape)
    _optional([("budget", budget, torch.int32, (a.n_req,)),
               ("kv_len_out", kv_len_out, torch.int32, (a.n_req,)),
               ("slot_src", slot_src, torch.int32, shape), ("status", status, torch.int32, (1,)),
               ("workspace", workspace, torch.uint8, (None,))])
    if budget is None:
        raise TypeError("budget must be a torch.Tensor, got NoneType")
    a.first, a.recent = _int32(first, "first"), _int32(recent, "recent")
    _pointers(a, tensors, [
        ("mass", mass), ("kv_len", kv_len), ("budget", budget), ("block_table", block_table),
        ("k_pool", k_pool), ("v_pool", v_pool), ("kv_len_out", kv_len_out),
        ("mass_out", mass_out), ("slot_src", slot_src)])
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_kv_evict", a, tensors, stream, prepare, workspace, sized=True)
