"""ctypes binding of the paged key/value cache operators: ``csa_rope_table``,
``csa_qk_norm_rope``, ``csa_kv_append`` and ``csa_paged_attn`` of
``include/csa.h`` (argument marshalling only).

Shapes, dtypes and strides are checked here, before anything reaches the
library; tensors must lie on one CUDA device, which need not be the current
one.  ``stream`` is a ``torch.cuda.Stream`` of that device (default: its current
stream); the caller orders it with the streams that made the tensors.  With
``prepare=True`` a call is marshalled once and returned: calling it only crosses
the C ABI, for tensors that stay in place (the prepared call keeps them alive).
"""

from __future__ import annotations

import ctypes
from ctypes import c_double, c_float, c_int32, c_int64, c_size_t, c_uint32, c_void_p

import torch

from . import _binding as B

PAGE = 128


class RopeTableArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("rope_dim", c_int32), ("n_pos", c_int32), ("pos0", c_int32),
        ("scaling", c_int32), ("orig_len", c_int32), ("theta", c_double), ("factor", c_double),
        ("beta_fast", c_double), ("beta_slow", c_double), ("attn_factor", c_double),
        ("cos", c_void_p), ("sin", c_void_p),
    ]


class QkNormRopeArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_rows", c_int32), ("n_q_heads", c_int32),
        ("n_k_heads", c_int32), ("head_dim", c_int32), ("norm", c_int32), ("eps", c_float),
        ("rope_layout", c_int32), ("rope_start", c_int32), ("rope_dim", c_int32),
        ("rope_cap", c_int32), ("q", c_void_p), ("k", c_void_p), ("q_out", c_void_p),
        ("k_out", c_void_p), ("q_row_stride", c_int64), ("k_row_stride", c_int64),
        ("q_out_row_stride", c_int64), ("k_out_row_stride", c_int64), ("q_gamma", c_void_p),
        ("k_gamma", c_void_p), ("row_pos", c_void_p), ("row_req", c_void_p),
        ("rope_cos", c_void_p), ("rope_sin", c_void_p), ("status_dev", c_void_p),
    ]


class KvAppendArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_rows", c_int32), ("n_heads", c_int32),
        ("head_dim", c_int32), ("fmt", c_int32), ("norm", c_int32), ("eps", c_float),
        ("rope_layout", c_int32), ("rope_start", c_int32), ("rope_dim", c_int32),
        ("rope_cap", c_int32), ("n_req", c_int32), ("max_blocks", c_int32),
        ("n_blocks", c_int32), ("k", c_void_p), ("v", c_void_p), ("k_row_stride", c_int64),
        ("v_row_stride", c_int64), ("k_gamma", c_void_p), ("row_req", c_void_p),
        ("row_pos", c_void_p), ("rope_cos", c_void_p), ("rope_sin", c_void_p),
        ("block_table", c_void_p), ("k_pool", c_void_p), ("v_pool", c_void_p),
        ("k_scale_pool", c_void_p), ("v_scale_pool", c_void_p), ("k_page_stride", c_int64),
        ("k_token_stride", c_int64), ("k_head_stride", c_int64), ("v_page_stride", c_int64),
        ("v_token_stride", c_int64), ("v_head_stride", c_int64), ("status_dev", c_void_p),
    ]


class PagedAttnArgs(ctypes.Structure):
    _fields_ = [
        ("struct_size", c_uint32), ("n_rows", c_int32), ("n_heads", c_int32),
        ("n_kv_heads", c_int32), ("head_dim", c_int32), ("causal", c_int32),
        ("window", c_int32), ("mode", c_int32), ("softmax_scale", c_float), ("n_req", c_int32),
        ("max_blocks", c_int32), ("n_blocks", c_int32), ("q", c_void_p),
        ("q_row_stride", c_int64), ("row_req", c_void_p), ("row_pos", c_void_p),
        ("kv_len", c_void_p), ("block_table", c_void_p), ("k_pool", c_void_p),
        ("v_pool", c_void_p), ("k_page_stride", c_int64), ("k_token_stride", c_int64),
        ("k_head_stride", c_int64), ("v_page_stride", c_int64), ("v_token_stride", c_int64),
        ("v_head_stride", c_int64), ("sink", c_void_p), ("out", c_void_p), ("lse", c_void_p),
        ("status_dev", c_void_p), ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


_CALLS = {"csa_rope_table": RopeTableArgs, "csa_qk_norm_rope": QkNormRopeArgs,
          "csa_kv_append": KvAppendArgs, "csa_paged_attn": PagedAttnArgs}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_LAYOUTS = {"adjacent": 0, "half": 1}


def _fn(name):
    f = getattr(B.lib(), name)
    if f.argtypes is None:
        f.argtypes = [ctypes.POINTER(_CALLS[name]), c_void_p]
        f.restype = c_int32
    return f


# ---------------------------------------------------------------- checks


def _want(t, name, dtype, shape):
    """Checks a tensor's kind, dtype and shape (None matches any size)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != len(shape) or any(w is not None and int(g) != w
                                    for g, w in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _dense(t, name, dtype, shape):
    _want(t, name, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _rows(t, name, shape):
    """A BF16 [rows, heads, dim] tensor whose rows may be strided; returns its
    row stride in bytes."""
    _want(t, name, torch.bfloat16, shape)
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    if n <= 1:
        return h * d * 2
    if t.stride(0) < h * d:
        raise ValueError(f"{name}: rows must not overlap")
    return t.stride(0) * 2


def _pool_strides(t, name):
    """Page, token and head strides in bytes of a BF16 pool [pages, 128,
    heads, dim] (a row's channels contiguous)."""
    n, _, h, d = t.shape
    if d > 1 and t.stride(3) != 1:
        raise ValueError(f"{name}: a head's channels must be contiguous")
    page, token, head = t.stride(0), t.stride(1), t.stride(2)
    if h == 1:
        head = d
    if n == 1:
        page = max(PAGE * token, h * head)
    if min(page, token, head) < d:
        raise ValueError(f"{name}: rows must not overlap")
    return page * 2, token * 2, head * 2


def _int32(x, name):
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit 32 bits, got {x}")
    return x


def _ptr(tensors, name, t):
    """The address of a checked tensor, noting its device."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if tensors and tensors[0].device != t.device:
        raise ValueError(f"{name} is on {t.device}, other tensors on {tensors[0].device}")
    tensors.append(t)
    return t.data_ptr()


def _rope(a, tensors, cos, sin, layout, start, dim):
    if (cos is None) != (sin is None):
        raise ValueError("rope_cos and rope_sin go together")
    if cos is None:
        return
    if layout not in _LAYOUTS:
        raise ValueError(f"rope_layout must be one of {sorted(_LAYOUTS)}, got {layout!r}")
    _dense(cos, "rope_cos", torch.float32, (None, None))
    _dense(sin, "rope_sin", torch.float32, tuple(cos.shape))
    a.rope_layout = _LAYOUTS[layout]
    a.rope_cap, a.rope_dim = _int32(cos.shape[0], "rope_cos"), _int32(2 * cos.shape[1], "rope_cos")
    if not 0 < a.rope_dim <= dim:
        raise ValueError(f"the tables rotate {a.rope_dim} channels of a head of {dim}")
    a.rope_start = dim - a.rope_dim if start is None else _int32(start, "rope_start")
    a.rope_cos, a.rope_sin = _ptr(tensors, "rope_cos", cos), _ptr(tensors, "rope_sin", sin)


# ---------------------------------------------------------------- launching


class _Call(B.PreparedCall):
    """A marshalled call on the device of its tensors, which it keeps alive."""

    def __init__(self, fn_name, args, workspace, tensors):
        _fn(fn_name)
        super().__init__(fn_name, args, workspace)
        self.tensors = tuple(tensors)
        self.device = tensors[0].device

    def __call__(self, stream=None):
        if stream is not None and stream.device != self.device:
            raise ValueError(f"{self.fn_name}: the stream is on {stream.device}, the tensors on "
                             f"{self.device}")
        index = self.device.index
        if torch.cuda.current_device() != index:
            with torch.cuda.device(index):
                return self(stream)
        # (the raw handle: a Stream object costs more than the launch)
        raw = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
        st = self.fn(*self._refs, raw)
        if st != B.CSA_OK:
            raise B.CsaError(self.fn_name, st)
        return self.workspace


def _launch(fn_name, a, tensors, stream, prepare, workspace=None, sized=False):
    if sized:
        with torch.cuda.device(tensors[0].device):
            a.workspace, a.workspace_bytes = None, 0
            st = _fn(fn_name)(ctypes.byref(a), None)  # size query
            if st != B.CSA_OK:
                raise B.CsaError(fn_name, st)
            need = int(a.workspace_bytes)
            if workspace is None or workspace.numel() < need:
                # allocated on the stream that uses it, so that it is not
                # handed to another while the call still runs
                with torch.cuda.stream(stream):
                    workspace = torch.empty(max(need, 256), dtype=torch.uint8,
                                            device=tensors[0].device)
        a.workspace = _ptr(tensors, "workspace", workspace)
        a.workspace_bytes = workspace.numel()
    call = _Call(fn_name, a, workspace, tensors)
    return call if prepare else call(stream)


def csa_rope_table(*, cos, sin, theta=10000.0, scaling="none", factor=1.0, orig_len=0,
                   beta_fast=32.0, beta_slow=1.0, attn_factor=1.0, pos0=0, stream=None,
                   prepare=False):
    """Fills FP32 ``cos`` and ``sin`` [n_pos, rope_dim / 2] with the tables of
    the positions ``pos0`` .. (``include/csa.h``: csa_rope_table).  ``scaling``
    is "none", "linear", "ntk" or "yarn"."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {sorted(_SCALINGS)}, got {scaling!r}")
    _dense(cos, "cos", torch.float32, (None, None))
    _dense(sin, "sin", torch.float32, tuple(cos.shape))
    a, tensors = RopeTableArgs(), []
    a.struct_size = ctypes.sizeof(a)
    a.n_pos, a.rope_dim = _int32(cos.shape[0], "cos"), _int32(2 * cos.shape[1], "cos")
    a.pos0 = _int32(pos0, "pos0")
    a.scaling, a.orig_len = _SCALINGS[scaling], _int32(orig_len, "orig_len")
    a.theta, a.factor, a.attn_factor = float(theta), float(factor), float(attn_factor)
    a.beta_fast, a.beta_slow = float(beta_fast), float(beta_slow)
    a.cos, a.sin = _ptr(tensors, "cos", cos), _ptr(tensors, "sin", sin)
    return _launch("csa_rope_table", a, tensors, stream, prepare)


def csa_qk_norm_rope(*, q, row_pos, k=None, q_out=None, k_out=None, row_req=None, norm=True,
                     q_gamma=None, k_gamma=None, eps=1e-6, rope_cos=None, rope_sin=None,
                     rope_layout="adjacent", rope_start=None, status=None, stream=None,
                     prepare=False):
    """RMS norm and rotation of every head of ``q`` [rows, heads, dim] and
    ``k`` (or None) in one pass (``include/csa.h``: csa_qk_norm_rope).  Without
    ``q_out`` / ``k_out`` the heads are replaced in place.  The tables' width
    gives the rotated channels; ``rope_start`` (default: the last ones) says
    where they begin.  ``rope_layout`` is "adjacent" or "half"."""
    a, tensors = QkNormRopeArgs(), []
    a.struct_size = ctypes.sizeof(a)
    q_out = q if q_out is None else q_out
    a.q_row_stride = _rows(q, "q", (None, None, None))
    n, h, d = (int(x) for x in q.shape)
    a.n_rows, a.n_q_heads, a.head_dim = (_int32(x, "q") for x in (n, h, d))
    a.q_out_row_stride = _rows(q_out, "q_out", (n, h, d))
    if k is not None:
        k_out = k if k_out is None else k_out
        a.k_row_stride = _rows(k, "k", (n, None, d))
        a.n_k_heads = _int32(k.shape[1], "k")
        a.k_out_row_stride = _rows(k_out, "k_out", tuple(k.shape))
    elif k_out is not None or k_gamma is not None:
        raise ValueError("k_out and k_gamma need k")
    _dense(row_pos, "row_pos", torch.int32, (n,))
    for name, x, dtype, shape in (("row_req", row_req, torch.int32, (n,)),
                                  ("q_gamma", q_gamma, torch.bfloat16, (d,)),
                                  ("k_gamma", k_gamma, torch.bfloat16, (d,)),
                                  ("status", status, torch.int32, (1,))):
        if x is not None:
            _dense(x, name, dtype, shape)
    if not norm and (q_gamma is not None or k_gamma is not None):
        raise ValueError("gammas need norm")
    a.norm, a.eps = 1 if norm else 0, float(eps)
    a.q, a.q_out = _ptr(tensors, "q", q), _ptr(tensors, "q_out", q_out)
    a.k = _ptr(tensors, "k", k)
    a.k_out = _ptr(tensors, "k_out", k_out) if k is not None else None
    a.q_gamma, a.k_gamma = _ptr(tensors, "q_gamma", q_gamma), _ptr(tensors, "k_gamma", k_gamma)
    a.row_pos, a.row_req = _ptr(tensors, "row_pos", row_pos), _ptr(tensors, "row_req", row_req)
    _rope(a, tensors, rope_cos, rope_sin, rope_layout, rope_start, d)
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_qk_norm_rope", a, tensors, stream, prepare)


def csa_kv_append(*, k, row_req, row_pos, block_table, k_pool, v=None, v_pool=None,
                  k_scale_pool=None, v_scale_pool=None, norm=False, k_gamma=None, eps=1e-6,
                  rope_cos=None, rope_sin=None, rope_layout="adjacent", rope_start=None,
                  status=None, stream=None, prepare=False):
    """Publishes the rows of ``k`` [rows, heads, dim] (normed and rotated on
    the way) and ``v`` (or None) in paged caches (``include/csa.h``:
    csa_kv_append).  Pools are BF16 [pages, 128, heads, dim], strided views
    included, or with scale pools (uint8 [pages, 128, heads, dim / 32]) MXFP8
    codes (uint8 [pages, 128, heads, dim]).  A pool of one head may come
    without its head dimension ([pages, 128, dim], scales [pages, 128, dim / 32])."""
    a, tensors = KvAppendArgs(), []
    a.struct_size = ctypes.sizeof(a)
    a.k_row_stride = _rows(k, "k", (None, None, None))
    n, h, d = (int(x) for x in k.shape)
    a.n_rows, a.n_heads, a.head_dim = (_int32(x, "k") for x in (n, h, d))
    if (v is None) != (v_pool is None):
        raise ValueError("v and v_pool go together")
    if v is not None:
        a.v_row_stride = _rows(v, "v", (n, h, d))
    low = k_scale_pool is not None
    if (v_scale_pool is not None) != (low and v is not None):
        raise ValueError("scale pools go with every MXFP8 pool, and with no other")
    a.fmt = B.CSA_FMT_MXFP8 if low else B.CSA_FMT_BF16

    def headed(t):
        return t.unsqueeze(2) if isinstance(t, torch.Tensor) and t.dim() == 3 and h == 1 else t

    k_pool, v_pool = headed(k_pool), headed(v_pool)
    k_scale_pool, v_scale_pool = headed(k_scale_pool), headed(v_scale_pool)
    pages = None
    for name, x, sc in (("k_pool", k_pool, k_scale_pool), ("v_pool", v_pool, v_scale_pool)):
        if name == "v_pool" and v is None:
            continue
        if low:
            _dense(x, name, torch.uint8, (pages, PAGE, h, d))
            _dense(sc, name.replace("pool", "scale_pool"), torch.uint8,
                   (x.shape[0], PAGE, h, d // 32))
        else:
            _want(x, name, torch.bfloat16, (pages, PAGE, h, d))
            st = _pool_strides(x, name)
            p = name[0]
            setattr(a, p + "_page_stride", st[0])
            setattr(a, p + "_token_stride", st[1])
            setattr(a, p + "_head_stride", st[2])
        pages = int(x.shape[0])
    a.n_blocks = _int32(pages, "pools")
    _dense(row_req, "row_req", torch.int32, (n,))
    _dense(row_pos, "row_pos", torch.int32, (n,))
    _dense(block_table, "block_table", torch.int32, (None, None))
    a.n_req, a.max_blocks = (_int32(x, "block_table") for x in block_table.shape)
    if k_gamma is not None:
        if not norm:
            raise ValueError("k_gamma needs norm")
        _dense(k_gamma, "k_gamma", torch.bfloat16, (d,))
    if status is not None:
        _dense(status, "status", torch.int32, (1,))
    a.norm, a.eps = 1 if norm else 0, float(eps)
    for name, x in (("k", k), ("v", v), ("k_gamma", k_gamma), ("row_req", row_req),
                    ("row_pos", row_pos), ("block_table", block_table), ("k_pool", k_pool),
                    ("v_pool", v_pool), ("k_scale_pool", k_scale_pool),
                    ("v_scale_pool", v_scale_pool)):
        setattr(a, name, _ptr(tensors, name, x))
    _rope(a, tensors, rope_cos, rope_sin, rope_layout, rope_start, d)
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_kv_append", a, tensors, stream, prepare)


def csa_paged_attn(*, q, row_req, row_pos, k_pool, v_pool, block_table, kv_len, out, lse=None,
                   sink=None, softmax_scale=None, causal=True, window=0, mode=B.CSA_MODE_AUTO,
                   status=None, workspace=None, stream=None, prepare=False):
    """Attention of the rows of ``q`` [rows, heads, dim] over paged keys and
    values [pages, 128, kv_heads, dim] (``include/csa.h``: csa_paged_attn).
    Returns the workspace, which a later call of the same sizes may be given;
    calls that overlap need one each.  ``mode`` (CSA_MODE_*) names the kernel;
    left to itself the call takes the rows as spread evenly over the block
    table's requests and the caches as long as its rows."""
    a, tensors = PagedAttnArgs(), []
    a.struct_size = ctypes.sizeof(a)
    a.q_row_stride = _rows(q, "q", (None, None, None))
    n, h, d = (int(x) for x in q.shape)
    a.n_rows, a.n_heads, a.head_dim = (_int32(x, "q") for x in (n, h, d))
    _want(k_pool, "k_pool", torch.bfloat16, (None, PAGE, None, d))
    _want(v_pool, "v_pool", torch.bfloat16, tuple(k_pool.shape))
    a.n_blocks, a.n_kv_heads = _int32(k_pool.shape[0], "pools"), _int32(k_pool.shape[2], "pools")
    if a.n_kv_heads < 1 or h % a.n_kv_heads:
        raise ValueError(f"{h} query heads do not divide among {a.n_kv_heads} key/value heads")
    a.k_page_stride, a.k_token_stride, a.k_head_stride = _pool_strides(k_pool, "k_pool")
    a.v_page_stride, a.v_token_stride, a.v_head_stride = _pool_strides(v_pool, "v_pool")
    _dense(block_table, "block_table", torch.int32, (None, None))
    a.n_req, a.max_blocks = (_int32(x, "block_table") for x in block_table.shape)
    _dense(kv_len, "kv_len", torch.int32, (a.n_req,))
    _dense(row_req, "row_req", torch.int32, (n,))
    _dense(row_pos, "row_pos", torch.int32, (n,))
    _dense(out, "out", torch.bfloat16, (n, h, d))
    for name, x, dtype, shape in (("lse", lse, torch.float32, (n, h)),
                                  ("sink", sink, torch.float32, (h,)),
                                  ("status", status, torch.int32, (1,)),
                                  ("workspace", workspace, torch.uint8, (None,))):
        if x is not None:
            _dense(x, name, dtype, shape)
    a.causal, a.window = 1 if causal else 0, _int32(window, "window")
    a.mode = _int32(mode, "mode")
    a.softmax_scale = float(d ** -0.5 if softmax_scale is None else softmax_scale)
    for name, x in (("q", q), ("row_req", row_req), ("row_pos", row_pos), ("kv_len", kv_len),
                    ("block_table", block_table), ("k_pool", k_pool), ("v_pool", v_pool),
                    ("sink", sink), ("out", out), ("lse", lse)):
        setattr(a, name, _ptr(tensors, name, x))
    a.status_dev = _ptr(tensors, "status", status)
    return _launch("csa_paged_attn", a, tensors, stream, prepare, workspace, sized=True)
