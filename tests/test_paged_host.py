"""Host side of the paged key/value cache operators (no GPU): struct layouts,
every refusal of the C entry points and of the binding, and pins of their
float64 definitions."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from test_abi_host import _c_layout

import prefill_csa_compress_gb300 as csa
from prefill_csa_compress_gb300 import _binding as B
from prefill_csa_compress_gb300 import _paged as P


@pytest.fixture(scope="module")
def L():
    from prefill_csa_compress_gb300 import build

    build.build()
    return B.lib()


@pytest.mark.parametrize("cname,S", [("csa_rope_table_args", P.RopeTableArgs),
                                     ("csa_qk_norm_rope_args", P.QkNormRopeArgs),
                                     ("csa_kv_append_args", P.KvAppendArgs),
                                     ("csa_paged_attn_args", P.PagedAttnArgs)])
def test_ctypes_layout_matches_c(cname, S):
    fields = [f for f, _ in S._fields_]
    got = _c_layout(cname, fields)
    assert got[0] == ctypes.sizeof(S)
    for f, off in zip(fields, got[1:]):
        assert getattr(S, f).offset == off, f


# one aligned host buffer stands for every tensor: a refused call never reads it
_buf = ctypes.create_string_buffer(4096)
_base = (ctypes.addressof(_buf) + 255) // 256 * 256

ROPE = dict(rope_dim=64, n_pos=16, theta=1e4, factor=1.0, attn_factor=1.0, cos=_base, sin=_base)
QK = dict(n_rows=4, n_q_heads=8, n_k_heads=2, head_dim=128, norm=1, eps=1e-6, rope_start=64,
          rope_dim=64, rope_cap=128, q=_base, k=_base, q_out=_base, k_out=_base, row_pos=_base,
          rope_cos=_base, rope_sin=_base)
APPEND = dict(n_rows=4, n_heads=2, head_dim=128, fmt=B.CSA_FMT_BF16, norm=1, eps=1e-6,
              rope_start=0, rope_dim=128, rope_cap=128, n_req=2, max_blocks=4, n_blocks=8,
              k=_base, v=_base, row_req=_base, row_pos=_base, rope_cos=_base, rope_sin=_base,
              block_table=_base, k_pool=_base, v_pool=_base)
ATTN = dict(n_rows=4, n_heads=8, n_kv_heads=2, head_dim=128, causal=1, softmax_scale=0.1, n_req=2,
            max_blocks=4, n_blocks=8, q=_base, row_req=_base, row_pos=_base, kv_len=_base,
            block_table=_base, k_pool=_base, v_pool=_base, out=_base, workspace=_base,
            workspace_bytes=1 << 40)
FP8 = dict(fmt=B.CSA_FMT_MXFP8, k_scale_pool=_base, v_scale_pool=_base)
INVALID, UNSUPPORTED = B.CSA_ERR_INVALID_ARG, B.CSA_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")

REFUSED = [
    ("csa_rope_table", ROPE, INVALID, [
        dict(struct_size=8), dict(n_pos=-1), dict(pos0=-1), dict(pos0=2 ** 31 - 1), dict(theta=1.0),
        dict(theta=NAN), dict(theta=INF), dict(attn_factor=0.0), dict(attn_factor=INF),
        dict(scaling=4), dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=2, factor=NAN),
        dict(scaling=3, factor=2.0), dict(scaling=3, factor=2.0, orig_len=64, beta_fast=1.0, beta_slow=2.0),
        dict(scaling=3, factor=2.0, orig_len=64, beta_fast=1.0, beta_slow=0.0),
        dict(cos=None), dict(sin=None), dict(cos=_base + 2)]),
    ("csa_rope_table", ROPE, UNSUPPORTED, [
        dict(rope_dim=0), dict(rope_dim=3), dict(rope_dim=514), dict(scaling=2, rope_dim=2, factor=2.0)]),
    ("csa_qk_norm_rope", QK, INVALID, [
        dict(struct_size=8), dict(n_rows=-1), dict(n_q_heads=0), dict(n_k_heads=-1),
        dict(norm=2), dict(eps=-1.0), dict(eps=NAN), dict(rope_sin=None), dict(rope_layout=2),
        dict(rope_cap=0), dict(rope_dim=0), dict(rope_start=-8), dict(rope_start=72),
        dict(rope_dim=136), dict(rope_cos=_base + 8), dict(q_row_stride=8 * 256 - 16),
        dict(q_row_stride=8 * 256 + 8), dict(k_row_stride=16), dict(q_out_row_stride=-2048),
        dict(k_out_row_stride=520), dict(q=None), dict(k=None), dict(q_out=None), dict(k_out=None),
        dict(row_pos=None), dict(q=_base + 8), dict(k_out=_base + 2), dict(q_gamma=_base + 8)]),
    ("csa_qk_norm_rope", QK, UNSUPPORTED, [
        dict(head_dim=0), dict(head_dim=520), dict(head_dim=132), dict(rope_start=4, rope_dim=64),
        dict(rope_start=0, rope_dim=12), dict(rope_start=0, rope_dim=24, rope_layout=1)]),
    ("csa_kv_append", APPEND, INVALID, [
        dict(struct_size=8), dict(n_rows=-1), dict(n_heads=0), dict(n_req=0), dict(max_blocks=0),
        dict(n_blocks=0), dict(norm=-1), dict(k=None), dict(row_req=None), dict(row_pos=None),
        dict(block_table=None), dict(k_pool=None), dict(v_pool=None), dict(k=_base + 8),
        dict(v=_base + 8), dict(v_pool=_base + 8), dict(k_gamma=_base + 2), dict(k_row_stride=256),
        dict(v_row_stride=520), dict(k_token_stride=256), dict(k_token_stride=520),
        dict(v_page_stride=512), dict(k_head_stride=-256), dict(k_head_stride=512),
        dict(FP8, k_scale_pool=None), dict(FP8, v_scale_pool=None), dict(rope_dim=144)]),
    ("csa_kv_append", APPEND, UNSUPPORTED, [
        dict(fmt=B.CSA_FMT_INT8), dict(fmt=9), dict(head_dim=516), dict(FP8, head_dim=120, rope_dim=64),
        dict(FP8, k_page_stride=1 << 20), dict(FP8, v_head_stride=256)]),
    ("csa_paged_attn", ATTN, INVALID, [
        dict(struct_size=8), dict(n_rows=-1), dict(n_req=0), dict(max_blocks=0), dict(n_blocks=0),
        dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(causal=2), dict(window=-1),
        dict(mode=3), dict(mode=-1), dict(softmax_scale=0.0), dict(softmax_scale=-1.0),
        dict(softmax_scale=NAN), dict(softmax_scale=INF), dict(q_row_stride=256),
        dict(k_token_stride=256), dict(v_head_stride=8), dict(k_page_stride=128),
        dict(workspace=_base + 16), dict(q=None), dict(row_req=None), dict(row_pos=None),
        dict(kv_len=None), dict(block_table=None), dict(k_pool=None), dict(v_pool=None),
        dict(out=None), dict(q=_base + 8), dict(out=_base + 8), dict(k_pool=_base + 8)]),
    ("csa_paged_attn", ATTN, UNSUPPORTED, [
        dict(head_dim=32), dict(head_dim=256), dict(n_heads=129, n_kv_heads=1), dict(n_rows=(1 << 24) + 1)]),
]


@pytest.mark.parametrize("name,base,status,change", [
    (n, b, s, c) for n, b, s, cs in REFUSED for c in cs],
    ids=lambda v: ",".join(f"{k}={x}" for k, x in v.items() if k != "cos")[:60] if isinstance(v, dict) and len(v) < 9 else None)
def test_refusals(L, name, base, status, change):
    a = P._CALLS[name]()
    a.struct_size = ctypes.sizeof(a)
    for k, v in {**base, **change}.items():
        setattr(a, k, v)
    assert P._fn(name)(ctypes.byref(a), None) == status


@pytest.mark.parametrize("name,base", [("csa_rope_table", dict(ROPE, n_pos=0)),
                                       ("csa_qk_norm_rope", dict(QK, n_rows=0)),
                                       ("csa_kv_append", dict(APPEND, n_rows=0)),
                                       ("csa_paged_attn", dict(ATTN, n_rows=0))])
def test_nothing_to_do_is_ok(L, name, base):
    a = P._CALLS[name]()
    a.struct_size = ctypes.sizeof(a)
    for k, v in base.items():
        setattr(a, k, v)
    before = csa.launch_count()
    assert P._fn(name)(ctypes.byref(a), None) == B.CSA_OK
    assert P._fn(name)(None, None) == INVALID
    assert csa.launch_count() == before


def test_attention_size_query(L):
    a = P.PagedAttnArgs()
    a.struct_size = ctypes.sizeof(a)
    for k, v in dict(ATTN, workspace=None, workspace_bytes=77).items():
        setattr(a, k, v)
    assert P._fn("csa_paged_attn")(ctypes.byref(a), None) == B.CSA_OK
    need = a.workspace_bytes
    assert need != 77
    if need:
        a.workspace, a.workspace_bytes = _base, need - 1
        assert P._fn("csa_paged_attn")(ctypes.byref(a), None) == INVALID


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_binding_refusals():
    """Shapes, dtypes and layouts are refused before any device is asked for;
    a call that is right but for its CPU tensors is refused last."""
    f32 = torch.zeros((16, 32))
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_rope_table(cos=f32, sin=f32.clone())
    with pytest.raises(ValueError, match="scaling"):
        csa.csa_rope_table(cos=f32, sin=f32, scaling="wide")
    with pytest.raises(ValueError, match="sin must have shape"):
        csa.csa_rope_table(cos=f32, sin=f32[:8])
    with pytest.raises(TypeError, match="cos must be"):
        csa.csa_rope_table(cos=f32.double(), sin=f32)

    qk = dict(q=_bf(4, 8, 64), row_pos=_i(4), k=_bf(4, 2, 64), rope_cos=f32, rope_sin=f32)
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_qk_norm_rope(**qk)
    for change, why in [(dict(q=_bf(4, 64)), "shape"), (dict(q=_bf(4, 64, 8).transpose(1, 2)), "contiguous"),
                        (dict(k=_bf(4, 2, 32)), "shape"), (dict(k=_bf(3, 2, 64)), "shape"),
                        (dict(q_out=_bf(4, 7, 64)), "shape"), (dict(row_pos=_i(5)), "shape"),
                        (dict(row_req=_i(3)), "shape"), (dict(q_gamma=_bf(32)), "shape"),
                        (dict(norm=False, q_gamma=_bf(64)), "norm"), (dict(k=None, k_gamma=_bf(64)), "need k"),
                        (dict(q=_bf(1, 8, 64).expand(4, 8, 64)), "overlap")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_qk_norm_rope(**{**qk, **change})
    with pytest.raises(TypeError, match="row_pos must be"):
        csa.csa_qk_norm_rope(**{**qk, "row_pos": _i(4).long()})
    with pytest.raises(TypeError, match="q must be"):
        csa.csa_qk_norm_rope(**{**qk, "q": _bf(4, 8, 64).half()})

    ap = dict(k=_bf(4, 2, 64), v=_bf(4, 2, 64), row_req=_i(4), row_pos=_i(4), block_table=_i(2, 3),
              k_pool=_bf(5, 128, 2, 64), v_pool=_bf(5, 128, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_kv_append(**ap)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    for change, why in [(dict(v=None), "together"), (dict(v_pool=None), "together"),
                        (dict(v=_bf(4, 1, 64)), "shape"), (dict(k_pool=_bf(5, 64, 2, 64)), "shape"),
                        (dict(v_pool=_bf(4, 128, 2, 64)), "shape"), (dict(row_req=_i(5)), "shape"),
                        (dict(block_table=_i(6)), "shape"), (dict(k_gamma=_bf(64)), "norm"),
                        (dict(k_scale_pool=u8(5, 128, 2, 2)), "scale pools"),
                        (dict(v_scale_pool=u8(5, 128, 2, 2)), "scale pools"),
                        (dict(k_pool=_bf(1, 128, 2, 64).expand(5, 128, 2, 64)), "overlap"),
                        (dict(k_pool=_bf(5, 128, 64, 2).transpose(2, 3)), "contiguous")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_kv_append(**{**ap, **change})
    with pytest.raises(TypeError, match="k_pool must be"):
        csa.csa_kv_append(**{**ap, "k_scale_pool": u8(5, 128, 2, 2), "v_scale_pool": u8(5, 128, 2, 2)})

    at = dict(q=_bf(4, 8, 64), row_req=_i(4), row_pos=_i(4), k_pool=_bf(5, 128, 2, 64),
              v_pool=_bf(5, 128, 2, 64), block_table=_i(2, 3), kv_len=_i(2), out=_bf(4, 8, 64))
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_paged_attn(**at)
    for change, why in [(dict(q=_bf(4, 7, 64), out=_bf(4, 7, 64)), "divide"), (dict(kv_len=_i(3)), "shape"),
                        (dict(v_pool=_bf(5, 128, 1, 64)), "shape"), (dict(lse=torch.zeros(4, 7)), "shape"),
                        (dict(out=_bf(4, 8, 128)[..., :64]), "contiguous"), (dict(sink=torch.zeros(2)), "shape"),
                        (dict(block_table=_i(2, 6)[:, ::2]), "contiguous")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_paged_attn(**{**at, **change})
    for change in (dict(window=2 ** 32 + 1), dict(mode=2 ** 32)):
        with pytest.raises(ValueError, match="32 bits"):
            csa.csa_paged_attn(**{**at, **change})
    with pytest.raises(ValueError, match="32 bits"):
        csa.csa_rope_table(cos=f32, sin=f32.clone(), pos0=2 ** 32)
    with pytest.raises(TypeError, match="sink must be"):
        csa.csa_paged_attn(**{**at, "sink": torch.zeros(8).double()})


# ---------------------------------------------------------------- the definitions


def test_rope_definition():
    f = PO.rope_frequencies(8, theta=100.0)
    assert np.allclose(f, [1, 100 ** -0.25, 100 ** -0.5, 100 ** -0.75])
    assert np.allclose(PO.rope_frequencies(8, theta=100.0, scaling="linear", factor=4.0), f / 4)
    # NTK: the fastest pair keeps its rotation, the slowest is stretched by the factor
    n = PO.rope_frequencies(64, scaling="ntk", factor=8.0)
    g = PO.rope_frequencies(64)
    assert n[0] == 1.0 and np.isclose(n[-1], g[-1] / 8.0)
    # the ramp: untouched where a pair turns > beta_fast times, divided where < beta_slow
    y = PO.rope_frequencies(64, scaling="yarn", factor=8.0, orig_len=4096)
    turns = g * 4096 / (2 * math.pi)
    assert np.array_equal(y[turns > 40], g[turns > 40])
    assert np.allclose(y[turns < 0.7], g[turns < 0.7] / 8.0, rtol=1e-14)
    assert np.all(y <= g) and np.all(y >= g / 8.0 * (1 - 1e-14))
    c, s = PO.rope_table(5, 8, pos0=7, attn_factor=2.0, theta=100.0)
    assert np.allclose(c[2], 2 * np.cos(9 * f)) and np.allclose(s[0], 2 * np.sin(7 * f))


@pytest.mark.parametrize("layout", ["adjacent", "half"])
def test_rotation_definition(layout):
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 16))
    c, s = PO.rope_table(50, 8, theta=100.0)
    y = PO.norm_rotate(x, [5, -1, 50], norm=False, cos=c, sin=s, layout=layout, start=4)
    assert np.array_equal(y[1:], x[1:])  # no position, past the tables
    assert np.array_equal(y[0, :, :4], x[0, :, :4]) and np.array_equal(y[0, :, 12:], x[0, :, 12:])
    r, z = x[0, :, 4:12], y[0, :, 4:12]
    a, b = (slice(0, 8, 2), slice(1, 8, 2)) if layout == "adjacent" else (slice(0, 4), slice(4, 8))
    got, want = z[:, a] + 1j * z[:, b], (r[:, a] + 1j * r[:, b]) * (c[5] + 1j * s[5])
    assert np.allclose(got, want)
    n = PO.norm_rotate(x, [0, 0, 0], eps=0.0, gamma=np.full(16, 3.0))
    assert np.allclose(np.sqrt(np.mean(n * n, -1)), 3.0)


def test_attention_definition():
    rng = np.random.default_rng(1)
    k, v = rng.standard_normal((2, 4, 128, 2, 8))
    q = rng.standard_normal((3, 4, 8))
    table, lens = np.array([[2, 0], [3, -1]]), [200, 90]
    o, lse, _ = PO.paged_attention(q, [0, 1, 1], [150, 20, 89], k, v, table, lens, 0.5, window=30)
    seq = np.concatenate([k[2], k[0]]), np.concatenate([v[2], v[0]])
    x = torch.from_numpy(0.5 * seq[0][121:151, 1] @ q[0, 3])
    assert np.allclose(o[0, 3], torch.softmax(x, 0).numpy() @ seq[1][121:151, 1])
    assert np.isclose(lse[0, 3], float(torch.logsumexp(x, 0)))
    # a sink is one more logit without a value; one seen position gives v * sigma(l - sink)
    o, lse, _ = PO.paged_attention(q[1:2], [1], [0], k, v, table, lens, 0.5, sink=[0.3] * 4)
    x = 0.5 * k[3, 0, 0] @ q[1, 0]
    assert np.allclose(o[0, 0], v[3, 0, 0] / (1 + math.exp(0.3 - x)))
    # nothing seen
    o, lse, _ = PO.paged_attention(q[:1], [0], [-1], k, v, table, lens, 0.5, sink=[0.3] * 4)
    assert not o.any() and np.allclose(lse, 0.3)
    assert PO.visible(10, 5) == (0, 5) and PO.visible(-1, 5) == (0, 0)
    assert PO.visible(10, 50, window=1) == (10, 11) and PO.visible(10, 50, causal=False, window=3) == (8, 50)
    assert PO.visible(40, 20, window=4) == (37, 37)


def test_mxfp8_exponent_definition():
    for amax, e in ((448.0, 0), (448.1, 1), (447.0, 0), (224.0, -1), (1.75, -8), (1.7501, -7), (0.0, -127)):
        assert PO.mxfp8_exponent(np.array([0.0, -amax])) == e
