"""Host side of the latent cache and eviction calls (no GPU): struct layouts, every
refusal of the C entry points and of the binding, and pins of their float64
definitions."""

import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO
from test_abi_host import _c_layout

import prefill_csa_compress_gb300 as csa
from prefill_csa_compress_gb300 import _binding as B
from prefill_csa_compress_gb300 import _cache as C
from prefill_csa_compress_gb300 import _paged as P


@pytest.fixture(scope="module")
def L():
    from prefill_csa_compress_gb300 import build

    build.build()
    return B.lib()


@pytest.mark.parametrize("cname,S", [("csa_latent_attn_args", C.LatentAttnArgs),
                                     ("csa_latent_expand_args", C.LatentExpandArgs),
                                     ("csa_attn_mass_args", C.AttnMassArgs),
                                     ("csa_kv_evict_args", C.KvEvictArgs),
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

LATENT = dict(n_rows=4, n_heads=8, causal=1, softmax_scale=0.1, n_req=2, max_blocks=4, n_blocks=8,
              q=_base, q_rope=_base, row_req=_base, row_pos=_base, kv_len=_base, block_table=_base,
              c_pool=_base, r_pool=_base, out=_base, workspace=_base, workspace_bytes=1 << 40)
EXPAND = dict(n_heads=8, n_req=2, max_blocks=4, n_blocks=8, out_max_blocks=4, n_out_blocks=8,
              kv_len=_base, block_table=_base, out_table=_base, c_pool=_base, r_pool=_base,
              w_uk=_base, w_uv=_base, k_pool=_base, v_pool=_base)
MASS = dict(n_rows=4, n_heads=8, n_kv_heads=2, head_dim=128, causal=1, softmax_scale=0.1, decay=1.0,
            n_req=2, max_blocks=4, n_blocks=8, q=_base, lse=_base, row_req=_base, row_pos=_base,
            kv_len=_base, block_table=_base, k_pool=_base, mass=_base, mass_out=_base,
            workspace=_base, workspace_bytes=1 << 40)
EVICT = dict(n_req=2, max_blocks=4, n_blocks=8, n_heads=2, k_dim=128, v_dim=64, mass=_base,
             kv_len=_base, budget=_base, block_table=_base, k_pool=_base, v_pool=_base,
             kv_len_out=_base, workspace=_base, workspace_bytes=1 << 40)
ATTN = dict(n_rows=4, n_heads=8, n_kv_heads=2, head_dim=192, v_dim=128, causal=1, softmax_scale=0.1,
            n_req=2, max_blocks=4, n_blocks=8, q=_base, row_req=_base, row_pos=_base, kv_len=_base,
            block_table=_base, k_pool=_base, v_pool=_base, out=_base, workspace=_base,
            workspace_bytes=1 << 40)
INVALID, UNSUPPORTED = B.CSA_ERR_INVALID_ARG, B.CSA_ERR_UNSUPPORTED
NAN, INF = float("nan"), float("inf")


def _gone(*names):
    return [{n: None} for n in names]


REFUSED = [
    ("csa_latent_attn", LATENT, INVALID, [
        dict(struct_size=8), dict(n_rows=-1), dict(n_req=0), dict(max_blocks=0), dict(n_blocks=0),
        dict(n_heads=0), dict(causal=2), dict(window=-1), dict(softmax_scale=0.0),
        dict(softmax_scale=NAN), dict(softmax_scale=INF), dict(q_row_stride=1024),
        dict(q_head_stride=1032), dict(q_head_stride=512), dict(q_head_stride=-1024),
        dict(q_head_stride=1024, q_row_stride=7 * 1024), dict(q_head_stride=3 * 1024, q_row_stride=1024),
        dict(q_row_stride=1 << 40), dict(q_rope_row_stride=64), dict(q_rope_head_stride=120),
        dict(c_token_stride=512), dict(c_page_stride=1024), dict(r_token_stride=136),
        dict(r_page_stride=128), dict(workspace=_base + 16), dict(q=_base + 8), dict(q_rope=_base + 2),
        dict(c_pool=_base + 8), dict(r_pool=_base + 8), dict(out=_base + 8)]
        + _gone("q", "q_rope", "row_req", "row_pos", "kv_len", "block_table", "c_pool", "r_pool", "out")),
    ("csa_latent_attn", LATENT, UNSUPPORTED, [
        dict(n_heads=129), dict(n_rows=(1 << 24) + 1), dict(max_blocks=(1 << 24) + 1)]),
    ("csa_latent_expand", EXPAND, INVALID, [
        dict(struct_size=8), dict(n_req=-1), dict(max_blocks=0), dict(n_blocks=0), dict(n_heads=0),
        dict(n_heads=65537), dict(out_max_blocks=0), dict(n_out_blocks=0), dict(c_token_stride=1008),
        dict(r_page_stride=-16), dict(w_uk_head_stride=1024), dict(w_uv_head_stride=131080),
        dict(k_token_stride=384), dict(k_head_stride=256), dict(v_head_stride=8),
        dict(v_page_stride=256), dict(c_pool=_base + 8), dict(r_pool=_base + 8), dict(w_uk=_base + 8),
        dict(w_uv=_base + 8), dict(k_pool=_base + 8), dict(v_pool=_base + 8)]
        + _gone("kv_len", "block_table", "out_table", "c_pool", "r_pool", "w_uk", "w_uv", "k_pool", "v_pool")),
    ("csa_latent_expand", EXPAND, UNSUPPORTED, [dict(max_blocks=1 << 24)]),
    ("csa_attn_mass", MASS, INVALID, [
        dict(struct_size=8), dict(n_rows=-1), dict(n_req=0), dict(max_blocks=0), dict(n_blocks=0),
        dict(n_heads=0), dict(n_kv_heads=0), dict(n_kv_heads=3), dict(n_heads=65538), dict(causal=-1),
        dict(window=-1), dict(softmax_scale=-1.0), dict(softmax_scale=NAN), dict(decay=-0.5),
        dict(decay=NAN), dict(decay=INF), dict(q_row_stride=256), dict(k_token_stride=256),
        dict(k_head_stride=8), dict(mass_row_stride=2044), dict(mass_out_row_stride=2050),
        dict(mass_out_row_stride=2052), dict(mass_row_stride=-4), dict(workspace=_base + 16),
        dict(q=_base + 8), dict(k_pool=_base + 8), dict(mass=_base + 2), dict(mass_out=_base + 1),
        dict(lse=_base + 2)]
        + _gone("q", "lse", "row_req", "row_pos", "kv_len", "block_table", "k_pool", "mass", "mass_out")),
    ("csa_attn_mass", MASS, UNSUPPORTED, [
        dict(head_dim=32), dict(head_dim=192), dict(n_heads=129, n_kv_heads=1),
        dict(n_rows=(1 << 24) + 1), dict(max_blocks=1 << 24)]),
    ("csa_kv_evict", EVICT, INVALID, [
        dict(struct_size=8), dict(n_req=-1), dict(max_blocks=0), dict(n_blocks=0), dict(n_heads=0),
        dict(n_heads=65537), dict(first=-1), dict(recent=-1), dict(k_token_stride=256),
        dict(v_token_stride=128), dict(v_head_stride=136), dict(mass_row_stride=2044),
        dict(mass_out=_base, mass_out_row_stride=2052), dict(mass_out_row_stride=2047),
        dict(workspace=_base + 16), dict(k_pool=_base + 8), dict(v_pool=_base + 8), dict(mass=_base + 2),
        dict(mass_out=_base + 2)]
        + _gone("mass", "kv_len", "budget", "block_table", "k_pool", "kv_len_out")),
    ("csa_kv_evict", EVICT, UNSUPPORTED, [
        dict(k_dim=4), dict(k_dim=520), dict(k_dim=100), dict(v_dim=0), dict(v_dim=12),
        dict(max_blocks=1 << 24)]),
    ("csa_paged_attn", ATTN, UNSUPPORTED, [
        dict(v_dim=0), dict(v_dim=192), dict(v_dim=64), dict(head_dim=128, v_dim=64),
        dict(head_dim=64, v_dim=128), dict(v_dim=-128)]),
    ("csa_paged_attn", ATTN, INVALID, [dict(k_token_stride=256), dict(v_token_stride=256),
                                       dict(q_row_stride=8 * 256)]),
]


def _args(name, **fields):
    a = P._CALLS[name]()
    a.struct_size = ctypes.sizeof(a)
    for k, v in fields.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("name,base,status,change", [
    (n, b, s, c) for n, b, s, cs in REFUSED for c in cs],
    ids=lambda v: ",".join(f"{k}={x}" for k, x in v.items())[:60] if isinstance(v, dict) and len(v) < 4 else None)
def test_refusals(L, name, base, status, change):
    assert P._fn(name)(ctypes.byref(_args(name, **{**base, **change})), None) == status


@pytest.mark.parametrize("name,base", [("csa_latent_attn", dict(LATENT, n_rows=0)),
                                       ("csa_latent_expand", dict(EXPAND, n_req=0)),
                                       ("csa_kv_evict", dict(EVICT, n_req=0)),
                                       ("csa_paged_attn", dict(ATTN, n_rows=0))])
def test_nothing_to_do_is_ok(L, name, base):
    before = csa.launch_count()
    assert P._fn(name)(ctypes.byref(_args(name, **base)), None) == B.CSA_OK
    assert P._fn(name)(None, None) == INVALID
    assert csa.launch_count() == before


@pytest.mark.parametrize("name,base", [("csa_latent_attn", LATENT), ("csa_attn_mass", MASS),
                                       ("csa_kv_evict", EVICT), ("csa_paged_attn", ATTN)])
def test_size_query(L, name, base):
    a = _args(name, **dict(base, workspace=None, workspace_bytes=77))
    assert P._fn(name)(ctypes.byref(a), None) == B.CSA_OK
    need = a.workspace_bytes
    assert need != 77
    if need:
        a.workspace, a.workspace_bytes = _base, need - 1
        assert P._fn(name)(ctypes.byref(a), None) == INVALID


@pytest.mark.parametrize("name,base", [
    ("csa_latent_attn", dict(LATENT, n_rows=8192, n_heads=64, n_req=1)),  # rows taken whole
    ("csa_latent_attn", dict(LATENT, n_rows=0)), ("csa_attn_mass", dict(MASS, n_req=64, max_blocks=128)),  # nothing split
    ("csa_attn_mass", dict(MASS, n_rows=0, n_req=64, max_blocks=128)), ("csa_kv_evict", dict(EVICT, n_req=0)),
    ("csa_paged_attn", dict(ATTN, n_rows=8192, n_heads=64, n_kv_heads=64)), ("csa_paged_attn", dict(ATTN, n_rows=0)),
    ("csa_paged_attn", dict(ATTN, n_rows=8192, head_dim=64, v_dim=64, n_heads=64, n_kv_heads=64))])
def test_size_query_is_never_zero(L, name, base):
    """A call whose workspace is NULL is a size query: a caller who allocates the bytes it
    is told has to hold a pointer then, also where nothing is split."""
    a = _args(name, **dict(base, workspace=None, workspace_bytes=0))
    assert P._fn(name)(ctypes.byref(a), None) == B.CSA_OK
    assert a.workspace_bytes >= 256

def test_paged_attention_struct_without_value_width(L):
    """A caller built before v_dim: its struct ends there, and values are as wide
    as keys."""
    a = _args("csa_paged_attn", **dict(ATTN, head_dim=128, v_dim=55, n_rows=0))
    assert P._fn("csa_paged_attn")(ctypes.byref(a), None) == UNSUPPORTED
    a.struct_size = P.PagedAttnArgs.v_dim.offset
    assert P._fn("csa_paged_attn")(ctypes.byref(a), None) == B.CSA_OK
    a.head_dim = 192
    assert P._fn("csa_paged_attn")(ctypes.byref(a), None) == UNSUPPORTED


def _bf(*s):
    return torch.zeros(s, dtype=torch.bfloat16)


def _i(*s):
    return torch.zeros(s, dtype=torch.int32)


def test_binding_refusals():
    """Shapes, dtypes and layouts are refused before any device is asked for;
    a call that is right but for its CPU tensors is refused last."""
    at = dict(q=_bf(4, 8, 512), q_rope=_bf(4, 8, 64), row_req=_i(4), row_pos=_i(4), c_pool=_bf(5, 128, 512),
              r_pool=_bf(5, 128, 64), block_table=_i(2, 3), kv_len=_i(2), out=_bf(4, 8, 512), softmax_scale=0.1)
    for change in (dict(), dict(q=_bf(8, 4, 512).transpose(0, 1)), dict(q_rope=_bf(4, 8, 576)[..., 512:]),
                   dict(c_pool=_bf(5, 128, 576)[..., :512], r_pool=_bf(5, 128, 576)[..., 512:]),
                   dict(q=_bf(0, 8, 512), q_rope=_bf(0, 8, 64), row_req=_i(0), row_pos=_i(0), out=_bf(0, 8, 512))):
        with pytest.raises(ValueError, match="CUDA"):
            csa.csa_latent_attn(**{**at, **change})
    for change, why in [(dict(q=_bf(4, 8, 576)), "shape"), (dict(q_rope=_bf(4, 7, 64)), "shape"),
                        (dict(q=_bf(4, 512, 8).transpose(1, 2)), "contiguous"), (dict(row_pos=_i(5)), "shape"),
                        (dict(q=_bf(1, 8, 512).expand(4, 8, 512)), "overlap"),
                        (dict(q=_bf(4, 1, 512).expand(4, 8, 512)), "overlap"),
                        (dict(c_pool=_bf(5, 128, 576)), "shape"), (dict(r_pool=_bf(4, 128, 64)), "shape"),
                        (dict(c_pool=_bf(1, 128, 512).expand(5, 128, 512)), "overlap"),
                        (dict(out=_bf(4, 8, 576)[..., :512]), "contiguous"), (dict(sink=torch.zeros(2)), "shape"),
                        (dict(window=2 ** 32 + 1), "32 bits"), (dict(lse=torch.zeros(4, 7)), "shape")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_latent_attn(**{**at, **change})
    with pytest.raises(TypeError, match="q must be"):
        csa.csa_latent_attn(**{**at, "q": _bf(4, 8, 512).half()})

    w = _bf(8, 256, 512)
    ex = dict(c_pool=at["c_pool"], r_pool=at["r_pool"], block_table=_i(2, 3), kv_len=_i(2), w_uk=w[:, :128],
              w_uv=w[:, 128:], k_pool=_bf(6, 128, 8, 192), v_pool=_bf(6, 128, 8, 128), out_table=_i(2, 7))
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_latent_expand(**ex)
    for change, why in [(dict(w_uk=w), "shape"), (dict(w_uv=w[:7, 128:]), "shape"),
                        (dict(w_uk=_bf(8, 512, 128).transpose(1, 2)), "contiguous"),
                        (dict(w_uk=_bf(1, 128, 512).expand(8, 128, 512)), "overlap"),
                        (dict(k_pool=_bf(6, 128, 8, 128)), "shape"), (dict(v_pool=_bf(5, 128, 8, 128)), "shape"),
                        (dict(out_table=_i(3, 7)), "shape"), (dict(first=_i(3)), "shape"), (dict(kv_len=_i(1)), "shape")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_latent_expand(**{**ex, **change})

    m = torch.zeros(2, 384)
    ms = dict(q=_bf(4, 8, 64), lse=torch.zeros(4, 8), row_req=_i(4), row_pos=_i(4), k_pool=_bf(5, 128, 2, 64),
              block_table=_i(2, 3), kv_len=_i(2), mass=m)
    for change in (dict(), dict(mass=None, mass_out=m, decay=0.0), dict(mass=torch.zeros(2, 500)[:, :384])):
        with pytest.raises(ValueError, match="CUDA"):
            csa.csa_attn_mass(**{**ms, **change})
    for change, why in [(dict(q=_bf(4, 7, 64), lse=torch.zeros(4, 7)), "divide"), (dict(mass=torch.zeros(2, 383)), "shape"),
                        (dict(mass=None), "needed"), (dict(mass=None, mass_out=m), "needed"),
                        (dict(lse=torch.zeros(4, 7)), "shape"), (dict(mass=torch.zeros(384, 2).t()), "contiguous"),
                        (dict(mass=torch.zeros(1, 384).expand(2, 384)), "overlap"), (dict(row_req=_i(3)), "shape")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_attn_mass(**{**ms, **change})

    ev = dict(mass=m, kv_len=_i(2), budget=_i(2), block_table=_i(2, 3), k_pool=_bf(5, 128, 2, 64))
    for change in (dict(), dict(v_pool=_bf(5, 128, 2, 128)), dict(k_pool=_bf(5, 128, 512), v_pool=_bf(5, 128, 64))):
        with pytest.raises(ValueError, match="CUDA"):
            csa.csa_kv_evict(**{**ev, **change})
    for change, why in [(dict(budget=_i(3)), "shape"), (dict(v_pool=_bf(5, 128, 1, 64)), "shape"),
                        (dict(mass_out=torch.zeros(2, 385)), "shape"), (dict(slot_src=_i(2, 3)), "shape"),
                        (dict(kv_len_out=_i(3)), "shape"), (dict(first=2 ** 31), "32 bits")]:
        with pytest.raises(ValueError, match=why):
            csa.csa_kv_evict(**{**ev, **change})
    with pytest.raises(TypeError, match="budget must be"):
        csa.csa_kv_evict(**{**ev, "budget": None})

    pa = dict(q=_bf(4, 8, 192), row_req=_i(4), row_pos=_i(4), k_pool=_bf(5, 128, 2, 192),
              v_pool=_bf(5, 128, 2, 128), block_table=_i(2, 3), kv_len=_i(2), out=_bf(4, 8, 128))
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_paged_attn(**pa)
    for change in (dict(v_pool=_bf(5, 128, 2, 192)), dict(out=_bf(4, 8, 192))):
        with pytest.raises(ValueError, match="shape"):
            csa.csa_paged_attn(**{**pa, **change})


# ---------------------------------------------------------------- the definitions


def test_latent_definition():
    """The absorbed form and the expanded one are the same function."""
    rng = np.random.default_rng(0)
    H, n = 3, 140
    c, r = rng.standard_normal((2, 128, 512)), rng.standard_normal((2, 128, 64))
    uk, uv = rng.standard_normal((2, H, 128, 512)) / 512 ** 0.5
    q = rng.standard_normal((2, H, 192))
    table = np.array([[1, 0]])
    qa = np.einsum("thd,hdc->thc", q[..., :128], uk)
    at = ([0, 0], [n - 1, 20], table, [n], 0.07)
    o, lse, _ = PO.latent_attention(qa, q[..., 128:], *at[:2], c, r, *at[2:], sink=[0.1] * H)
    k, v = PO.latent_expand(c.reshape(-1, 512), r.reshape(-1, 64), uk, uv)
    e, lse2, _ = PO.paged_attention(q, *at[:2], k.reshape(2, 128, H, 192), v.reshape(2, 128, H, 128), *at[2:],
                                    sink=[0.1] * H)
    assert np.allclose(np.einsum("thc,hdc->thd", o, uv), e) and np.allclose(lse, lse2)


def test_mass_definition():
    """Each row's weights add up to one; a window, an unmapped page and padding."""
    rng = np.random.default_rng(1)
    k, q = rng.standard_normal((3, 128, 2, 8)), rng.standard_normal((3, 4, 8))
    table = np.array([[2, 0], [1, -1]])
    req, pos, lens = [0, 1, -1], [200, 140, 3], [230, 150]
    _, lse, _ = PO.paged_attention(q, req, pos, k, k, table, lens, 0.4, window=60)
    m = PO.attention_mass(q, lse, req, pos, k, table, lens, 0.4, window=60)
    assert [len(x) for x in m] == lens
    assert np.isclose(m[0].sum(), 4) and np.isclose(m[1].sum(), 4)
    assert not m[0][:141].any() and m[0][141:201].all() and not m[0][201:].any()
    assert not m[1][128:].any()
    old = [np.full(230, 2.0), np.full(150, 3.0)]
    d = PO.attention_mass(q, lse, req, pos, k, table, lens, 0.4, window=60, mass=old, decay=0.5)
    assert np.allclose(d[0], m[0] + 1) and np.allclose(d[1], m[1] + 1.5)


def test_evict_definition():
    assert PO.evict([5, 1, 1, 7, math.nan, 3], 6, 3) == [0, 3, 5]
    assert PO.evict([1] * 6, 6, 3) == [0, 1, 2]  # ties: the lowest
    assert PO.evict([1] * 6, 6, 3, recent=2) == [0, 4, 5]
    assert PO.evict([1, 9, 8, 7], 4, 2, first=1) == [0, 1]
    assert PO.evict([0, 0, 0, 2, 1, 9], 6, 2, first=3) == [0, 1]  # more protected than kept: the lowest
    assert PO.evict([0, 0, math.inf, math.nan], 4, 2, recent=1) == [2, 3]
    assert PO.evict([4, 3], 2, 5) == [0, 1] and PO.evict([4, 3], 2, -1) == [] and PO.evict([], 0, 3) == []
    # kept slots before the cut stay, the others fill the holes in order
    assert PO.evict([9, 0, 9, 0, 9, 9], 6, 4) == [0, 4, 2, 5]
