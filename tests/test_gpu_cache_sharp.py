"""Latent attention in both forms and accumulated weights on inputs whose logits are
exact, so that a position counted twice or left out shows.

With q of a few +-1 and keys of +-1 every logit is a small whole number, whatever the
order of its sum, and softmax_scale = ln 2 makes each weight a power of two: rounding
the probabilities to BF16 changes nothing, and the products with values of +-1 add up
exactly (multiples of the smallest weight, below 2^24 of them).  What is left:
 - a weight's exponent x s - ref: s = scale log2(e) has two roundings (2^-23 |x|), ref,
   which is x s + 7 for the largest x, two (2^-23 |x|), and the sum one (|x s - ref| < 2^4
   wherever the weight counts: 2^-20), and 2^-22 for the exponential;
 - FP32 sums of the weights: a thread adds a tile (64 positions; a page of 128) after
   another, 16 and fewer additions beside that: (n / 64 + 16) 2^-24;
 - out rounded once to BF16 (2^-8), lse a sum and a product of FP32 numbers (2^-22).
Checks of the absorbed form also show, by the definition, that 64 positions less would
not pass.
"""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import prefill_csa_compress_gb300 as csa  # noqa: E402
from test_gpu_cache import DEV, H8, MASS_ROWS, Latent, Mass, _i32, _np, chunk, paged  # noqa: E402

LN2 = float(np.float32(math.log(2.0)))


def signs(rng, *shape):
    return torch.from_numpy(rng.choice([-1.0, 1.0], shape).astype(np.float32)).bfloat16().to(DEV)


def sparse(rng, rows, heads, dim, n, size):
    """[rows, heads, dim] with n channels of +-size a head, the rest zero."""
    q = np.zeros((rows, heads, dim), dtype=np.float32)
    for t in range(rows):
        for h in range(heads):
            q[t, h, rng.permutation(dim)[:n]] = rng.choice([-size, size], n)
    return torch.from_numpy(q).bfloat16().to(DEV)


def close(got, gl, o, ls, spread, skip, biggest, n):
    """out and lse within what is left; biggest: of the logits in units of ln 2."""
    assert (got[skip] == 77).all() and (gl[skip] == 77).all()
    got, gl, o, ls, spread = (x[~skip] for x in (got, gl, o, ls, spread))
    weight = LN2 * (biggest * 2.0 ** -22 + 2.0 ** -20) + 2.0 ** -22
    sums = (n / 64 + 16) * 2.0 ** -24
    tol = (H8 + weight + sums) * np.abs(o) + weight * spread + 1e-30
    assert (np.abs(got - o) <= tol).all(), (np.abs(got - o) / tol).max()
    none = np.isneginf(ls)
    assert np.array_equal(none, np.isneginf(gl))
    lt = weight + sums + 2.0 ** -22 * (np.abs(ls[~none]) + 16)
    assert (np.abs(gl[~none] - ls[~none]) <= lt).all(), (np.abs(gl[~none] - ls[~none]) / lt).max()
    return weight, sums


def shows(x, v, o, ls, weight, sums, at):
    """Whether the 64 positions from `at` on, left out of one row's sums (logits x,
    values v), would be outside close()'s tolerances for its out or lse."""
    w = np.exp(x - ls)
    lost = w[at:at + 64]
    o2 = (o - lost @ v[at:at + 64]) / (1 - lost.sum())
    tol = (H8 + weight + sums) * np.abs(o) + weight * (w @ np.abs(v))
    lt = weight + sums + 2.0 ** -22 * (abs(ls) + 16)
    return (np.abs(o2 - o) > tol).any() and abs(np.log1p(-lost.sum())) > lt


class Whole(Latent):
    """A latent case with whole logits: three channels of +-size a head."""

    def __init__(self, rows, lens, heads, *, size=1, zero=False, seed=0, **kw):
        super().__init__(rows, lens, heads, seed=seed, **kw)
        rng = np.random.default_rng(1000 + seed)
        for p in (self.c, self.r):
            unseen = torch.isnan(p)
            p.copy_(signs(rng, *p.shape))
            p[unseen] = float("nan")
        q = sparse(rng, len(rows), heads, 576, 0 if zero else 3, size)
        self.q, self.qr = q[..., :512], q[..., 512:]
        self.biggest = 0 if zero else 3 * size
        if self.sink is not None:
            self.sink = self.sink.round()

    def check(self, status=0):
        got, gl, st = self.call(softmax_scale=LN2)
        assert st == status
        q, qr, c, r = (_np(x) for x in (self.q, self.qr, self.c, self.r))
        sink = None if self.sink is None else _np(self.sink)
        o, ls, spread = PO.latent_attention(q, qr, self.req, self.pos, c, r, self.table, self.lens, LN2, sink=sink,
                                            **self.kw)
        skip = (self.req < 0) | (self.req >= len(self.lens))
        n = int(self.lens.max())
        weight, sums = close(got, gl, o, ls, spread, skip, self.biggest, n)
        if sink is None and self.biggest <= 3:
            for t in np.flatnonzero(~skip)[:3]:
                lo, hi = PO.visible(int(self.pos[t]), int(self.lens[self.req[t]]), self.kw["causal"], self.kw["window"])
                if hi - lo < 130:
                    continue
                j = np.arange(lo, hi)
                at = self.table[self.req[t], j // 128], j % 128
                for h in (0, self.q.shape[1] - 1):
                    x = LN2 * (c[at] @ q[t, h] + r[at] @ qr[t, h])
                    for lost in (0, (hi - lo) // 2, hi - lo - 64):
                        assert shows(x, c[at], o[t, h], ls[t, h], weight, sums, lost)


# ---------------------------------------------------------------- absorbed


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("rows,lens,heads,kw", [
    # equal shares of ragged contexts, cut items, many parts a row
    ([(0, 40000), (1, 500), (0, 39999), (2, 20000)], [40001, 501, 20001], 16, {}),
    ([(0, 17000)], [17001], 128, dict(window=9000)),
    ([(0, 20000)], [20001], 1, {}),
    ([(0, 5000), (1, 4990)], [5001, 4991], 70, {}),
    # few tiles: the shares are parts of an item, or an item each
    ([(0, 300)], [301], 64, {}), (chunk(0, 700, 9) + [(1, 200), (-1, 0), (2, 4)], [709, 201, 5], 24, {}),
    # rows of one request, windows, sinks
    (chunk(0, 100, 300), [400], 8, dict(window=130)), (chunk(0, 1000, 5), [1005], 128, dict(sink=True)),
    (chunk(0, 2000, 3) + chunk(1, 30, 70), [2003, 100], 33, dict(causal=False))])
def test_latent_attention_whole_logits(rows, lens, heads, kw, zero):
    Whole(rows, lens, heads, zero=zero, seed=heads, **kw).check()


def test_latent_attention_whole_logits_of_rows_taken_whole():
    """One request's items fill the SMs: no shares."""
    Whole(chunk(0, 200, 610), [810], 16, seed=2).check()


@pytest.mark.parametrize("rows,lens,heads", [
    ([(0, 20000)], [20001], 1), ([(0, 20000), (1, 9000)], [20001, 9001], 16), ([(0, 700)], [701], 128),
    (chunk(0, 200, 610), [810], 16)])
def test_latent_attention_waits_for_every_product(rows, lens, heads):
    """Calls between others' kernels (first launches, cold caches, warm ones): the
    products lag the softmax by more or less, and every tile's is in the outputs."""
    b = Whole(rows, lens, heads, zero=True, seed=2)
    b.check()
    want = b.call(softmax_scale=LN2)
    x = torch.randn(2048, 2048, device=DEV)
    flush = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for i in range(48):
        if i % 3 == 0:
            flush.fill_(i)
        elif i % 3 == 1:
            x = (x @ x).sort(dim=0)[0].softmax(1)
        got = b.call(softmax_scale=LN2)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]), i


@pytest.mark.parametrize("heads,rows_each", [(64, 200), (16, 700)])
def test_latent_attention_beside_other_work(heads, rows_each):
    """Rows taken whole while another stream's kernels come and go on the same SMs: no
    role of a CTA outruns another, no wait gives up, every call has the same bits."""
    lens = [rows_each + 40 * i for i in range(5)]
    rows = [x for b, n in enumerate(lens) for x in chunk(b, n - rows_each, rows_each)]
    b = Whole(rows, lens, heads, zero=True, seed=heads)
    out = torch.empty((len(rows), heads, 512), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((len(rows), heads), device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    call = csa.csa_latent_attn(
        q=b.q, q_rope=b.qr, row_req=_i32(b.req), row_pos=_i32(b.pos), c_pool=b.c, r_pool=b.r, block_table=_i32(b.table),
        kv_len=_i32(b.lens), out=out, lse=lse, softmax_scale=LN2, status=st, prepare=True)
    want = []  # equal weights: a row's output is the mean of what it sees
    for r, n in enumerate(lens):
        j = np.arange(n)
        c = b.c[torch.as_tensor(b.table[r, j // 128], device=DEV), torch.as_tensor(j % 128, device=DEV)].double()
        mean = c.cumsum(0) / torch.arange(1, n + 1, device=DEV)[:, None]
        want.append(mean[n - rows_each:])
    want = torch.cat(want)[:, None]
    side = torch.cuda.Stream()
    x = torch.randn(1 << 20, device=DEV)
    torch.cuda.synchronize()
    for i in range(150):
        out.fill_(77)
        lse.fill_(77)
        with torch.cuda.stream(side):
            torch.sort(x)
        call()
        torch.cuda.synchronize()
        assert int(st.item()) == 0, i
        if i == 0:
            assert ((out.double() - want).abs() <= (H8 + 2.0 ** -18) * want.abs() + 1e-30).all()
            first = out.clone(), lse.clone()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), i


@pytest.mark.parametrize("size", [32, 512])
def test_latent_attention_whole_large_logits(size):
    """Logits of +-96 and +-1536 times ln 2: references move, only the largest count."""
    Whole(chunk(0, 900, 3), [903], 8, size=size, seed=3).check()
    Whole([(0, 30000)], [30001], 64, size=size, seed=4).check()


def test_latent_cache_cut_whole_logits():
    """Attention over a latent cache that was cut, every kept position counted once."""
    rng = np.random.default_rng(14)
    lens, budget = [900, 260], [333, 259]
    b = Whole([(0, 899), (1, 259)], lens, 4, seed=14, causal=False)
    mass = torch.from_numpy(rng.random((2, b.table.shape[1] * 128)).astype(np.float32)).to(DEV)
    c0, r0 = _np(b.c), _np(b.r)
    kv_len = _i32(lens)
    csa.csa_kv_evict(mass=mass, kv_len=kv_len, budget=_i32(budget), block_table=_i32(b.table), k_pool=b.c, v_pool=b.r,
                     recent=8)
    got, gl, _ = b.call(kv_len=kv_len, softmax_scale=LN2)
    q, qr = _np(b.q), _np(b.qr)
    for t in range(2):
        kept = np.array(PO.evict(_np(mass[t]), lens[t], budget[t], 0, 8))
        at = b.table[t, kept // 128], kept % 128
        for h in range(4):
            x = LN2 * (c0[at] @ q[t, h] + r0[at] @ qr[t, h])
            ls = np.log(np.exp(x).sum())
            w = np.exp(x - ls)
            o = w @ c0[at]
            weight, sums = close(got[t:t + 1, h], gl[t:t + 1, h], o[None], np.array([ls]), (w @ np.abs(c0[at]))[None],
                                 np.zeros(1, bool), 3, len(kept))
            assert shows(x, c0[at], o, ls, weight, sums, 100)


# ---------------------------------------------------------------- expanded


@pytest.mark.parametrize("heads,kv_heads", [(7, 7), (20, 20), (12, 4), (32, 1)])
@pytest.mark.parametrize("rows,lens,kw", [
    (chunk(0, 300, 140) + chunk(1, 5, 3) + [(-1, 2)] + chunk(2, 900, 50), [440, 8, 950], {}),
    ([(b, 250 + b) for b in range(6)], [260] * 6, {}), ([(0, 3000)], [3001], {}),
    (chunk(0, 500, 200), [700], dict(window=200))])
def test_expanded_attention_whole_logits(heads, kv_heads, rows, lens, kw):
    rng = np.random.default_rng(heads)
    table, total = paged(rng, lens)
    k, v = signs(rng, total, 128, kv_heads, 192), signs(rng, total, 128, kv_heads, 128)
    q = sparse(rng, len(rows), heads, 192, 3, 1)
    req, pos = (np.array([r[i] for r in rows]) for i in range(2))
    out = torch.full((len(rows), heads, 128), 77.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((len(rows), heads), 77.0, device=DEV)
    csa.csa_paged_attn(q=q, row_req=_i32(req), row_pos=_i32(pos), k_pool=k, v_pool=v, block_table=_i32(table),
                       kv_len=_i32(lens), out=out, lse=lse, softmax_scale=LN2, **kw)
    torch.cuda.synchronize()
    o, ls, spread = PO.paged_attention(_np(q), req, pos, _np(k), _np(v), table, lens, LN2, **kw)
    close(_np(out), _np(lse), o, ls, spread, req < 0, 3, max(lens))


# ---------------------------------------------------------------- weights


def seen_counts(b):
    """How many (row, head) pairs see each position, a list of arrays."""
    out = [np.zeros(max(int(n), 0)) for n in b.lens]
    for r, p in zip(b.req, b.pos):
        if 0 <= r < len(out):
            lo, hi = PO.visible(int(p), len(out[r]), b.kw["causal"], b.kw["window"])
            out[r][lo:hi] += b.q.shape[1]
    return out


@pytest.mark.parametrize("rows,lens,kw", [(r, n, {}) for r, n in MASS_ROWS] + [
    (chunk(0, 0, 501) + chunk(1, 40, 333), [501, 373], {}), ([(0, 20000), (1, 300)], [20001, 301], {}),
    (chunk(0, 400, 300), [700], dict(window=129)), (chunk(0, 400, 40) + chunk(1, 2, 1), [440, 3], dict(causal=False)),
    ([(b, 40 * b) for b in range(200)], [40 * b + 1 for b in range(200)], {})])
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 64), (8, 2, 128), (21, 3, 64), (128, 1, 128), (16, 16, 64)])
def test_attention_mass_counts(rows, lens, kw, heads, kv_heads, dim):
    """Queries of zero against references of zero: every weight is one, and a
    position's sum the number of rows and heads that see it, exactly."""
    b = Mass(rows, lens, heads, kv_heads, dim, seed=heads, **kw)
    b.q.zero_()
    b.lse.zero_()
    out = torch.full_like(b.mass, 77.0)
    b.call(mass_out=out, decay=0.0)
    for r, want in enumerate(seen_counts(b)):
        assert np.array_equal(_np(out[r, :len(want)]), want), r
        assert (out[r, len(want):] == 77).all()


def test_attention_mass_references_that_are_not_finite():
    """A reference of -inf adds nothing, one of +inf zero; the other rows' and heads'
    sums are right."""
    b = Mass(chunk(0, 290, 4), [294], 4, 2, 64, seed=5)
    b.lse[1] = float("-inf")
    b.lse[2, 1] = float("inf")
    b.lse[3] = float("inf")
    out = torch.full_like(b.mass, 77.0)
    assert b.call(mass_out=out, decay=0.0) == 0
    q, k, lse = _np(b.q), _np(b.k), _np(b.lse)
    want = PO.attention_mass(q, lse, b.req, b.pos, k, b.table, b.lens, 64 ** -0.5)[0]
    # a logit is an FP32 sum of 64 products: 64 2^-24 of the sum of their sizes, the tensor
    # cores' truncation counted as a rounding twice; the exponent's own roundings beside a
    # reference of at most 16, the exponential, and sums of 16 weights
    sizes = max(np.abs(k[b.table[0, j // 128], j % 128, h // 2]) @ np.abs(q[t, h])
                for j in range(294) for t in (0, 2) for h in range(4))
    assert np.abs(lse[np.isfinite(lse)]).max() < 16
    e = 2 * 64 * 2.0 ** -24 * sizes / 8 + 2.0 ** -19 + 16 * 2.0 ** -24
    assert np.isfinite(e) and e < 1e-3
    got = _np(out[0, :294])
    assert (np.abs(got - want) <= e * want).all() and (want[291:293] > 0).all()
    # the definition without one of the pairs would not pass
    lse[2, 0] = np.inf
    less = PO.attention_mass(q, lse, b.req, b.pos, k, b.table, b.lens, 64 ** -0.5)[0]
    assert (np.abs(less - want)[:293] > e * want[:293]).all()
