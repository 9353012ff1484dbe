"""Rotary positions (a15, a16, a17) and cross attention (a18) on the GPU against the oracle, and runs of them with the
operators they stand beside.

Tolerances, from the arithmetic (u = half a step relative to the value: 2^-24 float32, 2^-8 bf16):
* table: the angle's fraction is exact to 2^-33 turns; the remainder, at most 1/4 of a half turn, becomes a float (u, of
  at most pi / 4), sine and cosine are off by 2 u at most each, the factor's product by u: 4 u of the factor.
* rotate: equal to the float32 steps of the definition, rounded once to the output's type, bit for bit.  With a norm
  the row's factor is off by (D / 2 + 8) u at most (its sum of squares of D terms by D u, the root halves it; mean, eps,
  reciprocal root 2 ulp, the two products), so a channel by that times |a c| + |b s|, 3 u more from the steps, and
  the output's rounding.
* rotated append: bytes and values equal.
* cross, with A = sum_j p_j |v_j| per channel and B = max_j sum_c |q_c k_jc| * scale per row: a logit is off by
  (D + 4) u B with float32 sums and by 4 u |logit| <= 4 u B in its scaling, reference and exponential, so a weight by
  e = (D + 8) 2^-23 B + 2^-21; in bf16 a weight is rounded to 2^-8 for the product with v; sums of n keys
  add n 2^-24, each of the parts and rescalings 2^-23 (at most n / 16 of them); the output's rounding 2^-8 or 2^-24 |o|."""

import math
import os

import numpy as np
import pytest
import torch

import oracle
from parity import set_force_simt

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _clean_status(lib):
    set_force_simt(False)
    yield
    set_force_simt(False)
    assert lib.bsa_device_status() == lib.BSA_OK


@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


def f64(t):
    return t.detach().double().cpu().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 2.0 ** -24


def rand(seed, *shape, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(*shape, generator=g)).to(dtype).to(DEV)


def tables(seed, *shape):
    a = torch.from_numpy(np.random.default_rng(seed).uniform(-4, 4, shape))
    return a.cos().float().to(DEV), a.sin().float().to(DEV)


# ---------------------------------------------------------------- a15 table

@pytest.mark.parametrize("T,P,axes", [(1, 64, 1), (5, 1, 1), (1021, 64, 3), (300, 20, 2), (77, 7, 1), (3, 128, 8), (2, 3, 2)])
def test_table(pl, T, P, axes):
    rng = np.random.default_rng(T + P)
    pos = rng.integers(-(1 << 31), 1 << 31, (T, axes))
    pos[0] = [-(1 << 31), (1 << 31) - 1, 0, -1, 1, 1 << 24, 3, 4][:axes]
    turns = rng.integers(-(1 << 63), 1 << 63, P)
    turns[: P // 2] >>= rng.integers(0, 50, P // 2)
    axis = rng.integers(0, axes, P)
    args = (torch.tensor(pos, dtype=torch.int32, device=DEV), torch.tensor(turns, device=DEV),
            torch.tensor(axis, dtype=torch.int32, device=DEV))
    cos, sin = pl.rotary_table(*args, factor=1.25)
    want = oracle.rotary_table(pos, turns, axis, 1.25)
    for got, w in zip((cos, sin), want):
        assert got.shape == (T, P) and np.max(np.abs(f64(got) - w)) <= 4 * 1.25 * 2.0 ** -24


def test_table_one_axis_out_and_no_tokens(pl):
    r = pl.rotary_frequencies(32, device=DEV)
    pos = torch.tensor([0, 1, 70000, -1], dtype=torch.int32, device=DEV)
    out = (torch.full((4, 16), 7.0, device=DEV), torch.full((4, 16), 7.0, device=DEV))
    assert r.table(pos, out=out) is out
    want = oracle.rotary_table(pos.tolist(), r.turns.tolist())
    assert all(np.max(np.abs(f64(g) - w)) <= 4 * 2.0 ** -24 for g, w in zip(out, want))
    cos, _ = r.table(pos[:0])
    assert cos.shape == (0, 16)


def test_table_latches_a_bad_axis(pl, lib):
    pos = torch.zeros(4, 2, dtype=torch.int32, device=DEV)
    pl.rotary_table(pos, torch.zeros(3, dtype=torch.int64, device=DEV), torch.tensor([0, 2, -1], dtype=torch.int32, device=DEV))
    assert lib.bsa_device_status() == lib.BSA_ERR_INDEX


# ---------------------------------------------------------------- a16 rotate

def oracle_rotate(x, cos, sin, interleaved, transpose, dtype):
    """[T, heads, D] float rows -> the definition's float32 steps, rounded to dtype."""
    y = oracle.rotate_f32(x.float().cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy(), interleaved, transpose)
    return torch.from_numpy(y).to(dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,HQ,H,D,P", [(1, 1, 1, 128, 64), (7, 24, 24, 128, 64), (129, 12, 3, 64, 20), (5, 3, 1, 64, 16),
                                        (33, 8, 2, 80, 40), (3, 5, 5, 256, 128), (6, 2, 1, 32, 8), (4, 3, 2, 16, 8),
                                        (9, 2, 2, 10, 3), (2, 1, 1, 2, 1), (3, 7, 2, 112, 24), (2, 64, 4, 250, 125)])
def test_rotate(pl, dtype, interleaved, T, HQ, H, D, P):
    rows = rand(T + D, T, HQ + 2 * H, D, dtype=dtype)
    q, k = rows[:, :HQ], rows[:, HQ:HQ + H]
    cos, sin = tables(P, T, P)
    for transpose in (False, True):
        for heads_first in (False, True):
            got = pl.rotate(q, k, cos, sin, interleaved=interleaved, transpose=transpose, heads_first=heads_first)
            for x, y in zip((q, k), got):
                want = oracle_rotate(x, cos, sin, interleaved, transpose, dtype)
                assert y.is_contiguous() and torch.equal((y.transpose(0, 1) if heads_first else y).cpu(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,P", [(128, 64), (64, 20), (80, 40), (64, 16), (34, 17), (256, 64)])
def test_rotate_with_norm(pl, dtype, interleaved, D, P):
    T, HQ, H, eps = 19, 6, 2, 1e-5
    rows = rand(D, T, HQ + H, D, dtype=dtype, scale=3.0)
    rows[3] = 0
    rows[4] *= 1e-3
    qw, kw = rand(1, D), rand(2, D)
    cos, sin = tables(P, T, P)
    got = pl.rotate(rows[:, :HQ], rows[:, HQ:], cos, sin, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=eps)
    for x, w, y in zip((rows[:, :HQ], rows[:, HQ:]), (qw, kw), got):
        n = oracle.rms_norm(f64(x), f64(w), eps)
        want = oracle.rotate(n, f64(cos), f64(sin), interleaved)
        mag = oracle.rotate(np.abs(n), np.abs(f64(cos)), -np.abs(f64(sin)), interleaved)
        mag = np.maximum(np.abs(mag), oracle.rotate(np.abs(n), np.abs(f64(cos)), np.abs(f64(sin)), interleaved))
        tol = (D / 2 + 8 + 3) * 2.0 ** -24 * mag + half_step(dtype) * np.abs(want) + 1e-30
        assert np.all(np.abs(f64(y) - want) <= tol * (1 + 2.0 ** -7))
    # a weight for one of the two alone
    one = pl.rotate(rows[:, :HQ], rows[:, HQ:], cos, sin, interleaved=interleaved, k_weight=kw, eps=eps)
    assert torch.equal(one[1], got[1])
    assert torch.equal(one[0], pl.rotate(rows[:, :HQ], None, cos, sin, interleaved=interleaved)[0])


@pytest.mark.parametrize("D,P", [(128, 64), (64, 20)])
def test_rotate_batches_strides_in_place(pl, D, P):
    B, T, HQ, H = 3, 11, 4, 2
    cos, sin = tables(1, T, P)
    each = tables(2, B, T, P)
    heads_first = rand(5, B, HQ, T, D, dtype=BF16)
    q, k = heads_first.transpose(1, 2), rand(6, T, B, H, D, dtype=BF16).transpose(0, 1)
    for c, s in ((cos, sin), each):
        got = pl.rotate(q, k, c, s)
        for b in range(B):
            cb, sb = (c, s) if c.dim() == 2 else (c[b], s[b])
            for x, y in zip((q, k), got):
                assert torch.equal(y[b].cpu(), oracle_rotate(x[b], cb, sb, False, False, BF16))
    want = pl.rotate(q, k, cos, sin)
    pl.rotate(q, k, cos, sin, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(heads_first.transpose(1, 2), q)
    # rows that start off 16 bytes
    odd = rand(7, T * HQ * D + 1, dtype=BF16)[1:].view(T, HQ, D)
    assert torch.equal(pl.rotate(odd, None, cos, sin)[0], pl.rotate(odd.clone(), None, cos, sin)[0])
    # no rows
    empty = pl.rotate(q[:, :0], k[:, :0], cos[:0], sin[:0])
    assert empty[0].shape == (B, 0, HQ, D)


def test_rotate_gradient_is_the_transposed_call(pl):
    """Against the formula (J^T g with J's columns from unit vectors) and against differences of the forward call."""
    T, H, D, P = 3, 2, 16, 6
    cos, sin = tables(3, T, P)
    x, g = rand(1, T, H, D), rand(2, T, H, D)
    for interleaved in (False, True):
        grad = pl.rotate(g, None, cos, sin, interleaved=interleaved, transpose=True)[0]
        jac = oracle.rotate(np.broadcast_to(np.eye(D), (T, D, D)), f64(cos), f64(sin), interleaved)  # [T, in, out]
        want = np.einsum("tio,tho->thi", jac, f64(g))
        assert np.max(np.abs(f64(grad) - want)) <= 3 * 2.0 ** -24 * 2 * np.max(np.abs(f64(g)))
        d = rand(4, T, H, D)
        step = (f64(pl.rotate(x + d, None, cos, sin, interleaved=interleaved)[0])
                - f64(pl.rotate(x - d, None, cos, sin, interleaved=interleaved)[0])) / 2
        # linear: the difference is exact but for the roundings of both calls and of x +- d
        size = 4 * 2 * np.max(np.abs(f64(x)) + np.abs(f64(d)))
        assert abs(np.sum(step * f64(g)) - np.sum(f64(d) * f64(grad))) <= T * H * D * 2.0 ** -24 * size * np.max(np.abs(f64(g)))


def test_rotate_keeps_infinities_and_nan_to_their_pair(pl):
    cos, sin = tables(9, 2, 64)
    x = rand(1, 2, 3, 128, dtype=BF16)
    y0 = pl.rotate(x, None, cos, sin)[0].clone()
    x[0, 1, 5], x[1, 2, 70] = float("nan"), float("inf")
    y = pl.rotate(x, None, cos, sin)[0]
    bad = torch.zeros(2, 3, 128, dtype=torch.bool, device=DEV)
    bad[0, 1, [5, 69]] = bad[1, 2, [6, 70]] = True
    assert torch.equal(torch.isfinite(y), ~bad) and torch.equal(y[~bad], y0[~bad])


# ---------------------------------------------------------------- a17 rotated append

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,HQ,H,D,P,page", [(1, 8, 1, 128, 64, 64), (37, 12, 3, 64, 32, 16), (5, 2, 2, 128, 32, 32),
                                             (9, 3, 1, 48, 20, 16), (6, 4, 2, 16, 8, 16), (11, 5, 1, 128, 24, 128),
                                             (3, 2, 2, 80, 40, 16), (4, 1, 1, 32, 1, 16), (200, 64, 4, 128, 64, 64)])
def test_append_rotated(pl, dtype, interleaved, T, HQ, H, D, P, page):
    rng = np.random.default_rng(T + D)
    rows = rand(T + P, T, HQ + 2 * H, D, dtype=dtype)
    q, k, v = rows[:, :HQ], rows[:, HQ:HQ + H], rows[:, HQ + H:]
    cos, sin = tables(T, T, P)
    n_pages = T // page + 2
    slots = torch.from_numpy(rng.permutation(n_pages * page)[:T]).to(DEV)
    if T > 3:
        slots[2] = -1
    scale = [torch.tensor(rng.uniform(0.05, 0.3, H), dtype=F32, device=DEV) for _ in range(2)]
    cache = pl.new_cache(n_pages, H, page, D)
    q_out = torch.full((T, HQ, D), 9.0, dtype=dtype, device=DEV)
    vals = tuple(torch.full((T, H, D), 9.0, dtype=dtype, device=DEV) for _ in range(2))
    assert pl.cache_append_rotated(k, v, slots, cache, cos, sin, *scale, interleaved=interleaved, values=vals, q=q,
                                   q_out=q_out) is q_out
    live = (slots >= 0).cpu()
    want_q = oracle_rotate(q, cos, sin, interleaved, False, dtype)
    assert torch.equal(q_out.cpu()[live], want_q[live]) and bool((q_out.cpu()[~live] == 9.0).all())
    kr = oracle.rotate_f32(k.float().cpu().numpy(), cos.cpu().numpy(), sin.cpu().numpy(), interleaved)
    want = oracle.empty_cache(n_pages, H, page, D)
    g = [s.cpu().numpy() for s in scale]
    for t in range(T):
        if live[t]:
            oracle.store(want, int(slots[t]), kr[t], v[t].float().cpu().numpy(), *g)
    assert np.array_equal(cache.cpu().numpy(), want)
    for t in range(0, T, max(1, T // 16)):
        if live[t]:
            for got, w in zip(vals, oracle.load(want, int(slots[t]), *g)):
                assert torch.equal(got[t].cpu(), torch.from_numpy(w).float().to(dtype))
        else:
            assert bool((vals[0][t] == 9.0).all())
    # without queries, values and scales: the same bytes as those of the steps by themselves
    one, two = pl.new_cache(n_pages, H, page, D), pl.new_cache(n_pages, H, page, D)
    assert pl.cache_append_rotated(k, v, slots, one, cos, sin, interleaved=interleaved) is None
    pl.cache_append(pl.rotate(k.float(), None, cos, sin, interleaved=interleaved)[0], v.float(), slots, two)
    assert torch.equal(one, two)


def test_append_rotated_odd_addresses_bad_slots_and_nan(pl, lib):
    T, HQ, H, D, P = 6, 3, 2, 64, 32
    cos, sin = tables(1, T, P)
    off = [rand(i, T * n * D + 1, dtype=BF16)[1:].view(T, n, D) for i, n in ((1, HQ), (2, H), (3, H))]
    slots = torch.tensor([0, 5, 17, 40, 63, 31], device=DEV)
    a, b = pl.new_cache(4, H, 16, D), pl.new_cache(4, H, 16, D)
    qa = pl.cache_append_rotated(off[1], off[2], slots, a, cos, sin, q=off[0])
    qb = pl.cache_append_rotated(off[1].clone(), off[2].clone(), slots, b, cos, sin, q=off[0].clone())
    assert torch.equal(a, b) and torch.equal(qa, qb)
    k = off[1].clone()
    k[1, 0, 3] = float("nan")  # pair (3, 35): groups 0 and 2 of that row read back as NaN
    pl.cache_append_rotated(k, off[2], slots, a, cos, sin)
    got = oracle.load(a.cpu().numpy(), 5)[0]
    bad = np.zeros((H, D), bool)
    bad[0, 0:16] = bad[0, 32:48] = True
    assert np.array_equal(np.isnan(got), bad)
    q_out = torch.zeros(T, HQ, D, dtype=BF16, device=DEV)
    slots[1] = 64
    before = a.clone()
    pl.cache_append_rotated(off[1], off[2], slots, a, cos, sin, q=off[0], q_out=q_out)
    assert lib.bsa_device_status() == lib.BSA_ERR_INDEX
    assert not q_out[1].any() and torch.equal(q_out[2], qa[2])
    assert torch.equal(a[0, :, 0, 5 * D // 2:6 * D // 2], before[0, :, 0, 5 * D // 2:6 * D // 2])  # slot 5: its K codes


# ---------------------------------------------------------------- a18 cross attention

def check_rows(o, lse, q, k, v, scale, dtype):
    """One sequence: o [n, HQ, D], lse [n, HQ] on the GPU against the oracle."""
    n, HQ, D = q.shape
    m, G = k.shape[0], HQ // k.shape[1]
    qd, kd, vd = f64(q), f64(k), f64(v)
    want, wlse = oracle.cross_attention(qd, kd, vd, scale)
    if m == 0:
        assert not f64(o).any() and np.all(np.isneginf(f64(lse)))
        return
    for hq in range(HQ):
        h = hq // G
        s = qd[:, hq] @ kd[:, h].T * scale
        p = np.exp(s - wlse[:, hq, None])
        A = p @ np.abs(vd[:, h])
        B = np.max(np.abs(qd[:, hq]) @ np.abs(kd[:, h]).T, axis=1, keepdims=True) * scale
        e = (D + 8) * 2.0 ** -23 * B + 2.0 ** -21
        sums = m * 2.0 ** -24 + m / 16 * 2.0 ** -23 + 2.0 ** -20
        weight = 2.0 ** -8 if dtype == BF16 else 0.0
        tol = A * (2 * e + sums + weight) + half_step(dtype) * np.abs(want[:, hq])
        err = np.abs(f64(o[:, hq]) - want[:, hq])
        assert np.all(err <= tol), (hq, float((err / tol).max()))
        lt = e[:, 0] + sums + 2.0 ** -23 * np.abs(wlse[:, hq])
        assert np.all(np.abs(f64(lse[:, hq]) - wlse[:, hq]) <= lt), hq


SHAPES = [  # B, N, M, HQ, H, D
    (1, 1, 1, 1, 1, 64), (2, 1, 7, 8, 1, 128), (3, 5, 130, 4, 2, 64), (1, 129, 128, 2, 2, 128), (2, 257, 300, 3, 1, 64),
    (1, 300, 1000, 16, 1, 128), (2, 40, 77, 24, 8, 80), (1, 3, 4000, 4, 1, 128), (1, 17, 65, 5, 5, 40), (2, 9, 33, 6, 2, 7),
    (1, 64, 512, 48, 3, 96), (1, 40, 300, 2, 2, 8), (2, 1, 90, 3, 1, 8), (1, 600, 129, 4, 4, 16), (4, 16, 2050, 16, 8, 64), (1, 2, 1, 128, 1, 128), (2, 70, 10, 2, 1, 1)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,M,HQ,H,D", SHAPES)
def test_cross_padded(pl, dtype, B, N, M, HQ, H, D):
    q, kv = rand(N, B, N, HQ, D, dtype=dtype, scale=2.0), rand(M, B, M, 2, H, D, dtype=dtype)
    k, v = kv[:, :, 0], kv[:, :, 1]
    for lens in (None, [M - b * M // B for b in range(B)]):
        kl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
        out, lse = pl.cross_attention(q, k, v, key_lens=kl)
        assert out.shape == q.shape and lse.shape == (B, N, HQ)
        for b in range(B):
            m = M if lens is None else lens[b]
            check_rows(out[b], lse[b], q[b], k[b, :m], v[b, :m], D ** -0.5, dtype)
        again = pl.cross_attention(q, k, v, key_lens=kl, need_lse=False)
        assert again[1] is None and torch.equal(again[0], out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("HQ,H,D", [(8, 2, 128), (3, 3, 64), (6, 2, 64), (16, 1, 128), (2, 2, 24)])
@pytest.mark.parametrize("n,m", [([3, 0, 1, 140], [70, 9, 0, 33]), ([1] * 9, [5, 400, 1, 0, 129, 128, 127, 64, 3000]),
                                 ([0, 0], [3, 4]), ([300, 2, 515], [1, 257, 640]), ([1, 1], [0, 0])])
def test_cross_packed(pl, dtype, HQ, H, D, n, m):
    starts = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV)  # noqa: E731
    T, M, pad = sum(n), sum(m), 5
    q = rand(1, T + pad, HQ, D, dtype=dtype, scale=2.0)
    k, v = rand(2, M, H, D, dtype=dtype), rand(3, M, H, D, dtype=dtype)
    qs, ks = starts(n), starts(m)
    out = torch.full((T + pad, HQ, D), 7.0, dtype=dtype, device=DEV)
    lse = torch.full((T + pad, HQ), 7.0, device=DEV)
    got = pl.cross_attention(q, k, v, query_start=qs, key_start=ks, out=out, lse=lse, scale=0.2)
    assert got[0] is out and got[1] is lse
    for b in range(len(n)):
        r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
        check_rows(out[r], lse[r], q[r], k[c], v[c], 0.2, dtype)
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    # packed queries over padded states
    if max(m) and T:
        kp, vp = (torch.full((len(m), max(m), H, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
        for b in range(len(m)):
            kp[b, :m[b]], vp[b, :m[b]] = k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]]
        o2, l2 = pl.cross_attention(q, kp, vp, query_start=qs, key_lens=torch.tensor(m, dtype=torch.int32, device=DEV),
                                    scale=0.2)
        for b in range(len(n)):
            r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
            check_rows(o2[r], l2[r], q[r], k[c], v[c], 0.2, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,HQ,H,D", [(1, 8, 2, 128), (200, 4, 4, 64), (9, 4, 2, 24), (300, 2, 2, 128)])
def test_cross_does_not_see_rows_that_do_not_count(pl, dtype, N, HQ, H, D):
    """NaN, infinities and the type's lowest value behind the lengths, and in a packed neighbour."""
    B, M, lens = 3, 300, [37, 256, 129]
    q, k, v = rand(1, B, N, HQ, D, dtype=dtype), rand(2, B, M, H, D, dtype=dtype), rand(3, B, M, H, D, dtype=dtype)
    kl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, wl = pl.cross_attention(q, k, v, key_lens=kl)
    for bad in (float("nan"), float("inf"), torch.finfo(dtype).min):
        for b in range(B):
            k[b, lens[b]:], v[b, lens[b]:] = bad, bad
        out, lse = pl.cross_attention(q, k, v, key_lens=kl)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    ks = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    kp, vp = (torch.cat([x[b, :lens[b]] for b in range(B)]) for x in (k, v))
    kp[ks[1]:ks[2]], vp[ks[1]:ks[2]] = float("nan"), float("nan")
    qs = torch.arange(0, B * N + 1, N, dtype=torch.int32, device=DEV)
    out, lse = pl.cross_attention(q.flatten(0, 1), kp, vp, query_start=qs, key_start=ks)
    for b in (0, 2):
        check_rows(out[b * N:(b + 1) * N], lse[b * N:(b + 1) * N], q[b], k[b, :lens[b]], v[b, :lens[b]], D ** -0.5, dtype)
    assert bool(torch.isnan(out[N:2 * N]).all())


@pytest.mark.parametrize("HQ,H,D", [(8, 2, 128), (3, 3, 64), (4, 1, 96)])
@pytest.mark.parametrize("n,m", [([1, 1, 1, 1], [9000, 0, 1, 4097]), ([2, 0, 1, 3, 1], [1500, 7000, 64, 63, 2000]), ([1], [20000]),
                                 ([1] * 40, [1100 + 37 * i for i in range(40)]), ([1, 0], [3, 5000])])
def test_cross_long_rows_in_equal_runs(pl, HQ, H, D, n, m):
    """Ragged rows cut at 64-key borders into one run a block: whole, cut once, cut many times, without keys."""
    starts = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV)  # noqa: E731
    T, M, pad = sum(n), sum(m), 3
    assert pl.bsa.bsa_cross_way(BF16, len(n), T + pad, M, HQ, H, D, True, True) == (2 if -(-(T + pad) // len(n)) * HQ // H <= 16 else 1)
    q = rand(1, T + pad, HQ, D, dtype=BF16, scale=2.0)
    k, v = rand(2, M, H, D, dtype=BF16), rand(3, M, H, D, dtype=BF16)
    qs, ks = starts(n), starts(m)
    out = torch.full((T + pad, HQ, D), 7.0, dtype=BF16, device=DEV)
    lse = torch.full((T + pad, HQ), 7.0, device=DEV)
    pl.cross_attention(q, k, v, query_start=qs, key_start=ks, out=out, lse=lse)
    for b in range(len(n)):
        r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
        check_rows(out[r], lse[r], q[r], k[c], v[c], D ** -0.5, BF16)
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    # padded, NaN behind the lengths
    most = max(m)
    kp, vp = (torch.full((len(m), most, H, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    for b in range(len(m)):
        kp[b, :m[b]], vp[b, :m[b]] = k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]]
    o2, l2 = pl.cross_attention(q[:T], kp, vp, query_start=qs, key_lens=torch.tensor(m, dtype=torch.int32, device=DEV))
    for b in range(len(n)):
        r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
        check_rows(o2[r], l2[r], q[r], k[c], v[c], D ** -0.5, BF16)


@pytest.mark.parametrize("HQ,H,D", [(8, 2, 128), (3, 3, 64), (12, 1, 96)])
@pytest.mark.parametrize("n,m", [([40, 33, 17, 64], [1200, 0, 100, 1285]), ([128, 1, 0, 30, 90], [128, 129, 900, 257, 1500]),
                                 ([20], [9000]), ([31] * 9, [512 + 131 * i for i in range(9)]), ([250, 3, 5, 7], [700, 3, 2000, 640])])
def test_cross_few_tokens_over_long_states(pl, HQ, H, D, n, m):
    """Half-filled row tiles over parts of the keys: none, one, two, many key tiles, masked last ones."""
    starts = lambda x: torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV)  # noqa: E731
    T, M = sum(n), sum(m)
    assert pl.bsa.bsa_cross_way(BF16, len(n), T, M, HQ, H, D, True, True) == 1
    q = rand(1, T, HQ, D, dtype=BF16, scale=2.0)
    k, v = rand(2, M, H, D, dtype=BF16), rand(3, M, H, D, dtype=BF16)
    qs, ks = starts(n), starts(m)
    out, lse = pl.cross_attention(q, k, v, query_start=qs, key_start=ks)
    most = max(m)
    kp, vp = (torch.full((len(m), most, H, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    for b in range(len(m)):
        kp[b, :m[b]], vp[b, :m[b]] = k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]]
    o2, l2 = pl.cross_attention(q, kp, vp, query_start=qs, key_lens=torch.tensor(m, dtype=torch.int32, device=DEV))
    for o, z in ((out, lse), (o2, l2)):
        for b in range(len(n)):
            r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
            check_rows(o[r], z[r], q[r], k[c], v[c], D ** -0.5, BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 56])
def test_cross_layouts(pl, dtype, D):
    """Heads first, slices of fused projections, states shared by the batch and by the heads, odd addresses."""
    B, N, M, HQ, H = 2, 150, 200, 8, 4
    q, k, v = rand(1, B, N, HQ, D, dtype=dtype), rand(2, B, M, H, D, dtype=dtype), rand(3, B, M, H, D, dtype=dtype)
    want, wl = pl.cross_attention(q, k, v)
    first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (q, k, v)]
    out, lse = pl.cross_attention(*first)
    assert out.stride() == first[0].stride() and lse.transpose(1, 2).is_contiguous()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    fused = torch.cat([k, v], 2)
    out, lse = pl.cross_attention(q, fused[:, :, :H], fused[:, :, H:])
    assert torch.equal(out, want) and torch.equal(lse, wl)
    odd = [torch.cat([torch.zeros(1, dtype=dtype, device=DEV), x.flatten()])[1:].view(x.shape) for x in (q, k, v)]
    out, lse = pl.cross_attention(*odd)
    for b in range(B):
        check_rows(out[b], lse[b], q[b], k[b], v[b], D ** -0.5, dtype)
    shared = [x[:1].expand(B, M, H, D) for x in (k, v)]
    out, lse = pl.cross_attention(q, *shared)
    for b in range(B):
        check_rows(out[b], lse[b], q[b], k[0], v[0], D ** -0.5, dtype)
    heads = [x[:, :, :1].expand(B, M, H, D) for x in (k, v)]
    out, lse = pl.cross_attention(q, *heads)
    for b in range(B):
        check_rows(out[b], lse[b], q[b], heads[0][b], heads[1][b], D ** -0.5, dtype)


@pytest.mark.parametrize("N", [1, 200])
def test_cross_extreme_logits(pl, N):
    """Logits up to some 1e4 either way (one key takes all), equal keys, a scale of 0."""
    B, M, H, D = 1, 260, 2, 64
    for dtype in (BF16, F32):
        q, k, v = rand(1, B, N, H, D, dtype=dtype, scale=60.0), rand(2, B, M, H, D, dtype=dtype, scale=60.0), rand(3, B, M, H, D, dtype=dtype)
        out, lse = pl.cross_attention(q, k, v)
        check_rows(out[0], lse[0], q[0], k[0], v[0], D ** -0.5, dtype)
        same = k[:, :1].expand(B, M, H, D).contiguous()
        out, lse = pl.cross_attention(q, same, v)
        check_rows(out[0], lse[0], q[0], same[0], v[0], D ** -0.5, dtype)
        out, lse = pl.cross_attention(q, k, v, scale=0.0)
        check_rows(out[0], lse[0], q[0], k[0], v[0], 0.0, dtype)
        assert np.allclose(f64(lse), math.log(M), atol=1e-5)


@pytest.mark.parametrize("N,M", [(1, 131072), (200, 131072), (3, 1 << 20), (2000, 65536)])
def test_cross_long_sums_of_one_sign(pl, N, M):
    """Values of 1 over equal keys: sums of products of one sign, which the tensor cores round towards zero, stay within
    an output's rounding of 1."""
    H, D = 2, 128
    q, k = rand(1, 1, N, H, D, dtype=BF16), rand(2, 1, M, H, D, dtype=BF16, scale=0.05)
    out, lse = pl.cross_attention(q, k, torch.ones_like(k))
    assert float((out.float() - 1).abs().max()) <= 2.0 ** -8
    want = torch.logsumexp((q[0, :1, 0].double() @ k[0, :, 0].double().T) * D ** -0.5, 1)
    assert float((lse[0, :1, 0].double() - want).abs().max()) <= 2.0 ** -18 * math.log(M) + M * 2.0 ** -24 / 16


@pytest.mark.parametrize("dtype,N,M", [(BF16, 1, 300), (BF16, 150, 300), (F32, 3, 100), (BF16, 1, 2000)])
def test_cross_offsets_past_32_bits(pl, dtype, N, M):
    """Sequences more than 2^32 bytes apart in one buffer, in every argument."""
    B, H, D = 2, 2, 64
    far = (1 << 31) + 64
    big = torch.empty(far + 4 * max(N, M) * H * D, dtype=dtype, device=DEV)
    at = [0]

    def place(x):
        y = big.as_strided(x.shape, (far, *x.stride()[1:]), at[0])
        at[0] += x[0].numel()
        return y.copy_(x)
    q, k, v = (rand(i, B, n, H, D, dtype=dtype) for i, n in ((1, N), (2, M), (3, M)))
    want, wl = pl.cross_attention(q, k, v)
    out = place(torch.zeros_like(q))
    got, lse = pl.cross_attention(place(q), place(k), place(v), out=out)
    assert torch.equal(got, want) and torch.equal(lse, wl)
    cos, sin = tables(1, N, D // 2)
    rot = pl.rotate(q, k[:, :N], cos, sin)
    at[0] = 0
    a, b = place(q), place(k[:, :N].contiguous())
    pl.rotate(a, b, cos, sin, out=(a, b))
    assert torch.equal(a, rot[0]) and torch.equal(b, rot[1])


def test_cross_bad_starts_and_lengths_are_latched(pl, lib):
    H, D = 2, 64
    q, k, v = rand(1, 30, H, D, dtype=BF16), rand(2, 50, H, D, dtype=BF16), rand(3, 50, H, D, dtype=BF16)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    good = pl.cross_attention(q, k, v, query_start=i32(0, 10, 20, 30), key_start=i32(0, 20, 30, 50))[0]
    for qs, ks, live in ((i32(0, 10, 31, 30), i32(0, 20, 30, 50), slice(0, 10)),
                         (i32(0, 10, 20, 30), i32(0, 20, 51, 50), slice(0, 10)),
                         (i32(0, 10, 20, 30), i32(-1, 20, 30, 50), slice(10, 30))):
        out = torch.zeros_like(q)
        pl.cross_attention(q, k, v, query_start=qs, key_start=ks, out=out)
        assert lib.bsa_device_status() == lib.BSA_ERR_INDEX
        assert torch.equal(out[live], good[live])
    qp, kp, vp = q.view(3, 10, H, D), k[:48].view(3, 16, H, D), v[:48].view(3, 16, H, D)
    want = pl.cross_attention(qp, kp, vp)[0]
    out = pl.cross_attention(qp, kp, vp, key_lens=i32(16, 17, -5))[0]
    assert lib.bsa_device_status() == lib.BSA_ERR_INDEX
    assert torch.equal(out[:2], want[:2]) and not out[2].any()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("stall", [0, 1, 4])
def test_cross_expired_wait_is_reported_and_recovers(pl, lib, D, stall):
    """A key tile that is never copied: the waits run out (after 1 ms under the switch), the kernel latches
    BSA_ERR_TIMEOUT and ends; the next call is as before."""
    B, N, M, H = 2, 1500, 700, 16
    q, k, v = rand(1, B, N, H, D, dtype=BF16), rand(2, B, M, H, D, dtype=BF16), rand(3, B, M, H, D, dtype=BF16)
    want, wl = pl.cross_attention(q, k, v)
    os.environ["BSA_TEST_STALL_TILE"] = str(stall)
    try:
        pl.cross_attention(q, k, v)
    finally:
        os.environ.pop("BSA_TEST_STALL_TILE")
    assert lib.bsa_device_status() == lib.BSA_ERR_TIMEOUT
    out, lse = pl.cross_attention(q, k, v)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,M,HQ,H,D", [(2, 40, 300, 4, 2, 64), (1, 300, 130, 2, 2, 128), (3, 1, 2000, 8, 2, 128), (2, 1, 500, 4, 4, 40)])
def test_cross_cuda_core_kernel_agrees(pl, lib, dtype, B, N, M, HQ, H, D):
    """The kernels that the switch takes out of play, and the one that remains."""
    q, k, v = rand(1, B, N, HQ, D, dtype=dtype), rand(2, B, M, H, D, dtype=dtype), rand(3, B, M, H, D, dtype=dtype)
    kl = torch.tensor([M - 7 * b for b in range(B)], dtype=torch.int32, device=DEV)
    out, lse = pl.cross_attention(q, k, v, key_lens=kl)
    lib.bsa_cross_workspace.cache_clear()  # the plan goes by the switch
    set_force_simt(True)
    try:
        assert lib.bsa_cross_way(dtype, B, N, M, HQ, H, D) == 0
        out2, lse2 = pl.cross_attention(q, k, v, key_lens=kl)
    finally:
        set_force_simt(False)
        lib.bsa_cross_workspace.cache_clear()
    for o, z in ((out, lse), (out2, lse2)):
        for b in range(B):
            check_rows(o[b], z[b], q[b], k[b, :M - 7 * b], v[b, :M - 7 * b], D ** -0.5, dtype)


@pytest.mark.parametrize("N,M", [(1, 3000), (300, 700)])
def test_cross_captured_and_on_another_stream(pl, N, M):
    """A captured call replays with new lengths and inputs, also while another stream works; two graphs have their own."""
    B, HQ, H, D = 2, 8, 4, 128
    q, k, v = rand(1, B, N, HQ, D, dtype=BF16), rand(2, B, M, H, D, dtype=BF16), rand(3, B, M, H, D, dtype=BF16)
    kl = torch.tensor([M, M // 2], dtype=torch.int32, device=DEV)
    want, wl = pl.cross_attention(q, k, v, key_lens=kl)
    outs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = pl.cross_attention(q, k, v, key_lens=kl)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], wl)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pl.cross_attention(q, k, v, key_lens=kl))
        graphs.append(g)
    kl.copy_(torch.tensor([M // 3, 0], dtype=torch.int32))
    q.mul_(0.5)
    fresh = pl.cross_attention(q, k, v, key_lens=kl)
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
            pl.cross_attention(q, k, v, key_lens=kl)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], fresh[0]) and torch.equal(o[1], fresh[1])


def test_refused_on_the_device(pl, lib):
    x, c = rand(1, 4, 2, 64, dtype=BF16), torch.zeros(4, 32, device=DEV)
    starts = torch.zeros(3, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="adjacent"):
        pl.rotate(rand(1, 4, 2, 128, dtype=BF16)[..., ::2], None, c, c)
    with pytest.raises(ValueError, match="cos_table"):
        pl.rotate(x, None, c.double(), c.double())
    with pytest.raises(ValueError, match="k:"):
        pl.rotate(x, x.float(), c, c)
    with pytest.raises(lib.BsaError):
        pl.rotate(x, None, c, c, q_weight=torch.ones(64, device=DEV), transpose=True)
    with pytest.raises(TypeError):
        pl.rotate(x.half(), None, c, c)
    with pytest.raises(ValueError, match="positions"):
        pl.rotary_table(torch.zeros(4, dtype=torch.int64, device=DEV), torch.zeros(8, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError, match="tables"):
        pl.cache_append_rotated(x, x, torch.zeros(4, dtype=torch.int64, device=DEV), pl.new_cache(1, 2, 16, 64), c[:3], c[:3])
    with pytest.raises(ValueError, match="without q"):
        pl.cache_append_rotated(x, x, torch.zeros(4, dtype=torch.int64, device=DEV), pl.new_cache(1, 2, 16, 64), c, c, q_out=x)
    with pytest.raises(ValueError, match="v:"):
        pl.cross_attention(x[None], x[None], x[None].float())
    with pytest.raises(ValueError, match="lse"):
        pl.cross_attention(x[None], x[None], x[None], lse=torch.zeros(1, 2, 4, device=DEV))
    with pytest.raises(ValueError, match="query_start"):
        pl.cross_attention(x, x, x, query_start=starts.long(), key_start=starts)
    with pytest.raises(lib.BsaError, match="scale"):
        pl.cross_attention(x[None], x[None], x[None], scale=-1.0)


# ---------------------------------------------------------------- together

def test_serving_step_of_a_rotated_cache_and_encoder_states(pl):
    """Two steps of three requests: tables, rotary table, rotated append, attention over the cache, cross attention to
    each request's states; a captured second step replays a smaller batch."""
    R, HQ, H, D, page, M, cap = 3, 4, 2, 64, 16, 40, 24
    cache = pl.TokenCache(R, 16, 6, H, D, page)
    freq = pl.rotary_frequencies(D // 2, scaling="parts", stretch=4.0, trained=64)
    states = rand(9, R, M, 2, H, D, dtype=BF16)
    mlens = [40, 0, 17]
    kl = torch.tensor(mlens, dtype=torch.int32, device=DEV)
    lens = [0, 0, 0]
    held = {r: [] for r in range(R)}
    for step_no, new in enumerate(([9, 4, 11], [10, 6, 11])):
        step = cache.step(torch.tensor(new, dtype=torch.int32, device=DEV), cap)
        cos, sin = freq.table(step.token_pos)
        rows = rand(20 + step_no, cap, HQ + 2 * H, D, dtype=BF16)
        vals = tuple(torch.zeros(cap, H, D, dtype=BF16, device=DEV) for _ in range(2))
        q = cache.append(rows[:, HQ:HQ + H], rows[:, HQ + H:], step, vals, rotary=(cos, sin), q=rows[:, :HQ])
        o, lse = cache.attend(q, step)
        c, cl = pl.cross_attention(o, states[:, :, 0], states[:, :, 1], key_lens=kl, query_start=step.query_start)
        start = 0
        for r in range(R):
            n = new[r] - lens[r]
            for i in range(n):
                t = start + i
                pos = lens[r] + i
                wc, ws = oracle.rotary_table([pos], freq.turns.tolist(), factor=freq.factor)
                assert np.max(np.abs(f64(cos[t]) - wc)) <= 4 * freq.factor * 2.0 ** -24
                held[r].append(vals[0][t])
            check_rows(c[start:start + n], cl[start:start + n], o[start:start + n], states[r, :mlens[r], 0],
                       states[r, :mlens[r], 1], D ** -0.5, BF16)
            for i in range(n):  # the values as stored are what the cache attention reads
                t, K = start + i, torch.stack(held[r][:lens[r] + i + 1]).float()
                want = oracle_rotate(rows[t:t + 1, :HQ], cos[t:t + 1], sin[t:t + 1], False, False, BF16)
                assert torch.equal(q[t:t + 1].cpu(), want)
                s = f64(q[t]).reshape(H, HQ // H, D) @ np.swapaxes(np.swapaxes(f64(K), 0, 1), 1, 2) * D ** -0.5
                w = np.log(np.exp(s).sum(-1)).reshape(-1)
                assert np.max(np.abs(f64(lse[t]) - w)) <= 2.0 ** -8 * np.max(np.abs(s)) + 1e-3
            start += n
        lens = list(new)


def test_video_step_rotate_block_sparse_cross(pl):
    """A video block's two attentions: norm and rotation into heads-first rows, block-sparse over them, cross attention
    of its output to a caption."""
    T, Hh, W, h, D, M = 4, 8, 16, 2, 128, 77
    N = T * Hh * W
    grid = torch.stack(torch.meshgrid(torch.arange(T), torch.arange(Hh), torch.arange(W), indexing="ij"), -1).view(N, 3)
    freq = pl.rotary_frequencies(D, sections=[44, 42, 42])
    cos, sin = freq.table(grid.int().to(DEV).contiguous())
    qkv = rand(1, 1, N, 3 * h, D, dtype=BF16)
    w = torch.ones(D, device=DEV)
    q, k = pl.rotate(qkv[:, :, :h], qkv[:, :, h:2 * h], cos, sin, interleaved=True, q_weight=w, k_weight=w, heads_first=True)
    v = qkv[:, :, 2 * h:].transpose(1, 2).contiguous()
    geom = pl.Geometry(T, Hh, W, 2, 4, 16)
    res = pl.block_sparse_attention(q[0], k[0], v[0], geom, geom.num_blocks)
    rows = qkv[0, :, :2 * h]
    x = oracle.rotate(oracle.rms_norm(f64(rows), np.ones(D), 1e-6), f64(cos), f64(sin), True)
    # every block kept: dense attention of the rotated rows, to the norm of the bf16 roundings of q, k, weights and output
    for i in range(h):
        want, _ = oracle.softmax_attention(x[:, i], x[:, h + i], f64(v[0, i]), D ** -0.5)
        assert np.linalg.norm(f64(res.out[i]) - want) <= 4 * 2.0 ** -8 * np.linalg.norm(want)
    text = rand(5, 1, M, 2, h, D, dtype=BF16)
    lens = torch.tensor([50], dtype=torch.int32, device=DEV)
    out, lse = pl.cross_attention(res.out[None].transpose(1, 2), text[:, :, 0], text[:, :, 1], key_lens=lens)
    check_rows(out[0], lse[0], res.out.transpose(0, 1), text[0, :50, 0], text[0, :50, 1], D ** -0.5, BF16)
