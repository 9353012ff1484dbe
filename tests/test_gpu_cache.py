"""The paged 4-bit cache on the GPU against its oracle: tables (a12), append (a13), attention (a14), and a run of
the three as a serving step uses them.

Tolerances, from the arithmetic (u = half a step relative to the value):
* tables and stored bytes: equal.
* attention, with A = sum_j p_j |v_j| per output channel and B = max_j sum_c |q_c k_jc| * scale per row:
  - a float32 logit is off by at most (D + 8) 2^-24 B from its sum and 2^-22 B from q in two float16 parts (bf16 q
    is exact in one), so a weight by twice that, and by 2^-22 from exp2;
  - a weight is held in float16 (u = 2^-11) for bf16 outputs, in two float16 parts (2^-22) for float32 ones;
  - float16's smallest step is 2^-24 and the tensor-core kernel holds 2^11 times each weight relative to a reference
    that is never above the row's largest logit, so no weight (the largest is at most 1) is held closer than half a
    step, 2^-25 2^-11 = 2^-36: F = 2^-36 sum_j |v_j| more per channel (it shows where a row's only large weight meets
    a zero of V: o ~ 1e-21 there, and A no larger);
  - sums over n keys add n 2^-24; the output's own rounding is u = 2^-8 |o| (bf16), 2^-24 |o| (float32).
  LSE: the logit's error, n 2^-24 + 2^-22 for the sum, 2^-24 |lse| for its rounding."""

import os

import numpy as np
import pytest
import torch

import oracle
from parity import set_force_simt

pytestmark = pytest.mark.gpu

DEV = "cuda"


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


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(x), device=DEV).to(dtype)


# ---------------------------------------------------------------- a12 tables

def tables_case(seed, R, P, max_pages, slack=3, kind="mixed"):
    """old, new lengths, table, pool, count: distinct pages, every request's held pages in its row."""
    rng = np.random.default_rng(seed)
    old = rng.integers(0, max_pages * P + 1, R)
    if kind == "mixed":
        new = np.where(rng.random(R) < 0.2, 0, np.clip(old + rng.integers(-3 * P, 3 * P, R), 0, max_pages * P))
    elif kind == "decode":
        old = np.minimum(old, max_pages * P - 1)
        new = old + 1
    elif kind == "prefill":
        old, new = np.zeros(R, np.int64), np.maximum(old, 1)
    else:  # finish
        new = np.zeros(R, np.int64)
    held, wanted = -(-old // P), -(-new // P)
    n_pages = max(1, int(held.sum() + np.maximum(wanted - held, 0).sum() - np.maximum(held - wanted, 0).sum()) + slack)
    n_pages = max(n_pages, int(held.sum()) + slack)
    ids = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    pool = np.full(n_pages, -7)
    pool[:n_pages - at] = ids[at:]
    return old, new, table, pool, n_pages - at


def run_tables(pl, old, new, P, table, pool, count, max_tokens, alias=False):
    t = dict(table=dev(table), pool=dev(pool), count=dev([count]), new=dev(new))
    R = len(old)
    out = (t["count"] if alias else dev([-9]), dev(np.full(R + 1, -9)), dev(np.full(max_tokens, -9)),
           dev(np.full(max_tokens, -9)), dev(np.full(max_tokens, -9), torch.int64))
    step = pl.cache_tables(dev(old), t["new"], P, t["table"], t["pool"], t["count"], max_tokens, out=out)
    return step, t


def check_tables(step, t, want, new, old):
    ok, table, pool, count, start, req, pos, slots = want
    assert np.array_equal(t["table"].cpu().numpy(), table)
    assert np.array_equal(t["pool"].cpu().numpy(), pool)
    assert step.pool_count.item() == count
    assert np.array_equal(step.query_start.cpu().numpy(), start)
    assert np.array_equal(step.token_req.cpu().numpy(), req)
    assert np.array_equal(step.token_pos.cpu().numpy(), pos)
    assert np.array_equal(step.slots.cpu().numpy(), slots)
    assert np.array_equal(t["new"].cpu().numpy(), new if ok else old)


@pytest.mark.parametrize("R,P,max_pages,kind,extra", [
    (1, 16, 1, "decode", 0), (1, 16, 4, "prefill", 5), (3, 16, 3, "mixed", 7), (64, 64, 20, "decode", 0),
    (64, 64, 20, "decode", 13), (33, 32, 9, "mixed", 1), (40, 1024, 2, "finish", 3), (257, 16, 5, "mixed", 100),
    (1024, 16, 3, "decode", 1), (1025, 16, 3, "mixed", 0), (37, 128, 40, "prefill", 2), (2500, 16, 4, "mixed", 9), (2400, 32, 5, "mixed", 3),
    (300, 16, 70, "prefill", 0), (60, 16, 300, "mixed", 5000), (1, 1024, 9, "prefill", 1),
    (700, 64, 17, "mixed", 30), (90, 16, 600, "finish", 1),
])
@pytest.mark.parametrize("alias", [False, True])
def test_tables(lib, pl, R, P, max_pages, kind, extra, alias):
    old, new, table, pool, count = tables_case(R + P, R, P, max_pages, kind=kind)
    most = int(np.maximum(new - old, 0).sum()) + extra
    want = oracle.cache_tables(old, new, P, table, pool, count, most)
    assert want[0]
    step, t = run_tables(pl, old, new, P, table, pool, count, most, alias)
    check_tables(step, t, want, new, old)


@pytest.mark.parametrize("R", [5, 1500, 2600])
@pytest.mark.parametrize("what", ["pages", "tokens", "negative", "long", "count", "overflow"])
def test_tables_refuse_as_a_whole(lib, pl, R, what):
    P, max_pages = 16, 4
    old, new, table, pool, count = tables_case(R, R, P, max_pages, slack=3 if what != "overflow" else 0, kind="mixed")
    most, code = int(np.maximum(new - old, 0).sum()), lib.BSA_ERR_INDEX
    if what == "pages":
        new = np.full(R, max_pages * P)
        most, count, code = R * P * max_pages, 0, lib.BSA_ERR_CAPACITY
    elif what == "tokens":
        most, code = most - 1, lib.BSA_ERR_CAPACITY
    elif what == "negative":
        new[R // 2] = -1
    elif what == "long":
        old[0] = max_pages * P + 1
    elif what == "count":
        count = len(pool) + 1
    else:  # more pages come back than the pool has room for
        old, new, count = np.full(R, max_pages * P), np.zeros(R, np.int64), len(pool)
        table = np.zeros((R, max_pages), np.int64)
    want = oracle.cache_tables(old, new, P, table, pool, count, most)
    assert not want[0]
    step, t = run_tables(pl, old, new, P, table, pool, count, most)
    check_tables(step, t, want, new, old)
    assert lib.bsa_device_status() == code


def test_tables_report_a_page_that_is_none(lib, pl):
    # a held page id outside the cache: its tokens have no slot; the rest of the step is done
    old, new, table, pool = [3, 3], [4, 4], np.array([[99], [1]]), np.arange(4)
    step, t = run_tables(pl, np.array(old), np.array(new), 16, table, pool, 0, 2)
    assert step.slots.tolist() == [-1, 19] and step.token_req.tolist() == [0, 1]
    assert lib.bsa_device_status() == lib.BSA_ERR_INDEX


def test_tables_shrink_undoes_grow(lib, pl):
    old, new, table, pool, count = tables_case(8, 50, 32, 12, kind="prefill")
    most = int(new.sum())
    t, a, b = dict(table=dev(table), pool=dev(pool), count=dev([count])), dev(old), dev(new)
    for x, y in ((a, b), (b, a), (a, b), (b, a)):
        out = (t["count"], torch.empty(51, dtype=torch.int32, device=DEV), torch.empty(most, dtype=torch.int32, device=DEV),
               torch.empty(most, dtype=torch.int32, device=DEV), torch.empty(most, dtype=torch.int64, device=DEV))
        pl.cache_tables(x, y.clone(), 32, t["table"], t["pool"], t["count"], most, out=out)
        if y is a:
            assert t["count"].item() == count and np.array_equal(t["pool"].cpu().numpy()[:count], pool[:count])


# ---------------------------------------------------------------- a13 append

def oracle_bytes(cache, slots, k, v, ks, vs):
    cache = cache.copy()
    for t, s in enumerate(slots):
        if s >= 0:
            oracle.store(cache, int(s), k[t], v[t], ks, vs)
    return cache


@pytest.mark.parametrize("T,H,D,P,dtype,scales,strided", [
    (1, 1, 16, 16, torch.float32, False, False), (1, 4, 128, 64, torch.bfloat16, True, True),
    (19, 3, 64, 16, torch.float32, True, True), (50, 2, 128, 32, torch.bfloat16, True, False),
    (33, 2, 48, 1024, torch.bfloat16, False, True), (17, 5, 80, 64, torch.float32, True, False),
    (130, 1, 128, 128, torch.bfloat16, False, True),
])
def test_append_bytes_and_values(lib, pl, T, H, D, P, dtype, scales, strided):
    rng = np.random.default_rng(T)
    rows = torch.tensor(rng.standard_normal((T, 3 * H, D)) * 10.0 ** rng.integers(-3, 3, (T, 3 * H, 1)), dtype=dtype)
    rows[0, 0] = 0  # a group of zeros
    n_pages = -(-(T + 3) // P) + 2
    slots = rng.permutation(n_pages * P)[:T]
    slots[rng.random(T) < 0.1] = -1
    cache0 = rng.integers(0, 256, (n_pages, H, P // 16, 18 * D)).astype(np.uint8)
    ks, vs = (rng.uniform(0.05, 2, (2, H)).astype(np.float32) if scales else (None, None))
    d = rows.to(DEV)
    k, v = (d[:, H:2 * H], d[:, 2 * H:]) if strided else (d[:, :H].contiguous(), d[:, H:2 * H].contiguous())
    cache = dev(cache0, torch.uint8)
    vals = tuple(torch.full((T, H, D), -77.0, dtype=dtype, device=DEV) for _ in range(2))
    dk, dv = (None if x is None else dev(x, torch.float32) for x in (ks, vs))
    pl.cache_append(k, v, dev(slots, torch.int64), cache, dk, dv, values=vals)
    want = oracle_bytes(cache0, slots, k.double().cpu().numpy(), v.double().cpu().numpy(), ks, vs)
    assert np.array_equal(cache.cpu().numpy(), want)
    for t in range(T):
        if slots[t] < 0:
            assert all((x[t] == -77).all() for x in vals)
            continue
        for got, x in zip(vals, oracle.load(want, int(slots[t]), ks, vs)):
            # code * scale is exact, the head's scale is one float32 product, the type one more rounding
            u = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
            assert (np.abs(got[t].double().cpu().numpy() - x) <= u * np.abs(x)).all()
    again = dev(cache0, torch.uint8)
    pl.cache_append(k, v, dev(slots, torch.int64), again, dk, dv)  # without the values: the same bytes
    assert torch.equal(again, cache)


def test_append_unaligned_rows(lib, pl):
    # rows whose addresses are not multiples of 16 bytes: same bytes as aligned ones
    T, H, D = 9, 2, 32
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.randn((T, 2 * H, D), device=DEV).to(dtype)
        flat = torch.zeros(T * (2 * H * D + 1) + 1, dtype=dtype, device=DEV)[1:]
        odd = flat.as_strided((T, 2 * H, D), (2 * H * D + 1, D, 1))
        odd.copy_(x)
        slots = torch.arange(T, device=DEV)
        a, b = pl.new_cache(1, H, 16, D), pl.new_cache(1, H, 16, D)
        pl.cache_append(x[:, :H], x[:, H:], slots, a)
        pl.cache_append(odd[:, :H], odd[:, H:], slots, b)
        assert torch.equal(a, b)


def test_append_borders_and_non_finite(lib, pl):
    # every rounding border of the codes at several scales (ties to the even code), float32 neighbours of the
    # borders, groups with NaN and infinities, the largest floats and subnormals
    steps = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    rows = []
    for s in [m / 8 * 2.0 ** e for m in range(8, 16) for e in (-6, -1, 0, 5)] + [3 * 2.0 ** -9]:
        x = np.zeros(16)
        x[0], x[1:8], x[8:15], x[15] = 6 * s, steps * s, -steps * s, 0
        rows.append(x)
        y = np.float32(x)
        rows += [np.nextafter(y, np.float32(np.inf)).astype(np.float64), np.nextafter(y, np.float32(-np.inf)).astype(np.float64)]
    for bad in (np.nan, np.inf, -np.inf):
        x = np.linspace(-3, 3, 16)
        x[7] = bad
        rows.append(x)
    rows += [np.full(16, 3.4e38), np.full(16, -1e-40), np.full(16, 2.0 ** -12), np.linspace(-2688, 2688, 16) * 1.01]
    # borders of the group scale: six times the midpoint of two E4M3 values, and its float32 neighbours
    for b in (1, 7, 8, 50, 51, 100, 125):
        mid = np.float32(3 * (oracle.e4m3_value(b) + oracle.e4m3_value(b + 1)))
        for top in (mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(1e9))):
            rows.append(np.linspace(-0.9, 1, 16) * float(top))
            rows[-1][15] = float(top)
    x = torch.tensor(np.array(rows), dtype=torch.float32)[:, None]
    T = x.shape[0]
    n_pages = -(-T // 16)
    cache = pl.new_cache(n_pages, 1, 16, 16)
    vals = tuple(torch.empty((T, 1, 16), device=DEV) for _ in range(2))
    pl.cache_append(x.to(DEV), -x.to(DEV), torch.arange(T, device=DEV), cache, values=vals)
    bytes_ = cache.cpu().numpy()
    for t in range(T):
        for which, r in ((0, x[t, 0].numpy()), (1, -x[t, 0].numpy())):
            codes, byte = oracle.quantise_group(r)
            got = oracle.load(bytes_, t)[which][0]
            if codes is None:
                assert np.isnan(got).all() and vals[which][t].isnan().all()
                continue
            want = np.array([oracle.code_value(int(c)) for c in codes]) * oracle.e4m3_value(byte)
            assert np.array_equal(got, want), (t, which)
            assert np.array_equal(vals[which][t, 0].double().cpu().numpy(), want)


def test_append_stores_the_sign_of_zero(lib, pl):
    """Bytes of zeros with a sign: in a group of numbers, of zeros, and where x / g underflows (g = 4)."""
    for dtype in (torch.float32, torch.bfloat16):
        tiny = 2.0 ** -149 if dtype == torch.float32 else 2.0 ** -133  # the smallest numbers
        rows = torch.zeros((5, 1, 32), dtype=dtype)
        rows[0] = torch.linspace(-3, 3, 32).to(dtype)
        rows[0, 0, 1::2] = -0.0
        rows[1, 0, ::3] = -0.0                       # groups of zeros only
        rows[2, 0] = torch.tensor([-tiny, tiny]).repeat(16).to(dtype)
        rows[2, 0, 0], rows[2, 0, 31] = 5.0, -5.0
        rows[3, 0] = torch.tensor([-tiny, 0.0, tiny, -0.0]).repeat(8).to(dtype)
        rows[4, 0, 20] = -448 * 6.0
        rows[4, 0, 21:] = -0.0
        for g in (1.0, 4.0):
            scale, slots = np.full(1, g, np.float32), np.arange(5)
            cache = torch.full((1, 1, 1, 18 * 32), 0xAA, dtype=torch.uint8, device=DEV)
            d = rows.to(DEV)
            pl.cache_append(d, -d, dev(slots, torch.int64), cache, dev(scale, torch.float32), dev(scale, torch.float32))
            x = rows.double().numpy()
            want = oracle_bytes(np.full((1, 1, 1, 18 * 32), 0xAA, np.uint8), slots, x, -x, scale, scale)
            assert np.array_equal(cache.cpu().numpy(), want), (dtype, g)


def test_append_reports_a_slot_outside_the_cache(lib, pl):
    x = torch.randn((3, 1, 16), device=DEV)
    cache = pl.new_cache(2, 1, 16, 16)
    pl.cache_append(x, x, dev([32, -2, 5], torch.int64), cache)
    assert lib.bsa_device_status() == lib.BSA_ERR_INDEX
    got = cache.cpu().numpy()
    assert got[1].sum() == 0 and np.array_equal(got, oracle_bytes(np.zeros_like(got), [-1, -1, 5], x.cpu().double().numpy(),
                                                                  x.cpu().double().numpy(), None, None))


# ---------------------------------------------------------------- a14 attention

def attend_case(seed, R, n, lo, hi, HQ, H, D, P, S, BS, dtype, sharp=1.0, scales=True):
    """A cache whose unseen bytes are all 0xff (NaN scales), lists in no order, and n tokens of each request."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(lo, hi + 1, R)
    max_pages = -(-hi // P)
    held = -(-lens // P)
    n_pages = int(held.sum()) + 2
    ids = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :held[r]] = ids[at:at + held[r]]
        at += held[r]
    cache = np.full((n_pages, H, P // 16, 18 * D), 0xFF, np.uint8)
    ch = np.arange(D)
    for r in range(R):
        p = np.arange(lens[r])
        page, strip, j = table[r][p // P], p % P // 16, p % 16
        for base, first, width in ((0, j * (D // 2), 1), (16 * D, j * (D // 16), 1)):
            w = D // 2 if base == 0 else D // 16
            cols = base + first[:, None] + np.arange(w)
            data = rng.integers(0, 256, (lens[r], H, w)) if base == 0 else rng.integers(0x28, 0x3C, (lens[r], H, w))
            cache[page[:, None, None], np.arange(H)[None, :, None], strip[:, None, None], cols[:, None, :]] = data
        c2 = np.arange(D // 2) * 2
        cols = 8 * D + ((c2 // 16) * 16 + j[:, None]) * 8 + c2 % 16 // 2
        cache[page[:, None, None], np.arange(H)[None, :, None], strip[:, None, None], cols[:, None, :]] = \
            rng.integers(0, 256, (lens[r], H, D // 2))
        cols = 17 * D + np.arange(D // 16) * 16 + j[:, None]
        cache[page[:, None, None], np.arange(H)[None, :, None], strip[:, None, None], cols[:, None, :]] = \
            rng.integers(0x20, 0x40, (lens[r], H, D // 16))
    assert ch.size == D
    T = R * n
    req = np.repeat(np.arange(R), n)
    pos = np.concatenate([np.arange(x - n, x) for x in lens]) if T else np.zeros(0, np.int64)
    q = torch.tensor(rng.standard_normal((T, HQ, D)) * sharp, dtype=dtype)
    ks, vs = (rng.uniform(0.2, 2, (2, H)).astype(np.float32) if scales else (None, None))
    idx = cnt = None
    if S:
        nblk = -(-max_pages * P // BS)
        idx, cnt = np.full((T, H, S), -1), np.zeros((T, H), np.int64)
        for t in range(T):
            for h in range(H):
                got = rng.permutation(nblk)[:S]
                if pos[t] >= 0 and rng.random() < 0.8:
                    got[0] = pos[t] // BS
                cnt[t, h] = rng.integers(0, len(got) + 1)
                idx[t, h, :len(got)] = got
    return dict(q=q, cache=cache, table=table, req=req, pos=pos, ks=ks, vs=vs, idx=idx, cnt=cnt, BS=BS)


def attend(pl, c, scale=None, **over):
    a = {**c, **over}
    f = torch.float32
    return pl.cache_attention(
        a["q"].to(DEV), dev(a["cache"], torch.uint8), dev(a["table"]), dev(a["req"]), dev(a["pos"]),
        None if a["ks"] is None else dev(a["ks"], f), None if a["vs"] is None else dev(a["vs"], f),
        None if a["idx"] is None else dev(a["idx"]), None if a["cnt"] is None else dev(a["cnt"]), a["BS"], scale)


def want_attend(c, scale=None):
    """Oracle output and LSE, and the two tolerances of the module's docstring."""
    D, bf16 = c["q"].shape[2], c["q"].dtype == torch.bfloat16
    q = c["q"].double().numpy()
    args = (c["cache"], c["table"], c["req"], c["pos"], c["ks"], c["vs"], c["idx"], c["cnt"], c["BS"], scale)
    o, lse = oracle.cache_attention(q, *args)
    scale = D ** -0.5 if scale is None else scale
    T, HQ, _ = q.shape
    H, P = c["cache"].shape[1], c["cache"].shape[2] * 16
    A, B, n, F = np.zeros_like(o), np.zeros((T, HQ)), np.zeros((T, HQ)), np.zeros_like(o)
    memo = {}
    for t in range(T):
        for h in range(H):
            if c["req"][t] < 0 or c["pos"][t] < 0:
                continue
            keys = np.arange(c["pos"][t] + 1) if c["idx"] is None else np.array(
                [b * c["BS"] + u for b in c["idx"][t, h, :max(0, c["cnt"][t, h])] for u in range(c["BS"])], dtype=np.int64)
            keys = keys[keys <= c["pos"][t]]
            if not len(keys):
                continue
            kv = []
            for x in keys:
                s = int(c["table"][c["req"][t], x // P]) * P + int(x) % P
                if s not in memo:
                    memo[s] = oracle.load(c["cache"], s, c["ks"], c["vs"])
                kv.append(memo[s])
            K, V = np.array([a[h] for a, _ in kv]), np.array([b[h] for _, b in kv])
            G = HQ // H
            for r in range(h * G, (h + 1) * G):
                x = K @ q[t, r] * scale
                p = np.exp(x - lse[t, r])
                A[t, r] = p @ np.abs(V)
                F[t, r] = 2.0 ** -36 * np.abs(V).sum(0)
                B[t, r] = (np.abs(K) @ np.abs(q[t, r])).max() * abs(scale)
                n[t, r] = len(keys)
    logit = B * ((D + 8) * 2.0 ** -24 + 2.0 ** -22)
    weight = 2 * logit + 2.0 ** -22 + n * 2.0 ** -24 + (2.0 ** -11 if bf16 else 2.0 ** -22)
    tol = F + A * weight[..., None] + np.abs(o) * (2.0 ** -8 if bf16 else 2.0 ** -24) * 1.01
    return o, lse, tol, logit + n * 2.0 ** -24 + 2.0 ** -22 + np.abs(np.where(np.isfinite(lse), lse, 0)) * 2.0 ** -24


def check_attend(out, lse, want):
    o, l, tol, ltol = want
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    live = ~np.isnan(l)
    assert np.isfinite(out[live]).all()
    err = np.abs(out - o)[live] - tol[live]
    assert err.max(initial=0) <= 0, "output off by %.3g over its tolerance" % err.max()
    empty = live & (l == -np.inf)
    assert (lse[empty] == -np.inf).all() and not out[empty].any()
    rest = live & (l != -np.inf)
    err = np.abs(lse - np.where(rest, l, 0))[rest] - ltol[rest]
    assert err.max(initial=0) <= 0, "LSE off by %.3g over its tolerance" % err.max()


ATTEND_CASES = [
    # R, n, lo, hi, HQ, H, D, P, S, BS, dtype
    (1, 1, 1, 1, 1, 1, 16, 16, 0, 0, torch.float32),
    (1, 1, 1, 1, 16, 1, 128, 64, 0, 0, torch.bfloat16),
    (3, 1, 5, 70, 8, 2, 128, 16, 0, 0, torch.bfloat16),
    (4, 2, 17, 200, 6, 2, 64, 32, 0, 0, torch.float32),
    (2, 1, 100, 300, 32, 2, 128, 64, 0, 0, torch.float32),
    (2, 3, 90, 333, 20, 1, 128, 128, 0, 0, torch.bfloat16),
    (2, 1, 65, 129, 40, 2, 64, 64, 0, 0, torch.bfloat16),
    (3, 1, 20, 100, 6, 3, 80, 16, 0, 0, torch.bfloat16),
    (2, 2, 30, 150, 5, 5, 48, 32, 0, 0, torch.float32),
    (3, 1, 64, 400, 16, 1, 128, 64, 5, 64, torch.bfloat16),
    (3, 2, 3, 500, 8, 2, 128, 16, 6, 32, torch.bfloat16),
    (2, 3, 8, 300, 8, 2, 64, 64, 4, 16, torch.float32),
    (2, 1, 300, 600, 32, 2, 128, 32, 3, 128, torch.bfloat16),
    (2, 2, 50, 400, 12, 3, 64, 128, 7, 48, torch.bfloat16),
    (2, 1, 40, 200, 4, 2, 96, 16, 3, 16, torch.float32),
    (1, 1, 700, 700, 7, 1, 128, 1024, 0, 0, torch.bfloat16),
    (1, 1, 600, 600, 2, 2, 128, 16, 40, 16, torch.float32),
]


@pytest.mark.parametrize("case", ATTEND_CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_attention(lib, pl, case):
    c = attend_case(sum(case[:-1]), *case)
    want = want_attend(c)
    check_attend(*attend(pl, c), want)
    set_force_simt(True)
    check_attend(*attend(pl, c), want)


def test_attention_running_maximum_moves_per_row(lib, pl):
    """Logits that grow along the keys, by other amounts in each head: every row's sum and output are rescaled by its
    own factor, tile after tile, in one warp's run as well as in a split row."""
    for dtype in (torch.float32, torch.bfloat16):
        for D in (64, 128):
            for HQ in (3, 8, 16):
                for R, n in ((1, 700), (60, 1500)):
                    c = attend_case(HQ, R, 1, n, n, HQ, 1, D, 64, 0, 0, dtype, scales=False)
                    c["cache"][..., 16 * D:17 * D] = 0x30  # K scales 0.5, but growing with the position below
                    for r in range(R):
                        for p in range(n):
                            c["cache"][c["table"][r, p // 64], 0, p % 64 // 16, 16 * D + p % 16 * (D // 16):
                                       16 * D + (p % 16 + 1) * (D // 16)] = 0x20 + min(0x30, p * 0x30 // n)
                    c["q"] = (c["q"].double() * torch.logspace(-1, 0.3, HQ, dtype=torch.float64)[:, None]).to(dtype)
                    out, lse = attend(pl, c)
                    pick = slice(0, 2)
                    d = {**c, "q": c["q"][pick], "req": c["req"][pick], "pos": c["pos"][pick]}
                    check_attend(out[pick], lse[pick], want_attend(d))


# Batches that are cut in each of the ways the tensor-core kernel has: a row to a cluster (few rows), equal runs of
# tiles with a join behind them (more rows than CTAs, or long ones), whole rows to clusters (many rows with lists),
# whole rows to warps (more rows than a start is searched for)
JOIN_8 = (120, 1, 1, 330, 32, 4, 128, 64, 0, 0, torch.bfloat16)
JOIN_16 = (80, 1, 1, 430, 64, 4, 128, 16, 0, 0, torch.bfloat16)
UNITS_8 = (150, 2, 2, 700, 32, 4, 128, 64, 5, 64, torch.bfloat16)
ROWS_8 = (70, 30, 30, 200, 8, 4, 64, 16, 6, 16, torch.bfloat16)
UNITS_16 = (150, 2, 2, 700, 64, 4, 128, 32, 9, 32, torch.bfloat16)
BATCHES = [
    # R, n, lo, hi, HQ, H, D, P, S, BS, dtype
    JOIN_8, JOIN_16, (40, 2, 2, 300, 8, 4, 64, 32, 0, 0, torch.float32),
    (40, 1, 1, 830, 32, 4, 128, 64, 0, 0, torch.bfloat16),
    (40, 1, 1, 830, 64, 4, 128, 16, 0, 0, torch.bfloat16),
    (23, 2, 2, 900, 8, 4, 64, 32, 0, 0, torch.float32),
    (3, 1, 9000, 30000, 40, 1, 64, 128, 0, 0, torch.bfloat16),
    (2, 1, 20000, 60000, 3, 1, 128, 64, 0, 0, torch.float32),
    UNITS_8, UNITS_16,
    (140, 3, 3, 600, 20, 4, 64, 16, 3, 128, torch.float32),
    ROWS_8,
    (70, 30, 30, 200, 36, 4, 64, 16, 6, 16, torch.float32),
    (180, 30, 30, 100, 4, 2, 64, 16, 0, 0, torch.bfloat16),
    (180, 30, 30, 60, 4, 4, 64, 16, 3, 16, torch.bfloat16),
]


@pytest.mark.parametrize("case", BATCHES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_attention_batches(lib, pl, case):
    c = attend_case(sum(case[:-1]), *case)
    T = c["q"].shape[0]
    rng = np.random.default_rng(T)
    pad = rng.random(T) < (0.05 if T > 10 else 0)
    c["req"] = np.where(pad, -1, c["req"])
    out, lse = attend(pl, c)
    again = attend(pl, c)
    live = torch.as_tensor(~pad, device=DEV)
    assert torch.equal(out[live], again[0][live]) and torch.equal(lse[live], again[1][live])  # fixed order of sums
    pick = np.sort(rng.permutation(T)[:40 if case[3] < 2000 else 2])
    d = {**c, "q": c["q"][pick], "req": c["req"][pick], "pos": c["pos"][pick]}
    if c["idx"] is not None:
        d["idx"], d["cnt"] = c["idx"][pick], c["cnt"][pick]
    pick = torch.as_tensor(pick, device=DEV)
    check_attend(out[pick], lse[pick], want_attend(d))
    # every row against the CUDA-core kernel: each is within its own tolerance of the exact row, bf16 outputs within
    # two roundings (2 * 2^-8 |o|) and both kernels' weights (2^-11 A, A <= sum p |v| <= max |v|)
    set_force_simt(True)
    o2, l2 = attend(pl, c)
    both = live[:, None] & torch.isfinite(l2)
    assert torch.equal(both, live[:, None] & torch.isfinite(lse))
    a, b = out.float()[both], o2.float()[both]
    u = 2.0 ** -8 if c["q"].dtype == torch.bfloat16 else 2.0 ** -14
    assert (a - b).norm() <= 2 * u * b.norm()
    assert (lse - l2)[both].abs().max() <= 2.0 ** -14 * (1 + l2[both].abs().max())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_sharp_and_scaled_logits(lib, pl, D, dtype):
    # logits of tens: a few keys carry each row, the running maximum moves, most weights underflow
    c = attend_case(5, 2, 1, 200, 500, 8, 2, D, 64, 0, 0, dtype, sharp=6.0)
    check_attend(*attend(pl, c), want_attend(c))
    for scale in (0.0, -0.05):
        check_attend(*attend(pl, c, scale=scale), want_attend(c, scale))
    c["q"] = c["q"] * (1e-6 if dtype == torch.float32 else 2.0 ** -20)
    check_attend(*attend(pl, c), want_attend(c))


@pytest.mark.parametrize("D", [64, 80, 128])
def test_attention_rows_without_keys_and_padding(lib, pl, D):
    c = attend_case(9, 3, 2, 40, 90, 8, 2, D, 16, 3, 32, torch.bfloat16)
    # columns for later blocks: a list entry past the table's last block is an error, not an unseen block
    c["table"] = np.pad(c["table"], ((0, 0), (0, 4)), constant_values=-1)
    c["cnt"][0], c["cnt"][1] = 0, -4          # empty lists
    c["pos"][2] = -1                          # a position of none
    c["idx"][3], c["cnt"][3] = c["pos"][3] // 32 + 1, 1  # only a later block
    c["req"][5] = -1                          # padding
    want = want_attend(c)
    T, HQ = c["q"].shape[:2]
    out = torch.full((T, HQ, D), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, HQ), 7.0, device=DEV)
    nb = lib.bsa_cache_attention_workspace(T, HQ, 2, D, 3 * 32)
    ws = torch.empty(max(nb, 16), dtype=torch.uint8, device=DEV)
    cache = dev(c["cache"], torch.uint8)
    lib.bsa_fwd_cache_tokens(c["q"].to(DEV), T, HQ, 2, D, cache, cache.shape[0], 16, dev(c["table"]), 3,
                             c["table"].shape[1], dev(c["req"]), dev(c["pos"]), dev(c["ks"], torch.float32),
                             dev(c["vs"], torch.float32), dev(c["idx"]), dev(c["cnt"]), 3, 32, D ** -0.5, out, lse, ws)
    check_attend(out, lse, want)
    assert (out[5] == 5).all() and (lse[5] == 7).all()
    assert np.isneginf(want[1][:4]).all()


def test_attention_counts_a_block_twice_that_is_listed_twice(lib, pl):
    for D in (48, 64, 128):
        c = attend_case(12, 2, 1, 100, 200, 4, 1, D, 16, 4, 16, torch.float32)
        c["idx"][:] = np.array([1, 3, 1, 0])
        c["cnt"][:] = 4
        check_attend(*attend(pl, c), want_attend(c))


def test_attention_reports_bad_indices_and_goes_on(lib, pl):
    for D in (48, 128):
        c = attend_case(13, 2, 1, 100, 200, 4, 2, D, 16, 4, 32, torch.bfloat16)
        c["idx"][:], c["cnt"][:] = np.array([0, 2, 1, 1]), 3
        good = want_attend(c)
        for change in ("block high", "block negative", "count", "page", "request", "position"):
            d = {k: (v.copy() if isinstance(v, np.ndarray) else v) for k, v in c.items()}
            want = good
            if change == "block high":
                d["idx"][0, 0, 1] = 1 << 20
            elif change == "block negative":
                d["idx"][0, 0, 1] = -1
            elif change == "count":
                d["cnt"][0, 0] = 9
                c4 = {**c, "cnt": c["cnt"].copy()}
                c4["cnt"][0, 0] = 4
                want = want_attend(c4)
            elif change == "page":
                d["table"][0, 4] = d["cache"].shape[0]  # keys 64..79: the first half of block 2
            elif change == "request":
                d["req"][0] = 2
            else:
                d["pos"][0] = d["table"].shape[1] * 16
            out, lse = attend(pl, d)
            assert lib.bsa_device_status() == lib.BSA_ERR_INDEX, change
            o, l, tol, ltol = (x[1:] for x in want)
            check_attend(out[1:], lse[1:], (o, l, tol, ltol))
            if change in ("block high", "block negative"):
                e = {**c, "idx": c["idx"].copy(), "cnt": c["cnt"].copy()}
                e["idx"][0, 0, :2], e["cnt"][0, 0] = [0, 1], 2
                check_attend(out, lse, want_attend(e))
            elif change == "page":
                e = {**c, "idx": c["idx"].copy(), "cnt": c["cnt"].copy(), "BS": 16}
                e["idx"] = np.tile(np.array([0, 1, 5, 2, 3]), (2, 2, 1))
                e["cnt"][:] = 5
                w = want_attend(e)
                check_attend(out[:1], lse[:1], tuple(x[:1] for x in w))
            elif change == "position":
                assert not out[0].any() and torch.isneginf(lse[0]).all()
            elif change == "count":
                check_attend(out, lse, want)


def test_attention_takes_strided_queries_and_lse_is_optional(lib, pl):
    for dtype in (torch.float32, torch.bfloat16):
        c = attend_case(14, 3, 2, 20, 90, 8, 2, 128, 32, 0, 0, dtype)
        wide = torch.randn((6, 12, 128)).to(dtype).to(DEV)
        wide[:, 2:10] = c["q"].to(DEV)
        a = attend(pl, {**c, "q": wide[:, 2:10]})
        odd = torch.zeros(6 * (8 * 128 + 1) + 1, dtype=dtype, device=DEV)[1:].as_strided((6, 8, 128), (8 * 128 + 1, 128, 1))
        odd.copy_(c["q"])
        b = attend(pl, {**c, "q": odd})
        check_attend(*a, want_attend(c))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        d = pl.cache_attention(c["q"].to(DEV), dev(c["cache"], torch.uint8), dev(c["table"]), dev(c["req"]), dev(c["pos"]),
                               dev(c["ks"], torch.float32), dev(c["vs"], torch.float32), need_lse=False)
        assert d[1] is None and torch.equal(d[0], a[0])


def test_attention_propagates_nan_and_infinity_that_a_row_sees(lib, pl):
    for D in (48, 128):
        c = attend_case(15, 2, 1, 40, 60, 4, 2, D, 16, 0, 0, torch.bfloat16)
        out, lse = attend(pl, c)
        d = {**c, "cache": c["cache"].copy()}
        p = int(c["pos"][0]) - 3
        d["cache"][c["table"][0, p // 16], 1, 0, 16 * D + p % 16 * (D // 16)] = 0x7F  # a NaN key of head 1, request 0
        o2, l2 = attend(pl, d)
        assert o2[0, 2:].isnan().all() and l2[0, 2:].isnan().all()
        assert torch.equal(o2[1], out[1]) and torch.equal(o2[0, :2], out[0, :2]) and torch.equal(l2[1], lse[1])
        q = c["q"].clone()
        q[1, 3, 5] = float("nan")
        o3, l3 = attend(pl, {**c, "q": q})
        assert o3[1, 3].isnan().all() and l3[1, 3].isnan() and torch.equal(o3[1, :3], out[1, :3])


@pytest.mark.parametrize("D", [64, 80, 128])
@pytest.mark.parametrize("HQ", [4, 16])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_attention_scale_that_is_no_number(lib, pl, D, HQ, dtype):
    c = attend_case(5, 2, 1, 20, 90, HQ, 1, D, 16, 0, 0, dtype)
    out, lse = attend(pl, c, scale=float("nan"))
    assert out.isnan().all() and lse.isnan().all()


@pytest.mark.parametrize("S", [0, 2])
def test_a_step_without_tokens(lib, pl, S):
    cache = pl.new_cache(2, 2, 16, 64)
    rows = torch.zeros((0, 2, 64), device=DEV)
    pl.cache_append(rows, rows, dev(np.zeros(0), torch.int64), cache, values=(rows, rows.clone()))
    lists = (dev(np.zeros((0, 2, S))), dev(np.zeros((0, 2))), 16) if S else ()
    out, lse = pl.cache_attention(rows, cache, dev(np.zeros((1, 2))), dev(np.zeros(0)), dev(np.zeros(0)), None, None, *lists)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)


@pytest.mark.parametrize("stall", [0, 2])
@pytest.mark.parametrize("case", [JOIN_8, JOIN_16, UNITS_8, UNITS_16, ROWS_8, ATTEND_CASES[9], ATTEND_CASES[15]],
                         ids=["join-8", "join-16", "units-8", "units-16", "rows-8", "split-lists", "split"])
def test_attention_expired_wait_is_reported_and_recovers(lib, pl, case, stall):
    """A tile that is never copied: its wait runs out (after 1 ms under the switch), the kernel latches
    BSA_ERR_TIMEOUT and ends, also where other warps and the join look for its parts; the next call is as before."""
    c = attend_case(sum(case[:-1]), *case)
    want = attend(pl, c)
    os.environ["BSA_TEST_STALL_TILE"] = str(stall)
    try:
        attend(pl, c)
    finally:
        os.environ.pop("BSA_TEST_STALL_TILE")
    status = lib.bsa_device_status()
    assert status == lib.BSA_ERR_TIMEOUT or (stall > 0 and status == lib.BSA_OK)  # not every warp has a third tile
    out, lse = attend(pl, c)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,D,P", [(torch.bfloat16, 128, 64), (torch.float32, 64, 16)])
def test_serving_steps(lib, pl, dtype, D, P):
    """Prompts, decode steps with a selection, a rollback, a finished and a new request, padded token arrays: every
    step's outputs against the oracle over the rows that were fed."""
    rng = np.random.default_rng(21)
    R, H, G, most = 4, 2, 4, 96
    ks, vs = (rng.uniform(0.02, 0.05, H).astype(np.float32) for _ in range(2))
    tc = pl.TokenCache(R, 14 * 64 // P, 4 * 64 // P, H, D, P, dev(ks, torch.float32), dev(vs, torch.float32))
    lens = np.zeros(R, np.int64)
    for new in ([40, 0, 17, 3], [41, 30, 18, 4], [42, 31, 15, 5], [43, 32, 0, 6], [44, 33, 21, 7]):
        new = np.array(new)
        step = tc.step(dev(new), most)
        n = int(np.maximum(new - lens, 0).sum())
        x = torch.tensor(rng.standard_normal((most, H * (G + 2), D)), dtype=dtype)
        d = x.to(DEV)
        vals = tuple(torch.zeros((most, H, D), dtype=dtype, device=DEV) for _ in range(2))
        tc.append(d[:, H * G:H * G + H], d[:, H * G + H:], step, values=vals)
        idx = dev(np.tile(np.array([2, 0, 1]), (most, H, 1)))
        cnt = dev(np.full((most, H), 2))
        for lists in (None, (idx, cnt, 16)):
            out, lse = tc.attend(d[:, :H * G], step, *(lists or ()))
            c = dict(q=x[:n, :H * G], cache=tc.cache.cpu().numpy(), table=tc.block_table.cpu().numpy(),
                     req=step.token_req.cpu().numpy()[:n], pos=step.token_pos.cpu().numpy()[:n], ks=ks, vs=vs,
                     idx=None if lists is None else idx.cpu().numpy()[:n],
                     cnt=None if lists is None else cnt.cpu().numpy()[:n], BS=16)
            check_attend(out[:n], lse[:n], want_attend(c))
        stored = [oracle.load(c["cache"], int(s), ks, vs) for s in step.slots.cpu().numpy()[:n]]
        for w in range(2):
            want = np.array([s[w] for s in stored])
            u = 2.0 ** -24 + (2.0 ** -8 if dtype == torch.bfloat16 else 0.0)
            assert (np.abs(vals[w][:n].double().cpu().numpy() - want) <= u * np.abs(want)).all()
            assert not vals[w][n:].any()
        assert step.token_req[n:].eq(-1).all()
        lens = new
    held = int((-(-lens // P)).sum())
    assert tc.pool_count.item() == tc.pool.numel() - held
    # a step that asks for more than there is changes nothing
    before = tc.block_table.clone(), tc.lens.clone(), tc.pool_count.clone()
    step = tc.step(dev(np.full(R, 4 * 64)), 4 * 4 * 64)
    assert step.token_req.eq(-1).all() and all(torch.equal(a, b) for a, b in zip(
        before, (tc.block_table, tc.lens, tc.pool_count)))
    assert lib.bsa_device_status() == lib.BSA_ERR_CAPACITY


def test_layers_share_tables(lib, pl):
    a = pl.TokenCache(2, 8, 4, 1, 64, 16)
    b = pl.TokenCache(2, 8, 4, 1, 64, 16, tables=a)
    step = a.step(dev([5, 9]), 14)
    x = torch.randn((14, 3, 64), device=DEV)
    for c, g in ((a, 1.0), (b, -1.0)):
        c.append(g * x[:, :1], x[:, 1:2], step)
        out, _ = c.attend(x[:, 2:], step)
        assert out.isfinite().all()
    with pytest.raises(ValueError):
        b.step(dev([6, 9]), 14)
    with pytest.raises(ValueError):
        pl.TokenCache(2, 8, 4, 1, 64, 32, tables=a)


def test_a_captured_step_replays_with_new_lengths(lib, pl):
    """Tables, append and attention captured once and replayed over other lengths and rows: equal to eager calls."""
    R, H, G, D, P, most = 3, 2, 4, 128, 16, 8
    eager, graph = (pl.TokenCache(R, 40, 12, H, D, P) for _ in range(2))
    lens, rows = dev([4, 0, 2]), torch.randn((most, H * (G + 2), D), device=DEV).bfloat16()

    def go(c):
        step = c.step(lens, most)
        c.append(rows[:, H * G:H * G + H], rows[:, H * G + H:], step)
        return step, c.attend(rows[:, :H * G], step)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        go(eager)
        go(graph)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step_g, (out_g, lse_g) = go(graph)
    for new in ([5, 2, 3], [6, 3, 3], [7, 0, 4], [8, 5, 5]):
        lens.copy_(dev(new))
        rows.copy_(torch.randn(rows.shape, device=DEV))
        step, (out, lse) = go(eager)
        g.replay()
        torch.cuda.synchronize()
        n = int(step.query_start[-1])
        assert all(torch.equal(a, b) for a, b in zip(step, step_g))
        assert torch.equal(out[:n], out_g[:n]) and torch.equal(lse[:n], lse_g[:n])
        assert torch.equal(eager.cache, graph.cache) and torch.equal(eager.block_table, graph.block_table)


@pytest.mark.parametrize("case", [JOIN_8, JOIN_16, UNITS_16, ROWS_8], ids=["join-8", "join-16", "units", "rows"])
def test_captured_batches_replay(lib, pl, case):
    """Large batches captured (the join behind its kernel, the clusters) and replayed over other positions, twice,
    beside a second graph of the same call: equal to eager calls."""
    c = attend_case(sum(case[:-1]), *case)
    f = torch.float32
    d = dict(q=c["q"].to(DEV), cache=dev(c["cache"], torch.uint8), table=dev(c["table"]), req=dev(c["req"]),
             pos=dev(c["pos"]), ks=dev(c["ks"], f), vs=dev(c["vs"], f), idx=None if c["idx"] is None else dev(c["idx"]),
             cnt=None if c["cnt"] is None else dev(c["cnt"]))

    def go():
        return pl.cache_attention(d["q"], d["cache"], d["table"], d["req"], d["pos"], d["ks"], d["vs"], d["idx"], d["cnt"],
                                  c["BS"])

    go()
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            got.append(go())
    for shift in (0, 3, 40):
        d["pos"].copy_(dev(np.maximum(c["pos"] - shift, -1)))
        want = go()
        for g, (out, lse) in zip(graphs, got):
            out.zero_(), lse.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_calls_on_two_streams_do_not_disturb_each_other(lib, pl):
    cases = [attend_case(30 + i, R, 1, lo, hi, 16, 2, 128, 64, 0, 0, torch.bfloat16)
             for i, R, lo, hi in ((0, 4, 300, 800), (1, 160, 20, 150))]
    want = [want_attend(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(attend(pl, cases[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for out, lse in got[i]:
            check_attend(out, lse, want[i])
            assert torch.equal(out, got[i][0][0])


def test_prefill_over_the_stored_values_agrees_with_decoding_them(lib, pl):
    """A prompt's rows appended with their values, prefilled by the query-outer kernel over those values, equal the
    same tokens attended through the cache, up to both kernels' roundings."""
    T, H, G, D, BS, S = 256, 1, 16, 128, 64, 3
    x = torch.randn((T, H * (G + 2), D), device=DEV).bfloat16()
    tc = pl.TokenCache(1, T // 64, T // 64, H, D)
    step = tc.step(dev([T]), T)
    vals = tuple(torch.empty((T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    tc.append(x[:, H * G:H * G + H], x[:, H * G + H:], step, values=vals)
    idx = torch.stack([torch.randperm(T // BS)[:S] for _ in range(T)]).int().view(T, H, S).to(DEV)
    cnt = torch.full((T, H), S, dtype=torch.int32, device=DEV)
    out, lse = tc.attend(x[:, :H * G], step, idx, cnt, BS)
    q = x[:, :H * G].contiguous()[None]
    want, wl = pl.nsa_qouter(q, vals[0][None], vals[1][None], idx[None], cnt[None], BS)
    # both are bf16 attention over the same values (exact in bf16): parity.py's bounds for such outputs, twice
    live = torch.isfinite(lse)
    assert torch.equal(live, torch.isfinite(wl[0]))
    a, b = out.float(), want[0].float()
    assert (a - b).abs().max() <= 2 * 2e-2 and (a - b).norm() / b.norm() <= 2 * 5e-3
    assert (lse - wl[0])[live].abs().max() <= 2e-3


# ---------------------------------------------------------------- every kernel that the sizes choose

WAYS = ("cuda cores", "split", "stream", "units", "rows")


def way_of(lib, c):
    """The kernel that this batch takes."""
    T, HQ, D = c["q"].shape
    H, P = c["cache"].shape[1], c["cache"].shape[2] * 16
    most = c["table"].shape[1] * P if c["idx"] is None else c["idx"].shape[2] * c["BS"]
    return WAYS[lib.bsa_cache_attention_way(T, HQ, H, D, c["q"].dtype, c["idx"] is not None, most)]


def asked(way, G, dtype):
    """Up to 8 heads in bfloat16 have no units: such batches are cut as a stream."""
    return "stream" if way == "units" and G <= 8 and dtype == torch.bfloat16 else way


def rows_of(c, pick):
    """The batch's tokens of these numbers."""
    return {**c, **{k: c[k][pick] for k in ("q", "req", "pos", "idx", "cnt") if c[k] is not None}}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["float32", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [3, 12])
@pytest.mark.parametrize("way", WAYS[1:])
def test_attention_every_kernel(lib, pl, way, G, D, dtype):
    """Each of the tensor-core kernels (way x up to 8 or more heads x D x type) on ragged rows with padding tokens:
    rows from across the batch against the oracle, all of them against the CUDA-core kernel (as in
    test_attention_batches), and twice the same bits."""
    R, n, lo, hi, P, S, BS = {"split": (3, 1, 300, 1300, 64, 0, 0), "stream": (130, 1, 1, 1300, 64, 0, 0),
                              "units": (150, 2, 2, 900, 32, 9, 64), "rows": (4, 700, 700, 1500, 16, 5, 64)}[way]
    c = attend_case(G + D, R, n, lo, hi, 4 * G, 4, D, P, S, BS, dtype)
    assert way_of(lib, c) == asked(way, G, dtype)
    T = R * n
    rng = np.random.default_rng(T)
    pad = rng.random(T) < (0.05 if T > 10 else 0)
    c["req"] = np.where(pad, -1, c["req"])
    out, lse = attend(pl, c)
    again = attend(pl, c)
    live = torch.as_tensor(~pad, device=DEV)
    assert torch.equal(out[live], again[0][live]) and torch.equal(lse[live], again[1][live])
    pick = np.unique(np.linspace(0, T - 1, 9).astype(int))
    check_attend(out[pick], lse[pick], want_attend(rows_of(c, pick)))
    set_force_simt(True)
    o2, l2 = attend(pl, c)
    both = live[:, None] & torch.isfinite(l2)
    assert torch.equal(both, live[:, None] & torch.isfinite(lse))
    a, b = out.float()[both], o2.float()[both]
    u = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -14
    assert (a - b).norm() <= 2 * u * b.norm()
    assert (lse - l2)[both].abs().max() <= 2.0 ** -14 * (1 + l2[both].abs().max())


def growing_case(seed, T, n, G, H, D, S, dtype):
    """T tokens of one request near its n-th key, whose K scales grow along the keys; with S, ascending lists of S
    blocks of 128.  Heads are sharp by other amounts, so each moves its maximum at other keys."""
    P, rng = 64, np.random.default_rng(seed)
    c = attend_case(seed, 1, 1, n, n, G * H, H, D, P, 0, 0, dtype, scales=False)
    p = np.arange(n)
    grow = (0x20 + p * 0x30 // n).astype(np.uint8)  # 2^-3 .. 2^3
    cols = 16 * D + (p % 16)[:, None] * (D // 16) + np.arange(D // 16)
    for h in range(H):
        c["cache"][c["table"][0, p // P][:, None], h, (p % P // 16)[:, None], cols] = grow[:, None]
    q = rng.standard_normal((T, G * H, D)) * np.logspace(-1, 0.3, G * H)[:, None]
    c["q"] = torch.tensor(q, dtype=dtype)
    c["req"], c["pos"] = np.zeros(T, np.int64), n - 1 - rng.integers(0, 100, T)
    if S:
        pool = np.argsort(rng.random((T, H, n // 128)), axis=2)[:, :, :S]
        c["idx"], c["cnt"], c["BS"] = np.sort(pool, axis=2), np.full((T, H), S), 128
    return c


# tokens, keys, KV heads, blocks of 128: rows of 23 tiles of 64 keys in runs of nine tiles a warp and more, whole rows
# of 20 tiles shared by a cluster's warps, whole rows of 20 tiles a warp; a row of 19 tiles over four warps
GROWING = {"split": (60, 1200, 4, 0), "stream": (700, 1500, 2, 0), "units": (300, 2000, 4, 10), "rows": (2800, 2000, 4, 10)}


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["float32", "bfloat16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [5, 16])
@pytest.mark.parametrize("way", WAYS[1:])
def test_attention_maxima_move_through_long_runs(lib, pl, way, G, D, dtype):
    """Each row's sum and output are rescaled by its own factor, many times in one warp's run of tiles."""
    T, n, H, S = GROWING[way]
    if way == "split" and G > 8:
        T = 40  # two CTAs an SM
    c = growing_case(G, T, n, G, H, D, S, dtype)
    assert way_of(lib, c) == asked(way, G, dtype)
    out, lse = attend(pl, c)
    pick = np.unique(np.linspace(0, T - 1, 7).astype(int))
    check_attend(out[pick], lse[pick], want_attend(rows_of(c, pick)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [8, 16])
@pytest.mark.parametrize("way,T", [("stream", 2000), ("units", 1216), ("rows", 8200)])
def test_attention_long_runs_do_not_shrink(lib, pl, way, T, G, D):
    """Rows of 2^19 keys, each in one warp's run, over values of one sign (2048 tokens, paged in again and again): the
    mean relative difference between bf16 and float32 outputs of the same queries.  A weight's rounding to float16 is
    at most 2^-11, taken as if all went one way; the outputs' own roundings (at most 2^-8, uniform, T G rows taken as
    one each) average to 2^-8 / sqrt(3 T G), five times that; float32 outputs are within 2^-14."""
    c = attend_case(G, 1, 1, 2048, 2048, G, 1, D, 1024, 0, 0, torch.bfloat16, scales=False)
    c["cache"][..., 8 * D:16 * D] &= 0x77
    c["table"] = np.tile(c["table"], (1, 256))
    n = c["table"].shape[1] * 1024
    c["q"] = torch.randn((T, G, D)).bfloat16()
    c["req"], c["pos"] = np.zeros(T, np.int64), np.full(T, n - 1)
    if way != "stream":
        c["idx"], c["cnt"], c["BS"] = np.tile(np.array([3, 0, 7, 1, 2, 6, 4, 5]), (T, 1, 1)), np.full((T, 1), 8), n // 8
    assert way_of(lib, c) == asked(way, G, torch.bfloat16)
    a = attend(pl, c)
    b = attend(pl, {**c, "q": c["q"].float()})
    short = ((a[0].double() - b[0].double()) / b[0].double()).mean().item()
    assert b[0].min() > 0 and abs(short) <= 2.0 ** -11 + 5 * 2.0 ** -8 / (3 * T * G) ** 0.5 + 2.0 ** -14, short
    assert (a[1] - b[1]).abs().max() <= 2.0 ** -14 * (1 + b[1].abs().max())


def on_device(c):
    """The arguments of cache_attention for this batch."""
    f = torch.float32
    return (c["q"].to(DEV), dev(c["cache"], torch.uint8), dev(c["table"]), dev(c["req"]), dev(c["pos"]),
            None if c["ks"] is None else dev(c["ks"], f), None if c["vs"] is None else dev(c["vs"], f),
            None if c["idx"] is None else dev(c["idx"]), None if c["cnt"] is None else dev(c["cnt"]), c["BS"])


def test_captured_long_runs_replay(lib, pl):
    """Runs of more than 128 tiles, whose sums are put aside in the workspace, captured in two graphs and replayed over
    other positions: the bits of eager calls, and rows within tolerance of the oracle."""
    c = growing_case(3, 400, 20000, 5, 2, 128, 0, torch.bfloat16)
    assert way_of(lib, c) == "stream"  # 800 rows of 311 tiles or more on 1824 warps
    args = on_device(c)
    pl.cache_attention(*args)
    torch.cuda.synchronize()
    graphs, got = [torch.cuda.CUDAGraph() for _ in range(2)], []
    for g in graphs:
        with torch.cuda.graph(g):
            got.append(pl.cache_attention(*args))
    for shift in (0, 5000, 3):
        args[4].copy_(dev(c["pos"] - shift))
        want = pl.cache_attention(*args)
        for g, (out, lse) in zip(graphs, got):
            out.zero_(), lse.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    pick = np.array([0, 399])
    check_attend(want[0][pick], want[1][pick], want_attend(rows_of({**c, "pos": c["pos"] - 3}, pick)))


ROWS_16 = (70, 30, 30, 200, 48, 4, 128, 16, 6, 16, torch.bfloat16)


@pytest.mark.parametrize("pair", [(JOIN_8, JOIN_16), (UNITS_16, UNITS_8), (ROWS_8, ROWS_16), (JOIN_8, ROWS_8)],
                         ids=["stream", "units", "rows", "stream-rows"])
def test_two_streams_keep_parts_and_counters_apart(lib, pl, pair):
    """Batches with parts in a workspace, a join launched early, or the stream's work counter, interleaved on two
    streams: the bits of calls made one by one."""
    assert {way_of(lib, attend_case(0, *x)) for x in pair} <= {"stream", "units", "rows"}
    args = [on_device(attend_case(sum(x[:-1]), *x)) for x in pair]
    want = []
    for a in args:
        want.append(pl.cache_attention(*a))
        torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for i in range(8):
        for s, a, to in zip(streams, args, got):
            with torch.cuda.stream(s):
                to.append(pl.cache_attention(*a))
        if i == 3:  # the other way round, behind a call on the first stream
            streams.reverse()
            streams[0].wait_stream(streams[1])
            streams[1].wait_stream(streams[0])
    torch.cuda.synchronize()
    for (o, l), to in zip(want, got):
        assert all(torch.equal(o, out) and torch.equal(l, lse) for out, lse in to)


@pytest.mark.parametrize("stall", [0, 2, 3])
@pytest.mark.parametrize("G", [5, 16])
@pytest.mark.parametrize("way", WAYS[1:])
def test_attention_wait_that_expires_late_is_reported(lib, pl, way, G, stall):
    """Runs of four tiles and more: a later tile of each warp is never copied, when parts have been written and rows
    claimed already.  The expiry (1 ms under the switch) is reported, and the next call is as before."""
    T, n, H, S = GROWING[way]
    if way == "split" and G > 8:
        T = 40
    c = growing_case(G, T, n, G, H, 128, S, torch.bfloat16)
    assert way_of(lib, c) == asked(way, G, torch.bfloat16)
    args = on_device(c)
    want = pl.cache_attention(*args)
    os.environ["BSA_TEST_STALL_TILE"] = str(stall)
    try:
        pl.cache_attention(*args)
    finally:
        os.environ.pop("BSA_TEST_STALL_TILE")
    assert lib.bsa_device_status() == lib.BSA_ERR_TIMEOUT
    out, lse = pl.cache_attention(*args)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------- offsets past 32 bits

@pytest.mark.parametrize("D", [80, 128])
def test_pages_past_32_bits_of_bytes(lib, pl, D):
    """Pages on both sides of the cache's 2^31st and 2^32nd byte hold what the same pages of a small cache hold."""
    H, P, G = 4, 64, 4
    page = H * (P // 16) * 18 * D
    n_pages = 2 ** 32 // page + 3
    ids = sorted({0, 2 ** 31 // page - 1, 2 ** 31 // page, 2 ** 31 // page + 1, 2 ** 32 // page - 1, 2 ** 32 // page, n_pages - 1})
    n = len(ids) * P - 5
    x = torch.randn((n, H * (G + 2), D), device=DEV).bfloat16()
    got = []
    for pages, ids_of in ((n_pages, ids), (len(ids), list(range(len(ids))))):
        cache = torch.full((pages, H, P // 16, 18 * D), 0xFF, dtype=torch.uint8, device=DEV)
        p = torch.arange(n, device=DEV)
        table = dev([ids_of])
        pl.cache_append(x[:, H * G:H * G + H], x[:, H * G + H:], table[0].long()[p // P] * P + p % P, cache)
        req, pos = dev(np.zeros(9)), dev(np.linspace(0, n - 1, 9).astype(int))
        out = pl.cache_attention(x[:9, :H * G], cache, table, req, pos)
        got.append((cache[dev(ids_of).long()], *out))
    assert all(torch.equal(a, b) for a, b in zip(*got)) and got[0][1].isfinite().all()


def test_rows_past_32_bits_of_elements(lib, pl):
    """Queries, outputs and appended rows past the 2^31st element: the last tokens as in a call of their own."""
    T, H, G, D, P = 2 ** 31 // (64 * 128) + 70, 4, 16, 128, 64
    q = torch.zeros((T, H * G, D), dtype=torch.bfloat16, device=DEV)
    q[-80:] = torch.randn((80, H * G, D), device=DEV)
    cache, table, n = pl.new_cache(3, H, P, D), dev([[2, 0, 1]]), 3 * P
    x, p = torch.randn((n, 2 * H, D), device=DEV).bfloat16(), torch.arange(n, device=DEV)
    pl.cache_append(x[:, :H], x[:, H:], table[0].long()[p // P] * P + p % P, cache)
    req, pos = torch.zeros(T, dtype=torch.int32, device=DEV), torch.arange(T, device=DEV).remainder(n).int()
    idx = torch.arange(T * H, device=DEV).remainder(12).int().view(T, H, 1)
    cnt = torch.ones((T, H), dtype=torch.int32, device=DEV)
    whole = pl.cache_attention(q, cache, table, req, pos, None, None, idx, cnt, 16)
    last = pl.cache_attention(q[-80:], cache, table, req[-80:], pos[-80:], None, None, idx[-80:], cnt[-80:], 16)
    empty = torch.isneginf(last[1])
    assert torch.equal(empty, torch.isneginf(whole[1][-80:])) and not empty.all()
    # one row to a warp or to a cluster: other orders of the same sums, so bf16 outputs are a rounding each apart
    a, b = whole[0][-80:].float(), last[0].float()
    assert (a - b).norm() <= 2 * 2.0 ** -8 * b.norm()
    assert (whole[1][-80:] - last[1])[~empty].abs().max() <= 2.0 ** -14 * (1 + last[1][~empty].abs().max())
    del q, whole, last
    H = 32
    T = 2 ** 31 // (2 * H * D) + 70
    rows = torch.zeros((T, 2 * H, D), dtype=torch.bfloat16, device=DEV)
    rows[-80:] = torch.randn((80, 2 * H, D), device=DEV)
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[-80:] = torch.arange(80, device=DEV).flip(0) + 11
    vals = tuple(torch.zeros((T, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    a, b = pl.new_cache(2, H, P, D), pl.new_cache(2, H, P, D)
    pl.cache_append(rows[:, :H], rows[:, H:], slots, a, values=vals)
    some = tuple(torch.zeros((80, H, D), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    pl.cache_append(rows[-80:, :H], rows[-80:, H:], slots[-80:], b, values=some)
    assert torch.equal(a, b) and a.any() and all(torch.equal(x[-80:], y) and not x[:-80].any() for x, y in zip(vals, some))
