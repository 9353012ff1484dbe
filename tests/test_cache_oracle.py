"""The paged 4-bit cache without a GPU: pins of its oracle, and what the entry points refuse."""

import numpy as np
import pytest
import torch

import oracle


@pytest.fixture(scope="module")
def bsa():
    from block_sparse_attention_tile_gb300.build import build
    build()
    from block_sparse_attention_tile_gb300 import bsa as mod
    return mod


# ---------------------------------------------------------------- numbers

def test_e4m3_values_are_torchs():
    want = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = np.array([oracle.e4m3_value(b) for b in range(256)])
    assert np.array_equal(got, want, equal_nan=True)


def test_every_code_times_scale_is_exact_in_float16_and_bfloat16():
    x = torch.tensor([oracle.code_value(c) * oracle.e4m3_value(b) for c in range(16) for b in range(256)
                      if b & 0x7F != 0x7F], dtype=torch.float64)
    assert torch.equal(x.half().double(), x) and torch.equal(x.bfloat16().double(), x)
    assert x.abs().max() == 2688 and x.abs()[x != 0].min() == 2.0 ** -10


def test_group_rounding_is_nearest_by_brute_force():
    rng = np.random.default_rng(0)
    steps = np.array([oracle.code_value(c) for c in range(8)])
    for i in range(300):
        x = np.float32(rng.standard_normal(16) * 10.0 ** rng.integers(-3, 4))
        codes, byte = oracle.quantise_group(x)
        s = oracle.e4m3_value(byte)
        top = float(np.abs(x).max())
        all_scales = np.array([oracle.e4m3_value(b) for b in range(127)])
        assert abs(s - top / 6) == np.abs(all_scales - top / 6).min()
        if s == 0:
            assert not np.any(codes & 7)
            continue
        got = np.array([oracle.code_value(int(c)) for c in codes])
        best = np.abs(np.abs(x)[:, None].astype(np.float64) / s - steps[None]).min(1)
        assert np.array_equal(np.abs(np.abs(x) / np.float64(s) - np.abs(got)), best)
        assert np.array_equal(np.sign(got)[got != 0], np.sign(x)[got != 0])


def test_group_rounding_ties_zero_and_non_finite():
    # with the scale at 1 (largest magnitude 6) the borders are ties: each goes to the even code
    x = np.zeros(16, np.float32)
    x[:9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -5]
    codes, byte = oracle.quantise_group(x)
    assert oracle.e4m3_value(byte) == 1.0
    assert [int(c) for c in codes[:9]] == [7, 0, 2, 2, 4, 4, 6, 6, 14]
    assert oracle.quantise_group(np.zeros(16))[1] == 0
    assert oracle.quantise_group(np.full(16, 1e9))[1] == 126  # saturates at 448
    for bad in (np.nan, np.inf, -np.inf):
        x[3] = bad
        assert oracle.quantise_group(x) == (None, 0x7F)


def test_store_then_load_gives_the_rounded_rows_and_touches_nothing_else():
    rng = np.random.default_rng(1)
    for H, P, D in ((2, 32, 48), (1, 16, 128)):
        cache = rng.integers(0, 256, oracle.empty_cache(3, H, P, D).shape).astype(np.uint8)
        before = cache.copy()
        k, v = rng.standard_normal((2, H, D))
        slot = 2 * P + P - 3
        oracle.store(cache, slot, k, v, k_scale=np.full(H, 0.5), v_scale=np.full(H, 0.25))
        K, V = oracle.load(cache, slot, np.full(H, 0.5), np.full(H, 0.25))
        for got, x, g in ((K, k, 0.5), (V, v, 0.25)):
            for h in range(H):
                for c in range(0, D, 16):
                    codes, byte = oracle.quantise_group(x[h, c:c + 16], g)
                    want = [oracle.code_value(int(q)) * oracle.e4m3_value(byte) * g for q in codes]
                    assert np.array_equal(got[h, c:c + 16], want)
        changed = {int(s) for s in range(3 * P)
                   if not all(np.array_equal(a, b, equal_nan=True)
                              for a, b in zip(oracle.load(cache, s), oracle.load(before, s)))}
        assert changed == {slot}
        # every bit of a strip belongs to one token: all 16 stored, all bytes overwritten
        full = np.full_like(cache, 255)
        for j in range(16):
            oracle.store(full, j, np.zeros((H, D)), np.zeros((H, D)))
        assert not full[0, :, 0].any() and (full[0, :, 1:] == 255).all()


# ---------------------------------------------------------------- tables

def _tables_state(rng, R, P, max_pages, slack):
    old = rng.integers(0, max_pages * P + 1, R)
    new = rng.integers(0, max_pages * P + 1, R)
    pages = -(-old // P)
    n_pages = int(pages.sum() + np.maximum(-(-new // P) - pages, 0).sum()) + slack
    ids = rng.permutation(n_pages)
    table = np.full((R, max_pages), -1)
    at = 0
    for r in range(R):
        table[r, :pages[r]] = ids[at:at + pages[r]]
        at += pages[r]
    pool = np.full(n_pages, -1)
    pool[:n_pages - at] = ids[at:]
    return old, new, table, pool, n_pages - at


def test_tables_hold_every_page_once_and_a_shrink_undoes_a_grow():
    rng = np.random.default_rng(2)
    for R, P, mp in ((1, 16, 4), (7, 32, 5), (20, 16, 9)):
        old, new, table, pool, count = _tables_state(rng, R, P, mp, 2)
        ok, table2, pool2, count2, start, req, pos, slots = oracle.cache_tables(old, new, P, table, pool, count, 10 ** 4)
        assert ok
        held = [int(table2[r, j]) for r in range(R) for j in range(-(-int(new[r]) // P))]
        assert sorted(held + [int(x) for x in pool2[:count2]]) == list(range(len(pool)))
        live = req >= 0
        assert live.sum() == np.maximum(new - old, 0).sum() == start[-1]
        assert len(set(slots[live].tolist())) == live.sum()
        grown = np.maximum(old, new)
        ok, t3, p3, c3, *_ = oracle.cache_tables(old, grown, P, table, pool, count, 10 ** 4)
        ok2, t4, p4, c4, *_ = oracle.cache_tables(grown, old, P, t3, p3, c3, 0)
        assert ok and ok2 and c4 == count and np.array_equal(p4[:count], pool[:count])


def test_tables_refuse_as_a_whole():
    P, table, pool = 16, np.full((2, 3), -1), np.arange(2)
    for old, new, most in (([0, 0], [17, 17], 99), ([0, 0], [5, 5], 9), ([0, 0], [49, 0], 99), ([0, -1], [1, 0], 9)):
        ok, t, p, c, start, req, pos, slots = oracle.cache_tables(old, new, P, table, pool, 2, most)
        assert not ok and c == 2 and np.array_equal(t, table) and not start.any() and (slots == -1).all()


# ---------------------------------------------------------------- attention

def test_cache_attention_is_softmax_over_the_stored_rows():
    rng = np.random.default_rng(3)
    H, G, P, D, n = 2, 3, 16, 32, 37
    cache, table = oracle.empty_cache(4, H, P, D), np.array([[2, 0, 3]])
    k, v = rng.standard_normal((2, n, H, D))
    slots = [int(table[0, p // P]) * P + p % P for p in range(n)]
    for p in range(n):
        oracle.store(cache, slots[p], k[p], v[p])
    got = [oracle.load(cache, s) for s in slots]
    K, V = (torch.tensor(np.stack([g[i] for g in got])).double() for i in (0, 1))
    q = rng.standard_normal((2, H * G, D))
    pos = [n - 1, 20]
    o, lse = oracle.cache_attention(q, cache, table, [0, 0], pos)
    for t in range(2):
        m = pos[t] + 1
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q[t])[:, None], K[:m].transpose(0, 1).repeat_interleave(G, 0),
            V[:m].transpose(0, 1).repeat_interleave(G, 0))[:, 0]
        assert np.allclose(o[t], want.numpy(), rtol=0, atol=1e-12)
        x = torch.einsum("hd,nhd->hn", torch.tensor(q[t]), K[:m].repeat_interleave(G, 1)) * D ** -0.5
        assert np.allclose(lse[t], x.logsumexp(1).numpy(), rtol=0, atol=1e-12)
    # all blocks listed once in any order: the same; a block of later keys adds nothing; none: zero and -inf
    idx = np.array([[[2, 0, 1, 5]] * H] * 2)
    o2, l2 = oracle.cache_attention(q, cache, np.pad(table, ((0, 0), (0, 5))), [0, 0], pos, block_indices=idx,
                                    block_counts=np.full((2, H), 4), block_size=16)
    assert np.allclose(o2, o, atol=1e-12) and np.allclose(l2, lse, atol=1e-12)
    o3, l3 = oracle.cache_attention(q, cache, table, [0, -1], [-1, 5])
    assert not o3[0].any() and (l3[0] == -np.inf).all() and np.isnan(o3[1]).all()


# ---------------------------------------------------------------- refusals (host checks: no CUDA call is made)

def _args(defaults, **changed):
    names = list(defaults)
    assert set(changed) <= set(names)
    return [changed.get(n, defaults[n]) for n in names]


TABLES = dict(old=16, new=16, R=4, P=64, table=16, max_pages=8, pool=16, n_pages=32, count=16, count_out=16, start=16,
              req=16, pos=16, slots=16, max_tokens=8, ws=16, ws_bytes=1 << 20, stream=None)
APPEND = dict(k=16, v=16, dtype=1, T=4, H=2, D=128, ks=256, vs=256, slots=16, cache=16, n_pages=4, P=64, k_scale=None,
              v_scale=None, k_val=None, v_val=None, stream=None)
ATTEND = dict(q=16, dtype=1, T=4, HQ=8, H=2, D=128, qs=1024, cache=16, n_pages=4, P=64, table=16, R=2, max_pages=4,
              req=16, pos=16, k_scale=None, v_scale=None, idx=16, cnt=16, S=4, BS=64, scale=0.1, out=16, lse=None,
              ws=32, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,word", [
    (dict(old=None), "null"), (dict(table=None), "null"), (dict(count_out=None), "null"), (dict(req=None), "null"),
    (dict(R=0), "sizes"), (dict(R=(1 << 20) + 1, max_pages=1), "sizes"), (dict(max_tokens=-1), "sizes"),
    (dict(max_tokens=(1 << 30) + 1), "sizes"),
    (dict(P=48), "power of two"), (dict(P=8), "power of two"), (dict(P=2048), "power of two"),
    (dict(R=1 << 16, max_pages=1 << 15), "2^31"), (dict(max_pages=1 << 26, R=1), "2^31"),
    (dict(ws=None, R=2401), "workspace"), (dict(ws_bytes=(8 + 2 * 2402) * 4 - 1, R=2401), "workspace"),
    (dict(ws=18, R=2401), "workspace"),
])
def test_tables_refusals(bsa, change, word):
    assert bsa._lib.bsa_cache_tables(*_args(TABLES, **change)) == bsa.BSA_ERR_INVALID_ARG
    assert word in bsa.bsa_last_error()


@pytest.mark.parametrize("change,word", [
    (dict(k=None), "null"), (dict(slots=None), "null"), (dict(cache=None), "null"), (dict(k_val=16), "together"),
    (dict(dtype=7), "dtype"), (dict(T=-1), "sizes"), (dict(H=0), "sizes"), (dict(D=40), "multiple of 16"),
    (dict(D=144), "multiple of 16"), (dict(P=100), "power of two"), (dict(ks=255), "stride"), (dict(vs=8), "stride"),
    (dict(cache=24), "aligned"),
])
def test_append_refusals(bsa, change, word):
    assert bsa._lib.bsa_cache_append(*_args(APPEND, **change)) == bsa.BSA_ERR_INVALID_ARG
    assert word in bsa.bsa_last_error()


@pytest.mark.parametrize("change,word,status", [
    (dict(q=None), "null", 1), (dict(pos=None), "null", 1), (dict(out=None), "null", 1), (dict(dtype=2), "dtype", 1),
    (dict(HQ=7), "sizes", 1), (dict(T=-1), "sizes", 1), (dict(R=0), "sizes", 1), (dict(P=24), "power of two", 1),
    (dict(D=8), "multiple of 16", 1), (dict(D=256), "multiple of 16", 1), (dict(qs=1023), "stride", 1),
    (dict(cache=17), "aligned", 1), (dict(out=24), "aligned", 1), (dict(idx=None), "together", 1), (dict(cnt=None), "together", 1),
    (dict(S=0), "block lists", 1), (dict(BS=0), "block lists", 1), (dict(S=1 << 20, BS=1 << 12), "block lists", 1),
    (dict(max_pages=1 << 26), "2^31", 1), (dict(BS=24), "multiple of 16", 2), (dict(n_pages=1 << 29), "strips", 1),
    (dict(ws=None, idx=None, cnt=None, max_pages=1 << 12), "workspace", 1),
    (dict(ws=16, idx=None, cnt=None, max_pages=1 << 12), "workspace", 1),
    (dict(ws_bytes=64, idx=None, cnt=None, max_pages=1 << 12), "workspace", 1),
])
def test_attention_refusals(bsa, change, word, status):
    assert bsa._lib.bsa_fwd_cache_tokens(*_args(ATTEND, **change)) == status
    assert word in bsa.bsa_last_error()


def test_append_of_too_many_rows(bsa):
    change = dict(T=(1 << 31) - 1, H=64, D=128, ks=64 * 128, vs=64 * 128)
    assert bsa._lib.bsa_cache_append(*_args(APPEND, **change)) == bsa.BSA_ERR_UNSUPPORTED


def test_an_empty_step_needs_no_launch(bsa):
    assert bsa._lib.bsa_cache_append(*_args(APPEND, T=0)) == bsa.BSA_OK
    assert bsa._lib.bsa_fwd_cache_tokens(*_args(ATTEND, T=0)) == bsa.BSA_OK


def test_an_empty_step_has_no_arrays(bsa):
    # an empty tensor's pointer is null
    assert bsa._lib.bsa_cache_append(*_args(APPEND, T=0, k=None, v=None, slots=None, v_val=16)) == bsa.BSA_OK
    assert bsa._lib.bsa_fwd_cache_tokens(*_args(ATTEND, T=0, q=None, req=None, pos=None, out=None, cnt=None, ws=None,
                                                ws_bytes=0)) == bsa.BSA_OK


def test_sizes(bsa):
    assert bsa.bsa_cache_bytes(3, 4, 64, 128) == 3 * 4 * 4 * 18 * 128 == oracle.empty_cache(3, 4, 64, 128).nbytes
    assert bsa.bsa_cache_bytes(1 << 20, 8, 128, 128) == (1 << 20) * 8 * 8 * 2304  # past 32 bits
    for bad in ((0, 1, 64, 128), (1, 1, 24, 128), (1, 1, 64, 100), (1, 1, 64, 256)):
        assert bsa.bsa_cache_bytes(*bad) == 0
    assert bsa.bsa_cache_tables_workspace(2401) == (8 + 2 * 2402) * 4 and bsa.bsa_cache_tables_workspace(2400) == 0


def test_way_of_sizes(bsa):
    way = bsa.bsa_cache_attention_way
    assert way(8, 8, 2, 96, torch.bfloat16, False, 600) == 0              # head sizes without a tensor-core kernel
    assert way(1, 64, 4, 128, torch.bfloat16, True, 16 * 64) == 1         # few rows: a cluster each
    assert way(48, 64, 8, 128, torch.bfloat16, False, 32768) == 2         # long rows: equal runs
    assert way(256, 64, 4, 128, torch.bfloat16, True, 16 * 128) == 3      # many lists of one length
    assert way(256, 32, 4, 128, torch.float32, True, 16 * 128) == 3
    assert way(256, 32, 4, 128, torch.bfloat16, True, 16 * 128) == 2      # three CTAs an SM: clusters of them do not fit
    assert way(3000, 32, 4, 128, torch.bfloat16, False, 1024) == 2
    assert way(2048, 64, 4, 128, torch.float32, True, 16 * 64) == 4       # more than six rows a warp
    for bad in (dict(T=0), dict(HQ=7), dict(H=0), dict(D=40), dict(D=144), dict(max_keys=0)):
        a = {**dict(T=8, HQ=8, H=2, D=64, dtype=torch.float32, lists=True, max_keys=64), **bad}
        assert way(*a.values()) == -1


def test_binding_refuses_tensors_that_do_not_fit(bsa):
    cpu = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bsa.bsa_cache_tables(cpu, cpu, 1, 16, cpu, 1, cpu, 1, cpu, cpu, cpu, cpu, cpu, cpu, 0, cpu)
    with pytest.raises(ValueError, match="old_lens"):
        bsa._expect("old_lens", cpu, torch.int32, 9, -1)
    with pytest.raises(ValueError, match="x: a contiguous"):
        bsa._expect("x", torch.zeros(8, 2, dtype=torch.int32)[:, 0], torch.int32, 8, -1)
    with pytest.raises(ValueError, match="x: a contiguous"):
        bsa._expect("x", cpu, torch.int64, 1, -1)
    rows = torch.zeros(3, 4, 32)
    assert bsa._rows("k", rows[:, :2], 3, 2, 32, torch.float32, -1)[1] == 128
    assert bsa._rows("k", rows[:1, :2], 1, 2, 32, torch.float32, -1)[1] == 64
    for bad in (rows[:, ::2], rows.transpose(0, 1), rows[..., ::2]):
        with pytest.raises(ValueError):
            bsa._rows("k", bad, bad.shape[0], bad.shape[1], bad.shape[2], torch.float32, -1)


def test_pipeline_refuses_a_cache_of_other_sizes(bsa):
    from block_sparse_attention_tile_gb300 import pipeline
    cache = pipeline.new_cache(2, 2, 16, 64, device="cpu")
    assert cache.shape == (2, 2, 1, 18 * 64) and not cache.any()
    with pytest.raises(ValueError):
        pipeline.new_cache(2, 2, 20, 64, device="cpu")
    rows = torch.zeros(1, 2, 32)
    with pytest.raises(ValueError, match="does not hold"):
        pipeline.cache_append(rows, rows, torch.zeros(1, dtype=torch.int64), cache)
    with pytest.raises(ValueError, match="does not hold"):
        pipeline.cache_attention(rows, cache, cache, None, None)


def test_token_cache_refuses_lengths_of_other_requests(bsa):
    from block_sparse_attention_tile_gb300 import pipeline
    c = pipeline.TokenCache(3, 4, 2, 1, 64, page_size=16, device="cpu")
    for R in (2, 4):
        with pytest.raises(ValueError, match="3 requests"):
            c.step(torch.zeros(R, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="another cache"):
        pipeline.TokenCache(3, 4, 2, 1, 64, page_size=16, device="cpu", tables=c).step(c.lens, 8)


@pytest.mark.parametrize("lists,word", [
    (dict(block_indices=(4, 8, 3)), "block_indices"), (dict(block_indices=(4, 2, 2, 3)), "block_indices"),
    (dict(block_indices=(8, 3)), "block_indices"), (dict(block_indices=(3, 2, 3)), "block_indices"),
    (dict(block_indices=(2, 4, 3)), "block_indices"),
    (dict(block_counts=(4, 8)), "block_counts"), (dict(block_counts=(4, 2, 3)), "block_counts"),
    (dict(block_counts=(8,)), "block_counts"), (dict(block_counts=(2, 4)), "block_counts"),
])
def test_attention_refuses_lists_of_other_heads(bsa, lists, word):
    """Tensors with enough elements in another order: their rows would be read as other rows."""
    from block_sparse_attention_tile_gb300 import pipeline
    T, HQ, H, D = 4, 8, 2, 64
    shapes = {"block_indices": (T, H, 3), "block_counts": (T, H), **lists}
    a = {k: torch.zeros(s, dtype=torch.int32) for k, s in shapes.items()}
    ints = torch.zeros(T, dtype=torch.int32)
    with pytest.raises(ValueError, match=word):
        pipeline.cache_attention(torch.zeros(T, HQ, D), pipeline.new_cache(2, H, 16, D, device="cpu"),
                                 torch.zeros(1, 2, dtype=torch.int32), ints, ints, block_size=16, **a)


@pytest.mark.parametrize("shape", [(2, 4, 64), (3, 2, 64), (4, 64, 2), (512,)])
def test_append_refuses_values_of_other_shapes(bsa, shape):
    from block_sparse_attention_tile_gb300 import pipeline
    T, H, D = 4, 2, 64
    rows = torch.zeros(T, H, D)
    for which in (0, 1):
        values = [torch.zeros(T, H, D), torch.zeros(T, H, D)]
        values[which] = torch.zeros(shape)
        with pytest.raises(ValueError, match="values"):
            pipeline.cache_append(rows, rows, torch.zeros(T, dtype=torch.int64),
                                  pipeline.new_cache(2, H, 16, D, device="cpu"), values=tuple(values))


@pytest.mark.parametrize("name", ["k_scale", "v_scale"])
@pytest.mark.parametrize("shape", [(8,), (1,), (2, 64), (4, 2)])
def test_scales_of_other_heads_are_refused(bsa, name, shape):
    from block_sparse_attention_tile_gb300 import pipeline
    T, HQ, H, D = 4, 8, 2, 64
    cache, rows = pipeline.new_cache(2, H, 16, D, device="cpu"), torch.zeros(T, H, D)
    ints, scale = torch.zeros(T, dtype=torch.int32), {name: torch.zeros(shape)}
    with pytest.raises(ValueError, match=name):
        pipeline.cache_attention(torch.zeros(T, HQ, D), cache, torch.zeros(1, 2, dtype=torch.int32), ints, ints, **scale)
    with pytest.raises(ValueError, match=name):
        pipeline.cache_append(rows, rows, torch.zeros(T, dtype=torch.int64), cache, **scale)


def test_longer_buffers_of_the_right_rows_pass_the_shape_checks(bsa):
    """Buffers for more tokens than the call's go on to the next check (here: no CUDA tensor)."""
    from block_sparse_attention_tile_gb300 import pipeline
    T, HQ, H, D = 4, 8, 2, 64
    ints, cache = torch.zeros(9, dtype=torch.int32), pipeline.new_cache(2, H, 16, D, device="cpu")
    with pytest.raises(ValueError, match="CUDA tensor"):
        pipeline.cache_attention(torch.zeros(T, HQ, D), cache, torch.zeros(1, 2, dtype=torch.int32), ints, ints,
                                 torch.zeros(H), torch.zeros(H), torch.zeros(9, H, 3, dtype=torch.int32),
                                 torch.zeros(9, H, dtype=torch.int32), 16)
    rows, long = torch.zeros(T, H, D), torch.zeros(9, H, D)
    with pytest.raises(ValueError, match="CUDA tensor"):
        pipeline.cache_append(rows, rows, torch.zeros(9, dtype=torch.int64), cache, values=(long, long))
