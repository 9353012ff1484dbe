"""Cross attention (a18): calls for which the kernel that their sizes name cannot read their addresses, and batches of more
sequences than one warp's lanes."""

import numpy as np
import pytest
import torch

from test_gpu_rotary_cross import check_rows, rand

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


def off_by_one(x):
    """The same rows from an address two bytes behind a 16-byte border."""
    return torch.cat([torch.zeros(1, dtype=x.dtype, device=DEV), x.flatten()])[1:].view(x.shape)


def median_ms(call):
    times = []
    for _ in range(7):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return sorted(times)[3]


@pytest.mark.parametrize("B,N,M,HQ,H,D", [(1, 1, 20000, 8, 2, 64), (3, 2, 5000, 4, 4, 128), (20, 1, 1500, 16, 1, 96), (2, 1, 300, 4, 2, 64)])
def test_odd_addresses_few_rows(pl, B, N, M, HQ, H, D):
    q, k, v = (off_by_one(rand(i, B, n, heads, D, dtype=BF16)) for i, n, heads in ((1, N, HQ), (2, M, H), (3, M, H)))
    assert pl.bsa.bsa_cross_way(BF16, B, N, M, HQ, H, D) == 2
    lens = [M - b * M // B for b in range(B)]
    out, lse = pl.cross_attention(q, k, v, key_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    for b in range(B):
        check_rows(out[b], lse[b], q[b], k[b, :lens[b]], v[b, :lens[b]], D ** -0.5, BF16)


def test_odd_addresses_few_rows_use_the_whole_card(pl):
    """One token over many states takes what the same kernel takes for a head dim of its own (within a factor of 4: whole
    rows take ten times as long)."""
    M, H = 131072, 8
    q, k = (off_by_one(rand(i, 1, n, H, 64, dtype=BF16)) for i, n in ((1, 1), (2, M)))
    q60, k60 = q[..., :60].contiguous(), k[..., :60].contiguous()
    assert median_ms(lambda: pl.cross_attention(q, k, k)) <= 4 * median_ms(lambda: pl.cross_attention(q60, k60, k60))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,N,M,HQ,H,D", [(3, 1, 2000, 8, 2, 128), (1, 70, 9000, 4, 4, 64), (2, 1, 500, 4, 4, 40), (640, 1, 1100, 1, 1, 64)])
def test_the_switch_between_two_calls(pl, monkeypatch, dtype, B, N, M, HQ, H, D):
    q, k, v = rand(1, B, N, HQ, D, dtype=dtype), rand(2, 1, M, H, D, dtype=dtype), rand(3, 1, M, H, D, dtype=dtype)
    k, v = k.expand(B, M, H, D), v.expand(B, M, H, D)
    rows = range(0, B, max(1, B // 5))
    monkeypatch.delenv("BSA_FORCE_SIMT", raising=False)
    for _ in range(2):
        out, lse = pl.cross_attention(q, k, v)
        for b in rows:
            check_rows(out[b], lse[b], q[b], k[b], v[b], D ** -0.5, dtype)
        monkeypatch.setenv("BSA_FORCE_SIMT", "1")


def many(seed, B, most, empty=5):
    """Mixed lengths, every `empty`-th sequence without any."""
    n = np.random.default_rng(seed).integers(1, most + 1, B)
    n[::empty] = 0
    return n.tolist()


def starts(x):
    return torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("B", [33, 64, 70])
@pytest.mark.parametrize("dtype,most,keys,HQ,H,D,way", [
    (BF16, 400, 700, 4, 2, 64, 1), (BF16, 300, 300, 2, 2, 128, 1), (BF16, 90, 9000, 1, 1, 64, 1), (F32, 60, 300, 2, 1, 64, 3),
    (F32, 3, 9000, 1, 1, 20, 3), (BF16, 40, 400, 3, 1, 50, 0), (BF16, 3, 9000, 1, 1, 60, 0)])
def test_more_sequences_than_lanes(pl, B, dtype, most, keys, HQ, H, D, way):
    """Packed and padded-ragged batches of more than 32 sequences, live and from a graph (whose schedule is fixed): the
    256-row kernel, float32 and the CUDA cores, whole and in parts."""
    n, m = many(B, B, most), many(B + 1, B, keys, 7)
    T, M = sum(n), sum(m)
    assert pl.bsa.bsa_cross_way(dtype, B, T + 3, M, HQ, H, D, True, True) == way
    q, k, v = rand(1, T + 3, HQ, D, dtype=dtype), rand(2, M, H, D, dtype=dtype), rand(3, M, H, D, dtype=dtype)
    qs, ks = starts(n), starts(m)

    def check(out, lse):
        for b in range(B):
            r, c = slice(int(qs[b]), int(qs[b + 1])), slice(int(ks[b]), int(ks[b + 1]))
            check_rows(out[r], lse[r], q[r], k[c], v[c], D ** -0.5, dtype)
        assert bool((out[T:] == 7).all()) and bool((lse[T:] == 7).all())

    def new():
        return torch.full((T + 3, HQ, D), 7.0, dtype=dtype, device=DEV), torch.full((T + 3, HQ), 7.0, device=DEV)
    out, lse = new()
    pl.cross_attention(q, k, v, query_start=qs, key_start=ks, out=out, lse=lse)
    check(out, lse)
    again = new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pl.cross_attention(q, k, v, query_start=qs, key_start=ks, out=again[0], lse=again[1])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    # the states padded, NaN behind the lengths
    kp, vp = (torch.full((B, max(m), H, D), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    for b in range(B):
        kp[b, :m[b]], vp[b, :m[b]] = k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]]
    padded = new()
    pl.cross_attention(q, kp, vp, query_start=qs, key_lens=torch.tensor(m, dtype=torch.int32, device=DEV), out=padded[0], lse=padded[1])
    check(*padded)
    # and the queries, as many of each
    count = min(max(n), 40)
    qp = rand(4, B, count, HQ, D, dtype=dtype)
    o, z = pl.cross_attention(qp, kp, vp, key_lens=torch.tensor(m, dtype=torch.int32, device=DEV))
    for b in range(0, B, 3):
        c = slice(int(ks[b]), int(ks[b + 1]))
        check_rows(o[b], z[b], qp[b], k[c], v[c], D ** -0.5, dtype)
