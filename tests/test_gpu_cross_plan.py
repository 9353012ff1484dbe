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
