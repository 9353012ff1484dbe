"""Cross attention (a18) over states so long, with rows so many, that no call cuts the keys: sums of one sign.

The keys are equal, so that every weight is 1, in bf16 too, and an output is the mean of its channel's values.  Tolerances,
with u = 2^-24 (a product with the tensor cores cuts its sum off: 2 u; an addition that rounds: u), relative to the mean:
* 256-row and 16-row kernels: at most 1024 products join a sum before it is put aside, 2048 u; the sums put aside are
  added up rounded, M / 16384 of them; some 8 u for the weights' sum and the division; half a step of the output.
* float32: 12 products a tile of 32 keys, 24 u; 128 tiles, 128 u; M / 4096 sums, each scaled and added, 2 u; 8 u.
* CUDA cores: 64 keys one after the other, 64 u, and M / 64 such sums, u each; 8 u; the weights' own sum likewise: doubled;
  half a step of the output."""

import pytest
import torch

from test_gpu_rotary_cross import check_rows

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


def equal_keys(pl, dtype, B, N, M, HQ, H, D, value=None):
    """The call's output and its exact value [H, D]; states shared by the batch."""
    g = torch.Generator(device=DEV).manual_seed(M + D)
    q = torch.randn(B, N, HQ, D, generator=g, device=DEV).to(dtype)
    k = torch.randn(H, D, generator=g, device=DEV).mul(0.3).to(dtype)
    if value is None:  # each channel's mean elsewhere between two values of bf16
        v = 1 + 0.7 / D * torch.arange(D, device=DEV) + 0.29 * torch.rand(M, H, D, generator=g, device=DEV)
    else:
        v = torch.full((M, H, D), value, device=DEV)
    v = v.to(dtype)
    out, lse = pl.cross_attention(q, k.expand(B, M, H, D).contiguous() if B == 1 else
                                  k.expand(M, H, D).contiguous().expand(B, M, H, D), v.expand(B, M, H, D))
    s = torch.einsum("bnhgd,hd->bnhg", q.double().unflatten(2, (H, HQ // H)), k.double()).flatten(2) * D ** -0.5
    want = s + torch.log(torch.tensor(float(M), dtype=torch.float64, device=DEV))
    assert float((lse.double() - want).abs().max()) <= (D + 8) * 2.0 ** -23 * float(s.abs().max() * 4 + 16) + M / 1024 * U + 1024 * U
    return out, v.double().mean(0)


def off(out, mean):
    """The largest distance from the mean (all of them below 2)."""
    want = mean.repeat_interleave(out.shape[2] // mean.shape[0], 0)
    return float(max((o.double() - want).abs().max() for o in out.flatten(0, 1).split(4096)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M", [1 << 18, (1 << 20) + 77])
def test_unsplit_long_sums_256_rows(pl, D, M):
    N = 19712  # 77 items: the keys stay in one piece
    assert pl.bsa.bsa_cross_way(BF16, 1, N, M, 1, 1, D) == 1
    assert pl.bsa.bsa_cross_workspace(BF16, 1, N, M, 1, 1, D, False, False) == 0
    out, mean = equal_keys(pl, BF16, 1, N, M, 1, 1, D)
    # half a step of 1 .. 2 is 2^-8
    most = off(out, mean)
    assert most <= 2.0 ** -8 + 2 * (2048 + M / 16384 + 8) * U


def moving_maxima(pl, dtype, B, N, M, HQ, H, D):
    """Logits that grow and fall along the states, so that sums are put aside under other maxima than the next ones'."""
    g = torch.Generator(device=DEV).manual_seed(N)
    q = torch.randn(B, N, HQ, D, generator=g, device=DEV).to(dtype)
    ramp = 0.2 + 4 * torch.sin(torch.arange(M, device=DEV) * (9.0 / M)).clamp(min=0)
    k = (torch.randn(M, H, D, generator=g, device=DEV) * ramp[:, None, None]).to(dtype)
    v = torch.randn(M, H, D, generator=g, device=DEV).to(dtype)
    out, lse = pl.cross_attention(q, k.expand(B, M, H, D), v.expand(B, M, H, D))
    rows = torch.arange(0, B * N, max(1, B * N // 150), device=DEV)
    check_rows(out.flatten(0, 1)[rows], lse.flatten(0, 1)[rows], q.flatten(0, 1)[rows], k, v, D ** -0.5, dtype)


@pytest.mark.parametrize("D", [64, 128])
def test_moving_maxima_256_rows(pl, D):
    moving_maxima(pl, BF16, 1, 19712, 40013, 1, 1, D)


@pytest.mark.parametrize("HQ,D", [(1, 64), (4, 128)])
@pytest.mark.parametrize("M", [1 << 19, (1 << 21) + 77])
def test_unsplit_long_sums_16_rows(pl, HQ, D, M):
    B = 640  # twice what runs at once: the rows are left whole, a quarter of the keys to a warp
    assert pl.bsa.bsa_cross_way(BF16, B, 1, M, HQ, 1, D) == 2
    assert pl.bsa.bsa_cross_workspace(BF16, B, 1, M, HQ, 1, D, False, False) == 0
    out, mean = equal_keys(pl, BF16, B, 1, M, HQ, 1, D)
    most = off(out, mean)
    assert most <= 2.0 ** -8 + 2 * (2048 + M / 16384 + 8) * U


@pytest.mark.parametrize("HQ,D", [(1, 64), (4, 128)])
def test_moving_maxima_16_rows(pl, HQ, D):
    moving_maxima(pl, BF16, 640, 1, 150013, HQ, 1, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("M", [1 << 17, 1 << 19])
def test_unsplit_long_sums_float32(pl, D, M):
    N = 39040
    assert pl.bsa.bsa_cross_way(F32, 1, N, M, 1, 1, D) == 3 and pl.bsa.bsa_cross_workspace(F32, 1, N, M, 1, 1, D, False, False) == 0
    out, mean = equal_keys(pl, F32, 1, N, M, 1, 1, D, 0.73)
    most = off(out, mean)
    assert most <= 0.73 * (24 + 128 + 2 * M / 4096 + 8) * U


@pytest.mark.parametrize("D", [7, 64, 128])
def test_long_sums_in_parts_float32(pl, D):
    N, M = 100, (1 << 20) + 77
    assert pl.bsa.bsa_cross_workspace(F32, 1, N, M, 1, 1, D, False, False) == 4 * 64 * N * (D + 1)  # 64 parts
    out, mean = equal_keys(pl, F32, 1, N, M, 1, 1, D, 0.73)
    most = off(out, mean)
    assert most <= 0.73 * (24 + 128 + 2 * M / 64 / 4096 + 2 * 64 + 8) * U


@pytest.mark.parametrize("N,HQ,H,D", [(39040, 1, 1, 64), (9760, 4, 1, 128), (100, 6, 2, 20)])
def test_moving_maxima_float32(pl, N, HQ, H, D):
    moving_maxima(pl, F32, 1, N, 10013 if N > 100 else 600013, HQ, H, D)


def test_unsplit_long_sums_cuda_cores(pl):
    N, M, D = 39040, 1 << 18, 4
    assert pl.bsa.bsa_cross_way(BF16, 1, N, M, 1, 1, D) == 0 and pl.bsa.bsa_cross_workspace(BF16, 1, N, M, 1, 1, D, False, False) == 0
    out, mean = equal_keys(pl, BF16, 1, N, M, 1, 1, D, 0.73)
    most = off(out, mean)
    assert most <= 2.0 ** -9 + 0.73 * 2 * (64 + M / 64 + 8) * U


@pytest.mark.parametrize("N,M,HQ,H,D", [(39040, 3013, 1, 1, 20), (700, 20013, 3, 1, 100), (3, 70000, 2, 2, 7)])
def test_moving_maxima_cuda_cores(pl, N, M, HQ, H, D):
    assert pl.bsa.bsa_cross_way(BF16, 1, N, M, HQ, H, D) == 0
    moving_maxima(pl, BF16, 1, N, M, HQ, H, D)


def test_items_longer_than_two_seconds(pl):
    """An item of 1.5 x 2^28 states (6.4 GB, K and V the same) takes the 256-row kernel some 3 s: its waits last as long."""
    N, M, D = 19712, 3 << 27, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    q, row = torch.randn(1, N, 1, D, generator=g, device=DEV).to(BF16), torch.randn(D, generator=g, device=DEV).to(BF16)
    k = torch.empty(1, M, 1, D, dtype=BF16, device=DEV).copy_(row)
    assert pl.bsa.bsa_cross_way(BF16, 1, N, M, 1, 1, D) == 1 and pl.bsa.bsa_cross_workspace(BF16, 1, N, M, 1, 1, D, False, False) == 0
    out, lse = pl.cross_attention(q, k, k)
    assert pl.bsa.bsa_device_status() == pl.bsa.BSA_OK
    # equal keys: the output is their row, but for half a step, and what 2^15 sums that were put aside are off
    most = float(((out.double() - row.double()) / row.double()).abs().max())
    assert most <= 2.0 ** -8 + 2 * (2048 + M / 16384 + 8) * U
