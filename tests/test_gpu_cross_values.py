"""Cross attention (a18) in float32 with the largest finite values and with infinities in rows that count.

Tolerance: logits are small, a weight is off by (D + 8) 2^-23 of the sum of |q_c k_c| and 2^-21, sums by 2^-20 (as in
test_gpu_rotary_cross.py), an output by that times the weighted magnitudes."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"
MOST = torch.finfo(torch.float32).max


@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


def call(pl, N, M, D, change):
    g = torch.Generator(device=DEV).manual_seed(N + M)
    q, k, v = (torch.randn(1, n, 2, D, generator=g, device=DEV) for n in (N, M, M))
    q[..., 1] = q[..., 1].abs() + 0.25
    change(q, k, v)
    out, lse = pl.cross_attention(q, k, v)
    qd, kd, vd = (x[0].double().transpose(0, 1) for x in (q, k, v))
    s = qd @ kd.transpose(1, 2) * D ** -0.5
    p = torch.softmax(s, -1)
    B = (qd.abs() @ kd.abs().transpose(1, 2) * D ** -0.5).nan_to_num(posinf=0).amax(-1, keepdim=True)
    tol = (p @ vd.abs().nan_to_num(posinf=0)) * (2 * ((D + 8) * 2.0 ** -23 * B + 2.0 ** -21) + 2.0 ** -20)
    return out[0].transpose(0, 1), lse[0].T.double(), p, vd, s, tol, B


@pytest.mark.parametrize("N,M,D", [(1, 40, 64), (70, 300, 128), (5, 9, 7), (200, 5000, 20)])
@pytest.mark.parametrize("value", [MOST, -MOST, MOST * (1 - 2.0 ** -12), MOST * (1 - 2.0 ** -11)])
def test_largest_values(pl, N, M, D, value):
    def change(q, k, v):
        v[0, M // 3, 0, D // 2] = value
        k[0, M // 2, 1, 1], q[..., 1] = value, 2.0 ** -127  # a logit of some 2
    out, lse, p, vd, s, tol, B = call(pl, N, M, D, change)
    assert bool(((out.double() - p @ vd).abs() <= tol).all())
    assert bool(((lse - torch.logsumexp(s, -1)).abs() <= ((D + 8) * 2.0 ** -23 * B + 2.0 ** -19)[..., 0]).all())


@pytest.mark.parametrize("N,M,D", [(1, 40, 64), (70, 300, 128), (5, 9, 7), (200, 5000, 20)])
def test_infinities(pl, N, M, D):
    """A key whose logit is -inf has no weight; one of +inf makes its rows NaN; an infinite value its channel infinite."""
    def change(q, k, v):
        k[0, M // 2, 0, 1] = -float("inf")
        v[0, M // 3, 0, D // 2] = float("inf")
        v[0, M // 3, 1, 0] = -float("inf")
    out, lse, p, vd, s, tol, B = call(pl, N, M, D, change)
    want = p @ vd
    assert bool((out[0, :, D // 2] == float("inf")).all()) and bool((out[1, :, 0] == -float("inf")).all())
    live = torch.isfinite(want)
    assert bool(((out.double() - want).abs() <= tol)[live].all()) and int((~live).sum()) == 2 * N
    assert bool(((lse - torch.logsumexp(s, -1)).abs() <= ((D + 8) * 2.0 ** -23 * B + 2.0 ** -19)[..., 0]).all())

    def change(q, k, v):
        k[0, M // 2, 0, 1] = float("inf")
    out = call(pl, N, M, D, change)[0]
    assert bool(out[0].isnan().all()) and bool(out[1].isfinite().all())
