"""Rotary positions and cross attention without a GPU: pins of the oracle, the frequencies, the refusals."""

import math

import numpy as np
import pytest
import torch

import oracle


def turns(f):
    return round(f / (2 * math.pi) * 2.0 ** 64)


def test_table_quarter_turns_and_far_positions():
    quarter = 1 << 62
    cos, sin = oracle.rotary_table([0, 1, 2, 3, 4, -1], [quarter])
    assert np.allclose(cos[:, 0], [1, 0, -1, 0, 1, 0], atol=1e-15) and np.allclose(sin[:, 0], [0, 1, 0, -1, 0, -1], atol=1e-15)
    # one radian a position at position 2^30, against the angle reduced with 80 digits of pi
    from decimal import Decimal, getcontext
    getcontext().prec = 80
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    t = int((Decimal(1) / (2 * pi) * (1 << 64)).to_integral_value())
    left = Decimal(1 << 30) % (2 * pi)
    cos, sin = oracle.rotary_table([1 << 30], [t])
    assert abs(cos[0, 0] - math.cos(float(left))) < 1e-9 and abs(sin[0, 0] - math.sin(float(left))) < 1e-9


def test_table_axes_and_factor():
    f = [turns(1.0), turns(0.5), turns(0.25)]
    cos, sin = oracle.rotary_table([[3, 5], [7, 11]], f, axis=[0, 1, 1], factor=1.5)
    want = np.array([[3.0, 2.5, 1.25], [7.0, 5.5, 2.75]])
    assert np.allclose(cos, 1.5 * np.cos(want)) and np.allclose(sin, 1.5 * np.sin(want))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotate_is_a_product_of_complex_numbers_and_its_transpose_takes_it_back(interleaved):
    rng = np.random.default_rng(1)
    x, angle = rng.standard_normal((3, 2, 10)), rng.standard_normal((3, 4))
    y = oracle.rotate(x, np.cos(angle), np.sin(angle), interleaved)
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if interleaved else (x[..., :4], x[..., 4:8])
    z = (a + 1j * b) * np.exp(1j * angle)[:, None]
    got = (y[..., 0:8:2], y[..., 1:8:2]) if interleaved else (y[..., :4], y[..., 4:8])
    assert np.allclose(got[0], z.real) and np.allclose(got[1], z.imag) and np.array_equal(y[..., 8:], x[..., 8:])
    assert np.allclose(oracle.rotate(y, np.cos(angle), np.sin(angle), interleaved, transpose=True), x)
    # logits depend on the distance alone
    c, s = oracle.rotary_table([5, 9, 1005, 1009], [turns(0.7), turns(0.01)])
    q, k = rng.standard_normal((2, 1, 1, 4))
    rot = lambda v, t: oracle.rotate(v, c[t:t + 1], s[t:t + 1], interleaved)  # noqa: E731
    assert np.allclose(np.sum(rot(q, 0) * rot(k, 1)), np.sum(rot(q, 2) * rot(k, 3)))


def test_rotate_f32_rounds_each_step():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((4, 1, 6)).astype(np.float32)
    c, s = (rng.standard_normal((4, 3)).astype(np.float32) for _ in range(2))
    y = oracle.rotate_f32(x, c, s)
    p, r = np.float32(x[1, 0, 2] * c[1, 2]), np.float32(x[1, 0, 5] * s[1, 2])
    assert y.dtype == np.float32 and y[1, 0, 2] == np.float32(p - r)
    assert np.max(np.abs(y - oracle.rotate(x, c, s))) < 1e-6


def test_cross_equals_a_library_attention():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((7, 4, 8)), rng.standard_normal((5, 2, 8)), rng.standard_normal((5, 2, 8))
    o, lse = oracle.cross_attention(q, k, v, 0.3)
    t = [torch.from_numpy(x).transpose(0, 1)[None] for x in (q, np.repeat(k, 2, 1), np.repeat(v, 2, 1))]
    want = torch.nn.functional.scaled_dot_product_attention(*t, scale=0.3)[0].transpose(0, 1).numpy()
    assert np.allclose(o, want)
    o, lse = oracle.cross_attention(q, k[:0], v[:0], 0.3)
    assert not o.any() and np.all(np.isneginf(lse))


# ---------------------------------------------------------------- the library without a GPU

@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300.build import build
    build()
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


@pytest.fixture(scope="module")
def bsa(pl):
    from block_sparse_attention_tile_gb300 import bsa as mod
    return mod


def radians(r):
    return np.array([int(t) % (1 << 64) for t in r.turns]) / 2.0 ** 64 * 2 * math.pi


def test_frequencies(pl):
    plain = pl.rotary_frequencies(128, device="cpu")
    want = 10000.0 ** (-np.arange(64) / 64)
    assert plain.axis is None and plain.factor == 1.0 and np.allclose(radians(plain), want, rtol=1e-15)
    axes = pl.rotary_frequencies(128, sections=[44, 42, 42], device="cpu")
    assert axes.axis.tolist() == [0] * 22 + [1] * 21 + [2] * 21
    assert np.allclose(radians(axes)[22:43], 10000.0 ** (-np.arange(21) / 21), rtol=1e-15)
    assert np.allclose(radians(pl.rotary_frequencies(64, scaling="linear", stretch=4.0, device="cpu")),
                       10000.0 ** (-np.arange(32) / 32) / 4, rtol=1e-14)
    base = radians(pl.rotary_frequencies(64, scaling="base", stretch=4.0, device="cpu"))
    assert np.isclose(base[0], 1.0) and np.isclose(base[-1], 10000.0 ** (-31 / 32) / 4)
    parts = pl.rotary_frequencies(128, scaling="parts", stretch=8.0, trained=4096, device="cpu")
    n = want * 4096 / (2 * math.pi)  # turns within the trained positions
    assert np.allclose(radians(parts)[n > 32], want[n > 32]) and np.allclose(radians(parts)[n < 1], want[n < 1] / 8)
    mid = (n > 1) & (n < 32)
    kept = (n[mid] - 1) / 31
    assert mid.any() and np.allclose(radians(parts)[mid], want[mid] * (kept + (1 - kept) / 8))
    assert math.isclose(parts.factor, 0.1 * math.log(8) + 1)


@pytest.mark.parametrize("bad", [dict(scaling="other"), dict(sections=[64, 63]), dict(sections=[63, 65]),
                                 dict(scaling="parts", stretch=2.0), dict(scaling="linear", stretch=0.5)])
def test_frequencies_refuse(pl, bad):
    with pytest.raises(ValueError):
        pl.rotary_frequencies(128, device="cpu", **bad)


def test_host_tensors_are_refused(pl):
    x = torch.zeros(4, 2, 16)
    c = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        pl.rotate(x, None, c, c)
    with pytest.raises(ValueError):
        pl.rotary_table(torch.zeros(4, dtype=torch.int32), torch.zeros(8, dtype=torch.int64))
    with pytest.raises(ValueError):
        pl.cross_attention(x[None], x[None], x[None])


def test_shapes_are_refused(pl):
    x, c = torch.zeros(2, 4, 3, 16), torch.zeros(4, 8)
    for kw in (dict(cos=c, sin=torch.zeros(4, 7)), dict(cos=torch.zeros(5, 8), sin=torch.zeros(5, 8)),
               dict(cos=c, sin=c, q_weight=torch.ones(15)), dict(cos=c, sin=c, out=(x[:1], None))):
        with pytest.raises(ValueError):
            pl.rotate(x, None, **kw)
    with pytest.raises(ValueError, match="three dimensions"):
        pl.cross_attention(x, x[0], x[0])
    with pytest.raises(ValueError, match="three dimensions"):
        pl.cross_attention(x, x, x[:, :3])
    with pytest.raises(ValueError, match="sequences"):
        pl.cross_attention(x, x, x, key_lens=torch.zeros(3, dtype=torch.int32))


def ints(n, *values):
    import ctypes
    return (ctypes.c_int64 * n)(*values)


def test_arguments_are_refused(bsa):
    lib, bad = bsa._lib, bsa.BSA_ERR_INVALID_ARG
    assert lib.bsa_rotary_table(None, 4, 1, 16, None, 8, 1.0, 16, 16, None) == bad and "null" in bsa.bsa_last_error()
    assert lib.bsa_rotary_table(16, 4, 3, 16, None, 8, 1.0, 16, 16, None) == bad and "axis" in bsa.bsa_last_error()
    assert lib.bsa_rotary_table(16, 4, 9, 16, 16, 8, 1.0, 16, 16, None) == bad and "axes=9" in bsa.bsa_last_error()
    assert lib.bsa_rotary_table(16, 4, 1, 16, None, 129, 1.0, 16, 16, None) == bad
    assert lib.bsa_rotary_table(None, 0, 1, 16, None, 8, 1.0, None, None, None) == bsa.BSA_OK

    def rotate(B=1, T=4, D=16, P=8, transpose=0, q=16, qw=None, H=0, k=None, eps=1e-6, dtype=1, st=ints(12)):
        return lib.bsa_rotate(dtype, B, T, D, P, 0, transpose, 16, 16, 0, q, 2, qw, 16, k, H, None, 16, st, eps, None)
    for kw, word in ((dict(P=9), "P=9"), (dict(D=258), "D=258"), (dict(P=0), "P=0"), (dict(q=None), "null"),
                     (dict(H=1), "null"), (dict(transpose=1, qw=16), "norm"), (dict(qw=16, eps=-1.0), "eps"),
                     (dict(qw=16, eps=float("nan")), "eps"), (dict(dtype=2), "dtype"), (dict(st=None), "strides"),
                     (dict(T=-1), "T=-1")):
        assert rotate(**kw) == bad and word in bsa.bsa_last_error(), kw
    assert rotate(T=0, q=None) == bsa.BSA_OK and rotate(B=0, q=None) == bsa.BSA_OK

    def append(T=4, D=64, P=32, q=16, q_out=32, HQ=4, q_stride=256, cos=16, page=16, k_val=16, v_val=16):
        return lib.bsa_cache_append_rotated(16, 16, 1, T, 2, D, 128, 128, 16, 16, 4, page, None, None, k_val, v_val, cos,
                                            16, P, 0, q, HQ, q_stride, q_out, None)
    for kw, word in ((dict(P=33), "P=33"), (dict(cos=None), "null"), (dict(q_out=None), "come together"),
                     (dict(q_stride=255), "stride"), (dict(HQ=0), "HQ"), (dict(D=72), "D must"), (dict(page=24), "page"),
                     (dict(v_val=None), "come together"), (dict(q_out=16), "must not be q")):
        assert append(**kw) == bad and word in bsa.bsa_last_error(), kw
    assert append(T=0) == bsa.BSA_OK

    def cross(B=2, N=4, M=8, HQ=4, H=2, D=64, dtype=1, qs=None, ks=None, kl=None, scale=0.1, q=16, ws=0, st=ints(15)):
        return lib.bsa_fwd_cross(q, 16, 16, dtype, B, N, M, HQ, H, D, st, qs, ks, kl, scale, 16, None, None, ws, None)
    for kw, word in ((dict(HQ=3), "HQ=3"), (dict(D=129), "D=129"), (dict(D=0), "D=0"), (dict(dtype=5), "dtype"),
                     (dict(ks=16, kl=16), "exclude"), (dict(scale=-1.0), "scale"), (dict(scale=float("inf")), "scale"),
                     (dict(scale=float("nan")), "scale"), (dict(q=None), "null"), (dict(st=None), "strides"),
                     (dict(B=-1), "B=-1"), (dict(M=100000), "workspace"), (dict(B=1 << 20, N=1 << 20), "sizes")):
        assert cross(**kw) == bad and word in bsa.bsa_last_error(), kw
    assert cross(N=0) == bsa.BSA_OK and cross(B=0) == bsa.BSA_OK
    assert bsa.bsa_cross_workspace(torch.bfloat16, 2, 4, 100000, 4, 2, 64, False, False) > 0
    assert bsa.bsa_cross_workspace(torch.bfloat16, 2, 4, 8, 3, 2, 64, False, False) == 0
    # 2^30 padded rows with their heads are too many, the same tokens packed are not
    assert bsa.bsa_cross_way(torch.bfloat16, 4096, 65536, 64, 64, 4, 128) == -1
    assert bsa.bsa_cross_way(torch.bfloat16, 4096, 65536, 1 << 20, 64, 4, 128, True, True) >= 0


def test_cross_sizes_whose_tiles_would_pass_32_bits_are_refused(bsa):
    """A tile's end may lie past the last state; it has to stay within 32 bits."""
    for dtype, D in ((torch.bfloat16, 64), (torch.bfloat16, 7), (torch.float32, 64)):
        for packed in (False, True):
            assert bsa.bsa_cross_way(dtype, 2, 1, 2 ** 30 - 1, 1, 1, D, packed, packed) >= 0
            for M in (2 ** 30, 2 ** 31 - 1):
                assert bsa.bsa_cross_way(dtype, 2, 1, M, 1, 1, D, packed, packed) == -1
                assert bsa.bsa_cross_workspace(dtype, 2, 1, M, 1, 1, D, packed, packed) == 0
