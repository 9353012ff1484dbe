"""Rotation and cross attention without a GPU: sizes that follow the kernel switch, and calls that are refused."""

import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pl():
    from block_sparse_attention_tile_gb300.build import build
    build()
    from block_sparse_attention_tile_gb300 import pipeline
    return pipeline


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", [(1, 1, 20000, 8, 2, 64), (1, 500, 20000, 4, 4, 128), (8, 1, 600, 8, 8, 128), (1, 2, 9000, 2, 2, 60)])
def test_cross_workspace_does_not_depend_on_the_switch(pl, monkeypatch, dtype, sizes):
    """A size that the binding keeps holds after BSA_FORCE_SIMT changes: the library asks for the same one."""
    def both():
        return (pl.bsa.bsa_cross_workspace(dtype, *sizes, False, False),
                pl.bsa._lib.bsa_cross_workspace(1 if dtype is torch.bfloat16 else 0, *sizes, 0, 0))
    monkeypatch.delenv("BSA_FORCE_SIMT", raising=False)
    cached, size = both()
    assert cached == size
    monkeypatch.setenv("BSA_FORCE_SIMT", "1")
    assert both() == (size, size) and pl.bsa.bsa_cross_way(dtype, *sizes) == 0


@pytest.mark.parametrize("positions,turns,axis", [((4, 3, 2), (8,), None), ((), (8,), None), ((4,), (8, 2), None), ((4, 2), (8, 2), (8, 2))])
def test_table_shapes_are_refused(pl, positions, turns, axis):
    """Positions of a batch, [B, T, axes], were read as B tokens."""
    i32 = torch.int32
    with pytest.raises(ValueError, match=r"positions \[T\] or \[T, axes\]"):
        pl.rotary_table(torch.zeros(positions, dtype=i32), torch.zeros(turns, dtype=torch.int64),
                        None if axis is None else torch.zeros(axis, dtype=i32))


@pytest.mark.parametrize("starts", [dict(query_start=(3, 2)), dict(query_start=()), dict(query_start=(3,), key_start=(3, 2))])
def test_start_shapes_are_refused(pl, starts):
    x = torch.zeros(4, 2, 16)
    kw = {n: torch.zeros(s, dtype=torch.int32) for n, s in starts.items()}
    with pytest.raises(ValueError, match="start"):
        pl.cross_attention(x, x if "key_start" in kw else x[None].expand(2, 4, 2, 16), x if "key_start" in kw else x[None].expand(2, 4, 2, 16), **kw)


def ints(*values):
    return (ctypes.c_int64 * len(values))(*values)


def test_rotate_refuses_a_negative_table_stride(pl):
    """The binding counts the table's rows from it: a negative one let the kernel read ahead of the table."""
    lib, st = pl.bsa._lib, ints(*[128, 32, 16] * 4)
    call = lambda stride: lib.bsa_rotate(1, 2, 4, 16, 8, 0, 0, 16, 16, stride, 64, 2, None, 64, None, 0, None, None, st, 1e-6, None)  # noqa: E731
    for stride in (-1, -32, -(1 << 40)):
        assert call(stride) == pl.bsa.BSA_ERR_INVALID_ARG and "table" in pl.bsa.bsa_last_error()


def test_rotate_refuses_outputs_over_other_rows(pl):
    """In place with other strides, or one output over the other tensor: rows were overwritten before they were read."""
    lib, B, T, HQ, H, D = pl.bsa._lib, 2, 4, 2, 2, 16
    rows, heads = (T * HQ * D, HQ * D, D), (T * HQ * D, D, T * D)  # batch, token, head: [B, T, H, D] and [B, H, T, D]
    def call(q, q_out, k, k_out, q_in=rows, q_to=rows, k_in=rows, k_to=rows, T=T):  # noqa: E306
        return lib.bsa_rotate(1, B, T, D, 8, 0, 0, 16, 16, 0, q, HQ, None, q_out, k, H, None, k_out, ints(*q_in, *q_to, *k_in, *k_to), 1e-6, None)
    for kw in (dict(q=4096, q_out=4096, k=8192, k_out=12288, q_to=heads), dict(q=4096, q_out=8192, k=12288, k_out=12288, k_to=heads),
               dict(q=4096, q_out=8192, k=8192, k_out=4096), dict(q=4096, q_out=4096, k=4096, k_out=8192),
               dict(q=4096, q_out=8192, k=12288, k_out=8192), dict(q=4096, q_out=8192, k=12288, k_out=4096)):
        assert call(**kw) == pl.bsa.BSA_ERR_INVALID_ARG and "overlap" in pl.bsa.bsa_last_error(), kw
    assert call(4096, 4096, 8192, 8192, q_to=heads, T=0) == pl.bsa.BSA_OK


def test_append_rotated_refuses_values_over_its_inputs(pl):
    """A key's partner channels are read by another thread than the one that writes its value."""
    def call(k=4096, v=8192, k_val=12288, v_val=16384):
        return pl.bsa._lib.bsa_cache_append_rotated(k, v, 1, 4, 2, 64, 128, 128, 64, 4096 * 16, 4, 16, None, None, k_val, v_val, 16,
                                                    16, 32, 0, None, 0, 0, None, None)
    for kw in (dict(k_val=4096), dict(v_val=8192), dict(k_val=8192), dict(v_val=4096), dict(k_val=16384)):
        assert call(**kw) == pl.bsa.BSA_ERR_INVALID_ARG and "overlap" in pl.bsa.bsa_last_error(), kw
