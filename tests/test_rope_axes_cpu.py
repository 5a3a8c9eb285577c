"""Rotary positions with several axes: pair lists and refusals that need no GPU."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def test_rope_axes(pkv):
    assert pkv.rope_axes((2, 1, 3)) == [0, 0, 1, 2, 2, 2]
    assert pkv.rope_axes((2, 1, 3), dealt=True) == [0, 1, 2, 0, 2, 2]
    assert pkv.rope_axes((24, 20, 20), True) == [i % 3 for i in range(60)] + [0] * 4
    assert pkv.rope_axes((0, 2)) == [1, 1] and pkv.rope_axes((4,)) == [0] * 4
    for bad in ((), (0, 0), (3, -1), (1,) * 9):
        with pytest.raises(ValueError):
            pkv.rope_axes(bad)


@pytest.mark.parametrize("axes", [[0, 1, 2], [0, 1, 2, 8], [0, -1, 1, 1], []])
def test_rope_refuses_axes(pkv, axes):
    with pytest.raises(ValueError):
        pkv.Rope(torch.ones(4, dtype=torch.float64), device="cpu", axes=axes)
    with pytest.raises(ValueError):
        pkv.Rope(None, axes=[0, 1])


def test_rope_keeps_axes(pkv):
    r = pkv.Rope(torch.ones(4, dtype=torch.float64), device="cpu", axes=[0, 2, 1, 0])
    assert r.num_axes == 3 and r.axis.tolist() == [0, 2, 1, 0] and r.desc.num_axes == 3 and r.desc.axis == r.axis.data_ptr()
    r = pkv.Rope(torch.ones(4, dtype=torch.float64), device="cpu", axes=[0, 0, 0, 0])
    assert r.num_axes == 1 and r.axis is None and not r.desc.axis


@pytest.mark.parametrize("shape", [(5,), (5, 2), (4, 3), (5, 3, 1)])
def test_positions_shape(pkv, shape):
    r = pkv.Rope(torch.ones(4, dtype=torch.float64), device="cpu", axes=[0, 2, 1, 0])
    q = torch.zeros(5, 2, 8)
    with pytest.raises(ValueError):
        pkv.norm_rope(r, q, None, torch.zeros(shape, dtype=torch.int32))


@pytest.mark.parametrize("axes,ptr", [(2, 0), (-1, 64), (9, 64), (0, 64), (1, 64)])
def test_c_entry_refuses(pkv, axes, ptr):
    from paged_kv_decode_13_gb300 import _lib
    d = _lib.RopeDesc(turns=64, rot_dim=8, interleaved=0, mscale=1.0, eps=1e-6, axis=ptr or None, num_axes=axes)
    rows = _lib.RowsDesc(q=64, q_out=64, q_stride=16, q_out_stride=16, q_heads=2, total_rows=1, positions=64)
    assert _lib.lib.pkv_norm_rope(ctypes.byref(d), _lib.BF16, 8, 0, ctypes.byref(rows), None) == _lib.EINVAL
