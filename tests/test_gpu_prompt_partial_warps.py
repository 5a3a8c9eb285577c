"""Prompt attention where some lanes of a warp hold no row: groups that do not fill a tile, segments that end inside a
warp, rows that add up a hidden key's products while others write."""
import pytest
import torch

from tests.test_gpu_prompt import check, make, run, table

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


@pytest.mark.parametrize("hq,hkv", [(5, 1), (14, 2), (11, 1), (3, 1), (27, 1)])
@pytest.mark.parametrize("D", [64, 72, 128, 200, 256])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("odd", [False, True])
def test_rows_end_inside_a_warp(pkv, hq, hkv, D, dtype, odd):
    si, rows = table([9, 1, 131, 2, 47, 301, 33])
    q, k, v = make(hq + D, rows, hq, hkv, D)
    seen = torch.ones(rows, dtype=torch.bool)
    if odd:    # an infinity and a NaN in V that only the rows behind them see
        for q0, n, _, _ in si.tolist():
            if n > 8:
                v[q0 + n - 3, :, 5] = float("inf")
                v[q0 + n - 2, 0, D - 1] = float("nan")
                seen[q0 + n - 3:q0 + n] = False
    out, lse, err = run(pkv, q, k, v, si, out_dtype=dtype)
    assert err == 0
    clean = torch.nan_to_num(v, nan=0.0, posinf=0.0)     # (hidden from the rows that are compared)
    check(out, lse, q, k, clean, si, rows=seen)
    if odd:
        for q0, n, _, _ in si.tolist():
            if n > 8:
                assert bool(torch.isinf(out[q0 + n - 3, :, 5]).all() and torch.isinf(out[q0 + n - 1, :, 5]).all())
                assert bool(out[q0 + n - 2:q0 + n, :hq // hkv, D - 1].isnan().all())
