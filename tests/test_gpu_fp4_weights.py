"""Attention over a 4-bit cache whose softmax weights span many octaves.

Every page holds one key of weight 1 and fifteen of weight 2^-e; the values
of the first are zero, so the output is what the small weights carry.  A weight w
is off by its rounding to fp16, 2^-11 w in fp16's normal range (half a step) and
2^-32 below it (weights are held 2^7 above the largest one's scale, so
half of fp16's smallest step, 2^-25, stands for 2^-32), by its exponent: e log2
units from two fp32 roundings of the scale and the product (2^-23 e each, times ln 2),
and by exp2 (2^-22); the sum of weights by the same in relative terms, and their
addition by n 2^-24: |out - ref| <= sum |v| (w r + 2^-32) / sum w + 2 r |ref|,
r = 2^-11 + 2^-22 e + 2^-21 + n 2^-24."""
import numpy as np
import pytest
import torch

from tests import fp4_ref as R

pytestmark = pytest.mark.gpu
BIG = 1 << 20


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


@pytest.mark.parametrize("D,q_heads,max_kv", [(64, 1, 0), (128, 1, 0), (256, 1, 0), (64, 16, 0), (128, 16, 0), (256, 16, 0), (64, 32, 0), (128, 32, 0),
                                              (64, 1, BIG), (128, 1, BIG), (256, 16, BIG), (128, 32, BIG), (128, 64, BIG), (128, 128, BIG)])
@pytest.mark.parametrize("e", [12, 20, 26, 30])
def test_small_weights_reach_the_output(pkv, D, q_heads, max_kv, e):
    n = 2048
    blocks = n // 16
    k, v = np.zeros((blocks, 16, 1, D)), np.full((blocks, 16, 1, D), 6.0)
    for b in range(blocks):
        k[b, b % 16, 0, 0] = 6.0
        v[b, b % 16] = 0.0
    pools = [torch.from_numpy(R.pack(*R.quantise(x), i)).cuda() for x, i in ((k, False), (v, True))]
    assert all(np.array_equal(R.pool_values(p.cpu().numpy(), i), x) for p, i, x in ((pools[0], False, k), (pools[1], True, v)))
    cache = pkv.PagedKVCache([pools[0]], [pools[1]], torch.arange(blocks, dtype=torch.int32, device="cuda").view(1, -1))
    q = torch.zeros(1, q_heads, D, dtype=torch.bfloat16)
    q[..., 0] = 1.0
    scale = float(np.float32(e * np.log(2.0) / 6.0))
    out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
    si = torch.tensor([[0, 1, 0, n]], dtype=torch.int32, device="cuda")
    if max_kv:
        assert pkv.attend_workspace_bytes(cache, q_heads, 1, 1, max_kv) > 0
    pkv.attend_varlen(cache, 0, q.cuda(), si, out, err, 1, max_kv or n, scale, lse=lse)
    w = np.exp(-6.0 * scale)
    total = blocks * (1 + 15 * w)
    ref, r = blocks * 15 * w * 6.0 / total, 2.0 ** -11 + e * 2.0 ** -22 + 2.0 ** -21 + n * 2.0 ** -24
    lim = blocks * 15 * 6.0 * (w * r + 2.0 ** -32) / total + 2 * r * ref
    assert int(err.item()) == 0
    worst = float(np.abs(out.cpu().numpy().astype(np.float64) - ref).max())
    assert worst <= lim, f"{worst} above {lim}; the output is {ref}"
    want = 6.0 * scale + np.log(total)
    assert np.abs(lse.cpu().numpy() - want).max() <= want * 2.0 ** -21 + n * 2.0 ** -24
