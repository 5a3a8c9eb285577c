"""Rotary positions with several axes (norm_rope, norm_rope_append) on the GPU
against the 64-bit definition: pair i of a row is turned by the row's position
on axis[i].  Tolerances are those of test_gpu_rope.py: an axis changes which
position a pair takes and nothing of its arithmetic.
"""
import numpy as np
import pytest
import torch

import workloads
from tests import fp4_ref as F4
from tests import gpu_util as U
from tests import test_gpu_rope as T

pytestmark = pytest.mark.gpu
pkv = T.pkv


def check_axes(got, x, weight, eps, freq, axis, pos, mscale, interleaved, dtype):
    """Row by row: turning pair i by pos[axis[i]] * freq[i] is turning it by position 1 at that frequency."""
    for r in range(got.shape[0]):
        own = torch.tensor(pos[r][axis].astype(np.float64)) * freq.double()
        T.check_rows(got[r:r + 1], x[r:r + 1], weight, eps, own, np.ones(1), mscale, interleaved, dtype)


def positions(rows, axes, seed, far=1 << 16):
    g = torch.Generator().manual_seed(seed)
    p = torch.randint(0, far, (rows, axes), generator=g, dtype=torch.int32)
    p[0] = 0
    return p


CASES = [  # D, sections, dealt, interleaved, dtype
    (128, (16, 24, 24), False, False, torch.bfloat16), (128, (24, 20, 20), True, False, torch.bfloat16),
    (80, (20, 20), False, False, torch.bfloat16), (80, (7, 4), True, True, torch.float32), (64, (1, 0, 2), False, False, torch.bfloat16),
    (256, (32, 32, 32, 32), True, True, torch.bfloat16), (72, (5, 6), False, False, torch.float32), (8, (1, 1, 1, 1), False, True, torch.float32),
    (64, (4,) * 8, True, False, torch.bfloat16),
]


@pytest.mark.parametrize("D,sections,dealt,interleaved,dtype", CASES)
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_axes(pkv, D, sections, dealt, interleaved, dtype, norm):
    rows, hq, hkv = 6, 7, 3
    q, k, _, wq, wk = T.make(D, rows, hq, hkv, D, dtype)
    axis = np.array(pkv.rope_axes(sections, dealt))
    freq, m = pkv.rope_inv_freq(2 * len(axis))
    rope = pkv.Rope(freq, interleaved, mscale=m, q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-5, device="cuda", axes=axis)
    pos = positions(rows, len(sections), D)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pkv.norm_rope(rope, q, k, pos.cuda(), qo, ko)
    check_axes(qo, q, wq if norm else None, 1e-5, freq, axis, pos.numpy(), m, interleaved, dtype)
    check_axes(ko, k, wk if norm else None, 1e-5, freq, axis, pos.numpy(), m, interleaved, dtype)
    pkv.norm_rope(rope, q, k, pos.cuda())   # in place: bit for bit the same
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("rows", [1, 333, 5000])
def test_equal_positions_are_one_axis(pkv, rows):
    """Rows whose axes agree (text) come out as without axes, bit for bit."""
    D = 128
    q, k, _, wq, wk = T.make(rows, rows, 8, 2, D, torch.bfloat16)
    freq, _ = pkv.rope_inv_freq(D)
    one = pkv.Rope(freq, q_weight=wq, k_weight=wk, device="cuda")
    many = pkv.Rope(freq, q_weight=wq, k_weight=wk, device="cuda", axes=pkv.rope_axes((22, 21, 21), True))
    pos = positions(rows, 1, 3, 1 << 30)[:, 0].cuda()
    a, b = [[torch.empty_like(q), torch.empty_like(k)] for _ in range(2)]
    pkv.norm_rope(one, q, k, pos, *a)
    pkv.norm_rope(many, q, k, pos[:, None].expand(-1, 3).contiguous(), *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64)])
@pytest.mark.parametrize("max_q", [1, 37])
def test_append_axes(pkv, dtype, D, max_q):
    w = U.nan_tails(workloads.spec_verify(S=6, max_q=max_q, len_lo=max_q, len_hi=200, seed=D, q_heads=12, kv_heads=3, head_dim=D, dtype=dtype))
    freq, m = pkv.rope_inv_freq(D)
    axis = np.array(pkv.rope_axes((D // 2 - 2 * (D // 8), D // 8, D // 8), True))
    pos = positions(w.total_rows, 3, D)
    _, cache, qo, ko, vo, err, wq, wk = T.run_append(pkv, w, dict(axes=axis), freq, True, positions=pos.cuda())
    assert err == 0
    _, rows = T.cache_positions(w)
    check_axes(qo[rows], w.q[0][rows], wq, 1e-6, freq, axis, pos.numpy()[rows], m, False, dtype)
    check_axes(ko[rows], w.k_new[0][rows], wk, 1e-6, freq, axis, pos.numpy()[rows], m, False, dtype)
    assert torch.equal(vo[rows].cpu(), w.v_new[0][rows])
    w.k_new[0], w.v_new[0] = ko.cpu(), vo.cpu()
    kp, vp, e = U.oracle_append_pools(w, 0)
    assert e == 0 and U.pool_bytes(cache.k[0]) == kp.tobytes() and U.pool_bytes(cache.v[0]) == vp.tobytes()


def test_append_without_positions_takes_the_cache_position_on_every_axis(pkv):
    w = workloads.spec_verify(S=3, max_q=5, len_lo=8, len_hi=90, seed=1, q_heads=4, kv_heads=2, head_dim=64, dtype=torch.bfloat16)
    freq, _ = pkv.rope_inv_freq(64)
    got = []
    for axes in (None, pkv.rope_axes((12, 10, 10))):
        _, cache, qo, ko, _, err, _, _ = T.run_append(pkv, w, dict(axes=axes), freq, True)
        assert err == 0
        got.append((qo, ko, cache.k[0]))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_append_axes_four_bit(pkv):
    """The 4-bit append turns its K rows the same way: k_out is the quantised form of the turned row."""
    D, rows, S = 128, 40, 2
    g = torch.Generator().manual_seed(7)
    k, v = [torch.randn(rows, 2, D, generator=g).bfloat16().cuda() for _ in range(2)]
    pools = [torch.zeros(8, 2, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    si = torch.tensor([[0, 23, 0, 30], [23, 17, 1, 17]], dtype=torch.int32, device="cuda")
    freq, _ = pkv.rope_inv_freq(D)
    rope = pkv.Rope(freq, device="cuda", axes=pkv.rope_axes((16, 24, 24)))
    pos = positions(rows, 3, 2).cuda()
    turned, ko, err = torch.empty_like(k), torch.empty_like(k), pkv.new_err_flags()
    pkv.norm_rope(rope, None, k, pos, None, turned)
    cache = pkv.PagedKVCache([pools[0]], [pools[1]], table)
    pkv.norm_rope_append(cache, 0, rope, None, k, v, si, None, err, positions=pos, k_out=ko)
    assert int(err.item()) == 0
    assert np.array_equal(U.f64(ko), F4.values(*F4.quantise(U.f64(turned))))


def test_axis_past_the_last_counts_as_the_last(pkv):
    """An axis number that only the device sees stays inside the row's positions."""
    rope = pkv.Rope(pkv.rope_inv_freq(64)[0], device="cuda", axes=[0] * 16 + [1] * 16)
    q = torch.randn(9, 4, 64, device="cuda")
    pos = positions(9, 2, 5).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    pkv.norm_rope(rope, q, None, pos, a)
    rope.axis[20:] = 255
    pkv.norm_rope(rope, q, None, pos, b)
    assert torch.equal(a, b)


def test_captured_axes(pkv):
    """One capture serves the positions that are in the buffer at each replay."""
    rope = pkv.Rope(pkv.rope_inv_freq(128)[0], device="cuda", axes=pkv.rope_axes((22, 21, 21)))
    q, k, _, _, _ = T.make(1, 4, 8, 2, 128, torch.bfloat16)
    pos = torch.zeros(4, 3, dtype=torch.int32, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.norm_rope(rope, q, k, pos, qo, ko)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.norm_rope(rope, q, k, pos, qo, ko)
    for seed in (1, 2):
        pos.copy_(positions(4, 3, seed))
        graph.replay()
        a, b = torch.empty_like(q), torch.empty_like(k)
        pkv.norm_rope(rope, q, k, pos, a, b)
        assert torch.equal(a, qo) and torch.equal(b, ko)
