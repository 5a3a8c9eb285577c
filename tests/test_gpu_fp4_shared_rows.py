"""Appends to a 4-bit cache whose segments share rows of k_new and v_new: each
segment gets the row's K and V, as in the other cache types."""
import numpy as np
import pytest
import torch

import workloads
from tests import fp4_ref as R
from tests import gpu_util as U
from tests.test_gpu_fp4 import Fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def workload(D, segments, rows, kv_heads=3):
    w = workloads.batched(S=6, max_len=160, lengths=[160] * 6, q_heads=kv_heads, kv_heads=kv_heads, head_dim=D, seed=D)
    g = torch.Generator().manual_seed(rows)
    w.q, w.k_new, w.v_new = [[torch.randn(rows, kv_heads, D, generator=g).bfloat16()] for _ in range(3)]
    w.block_table[5, 1] = -4
    w.seq_info = torch.tensor(segments, dtype=torch.int32)
    return w


SEGMENTS = [
    [[0, 1, 0, 20], [0, 1, 1, 33]],                                           # one token, two sequences
    [[0, 7, 0, 40], [4, 6, 1, 70], [5, 1, 2, 1], [20, 3, 3, 9]],              # overlapping steps
    [[3, 4, 5, 20], [0, 9, 1, 50], [2, 70, 0, 90], [40, 30, 3, 155]],         # the lowest segment is on a bad page
    [[3, 4, 0, 3], [3, 4, 9, 20], [3, 4, 1, 33], [0, 90, 2, 91], [6, 2, 5, 18]],  # refused ones among them
    [[i % 5, 3, i % 5, 30 + 3 * i] for i in range(40)],                       # many; sequence i % 5 goes on
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("segments", SEGMENTS)
def test_each_segment_gets_k_and_v(pkv, D, segments):
    w = workload(D, segments, 100)
    f, err = Fp4(pkv, w), pkv.new_err_flags()
    kn, vn = w.k_new[0].cuda(), w.v_new[0].cuda()
    pkv.append(f.cache, 0, kn, vn, w.seq_info.cuda(), err)
    want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
    assert int(err.item()) == e >> 1   # (the oracle counts its bits from 1)
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    f.check_guards()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("segments", [
    [[0, 1, 0, 20]] * 2, [[3, 1, 1, 33], [0, 1, 0, 20]] + [[1, 1, 2, 50]] * 6,    # a padded decode step
    [[0, 7, 0, 40]] * 3 + [[10, 60, 2, 71]] * 2, [[5, 31, 1, 39], [10, 20, 1, 33], [0, 3, 0, 3]],   # and a piece of a segment again
])
def test_the_same_slot_twice_with_the_same_row(pkv, D, segments):
    w = workload(D, segments, 100)
    want = None
    for _ in range(10):
        f, err = Fp4(pkv, w), pkv.new_err_flags()
        pkv.append(f.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), err)
        if want is None:
            want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
        assert int(err.item()) == e == 0
        for i in (0, 1):
            assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]


ONE_EACH = [[2 * i, 2, i % 5, 10 + 3 * i] for i in range(45)]
LONG_TABLES = [
    ONE_EACH, ONE_EACH[::-1], ONE_EACH + [[0, 0, 0, 0]] * 60,                  # in order, backwards, padded behind
    [[0, 0, 0, 0]] * 3 + ONE_EACH, ONE_EACH + [[0, 0, 0, 0], [20, 2, 4, 3]],  # empty ones in front of others, one of which shares
    ONE_EACH[:40] + [[79, 3, 4, 6]], [[0, 90, 3, 95]] + ONE_EACH[:3] + ONE_EACH[4::5],   # the last row again; one segment over all
    [[-1, 2, 0, 9], [5, -3, 1, 9]] + ONE_EACH + [[2, 99, 1, 120], [88, 4, 3, 150]],   # refused ones
]


@pytest.mark.parametrize("segments", LONG_TABLES)
def test_long_tables(pkv, segments):
    """More segments than a warp has lanes, sharing rows or not, in any order."""
    w = workload(64, segments, 100)
    f, err = Fp4(pkv, w), pkv.new_err_flags()
    pkv.append(f.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), err)
    want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
    assert int(err.item()) == e >> 1
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    f.check_guards()


@pytest.mark.parametrize("segments", SEGMENTS)
@pytest.mark.parametrize("given", [False, True])
def test_rotated_and_in_place(pkv, segments, given):
    """With a rotation: turned once, by the given position or by its place in the lowest segment that takes the row; q and k change in place."""
    D, rows = 128, 100
    w = workload(D, segments, rows)
    f, err = Fp4(pkv, w), pkv.new_err_flags()
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda")
    pos, live = np.full(rows, -1), np.zeros(rows, bool)
    for q0, n, col, kend in segments:
        if col >= 6 or n > kend or (col == 5 and kend > 16):
            continue
        for i in range(n):
            if pos[q0 + i] < 0:
                pos[q0 + i] = kend - n + i
            live[q0 + i] = True
    if given:
        pos = np.arange(rows) * 17 % 4001
    dpos = torch.from_numpy(np.maximum(pos, 0).astype(np.int32)).cuda()
    k2 = w.k_new[0].cuda()
    q2 = w.q[0].cuda()
    pkv.norm_rope(rope, q2, k2, dpos)
    q, kn, vn = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda()
    vo = vn.clone()
    pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, w.seq_info.cuda(), None, err, positions=dpos if given else None, k_out=kn, v_out=vo)
    want, e = f.oracle_bytes(k2.cpu(), w.v_new[0])
    assert int(err.item()) == e >> 1   # (the oracle counts its bits from 1)
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    dead = torch.from_numpy(~live).cuda()
    for got, x, y in ((q, q2, w.q[0]), (kn, torch.from_numpy(R.values(*R.quantise(U.f64(k2)))).bfloat16().cuda(), w.k_new[0]),
                      (vo, torch.from_numpy(R.values(*R.quantise(U.f64(w.v_new[0])))).bfloat16().cuda(), w.v_new[0])):
        assert torch.equal(got[~dead], x[~dead]) and torch.equal(got[dead], y.cuda()[dead])
