"""Rows that several segments of a call hold, in an 8-bit cache: their queries are turned once, in place too."""
import numpy as np
import pytest
import torch

import workloads
from tests.test_gpu_fp8 import Fp8, check_append

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


TABLES = [
    [[0, 7, 0, 20], [20, 9, 1, 30], [0, 7, 0, 20], [20, 9, 1, 30], [20, 9, 1, 30]],     # a padded batch
    [[0, 5, 0, 20], [3, 20, 1, 40], [2, 2, 2, 33]],                                     # sequences that begin with the same rows
    [[10, 12, 3, 40], [0, 5, 9, 20], [3, 20, 1, 40], [2, 2, 2, 33], [4, 1, 0, 1]],      # the lowest on a bad page or refused
    [[i % 30, 1, i % 3, 10 + i] for i in range(100)],                                   # more than a warp has lanes
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("table", TABLES)
@pytest.mark.parametrize("given", [False, True])
def test_queries_in_place(pkv, D, table, given):
    w = workloads.batched(S=4, max_len=128, lengths=[128] * 4, q_heads=8, kv_heads=2, head_dim=D)
    w.block_table[3, 2] = 1 << 20
    rows = 40
    g = torch.Generator().manual_seed(D)
    q, kn, vn = [torch.randn(rows, h, D, generator=g).bfloat16().cuda() for h in (8, 2, 2)]
    wq, wk = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)]
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], q_weight=wq, k_weight=wk, device="cuda")
    positions = torch.randint(0, 5000, (rows,), generator=g, dtype=torch.int32) if given else None
    valid = [s for s in table if s[2] < 3]
    at, new = np.zeros(rows, np.int32), np.zeros(rows, bool)
    for q0, n, _, kend in reversed(valid):
        at[q0:q0 + n], new[q0:q0 + n] = np.arange(kend - n, kend), True
    want = q.clone()
    pkv.norm_rope(rope, want, kn.clone(), positions.cuda() if given else torch.from_numpy(at).cuda())
    want = torch.where(torch.from_numpy(new).cuda()[:, None, None], want, q)
    w.seq_info = torch.tensor(table, dtype=torch.int32)
    for _ in range(3):
        f, err, turned = Fp8(pkv, w), pkv.new_err_flags(), q.clone()
        pkv.norm_rope_append(f.cache, 0, rope, turned, kn, vn, w.seq_info.cuda(), None, err, positions=None if not given else positions.cuda())
        torch.cuda.synchronize()
        bad = {s[2] for s in table if s not in valid}
        assert int(err.item()) == (1 if 9 in bad else 0) | (8 if 3 in bad else 0)
        assert torch.equal(turned, want)
        f.check_guards()
        if given:    # (otherwise a row's k differs from segment to segment)
            k2 = kn.clone()
            pkv.norm_rope(rope, None, k2, positions.cuda())
            check_append(f, f.bytes, k2, vn, None, None, si=valid)
