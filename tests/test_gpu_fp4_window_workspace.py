"""Attention over a 4-bit cache with a window and a workspace that the size query
(which knows no window) does not ask for."""
import random

import pytest
import torch

import workloads
from tests.test_gpu_fp4 import Fp4, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def differing_bounds(pkv, f, w):
    """(segments, max_kv, window) for which max_kv keys need no workspace, and the few less that the window leaves do.

    They are rare: the cost of clusters steps with the keys, that of shares does not."""
    r, found = random.Random(1), []
    for _ in range(6000):
        S, max_kv = r.randint(5, 512), int(2 ** r.uniform(11, 16.5))
        if pkv.attend_workspace_bytes(f.cache, w.q_heads, S, 1, max_kv) == 0:
            for cut in (16, 32, 64):
                if pkv.attend_workspace_bytes(f.cache, w.q_heads, S, 1, max_kv - cut):
                    found.append((S, max_kv, max_kv - cut - 1))
                    break
    return found


def test_a_small_workspace_is_taken_where_none_is_asked_for(pkv):
    tried = 0
    for D, q_heads, kv_heads in ((128, 1, 1), (128, 32, 1), (128, 64, 2), (256, 1, 1), (64, 2, 2)):
        w = workloads.batched(S=5, max_len=2000, seed=D, lengths=[1500, 3, 700, 2000, 1], q_heads=q_heads, kv_heads=kv_heads, head_dim=D)
        f = Fp4(pkv, w)
        for S, max_kv, window in differing_bounds(pkv, f, w)[:2]:
            si = torch.cat([w.seq_info, torch.zeros(S - w.num_segments, 4, dtype=torch.int32)]).cuda()
            q = w.q[0].cuda()
            out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
            buf = torch.full((8192,), 0xA5, dtype=torch.uint8, device="cuda")
            pkv.attend_varlen(f.cache, 0, q, si, out, err, 1, max_kv, w.scale, w.causal, window, lse=lse, workspace=buf[:256])
            assert int(err.item()) == 0 and bool((buf == 0xA5).all())
            check(f, out, lse, window=window)
            tried += 1
            # one below the size asked for is refused still
            with pytest.raises(pkv.PkvError):
                pkv.attend_varlen(f.cache, 0, q, si, out, err, 1, window + 1, w.scale, w.causal, 0, lse=lse, workspace=buf[:256])
    assert tried > 0
