"""Rejected drafts in an 8-bit cache: what a rewind leaves of them."""
import numpy as np
import pytest
import torch

import workloads
from tests import fp8_ref as R
from tests import gpu_util as U
from tests.test_gpu_fp8 import attend, check, check_append, run_append, zeroed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def values(f, n):
    """What the sequence's first n tokens are held as, K and V, and the scales of their pages [pages, H]."""
    w, out = f.w, []
    blocks = w.block_table[0, :-(-n // 16)].numpy()
    for i in (0, 1):
        v = R.pool_values(f.host(i))[blocks]
        out.append((v.reshape(-1, *v.shape[2:])[:n], R.scale(R.unpack(f.host(i))[1][blocks])))
    return out


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("size", [0.5, 8.0, float("inf")])
@pytest.mark.parametrize("first,drafts", [(21, 6), (21, 20), (32, 5), (47, 1)])
def test_rejected_drafts(pkv, D, size, first, drafts):
    """Tokens before the drafts lose at most 2^-10 of the scale that these made; pages without such tokens start afresh."""
    w = workloads.batched(S=1, max_len=96, lengths=[96], q_heads=4, kv_heads=2, head_dim=D)
    f, g = zeroed(pkv, w), torch.Generator().manual_seed(D)
    si, err = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), pkv.new_err_flags()

    def step(n, end, big=1.0):
        rows = [torch.randn(n, 2, D, generator=g) for _ in range(2)]
        for x in rows:
            x[n // 2, 0] *= 1.0 if np.isinf(big) else big
            if np.isinf(big):
                x[n // 2, 0, 3] = big
        rows = [x.bfloat16() for x in rows]
        w.seq_info = torch.tensor([[0, n, 0, end]], dtype=torch.int32)
        before = [f.host(i).copy() for i in (0, 1)]
        ko, vo, e = run_append(pkv, f, *rows)
        assert e == 0
        check_append(f, before, *rows, ko, vo)
        return rows

    step(first, first)
    kept = values(f, first)
    step(drafts, first + drafts, size)
    raised = values(f, first)
    si.copy_(w.seq_info)
    pkv.rewind(f.cache, si, torch.tensor([drafts], dtype=torch.int32, device="cuda"), err)
    assert int(err.item()) == 0 and si.tolist() == [[0, drafts, 0, first]]
    for (a, _), (b, s) in zip(kept, raised):
        lim = 2.0 ** -10 * np.repeat(s, 16, 0)[:first, :, None]
        assert (np.abs(a - b) <= lim).all()
        whole = first // 16 * 16
        assert np.array_equal(a[:whole], b[:whole])      # pages before that of the first draft
    rows = step(3, first + 3)
    after = values(f, first + 3)
    for (b, s), (c, t), x in zip(raised, after, rows):
        # the new rows do not move the tokens again, unless they are the larger ones
        same = t[:-(-first // 16)] == s
        assert np.array_equal(np.repeat(same, 16, 0)[:first, :, None] & (b != c[:first]), np.zeros_like(b, bool))
        # and are held to half a step, or 2^-10 of their page's scale
        scale = np.repeat(t, 16, 0)[first:first + 3, :, None]
        x = U.f64(x)
        assert (np.abs(c[first:] - x) <= np.abs(x) * 2.0 ** -4 + 2.0 ** -10 * scale).all()
        if first % 16 == 0:
            assert (t[first // 16] <= 2.0 ** -5).all()   # (448 2^-5 = 14, beyond any of these rows)
    w.q = [torch.randn(3, 4, D, generator=g).bfloat16()]
    out, lse, e = attend(pkv, f, causal=True, max_q=3)
    assert e == 0
    check(f, out, lse, causal=True)
