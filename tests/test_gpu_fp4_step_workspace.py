"""Captured steps over 4-bit caches whose launches merge through a workspace: two
at a time on two streams, and one whose bounds change."""
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


def make(pkv, hq, hkv, D, lens, seed, max_kv, dtype=torch.float32, with_rope=False):
    """A step of one token a sequence over a cache of `lens` tokens of history, with its rows in place."""
    from paged_kv_decode_13_gb300.graph import DecodeStep
    g = torch.Generator().manual_seed(seed)
    width = max(lens) // 16 + 1
    pools = [[torch.from_numpy(R.pack(*R.quantise(torch.randn(len(lens) * width, 16, hkv, D, generator=g).numpy()), bool(i))).cuda() for _ in range(2)]
             for i in range(2)]
    bt = torch.randperm(len(lens) * width, generator=g).to(torch.int32).view(len(lens), width).cuda()
    cache = pkv.PagedKVCache(*pools, bt)
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda") if with_rope else None
    step = DecodeStep(cache, hq, rows=len(lens), num_segments=len(lens), max_kv=max_kv, with_lse=True, rope=rope, out_dtype=dtype)
    step.seq_info.copy_(torch.tensor([[i, 1, i, n + 1] for i, n in enumerate(lens)], dtype=torch.int32))
    for t in step.q + step.k_new + step.v_new:
        t.copy_(torch.randn(t.shape, generator=g))
    return step


@pytest.mark.parametrize("with_rope", [False, True])
def test_two_runners_at_once(pkv, with_rope):
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner
    steps = [make(pkv, 16, 4, 128, [4000, 17, 2900, 1, 3500], 1, BIG, with_rope=with_rope),
             make(pkv, 32, 8, 128, [900, 3100, 2000, 5000, 64, 700, 1500], 2, BIG, dtype=torch.bfloat16, with_rope=with_rope),
             make(pkv, 64, 1, 128, [3000, 400], 3, BIG, with_rope=with_rope)]          # the wide kernel
    want = []
    for st in steps:
        assert st.ws is not None
        st.run()
        torch.cuda.synchronize()
        want.append(st.outputs.clone())
        assert int(st.err.item()) == 0 and bool(st.outputs.view(torch.uint8).any())
    runners, streams = [DecodeGraphRunner(st) for st in steps], [torch.cuda.Stream() for _ in steps]
    for r in runners:
        r.step()
    torch.cuda.synchronize()
    for a, b in ((0, 1), (1, 2), (0, 2)):
        for i in (a, b):
            steps[i].outputs.zero_()
        torch.cuda.synchronize()
        for _ in range(30):
            for i in (a, b):
                with torch.cuda.stream(streams[i]):
                    runners[i].step()
        torch.cuda.synchronize()
        for i in (a, b):
            assert torch.equal(steps[i].outputs, want[i]) and int(steps[i].err.item()) == 0


def test_rebound_step_captures_again(pkv):
    """New bounds that need no workspace free it; a capture that holds it is not replayed."""
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner
    st = make(pkv, 16, 4, 128, [400, 17, 290, 1, 350], 1, BIG)
    runner = DecodeGraphRunner(st)
    runner.step()
    torch.cuda.synchronize()
    want, ws = st.outputs.clone(), st.ws
    runner.rebind(st.cache)                         # the same bucket and generation, but max_kv is the bucket's now
    assert ws is not None and st.ws is None and st.max_kv == st.cache.bucket
    del ws
    junk = torch.full((32 << 20,), 0x77, dtype=torch.uint8, device="cuda")   # takes over the old one's memory
    st.outputs.zero_()
    runner.step()
    torch.cuda.synchronize()
    assert runner.captures == 2 and bool((junk == 0x77).all())
    a, b = [o[:st.out[0].numel() * 2 * 4].view(torch.float32).double().cpu().numpy() for o in (want, st.outputs)]
    assert np.abs(a - b).max() <= np.abs(a).max() * 2.0 ** -10 and int(st.err.item()) == 0   # weights rounded against another reference
