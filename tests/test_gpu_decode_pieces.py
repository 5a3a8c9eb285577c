"""A DecodeStep with a rope whose segments are pieces of one sequence: a later
piece attends to the keys that an earlier one appends in the same step."""
import pytest
import torch

from tests import fp4_ref as R

pytestmark = pytest.mark.gpu
LAYERS, HQ, HKV, D = 4, 8, 2, 128


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("pieces", [[40, 40, 40], [1, 1, 1, 1], [16, 64, 3, 100]])
def test_pieces_of_one_sequence(pkv, fp4, pieces):
    """The step equals the append and, once all of it has ended, the attention; again and again from other keys."""
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner, DecodeStep
    rows, width, g = sum(pieces), 100, torch.Generator().manual_seed(len(pieces))
    shape = (width, HKV, 9 * D) if fp4 else (width, 16, HKV, D)
    made = []
    for _ in range(2):
        pools = [[torch.zeros(shape, dtype=torch.uint8 if fp4 else torch.bfloat16, device="cuda") for _ in range(LAYERS)] for _ in range(2)]
        made.append(pkv.PagedKVCache(*pools, torch.randperm(width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, -1).cuda()))
    cache, eager = made
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda")
    step = DecodeStep(cache, HQ, rows=rows, num_segments=len(pieces), max_q_len=max(pieces), causal=True, with_lse=True, rope=rope)
    ends = torch.tensor(pieces).cumsum(0) + 777
    step.seq_info.copy_(torch.tensor([[int(e) - 777 - n, n, 0, int(e)] for n, e in zip(pieces, ends)], dtype=torch.int32))
    runner, err = DecodeGraphRunner(step), pkv.new_err_flags()
    for it in range(8):
        for t in step.q + step.k_new + step.v_new:
            t.copy_(torch.randn(t.shape, generator=g))
        for c in (cache, eager):                    # other older keys than the last time's
            for la in range(LAYERS):
                for i, p in enumerate((c.k[la], c.v[la])):
                    x = torch.randn(width, 16, HKV, D, generator=torch.Generator().manual_seed(it * 10 + la * 2 + i)) * 2
                    p.copy_(torch.from_numpy(R.pack(*R.quantise(x.numpy()), bool(i))) if fp4 else x)
        torch.cuda.synchronize()
        runner.step()
        torch.cuda.synchronize()
        for la in range(LAYERS):
            q = step.q[la].clone()
            pkv.norm_rope_append(eager, la, rope, q, step.k_new[la], step.v_new[la], step.seq_info, None, err)
            torch.cuda.synchronize()
            out, lse = torch.empty_like(step.out[la]), torch.empty_like(step.lse[la])
            pkv.attend_varlen(eager, la, q, step.seq_info, out, err, max(pieces), step.max_kv, step.scale, causal=True, lse=lse)
            torch.cuda.synchronize()
            assert torch.equal(cache.k[la], eager.k[la]) and torch.equal(cache.v[la], eager.v[la])
            assert torch.equal(step.out[la], out) and torch.equal(step.lse[la], lse)
    assert int(step.err.item()) == 0 and int(err.item()) == 0
