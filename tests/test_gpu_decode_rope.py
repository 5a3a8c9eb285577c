"""DecodeStep over rows as the projections give them: norm + rotary + append,
then attention, layer after layer, over bf16 and 4-bit caches, captured and replayed.

A replay must equal the operators called one by one (norm_rope, append,
attend_varlen; their own tests compare them with the definitions), and at every step
the turned queries and the attention over what the pools then hold meet the 64-bit
definitions: the queries within the norm + rotary tolerance, the attention
within the 4-bit kernels' tolerance or the 2e-3 of the bf16 tests."""
import numpy as np
import pytest
import torch

import workloads
from tests import fp4_ref as R
from tests import gpu_util as U
from tests import test_gpu_fp4 as F
from tests.test_gpu_rope import check_rows

pytestmark = pytest.mark.gpu
LAYERS, HQ, HKV, D, LENS, Q = 3, 8, 2, 128, [40, 0, 611, 15], [1, 1, 4, 2]


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def caches(pkv, fp4):
    """Two equal caches with LENS tokens of history."""
    w = workloads.batched(S=4, max_len=704, lengths=[n + 32 for n in LENS], num_layers=LAYERS, q_heads=HQ, kv_heads=HKV, head_dim=D, seed=5)
    made = []
    for _ in range(2):
        pools = []
        for i, side in enumerate((w.k, w.v)):
            x = [torch.nan_to_num(t.float(), nan=0.0) * (1 - i + 1) for t in side]
            pools.append([torch.from_numpy(R.pack(*R.quantise(t.numpy()), bool(i))).cuda() if fp4 else t.bfloat16().cuda() for t in x])
        made.append(pkv.PagedKVCache(*pools, w.block_table.cuda(), bucket=w.bucket))
    return w, made


@pytest.mark.parametrize("fp4,out_dtype", [(False, torch.float32), (True, torch.float32), (True, torch.bfloat16)])
@pytest.mark.parametrize("max_kv,shares", [(704, False), (1 << 20, True)])
@pytest.mark.parametrize("per_layer", [False, True])
def test_rope_steps_in_a_graph(pkv, fp4, out_dtype, max_kv, shares, per_layer):
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner, DecodeStep
    w, (cache, eager) = caches(pkv, fp4)
    rows, g = sum(Q) + 1, torch.Generator().manual_seed(3)          # one padding row at the end
    freq, _ = pkv.rope_inv_freq(64)
    weight = lambda: (1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda()  # noqa: E731
    ropes = [pkv.Rope(freq, q_weight=weight(), k_weight=weight(), device="cuda") for _ in range(LAYERS if per_layer else 1)]
    step = DecodeStep(cache, HQ, rows=rows, num_segments=4, max_q_len=4, max_kv=max_kv, causal=True, with_lse=True, advance=True,
                      rope=ropes if per_layer else ropes[0], out_dtype=out_dtype)
    if fp4:
        assert (pkv.attend_workspace_bytes(cache, HQ, 4, 4, max_kv) > 0) == shares
    assert step.launch_count() == 2 * LAYERS + 1
    runner = DecodeGraphRunner(step)
    q0 = np.cumsum([0] + Q[:-1])
    step.seq_info.copy_(torch.tensor([[int(a), n, s, LENS[s] + n] for s, (a, n) in enumerate(zip(q0, Q))], dtype=torch.int32))
    err = pkv.new_err_flags()
    for it in range(6):
        si = step.seq_info.clone()
        fresh = [(torch.randn(t.shape, generator=g) * s).bfloat16() for ts, s in ((step.q, 2.0), (step.k_new, 1.0), (step.v_new, 1.0)) for t in ts]
        step.step_inputs.copy_(torch.cat([t.view(torch.uint8).reshape(-1) for t in fresh]))
        runner.step()
        pos = np.zeros(rows, np.int32)
        for a, n, _, e in si.tolist():
            pos[a:a + n] = np.arange(e - n, e)
        dpos = torch.from_numpy(pos).cuda()
        for la in range(LAYERS):
            rope = ropes[la if per_layer else 0]
            q, k, v = step.q[la].clone(), step.k_new[la].clone(), step.v_new[la].clone()
            pkv.norm_rope(rope, q, k, dpos)
            pkv.append(eager, la, k, v, si, err)
            out, lse = torch.empty_like(step.out[la]), torch.empty_like(step.lse[la])
            pkv.attend_varlen(eager, la, q, si, out, err, 4, max_kv, step.scale, causal=True, lse=lse)
            torch.cuda.synchronize()
            assert torch.equal(step.q_rot[la][:-1], q[:-1]) and (step.q_rot[la][-1] == 0).all()
            assert torch.equal(cache.k[la], eager.k[la]) and torch.equal(cache.v[la], eager.v[la])
            assert torch.equal(step.out[la], out) and torch.equal(step.lse[la], lse)
            assert (out[-1] == 0).all() and torch.isinf(lse[-1]).all()
            check_rows(q[:-1], step.q[la][:-1], rope.q_weight, rope.eps, freq, pos[:-1], 1.0, False, torch.bfloat16)
            if fp4:
                check_fp4(eager, la, w, q, si, out, lse, step.scale)
            else:
                ref, _, e = F.O.attend(U.f64(q), U.f64(eager.k[la]), U.f64(eager.v[la]), w.block_table.numpy(), si.cpu().numpy(),
                                       step.scale, causal=True)
                assert e == 0 and float(np.abs(U.f64(out) - ref).max()) <= 2e-3 * max(1.0, float(eager.v[la].float().abs().max()))
    assert runner.captures == 1 and int(step.err.item()) == 0 and int(err.item()) == 0
    assert step.seq_info[:, 3].tolist() == [LENS[s] + 7 * n for s, n in enumerate(Q)]


def check_fp4(cache, layer, w, q, si, out, lse, scale):
    f = F.Fp4.__new__(F.Fp4)
    f.w, f.first_valid = w, None
    f.host = lambda i: (cache.k if i == 0 else cache.v)[layer].cpu().numpy()
    assert abs(w.scale - scale) < 1e-7 * scale
    w.seq_info, w.causal = si.cpu(), True
    F.check(f, out, lse, q=q)


def test_plain_step_over_a_4bit_cache(pkv):
    """Without a rope: append_attend, and the two calls, give the same step."""
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner, DecodeStep
    w, (a, b) = caches(pkv, True)
    steps = [DecodeStep(c, HQ, rows=4, num_segments=4, max_kv=704, fused=fused, with_lse=True) for c, fused in ((a, True), (b, False))]
    g = torch.Generator().manual_seed(4)
    rows = torch.cat([torch.randn(n, generator=g).bfloat16().view(torch.uint8) for n in [4 * HQ * D] * LAYERS + [4 * HKV * D] * 2 * LAYERS])
    for st in steps:
        st.step_inputs.copy_(rows)
        st.seq_info.copy_(torch.tensor([[i, 1, i, n + 1] for i, n in enumerate(LENS)], dtype=torch.int32))
        assert st.launch_count() == 2 * LAYERS
        DecodeGraphRunner(st).step()
    torch.cuda.synchronize()
    assert torch.equal(steps[0].outputs, steps[1].outputs) and int(steps[0].err.item()) == int(steps[1].err.item()) == 0
    for la in range(LAYERS):
        assert torch.equal(a.k[la], b.k[la]) and torch.equal(a.v[la], b.v[la])
        check_fp4(a, la, w, steps[0].q[la], steps[0].seq_info, steps[0].out[la], steps[0].lse[la], steps[0].scale)


def test_step_refusals(pkv):
    from paged_kv_decode_13_gb300.graph import DecodeStep
    _, (cache, _) = caches(pkv, False)
    freq, _ = pkv.rope_inv_freq(D)
    with pytest.raises(ValueError):
        DecodeStep(cache, HQ, rope=[pkv.Rope(freq, device="cuda")] * (LAYERS - 1))
    with pytest.raises(ValueError):
        DecodeStep(cache, HQ, out_dtype=torch.bfloat16)
