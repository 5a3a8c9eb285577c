"""A captured DecodeStep whose ropes have several axes: positions that are not the rows' places in the cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8, torch.float8_e4m3fn])
@pytest.mark.parametrize("axes", [None, (32, 16, 16)])
def test_captured_steps_after_an_image(pkv, dtype, axes):
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner, DecodeStep
    L, Hq, Hkv, D, n = 2, 8, 2, 128, 100
    cache, plain = [pkv.PagedKVCache.allocate(L, Hkv, D, 256, dtype=dtype) for _ in range(2)]
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda", axes=None if axes is None else pkv.rope_axes(axes, dealt=True))
    step = DecodeStep(cache, Hq, max_kv=256, advance=True, rope=rope, positions=True)
    run = DecodeGraphRunner(step)
    g = torch.Generator().manual_seed(0)
    # n rows of text and an image are in the cache, text position 40 (so far) on every axis
    q, kn, vn = [torch.randn(n, h, D, generator=g).bfloat16().cuda() for h in (Hq, Hkv, Hkv)]
    at = torch.randint(0, 40, (n,) if axes is None else (n, 3), generator=g, dtype=torch.int32).cuda()
    si, err = torch.tensor([[0, n, 0, n]], dtype=torch.int32, device="cuda"), pkv.new_err_flags()
    for c in (cache, plain):
        for layer in range(L):
            pkv.norm_rope_append(c, layer, rope, q, kn, vn, si, torch.empty_like(q), err, positions=at)
    step.seq_info.copy_(torch.tensor([[0, 1, 0, n + 1]], dtype=torch.int32))
    si = step.seq_info.clone()
    for t in range(20):
        step.positions.fill_(40 + t)
        for layer in range(L):
            for dst in (step.q, step.k_new, step.v_new):
                dst[layer].copy_(torch.randn(dst[layer].shape, generator=g).bfloat16())
        run.step()
        for layer in range(L):
            turned = torch.empty_like(step.q[layer])
            pkv.norm_rope_append(plain, layer, rope, step.q[layer], step.k_new[layer], step.v_new[layer], si, turned, err, positions=step.positions)
            out = torch.empty(1, Hq, D, device="cuda")
            pkv.attend_varlen(plain, layer, turned, si, out, err, 1, 256, step.scale)
            assert torch.equal(step.q_rot[layer], turned) and torch.equal(step.out[layer], out)
            # what the row's place in the cache would give is something else
            other = step.q[layer].clone()
            pkv.norm_rope(rope, other, None, (si[:, 3] - 1).contiguous() if axes is None else (si[:, 3:] - 1).expand(1, 3).contiguous())
            assert not torch.equal(other, turned)
        pkv.advance(si)
    assert int(err.item()) == 0 and int(step.err.item()) == 0 and torch.equal(si, step.seq_info)
