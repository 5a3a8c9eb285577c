"""bf16 and fp32 attention at positions up to the largest that a segment may end
at, 2^31 - 33: the same pages at near and at far positions give the same results."""
import pytest
import torch

pytestmark = pytest.mark.gpu
END = 0x7FFFFFFF - 32
PAGES, H, D = 64, 2, 128          # pages of the sequence that exist: its last ones


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


@pytest.fixture(scope="module")
def tables():
    ids = torch.randperm(PAGES, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
    last = END // 16 + 1
    table = torch.full((1, 1 << 27), -1, dtype=torch.int32, device="cuda")
    table[0, last - PAGES:last] = ids
    yield table, ids.view(1, -1), (last - PAGES) * 16


@pytest.mark.parametrize("dtype,flags", [(torch.bfloat16, 0), (torch.bfloat16, 1), (torch.bfloat16, 2), (torch.bfloat16, 8), (torch.float32, 0)])
@pytest.mark.parametrize("q_heads,q_len,window,causal", [(2, 1, 300, False), (8, 1, 700, True), (16, 9, 500, True), (64, 4, 333, True), (64, 40, 600, False)])
@pytest.mark.parametrize("fused", [False, True])
def test_attention(pkv, tables, dtype, flags, q_heads, q_len, window, causal, fused):
    far_table, near_table, shift = tables
    g = torch.Generator().manual_seed(q_heads)
    pools = [torch.randn(PAGES, 16, H, D, generator=g).to(dtype).cuda() for _ in range(2)]
    q, kn, vn = [torch.randn(q_len, h, D, generator=g).to(dtype).cuda() for h in (q_heads, H, H)]
    for back in (0, 1, 15, 20):
        got = []
        for table, end in ((far_table, END - back), (near_table, END - back - shift)):
            cache = pkv.PagedKVCache([pools[0].clone()], [pools[1].clone()], table)
            si = torch.tensor([[0, q_len, 0, end]], dtype=torch.int32, device="cuda")
            out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
            if fused:
                pkv.append_attend(cache, 0, q, kn, vn, si, out, err, q_len, 1 << 31, D ** -0.5, causal, window, lse=lse, flags=flags)
            else:
                pkv.append(cache, 0, kn, vn, si, err)
                pkv.attend_varlen(cache, 0, q, si, out, err, q_len, 1 << 31, D ** -0.5, causal, window, lse=lse, flags=flags & ~pkv.FLAG_PDL)
            assert int(err.item()) == 0
            got.append((out, lse, cache.k[0], cache.v[0]))
        assert all(torch.equal(a, b) for a, b in zip(*got))
