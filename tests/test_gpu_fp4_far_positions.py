"""Positions up to the largest that a segment may end at, 2^31 - 33: the same
pages at near and at far positions give the same results, bit for bit."""
import pytest
import torch

from tests import fp4_ref as R

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
def caches(pkv):
    g = torch.Generator().manual_seed(0)
    pools = [torch.from_numpy(R.pack(*R.quantise(torch.randn(PAGES, 16, H, D, generator=g).numpy()), bool(i))).cuda() for i in (0, 1)]
    ids = torch.randperm(PAGES, generator=g).to(torch.int32).cuda()
    last = END // 16 + 1
    table = torch.full((1, 1 << 27), -1, dtype=torch.int32, device="cuda")
    table[0, last - PAGES:last] = ids
    far = pkv.PagedKVCache([pools[0].clone()], [pools[1].clone()], table)
    near = pkv.PagedKVCache([pools[0].clone()], [pools[1].clone()], ids.view(1, -1))
    yield far, near, (last - PAGES) * 16
    del far, table


@pytest.mark.parametrize("max_kv", [1000, 1 << 31])
@pytest.mark.parametrize("q_heads,q_len,window,causal", [(2, 1, 300, False), (8, 1, 700, True), (16, 9, 500, True), (64, 4, 333, True), (64, 40, 600, False)])
@pytest.mark.parametrize("back", [0, 1, 15, 20])
def test_attention(pkv, caches, max_kv, q_heads, q_len, window, causal, back):
    far, near, shift = caches
    g = torch.Generator().manual_seed(q_heads)
    q = torch.randn(q_len, q_heads, D, generator=g).bfloat16().cuda()
    got = []
    for cache, end in ((far, END - back), (near, END - back - shift)):
        si = torch.tensor([[0, q_len, 0, end]] + [[0, 0, 0, 0]] * 40, dtype=torch.int32, device="cuda")
        for flags in (0, pkv.FLAG_PDL):
            out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
            pkv.attend_varlen(cache, 0, q, si, out, err, q_len, max_kv, D ** -0.5, causal, window, lse=lse, flags=flags)
            assert int(err.item()) == 0 and bool(out.isfinite().all())
            got.append((out, lse))
    assert all(torch.equal(a, b) for o in got[1:] for a, b in zip(got[0], o))


@pytest.mark.parametrize("q_len,back", [(1, 0), (5, 3), (100, 0), (100, 7)])
def test_append(pkv, caches, q_len, back):
    far, near, shift = caches
    g = torch.Generator().manual_seed(q_len)
    q, kn, vn = [torch.randn(q_len, h, D, generator=g).bfloat16().cuda() for h in (4, H, H)]
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda")
    pos = torch.arange(END - back - q_len, END - back, dtype=torch.int32, device="cuda")
    q2, err = q.clone(), pkv.new_err_flags()
    for cache, end, positions, rows in ((far, END - back, None, q), (near, END - back - shift, pos, q2)):
        si = torch.tensor([[0, q_len, 0, end]], dtype=torch.int32, device="cuda")
        pkv.norm_rope_append(cache, 0, rope, rows, kn, vn, si, None, err, positions=positions)
    assert int(err.item()) == 0 and torch.equal(q, q2)
    assert torch.equal(far.k[0], near.k[0]) and torch.equal(far.v[0], near.v[0])
    si = torch.tensor([[0, q_len, 0, END + 1]], dtype=torch.int32, device="cuda")
    pkv.norm_rope_append(far, 0, rope, q, kn, vn, si, None, err)
    assert int(err.item()) == 1 and torch.equal(q, q2) and torch.equal(far.k[0], near.k[0])
