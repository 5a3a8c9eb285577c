"""The 8-bit cache on the GPU: the append bit for bit against the format's
definition, attention against the fp64 oracle over the stored values.

Tolerances of attention are those of the 4-bit cache (test_gpu_fp4.py, `check`):
scores are fp32 sums of exact products there and here, and weights are rounded to
fp16.  Here it is the weight times its page's V scale that is rounded, 2^-11 of itself or
2^-25 of the unit in which the row's largest such product is at least 2^7 over a scale 2^e
with 448 * 2^e at most twice the largest |v|: n 2^-25 vmax covers n * 2^-32 * 2 vmax.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import oracle as O
from tests import fp8_ref as R
from tests import gpu_util as U
from tests.test_gpu_fp4 import BIG, attend, check, shares, with_empty_segments

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


class Fp8:
    """A bf16 workload's pools in 8 bits: bytes on the host, and the cache on the device."""

    def __init__(self, pkv, w, garbage=True, first_valid=None, kscale=4.0, spread=0.0):
        self.w, self.bytes = w, []
        r = np.random.default_rng(7)
        for t, sc in ((w.k[0], kscale), (w.v[0], 1.0)):
            x = t.float().double().numpy()
            dead = np.isnan(x).any(-1).any(-1)  # [blocks, 16]: slots no segment reads
            x = np.nan_to_num(x, nan=0.0) * sc
            if spread:   # pages far apart in size
                x *= 2.0 ** r.integers(-spread, spread + 1, (x.shape[0], 1, x.shape[2], 1)).astype(float)
            b = R.exponent(np.abs(x).max((1, 3)))
            c = R.codes_of(x, b[:, None, :, None])
            m = np.zeros(b.shape, np.int64)
            if garbage:  # dead slots hold any codes, NaN ones among them; dead pages any scale and mask
                c[dead] = r.integers(0, 256, c[dead].shape)
                gone = dead.all(1)
                b[gone], m[gone] = r.integers(0, 256, b[gone].shape), r.integers(0, 65536, m[gone].shape)
            self.bytes.append(R.pack(c, b, m))
        self.guards, pools = [], []
        for b in self.bytes:
            buf = torch.full((b.size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
            view = buf[4096:4096 + b.size].view(b.shape)
            view.copy_(torch.from_numpy(b))
            self.guards.append(buf)
            pools.append(view.view(torch.float8_e4m3fn))
        fv = None if first_valid is None else torch.as_tensor(first_valid, dtype=torch.int32).cuda()
        self.cache = pkv.PagedKVCache([pools[0]], [pools[1]], w.block_table.cuda(), ring_rows=w.ring_rows, bucket=w.bucket, first_valid=fv)
        self.first_valid = first_valid

    def check_guards(self):
        for b in self.guards:
            assert bool((b[:4096] == 0x5A).all()) and bool((b[-4096:] == 0x5A).all()), "write outside a pool"

    def host(self, i):
        return (self.cache.k if i == 0 else self.cache.v)[0].view(torch.uint8).cpu().numpy()

    def ref(self, q, causal, window):
        w = self.w
        k, v = [np.nan_to_num(R.pool_values(self.host(i)), nan=0.0) for i in (0, 1)]
        live = np.zeros(k.shape[:2], bool)   # what no segment reads counts for nothing in a tolerance
        for _, _, col, kend in w.seq_info.tolist():
            span = min(w.ring_rows or kend, w.block_table.shape[1] * 16)
            at = np.arange(max(span, 0))
            blk = w.block_table.numpy()[col, at // 16]
            ok = (blk >= 0) & (blk < len(k))
            live[blk[ok], at[ok] % 16] = True
        k, v = [np.where(live[..., None, None], x, 0.0) for x in (k, v)]
        out, lse, err = O.attend(U.f64(q), k, v, w.block_table.numpy(), w.seq_info.numpy(), w.scale, causal=causal, window=window,
                                 ring_rows=w.ring_rows, first_valid=self.first_valid)
        return out, lse, err, k, v


def run_append(pkv, f, kn, vn, si=None, outs=True, **kw):
    w, err = f.w, pkv.new_err_flags()
    kn, vn = kn.cuda(), vn.cuda()
    ko, vo = torch.full_like(kn, 9), torch.full_like(vn, 9)
    pkv.norm_rope_append(f.cache, 0, None, None, kn, vn, (w.seq_info if si is None else si).cuda(), None, err, window=w.window,
                         k_out=ko if outs else None, v_out=vo if outs else None, **kw)
    torch.cuda.synchronize()
    f.check_guards()
    return ko, vo, int(err.item())


def check_append(f, before, kn, vn, ko, vo, si=None):
    """The pools are what the definition makes of `before`, bit for bit, and the rows out what they hold."""
    w = f.w
    for i, (x, got) in enumerate(((kn, ko), (vn, vo))):
        want = before[i].copy()
        held = R.append(want, w.block_table.numpy(), w.seq_info if si is None else si, U.f64(x), w.ring_rows)
        assert f.host(i).tobytes() == want.tobytes(), "KV"[i]
        if got is not None:
            assert np.array_equal(U.f64(got), held, equal_nan=True)


def zeroed(pkv, w):
    """The same cache with empty pools."""
    f = Fp8(pkv, w, garbage=False)
    for i, p in enumerate((f.cache.k[0], f.cache.v[0])):
        p.view(torch.uint8).zero_()
        f.bytes[i] = np.zeros_like(f.bytes[i])
    return f


# ---------------------------------------------------------------- the append

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 3, 50])
def test_append_is_bit_exact(pkv, D, max_q):
    w = U.nan_tails(workloads.spec_verify(S=7, max_q=max_q, len_lo=max_q, len_hi=150, seed=D + max_q, q_heads=6, kv_heads=3, head_dim=D))
    w.k_new[0] *= torch.exp(2 * torch.randn(w.total_rows, 3, D)).bfloat16()
    f = Fp8(pkv, w)
    ko, vo, err = run_append(pkv, f, w.k_new[0], w.v_new[0])
    assert err == 0
    check_append(f, f.bytes, w.k_new[0], w.v_new[0], ko, vo)
    g, e = Fp8(pkv, w), pkv.new_err_flags()     # the plain entry point does the same
    pkv.append(g.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), e)
    assert torch.equal(g.cache.k[0].view(torch.uint8), f.cache.k[0].view(torch.uint8)) and torch.equal(
        g.cache.v[0].view(torch.uint8), f.cache.v[0].view(torch.uint8))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("steps", [[1] * 40, [7, 9, 16, 1, 1, 25, 5], [64], [15, 1, 1, 47]])
def test_append_step_by_step(pkv, D, steps):
    """A sequence that grows over its pages, its rows larger and smaller as it goes: scales grow and codes follow."""
    w = workloads.batched(S=1, max_len=64, lengths=[64], q_heads=2, kv_heads=2, head_dim=D)
    f = zeroed(pkv, w)
    g = torch.Generator().manual_seed(D)
    end = 0
    for n in steps:
        end += n
        kn, vn = [(torch.randn(n, 2, D, generator=g) * torch.exp2(torch.randint(-12, 13, (n, 2, 1), generator=g).float())).bfloat16() for _ in range(2)]
        w.seq_info = torch.tensor([[0, n, 0, end]], dtype=torch.int32)
        before = [f.host(0).copy(), f.host(1).copy()]
        ko, vo, err = run_append(pkv, f, kn, vn)
        assert err == 0
        check_append(f, before, kn, vn, ko, vo)


def test_append_special_values(pkv):
    D = 128
    w = workloads.batched(S=1, max_len=32, lengths=[32], q_heads=2, kv_heads=2, head_dim=D)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(32, 2, D, generator=g)
    x[0] = 0.0
    x[1, 0, 5] = float("nan")
    x[2, 0, 7], x[2, 0, 8] = float("inf"), float("-inf")      # saturates page 0 of head 0
    x[3, 1] = 1e-40                                            # bf16 subnormals
    x[4, 1, :] = -0.0
    x[17, 0] = 448.0
    x[18, 0, 3] = 464.0                                        # 448 and just above: the next scale
    x[20, 1, :] = float("nan")
    x[21, 1, 4] = 3.3e38
    for order in ([32], [1] * 32, [2, 1, 29]):
        f, at = zeroed(pkv, w), 0
        for n in order:
            rows = x[at:at + n].bfloat16()
            at += n
            w.seq_info = torch.tensor([[0, n, 0, at]], dtype=torch.int32)
            before = [f.host(0).copy(), f.host(1).copy()]
            ko, vo, err = run_append(pkv, f, rows, -rows)
            assert err == 0
            check_append(f, before, rows, -rows, ko, vo)
        vals = R.pool_values(f.host(0))[w.block_table[0, :2].numpy()].reshape(32, 2, D)
        assert np.isnan(vals[1, 0]).all() and not np.isnan(vals[1, 1]).any() and np.isnan(vals[20, 1]).all()
        assert vals[2, 0, 7] == 448.0 * 2.0 ** 119 and vals[2, 0, 8] == -448.0 * 2.0 ** 119
    # a page's first slot starts it afresh, NaN marks and all
    w.seq_info = torch.tensor([[0, 1, 0, 1]], dtype=torch.int32)
    before = [f.host(0).copy(), f.host(1).copy()]
    one = torch.full((1, 2, D), 0.5).bfloat16()
    ko, vo, err = run_append(pkv, f, one, one)
    check_append(f, before, one, one, ko, vo)
    assert (U.f64(ko) == 0.5).all()


def test_append_ring_and_bad_segments(pkv):
    w = workloads.long_context(S=3, kv_len=1000, window=100, ring_rows=128, q_heads=4, kv_heads=2, head_dim=64)
    g = torch.Generator().manual_seed(5)
    rows = 40
    w.q, w.k_new, w.v_new = [[(4 * torch.randn(rows, h, 64, generator=g)).bfloat16()] for h in (4, 2, 2)]
    w.block_table[1, 3] = -7
    # a step that wraps; one whose ring is too short; one on a bad page; one beyond the rows; an empty one
    w.seq_info = torch.tensor([[20, 20, 2, 1000], [0, 7, 0, 129], [7, 2, 1, 50], [39, 2, 0, 200], [9, 0, 1, 5]], dtype=torch.int32)
    w.window = 100
    f = Fp8(pkv, w, garbage=False)
    ko, vo, err = run_append(pkv, f, w.k_new[0], w.v_new[0])
    assert err == 1 | 8
    check_append(f, f.bytes, w.k_new[0], w.v_new[0], ko, vo, si=w.seq_info[:2])
    assert (ko[7:20] == 9).all() and (vo[7:20] == 9).all() and not (ko[20:] == 9).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kend", [1000, 1003, 77, 128])
def test_append_a_whole_ring(pkv, D, kend):
    """As many rows as the ring holds: its last new page is also its first one."""
    w = workloads.long_context(S=1, kv_len=kend, window=1, ring_rows=64, q_heads=3, kv_heads=3, head_dim=D)
    g = torch.Generator().manual_seed(kend)
    w.k_new, w.v_new = [[torch.randn(64, 3, D, generator=g).bfloat16()] for _ in range(2)]
    w.seq_info, w.window = torch.tensor([[0, 64, 0, kend]], dtype=torch.int32), 1
    f = Fp8(pkv, w)
    ko, vo, err = run_append(pkv, f, w.k_new[0], w.v_new[0])
    assert err == 0
    check_append(f, f.bytes, w.k_new[0], w.v_new[0], ko, vo)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("table", [
    [[0, 7, 0, 20], [7, 1, 0, 21], [8, 2, 0, 23], [10, 20, 0, 43], [35, 5, 0, 58], [30, 5, 1, 5]],    # pieces of one sequence
    [[35, 5, 0, 58], [10, 20, 0, 43], [30, 5, 1, 5], [8, 2, 0, 23], [0, 7, 0, 20], [7, 1, 0, 21]],    # in another order
    [[0, 7, 0, 20], [20, 9, 1, 30], [0, 7, 0, 20], [20, 9, 1, 30], [20, 9, 1, 30]],                   # a padded batch
    [[0, 7, 0, 20], [9, 3, 0, 18], [30, 2, 0, 20]],                                                   # rows for slots that others write too
    [[0, 7, 0, 20]] + [[0, 3, 9, 20], [5, 0, 0, 21]] * 40 + [[10, 3, 0, 23]],                         # refused and empty ones between, more than a warp has lanes
])
def test_append_segments_that_share_a_page(pkv, D, table):
    w = workloads.batched(S=2, max_len=64, lengths=[64, 64], q_heads=2, kv_heads=2, head_dim=D)
    g = torch.Generator().manual_seed(D)
    kn, vn = [(torch.randn(40, 2, D, generator=g) * torch.exp2(torch.randint(-5, 6, (40, 2, 1), generator=g).float())).bfloat16() for _ in range(2)]
    w.seq_info = torch.tensor(table, dtype=torch.int32)
    valid = [s for s in table if s[2] < 2]
    twice = len({(c, k - i) for _, n, c, k in valid for i in range(n)}) < sum(n for _, n, _, _ in valid)
    for _ in range(3):
        f = Fp8(pkv, w)
        ko, vo, err = run_append(pkv, f, kn, vn)
        assert err == (1 if len(valid) < len(table) else 0)
        check_append(f, f.bytes, kn, vn, None if twice else ko, None if twice else vo, si=valid)


def test_append_piece_on_a_bad_page_does_not_own_it(pkv):
    """A segment refused for a bad page leaves its good ones to the segments after it."""
    w = workloads.batched(S=1, max_len=64, lengths=[64], q_heads=2, kv_heads=2, head_dim=64)
    w.block_table[0, 2] = 4000
    kn, vn = [torch.randn(30, 2, 64).bfloat16() for _ in range(2)]
    w.seq_info = torch.tensor([[0, 20, 0, 40], [20, 6, 0, 26]], dtype=torch.int32)
    f = Fp8(pkv, w)
    ko, vo, err = run_append(pkv, f, kn, vn)
    assert err == 8 and (ko[:20] == 9).all()
    check_append(f, f.bytes, kn, vn, ko, vo, si=w.seq_info[1:])


@pytest.mark.parametrize("D,rot,interleaved,norm", [(64, 64, False, True), (128, 128, False, True), (128, 64, True, False), (256, 256, False, True),
                                                    (128, 44, False, True), (64, 10, False, False), (256, 128, True, True), (128, 0, False, True)])
def test_norm_rope_into_fp8(pkv, D, rot, interleaved, norm):
    """The fused call stores what norm_rope's bf16 rows are held as; q comes out as norm_rope's, bit for bit."""
    w = workloads.spec_verify(S=4, max_q=20, len_lo=20, len_hi=90, seed=1, q_heads=8, kv_heads=2, head_dim=D)
    f = Fp8(pkv, w)
    freq, m = pkv.rope_inv_freq(rot, scaling="yarn", factor=8.0, trained_len=32) if rot else (None, 1.0)
    wq, wk = [(1 + 0.2 * torch.randn(D)).bfloat16().cuda() if norm else None for _ in range(2)]
    rope = pkv.Rope(freq, interleaved, mscale=m, q_weight=wq, k_weight=wk, device="cuda")
    err = pkv.new_err_flags()
    q, kn, vn, si = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda()
    qo, ko, vo = torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
    pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, si, qo, err, k_out=ko, v_out=vo)
    pos = np.concatenate([np.arange(k - n, k) for _, n, _, k in w.seq_info.tolist()]).astype(np.int32)
    q2, k2 = q.clone(), kn.clone()
    pkv.norm_rope(rope, q2, k2, torch.from_numpy(pos).cuda())
    assert int(err.item()) == 0 and torch.equal(q2, qo)
    check_append(f, f.bytes, k2, vn, ko, vo)
    # in place, from a projection's output, with given positions and several axes
    if rot >= 44:
        axes = pkv.rope_axes((rot // 2 - 2 * (rot // 8), rot // 8, rot // 8), True)
        rope = pkv.Rope(freq, interleaved, mscale=m, q_weight=wq, k_weight=wk, device="cuda", axes=axes)
        p3 = torch.randint(0, 1 << 20, (w.total_rows, 3), dtype=torch.int32, device="cuda")
        qkv = torch.cat([q, kn, vn, torch.ones_like(vn)], 1)
        a, b, c = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:12]
        q2, k2 = q.clone(), kn.clone()
        pkv.norm_rope(rope, q2, k2, p3)
        g = Fp8(pkv, w)
        pkv.norm_rope_append(g.cache, 0, rope, a, b, c, si, None, err, positions=p3, k_out=b, v_out=c)
        assert int(err.item()) == 0 and torch.equal(a, q2) and (qkv[:, 12:] == 1).all()
        check_append(g, g.bytes, k2, vn, b, c)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_single_rows_beside_empty_slots(pkv, D):
    """A page's slots without a new row take no part, whatever a norm with eps 0 makes of nothing."""
    w = workloads.batched(S=3, max_len=64, lengths=[64, 40, 17], q_heads=4, kv_heads=2, head_dim=D)
    f = Fp8(pkv, w)
    freq, _ = pkv.rope_inv_freq(D)
    wq, wk = [(1 + 0.2 * torch.randn(D)).bfloat16().cuda() for _ in range(2)]
    rope = pkv.Rope(freq, q_weight=wq, k_weight=wk, eps=0.0, device="cuda")
    q, kn, vn, si, err = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), pkv.new_err_flags()
    qo, ko, vo = torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
    pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, si, qo, err, k_out=ko, v_out=vo)
    q2, k2 = q.clone(), kn.clone()
    pkv.norm_rope(rope, q2, k2, (w.seq_info[:, 3] - 1).cuda())
    assert int(err.item()) == 0 and torch.equal(q2, qo)
    check_append(f, f.bytes, k2, vn, ko, vo)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_many_rows(pkv, D):
    """Ragged prompts with gaps, a refused segment and a bad page among them."""
    w = workloads.batched(S=6, max_len=1024, lengths=[700, 300, 17, 900, 64, 333], q_heads=4, kv_heads=2, head_dim=D, seed=1)
    w.block_table[4, 1] = -3
    rows = 2300
    g = torch.Generator().manual_seed(3)
    kn, vn = [torch.randn(rows, 2, D, generator=g).bfloat16() for _ in range(2)]
    good = [[1000, 700, 0, 700], [5, 299, 1, 300], [400, 10, 2, 17], [1701, 500, 3, 900]]
    w.seq_info = torch.tensor(good + [[420, 40, 4, 64], [900, 50, 5, 40]], dtype=torch.int32)
    f = Fp8(pkv, w)
    ko, vo, err = run_append(pkv, f, kn, vn)
    assert err == 1 | 8
    check_append(f, f.bytes, kn, vn, ko, vo, si=good)


def test_to_contiguous_reads_back(pkv):
    for D in (64, 128, 256):
        cache = pkv.PagedKVCache.allocate(2, 3, D, 512, dtype=torch.float8_e4m3fn)
        n = 77
        kn, vn = [torch.randn(n, 3, D).bfloat16().cuda() for _ in range(2)]
        kn[5, 1, 3] = float("nan")
        si, err = torch.tensor([[0, n, 0, n]], dtype=torch.int32, device="cuda"), pkv.new_err_flags()
        ko, vo = torch.empty_like(kn), torch.empty_like(vn)
        pkv.norm_rope_append(cache, 1, None, None, kn, vn, si, None, err, k_out=ko, v_out=vo)
        for m in (n, 1, 16, 33):
            buf = torch.full((2, 3 * m * D + 16), 5.0, dtype=torch.bfloat16, device="cuda")
            a, b = [buf[i, :3 * m * D].view(3, m, D) for i in range(2)]
            pkv.to_contiguous(cache, 1, m, a, b)
            assert np.array_equal(U.f64(a), U.f64(ko[:m].transpose(0, 1)), equal_nan=True) and torch.equal(b, vo[:m].transpose(0, 1))
            assert (buf[:, 3 * m * D:] == 5).all()


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqused", [1, 2, 15, 16, 17, 300, 1000, 1024])
def test_one_token(pkv, D, seqused):
    w = U.nan_tails(workloads.sensenova(seqused, 1024, num_layers=1, seed=seqused, head_dim=D))
    f = Fp8(pkv, w)
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = attend(pkv, f, out_dtype=dt, max_kv=1024)
        assert err == 0
        check(f, out, lse)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 3), (7, 1), (8, 1), (12, 3), (9, 1), (16, 1), (40, 2), (33, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_groups(pkv, q_heads, kv_heads, D):
    w = U.nan_tails(workloads.batched(S=5, max_len=700, seed=q_heads, q_heads=q_heads, kv_heads=kv_heads, head_dim=D))
    f = Fp8(pkv, w)
    for kw in ({"max_kv": 700}, {"max_kv": BIG}):
        out, lse, err = attend(pkv, f, **kw)
        assert err == 0
        check(f, out, lse)


@pytest.mark.parametrize("num_splits", [0, 1, 2, 3, 5, 8, 13, 16])
def test_splits(pkv, num_splits):
    w = U.nan_tails(workloads.batched(S=3, max_len=5000, seed=1, lengths=[5000, 2049, 3]))
    f = Fp8(pkv, w)
    out, lse, err = attend(pkv, f, num_splits=num_splits)
    assert err == 0
    check(f, out, lse)
    again, lse2, _ = attend(pkv, f, num_splits=num_splits)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("max_q,q_heads", [(2, 8), (5, 16), (16, 64), (40, 16)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_kv", [None, BIG])
def test_wide_groups(pkv, max_q, q_heads, causal, D, max_kv):
    w = U.nan_tails(workloads.spec_verify(S=5, max_q=max_q, len_lo=max_q, len_hi=900, seed=max_q, q_heads=q_heads, kv_heads=8 if q_heads > 8 else 2,
                                          head_dim=D, causal=causal))
    f = Fp8(pkv, w)
    out, lse, err = attend(pkv, f, max_kv=max_kv)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 899, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_heads", [16, 64])
def test_windows(pkv, window, causal, q_heads):
    w = workloads.spec_verify(S=6, max_q=9, len_lo=9, len_hi=900, seed=window, q_heads=q_heads, kv_heads=4, causal=causal)
    f = Fp8(pkv, w)
    out, lse, err = attend(pkv, f, window=window)
    assert err == 0
    check(f, out, lse, window=window)


@pytest.mark.parametrize("D,window,ring,kv", [(128, 100, 112, 1000), (64, 33, 64, 5000), (256, 512, 512, 3001)])
@pytest.mark.parametrize("q_heads", [8, 80])
def test_rings(pkv, D, window, ring, kv, q_heads):
    w = workloads.long_context(S=3, kv_len=kv, window=window, ring_rows=ring, q_heads=q_heads, kv_heads=2, head_dim=D)
    f = Fp8(pkv, w, garbage=False)
    out, lse, err = attend(pkv, f)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("max_q,q_heads,window", [(1, 8, 0), (12, 32, 0), (12, 32, 40)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("max_kv", [None, BIG])
def test_left_padding(pkv, max_q, q_heads, window, causal, max_kv):
    w = workloads.spec_verify(S=5, max_q=max_q, len_lo=60, len_hi=400, seed=3, q_heads=q_heads, kv_heads=4, causal=causal)
    ends = w.seq_info[:, 3].tolist()
    fv = [0, 17, ends[2] - 1, ends[3] + 5, max(ends[4] - max_q // 2 - 1, 0)]
    f = Fp8(pkv, w, first_valid=np.array(fv, np.int32))
    out, lse, err = attend(pkv, f, window=window, max_kv=max_kv)
    assert err == 0
    check(f, out, lse, window=window)


def test_uncovered_empty_and_overlapping_rows(pkv):
    w = workloads.batched(S=3, max_len=100, seed=2, q_heads=8, kv_heads=2)
    w.q = [torch.randn(10, 8, 128).bfloat16()]
    w.seq_info = torch.tensor([[7, 1, 0, 40], [2, 3, 1, 30], [5, 0, 2, 9]], dtype=torch.int32)
    w.block_table[0, :7], w.block_table[1, :7] = torch.arange(7), torch.arange(7)
    w.max_q_len = 3
    f = Fp8(pkv, w)
    for max_kv in (None, BIG):
        out, lse, err = attend(pkv, f, causal=True, max_kv=max_kv)
        assert err == 0
        check(f, out, lse, causal=True)
        dead = [0, 1, 5, 6, 8, 9]
        assert (out[dead] == 0).all() and torch.isinf(lse[dead]).all()
    w.seq_info = torch.tensor([[0, 3, 0, 40], [2, 3, 1, 30]], dtype=torch.int32)
    assert attend(pkv, f, causal=True)[2] == 32
    w.seq_info = torch.zeros(0, 4, dtype=torch.int32)
    out, lse, err = attend(pkv, f, max_q=1)
    assert err == 0 and (out == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("seg,bit", [((2, 1, 9, 5), 1), ((-1, 2, 0, 9), 1), ((2, 9, 0, 9), 1), ((2, 3, 0, 2), 1), ((2, 1, 0, 4096), 2),
                                     ((2, 2, 1, 33), 8), ((2, 2, 1, 690), 8), ((2, 4, 0, 9), 16)])
def test_bad_segments_read_zero(pkv, seg, bit):
    w = workloads.batched(S=2, max_len=700, seed=4, lengths=[700, 690], q_heads=16, kv_heads=2)
    w.block_table[1, 1] = 4000
    w.q = [torch.randn(6, 16, 128).bfloat16()]
    f = Fp8(pkv, w)
    for kw in ({"num_splits": 0}, {"num_splits": 1}, {"num_splits": 4}, {"max_kv": BIG}):
        w.seq_info = torch.tensor([seg, [0, 2, 0, 600]], dtype=torch.int32)
        out, lse, err = attend(pkv, f, causal=True, max_q=3, **kw)
        assert err == bit
        assert (out[2:] == 0).all() and torch.isinf(lse[2:]).all()
        w.seq_info = w.seq_info[1:]
        check(f, out, lse, causal=True, rows=np.arange(6) < 2)


@pytest.mark.parametrize("q_heads", [8, 64])
@pytest.mark.parametrize("max_kv", [None, BIG])
def test_nan_reaches_only_rows_that_see_it(pkv, q_heads, max_kv):
    w = workloads.spec_verify(S=1, max_q=8, len_lo=200, len_hi=200, seed=6, q_heads=q_heads, kv_heads=2)
    w.seq_info = torch.tensor([[0, 8, 0, 200]], dtype=torch.int32)
    w.q = [torch.randn(8, q_heads, 128).bfloat16()]
    f = Fp8(pkv, w)
    half = q_heads // 2
    for tok in (197, 192, 40, 199):                 # inside the step, its first, one that every row sees, the last
        page = int(w.block_table[0, tok // 16])
        see = np.arange(192, 200) >= tok
        for which, pool in ((0, f.cache.k[0]), (1, f.cache.v[0])):
            raw, keep = pool.view(torch.uint8), pool.view(torch.uint8).clone()
            bit = 1 << tok % 16
            raw[page, 1, 16 * 128 + 2] = bit & 255   # kv head 1
            raw[page, 1, 16 * 128 + 3] = bit >> 8
            out, lse, err = attend(pkv, f, causal=True, max_kv=max_kv)
            o, l = out.isnan().cpu().numpy(), lse.isnan().cpu().numpy()
            want = np.zeros((8, q_heads, 128), bool)
            want[see, half:] = True
            assert err == 0 and (o == want).all()
            assert (l == (want[..., 0] if which == 0 else False)).all()
            raw.copy_(keep)
    q = w.q[0].clone()
    q[3, 2, 7] = float("nan")
    out, lse, _ = attend(pkv, f, q=q, causal=True, max_kv=max_kv)
    assert out[3, 2].isnan().all() and lse[3, 2].isnan() and int(out.isnan().any(-1).sum()) == 1


@pytest.mark.parametrize("q_heads,max_q", [(8, 1), (16, 1), (32, 5), (64, 9)])
@pytest.mark.parametrize("spread", [3, 9])
@pytest.mark.parametrize("max_kv", [None, BIG])
def test_pages_of_different_scales(pkv, q_heads, max_q, spread, max_kv):
    """K and V pages up to 2^18 apart: a large V scale that comes late moves what was summed before it.

    vmax in the tolerance is that of the largest page, which is what the weights' rounding counts against."""
    w = workloads.spec_verify(S=4, max_q=max_q, len_lo=300, len_hi=700, seed=max_q, q_heads=q_heads, kv_heads=2)
    f = Fp8(pkv, w, kscale=2.0 ** -spread, spread=spread)
    out, lse, err = attend(pkv, f, max_kv=max_kv)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("q_heads", [4, 64])
@pytest.mark.parametrize("max_kv", [None, BIG])
def test_small_pages_behind_a_large_one(pkv, q_heads, max_kv):
    """Weights that go to pages of small V values are not lost behind a page of large ones that nobody looks at.

    The rows look at one key each, in a page 2^-12 as large as the page before it: what the
    large page adds is below e^-60 of it, so the row is that key's V but for 2^-11 of it, and half a step of bf16."""
    D = 128
    w = workloads.batched(S=1, max_len=64, lengths=[64], q_heads=q_heads, kv_heads=2, head_dim=D)
    f = zeroed(pkv, w)
    k, v = torch.zeros(64, 2, D), torch.randn(64, 2, D)
    k[:, :, 0] = -64.0
    k[37, :, 0] = 64.0
    v[:32] *= 2.0 ** 12
    w.seq_info = torch.tensor([[0, 64, 0, 64]], dtype=torch.int32)
    _, vo, err = run_append(pkv, f, k.bfloat16(), v.bfloat16())
    q = torch.zeros(1, q_heads, D)
    q[..., 0] = D ** 0.5
    w.seq_info = torch.tensor([[0, 1, 0, 64]], dtype=torch.int32)
    out, lse, err = attend(pkv, f, q=q.bfloat16(), max_q=1, max_kv=max_kv)
    want = vo[37].repeat_interleave(q_heads // 2, 0).float()
    assert err == 0 and bool(((out[0] - want).abs() <= 2.0 ** -10 * want.abs() + 2.0 ** -30).all())


def test_query_magnitudes(pkv):
    w = workloads.batched(S=4, max_len=300, seed=5, q_heads=8, kv_heads=2)
    f = Fp8(pkv, w)
    base = w.q[0].clone()

    def go(q, scale, max_kv=300):
        out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
        pkv.attend_varlen(f.cache, 0, q.cuda(), w.seq_info.cuda(), out, err, 1, max_kv, scale, lse=lse)
        assert int(err.item()) == 0
        return out, lse

    for max_kv in (300, BIG):
        out, lse = go(base, w.scale, max_kv)
        for e in (-100, -40, 40, 100):
            got, l2 = go((base.float() * 2.0 ** e).bfloat16(), w.scale * 2.0 ** -e, max_kv)
            assert torch.equal(got, out) and torch.equal(l2, lse)
        got, l2 = go(-base, -w.scale, max_kv)
        assert torch.allclose(got, out, rtol=0, atol=1e-6) and torch.allclose(l2, lse, rtol=1e-6)
        got, l2 = go(base, 0.0, max_kv)
        for s, (_, _, _, kend) in enumerate(w.seq_info.tolist()):
            assert torch.allclose(l2[s], torch.full_like(l2[s], float(np.log(kend))), rtol=1e-5)


def test_long_cache_offsets(pkv):
    """A pool whose bytes pass 2^32: block ids far into it are read and written where they are."""
    D, H = 256, 8
    blocks = (1 << 32) // ((16 * D + 16) * H) + 64
    pools = [torch.zeros(blocks, H, 16 * D + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    bt = torch.tensor([[blocks - 1, 3, blocks - 2]], dtype=torch.int32, device="cuda")
    cache = pkv.PagedKVCache([pools[0]], [pools[1]], bt)
    g = torch.Generator().manual_seed(0)
    kn, vn = [torch.randn(40, H, D, generator=g).bfloat16().cuda() for _ in range(2)]
    si = torch.tensor([[0, 40, 0, 40]], dtype=torch.int32, device="cuda")
    err = pkv.new_err_flags()
    ko, vo = torch.empty_like(kn), torch.empty_like(vn)
    pkv.norm_rope_append(cache, 0, None, None, kn, vn, si, None, err, k_out=ko, v_out=vo)
    q = torch.randn(40, H, D, generator=g).bfloat16().cuda()
    out = torch.empty(40, H, D, device="cuda")
    pkv.attend_varlen(cache, 0, q, si, out, err, 40, 40, D ** -0.5, causal=True)
    ref = torch.nn.functional.scaled_dot_product_attention(*[t.double().transpose(0, 1) for t in (q, ko, vo)], is_causal=True).transpose(0, 1)
    assert int(err.item()) == 0 and float((out.double() - ref).abs().max()) < float(vo.abs().max()) * 2.0 ** -10
    assert [int((p.view(torch.uint8).view(blocks, -1).count_nonzero(1) > 0).sum()) for p in pools] == [3, 3]


def test_append_attend_is_the_two_calls(pkv):
    w = U.nan_tails(workloads.spec_verify(S=4, max_q=5, len_lo=5, len_hi=300, seed=9, q_heads=16, kv_heads=4))
    q, kn, vn, si = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda()
    res = []
    for fn in ("two", "append_attend", "append_attend_noalloc"):
        f = Fp8(pkv, w)
        out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
        if fn == "two":
            pkv.append(f.cache, 0, kn, vn, si, err)
            pkv.attend_varlen(f.cache, 0, q, si, out, err, 5, 300, w.scale, causal=True, lse=lse)
        else:
            getattr(pkv, fn)(f.cache, 0, q, kn, vn, si, out, err, 5, 300, w.scale, causal=True, lse=lse)
        assert int(err.item()) == 0
        res.append((out, lse, f.cache.k[0].view(torch.uint8), f.cache.v[0].view(torch.uint8)))
        w.causal = True
        check(f, out, lse)
    for r in res[1:]:
        assert all(torch.equal(x, y) for x, y in zip(res[0], r))


@pytest.mark.parametrize("ring", [0, 64])
def test_steps_with_an_early_start(pkv, ring):
    """Decode steps whose attention is launched behind the append with an early start: in a ring, the append moves the scale of
    older tokens in its page, which the attention must not read before it is done."""
    S, D, n = 40, 128, 60
    w = workloads.long_context(S=S, kv_len=200, window=48 if ring else 0, ring_rows=ring, q_heads=8, kv_heads=2, head_dim=D)
    f = zeroed(pkv, w)
    g = torch.Generator().manual_seed(ring)
    err = pkv.new_err_flags()
    kn, vn = [(torch.randn(n, S, 2, D, generator=g) * torch.exp2(torch.arange(n).float() / 4)[:, None, None, None]).bfloat16().cuda() for _ in range(2)]
    q = (0.01 * torch.randn(n, S, 8, D, generator=g)).bfloat16().cuda()
    got = [torch.empty(n, S, 8, D, device="cuda") for _ in range(2)]
    for i, flags in enumerate((0, pkv.FLAG_PDL)):
        for p in (f.cache.k[0], f.cache.v[0]):
            p.view(torch.uint8).zero_()
        si = torch.tensor([[s, 1, s, 1] for s in range(S)], dtype=torch.int32, device="cuda")
        for t in range(n):
            pkv.append(f.cache, 0, kn[t], vn[t], si, err, window=w.window)
            pkv.attend_varlen(f.cache, 0, q[t], si, got[i][t], err, 1, 200, w.scale, causal=True, window=w.window, flags=flags)
            pkv.advance(si)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
    assert torch.equal(got[0], got[1])


def test_side_stream_and_graph(pkv):
    """Captured on a side stream and replayed at other lengths."""
    w = workloads.batched(S=3, max_len=600, seed=3, lengths=[600, 77, 350], q_heads=8, kv_heads=2)
    f = Fp8(pkv, w)
    q, kn, vn = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda()
    si, err = w.seq_info.cuda(), pkv.new_err_flags()
    out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
    freq, _ = pkv.rope_inv_freq(128)
    rope, qo = pkv.Rope(freq, device="cuda"), torch.empty_like(q)

    def step():
        pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, si, qo, err)
        pkv.attend_varlen(f.cache, 0, qo, si, out, err, 1, 600, w.scale, lse=lse, flags=pkv.FLAG_PDL)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for lens in ([600, 77, 350], [1, 16, 17], [33, 64, 349]):
        w.seq_info[:, 3] = torch.tensor(lens, dtype=torch.int32)
        si.copy_(w.seq_info)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], out) and torch.equal(got[1], lse) and int(err.item()) == 0
        check(f, out, lse, q=qo.cpu())


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("rows", [1023, 1024, 2600])
@pytest.mark.parametrize("in_place", [False, True])
def test_queries_of_long_steps(pkv, D, rows, in_place):
    """The queries of many rows: as norm_rope turns them; rows of no segment and of refused ones stay as they were."""
    g = torch.Generator().manual_seed(rows)
    ql = [1, 700, 0, 33, rows - 764, 20]
    w = workloads.batched(S=6, max_len=2000, lengths=[n + 5 for n in ql], q_heads=4, kv_heads=1, head_dim=D)
    q0 = [sum(ql[:i]) for i in range(6)]
    w.seq_info = torch.tensor([[a, n, i, n + 5] for i, (a, n) in enumerate(zip(q0, ql))], dtype=torch.int32)
    w.seq_info[3, 2] = 6          # no such sequence
    w.block_table[5, 1] = 1 << 20   # no such page
    valid = [s for i, s in enumerate(w.seq_info.tolist()) if i not in (3, 5)]
    total = rows                  # the last ten belong to none
    kn, vn = [torch.randn(total, 1, D, generator=g).bfloat16() for _ in range(2)]
    q = torch.randn(total, 4, D, generator=g).bfloat16().cuda()
    wq, wk = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)]
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], q_weight=wq, k_weight=wk, device="cuda")
    f, err = Fp8(pkv, w), pkv.new_err_flags()
    pos, new = np.zeros(total, np.int32), np.zeros(total, bool)
    for a, n, _, kend in valid:
        pos[a:a + n], new[a:a + n] = np.arange(kend - n, kend), True
    q2, k2 = q.clone(), kn.cuda()
    pkv.norm_rope(rope, q2, k2, torch.from_numpy(pos).cuda())
    new = torch.from_numpy(new).cuda()
    qo = q.clone() if in_place else torch.full_like(q, 9)
    want = torch.where(new[:, None, None], q2, qo)
    ko, vo = torch.full_like(k2, 9), torch.full_like(k2, 9)
    pkv.norm_rope_append(f.cache, 0, rope, qo if in_place else q, kn.cuda(), vn.cuda(), w.seq_info.cuda(), None if in_place else qo, err, k_out=ko, v_out=vo)
    torch.cuda.synchronize()
    assert int(err.item()) == 1 | 8 and torch.equal(qo, want)
    f.check_guards()
    check_append(f, f.bytes, k2, vn, ko, vo, si=valid)


@pytest.mark.parametrize("with_rope", [False, True])
@pytest.mark.parametrize("S", [1, 6])
def test_decode_step(pkv, with_rope, S):
    """A captured DecodeStep over an 8-bit cache, replayed as its sequences grow."""
    from paged_kv_decode_13_gb300.graph import DecodeGraphRunner, DecodeStep
    L, Hq, Hkv, D = 2, 8, 2, 128
    pools = [[torch.zeros(S * 8, Hkv, 16 * D + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(L)] for _ in range(2)]
    table = torch.randperm(S * 8, generator=torch.Generator().manual_seed(1)).int().view(S, 8)
    cache = pkv.PagedKVCache(pools[0], pools[1], table.cuda())
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], device="cuda") if with_rope else None
    step = DecodeStep(cache, Hq, rows=S, num_segments=S, max_kv=128, advance=True, rope=rope, with_lse=True, out_dtype=torch.bfloat16)
    run = DecodeGraphRunner(step)
    step.seq_info.copy_(torch.tensor([[s, 1, s, 1] for s in range(S)], dtype=torch.int32))
    g = torch.Generator().manual_seed(2)
    ref = [[torch.zeros(S * 8, Hkv, 16 * D + 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(L)] for _ in range(2)]
    plain = pkv.PagedKVCache(ref[0], ref[1], table.cuda())
    si, err = step.seq_info.clone(), pkv.new_err_flags()
    for t in range(40):
        for layer in range(L):
            for dst in (step.q, step.k_new, step.v_new):
                dst[layer].copy_((torch.randn(dst[layer].shape, generator=g) * 2.0 ** (t % 5)).bfloat16())
        run.step()
        for layer in range(L):
            q = step.q[layer].clone()
            pkv.norm_rope_append(plain, layer, rope, q, step.k_new[layer], step.v_new[layer], si, None, err)
            out, lse = torch.empty_like(q), torch.empty(S, Hq, device="cuda")
            pkv.attend_varlen(plain, layer, q, si, out, err, 1, 128, step.scale, lse=lse, workspace=step.ws)
            assert torch.equal(out, step.out[layer]) and torch.equal(lse, step.lse[layer])
        pkv.advance(si)
    assert int(err.item()) == 0 and int(step.err.item()) == 0 and torch.equal(si, step.seq_info)
    for a, b in zip(pools[0] + pools[1], ref[0] + ref[1]):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- equal shares

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [16], [17, 1, 5000], [2999, 0, 40, 2998, 1], [9000]])
def test_shares(pkv, D, lengths):
    w = U.nan_tails(workloads.batched(S=len(lengths), max_len=max(lengths), seed=D, lengths=lengths, q_heads=8, kv_heads=2, head_dim=D))
    w.seq_info[:, 1] = (w.seq_info[:, 3] > 0).int()
    f = Fp8(pkv, w)
    assert shares(pkv, f, 1)
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = attend(pkv, f, out_dtype=dt, max_kv=BIG)
        assert err == 0
        check(f, out, lse)
    again, lse2, _ = attend(pkv, f, out_dtype=dt, max_kv=BIG)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_shares_many_segments(pkv):
    S = 300
    lengths = torch.randint(0, 200, (S,), generator=torch.Generator().manual_seed(1)).tolist()
    w = workloads.batched(S=S, max_len=200, lengths=[max(n, 1) for n in lengths], q_heads=8, kv_heads=2)
    w.seq_info[:, 1] = (torch.tensor(lengths) > 0).int()
    f = Fp8(pkv, w)
    out, lse, err = attend(pkv, f, max_kv=BIG)
    assert err == 0
    check(f, out, lse)


def test_shares_with_empty_segments(pkv):
    w = with_empty_segments(workloads.batched(S=5, max_len=900, seed=3, q_heads=8, kv_heads=2), 7)
    f = Fp8(pkv, w)
    out, lse, err = attend(pkv, f, max_kv=BIG)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("q_heads,max_q", [(8, 1), (16, 4), (32, 4), (64, 9)])
@pytest.mark.parametrize("window", [1000, 3000])
@pytest.mark.parametrize("padded", [False, True])
def test_shares_with_windows(pkv, q_heads, max_q, window, padded):
    w = workloads.spec_verify(S=7, max_q=max_q, len_lo=max_q, len_hi=6000, seed=q_heads + window, q_heads=q_heads, kv_heads=8)
    ends = w.seq_info[:, 3].tolist()
    fv = np.array([0, 17, ends[2] - 1, ends[3] + 5, max(ends[4] - 5, 0), 3, 0], np.int32) if padded else None
    f = Fp8(pkv, w, first_valid=fv)
    with_empty_segments(w, 500)
    out, lse, err = attend(pkv, f, max_q=max_q, max_kv=BIG, window=window)
    assert err == 0
    check(f, out, lse, window=window)


@pytest.mark.parametrize("D,window,ring,kv", [(128, 3000, 3024, 5000), (64, 2000, 2000, 3000), (256, 2000, 2000, 3001)])
@pytest.mark.parametrize("q_heads", [8, 288])
def test_shares_with_rings(pkv, D, window, ring, kv, q_heads):
    w = workloads.long_context(S=3, kv_len=kv, window=window, ring_rows=ring, q_heads=q_heads, kv_heads=8, head_dim=D)
    f = Fp8(pkv, w, garbage=False, first_valid=np.array([0, kv - 100, kv + 5], np.int32))
    with_empty_segments(w, 500)
    out, lse, err = attend(pkv, f, max_q=1, max_kv=BIG, window=window)
    assert err == 0
    check(f, out, lse, window=window)
