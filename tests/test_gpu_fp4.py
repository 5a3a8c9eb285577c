"""The 4-bit cache on the GPU: the append bit for bit against the format's
definition, attention against the fp64 oracle over the stored values.

Tolerances of attention, from the arithmetic: a score is an fp32 sum of D
exact products, off by at most D 2^-24 sum|q k| scale =: d; a weight exp(x - m)
then by d relative, its exp2 and rounding to fp16 by 2^-11 (or 2^-25 absolute
below fp16's normal range, against a sum of weights of at least 1), and the
sum of weights by d again: |out - ref| <= vmax (2^-11 + n 2^-25 + 2 d + 2^-18),
plus half a step (2^-8 relative) where out is bf16.  lse: d + n 2^-24 + 2^-21 |lse|.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import oracle as O
from tests import fp4_ref as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


class Fp4:
    """A bf16 workload's pools in 4 bits: bytes on the host, and the cache on the device."""

    def __init__(self, pkv, w, garbage=True, first_valid=None, kscale=4.0):
        # the workload's K is N(0, 1) / sqrt(D): make scores spread, as real keys do
        self.w, self.bytes = w, []
        nan = [torch.isnan(t.float()).any(-1).any(-1).numpy() for t in (w.k[0], w.v[0])]
        for t, is_v, sc in ((w.k[0], False, kscale), (w.v[0], True, 1.0)):
            x = torch.nan_to_num(t.float(), nan=0.0).numpy() * sc
            c, s = R.quantise(x.astype(np.float64))
            if garbage:   # slots no segment reads: any bytes, NaN and infinite scales among them
                dead = nan[int(is_v)]
                r = np.random.default_rng(7)
                c[dead] = r.integers(0, 16, c[dead].shape)
                s[dead] = r.choice([0xFF, 0xF8, 0x80, 0xF9], s[dead].shape)
            self.bytes.append(R.pack(c, s, is_v))
        self.guards = []
        pools = []
        for b in self.bytes:
            buf = torch.full((b.size + 8192,), 0x5A, dtype=torch.uint8, device="cuda")
            view = buf[4096:4096 + b.size].view(b.shape)
            view.copy_(torch.from_numpy(b))
            self.guards.append(buf)
            pools.append(view)
        fv = None if first_valid is None else torch.as_tensor(first_valid, dtype=torch.int32).cuda()
        self.cache = pkv.PagedKVCache([pools[0]], [pools[1]], w.block_table.cuda(), ring_rows=w.ring_rows, bucket=w.bucket, first_valid=fv)
        self.first_valid = first_valid

    def check_guards(self):
        for b in self.guards:
            assert bool((b[:4096] == 0x5A).all()) and bool((b[-4096:] == 0x5A).all()), "write outside a pool"

    def oracle_bytes(self, ko, vo):
        """Codes and scales of both pools after the oracle's append of the rows ko, vo (quantised here)."""
        w, got, err = self.w, [], 0
        parts = [R.unpack(self.bytes[i], bool(i)) + R.quantise(U.f64(x)) for i, x in enumerate((ko, vo))]
        for part in (0, 1):
            kp, vp = parts[0][part].copy(), parts[1][part].copy()
            err |= O.append(kp, vp, w.block_table.numpy(), w.seq_info.numpy(), parts[0][2 + part], parts[1][2 + part],
                            ring_rows=w.ring_rows, window=w.window, causal=w.causal)
            got.append((kp, vp))
        return [R.pack(got[0][i], got[1][i], bool(i)) for i in (0, 1)], err

    def ref(self, q, causal, window):
        w = self.w
        k, v = [np.nan_to_num(R.pool_values(self.host(i), bool(i)), nan=0.0, posinf=0.0, neginf=0.0) for i in (0, 1)]
        out, lse, err = O.attend(U.f64(q), k, v, w.block_table.numpy(), w.seq_info.numpy(), w.scale, causal=causal, window=window,
                                 ring_rows=w.ring_rows, first_valid=self.first_valid)
        return out, lse, err, k, v

    def host(self, i):
        return (self.cache.k if i == 0 else self.cache.v)[0].cpu().numpy()


def attend(pkv, f, q=None, causal=None, window=None, out_dtype=torch.float32, num_splits=0, max_q=None, max_kv=None, flags=0):
    w = f.w
    q = (w.q[0] if q is None else q).cuda()
    buf = torch.full((q.numel() + 2048,), 5.0, dtype=out_dtype, device="cuda")
    out = buf[1024:1024 + q.numel()].view(q.shape)
    lse = torch.full(q.shape[:2], 3.0, device="cuda")
    err = pkv.new_err_flags()
    mk = max_kv or max(int(w.seq_info[:, 3].max()) if w.num_segments else 1, 1)
    pkv.attend_varlen(f.cache, 0, q, w.seq_info.cuda(), out, err, max_q or w.max_q_len, mk, w.scale, w.causal if causal is None else causal,
                      w.window if window is None else window, lse=lse, num_splits=num_splits, flags=flags)
    torch.cuda.synchronize()
    assert bool((buf[:1024] == 5).all()) and bool((buf[-1024:] == 5).all()), "write outside the output"
    f.check_guards()
    return out, lse, int(err.item())


def check(f, out, lse, q=None, causal=None, window=None, rows=None):
    w = f.w
    causal, window = w.causal if causal is None else causal, w.window if window is None else window
    q = w.q[0] if q is None else q
    ref, ref_lse, err, k, v = f.ref(q, causal, window)
    assert err == 0
    D, n = w.head_dim, int(w.seq_info[:, 3].max())
    vmax, kmax = np.abs(v).max(), np.abs(k).reshape(-1, D).sum(-1).max()
    d = D * 2.0 ** -24 * float(np.abs(U.f64(q)).max()) * kmax * w.scale
    tol = vmax * (2.0 ** -11 + n * 2.0 ** -25 + 2 * d + 2.0 ** -18)
    got = U.f64(out)
    rows = np.ones(len(got), bool) if rows is None else rows
    assert np.isfinite(got[rows]).all()
    lim = tol + (2.0 ** -8 * (np.abs(ref) + tol) if out.dtype == torch.bfloat16 else 0)
    worst = float((np.abs(got - ref) / lim)[rows].max())
    assert worst <= 1, f"{worst} times the tolerance"
    gl = U.f64(lse)[rows]
    el = ref_lse[rows]
    assert (np.isinf(gl) == np.isinf(el)).all()
    fin = np.isfinite(el)
    assert (np.abs(gl[fin] - el[fin]) <= d + n * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(el[fin]))).all()


# ---------------------------------------------------------------- the append

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 3, 50])
def test_append_is_bit_exact(pkv, D, max_q):
    w = U.nan_tails(workloads.spec_verify(S=7, max_q=max_q, len_lo=max_q, len_hi=150, seed=D + max_q, q_heads=6, kv_heads=3, head_dim=D))
    w.k_new[0] *= torch.exp(2 * torch.randn(w.total_rows, 3, D)).bfloat16()
    f = Fp4(pkv, w)
    err = pkv.new_err_flags()
    kn, vn = w.k_new[0].cuda(), w.v_new[0].cuda()
    ko, vo = torch.full_like(kn, 9), torch.full_like(vn, 9)
    pkv.norm_rope_append(f.cache, 0, None, None, kn, vn, w.seq_info.cuda(), None, err, k_out=ko, v_out=vo)
    want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
    assert e == 0 and int(err.item()) == 0
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    assert np.array_equal(U.f64(ko), R.values(*R.quantise(U.f64(kn)))) and np.array_equal(U.f64(vo), R.values(*R.quantise(U.f64(vn))))
    f.check_guards()
    # the plain entry point does the same
    g = Fp4(pkv, w)
    pkv.append(g.cache, 0, kn, vn, w.seq_info.cuda(), err)
    assert torch.equal(g.cache.k[0], f.cache.k[0]) and torch.equal(g.cache.v[0], f.cache.v[0])


def test_append_special_values(pkv):
    w = workloads.sensenova(40, 64, num_layers=1, q_heads=4, kv_heads=2)
    nan, inf = float("nan"), float("inf")
    for t in (w.k_new[0], w.v_new[0]):
        t[0, 0, 3], t[0, 0, 20], t[0, 0, 40], t[0, 1, 50] = nan, inf, -inf, 65000.0
        t[0, 0, 64:80], t[0, 0, 80:96], t[0, 0, 96:112], t[0, 0, 112:128] = 0.0, -0.0, 1e-5, 6e-5
        t[0, 1, 0:16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
        t[0, 1, 16:32] = torch.linspace(-1e-38, 1e-38, 16).bfloat16()
    f = Fp4(pkv, w)
    err = pkv.new_err_flags()
    pkv.append(f.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), err)
    want, _ = f.oracle_bytes(w.k_new[0], w.v_new[0])
    for i in (0, 1):
        a, b = R.unpack(f.host(i), bool(i)), R.unpack(want[i], bool(i))
        assert np.array_equal(a[1], b[1])
        live = np.repeat(b[1] != 0xFF, 16, -1)       # codes under a NaN scale mean nothing
        assert np.array_equal(a[0][live], b[0][live])


def test_append_ring_and_bad_segments(pkv):
    w = workloads.long_context(S=3, kv_len=1000, window=100, ring_rows=128, q_heads=4, kv_heads=2, head_dim=64)
    g = torch.Generator().manual_seed(5)
    rows = 40
    w.q, w.k_new, w.v_new = [[torch.randn(rows, h, 64, generator=g).bfloat16()] for h in (4, 2, 2)]
    w.block_table[1, 3] = -7
    # a step that wraps; one whose ring is too short; one on a bad page; one beyond the rows; an empty one
    w.seq_info = torch.tensor([[20, 20, 2, 1000], [0, 7, 0, 129], [7, 2, 1, 50], [39, 2, 0, 200], [9, 0, 1, 5]], dtype=torch.int32)
    f = Fp4(pkv, w)
    err = pkv.new_err_flags()
    kn, vn = w.k_new[0].cuda(), w.v_new[0].cuda()
    ko, vo = torch.full_like(kn, 9), torch.full_like(vn, 9)
    pkv.norm_rope_append(f.cache, 0, None, None, kn, vn, w.seq_info.cuda(), None, err, window=100, k_out=ko, v_out=vo)
    w.window = 100
    want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
    assert int(err.item()) == 1 | 8
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    assert (ko[7:20] == 9).all() and (vo[7:20] == 9).all() and not (ko[20:] == 9).all()


@pytest.mark.parametrize("D", [64, 128])
def test_norm_rope_into_fp4(pkv, D):
    """The fused call stores what norm_rope's bf16 rows quantise to."""
    w = workloads.spec_verify(S=4, max_q=20, len_lo=20, len_hi=90, seed=1, q_heads=8, kv_heads=2, head_dim=D)
    f = Fp4(pkv, w)
    freq, m = pkv.rope_inv_freq(D, scaling="yarn", factor=8.0, trained_len=32)
    wq, wk = [(1 + 0.2 * torch.randn(D)).bfloat16().cuda() for _ in range(2)]
    rope = pkv.Rope(freq, mscale=m, q_weight=wq, k_weight=wk, device="cuda")
    err = pkv.new_err_flags()
    q, kn, vn, si = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda()
    qo, ko, vo = torch.empty_like(q), torch.empty_like(kn), torch.empty_like(vn)
    pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, si, qo, err, k_out=ko, v_out=vo)
    pos = np.concatenate([np.arange(k - n, k) for _, n, _, k in w.seq_info.tolist()]).astype(np.int32)
    q2, k2 = q.clone(), kn.clone()
    pkv.norm_rope(rope, q2, k2, torch.from_numpy(pos).cuda())
    assert torch.equal(q2, qo) and int(err.item()) == 0
    want, e = f.oracle_bytes(k2.cpu(), w.v_new[0])
    assert e == 0
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    assert np.array_equal(U.f64(ko), R.values(*R.quantise(U.f64(k2))))


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("seqused", [1, 2, 15, 16, 17, 300, 1000, 1024])
def test_one_token(pkv, D, seqused):
    w = U.nan_tails(workloads.sensenova(seqused, 1024, num_layers=1, seed=seqused, head_dim=D))
    f = Fp4(pkv, w)
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = attend(pkv, f, out_dtype=dt, max_kv=1024)
        assert err == 0
        check(f, out, lse)


@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (3, 3), (7, 1), (8, 1), (12, 3), (9, 1), (16, 1), (40, 2), (33, 1)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_groups(pkv, q_heads, kv_heads, D):
    w = U.nan_tails(workloads.batched(S=5, max_len=700, seed=q_heads, q_heads=q_heads, kv_heads=kv_heads, head_dim=D))
    f = Fp4(pkv, w)
    out, lse, err = attend(pkv, f, max_kv=700)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("num_splits", [0, 1, 2, 3, 5, 8, 13, 16])
def test_splits(pkv, num_splits):
    w = U.nan_tails(workloads.batched(S=3, max_len=5000, seed=1, lengths=[5000, 2049, 3]))
    f = Fp4(pkv, w)
    out, lse, err = attend(pkv, f, num_splits=num_splits)
    assert err == 0
    check(f, out, lse)
    again, lse2, _ = attend(pkv, f, num_splits=num_splits)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("max_q,q_heads", [(2, 8), (5, 16), (16, 64), (40, 16)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_wide_groups(pkv, max_q, q_heads, causal, D):
    w = U.nan_tails(workloads.spec_verify(S=5, max_q=max_q, len_lo=max_q, len_hi=900, seed=max_q, q_heads=q_heads, kv_heads=8 if q_heads > 8 else 2,
                                          head_dim=D, causal=causal))
    f = Fp4(pkv, w)
    out, lse, err = attend(pkv, f)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 899, 5000])
@pytest.mark.parametrize("causal", [True, False])
def test_windows(pkv, window, causal):
    w = workloads.spec_verify(S=6, max_q=9, len_lo=9, len_hi=900, seed=window, q_heads=16, kv_heads=4, causal=causal)
    f = Fp4(pkv, w)
    out, lse, err = attend(pkv, f, window=window)
    assert err == 0
    check(f, out, lse, window=window)


@pytest.mark.parametrize("D,window,ring,kv", [(128, 100, 112, 1000), (64, 33, 64, 5000), (256, 512, 512, 3001)])
def test_rings(pkv, D, window, ring, kv):
    w = workloads.long_context(S=3, kv_len=kv, window=window, ring_rows=ring, q_heads=8, kv_heads=2, head_dim=D)
    f = Fp4(pkv, w, garbage=False)
    out, lse, err = attend(pkv, f)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("max_q,q_heads,window", [(1, 8, 0), (12, 32, 0), (12, 32, 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_left_padding(pkv, max_q, q_heads, window, causal):
    w = workloads.spec_verify(S=5, max_q=max_q, len_lo=60, len_hi=400, seed=3, q_heads=q_heads, kv_heads=4, causal=causal)
    ends = w.seq_info[:, 3].tolist()
    fv = [0, 17, ends[2] - 1, ends[3] + 5, max(ends[4] - max_q // 2 - 1, 0)]  # none, some, all but one, more than all, inside the step
    f = Fp4(pkv, w, first_valid=np.array(fv, np.int32))
    out, lse, err = attend(pkv, f, window=window)
    assert err == 0
    check(f, out, lse, window=window)


def test_uncovered_empty_and_overlapping_rows(pkv):
    w = workloads.batched(S=3, max_len=100, seed=2, q_heads=8, kv_heads=2)
    w.q = [torch.randn(10, 8, 128).bfloat16()]
    w.seq_info = torch.tensor([[7, 1, 0, 40], [2, 3, 1, 30], [5, 0, 2, 9]], dtype=torch.int32)
    w.block_table[0, :7], w.block_table[1, :7] = torch.arange(7), torch.arange(7)
    w.max_q_len = 3
    f = Fp4(pkv, w)
    out, lse, err = attend(pkv, f, causal=True)
    assert err == 0
    check(f, out, lse, causal=True)
    dead = [0, 1, 5, 6, 8, 9]
    assert (out[dead] == 0).all() and torch.isinf(lse[dead]).all()
    w.seq_info = torch.tensor([[0, 3, 0, 40], [2, 3, 1, 30]], dtype=torch.int32)
    _, _, err = attend(pkv, f, causal=True)
    assert err == 32
    w.seq_info = torch.zeros(0, 4, dtype=torch.int32)
    out, lse, err = attend(pkv, f, max_q=1)
    assert err == 0 and (out == 0).all() and torch.isinf(lse).all()


@pytest.mark.parametrize("seg,bit", [((2, 1, 9, 5), 1), ((-1, 2, 0, 9), 1), ((2, 9, 0, 9), 1), ((2, 3, 0, 2), 1), ((2, 1, 0, 4096), 2),
                                     ((2, 2, 1, 33), 8), ((2, 2, 1, 690), 8), ((2, 4, 0, 9), 16)])
def test_bad_segments_read_zero(pkv, seg, bit):
    w = workloads.batched(S=2, max_len=700, seed=4, lengths=[700, 690], q_heads=16, kv_heads=2)
    w.block_table[1, 1] = 4000
    w.q = [torch.randn(6, 16, 128).bfloat16()]
    f = Fp4(pkv, w)
    for splits in (0, 1, 4):
        w.seq_info = torch.tensor([seg, [0, 2, 0, 600]], dtype=torch.int32)
        out, lse, err = attend(pkv, f, causal=True, max_q=3, num_splits=splits)
        assert err == bit
        assert (out[2:] == 0).all() and torch.isinf(lse[2:]).all()
        w.seq_info = w.seq_info[1:]
        check(f, out, lse, causal=True, rows=np.arange(6) < 2)


def test_nan_reaches_only_rows_that_see_it(pkv):
    w = workloads.spec_verify(S=1, max_q=8, len_lo=200, len_hi=200, seed=6, q_heads=8, kv_heads=2)
    w.seq_info = torch.tensor([[0, 8, 0, 200]], dtype=torch.int32)
    w.q = [torch.randn(8, 8, 128).bfloat16()]
    f = Fp4(pkv, w)
    page, tok = int(w.block_table[0, 197 // 16]), 197 % 16
    for which, pool in ((0, f.cache.k[0]), (1, f.cache.v[0])):
        c, s = R.unpack(pool.cpu().numpy(), bool(which))
        keep = pool.clone()
        s[page, tok, 1, 2] = 0xFF                       # columns 32..47 of kv head 1
        pool.copy_(torch.from_numpy(R.pack(c, s, bool(which))))
        out, lse, err = attend(pkv, f, causal=True)
        o, l = out.isnan().cpu().numpy(), lse.isnan().cpu().numpy()
        see = np.arange(192, 200) >= 197
        want = np.zeros((8, 8, 128), bool)
        if which == 0:                                  # the whole row of the kv head's query heads
            want[see, 4:] = True
            assert (l[:, 4:] == see[:, None]).all() and not l[:, :4].any()
        else:
            want[see, 4:, 32:48] = True
            assert not l.any()
        assert (o == want).all()
        pool.copy_(keep)
    q = w.q[0].clone()
    q[3, 2, 7] = float("nan")
    out, lse, _ = attend(pkv, f, q=q, causal=True)
    assert out[3, 2].isnan().all() and lse[3, 2].isnan() and int(out.isnan().any(-1).sum()) == 1


def test_query_magnitudes(pkv):
    """Rows far below and above fp16's range score as they are."""
    w = workloads.batched(S=4, max_len=300, seed=5, q_heads=8, kv_heads=2)
    f = Fp4(pkv, w)
    base = w.q[0].clone()
    out, lse, _ = attend(pkv, f)
    for e in (-100, -40, 40, 100):
        q = (base.float() * 2.0 ** e).bfloat16()
        keep = w.seq_info
        got, l2, err = attend_scaled(pkv, f, q, w.scale * 2.0 ** -e)
        assert err == 0 and torch.equal(got, out) and torch.equal(l2, lse)


def attend_scaled(pkv, f, q, scale):
    w = f.w
    out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
    pkv.attend_varlen(f.cache, 0, q.cuda(), w.seq_info.cuda(), out, err, w.max_q_len, int(w.seq_info[:, 3].max()), scale, w.causal, w.window, lse=lse)
    return out, lse, int(err.item())


def test_long_cache_offsets(pkv):
    """A pool whose bytes pass 2^32: block ids far into it are read and written where they are."""
    D, H = 256, 8
    blocks = (1 << 32) // (9 * D * H) + 64
    pools = [torch.zeros(blocks, H, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
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
    n = [int((p.view(blocks, -1).count_nonzero(1) > 0).sum()) for p in pools]
    assert n == [3, 3]


def test_append_attend_is_the_two_calls(pkv):
    w = U.nan_tails(workloads.spec_verify(S=4, max_q=5, len_lo=5, len_hi=300, seed=9, q_heads=16, kv_heads=4))
    a, b = Fp4(pkv, w), Fp4(pkv, w)
    q, kn, vn, si = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda()
    res = []
    for f, fn in ((a, "two"), (b, "append_attend"), (Fp4(pkv, w), "append_attend_noalloc")):
        out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
        if fn == "two":
            pkv.append(f.cache, 0, kn, vn, si, err)
            pkv.attend_varlen(f.cache, 0, q, si, out, err, 5, 300, w.scale, causal=True, lse=lse)
        else:
            getattr(pkv, fn)(f.cache, 0, q, kn, vn, si, out, err, 5, 300, w.scale, causal=True, lse=lse)
        assert int(err.item()) == 0
        res.append((out, lse, f.cache.k[0], f.cache.v[0]))
    for r in res[1:]:
        assert all(torch.equal(x, y) for x, y in zip(res[0], r))
    w.causal = True
    check(a, res[0][0], res[0][1])


def test_rewind_on_fp4(pkv):
    w = workloads.batched(S=2, max_len=100, lengths=[100, 50], q_heads=4, kv_heads=2)
    f = Fp4(pkv, w)
    si, err = w.seq_info.cuda(), pkv.new_err_flags()
    pkv.rewind(f.cache, si, torch.tensor([3, 0], dtype=torch.int32, device="cuda"), err)
    pkv.advance(si)
    assert si[:, 3].tolist() == [98, 51] and int(err.item()) == 0


def test_side_stream_and_graph(pkv):
    """Captured on a side stream and replayed at other lengths; two graphs at once."""
    w = workloads.batched(S=3, max_len=600, seed=3, lengths=[600, 77, 350], q_heads=8, kv_heads=2)
    f = Fp4(pkv, w)
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


# ---------------------------------------------------------------- equal shares: launches whose bounds are large
#
# The launch bounds decide (max_kv is one), so a large max_kv runs small cases there.

BIG = 1 << 20


def shares(pkv, f, max_q):
    w = f.w
    return pkv.attend_workspace_bytes(f.cache, w.q_heads, w.num_segments, max_q, BIG) > 0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lengths", [[1], [16], [17, 1, 5000], [3000, 0, 40, 2999, 1], [9000]])
def test_shares(pkv, D, lengths):
    w = U.nan_tails(workloads.batched(S=len(lengths), max_len=max(lengths), seed=D, lengths=lengths, q_heads=8, kv_heads=2, head_dim=D))
    w.seq_info[:, 1] = (w.seq_info[:, 3] > 0).int()
    f = Fp4(pkv, w)
    assert shares(pkv, f, 1)
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = attend(pkv, f, out_dtype=dt, max_kv=BIG)
        assert err == 0
        check(f, out, lse)
    again, lse2, _ = attend(pkv, f, out_dtype=dt, max_kv=BIG)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_heads,kv_heads,max_q", [(1, 1, 1), (8, 1, 1), (12, 3, 2), (4, 4, 8), (7, 1, 1)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 33, 700])
def test_shares_groups_and_windows(pkv, q_heads, kv_heads, max_q, causal, window):
    w = U.nan_tails(workloads.spec_verify(S=9, max_q=max_q, len_lo=max_q, len_hi=2000, seed=q_heads, q_heads=q_heads, kv_heads=kv_heads, causal=causal))
    f = Fp4(pkv, w)
    assert shares(pkv, f, max_q)
    ws = pkv.new_workspace(f.cache, q_heads, 9, max_q, BIG)
    out, lse, err = torch.empty(w.q[0].shape, device="cuda"), torch.empty(w.q[0].shape[:2], device="cuda"), pkv.new_err_flags()
    buf = torch.full((ws.numel() + 4096,), 0xA5, dtype=torch.uint8, device="cuda")   # garbage in it, a guard behind it
    pkv.attend_varlen(f.cache, 0, w.q[0].cuda(), w.seq_info.cuda(), out, err, max_q, BIG, w.scale, causal, window, lse=lse, workspace=buf[:ws.numel()])
    assert int(err.item()) == 0 and bool((buf[ws.numel():] == 0xA5).all())
    check(f, out, lse, window=window)


def test_shares_many_segments(pkv):
    g = torch.Generator().manual_seed(1)
    lengths = torch.randint(1, 400, (512,), generator=g).tolist()
    w = workloads.batched(S=512, max_len=400, lengths=lengths, q_heads=2, kv_heads=1, head_dim=64)
    f = Fp4(pkv, w)
    assert shares(pkv, f, 1)
    out, lse, err = attend(pkv, f, max_kv=BIG)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("D,window,ring,kv", [(128, 1000, 1008, 5000), (64, 333, 352, 5000), (256, 512, 512, 3001)])
def test_shares_rings_and_padding(pkv, D, window, ring, kv):
    w = workloads.long_context(S=3, kv_len=kv, window=window, ring_rows=ring, q_heads=8, kv_heads=2, head_dim=D)
    f = Fp4(pkv, w, garbage=False, first_valid=np.array([0, kv - 100, kv + 5], np.int32))
    assert shares(pkv, f, 1)
    ws = pkv.new_workspace(f.cache, 8, 3, 1, BIG)
    out, lse, err = torch.empty(w.q[0].shape, device="cuda"), torch.empty(w.q[0].shape[:2], device="cuda"), pkv.new_err_flags()
    # (with a window the bound is the window's: enough kv heads and segments, or an ample window)
    pkv.attend_varlen(f.cache, 0, w.q[0].cuda(), w.seq_info.cuda(), out, err, 1, BIG, w.scale, w.causal, window, lse=lse, workspace=ws)
    assert int(err.item()) == 0
    check(f, out, lse)
    w = U.nan_tails(workloads.batched(S=5, max_len=3000, seed=2, q_heads=8, kv_heads=2, head_dim=D))
    fv = np.array([0, 5, 2999, 4000, 17], np.int32)
    f = Fp4(pkv, w, first_valid=fv)
    out, lse, err = attend(pkv, f, max_kv=BIG)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("seg,bit", [((2, 1, 9, 5), 1), ((-1, 2, 0, 9), 1), ((2, 9, 0, 9), 1), ((2, 1, 0, 99999), 2),
                                     ((2, 2, 1, 33), 8), ((2, 2, 1, 5990), 8), ((2, 2, 1, 17), 8), ((2, 4, 0, 9), 16)])
def test_shares_bad_segments_read_zero(pkv, seg, bit):
    w = workloads.batched(S=2, max_len=6000, seed=4, lengths=[6000, 5990], q_heads=4, kv_heads=2)
    w.block_table[1, 1] = 4000
    w.q = [torch.randn(6, 4, 128).bfloat16()]
    f = Fp4(pkv, w)
    w.seq_info = torch.tensor([seg, [0, 2, 0, 5900]], dtype=torch.int32)
    assert shares(pkv, f, 3)
    out, lse, err = attend(pkv, f, causal=True, max_q=3, max_kv=BIG)
    assert err == bit
    assert (out[2:] == 0).all() and torch.isinf(lse[2:]).all()
    w.seq_info = w.seq_info[1:]
    check(f, out, lse, causal=True, rows=np.arange(6) < 2)
    w.seq_info = torch.tensor([[0, 3, 0, 40], [2, 3, 0, 30]], dtype=torch.int32)
    assert attend(pkv, f, causal=True, max_q=3, max_kv=BIG)[2] == 32
    w.seq_info = torch.tensor([[7, 1, 0, 40]], dtype=torch.int32)   # past the rows: nothing is left to attend
    out, lse, err = attend(pkv, f, max_q=1, max_kv=BIG)
    assert err == 1 and (out == 0).all()


def test_shares_nan(pkv):
    w = workloads.spec_verify(S=1, max_q=4, len_lo=5000, len_hi=5000, seed=6, q_heads=4, kv_heads=2)
    w.seq_info = torch.tensor([[0, 4, 0, 5000]], dtype=torch.int32)
    w.q = [torch.randn(4, 4, 128).bfloat16()]
    f = Fp4(pkv, w)
    for at, see in ((4998, np.arange(4996, 5000) >= 4998), (1234, np.ones(4, bool))):
        pool = f.cache.v[0]
        keep = pool.clone()
        c, s = R.unpack(pool.cpu().numpy(), True)
        s[int(w.block_table[0, at // 16]), at % 16, 1, 2] = 0xFF
        pool.copy_(torch.from_numpy(R.pack(c, s, True)))
        out, lse, err = attend(pkv, f, causal=True, max_q=4, max_kv=BIG)
        want = np.zeros((4, 4, 128), bool)
        want[see, 2:, 32:48] = True
        assert err == 0 and (out.isnan().cpu().numpy() == want).all() and not lse.isnan().any()
        pool.copy_(keep)


def test_shares_in_graphs(pkv):
    """Two captured graphs, each with its own workspace from the allocator, replayed on two streams."""
    w = workloads.batched(S=4, max_len=4000, seed=3, q_heads=16, kv_heads=4)
    f = Fp4(pkv, w)
    q, si, err = w.q[0].cuda(), w.seq_info.cuda(), pkv.new_err_flags()
    want, want_lse, _ = attend(pkv, f, max_kv=BIG)
    made = []
    for _ in range(2):
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            for _ in range(3):
                pkv.attend_varlen(f.cache, 0, q, si, out, err, 1, BIG, w.scale, lse=lse, flags=pkv.FLAG_PDL)
        made.append((g, st, out, lse))
    for _ in range(20):
        for g, st, _, _ in made:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for _, _, out, lse in made:
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    assert int(err.item()) == 0


# ---------------------------------------------------------------- equal shares of wide groups (head_dim 128: the tcgen05 kernel)

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads,max_q", [(16, 1, 1), (17, 1, 1), (8, 2, 5), (64, 8, 16), (8, 1, 16), (16, 2, 40)])
@pytest.mark.parametrize("causal", [True, False])
def test_shares_wide(pkv, D, q_heads, kv_heads, max_q, causal):
    w = U.nan_tails(workloads.spec_verify(S=5, max_q=max_q, len_lo=max_q, len_hi=1500, seed=max_q + q_heads, q_heads=q_heads, kv_heads=kv_heads,
                                          head_dim=D, causal=causal))
    f = Fp4(pkv, w)
    assert shares(pkv, f, max_q) == (D != 256 or q_heads // kv_heads * max_q <= 256)   # at most 16 row tiles
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = attend(pkv, f, out_dtype=dt, max_kv=BIG, max_q=max_q)
        assert err == 0
        check(f, out, lse)
    again, lse2, _ = attend(pkv, f, out_dtype=dt, max_kv=BIG, max_q=max_q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window", [1, 17, 64, 333, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("padded", [False, True])
def test_shares_wide_windows_and_padding(pkv, window, causal, padded):
    w = U.nan_tails(workloads.spec_verify(S=6, max_q=9, len_lo=20, len_hi=900, seed=window, q_heads=16, kv_heads=2, causal=causal))
    ends = w.seq_info[:, 3].tolist()
    fv = np.array([0, 17, ends[2] - 1, ends[3] + 5, max(ends[4] - 5, 0), 3], np.int32) if padded else None
    f = Fp4(pkv, w, first_valid=fv)
    ws = pkv.new_workspace(f.cache, 16, 6, 9, BIG)
    assert ws is not None
    out, lse, err = torch.empty(w.q[0].shape, device="cuda"), torch.empty(w.q[0].shape[:2], device="cuda"), pkv.new_err_flags()
    pkv.attend_varlen(f.cache, 0, w.q[0].cuda(), w.seq_info.cuda(), out, err, 9, BIG, w.scale, causal, window if window < 5000 else 0, lse=lse, workspace=ws)
    assert int(err.item()) == 0
    check(f, out, lse, window=window if window < 5000 else 0)


def test_shares_wide_ring(pkv):
    w = workloads.long_context(S=3, kv_len=5000, window=2000, ring_rows=2016, q_heads=16, kv_heads=2, head_dim=128)
    g = torch.Generator().manual_seed(3)
    w.q = [torch.randn(30, 16, 128, generator=g).bfloat16()]
    w.seq_info = torch.tensor([[0, 10, 0, 5000], [10, 3, 1, 2100], [13, 17, 2, 40]], dtype=torch.int32)
    w.max_q_len = 17
    f = Fp4(pkv, w, garbage=False)
    assert shares(pkv, f, 17)
    out, lse, err = attend(pkv, f, max_kv=BIG)
    assert err == 0
    check(f, out, lse)


@pytest.mark.parametrize("seg,bit", [((2, 1, 9, 5), 1), ((-1, 2, 0, 9), 1), ((2, 9, 0, 9), 1), ((2, 1, 0, 99999), 2),
                                     ((2, 2, 1, 33), 8), ((2, 2, 1, 5990), 8), ((2, 2, 1, 17), 8), ((2, 4, 0, 9), 16)])
def test_shares_wide_bad_segments_read_zero(pkv, seg, bit):
    w = workloads.batched(S=2, max_len=6000, seed=4, lengths=[6000, 5990], q_heads=48, kv_heads=2)
    w.block_table[1, 1] = 4000
    w.q = [torch.randn(6, 48, 128).bfloat16()]
    f = Fp4(pkv, w)
    w.seq_info = torch.tensor([seg, [0, 2, 0, 5900]], dtype=torch.int32)
    assert shares(pkv, f, 3)
    out, lse, err = attend(pkv, f, causal=True, max_q=3, max_kv=BIG)
    assert err == bit
    assert (out[2:] == 0).all() and torch.isinf(lse[2:]).all()
    w.seq_info = w.seq_info[1:]
    check(f, out, lse, causal=True, rows=np.arange(6) < 2)


def test_shares_wide_nan(pkv):
    w = workloads.spec_verify(S=1, max_q=8, len_lo=5000, len_hi=5000, seed=6, q_heads=16, kv_heads=2)
    w.seq_info = torch.tensor([[0, 8, 0, 5000]], dtype=torch.int32)
    w.q = [torch.randn(8, 16, 128).bfloat16()]
    f = Fp4(pkv, w)
    for which, at in ((1, 4997), (1, 1234), (1, 4992), (0, 4997), (0, 777)):
        pool = (f.cache.k if which == 0 else f.cache.v)[0]
        keep = pool.clone()
        c, s = R.unpack(pool.cpu().numpy(), bool(which))
        s[int(w.block_table[0, at // 16]), at % 16, 1, 2] = 0xFF
        pool.copy_(torch.from_numpy(R.pack(c, s, bool(which))))
        out, lse, err = attend(pkv, f, causal=True, max_q=8, max_kv=BIG)
        see = np.arange(4992, 5000) >= at
        want = np.zeros((8, 16, 128), bool)
        want[see, 8:, (32 if which else 0):(48 if which else 128)] = True
        assert err == 0 and (out.isnan().cpu().numpy() == want).all()
        assert (lse.isnan().cpu().numpy() == (want.all(-1))).all()
        pool.copy_(keep)
    q = w.q[0].clone()
    q[3, 2, 7] = float("nan")
    out, lse, _ = attend(pkv, f, q=q, causal=True, max_q=8, max_kv=BIG)
    assert out[3, 2].isnan().all() and lse[3, 2].isnan() and int(out.isnan().any(-1).sum()) == 1


@pytest.mark.parametrize("q_heads", [4, 64])
def test_shares_scales_and_magnitudes(pkv, q_heads):
    """A negative and a zero softmax scale, and queries far from fp16's range."""
    w = workloads.batched(S=4, max_len=900, seed=5, q_heads=q_heads, kv_heads=2)
    f = Fp4(pkv, w)
    base = w.q[0].clone()

    def go(q, scale):
        out, lse, err = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda"), pkv.new_err_flags()
        pkv.attend_varlen(f.cache, 0, q.cuda(), w.seq_info.cuda(), out, err, 1, BIG, scale, lse=lse)
        assert int(err.item()) == 0
        return out, lse
    out, lse = go(base, w.scale)
    for e in (-100, -40, 40, 100):
        got, l2 = go((base.float() * 2.0 ** e).bfloat16(), w.scale * 2.0 ** -e)
        assert torch.equal(got, out) and torch.equal(l2, lse)
    got, l2 = go(-base, -w.scale)
    assert torch.allclose(got, out, rtol=0, atol=1e-6) and torch.allclose(l2, lse, rtol=1e-6)
    got, l2 = go(base, 0.0)
    for s, (_, _, col, kend) in enumerate(w.seq_info.tolist()):
        assert torch.allclose(l2[s], torch.full_like(l2[s], float(np.log(kend))), rtol=1e-5)


# ---------------------------------------------------------------- appends of many rows

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_many_rows(pkv, D, rotate):
    lengths = [700, 300, 17, 900, 64, 333]
    w = workloads.batched(S=6, max_len=1024, lengths=lengths, q_heads=4, kv_heads=2, head_dim=D, seed=1)
    w.block_table[4, 1] = -3
    rows = 2300
    g = torch.Generator().manual_seed(3)
    w.q, w.k_new, w.v_new = [[torch.randn(rows, h, D, generator=g).bfloat16()] for h in (4, 2, 2)]
    good = [[1000, 700, 0, 700], [5, 299, 1, 300], [400, 10, 2, 17], [1701, 500, 3, 900]]
    w.seq_info = torch.tensor(good + [[420, 40, 4, 64], [900, 50, 5, 40]], dtype=torch.int32)
    f = Fp4(pkv, w)
    q, kn, vn, err = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), pkv.new_err_flags()
    qo, ko, vo = torch.full_like(q, 9), torch.full_like(kn, 9), torch.full_like(vn, 9)
    freq, m = pkv.rope_inv_freq(D)
    rope = pkv.Rope(freq, device="cuda") if rotate else None
    pkv.norm_rope_append(f.cache, 0, rope, q, kn, vn, w.seq_info.cuda(), qo, err, k_out=ko, v_out=vo)
    assert int(err.item()) == 1 | 8
    w.seq_info = torch.tensor(good, dtype=torch.int32)
    live, k2 = torch.zeros(rows, dtype=torch.bool), kn.clone()
    pos = torch.zeros(rows, dtype=torch.int32)
    for q0, n, _, kend in good:
        live[q0:q0 + n] = True
        pos[q0:q0 + n] = torch.arange(kend - n, kend, dtype=torch.int32)
    q2 = q.clone()
    if rotate:
        pkv.norm_rope(rope, q2, k2, pos.cuda())
    want, e = f.oracle_bytes(k2.cpu(), w.v_new[0])
    assert e == 0
    for i in (0, 1):
        assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]
    for got, x in ((qo, q2), (ko, torch.from_numpy(R.values(*R.quantise(U.f64(k2)))).bfloat16().cuda()),
                   (vo, torch.from_numpy(R.values(*R.quantise(U.f64(vn)))).bfloat16().cuda())):
        assert torch.equal(got[live.cuda()], x[live.cuda()]) and (got[~live.cuda()] == 9).all()


# ---------------------------------------------------------------- appends that meet in a page

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kend", [1000, 1003, 77, 128])
def test_append_a_whole_ring(pkv, D, kend):
    """As many rows as the ring holds: its last new page is also its first one, cut between two tokens of a byte."""
    w = workloads.long_context(S=1, kv_len=kend, window=1, ring_rows=64, q_heads=3, kv_heads=3, head_dim=D)
    g = torch.Generator().manual_seed(kend)
    w.q, w.k_new, w.v_new = [[torch.randn(64, 3, D, generator=g).bfloat16()] for _ in range(3)]
    w.seq_info, w.window = torch.tensor([[0, 64, 0, kend]], dtype=torch.int32), 1
    want = None
    for _ in range(5):
        f, err = Fp4(pkv, w), pkv.new_err_flags()
        pkv.append(f.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), err, window=1)
        if want is None:
            want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
        assert e == 0 and int(err.item()) == 0
        for i in (0, 1):
            assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]


@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_segments_that_share_a_page(pkv, D):
    """Consecutive pieces of one sequence in one call, and tails of two sequences in a shared page."""
    w = workloads.batched(S=2, max_len=64, lengths=[64, 64], q_heads=2, kv_heads=2, head_dim=D)
    g = torch.Generator().manual_seed(D)
    w.q, w.k_new, w.v_new = [[torch.randn(40, 2, D, generator=g).bfloat16()] for _ in range(3)]
    w.block_table[1, 0] = w.block_table[0, 3]
    w.seq_info = torch.tensor([[0, 7, 0, 20], [7, 1, 0, 21], [8, 2, 0, 23], [10, 20, 0, 43], [30, 5, 1, 5], [35, 5, 0, 58]], dtype=torch.int32)
    for _ in range(5):
        f, err = Fp4(pkv, w), pkv.new_err_flags()
        pkv.append(f.cache, 0, w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), err)
        want, e = f.oracle_bytes(w.k_new[0], w.v_new[0])
        assert e == 0 and int(err.item()) == 0
        for i in (0, 1):
            assert f.host(i).tobytes() == want[i].tobytes(), "KV"[i]


def test_shares_on_a_given_stream(pkv):
    """stream= takes the call and its workspace to that stream: nothing on the current one is disturbed."""
    w = workloads.batched(S=4, max_len=4000, seed=3, q_heads=16, kv_heads=4)
    f = Fp4(pkv, w)
    q, si, err = w.q[0].cuda(), w.seq_info.cuda(), pkv.new_err_flags()
    want, want_lse, _ = attend(pkv, f, max_kv=BIG)
    n = pkv.attend_workspace_bytes(f.cache, 16, 4, 1, BIG)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    bufs = []
    for i in range(20):
        out, lse = torch.empty(q.shape, device="cuda"), torch.empty(q.shape[:2], device="cuda")
        st.wait_stream(torch.cuda.current_stream())
        pkv.attend_varlen(f.cache, 0, q, si, out, err, 1, BIG, w.scale, lse=lse, stream=st)
        bufs.append((out, lse, torch.full((n,), i, dtype=torch.uint8, device="cuda")))   # the current stream's own use of such a block
    torch.cuda.synchronize()
    for i, (out, lse, b) in enumerate(bufs):
        assert torch.equal(out, want) and torch.equal(lse, want_lse) and bool((b == i).all())
    assert int(err.item()) == 0


# ---------------------------------------------------------------- equal shares with a window: the window bounds the work, so many (empty) segments

def with_empty_segments(w, n):
    w.seq_info = torch.cat([w.seq_info, torch.zeros(n - w.num_segments, 4, dtype=torch.int32)])
    return w


def attend_in_shares(pkv, f, max_q, window):
    """Attention with a workspace, which must have been used."""
    w = f.w
    n = pkv.attend_workspace_bytes(f.cache, w.q_heads, w.num_segments, max_q, BIG)
    assert n > 0
    ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse, err = torch.empty(w.q[0].shape, device="cuda"), torch.empty(w.q[0].shape[:2], device="cuda"), pkv.new_err_flags()
    pkv.attend_varlen(f.cache, 0, w.q[0].cuda(), w.seq_info.cuda(), out, err, max_q, BIG, w.scale, w.causal, window, lse=lse, workspace=ws)
    assert int(err.item()) == 0 and not bool((ws == 0xA5).all()), "not run as shares"
    return out, lse


@pytest.mark.parametrize("q_heads,max_q", [(8, 1), (16, 4), (32, 4), (64, 9)])
@pytest.mark.parametrize("window", [1000, 3000])
@pytest.mark.parametrize("padded", [False, True])
def test_shares_with_windows(pkv, q_heads, max_q, window, padded):
    w = workloads.spec_verify(S=7, max_q=max_q, len_lo=max_q, len_hi=6000, seed=q_heads + window, q_heads=q_heads, kv_heads=8)
    ends = w.seq_info[:, 3].tolist()
    fv = np.array([0, 17, ends[2] - 1, ends[3] + 5, max(ends[4] - 5, 0), 3, 0], np.int32) if padded else None
    f = Fp4(pkv, w, first_valid=fv)
    with_empty_segments(w, 500)
    out, lse = attend_in_shares(pkv, f, max_q, window)
    check(f, out, lse, window=window)


@pytest.mark.parametrize("D,window,ring,kv", [(128, 3000, 3024, 5000), (64, 2000, 2000, 3000), (256, 2000, 2000, 3001)])
@pytest.mark.parametrize("q_heads", [8, 288])
def test_shares_with_rings(pkv, D, window, ring, kv, q_heads):
    w = workloads.long_context(S=3, kv_len=kv, window=window, ring_rows=ring, q_heads=q_heads, kv_heads=8, head_dim=D)
    f = Fp4(pkv, w, garbage=False, first_valid=np.array([0, kv - 100, kv + 5], np.int32))
    with_empty_segments(w, 500)
    out, lse = attend_in_shares(pkv, f, 1, window)
    check(f, out, lse, window=window)
