"""norm_rope and norm_rope_append on the GPU against the 64-bit definition.

Tolerances.  A rotated value is m (u c - w s) with u = x r w: fp32 products
and one fused add (3 roundings of 2^-24), r = rsqrt (its argument's sum of D
squares, at most (D / 8 + 8) 2^-24 in this order of summing, halved by the
root; the call 2 ulp), c and s from an angle of 2^-24 relative error in half
turns (at most pi 2^-24 rad) and 2 ulp.  All in all less than 2^-18 of
m (|u| + |w|) for D <= 256, then one rounding to the rows' type: half a step,
2^-8 (bf16) or 2^-24 (fp32) of the value.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import oracle as O
from tests import fp4_ref as R
from tests import gpu_util as U

pytestmark = pytest.mark.gpu
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def make(seed, rows, hq, hkv, D, dtype):
    g = torch.Generator().manual_seed(seed)
    q, k, v = [torch.randn(rows, h, D, generator=g).mul(s).to(dtype).cuda() for h, s in ((hq, 1.5), (hkv, 3.0), (hkv, 0.5))]
    wq, wk = [(1 + 0.3 * torch.randn(D, generator=g)).to(dtype).cuda() for _ in range(2)]
    return q, k, v, wq, wk


def check_rows(got, x, weight, eps, freq, pos, mscale, interleaved, dtype):
    f = None if freq is None else freq.double().numpy()
    w = None if weight is None else U.f64(weight)
    want = R.norm_rope(U.f64(x), w, eps, f, pos, mscale, interleaved)
    # the size |u| + |w| of the pair a value is made of, before the rotation
    size = np.abs(R.norm_rope(U.f64(x), w, eps, None, pos))
    if f is not None:
        r = 2 * len(f)
        a, b = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
        pair = abs(mscale) * (size[..., a] + size[..., b])
        size[..., a] = size[..., b] = pair
    tol = 2.0 ** -18 * size + HALF[dtype] * (np.abs(want) + 2.0 ** -18 * size)
    got = U.f64(got)
    assert np.isfinite(got).all()
    worst = float((np.abs(got - want) / np.maximum(tol, 1e-300)).max())
    assert worst <= 1.0, f"{worst} times the tolerance"


# head dims that fill no power of two of lanes, halves that are no whole lanes, heads that fill no warp
SHAPES = [(64, 64), (128, 128), (256, 256), (128, 64), (128, 32), (80, 80), (72, 24), (64, 2), (256, 66), (8, 8), (8, 4), (128, 0), (200, 120)]


@pytest.mark.parametrize("D,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_shapes(pkv, D, rot, interleaved, dtype, norm):
    rows, hq, hkv = 5, 7, 3
    q, k, v, wq, wk = make(D + rot, rows, hq, hkv, D, dtype)
    freq, m = pkv.rope_inv_freq(rot) if rot else (None, 1.0)
    rope = pkv.Rope(freq, interleaved, q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-5, device="cuda")
    pos = torch.tensor([0, 1, 17, 4095, 131071], dtype=torch.int32)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    pkv.norm_rope(rope, q, k, pos.cuda(), qo, ko)
    check_rows(qo, q, wq if norm else None, 1e-5, freq, pos.numpy(), m, interleaved, dtype)
    check_rows(ko, k, wk if norm else None, 1e-5, freq, pos.numpy(), m, interleaved, dtype)
    # in place: bit for bit the same
    pkv.norm_rope(rope, q, k, pos.cuda())
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_far_positions_and_scalings(pkv, scaling):
    freq, m = pkv.rope_inv_freq(128, 500000.0, scaling, factor=32.0, trained_len=4096)
    pos = torch.tensor([2 ** 31 - 1, -1, -(2 ** 31), 10 ** 9 + 7, -12345, 2 ** 24 + 1], dtype=torch.int32)
    q, k, _, wq, _ = make(3, 6, 4, 2, 128, torch.float32)
    rope = pkv.Rope(freq, False, mscale=m, q_weight=wq, device="cuda")
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.norm_rope(rope, q, k, pos.cuda(), qo, ko)
    # the reference's own angle loses pos * 2^-53 turns: 1e-6 at 2^31, so it is reduced exactly first
    from fractions import Fraction
    ang = np.array([[float(Fraction(int(p)) * Fraction(float(f)) % Fraction(2 * np.pi)) for f in freq] for p in pos])
    x = R.norm_rope(U.f64(q), U.f64(wq), 1e-6, None, None)
    u, w = x[..., :64], x[..., 64:]
    c, s = m * np.cos(ang)[:, None], m * np.sin(ang)[:, None]
    want = np.concatenate([u * c - w * s, w * c + u * s], -1)
    # Two more terms: Fraction(2 * pi) is off by 2.4e-16, times pos * freq / 2 pi turns (3.4e8): 9e-8 rad here;
    # 1 / 2 pi in the turns by 2^-54, and the turns by 2^-53, of a turn a position: 2^31 * 2^-52 * 2 pi = 3e-6 rad.
    tol = (2.0 ** -18 + 4e-6) * m * np.concatenate([np.abs(u) + np.abs(w)] * 2, -1)
    assert (np.abs(U.f64(qo) - want) <= tol).all()


def test_one_side_only_and_strided_rows(pkv):
    rows, hq, hkv, D = 9, 12, 4, 128
    g = torch.Generator().manual_seed(1)
    qkv = torch.randn(rows, (hq + 2 * hkv) * D + 24, generator=g).bfloat16().cuda()
    q, k = qkv[:, :hq * D].unflatten(1, (hq, D)), qkv[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
    keep = qkv.clone()
    freq, _ = pkv.rope_inv_freq(D)
    rope = pkv.Rope(freq, device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 31
    qo = torch.empty(rows, hq, D, dtype=torch.bfloat16, device="cuda")
    pkv.norm_rope(rope, q, None, pos, qo)
    check_rows(qo, q, None, 0, freq, pos.cpu().numpy(), 1.0, False, torch.bfloat16)
    ko = torch.empty(rows, hkv, D, dtype=torch.bfloat16, device="cuda")
    pkv.norm_rope(rope, None, k, pos, None, ko)
    check_rows(ko, k, None, 0, freq, pos.cpu().numpy(), 1.0, False, torch.bfloat16)
    assert torch.equal(qkv, keep)
    pkv.norm_rope(rope, q, k, pos)   # in place in the projection's output: the rest of it stays
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, (hq + hkv) * D:], keep[:, (hq + hkv) * D:])


def test_empty_and_nan_rows(pkv):
    freq, _ = pkv.rope_inv_freq(64)
    rope = pkv.Rope(freq, device="cuda")
    pkv.norm_rope(rope, torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda"), None, torch.zeros(0, dtype=torch.int32, device="cuda"))
    q = torch.ones(2, 3, 64, dtype=torch.float32, device="cuda")
    q[0, 1, 5] = float("nan")
    part = pkv.Rope(pkv.rope_inv_freq(8)[0], device="cuda")
    q[1, 2, 40] = float("inf")
    out = torch.empty_like(q)
    pkv.norm_rope(part, q, None, torch.tensor([3, 4], dtype=torch.int32, device="cuda"), out)
    bad = ~torch.isfinite(out)
    assert bad[0, 1, 1] and bad[0, 1, 5] and bad[1, 2, 40] and int(bad.sum()) == 3   # a pair, and a column that is not rotated


# ---------------------------------------------------------------- with the append

def appended(w, pool_dtype):
    kp, vp = w.k[0].clone(), w.v[0].clone()
    return kp, vp


def run_append(pkv, w, rope_kw, freq, norm, positions=None, q_out=True, seed=0, outs=True):
    """norm_rope_append of w's step and its checks against the definition and the oracle's append."""
    dtype = w.dtype
    wq, wk = make(seed, 1, 1, 1, w.head_dim, dtype)[3:]
    rope = pkv.Rope(freq, q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-6, device="cuda", **rope_kw)
    cache = U.device_cache(pkv, w, canary=True)
    q, kn, vn, si = w.q[0].cuda(), w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda()
    err = pkv.new_err_flags()
    qo, ko, vo = torch.full_like(q, 9.0), torch.full_like(kn, 9.0), torch.full_like(vn, 9.0)
    pkv.norm_rope_append(cache, 0, rope, q, kn, vn, si, qo, err, window=w.window, positions=positions,
                         k_out=ko if outs else None, v_out=vo if outs else None)
    torch.cuda.synchronize()
    U.check_canaries(cache)
    return rope, cache, qo, ko, vo, int(err.item()), wq, wk


def cache_positions(w):
    pos = np.zeros(w.total_rows, np.int64)
    rows = np.zeros(w.total_rows, bool)
    for q0, ql, col, kend in w.seq_info.tolist():
        pos[q0:q0 + ql] = np.arange(kend - ql, kend)
        rows[q0:q0 + ql] = True
    return pos, rows


def check_append(w, cache, qo, ko, vo, wq, wk, norm, freq, pos, mscale, interleaved, rows):
    dtype = w.dtype
    check_rows(qo[rows], w.q[0][rows], wq if norm else None, 1e-6, freq, pos[rows], mscale, interleaved, dtype)
    check_rows(ko[rows], w.k_new[0][rows], wk if norm else None, 1e-6, freq, pos[rows], mscale, interleaved, dtype)
    assert torch.equal(vo[rows].cpu(), w.v_new[0][rows])
    # the pools: the oracle's append of the rows that came out, bit for bit, and nothing else
    w.k_new[0], w.v_new[0] = ko.cpu(), vo.cpu()
    kp, vp, err = U.oracle_append_pools(w, 0)
    assert err == 0
    assert U.pool_bytes(cache.k[0]) == kp.tobytes() and U.pool_bytes(cache.v[0]) == vp.tobytes()


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.bfloat16, 80), (torch.bfloat16, 256), (torch.float32, 64), (torch.float32, 256)])
@pytest.mark.parametrize("interleaved,norm", [(False, True), (True, False)])
@pytest.mark.parametrize("max_q", [1, 37])
def test_append_ragged(pkv, dtype, D, interleaved, norm, max_q):
    w = U.nan_tails(workloads.spec_verify(S=6, max_q=max_q, len_lo=max_q, len_hi=200, seed=D, q_heads=12, kv_heads=3, head_dim=D, dtype=dtype))
    rot = D // 2 if interleaved else D
    freq, m = pkv.rope_inv_freq(rot, scaling="yarn", factor=4.0, trained_len=64)
    _, cache, qo, ko, vo, err, wq, wk = run_append(pkv, w, dict(interleaved=interleaved, mscale=m), freq, norm)
    assert err == 0
    pos, rows = cache_positions(w)
    check_append(w, cache, qo, ko, vo, wq, wk, norm, freq, pos, m, interleaved, rows)


def test_append_given_positions_ring_and_gaps(pkv):
    # a ring that wraps inside the step, rows between segments that belong to none, positions of the caller's own
    w = workloads.long_context(S=3, kv_len=1000, window=100, ring_rows=128, q_heads=8, kv_heads=2, head_dim=64)
    g = torch.Generator().manual_seed(5)
    rows = 40
    w.q, w.k_new, w.v_new = [[torch.randn(rows, h, 64, generator=g).bfloat16()] for h in (8, 2, 2)]
    w.seq_info = torch.tensor([[20, 20, 2, 1000], [0, 7, 0, 129], [9, 0, 1, 5], [8, 1, 1, 1]], dtype=torch.int32)
    positions = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    freq, m = pkv.rope_inv_freq(64)
    _, cache, qo, ko, vo, err, wq, wk = run_append(pkv, w, {}, freq, True, positions=positions.cuda())
    assert err == 0
    _, live = cache_positions(w)
    live[9:20] = False
    assert (qo[~live] == 9).all() and (ko[~live] == 9).all() and (vo[~live] == 9).all()
    check_append(w, cache, qo, ko, vo, wq, wk, True, freq, positions.numpy(), m, False, live)


def test_append_without_rope_is_append(pkv):
    w = workloads.batched(S=5, max_len=90, seed=2)
    a, b = U.device_cache(pkv, w), U.device_cache(pkv, w)
    kn, vn, si, err = w.k_new[0].cuda(), w.v_new[0].cuda(), w.seq_info.cuda(), pkv.new_err_flags()
    pkv.append(a, 0, kn, vn, si, err)
    pkv.norm_rope_append(b, 0, None, None, kn, vn, si, None, err)
    assert torch.equal(a.k[0], b.k[0]) and torch.equal(a.v[0], b.v[0]) and int(err.item()) == 0


BAD = [((0, 1, 9, 5), 1), ((-1, 2, 0, 9), 1), ((0, 9, 0, 9), 1), ((0, 3, 0, 2), 1), ((0, 1, 0, 4096), 2), ((0, 2, 1, 40), 8), ((4, 0, -1, 3), 1)]


@pytest.mark.parametrize("seg,bit", BAD)
def test_bad_segments_write_nothing(pkv, seg, bit):
    w = workloads.batched(S=2, max_len=64, seed=4, lengths=[64, 33])
    # column 1 lists 3 pages; its last one is outside the pool
    w.block_table[1, 2] = 4000 if bit == 8 else w.block_table[1, 2]
    w.q, w.k_new, w.v_new = [[torch.randn(4, h, 128).bfloat16()] for h in (32, 8, 8)]
    w.seq_info = torch.tensor([seg, [2, 2, 0, 60]], dtype=torch.int32)
    freq, _ = pkv.rope_inv_freq(128)
    _, cache, qo, ko, vo, err, _, _ = run_append(pkv, w, {}, freq, False)
    assert err == bit
    for t in (qo, ko, vo):
        assert (t[:2] == 9).all() and not (t[2:] == 9).all()
    w.seq_info = w.seq_info[1:]
    w.k_new[0], w.v_new[0] = ko.cpu(), vo.cpu()
    kp, vp, e = U.oracle_append_pools(w, 0)
    assert U.pool_bytes(cache.k[0]) == kp.tobytes() and U.pool_bytes(cache.v[0]) == vp.tobytes()


def test_many_rows_and_unsorted_segments(pkv):
    # more rows than a warp each, segments in no order, more than a warp's worth of them
    S, rows = 70, 0
    g = torch.Generator().manual_seed(8)
    qlens = torch.randint(1, 60, (S,), generator=g).tolist()
    lengths = [n + int(torch.randint(0, 50, (1,), generator=g)) for n in qlens]
    w = workloads.batched(S=S, max_len=128, lengths=lengths, q_heads=4, kv_heads=2, head_dim=64, seed=9)
    order = torch.randperm(S, generator=g).tolist()
    si = []
    for s in order:
        si.append([rows, qlens[s], s, lengths[s]])
        rows += qlens[s]
    w.seq_info = torch.tensor([si[i] for i in torch.randperm(S, generator=g).tolist()], dtype=torch.int32)
    w.q, w.k_new, w.v_new = [[torch.randn(rows, h, 64, generator=g).bfloat16()] for h in (4, 2, 2)]
    freq, _ = pkv.rope_inv_freq(64)
    _, cache, qo, ko, vo, err, wq, wk = run_append(pkv, w, {}, freq, True)
    assert err == 0
    pos, live = cache_positions(w)
    check_append(w, cache, qo, ko, vo, wq, wk, True, freq, pos, 1.0, False, live)


# ---------------------------------------------------------------- many rows: through shared memory

@pytest.mark.parametrize("dtype,D,rot,interleaved,hq,hkv", [
    (torch.bfloat16, 128, 128, False, 8, 2), (torch.bfloat16, 128, 64, True, 7, 3), (torch.bfloat16, 72, 24, False, 5, 1),
    (torch.float32, 64, 64, False, 4, 2), (torch.float32, 80, 18, False, 3, 1), (torch.bfloat16, 256, 256, False, 64, 8),
])
@pytest.mark.parametrize("norm", [False, True])
def test_many_rows(pkv, dtype, D, rot, interleaved, hq, hkv, norm):
    rows = 1501
    g = torch.Generator().manual_seed(rows + D)
    q, k, v, wq, wk = make(D, rows, hq, hkv, D, dtype)
    freq, m = pkv.rope_inv_freq(rot, scaling="yarn", factor=4.0, trained_len=512)
    rope = pkv.Rope(freq, interleaved, mscale=m, q_weight=wq if norm else None, k_weight=wk if norm else None, eps=1e-6, device="cuda")
    pos = torch.randint(0, 1 << 20, (rows,), generator=g, dtype=torch.int32)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pkv.norm_rope(rope, q, k, pos.cuda(), qo, ko)
    check_rows(qo, q, wq if norm else None, 1e-6, freq, pos.numpy(), m, interleaved, dtype)
    check_rows(ko, k, wk if norm else None, 1e-6, freq, pos.numpy(), m, interleaved, dtype)
    pkv.norm_rope(rope, q, k, pos.cuda())       # in place, through the stages
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 128), (torch.float32, 64)])
def test_many_rows_append(pkv, dtype, D):
    """Ragged prompts with gaps, a refused segment and a bad page among them."""
    lengths = [700, 300, 17, 900, 64, 333]
    w = workloads.batched(S=6, max_len=1024, lengths=lengths, q_heads=6, kv_heads=2, head_dim=D, dtype=dtype, seed=1)
    w.block_table[4, 1] = -3
    rows = 2300
    g = torch.Generator().manual_seed(3)
    w.q, w.k_new, w.v_new = [[torch.randn(rows, h, D, generator=g).to(dtype)] for h in (6, 2, 2)]
    w.seq_info = torch.tensor([[1000, 700, 0, 700], [5, 299, 1, 300], [400, 10, 2, 17], [1701, 500, 3, 900], [420, 40, 4, 64], [900, 50, 5, 40]],
                              dtype=torch.int32)
    freq, m = pkv.rope_inv_freq(D)
    _, cache, qo, ko, vo, err, wq, wk = run_append(pkv, w, {}, freq, True)
    assert err == 1 | 8
    w.seq_info = w.seq_info[:4]
    pos, live = cache_positions(w)
    assert (qo[~live] == 9).all() and (ko[~live] == 9).all() and (vo[~live] == 9).all()
    check_append(w, cache, qo, ko, vo, wq, wk, True, freq, pos, 1.0, False, live)
