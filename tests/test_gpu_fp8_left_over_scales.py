"""The scale of a ring's 8-bit page after the tokens that made it are gone: overwritten, passed by the
window, or an earlier sequence's.

Bit for bit against the rule, in numpy: a ring page's scale does not get smaller unless it is more than 2^6 above
what the new rows and the tokens that count need; then it is what they need.  The tokens
count whose position some row from this step on may see.  Others of the ring
stay, saturated; slots that the sequence has not come to hold nothing.  Flat caches keep a page's
scale while it has tokens before the last new row.
"""
import numpy as np
import pytest
import torch

import workloads
from tests import fp8_ref as R
from tests import gpu_util as U
from tests.test_gpu_fp8 import Fp8, check, attend

pytestmark = pytest.mark.gpu
SLACK = 6


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def write_page(block, new, kept, count, ring):
    D = block.shape[-1] // 16 - 1
    c, b0, m0 = (x[0] for x in R.unpack(block[None, None]))
    c, b0, m0 = c[:, 0], min(int(b0[0]), 246), int(m0[0])
    nan = {t for t, x in new.items() if np.isnan(x).any()}
    clean = {t: np.where(np.isnan(x), 0.0, x) for t, x in new.items()}
    b = int(R.exponent(max(np.abs(x).max() for x in clean.values())))
    mask = sum(1 << t for t in nan)
    if kept:
        mask |= m0 & sum(1 << t for t in kept)
        least = b0
        if ring and b0 > b + SLACK:
            theirs = int(R.exponent(max([float(R.MAGS[c[t] & 127].max()) * 2.0 ** (b0 - 127) for t in count], default=0.0)))
            if max(theirs, b) + SLACK < b0:
                least = max(theirs, 1)
        b = max(b, least)
        if b0 and b != b0:
            for t in kept:
                c[t] = R.codes_of(np.where(c[t] >= 128, -1.0, 1.0) * R.MAGS[c[t] & 127] * 2.0 ** (b0 - b), 127)
    for t, x in clean.items():
        c[t] = np.where(np.isnan(new[t]), 0, R.codes_of(x, b))
    held = {t: np.full(D, np.nan) if t in nan else R.values_of(c[t], b) for t in new}
    return R.pack(c[None, :, None], np.array([[b]]), np.array([[mask]]), block[None, None])[0, 0], held


def append(pool, table, seq_info, rows, ring, window):
    held = np.full(rows.shape, 9.0)
    pages, span = {}, {}
    for q0, n, col, kend in np.asarray(seq_info).tolist():
        lo, hi = span.get(col, (kend - n, kend))
        span[col] = min(lo, kend - n), max(hi, kend)
        for i in range(n):
            at = (kend - n + i) % ring if ring else kend - n + i
            pages.setdefault((col, at // 16), {})[at % 16] = q0 + i
    for (col, tp), slots in pages.items():
        first, kend = span[col]
        if ring:
            last = {t: kend - 1 - (kend - 1 - (tp * 16 + t)) % ring for t in range(16) if t not in slots}
            kept = [t for t, at in last.items() if at >= 0]
            count = [t for t in kept if last[t] > first - window]
        else:
            kept = count = [t for t in range(max(slots)) if t not in slots]
        block = int(table[col, tp])
        for h in range(pool.shape[1]):
            pool[block, h], out = write_page(pool[block, h], {t: rows[r, h] for t, r in slots.items()}, kept, count, ring)
            for t, r in slots.items():
                held[r, h] = out[t]
    return held


class Ring:
    """S sequences over rings (ring 0: flat) whose pools hold anything at first."""

    def __init__(self, pkv, S, D, ring, window, left_over=True, cap=256):
        self.w = workloads.long_context(S=S, kv_len=64, window=window, ring_rows=ring, q_heads=4, kv_heads=2, head_dim=D) if ring else \
            workloads.batched(S=S, max_len=cap, lengths=[cap] * S, q_heads=4, kv_heads=2, head_dim=D)
        self.f = Fp8(pkv, self.w, garbage=False)
        self.pkv, self.window = pkv, window
        r = np.random.default_rng(3)
        for i, p in enumerate((self.f.cache.k[0], self.f.cache.v[0])):
            b = self.f.bytes[i]
            b[:] = 0
            if left_over:  # of an earlier sequence: large scales, NaN marks, any codes
                c = r.integers(0, 256, (len(b), 16, 2, D)).astype(np.uint8)
                b[:] = R.pack(np.where((c & 127) == 127, 5, c), r.integers(180, 247, (len(b), 2)), r.integers(0, 65536, (len(b), 2)))
            p.view(torch.uint8).copy_(torch.from_numpy(b))

    def step(self, table, kn, vn):
        w, err = self.w, self.pkv.new_err_flags()
        before = [self.f.host(i).copy() for i in (0, 1)]
        kn, vn = kn.cuda(), vn.cuda()
        ko, vo = torch.full_like(kn, 9), torch.full_like(vn, 9)
        self.pkv.norm_rope_append(self.f.cache, 0, None, None, kn, vn, torch.tensor(table, dtype=torch.int32).cuda(), None, err,
                                  window=self.window, k_out=ko, v_out=vo)
        assert int(err.item()) == 0
        self.f.check_guards()
        for i, (x, got) in enumerate(((kn, ko), (vn, vo))):
            held = append(before[i], w.block_table.numpy(), table, U.f64(x), w.ring_rows, self.window)
            assert np.array_equal(U.f64(got), held, equal_nan=True), "KV"[i]
            assert self.f.host(i).tobytes() == before[i].tobytes(), "KV"[i]
        return ko, vo


def close(got, x, spread=16.0):
    """Rows of one size are held to half a step of e4m3 of each value (2^-4), or, where the value is small, of
    2^-10 of a scale that holds 2^SLACK times the largest (448 of it being at least half of that)."""
    got, x = U.f64(got), U.f64(x)
    lim = np.abs(x) * 2.0 ** -4 + 2.0 ** -10 * 2.0 ** (SLACK + 1) * np.abs(x).max() * spread / 448
    assert (np.abs(got - x) <= lim).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,ring", [(32, 48), (33, 64), (48, 48), (7, 16)])
def test_a_new_sequence_in_old_pages(pkv, D, window, ring):
    r, g = Ring(pkv, 2, D, ring, window), torch.Generator().manual_seed(D)
    n = [0, 0]
    for t in range(3 * ring // 2):
        rows = torch.randn(2, 2, 2, D, generator=g).bfloat16()
        n = [n[0] + 1, n[1] + 1]
        ko, vo = r.step([[0, 1, 0, n[0]], [1, 1, 1, n[1]]], rows[0], rows[1])
        close(ko, rows[0])
        close(vo, rows[1])


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("window,ring", [(32, 48), (48, 48), (20, 96)])
@pytest.mark.parametrize("odd", [2.0 ** 30, float("inf"), float("nan")])
@pytest.mark.parametrize("q", [1, 3])
def test_an_outlier_ages_out(pkv, D, window, ring, odd, q):
    """One token among ordinary ones: rows are held well again once no row sees it."""
    if window + q - 1 > ring:
        pytest.skip("the ring is too short for the step")
    r, g = Ring(pkv, 2, D, ring, window, left_over=False), torch.Generator().manual_seed(D + q)
    end, at = 0, 21
    while end < 3 * ring:
        first, end = end, end + q
        rows = torch.randn(2, 2 * q, 2, D, generator=g).bfloat16()
        if first <= at < end:
            rows[:, at - first, 0, 3] = odd     # of the first sequence's head 0
        ko, vo = r.step([[0, q, 0, end], [q, q, 1, end]], rows[0], rows[1])
        if first >= at + window or end <= at // 16 * 16:
            close(ko, rows[0])
            close(vo, rows[1])
        else:
            close(ko[q:], rows[0][q:])
    r.w.seq_info = torch.tensor([[0, 1, 0, end], [1, 1, 1, end]], dtype=torch.int32)
    out, lse, err = attend(pkv, r.f, max_q=1, causal=True, window=window)
    assert err == 0
    check(r.f, out, lse, causal=True, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window,ring", [(0, 0), (20, 64), (40, 48)])
def test_any_steps(pkv, D, window, ring):
    """Steps of any length and size, pieces of a sequence, rewinds: the rule, bit for bit."""
    r, g = Ring(pkv, 2, D, ring, window, left_over=bool(ring)), torch.Generator().manual_seed(D + ring)
    rng = np.random.default_rng(D + ring)
    ends = [0, 0]
    for _ in range(60):
        table, q0 = [], 0
        for col in (0, 1):
            n = int(rng.integers(1, min(ring - window + 2, 20) if ring else 20))
            back = int(rng.integers(0, min(ends[col], ring - window + 1 if ring else 12) + 1)) if rng.random() < 0.3 else 0
            ends[col] += n - back
            if not ring and ends[col] > 256:
                ends[col] = n
            cut = int(rng.integers(0, n)) if rng.random() < 0.5 else 0
            if cut:
                table.append([q0, cut, col, ends[col] - n + cut])
            table.append([q0 + cut, n - cut, col, ends[col]])
            q0 += n
        size = torch.exp2(torch.randint(-12, 13, (2, q0, 2, 1), generator=g).float() * float(rng.integers(0, 4)))
        rows = (torch.randn(2, q0, 2, D, generator=g) * size).bfloat16()
        r.step([table[i] for i in rng.permutation(len(table))], rows[0], rows[1])


def test_a_rewound_ring_gives_back_its_tokens(pkv):
    """Tokens that the window had passed are as they were, if they are no larger than 2^6 times what came after them."""
    D, window, ring = 64, 20, 64
    r, g = Ring(pkv, 1, D, ring, window), torch.Generator().manual_seed(1)
    held = []
    for t in range(80):
        rows = torch.randn(2, 1, 2, D, generator=g).bfloat16()
        held.append(r.step([[0, 1, 0, t + 1]], rows[0], rows[1])[0])
    k = R.pool_values(r.f.host(0))
    for at in range(80 - ring, 80):
        got = k[int(r.w.block_table[0, at % ring // 16]), at % ring % 16]
        assert np.abs(got - U.f64(held[at][0])).max() <= 2.0 ** -10 * 2.0 ** (SLACK + 1) * 6 / 224
