"""Attention over an 8-bit cache whose V pages are far apart in scale: what a row
does not see, or hardly weighs, costs it nothing.

Tolerance, of each row by itself.  With weights p (of sum L) and V = code * 2^e: scores are fp32 sums
of exact products, off by d = D 2^-24 max|q| sum|k| scale; a weight of the product is rounded to
fp16, by 2^-11 of itself or by 2^-25 in a unit in which the row's largest p 2^e is 2^7 at least, 448 times
that in each of n keys; 2^-16 is for exponentials and the sums.  So the error is at most
(2^-11 + 2 d + 2^-16) A + 448 n 2^-32 B, with A = sum p |V| / L and B = sum p 2^e / L >= max p 2^e / L.
A weight below 2^-126 of the row's largest may count as zero: 2^(score - largest score) is then below the least
normal fp32 number, 2^-126, in the factor by which a split's or warp's sums join those of the one that holds the
largest score.  That is at most the part of A that such keys have.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import oracle as O
from tests import fp8_ref as R
from tests import gpu_util as U
from tests.test_gpu_fp4 import BIG, attend
from tests.test_gpu_fp8 import Fp8

pytestmark = pytest.mark.gpu
D2E = 1.4426950408889634


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def set_pool(f, i, codes=None, b=None):
    """Codes [blocks, 16, H, D] and biased exponents [blocks, H] of pool i, on the device too."""
    c, b0, m = R.unpack(f.host(i))
    f.bytes[i] = R.pack(c if codes is None else codes, b0 if b is None else b, m)
    (f.cache.k if i == 0 else f.cache.v)[0].view(torch.uint8).copy_(torch.from_numpy(f.bytes[i]))


def check_rows(f, out, q, causal, window, rows, light=()):
    """light: pages whose keys all have weights below 2^-126 of the row's largest."""
    w = f.w
    D, n = w.head_dim, int(w.seq_info[:, 3].max())
    k, v = [np.nan_to_num(R.pool_values(f.host(i)), nan=0.0) for i in (0, 1)]
    _, b, _ = R.unpack(f.host(1))
    unit = np.broadcast_to(R.scale(b)[:, None, :, None], v.shape)
    ref, a, c = [O.attend(U.f64(q), k, x, w.block_table.numpy(), w.seq_info.numpy(), w.scale, causal=causal, window=window)[0]
                 for x in (v, np.abs(v), np.ascontiguousarray(unit))]
    d = D * 2.0 ** -24 * float(np.abs(U.f64(q)).max()) * np.abs(k).reshape(-1, D).sum(-1).max() * w.scale
    lim = (2.0 ** -11 + 2 * d + 2.0 ** -16) * a + 448 * n * 2.0 ** -32 * c
    if len(light):
        only = np.zeros_like(v)
        only[light] = np.abs(v[light])
        lim = lim + O.attend(U.f64(q), k, only, w.block_table.numpy(), w.seq_info.numpy(), w.scale, causal=causal, window=window)[0]
    got = U.f64(out)
    assert np.isfinite(got[rows]).all()
    worst = float((np.abs(got - ref)[rows] / lim[rows]).max())
    assert worst <= 1, f"{worst} times the tolerance"


def table(lens, ql):
    return torch.tensor([[i * ql, ql, i, n] for i, n in enumerate(lens)], dtype=torch.int32)


SHAPES = [(64, 4, 1), (128, 8, 1), (256, 8, 1), (64, 32, 1), (128, 16, 1), (128, 32, 1), (256, 16, 1), (128, 64, BIG)]


@pytest.mark.parametrize("D,q_heads,max_kv", SHAPES)
@pytest.mark.parametrize("behind", ["causal", "window"])
def test_a_page_hidden_from_rows(pkv, D, q_heads, max_kv, behind):
    """The last page holds one token, under the scale of an infinity, which only the last row sees; or the first
    pages are under it, behind the window of every row but the first."""
    ql, lens, window = 4, [113, 273], 0
    w = workloads.batched(S=2, max_len=288, lengths=lens, q_heads=q_heads, kv_heads=2, head_dim=D, seed=D)
    w.q = [torch.randn(2 * ql, q_heads, D, generator=torch.Generator().manual_seed(1)).bfloat16()]
    w.seq_info = table(lens, ql)
    f = Fp8(pkv, w, garbage=False, kscale=1.0)
    b = R.unpack(f.host(1))[1]
    rows = np.ones(2 * ql, bool)
    bt = w.block_table.numpy()
    if behind == "causal":
        for i, n in enumerate(lens):
            b[bt[i, n // 16]] = 246
        rows[ql - 1::ql] = False
    else:
        # the first row sees key n - 4 - window + 1 = 16 m - 1 of page m - 1, the others begin at page m
        window = 63
        for i, n in enumerate(lens):
            first = n - ql - window + 1
            assert first % 16 == 15
            b[bt[i, :first // 16 + 1]] = 246
        rows[0::ql] = False
    set_pool(f, 1, b=b)
    out, _, err = attend(pkv, f, causal=True, window=window, max_q=ql, max_kv=max_kv if max_kv > 1 else 288)
    assert err == 0
    check_rows(f, out, w.q[0], True, window, rows)


@pytest.mark.parametrize("D,q_heads,max_kv", SHAPES)
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("splits", [0, 1])
def test_a_page_without_weight(pkv, D, q_heads, max_kv, where, splits):
    """Every row sees a page under 2^60 whose keys have 2^-180 of the others' weight: 2^-120 of them in the products."""
    n, ql = 256, 4
    w = workloads.batched(S=1, max_len=n, lengths=[n], q_heads=q_heads, kv_heads=2, head_dim=D, seed=D)
    g = torch.Generator().manual_seed(2)
    q = torch.randn(ql, q_heads, D, generator=g)
    q[..., 0] = 16.0
    w.q = [q.bfloat16()]
    w.seq_info = table([n], ql)
    f = Fp8(pkv, w, garbage=False, kscale=0.05)
    page = w.block_table.numpy()[0, {"first": 0, "middle": 7, "last": 15}[where]]
    kc, kb, _ = R.unpack(f.host(0))
    k = R.values_of(kc, kb[:, None, :, None])
    k[..., 0] = 0.0
    k[page, :, :, 0] = -180 / (16.0 * w.scale * D2E)
    kb = R.exponent(np.abs(k).max((1, 3)))
    set_pool(f, 0, R.codes_of(k, kb[:, None, :, None]), kb)
    b = R.unpack(f.host(1))[1]
    b[page] = 127 + 60
    set_pool(f, 1, b=b)
    out, _, err = attend(pkv, f, causal=False, max_q=ql, max_kv=max_kv if max_kv > 1 else n, num_splits=0 if max_kv > 1 else splits)
    assert err == 0
    check_rows(f, out, w.q[0], False, 0, np.ones(ql, bool))


@pytest.mark.parametrize("D,q_heads,max_kv", SHAPES)
@pytest.mark.parametrize("spread", [20, 55])
def test_pages_of_any_scale(pkv, D, q_heads, max_kv, spread):
    """V pages up to 2^(2 spread) apart in any order, some all zero, seen by some rows and not by others."""
    ql, lens = 4, [400, 37, 210]
    w = workloads.batched(S=3, max_len=400, lengths=lens, q_heads=q_heads, kv_heads=2, head_dim=D, seed=D)
    w.q = [torch.randn(3 * ql, q_heads, D, generator=torch.Generator().manual_seed(1)).bfloat16()]
    w.seq_info = table(lens, ql)
    f = Fp8(pkv, w, garbage=False, kscale=2.0)
    c, b, m = R.unpack(f.host(1))
    r = np.random.default_rng(spread)
    b = 127 + r.integers(-spread, spread + 1, b.shape)
    zero = r.random(b.shape) < 0.1
    b[zero] = 0
    c[np.broadcast_to(zero[:, None, :, None], c.shape)] = 0
    set_pool(f, 1, c, b)
    for causal, window in ((True, 0), (True, 33), (False, 50)):
        out, _, err = attend(pkv, f, causal=causal, window=window, max_q=ql, max_kv=max_kv if max_kv > 1 else 400)
        assert err == 0
        check_rows(f, out, w.q[0], causal, window, np.ones(3 * ql, bool))


@pytest.mark.parametrize("D,q_heads,max_kv", SHAPES)
@pytest.mark.parametrize("depth", [90, 115, 120, 129])
def test_a_light_page_that_counts(pkv, D, q_heads, max_kv, depth):
    """Keys of 2^-depth of the largest weight whose V is 2^80, beside V of 2^-110: it is they that the row reads."""
    n, ql = 64, 4
    w = workloads.batched(S=1, max_len=n, lengths=[n], q_heads=q_heads, kv_heads=2, head_dim=D, seed=D)
    q = torch.zeros(ql, q_heads, D)
    q[..., 0] = 16.0
    w.q = [q.bfloat16()]
    w.seq_info = table([n], ql)
    f = Fp8(pkv, w, garbage=False, kscale=1.0)
    k = np.zeros_like(R.values_of(*[x if i == 0 else x[:, None, :, None] for i, x in enumerate(R.unpack(f.host(0))[:2])]))
    page = w.block_table.numpy()[0, 2]
    k[page, :, :, 0] = -depth / (16.0 * w.scale * D2E)
    kb = R.exponent(np.abs(k).max((1, 3)))
    set_pool(f, 0, R.codes_of(k, kb[:, None, :, None]), kb)
    b = np.full_like(R.unpack(f.host(1))[1], 127 - 110)
    b[page] = 127 + 80
    set_pool(f, 1, b=b)
    out, _, err = attend(pkv, f, causal=False, max_q=ql, max_kv=max_kv if max_kv > 1 else n, num_splits=0 if max_kv > 1 else 1)
    assert err == 0
    exponent = float(R.pool_values(f.host(0))[page, 0, 0, 0]) * 16.0 * w.scale * D2E   # (of the code nearest to it)
    check_rows(f, out, w.q[0], False, 0, np.ones(ql, bool), light=[page] if exponent < -126 else [])
