"""Attention of packed prompts over their own rows (attend_prompt) against the
definition in 64 bits.

Tolerances, from the arithmetic: a score is an fp32 sum of D exact products, off by
at most d = D 2^-24 max sum|q k| scale; a weight exp(x - m) by d relative, by
its exp2 (2^-22, and 2^-24 times its argument's size, below 2^-17 for weights that
count) and by its rounding to bf16, half a step, 2^-8; the sum of weights by
d + 2^-18.  |out - ref| <= (2^-8 + 2 d + 2^-16) * sum p|v| / sum p, plus half a step (2^-8
relative) where out is bf16.  lse: d + n 2^-24 + 2^-21 (1 + |lse|).
"""
import numpy as np
import pytest
import torch

from tests import fp8_ref as R8
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def make(seed, rows, hq, hkv, D, fused=False, kscale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, v = [(s * torch.randn(rows, h, D, generator=g, device="cuda")).bfloat16() for h, s in ((hq, 2.0), (hkv, kscale), (hkv, 0.7))]
    if fused:   # slices of one projection's output, with columns of something else behind them
        all_ = torch.cat([q, k, v, torch.full_like(v, float("nan"))], 1)
        q, k, v = all_[:, :hq], all_[:, hq:hq + hkv], all_[:, hq + hkv:hq + 2 * hkv]
    return q, k, v


def table(lens, gap=0, first=0):
    out, at = [], first
    for i, n in enumerate(lens):
        out.append([at, n, i, n])
        at += n + gap
    return torch.tensor(out, dtype=torch.int32).view(-1, 4), at


def run(pkv, q, k, v, si, scale=None, causal=True, window=0, out_dtype=torch.float32, max_len=None, lse=True):
    buf = torch.full((q.numel() + 2048,), 5.0, dtype=out_dtype, device="cuda")
    out = buf[1024:1024 + q.numel()].view(q.shape)
    ls = torch.full(q.shape[:2], 3.0, device="cuda") if lse else None
    err = pkv.new_err_flags()
    m = max_len or max([int(x[1]) for x in si.tolist()] + [1])
    pkv.attend_prompt(q, k, v, si.cuda(), out, err, m, scale or q.shape[2] ** -0.5, causal, window, lse=ls)
    torch.cuda.synchronize()
    assert bool((buf[:1024] == 5).all()) and bool((buf[-1024:] == 5).all()), "write outside the output"
    return out, ls, int(err.item())


def reference(q, k, v, segs, scale, causal, window):
    """out, lse, the sum p|v| / sum p and d of the docstring, per row; rows of no segment 0 and -inf."""
    rows, hq, D = q.shape
    G = hq // k.shape[1]
    out, size = [torch.zeros(rows, hq, D, dtype=torch.float64, device="cuda") for _ in range(2)]
    lse = torch.full((rows, hq), -np.inf, dtype=torch.float64, device="cuda")
    d = torch.zeros(rows, hq, dtype=torch.float64, device="cuda")
    for q0, n, _, _ in segs:
        if n == 0:
            continue
        r = slice(q0, q0 + n)
        qq, kk, vv = [t[r].double().transpose(0, 1) for t in (q, k, v)]
        kk, vv = kk.repeat_interleave(G, 0), vv.repeat_interleave(G, 0)
        i = torch.arange(n, device="cuda")
        hi = i + 1 if causal else torch.full_like(i, n)
        lo = (hi - window).clamp(min=0) if window else torch.zeros_like(i)
        see = (i[None] >= lo[:, None]) & (i[None] < hi[:, None])
        x = (qq @ kk.transpose(1, 2) * scale).masked_fill(~see, -np.inf)
        p = torch.softmax(x, -1)
        out[r], lse[r] = (p @ vv).transpose(0, 1), torch.logsumexp(x, -1).T
        size[r] = (p @ vv.abs()).transpose(0, 1)
        d[r] = ((qq.abs() @ kk.abs().transpose(1, 2)).masked_fill(~see, 0).amax(-1) * abs(scale) * D * 2.0 ** -24).T
    return out, lse, size, d


def check(got, lse, q, k, v, segs, scale=None, causal=True, window=0, rows=None):
    scale = scale or q.shape[2] ** -0.5
    segs = segs.tolist() if torch.is_tensor(segs) else segs
    ref, rl, size, d = reference(q, k, v, segs, scale, causal, window)
    rows = torch.ones(len(q), dtype=torch.bool) if rows is None else rows
    tol = (2.0 ** -8 + 2 * d + 2.0 ** -16)[..., None] * size + 1e-30
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    assert bool(torch.isfinite(got[rows]).all())
    worst = float(((got.double() - ref).abs() / tol)[rows].max())
    assert worst <= 1, f"{worst} times the tolerance"
    if lse is not None:
        gl, el = lse.double()[rows], rl[rows]
        assert torch.equal(torch.isinf(gl), torch.isinf(el))
        fin = torch.isfinite(el)
        n = max([s[1] for s in segs] + [1])
        assert bool(((gl - el).abs()[fin] <= (d[rows] + n * 2.0 ** -24 + 2.0 ** -21 * (1 + el.abs()))[fin]).all())


HEADS = [(1, 1), (3, 3), (7, 1), (8, 1), (12, 3), (32, 8), (40, 8), (64, 1), (100, 1), (128, 1)]


@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_head_groups(pkv, hq, hkv, D):
    si, rows = table([200, 1, 333, 64])
    q, k, v = make(hq + D, rows, hq, hkv, D, fused=hq % 3 == 0)
    out, lse, err = run(pkv, q, k, v, si)
    assert err == 0
    check(out, lse, q, k, v, si)


@pytest.mark.parametrize("D", [8, 40, 64, 72, 80, 128, 136, 200, 256])
@pytest.mark.parametrize("lens", [[1], [2, 0, 3], [127, 128, 129], [31, 32, 33, 1, 255, 256, 257], [1000, 777]])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(pkv, D, lens, causal):
    si, rows = table(lens, first=3)
    q, k, v = make(sum(lens) + D, rows + 5, 8, 2, D, fused=True)
    for dt in (torch.float32, torch.bfloat16):
        out, lse, err = run(pkv, q, k, v, si, causal=causal, out_dtype=dt)
        assert err == 0
        check(out, lse, q, k, v, si, causal=causal)


@pytest.mark.parametrize("window", [1, 2, 63, 64, 128, 200, 1000, 5000])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (3, 3, 64), (16, 1, 256), (1, 1, 128)])
def test_windows(pkv, window, causal, hq, hkv, D):
    si, rows = table([700, 129, 40, 1])
    q, k, v = make(window, rows, hq, hkv, D)
    out, lse, err = run(pkv, q, k, v, si, causal=causal, window=window)
    assert err == 0
    check(out, lse, q, k, v, si, causal=causal, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_long(pkv, D):
    """Many blocks a row: the stage ring goes round, references move, several items a segment."""
    si, rows = table([2500, 1300])
    q, k, v = make(D, rows, 4, 1, D, kscale=1.0)
    k *= torch.linspace(0.1, 2, rows, device="cuda")[:, None, None].bfloat16()   # scores that grow along the keys
    for causal in (True, False):
        out, lse, err = run(pkv, q, k, v, si, causal=causal)
        assert err == 0
        check(out, lse, q, k, v, si, causal=causal)
        again, lse2, _ = run(pkv, q, k, v, si, causal=causal)
        assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_large_bound_and_no_lse(pkv):
    si, rows = table([77, 300])
    q, k, v = make(1, rows, 8, 2, 128)
    a = run(pkv, q, k, v, si)
    b = run(pkv, q, k, v, si, max_len=1 << 30)
    c = run(pkv, q, k, v, si, lse=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and torch.equal(a[0], c[0]) and a[2] == b[2] == c[2] == 0


def test_uncovered_overlapping_and_no_segments(pkv):
    q, k, v = make(2, 300, 8, 2, 128)
    si = torch.tensor([[200, 70, 0, 70], [10, 100, 1, 100], [150, 0, 5, 0]], dtype=torch.int32)
    out, lse, err = run(pkv, q, k, v, si)
    assert err == 0
    check(out, lse, q, k, v, si)
    dead = torch.ones(300, dtype=torch.bool)
    dead[200:270] = dead[10:110] = False
    assert bool((out[dead] == 0).all()) and bool(torch.isinf(lse[dead]).all())
    si[1, 1] = si[1, 3] = 191
    assert run(pkv, q, k, v, si)[2] == 32
    out, lse, err = run(pkv, q, k, v, torch.zeros(0, 4, dtype=torch.int32))
    assert err == 0 and bool((out == 0).all()) and bool(torch.isinf(lse).all())


@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 8, 1), (256, 6, 2)])
@pytest.mark.parametrize("S", [31, 33, 100])
def test_long_tables(pkv, D, hq, hkv, S):
    """Prompts of all lengths side by side and in any order, empty and refused ones between them, rows of none at the end."""
    g = torch.Generator().manual_seed(S)
    lens = [int(x) for x in torch.randint(0, 60, (S,), generator=g)]
    lens[S // 2], lens[S - 1], lens[0] = 700, 301, 0
    si, rows = table(lens, gap=1)
    rows += 40
    si = si[torch.randperm(S, generator=g)]
    bad = int((si[:, 1] == 301).nonzero()[0, 0])
    q, k, v = make(5, rows, hq, hkv, D)
    out, lse, err = run(pkv, q, k, v, si, max_len=5000)
    assert err == 0
    check(out, lse, q, k, v, si)
    si[bad, 3] -= 1
    good = torch.cat([si[:bad], si[bad + 1:]])
    a, b, err = run(pkv, q, k, v, si, max_len=5000)
    live = torch.zeros(rows, dtype=torch.bool)
    for q0, n, _, _ in good.tolist():
        live[q0:q0 + n] = True
    assert err == 1 and torch.equal(a[live], out[live]) and torch.equal(b[live], lse[live])
    assert bool((a[~live] == 0).all()) and bool(torch.isinf(b[~live]).all())


def test_no_rows(pkv):
    q, k, v = make(7, 0, 8, 2, 128)
    for si in (torch.zeros(0, 4, dtype=torch.int32), torch.zeros(3, 4, dtype=torch.int32)):
        err = pkv.new_err_flags()
        pkv.attend_prompt(q, k, v, si.cuda(), torch.empty_like(q), err, 5, 0.1)
        assert int(err.item()) == 0


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (256, 4, 1)])
def test_many_bad_items(pkv, D, hq, hkv):
    """More items to run again than the list holds, after others with a bad row in one warp only."""
    rows, G = 160 * 190, hq // hkv
    q, k, v = make(8, rows, hq, hkv, D)
    si, _ = table([190] * 160)
    clean, lse0, _ = run(pkv, q, k, v, si)
    bad = v.clone()
    i = torch.arange(rows, device="cuda")
    n, at = i // 190, i % 190
    bad[(at == 189) & (n % 7 != 0), 0, 5] = float("inf")   # seen by the last row alone
    bad[(at == 0) & (n % 7 == 3), hkv - 1, 2] = float("nan")  # and by all
    out, lse, err = run(pkv, q, k, bad, si)
    last = torch.zeros_like(out, dtype=torch.bool)
    last[(at == 189) & (n % 7 != 0), :G, 5] = True
    every = torch.zeros_like(last)
    every[n % 7 == 3, (hkv - 1) * G:, 2] = True
    assert err == 0 and torch.equal(lse, lse0) and torch.equal(out[~(last | every)], clean[~(last | every)])
    assert bool(out[every].isnan().all()) and bool((out[last & ~every] == float("inf")).all())


@pytest.mark.parametrize("D,hq,hkv", [(128, 8, 2), (256, 4, 1)])
def test_the_same_rows_in_many_segments(pkv, D, hq, hkv):
    """An error, but every row of every segment is computed all the same."""
    q, k, v = make(6, 640, hq, hkv, D)
    si = torch.tensor([[0, 640, 0, 640]], dtype=torch.int32)
    one = run(pkv, q, k, v, si)
    many = run(pkv, q, k, v, torch.cat([si] * 40 + [torch.tensor([[0, 0, 0, 0]], dtype=torch.int32)] * 3))
    assert many[2] == 32 and torch.equal(one[0], many[0]) and torch.equal(one[1], many[1])


@pytest.mark.parametrize("seg,bit", [((50, 10, 0, 11), 1), ((50, 10, 0, 9), 1), ((-1, 20, 0, 20), 1), ((90, 20, 0, 20), 1), ((50, -3, 0, -3), 1),
                                     ((2 ** 31 - 5, 10, 0, 10), 1), ((50, 45, 0, 45), 16)])
@pytest.mark.parametrize("D", [128, 256])
def test_refused_segments_read_zero(pkv, seg, bit, D):
    q, k, v = make(3, 100, 4, 2, D)
    si = torch.tensor([seg, [0, 40, 9, 40]], dtype=torch.int32)
    out, lse, err = run(pkv, q, k, v, si, max_len=40)
    assert err == bit
    check(out, lse, q, k, v, si[1:])
    assert bool((out[40:] == 0).all()) and bool(torch.isinf(lse[40:]).all())


@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 2), (128, 8, 2), (128, 3, 3), (256, 4, 1), (80, 16, 1)])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 100])
def test_a_bad_key_reaches_only_rows_that_see_it(pkv, D, hq, hkv, value, window):
    """In V: the column, of the rows of its kv head that see the key.  In K (a NaN): those rows whole.  All others stay bit for bit."""
    lens = [300, 150, 40]
    si, rows = table(lens)
    q, k, v = make(4, rows, hq, hkv, D)
    clean, lse0, _ = run(pkv, q, k, v, si, window=window)
    G = hq // hkv
    for key in (0, 5, 128, 200, 299, 300, 449, 450, 489):
        seg = next(s for s in si.tolist() if s[0] <= key < s[0] + s[1])
        i = torch.arange(rows, device="cuda")
        sees = (i >= key) & (i < seg[0] + seg[1]) & ((i < key + window) if window else True)
        bad = v.clone()
        bad[key, hkv - 1, 3] = value
        out, lse, err = run(pkv, q, k, bad, si, window=window)
        want = torch.zeros_like(out, dtype=torch.bool)
        want[sees, (hkv - 1) * G:, 3] = True
        assert err == 0 and torch.equal(lse, lse0)
        assert torch.equal(out[~want], clean[~want])
        if np.isnan(value):
            assert bool(out[want].isnan().all())
        else:   # the weight times the infinity; a weight that vanished makes it NaN
            assert not bool(torch.isfinite(out[want]).any()) and bool((out[want].isnan() | (out[want] == value)).all())
            assert bool((out[key, (hkv - 1) * G:, 3] == value).all())
        if np.isnan(value):
            bad = k.clone()
            bad[key, hkv - 1, 3] = value
            out, lse, err = run(pkv, q, bad, v, si, window=window)
            want = torch.zeros_like(out, dtype=torch.bool)
            want[sees, (hkv - 1) * G:] = True
            assert err == 0 and torch.equal(out[~want], clean[~want]) and bool(out[want].isnan().all())
            assert torch.equal(lse[~want[..., 0]], lse0[~want[..., 0]]) and bool(lse[want[..., 0]].isnan().all())


def test_bad_rows_everywhere(pkv):
    """A prompt whose second half is NaN leaves the first half as it is; so does one beside a prompt of NaN."""
    si, rows = table([400, 300])
    q, k, v = make(5, rows, 8, 2, 128)
    clean, lse0, _ = run(pkv, q, k, v, si)
    bad = v.clone()
    bad[200:400] = float("nan")
    out, lse, err = run(pkv, q, k, bad, si)
    assert err == 0 and torch.equal(out[:200], clean[:200]) and torch.equal(out[400:], clean[400:]) and bool(out[200:400].isnan().all())
    bad = [t.clone() for t in (q, k, v)]
    for t in bad:
        t[400:] = float("nan")
    out, lse, err = run(pkv, *bad, si)
    assert err == 0 and torch.equal(out[:400], clean[:400]) and torch.equal(lse[:400], lse0[:400]) and bool(out[400:].isnan().all())


def test_magnitudes(pkv):
    si, rows = table([150, 33])
    q, k, v = make(6, rows, 4, 2, 128)
    base, lse0, _ = run(pkv, q, k, v, si)
    for e in (-60, -20, 20, 60):
        out, lse, err = run(pkv, (q.float() * 2.0 ** e).bfloat16(), k, v, si, scale=128 ** -0.5 * 2.0 ** -e)
        assert err == 0 and torch.equal(out, base) and torch.equal(lse, lse0)
    # scores far apart: one key takes all
    big = (k.float() * 100).bfloat16()
    out, lse, err = run(pkv, q, big, v, si)
    assert err == 0
    check(out, lse, q, big, v, si)


def test_captured_on_a_side_stream(pkv):
    """One capture serves the tables and rows that are there at each replay; two graphs may run at once."""
    q, k, v = make(7, 600, 8, 2, 128)
    sis = [table(x)[0] for x in ([300, 200, 100], [1, 16, 17], [600, 0, 0], [128, 129, 256])]
    si, err = sis[0].cuda(), pkv.new_err_flags()
    outs = [torch.empty(600, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for s, out in zip(streams, outs):
        with torch.cuda.stream(s):
            pkv.attend_prompt(q, k, v, si, out, err, 600, 128 ** -0.5)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                pkv.attend_prompt(q, k, v, si, out, err, 600, 128 ** -0.5)
            graphs.append(g)
    for x in sis:
        si.copy_(x)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and int(err.item()) == 0
        check(outs[0], None, q, k, v, x)


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_a_prompt_and_the_steps_after_it(pkv, kind):
    """What a user does with them: rows of text and images are normalised, turned on three axes and appended, attended
    over as a prompt, and then decoded over the cache, token by token, with the same results as attention over the cache's own values."""
    D, Hq, Hkv, lens, steps = 128, 8, 2, [150, 37], 5
    si, rows = table(lens)
    si = si.cuda()
    nb = [16, 8]
    dt = torch.bfloat16 if kind == "bf16" else torch.float8_e4m3fn
    shape = (24, 16, Hkv, D) if kind == "bf16" else (24, Hkv, 16 * D + 16)
    pools = [torch.zeros(shape, dtype=torch.uint8 if kind == "fp8" else dt, device="cuda").view(dt) for _ in range(2)]
    bt = torch.full((2, 16), -1, dtype=torch.int32)
    bt[0], bt[1, :8] = torch.arange(8, 24), torch.arange(8)
    cache = pkv.PagedKVCache([pools[0]], [pools[1]], bt.cuda())
    g = torch.Generator(device="cuda").manual_seed(9)
    wq, wk = [(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).bfloat16() for _ in range(2)]
    rope = pkv.Rope(pkv.rope_inv_freq(D)[0], q_weight=wq, k_weight=wk, axes=pkv.rope_axes((22, 21, 21), True))
    qkv = torch.randn(rows, Hq + 2 * Hkv, D, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.randint(0, 500, (rows, 3), generator=g, device="cuda", dtype=torch.int32)
    turned_q, turned_k = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device="cuda"), torch.empty(rows, Hkv, D, dtype=torch.bfloat16, device="cuda")
    pkv.norm_rope(rope, q, k, pos, turned_q, turned_k)
    err, held = pkv.new_err_flags(), [torch.empty_like(turned_k) for _ in range(2)]
    pkv.norm_rope_append(cache, 0, rope, q, k, v, si, None, err, positions=pos, k_out=held[0], v_out=held[1])
    assert torch.equal(q, turned_q)
    out = torch.empty(rows, Hq, D, dtype=torch.bfloat16, device="cuda")
    pkv.attend_prompt(q, turned_k, v, si, out, err, 150, D ** -0.5)
    assert int(err.item()) == 0
    check(out, None, turned_q, turned_k, v, si)
    if kind == "bf16":   # the same rows through the cache
        over = torch.empty(rows, Hq, D, device="cuda")
        pkv.attend_varlen(cache, 0, turned_q, si, over, err, 150, 150, D ** -0.5, causal=True)
        check(over, None, turned_q, turned_k, v, si)
    keys = [[held[0][s:s + n], held[1][s:s + n]] for s, n, _, _ in si.tolist()]
    step = torch.tensor([[0, 1, 0, lens[0] + 1], [1, 1, 1, lens[1] + 1]], dtype=torch.int32, device="cuda")
    for t in range(steps):
        a, b, c = [torch.randn(2, h, D, generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv)]
        p3 = torch.full((2, 3), 500 + t, dtype=torch.int32, device="cuda")
        ko, vo = torch.empty_like(b), torch.empty_like(c)
        pkv.norm_rope_append(cache, 0, rope, a, b, c, step, None, err, positions=p3, k_out=ko, v_out=vo)
        one, lse = torch.empty(2, Hq, D, device="cuda"), torch.empty(2, Hq, device="cuda")
        pkv.attend_varlen(cache, 0, a, step, one, err, 1, 256, D ** -0.5, lse=lse)
        for s in range(2):
            n = lens[s] + t + 1
            page = bt[s, :(n + 15) // 16].long().cuda()
            kk, vv = [(torch.tensor(R8.pool_values(x.view(torch.uint8)[page].cpu().numpy())) if kind == "fp8" else x[page].double().cpu())
                      .reshape(-1, Hkv, D)[:n].repeat_interleave(Hq // Hkv, 1) for x in pools]
            x = torch.einsum("hd,nhd->hn", a[s].double().cpu(), kk) * D ** -0.5
            ref = torch.einsum("hn,nhd->hd", torch.softmax(x, -1), vv)
            assert float((one[s].double().cpu() - ref).abs().max()) <= 2e-3 * max(1.0, float(vv.abs().max()))
            # what the cache holds is the rows as they came out, but that an 8-bit page's scale may have grown since
            mine = torch.cat([keys[s][1], vo[s:s + 1]]).double().cpu()
            far = (mine.repeat_interleave(Hq // Hkv, 1) - vv).abs()
            assert float(far.max()) <= (0 if kind == "bf16" else 2.0 ** -12 * float(vv.abs().max()))
            keys[s] = [torch.cat([keys[s][0], ko[s:s + 1]]), torch.cat([keys[s][1], vo[s:s + 1]])]
        pkv.advance(step)
    assert int(err.item()) == 0
