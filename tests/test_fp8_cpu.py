"""The 8-bit cache: what needs no GPU.  The reference of the format itself, and refusals before any launch."""
import ctypes

import numpy as np
import pytest
import torch

from tests import fp8_ref as R


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from paged_kv_decode_13_gb300 import _lib
    return _lib


@pytest.fixture(scope="module")
def pkv(lib):
    import paged_kv_decode_13_gb300 as m
    return m


# ---------------------------------------------------------------- the format

@pytest.mark.parametrize("D", [64, 128, 256])
def test_block_places_are_a_bijection(D):
    at = R.places(D)
    assert sorted(at.ravel()) == list(range(16 * D))
    assert (at // D == np.arange(16)[:, None]).all()   # a token's row is contiguous
    r = np.random.default_rng(0)
    c, b, m = r.integers(0, 256, (3, 16, 2, D)).astype(np.uint8), r.integers(0, 247, (3, 2)), r.integers(0, 65536, (3, 2))
    back = R.unpack(R.pack(c, b, m))
    assert all((x == y).all() for x, y in zip(back, (c, b, m)))


def test_codes_are_e4m3():
    """The numbers of the codes, and the rounding, against torch's own cast."""
    c = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    v = c.view(torch.float8_e4m3fn).double().numpy()
    ok = ~np.isnan(v)
    assert (R.values_of(c.numpy(), 127)[ok] == v[ok]).all() and list(c.numpy()[~ok]) == [127, 255]
    x = torch.cat([torch.randn(4000) * s for s in (1e-4, 1e-2, 1.0, 100.0)] + [torch.tensor(R.FINITE), torch.tensor((R.FINITE[1:] + R.FINITE[:-1]) / 2)]).float()
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (R.codes_of(x.double().numpy(), 127) == want).all()


def test_exponent_is_the_smallest_that_fits():
    for a in (1.0, 448.0, 449.0, 1.75, 1.7578125, 1e-30, 3.3e38, 2.0 ** -133, np.inf):
        b = int(R.exponent(a))
        assert 1 <= b <= 246 and (a <= 448.0 * R.scale(b) or b == 246) and (b == 1 or a > 448.0 * R.scale(b - 1))
    assert R.exponent(0.0) == 0 and R.scale(0) == 0 and R.exponent(448.0) == 127 and R.exponent(450.0) == 128


def test_moving_a_page_to_a_larger_scale():
    """Codes that follow a scale stay what they were down to 2^-6 of it, and are off by at most 2^-10 of it below."""
    D, r = 64, np.random.default_rng(1)
    block = np.zeros(16 * D + 16, np.uint8)
    a = r.normal(size=D)
    block, held = R.write_page(block, {0: a}, [])
    before = held[0]
    assert (np.abs(before - a) <= np.maximum(2.0 ** -4 * np.abs(a), 2.0 ** -10 * R.scale(int(block[16 * D])))).all()
    for step in range(1, 12):
        block, _ = R.write_page(block, {step: a * 2.0 ** step}, list(range(step)))
        s = R.scale(int(block[16 * D]))
        now = R.pool_values(block[None, None])[0, 0, 0]
        big = np.abs(before) >= s * 2.0 ** -6
        assert (now[big] == before[big]).all() and (np.abs(now - before) <= step * 2.0 ** -10 * s).all()


# ---------------------------------------------------------------- refusals at the C entry points

def _desc(lib, **kw):
    fake = (ctypes.c_void_p * 1)(0x1000)
    d = lib.CacheDesc(num_layers=1, kv_heads=2, head_dim=64, dtype=lib.FP8, num_blocks=32, max_seqs=1, max_blocks_per_seq=32, ring_rows=0,
                      k=ctypes.cast(fake, ctypes.c_void_p), v=ctypes.cast(fake, ctypes.c_void_p), block_table=0x2000, bucket=512, generation=0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d, fake


def _rows(lib, **kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, q_out=0x40000, q_stride=512, k_stride=128, v_stride=128, q_out_stride=512,
             k_out_stride=128, v_out_stride=128, q_heads=8, total_rows=4, positions=None)
    a.update(kw)
    return lib.RowsDesc(**a)


def _append(lib, desc, rope=None, rows=None, si=0x60000, S=1, window=0, err=0x70000, layer=0):
    d, keep = desc
    return lib.lib.pkv_norm_rope_append(ctypes.byref(d), layer, ctypes.byref(rope) if rope else None, ctypes.byref(rows) if rows else None,
                                        si, S, window, err, None)


@pytest.mark.parametrize("field,value,status", [("head_dim", 80, -2), ("head_dim", 32, -2), ("head_dim", 192, -2), ("kv_heads", 0, -1),
                                                ("num_blocks", 0, -1), ("ring_rows", 24, -1), ("dtype", 4, -2)])
def test_cache_refusals(lib, field, value, status):
    assert _append(lib, _desc(lib, **{field: value}), rows=_rows(lib)) == status
    d, keep = _desc(lib, **{field: value})
    assert lib.lib.pkv_attend_varlen(ctypes.byref(d), 0, 0x4000, 8, 1, 0x5000, 1, 1, 512, 0, 0.125, 0, 0, 0x6000, None, None, 0,
                                     0x7000, 0, None) == status
    assert lib.lib.pkv_to_contiguous(ctypes.byref(d), 0, 4, 0x4000, 0x4000, None) == status


def test_append_refusals(lib):
    for bad in (dict(q=0x10008), dict(k=0x20004), dict(v=None), dict(k=None), dict(q_out=None), dict(q=None), dict(q_heads=0), dict(q_stride=504),
                dict(k_stride=120), dict(v_stride=130), dict(k_out=0x40002), dict(positions=0x50002), dict(total_rows=-1)):
        assert _append(lib, _desc(lib), rows=_rows(lib, **bad)) == -1, bad
    for bad in (dict(si=None), dict(si=0x60008), dict(S=-1), dict(window=-1), dict(err=None), dict(layer=1), dict(layer=-1)):
        assert _append(lib, _desc(lib), rows=_rows(lib), **bad) == -1, bad
    assert _append(lib, _desc(lib), rows=_rows(lib), S=0) == 0


def test_copying_calls(lib):
    d, keep = _desc(lib)
    e, keep2 = _desc(lib, bucket=1024)
    L, ref = lib.lib, ctypes.byref(d)
    assert L.pkv_seq_clone(ref, 0, 0, 4, 0x7000, None) == -2
    assert L.pkv_resize_bucket(ref, ctypes.byref(e), 10, None) == -2
    assert L.pkv_load_prefix(ref, None, None, 5, 128, 64, None) == -2
    for bad, st in (((0, 513, 0x4000, 0x4000), -4), ((0, -1, 0x4000, 0x4000), -4), ((1, 4, 0x4000, 0x4000), -1), ((0, 4, None, 0x4000), -1), ((0, 4, 0x4000, 0x4008), -1)):
        assert L.pkv_to_contiguous(ref, *bad, None) == st
    assert L.pkv_to_contiguous(ref, 0, 0, None, None, None) == 0
    assert L.pkv_rewind(ref, 0x5000, 0, None, 0, 0x7000, None) == 0


def test_attention_refusals(lib):
    d, keep = _desc(lib)
    L, ref = lib.lib, ctypes.byref(d)

    def attend(**kw):
        a = dict(layer=0, q=0x4000, hq=8, rows=1, si=0x5000, S=1, mq=1, mk=512, ns=0, scale=1.0, causal=0, window=0, out=0x6000,
                 lse=None, err=0x7000, flags=0)
        a.update(kw)
        return L.pkv_attend_varlen(ref, a["layer"], a["q"], a["hq"], a["rows"], a["si"], a["S"], a["mq"], a["mk"], a["ns"], a["scale"],
                                   a["causal"], a["window"], a["out"], a["lse"], None, 0, a["err"], a["flags"], None)

    for bad in (dict(hq=3), dict(hq=0), dict(layer=1), dict(q=0x4004), dict(q=None), dict(si=0x5004), dict(si=None), dict(err=None), dict(out=None),
                dict(out=0x6004), dict(lse=0x6002), dict(causal=2), dict(window=-1), dict(ns=17), dict(mq=0), dict(mk=0), dict(S=65536), dict(rows=-1)):
        assert attend(**bad) == -1, bad
    assert attend(rows=0, S=0) == 0


def test_workspace_bounds(lib):
    d, keep = _desc(lib, kv_heads=64)
    size = lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 512, 512, 1, 1 << 20, 0, 0)
    assert 0 < size < 25 << 20
    assert lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 512, 512, 1, (1 << 62), 0, 0) == size
    d, keep = _desc(lib)
    assert lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 8, 1, 1, 16, 0, 0) == 0


# ---------------------------------------------------------------- refusals of the binding

def test_pools(pkv):
    bt = torch.zeros(1, 4, dtype=torch.int32)
    pool = torch.zeros(4, 2, 16 * 64 + 16, dtype=torch.uint8).view(torch.float8_e4m3fn)
    c = pkv.PagedKVCache([pool], [pool.clone()], bt)
    assert (c.kv_heads, c.head_dim, c.row_dtype, c.dtype) == (2, 64, torch.bfloat16, torch.float8_e4m3fn)
    for bad in (pool.view(4, 2, 65, 16), pool[:, :, :16].contiguous(), torch.zeros(4, 2, 1035, dtype=torch.uint8).view(torch.float8_e4m3fn)):
        with pytest.raises(ValueError):
            pkv.PagedKVCache([bad], [bad], bt)
    a = pkv.PagedKVCache.allocate(2, 3, 128, 512, dtype=torch.float8_e4m3fn, device="cpu")
    assert a.k[0].shape == (32, 3, 16 * 128 + 16) and a.reusable_for(2, 3, 128, torch.float8_e4m3fn, 512)
    assert not a.reusable_for(2, 3, 128, torch.uint8, 512)


def test_rows_and_tensors(pkv):
    cache = pkv.PagedKVCache.allocate(1, 2, 64, 512, dtype=torch.float8_e4m3fn, device="cpu")
    si, err = torch.tensor([[0, 2, 0, 2]], dtype=torch.int32), pkv.new_err_flags("cpu")
    q, out = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.empty(2, 4, 64)
    good = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for k, v in ((good.float(), good), (good, good.half()), (good, good[:1]), (good.to(torch.float8_e4m3fn), good)):
        with pytest.raises(ValueError):
            pkv.append(cache, 0, k, v, si, err)
        with pytest.raises(ValueError):
            pkv.norm_rope_append(cache, 0, None, None, k, v, si, None, err)
        for fn in (pkv.append_attend, pkv.append_attend_noalloc):
            with pytest.raises(ValueError):
                fn(cache, 0, q, k, v, si, out, err, 2, 512, 0.125)
    for bq, bo, bl in ((q.float(), out, None), (q, out.half(), None), (q, out[:1], None), (q, out, torch.empty(2, 3)), (q, out, torch.empty(2, 4).bfloat16())):
        with pytest.raises(ValueError):
            pkv.attend_varlen(cache, 0, bq, si, bo, err, 2, 512, 0.125, lse=bl)
    kv = torch.empty(2, 5, 64, dtype=torch.bfloat16)
    for a, b in ((kv.float(), kv), (kv, kv[:, :4]), (kv[:, ::2], kv)):
        with pytest.raises(ValueError):
            pkv.to_contiguous(cache, 0, 5, a, b)
