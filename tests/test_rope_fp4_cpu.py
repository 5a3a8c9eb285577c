"""Norm + rotary + append and the 4-bit cache: what needs no GPU.  Host
functions, struct layouts, refusals before any launch, and the reference of the
format itself."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import fp4_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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
@pytest.mark.parametrize("is_v", [False, True])
def test_block_places_are_a_bijection(D, is_v):
    at, nib, sc = R.places(D, is_v)
    assert len(set((2 * at + nib).ravel())) == 16 * D and at.max() == 8 * D - 1
    assert sorted(sc.ravel()) == list(range(8 * D, 9 * D))
    codes = np.random.default_rng(0).integers(0, 16, (3, 16, 2, D)).astype(np.uint8)
    scales = np.random.default_rng(1).integers(0, 256, (3, 16, 2, D // 16)).astype(np.uint8)
    back = R.unpack(R.pack(codes, scales, is_v), is_v)
    assert (back[0] == codes).all() and (back[1] == scales).all()


def test_quantise_reference():
    # ties go to the even code: with s = 1 (max 6) each border between codes
    x = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, 0, -0.0, 0.26, 0.74, 2.51, 5.01])
    c, s = R.quantise(x)
    assert s[0] == 0x78 and R.SCALES[0x78] == 1.0
    assert list(R.values(c, s)) == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, 0, 0, 0.5, 0.5, 3, 6]
    # the relative error of a value is at most half a step of its group's scale, a sixteenth for the scale itself
    g = np.random.default_rng(0).normal(size=(1000, 64))
    v = R.values(*R.quantise(g))
    top = np.abs(g.reshape(1000, 4, 16)).max(-1, keepdims=True)
    assert (np.abs((v - g).reshape(1000, 4, 16)) <= top / 6 * (1 + 1 / 16) + 1e-12).all()
    # a group with a NaN reads NaN, an infinity saturates, tiny groups vanish
    assert np.isnan(R.values(*R.quantise(np.r_[np.nan, np.ones(15)]))).all()
    assert R.values(*R.quantise(np.r_[np.inf, np.zeros(15)]))[0] == 6 * 10240
    assert (R.values(*R.quantise(np.full(16, 1e-6))) == 0).all()


# ---------------------------------------------------------------- host functions

@pytest.mark.parametrize("rot", [2, 24, 64, 128, 256])
def test_inv_freq_scalings(pkv, rot):
    i = np.arange(rot // 2)
    f = 10000.0 ** (-2.0 * i / rot)
    got, m = pkv.rope_inv_freq(rot, 10000.0)
    assert m == 1.0 and np.allclose(got.numpy(), f, rtol=1e-14)
    got, m = pkv.rope_inv_freq(rot, 10000.0, "linear", factor=8.0)
    assert m == 1.0 and np.allclose(got.numpy(), f / 8, rtol=1e-14)
    if rot > 2:
        got, m = pkv.rope_inv_freq(rot, 10000.0, "ntk", factor=4.0)
        assert m == 1.0 and np.allclose(got.numpy(), (10000.0 * 4.0 ** (rot / (rot - 2))) ** (-2.0 * i / rot), rtol=1e-13)
        # its slowest pair is stretched by the factor, its fastest kept
        assert got[0] == 1.0 and np.isclose(got[-1], f[-1] / 4, rtol=1e-12)
    got, m = pkv.rope_inv_freq(rot, 10000.0, "yarn", factor=16.0, trained_len=8192)
    assert np.isclose(m, 0.1 * np.log(16) + 1)
    turns = 8192 * f / (2 * np.pi)
    got = got.numpy()
    assert ((got <= f * (1 + 1e-14)) & (got >= f / 16 * (1 - 1e-14))).all()
    if rot >= 64:
        assert np.allclose(got[turns > 40], f[turns > 40]) and np.allclose(got[turns < 0.7], f[turns < 0.7] / 16)


def test_turns_are_exact_fractions(lib):
    inv = np.array([1.0, 10000.0 ** -0.5, 1e-4, 0.0, 7.5, -0.3, 2 * np.pi])
    turns = np.zeros(len(inv), np.uint64)
    assert lib.lib.pkv_rope_turns(inv.ctypes.data, len(inv), turns.ctypes.data) == 0
    for f, t in zip(inv, turns):
        want = (f / (2 * np.pi)) % 1.0
        d = abs(int(t) / 2.0 ** 64 - want)
        assert min(d, 1 - d) < 2.0 ** -52
    bad = np.array([1.0, np.inf])
    assert lib.lib.pkv_rope_turns(bad.ctypes.data, 2, turns.ctypes.data) == -1
    assert lib.lib.pkv_rope_turns(None, 1, turns.ctypes.data) == -1
    assert lib.lib.pkv_rope_turns(None, 0, None) == 0


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1, 0, 32, 1), (7, 1e4, 0, 1, 0, 32, 1), (64, 1.0, 0, 1, 0, 32, 1), (64, float("nan"), 0, 1, 0, 32, 1),
    (64, 1e4, 4, 1, 0, 32, 1), (64, 1e4, -1, 1, 0, 32, 1), (64, 1e4, 1, 0.5, 0, 32, 1), (64, 1e4, 1, float("inf"), 0, 32, 1),
    (2, 1e4, 2, 2, 0, 32, 1), (64, 1e4, 3, 2, 0, 32, 1), (64, 1e4, 3, 2, 4096, 1, 32), (64, 1e4, 3, 2, 4096, 32, 0),
])
def test_inv_freq_refusals(lib, args):
    out, m = np.zeros(128), ctypes.c_double()
    assert lib.lib.pkv_rope_inv_freq(*args, out.ctypes.data, ctypes.addressof(m)) == -1


# ---------------------------------------------------------------- layouts and refusals at the C entry points

@pytest.mark.parametrize("struct,mirror", [("pkv_rope", "RopeDesc"), ("pkv_rows", "RowsDesc")])
def test_struct_layouts_match_compiled_header(lib, tmp_path, struct, mirror):
    m = getattr(lib, mirror)
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "pkv.h"\n'
                   f'int main(void) {{ printf("%zu", sizeof({struct}));\n'
                   + "".join(f'  printf(" %zu", offsetof({struct}, {n}));\n' for n, _ in m._fields_) + "  return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(m)] + [getattr(m, n).offset for n, _ in m._fields_]


def _desc(lib, **kw):
    fake = (ctypes.c_void_p * 2)(0x1000, 0x2000)
    d = lib.CacheDesc(num_layers=1, kv_heads=2, head_dim=64, dtype=lib.FP4, num_blocks=32, max_seqs=1,
                      max_blocks_per_seq=32, ring_rows=0, reserved0=0, k=ctypes.cast(fake, ctypes.c_void_p),
                      v=ctypes.cast(ctypes.byref(fake, 8), ctypes.c_void_p), block_table=0x3000, bucket=512, generation=0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d, fake


def _rows(lib, **kw):
    a = dict(q=0x10000, k=0x20000, v=0x30000, q_out=0x40000, q_stride=512, k_stride=128, v_stride=128, q_out_stride=512,
             k_out_stride=128, v_out_stride=128, q_heads=8, total_rows=4, positions=None)
    a.update(kw)
    return lib.RowsDesc(**a)


def _rope(lib, **kw):
    a = dict(turns=0x50000, rot_dim=64, interleaved=0, mscale=1.0, eps=1e-6, q_weight=None, k_weight=None)
    a.update(kw)
    return lib.RopeDesc(**a)


def _append(lib, cache=None, rope=None, rows=None, si=0x60000, S=1, window=0, err=0x70000, layer=0):
    d, keep = cache or _desc(lib)
    return lib.lib.pkv_norm_rope_append(ctypes.byref(d), layer, ctypes.byref(rope) if rope else None, ctypes.byref(rows) if rows else None,
                                        si, S, window, err, None)


@pytest.mark.parametrize("field,value,status", [
    ("head_dim", 80, -2), ("head_dim", 32, -2), ("head_dim", 192, -2), ("dtype", 3, -2), ("kv_heads", 0, -1),
    ("num_blocks", 0, -1), ("ring_rows", 24, -1),
])
def test_fp4_cache_refusals(lib, field, value, status):
    assert _append(lib, cache=_desc(lib, **{field: value}), rows=_rows(lib)) == status
    d, keep = _desc(lib, **{field: value})
    assert lib.lib.pkv_attend_varlen(ctypes.byref(d), 0, 0x4000, 8, 1, 0x5000, 1, 1, 512, 0, 0.125, 0, 0, 0x6000, None, None, 0,
                                     0x7000, 0, None) == status


def test_copying_calls_refuse_fp4(lib):
    d, keep = _desc(lib)
    e, keep2 = _desc(lib, bucket=1024)
    L, ref = lib.lib, ctypes.byref(d)
    assert L.pkv_seq_clone(ref, 0, 0, 4, 0x7000, None) == -2
    assert L.pkv_resize_bucket(ref, ctypes.byref(e), 10, None) == -2
    assert L.pkv_load_prefix(ref, None, None, 5, 128, 64, None) == -2
    assert L.pkv_to_contiguous(ref, 0, 4, 0x4000, 0x4000, None) == -2
    assert L.pkv_rewind(ref, 0x5000, 0, None, 0, 0x7000, None) == 0  # only reads the ring rule


def test_fp4_attention_refusals(lib):
    d, keep = _desc(lib)
    L, ref = lib.lib, ctypes.byref(d)

    def attend(**kw):
        a = dict(layer=0, q=0x4000, hq=8, rows=1, si=0x5000, S=1, mq=1, mk=512, ns=0, scale=1.0, causal=0, window=0, out=0x6000,
                 lse=None, err=0x7000, flags=0)
        a.update(kw)
        return L.pkv_attend_varlen(ref, a["layer"], a["q"], a["hq"], a["rows"], a["si"], a["S"], a["mq"], a["mk"], a["ns"], a["scale"],
                                   a["causal"], a["window"], a["out"], a["lse"], None, 0, a["err"], a["flags"], None)

    for bad in (dict(hq=3), dict(hq=0), dict(layer=1), dict(layer=-1), dict(q=0x4004), dict(q=None), dict(si=0x5004), dict(si=None),
                dict(err=None), dict(out=None), dict(out=0x6004), dict(lse=0x6002), dict(causal=2), dict(window=-1), dict(ns=17),
                dict(ns=-1), dict(mq=0), dict(mk=0), dict(S=-1), dict(S=65536), dict(rows=-1)):
        assert attend(**bad) == -1, bad
    assert attend(rows=0, S=0) == 0
    assert L.pkv_append_attend(ref, 0, 0x4000, None, None, 8, 1, 0x5000, 1, 1, 512, 0, 1.0, 0, 0, 0x6000, None, None, 0, 0x7000, 0, None) == -1
    assert L.pkv_append_attend(ref, 0, 0x4000, 0x8000, 0x9000, 8, 1, 0x5000, 1, 1, 512, 0, 1.0, 0, 0, 0x6004, None, None, 0, 0x7000, 0, None) == -1
    assert L.pkv_attend_workspace_bytes(ref, 8, 4, 1, 512, 0, 0) == 0
    assert L.pkv_attend_workspace_bytes(ref, 3, 4, 1, 512, 0, 0) == -1


def test_bf16_output_is_for_fp4_only(lib):
    d, keep = _desc(lib, dtype=lib.BF16)
    assert lib.lib.pkv_attend_varlen(ctypes.byref(d), 0, 0x4000, 8, 1, 0x5000, 1, 1, 512, 0, 0.125, 0, 0, 0x6000, None, None, 0,
                                     0x7000, lib.FLAG_OUT_BF16, None) == -2


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_append_refusals(lib, dtype):
    def go(rope=None, cache=None, **kw):
        call = {k: kw.pop(k) for k in ("si", "S", "window", "err", "layer") if k in kw}
        return _append(lib, cache=cache or _desc(lib, dtype=dtype), rope=rope, rows=_rows(lib, **kw), **call)

    for bad in (dict(q=0x10008), dict(k=0x20004), dict(v=None), dict(k=None), dict(q_out=None), dict(q=None), dict(q_heads=0),
                dict(q_stride=504), dict(k_stride=120), dict(v_stride=130), dict(q_out=0x40002), dict(k_out=0x40002),
                dict(v_out=0x40001), dict(k_out=0x40000, k_out_stride=64), dict(positions=0x50002), dict(total_rows=-1),
                dict(q_heads=-1), dict(si=None), dict(si=0x60008), dict(S=-1), dict(window=-1), dict(err=None), dict(layer=1),
                dict(layer=-1)):
        assert go(**bad) == -1, bad
    for bad in (dict(rot_dim=63), dict(rot_dim=-2), dict(rot_dim=66), dict(interleaved=2), dict(turns=None), dict(turns=0x50004),
                dict(q_weight=0x50008), dict(k_weight=0x50002)):
        assert go(rope=_rope(lib, **bad)) == -1, bad
    assert _append(lib, cache=_desc(lib, dtype=dtype)) == -1          # no rows
    assert go(S=0) == 0                                                 # nothing to place, nothing launched


def test_norm_rope_refusals(lib):
    L = lib.lib

    def go(rope=None, dtype=0, dim=64, kv=2, **kw):
        a = dict(v=None, k_out=0x80000, positions=0x90000)
        a.update(kw)
        return L.pkv_norm_rope(ctypes.byref(rope or _rope(lib)), dtype, dim, kv, ctypes.byref(_rows(lib, **a)), None)

    assert L.pkv_norm_rope(None, 0, 64, 2, ctypes.byref(_rows(lib, v=None, k_out=0x80000, positions=0x90000)), None) == -1
    for bad in (dict(v=0x30000), dict(v_out=0x30000), dict(k_out=None), dict(k=None), dict(q=None), dict(positions=None),
                dict(q=None, k=None, q_out=None, k_out=None, q_heads=0), dict(kv=-1), dict(q_stride=100)):
        assert go(**bad) == -1, bad
    assert go(dtype=2) == -2 and go(dim=60) == -2 and go(dim=264) == -2 and go(dim=0) == -2
    assert go(total_rows=0) == 0


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refusals(pkv):
    cpu = dict(device="cpu")
    f = pkv.rope_inv_freq(64)[0]
    with pytest.raises(ValueError):
        pkv.rope_inv_freq(64, scaling="twice")
    with pytest.raises(pkv.PkvError):
        pkv.rope_inv_freq(63)
    with pytest.raises(ValueError):
        pkv.Rope(f.view(1, -1), **cpu)
    with pytest.raises(pkv.PkvError):
        pkv.Rope(torch.tensor([float("nan")]), **cpu)
    with pytest.raises(ValueError):
        pkv.Rope(f, q_weight=torch.ones(64, dtype=torch.float16), **cpu)
    rope = pkv.Rope(f, q_weight=torch.ones(64, dtype=torch.bfloat16), **cpu)
    q, pos = torch.zeros(3, 4, 64, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    for bad in (dict(q=q.float()), dict(q=q.half()), dict(q=q[..., ::2]), dict(q=q.transpose(1, 2)), dict(positions=pos.long()),
                dict(positions=pos[:2]), dict(q_out=q[:2]), dict(q_out=q.float()), dict(k=q[:, :, :32]), dict(q=None), dict(q=q[0])):
        a = dict(q=q, k=None, positions=pos)
        a.update(bad)
        with pytest.raises(ValueError):
            pkv.norm_rope(rope, **a)
    with pytest.raises(ValueError):
        pkv.norm_rope(pkv.Rope(pkv.rope_inv_freq(128)[0], **cpu), q, None, pos)  # more rotated columns than the head has
    pool, bt = torch.zeros(4, 2, 9 * 64, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        pkv.PagedKVCache([pool.view(4, 1, 2, -1)], [pool.view(4, 1, 2, -1)], bt)
    with pytest.raises(ValueError):
        pkv.PagedKVCache([pool[:, :, :64].contiguous()], [pool[:, :, :64].contiguous()], bt)
    c = pkv.PagedKVCache([pool], [pool.clone()], bt)
    assert (c.kv_heads, c.head_dim, c.row_dtype, c.bucket) == (2, 64, torch.bfloat16, 64)
    kn, si, err = torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    for bad in (dict(k_new=kn.float()), dict(k_new=kn[:, :1]), dict(seq_info=si.long()), dict(seq_info=si[0]), dict(v_out=kn.float()),
                dict(q=kn), dict(positions=torch.zeros(2, dtype=torch.int32))):
        a = dict(rope=None, q=None, k_new=kn, v_new=kn, seq_info=si, q_out=None, err=err)
        a.update(bad)
        if "q" in bad:
            a["q_out"] = kn.float()
        with pytest.raises(ValueError):
            pkv.norm_rope_append(c, 0, **a)


@pytest.mark.parametrize("q,out,lse", [
    (torch.float32, (torch.float32, (2, 4, 64)), None), (torch.bfloat16, (torch.float16, (2, 4, 64)), None),
    (torch.bfloat16, (torch.float32, (1, 4, 64)), None), (torch.bfloat16, (torch.bfloat16, (2, 4, 128)), None),
    (torch.bfloat16, (torch.float32, (2, 4, 64)), (torch.float32, (2, 3))), (torch.bfloat16, (torch.float32, (2, 4, 64)), (torch.bfloat16, (2, 4))),
])
def test_attention_over_fp4_checks_its_tensors(q, out, lse):
    import paged_kv_decode_13_gb300 as pkv
    cache = pkv.PagedKVCache.allocate(1, 2, 64, 512, dtype=torch.uint8, device="cpu")
    si, err = torch.tensor([[0, 2, 0, 2]], dtype=torch.int32), pkv.new_err_flags("cpu")
    lse = None if lse is None else torch.empty(lse[1], dtype=lse[0])
    with pytest.raises(ValueError):
        pkv.attend_varlen(cache, 0, torch.zeros(2, 4, 64, dtype=q), si, torch.empty(out[1], dtype=out[0]), err, 2, 512, 0.125, lse=lse)


def test_rows_for_fp4_are_bf16():
    import paged_kv_decode_13_gb300 as pkv
    cache = pkv.PagedKVCache.allocate(1, 2, 64, 512, dtype=torch.uint8, device="cpu")
    si, err = torch.tensor([[0, 2, 0, 2]], dtype=torch.int32), pkv.new_err_flags("cpu")
    q, out = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.empty(2, 4, 64)
    good = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    for k, v in ((good.float(), good), (good, good.half()), (good, good[:1])):
        with pytest.raises(ValueError):
            pkv.append(cache, 0, k, v, si, err)
        for fn in (pkv.append_attend, pkv.append_attend_noalloc):
            with pytest.raises(ValueError):
                fn(cache, 0, q, k, v, si, out, err, 2, 512, 0.125)
    with pytest.raises(ValueError):
        pkv.append_attend_noalloc(cache, 0, q, good, good, si, out.half(), err, 2, 512, 0.125)


def test_workspace_bounds_do_not_overflow(lib):
    """Any bounds give a size or a refusal, the largest ones a size that does not grow with them."""
    d, keep = _desc(lib, kv_heads=64)
    size = lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 512, 512, 1, 1 << 20, 0, 0)
    assert 0 < size < 25 << 20
    assert lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 512, 512, 1, (1 << 62), 0, 0) == size
    assert lib.lib.pkv_attend_workspace_bytes(ctypes.byref(d), 512, 512, 1, 16, 0, 0) == 0
