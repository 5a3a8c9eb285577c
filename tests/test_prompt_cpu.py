"""attend_prompt: refusals before any launch, at the C entry point and in the binding."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def pkv():
    import __graft_entry__
    __graft_entry__.build()
    import paged_kv_decode_13_gb300 as m
    return m


def call(pkv, D=64, hkv=2, si=0x60000, S=1, max_len=10, scale=0.125, causal=1, window=0, out=0x70000, lse=None, err=0x80000, flags=0, **kw):
    from paged_kv_decode_13_gb300 import _lib
    a = dict(q=0x10000, k=0x20000, v=0x30000, q_stride=512, k_stride=128, v_stride=128, q_heads=8, total_rows=4)
    a.update(kw)
    r = _lib.RowsDesc(**a)
    return _lib.lib.pkv_attend_prompt(D, hkv, ctypes.byref(r), si, S, max_len, scale, causal, window, out, lse, err, flags, None)


@pytest.mark.parametrize("bad", [
    dict(hkv=0), dict(hkv=3), dict(q_heads=0), dict(q_heads=-8), dict(total_rows=-1), dict(q=None), dict(k=None), dict(v=None), dict(q=0x10008),
    dict(k=0x20002), dict(v=0x30004), dict(q_stride=504), dict(q_stride=516), dict(k_stride=120), dict(v_stride=132), dict(si=None), dict(si=0x60004),
    dict(S=-1), dict(S=65536), dict(max_len=0), dict(max_len=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
    dict(causal=2), dict(causal=-1), dict(window=-1), dict(out=None), dict(out=0x70008), dict(lse=0x90002), dict(err=None), dict(flags=1), dict(flags=4),
    dict(q_out=0x10000), dict(k_out=0x10000), dict(v_out=0x10000), dict(positions=0x10000), dict(S=65535, hkv=8, max_len=1 << 30, total_rows=1 << 30),
])
def test_refusals(pkv, bad):
    assert call(pkv, **bad) == -1


def test_unsupported_and_empty(pkv):
    for D in (0, -8, 4, 60, 264):
        assert call(pkv, D=D, q_stride=1 << 14, k_stride=1 << 12, v_stride=1 << 12) == -2
    assert call(pkv, hkv=1, q_heads=129, q_stride=129 * 64) == -2
    assert call(pkv, total_rows=0) == 0 and call(pkv, total_rows=0, S=0, si=None, q=None, k=None, v=None) == 0


def test_no_rows_need_no_output(pkv):
    assert call(pkv, total_rows=0, out=None) == 0 and call(pkv, total_rows=0, out=None, q=None, k=None, v=None) == 0
    assert call(pkv, total_rows=0, out=0x70008) == -1 and call(pkv, total_rows=0, err=None) == -1


def test_binding_checks(pkv):
    q, kv = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    si, err, out = torch.tensor([[0, 5, 0, 5]], dtype=torch.int32), pkv.new_err_flags("cpu"), torch.zeros(5, 4, 64)
    good = dict(q=q, k=kv, v=kv, seq_info=si, out=out, err=err, max_len=5, scale=0.125)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=kv[:4]), dict(k=kv.half()), dict(v=kv[:, :1]), dict(k=kv[..., :32]), dict(q=q.transpose(0, 1)),
                dict(v=torch.zeros(5, 64, 2).transpose(1, 2).bfloat16()), dict(out=out.half()), dict(out=out[:4]), dict(out=torch.zeros(5, 4, 128)[..., :64]),
                dict(lse=torch.zeros(5, 3)), dict(lse=torch.zeros(5, 4).bfloat16()), dict(seq_info=si.long()), dict(seq_info=si[0])):
        with pytest.raises(ValueError):
            pkv.attend_prompt(**{**good, **bad})
    with pytest.raises(ValueError):   # host tensors
        pkv.attend_prompt(**good)
