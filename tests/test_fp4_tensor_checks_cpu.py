"""Calls over a 4-bit cache whose tensors do not fit it are refused before
anything is launched: the kernels index rows by the cache's own heads and head_dim."""
import pytest
import torch

import paged_kv_decode_13_gb300 as pkv

BF = torch.bfloat16


def tensors():
    cache = pkv.PagedKVCache.allocate(1, 2, 128, 512, dtype=torch.uint8, device="cpu")
    return dict(cache=cache, q=torch.zeros(3, 4, 128, dtype=BF), k_new=torch.zeros(3, 2, 128, dtype=BF), v_new=torch.zeros(3, 2, 128, dtype=BF),
                seq_info=torch.tensor([[0, 3, 0, 3]], dtype=torch.int32), out=torch.zeros(3, 4, 128), err=pkv.new_err_flags("cpu"),
                lse=torch.zeros(3, 4))


BAD_ATTEND = [
    dict(q=torch.zeros(3, 4, 64, dtype=BF), out=torch.zeros(3, 4, 64)), dict(q=torch.zeros(3, 4, 256, dtype=BF), out=torch.zeros(3, 4, 256)),
    dict(q=torch.zeros(3, 512, dtype=BF), out=torch.zeros(3, 512)), dict(out=torch.zeros(3, 4, 64)), dict(out=torch.zeros(2, 4, 128)),
    dict(lse=torch.zeros(3, 8)[:, ::2]), dict(lse=torch.zeros(2, 4)), dict(seq_info=torch.zeros(1, 4, dtype=torch.int64)),
    dict(seq_info=torch.zeros(4, dtype=torch.int32)), dict(seq_info=torch.zeros(1, 3, dtype=torch.int32)),
]
BAD_NEW = [
    dict(k_new=torch.zeros(2, 2, 128, dtype=BF), v_new=torch.zeros(2, 2, 128, dtype=BF)),     # fewer rows than q
    dict(k_new=torch.zeros(3, 1, 128, dtype=BF), v_new=torch.zeros(3, 1, 128, dtype=BF)),
    dict(k_new=torch.zeros(3, 2, 64, dtype=BF), v_new=torch.zeros(3, 2, 64, dtype=BF)),
    dict(k_new=torch.zeros(3, 4, 64, dtype=BF), v_new=torch.zeros(3, 4, 64, dtype=BF)),
    dict(v_new=torch.zeros(3, 256, dtype=BF)), dict(k_new=torch.zeros(768, dtype=BF), v_new=torch.zeros(768, dtype=BF)),
]


def attend(t, fn):
    new = () if fn is pkv.attend_varlen else (t["k_new"], t["v_new"])
    fn(t["cache"], 0, t["q"], *new, t["seq_info"], t["out"], t["err"], 3, 512, 0.1, lse=t["lse"])


@pytest.mark.parametrize("fn", [pkv.attend_varlen, pkv.append_attend, pkv.append_attend_noalloc])
@pytest.mark.parametrize("bad", range(len(BAD_ATTEND)))
def test_attention_refuses(fn, bad):
    with pytest.raises(ValueError):
        attend({**tensors(), **BAD_ATTEND[bad]}, fn)


@pytest.mark.parametrize("fn", [pkv.append_attend, pkv.append_attend_noalloc])
@pytest.mark.parametrize("bad", range(len(BAD_NEW)))
def test_append_attend_refuses(fn, bad):
    with pytest.raises(ValueError):
        attend({**tensors(), **BAD_NEW[bad]}, fn)


@pytest.mark.parametrize("bad", range(1, len(BAD_NEW)))
def test_append_refuses(bad):
    t = {**tensors(), **BAD_NEW[bad]}
    with pytest.raises(ValueError):
        pkv.append(t["cache"], 0, t["k_new"], t["v_new"], t["seq_info"], t["err"])


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 3


@pytest.mark.parametrize("name", ["k", "v", "block_table", "first_valid"])
def test_a_cache_is_on_one_device(name):
    a = dict(k=torch.zeros(4, 2, 9 * 64, dtype=torch.uint8), v=torch.zeros(4, 2, 9 * 64, dtype=torch.uint8), block_table=torch.zeros(1, 4, dtype=torch.int32),
             first_valid=torch.zeros(1, dtype=torch.int32))
    pkv.PagedKVCache([a["k"]], [a["v"]], a["block_table"], first_valid=a["first_valid"])
    a[name] = a[name].as_subclass(Elsewhere)
    with pytest.raises(ValueError):
        pkv.PagedKVCache([a["k"]], [a["v"]], a["block_table"], first_valid=a["first_valid"])


@pytest.mark.parametrize("name", ["q", "out", "lse", "seq_info", "err", "k_new", "v_new"])
def test_tensors_of_another_device(name):
    t = tensors()
    t[name] = t[name].as_subclass(Elsewhere)
    for fn in (pkv.append_attend, pkv.append_attend_noalloc) + (() if name in ("k_new", "v_new") else (pkv.attend_varlen,)):
        with pytest.raises(ValueError):
            attend(t, fn)
    if name not in ("q", "out", "lse"):
        with pytest.raises(ValueError):
            pkv.append(t["cache"], 0, t["k_new"], t["v_new"], t["seq_info"], t["err"])
        with pytest.raises(ValueError):
            pkv.norm_rope_append(t["cache"], 0, None, None, t["k_new"], t["v_new"], t["seq_info"], None, t["err"])


def test_rows_may_come_flat(monkeypatch):
    """(rows, heads * head_dim) says the same as (rows, heads, head_dim)."""
    from paged_kv_decode_13_gb300 import api
    seen = []
    monkeypatch.setattr(api.lib, "pkv_append", lambda *a: seen.append(a) or 0)
    monkeypatch.setattr(api, "_stream", lambda s: 0)
    t = tensors()
    pkv.append(t["cache"], 0, t["k_new"], t["v_new"], t["seq_info"], t["err"])
    pkv.append(t["cache"], 0, t["k_new"].view(3, 256), t["v_new"].view(3, 256), t["seq_info"], t["err"])
    assert len(seen) == 2 and seen[0][2:] == seen[1][2:]
