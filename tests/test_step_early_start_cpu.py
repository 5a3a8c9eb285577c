"""When a DecodeStep lets a layer's attention start before the launch in front of
it has finished: never where that launch may be writing older keys of the step."""
import pytest
import torch

import paged_kv_decode_13_gb300 as pkv
from paged_kv_decode_13_gb300 import graph


def early(monkeypatch, rope, dtype=torch.bfloat16, **kw):
    flags = []
    for name in ("attend_varlen", "append_attend"):
        monkeypatch.setattr(graph, name, lambda *a, **k: flags.append(bool(k["flags"] & pkv.FLAG_PDL)))
    for name in ("append", "norm_rope_append"):
        monkeypatch.setattr(graph, name, lambda *a, **k: None)
    cache = pkv.PagedKVCache.allocate(3, 2, 64, 512, dtype=dtype, device="cpu")
    r = pkv.Rope(pkv.rope_inv_freq(64)[0], device="cpu") if rope else None
    graph.DecodeStep(cache, 4, rope=r, **kw).run()
    return flags


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.uint8])
@pytest.mark.parametrize("fused", [True, False])
def test_behind_an_append_of_several_segments(monkeypatch, dtype, fused):
    two = dict(rows=2, num_segments=2, dtype=dtype, fused=fused)
    assert early(monkeypatch, True, **two) == [False] * 3
    assert early(monkeypatch, True, pdl=True, **two) == [True] * 3
    assert early(monkeypatch, True, pdl=False, **two) == [False] * 3
    assert early(monkeypatch, True, dtype=dtype, fused=fused) == [True] * 3      # one segment reads what it writes after its wait
    assert early(monkeypatch, True, dtype=dtype, fused=fused, pdl=False) == [False] * 3


@pytest.mark.parametrize("pdl", [None, True, False])
def test_without_a_rope(monkeypatch, pdl):
    for n in (1, 2):
        kw = dict(rows=n, num_segments=n, pdl=pdl)
        assert early(monkeypatch, False, **kw) == [False] + [pdl is not False] * 2
        assert early(monkeypatch, False, fused=False, **kw) == [False] * 3
