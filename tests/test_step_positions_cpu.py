"""The positions of a DecodeStep: what its ropes' angles are taken from."""
import pytest
import torch

import paged_kv_decode_13_gb300 as pkv
from paged_kv_decode_13_gb300 import graph


def rope(axes=None):
    return pkv.Rope(pkv.rope_inv_freq(64)[0], device="cpu", axes=None if axes is None else pkv.rope_axes(axes))


def taken(monkeypatch, **kw):
    got = []
    monkeypatch.setattr(graph, "attend_varlen", lambda *a, **k: None)
    monkeypatch.setattr(graph, "norm_rope_append", lambda *a, **k: got.append(k["positions"]))
    step = graph.DecodeStep(pkv.PagedKVCache.allocate(3, 2, 64, 512, device="cpu"), 4, rows=5, **kw)
    step.run()
    return step, got


def test_positions_reach_every_layer(monkeypatch):
    for axes, shape in ((None, (5,)), ((16, 8, 8), (5, 3))):
        step, got = taken(monkeypatch, rope=rope(axes), positions=True)
        assert step.positions.shape == shape and step.positions.dtype == torch.int32 and len(got) == 3
        assert all(p is step.positions for p in got)
        at = step.positions.data_ptr() - step.inputs.data_ptr()
        assert 0 < at < step.step_inputs.numel() <= step.seq_info.data_ptr() - step.inputs.data_ptr()
        step, got = taken(monkeypatch, rope=rope(axes))
        assert step.positions is None and got == [None] * 3


def test_positions_without_a_rope_or_of_mixed_ropes_are_refused(monkeypatch):
    with pytest.raises(ValueError):
        taken(monkeypatch, positions=True)
    with pytest.raises(ValueError):
        taken(monkeypatch, positions=True, rope=[rope(), rope((16, 16)), rope()])
