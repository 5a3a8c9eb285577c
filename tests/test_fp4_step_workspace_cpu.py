"""A DecodeStep over a 4-bit cache owns the workspace that its launches merge
through: nothing is left for a call to allocate inside a capture."""
import pytest
import torch

import paged_kv_decode_13_gb300 as pkv
from paged_kv_decode_13_gb300 import graph


def step(max_kv, **kw):
    cache = pkv.PagedKVCache.allocate(2, 8, 128, 512, dtype=torch.uint8, device="cpu")
    return graph.DecodeStep(cache, 32, rows=4, num_segments=4, max_kv=max_kv, **kw)


@pytest.mark.parametrize("fused,rope", [(True, False), (False, False), (True, True)])
def test_every_call_gets_the_steps_workspace(monkeypatch, fused, rope):
    given = []

    def record(*a, workspace=None, **kw):
        given.append(workspace)

    for name in ("attend_varlen", "append_attend"):
        monkeypatch.setattr(graph, name, record)
    for name in ("append", "norm_rope_append"):
        monkeypatch.setattr(graph, name, lambda *a, **kw: None)
    ropes = pkv.Rope(pkv.rope_inv_freq(128)[0], device="cpu") if rope else None
    steps = [step(1 << 20, fused=fused, rope=ropes) for _ in range(2)]
    need = pkv.attend_workspace_bytes(steps[0].cache, 32, 4, 1, 1 << 20)
    assert need > 0
    for st in steps:
        st.run()
    assert len(given) == 4 and all(w is not None and w.numel() == need for w in given)
    assert given[0] is given[1] and given[2] is given[3] and given[0].data_ptr() != given[2].data_ptr()


def test_no_workspace_where_the_bounds_need_none():
    assert step(512).ws is None
    assert step(1 << 20, num_splits=4).ws is None


def test_a_workspace_of_the_right_size_is_kept():
    st = step(1 << 20)
    ws = st.ws
    st.size_workspace()
    assert st.ws is ws
    st.max_kv = 512
    st.size_workspace()
    assert st.ws is None
