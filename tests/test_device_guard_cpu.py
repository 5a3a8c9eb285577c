"""Every call runs with its cache's device current, and on that device's stream,
whichever device is current when it is made."""
import contextlib

import pytest
import torch

import paged_kv_decode_13_gb300 as pkv
from paged_kv_decode_13_gb300 import api


@pytest.fixture
def machine(monkeypatch):
    """Two devices that only keep a record: the device current at each library call, and its stream (100 + device)."""
    state = {"current": 0, "calls": []}

    @contextlib.contextmanager
    def device(d):
        old, state["current"] = state["current"], d
        yield
        state["current"] = old

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: state["current"], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: state["current"])
    monkeypatch.setattr(torch.cuda, "device", device)

    class Lib:
        def __getattr__(self, name):
            def call(*a):
                state["calls"].append((name, state["current"], None if name.endswith("_bytes") else a[-1]))
                return 0
            return call

    monkeypatch.setattr(api, "lib", Lib())
    return state


class On1(torch.Tensor):
    def get_device(self):
        return 1


def on1(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype).as_subclass(On1)


def calls(cache, rows_dtype):
    new, si, err = on1(1, 2, 64, dtype=rows_dtype), on1(1, 4, dtype=torch.int32), on1(1, dtype=torch.int32)
    q, out = on1(1, 4, 64, dtype=rows_dtype), on1(1, 4, 64, dtype=torch.float32)
    yield "pkv_append", lambda: pkv.append(cache, 0, new, new, si, err)
    yield "pkv_attend_varlen", lambda: pkv.attend_varlen(cache, 0, q, si, out, err, 1, 64, 0.1)
    yield "pkv_append_attend", lambda: pkv.append_attend(cache, 0, q, new, new, si, out, err, 1, 64, 0.1)
    yield "pkv_append_attend_noalloc", lambda: pkv.append_attend_noalloc(cache, 0, q, new, new, si, out, err, 1, 64, 0.1)
    yield "pkv_norm_rope_append", lambda: pkv.norm_rope_append(cache, 0, None, None, new, new, si, None, err)
    yield "pkv_rewind", lambda: pkv.rewind(cache, si, on1(1, dtype=torch.int32), err)
    yield "pkv_advance", lambda: pkv.advance(si)
    yield "pkv_attend_workspace_bytes", lambda: pkv.attend_workspace_bytes(cache, 4, 1, 1, 64)
    yield "pkv_seqinfo_from_seqused", lambda: pkv.seqinfo_from_seqused(on1(2, dtype=torch.int32), on1(1, dtype=torch.int32), si)
    yield "pkv_seq_clone", lambda: pkv.seq_clone(cache, 0, 0, 1, err)
    yield "pkv_resize_bucket", lambda: pkv.resize_bucket(cache, cache, 1)
    yield "pkv_to_contiguous", lambda: pkv.to_contiguous(cache, 0, 1, new, new)
    yield "pkv_load_prefix", lambda: pkv.load_prefix(cache, [new], [new])


@pytest.mark.parametrize("fp4", [False, True])
@pytest.mark.parametrize("current", [0, 1])
def test_the_caches_device_is_current(machine, fp4, current):
    shape = (4, 2, 9 * 64) if fp4 else (4, 16, 2, 64)
    pool = on1(*shape, dtype=torch.uint8 if fp4 else torch.bfloat16)
    cache = pkv.PagedKVCache([pool], [pool], on1(1, 4, dtype=torch.int32))
    machine["current"] = current
    for name, call in calls(cache, torch.bfloat16):
        if name == "pkv_load_prefix" and fp4:
            continue
        machine["calls"].clear()
        call()
        assert [c[0] for c in machine["calls"]] == [name]
        _, device, stream = machine["calls"][0]
        assert device == 1 and stream in (None, 101), name
        assert machine["current"] == current
