"""With a window the keys that it leaves decide how attention over a 4-bit
cache is cut: no workspace is taken for a launch that would not use it."""
import pytest
import torch

import paged_kv_decode_13_gb300 as pkv
from paged_kv_decode_13_gb300 import api, graph


def cache(D=128):
    return pkv.PagedKVCache.allocate(1, 8, D, 512, dtype=torch.uint8, device="cpu")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 16])
def test_taken_as_the_windows_keys_need(D, max_q):
    c, seen = cache(D), set()
    for max_kv in (512, 8192, 1 << 17, 1 << 20):
        for window in (0, 1, 100, 4096, 1 << 17, 1 << 30):
            keys = min(max_kv, window + max_q) if window else max_kv
            n = pkv.attend_workspace_bytes(c, 32, 8, max_q, keys)
            ws = api._fp4_workspace(c, 32, 8, max_q, max_kv, window, 0, None)
            assert (0 if ws is None else ws.numel()) == n
            seen.add(n > 0)
            st = graph.DecodeStep(c, 32, rows=8 * max_q, num_segments=8, max_q_len=max_q, max_kv=max_kv, window=window)
            assert (0 if st.ws is None else st.ws.numel()) == n
    assert seen == {False, True}
