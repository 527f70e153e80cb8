"""CPU: the compressed layer's workspaces, with a stand-in for the library's calls."""
import threading
import weakref
from types import SimpleNamespace

import pytest
import torch

import compressed_sparse_long_gb300 as v4a
from compressed_sparse_long_gb300 import layer


@pytest.fixture
def calls(monkeypatch):
    """The layer's calls that take a workspace; `during` runs inside each, `made` lists the
    workspaces that were allocated."""
    w = SimpleNamespace(during=lambda ws: None, made=[])

    def call(*a):
        ws = [t for t in a if isinstance(t, torch.Tensor) and t.dtype is torch.uint8][-1]
        w.made.append(weakref.ref(ws))
        w.during(ws.data_ptr())
    for name in ("v4a_index_topk", "v4a_attn_decode", "v4a_attn_prefill", "v4a_attn_decode_q8"):
        monkeypatch.setattr(layer, name, call)
    for name in ("v4a_index_topk_workspace_size", "v4a_attn_workspace_size", "v4a_attn_q8_workspace_size"):
        monkeypatch.setattr(layer, name, lambda *a: 4096)
    pool = SimpleNamespace(c=None)
    cfg = v4a.layer_cfg(v4a.C4A, v4a.BF16_FP8, 512, 64, 64, 64, 128, 8, 4, -4, 128, 10000.0, 1e-6, 0.04)
    lay = layer.Layer(cfg, None, None, None, pool, pool, pool, pool, top_k=64)
    seq, pos = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)
    q = torch.zeros(2, 64, 512, dtype=torch.bfloat16)
    w.forms = dict(index=lambda: lay.index_topk(seq, pos, 900, None, None),
                   decode=lambda: lay.attention(seq, pos, 900, q),
                   prefill=lambda: lay.attention(seq, pos, 900, q, prefill=True),
                   q8=lambda: lay.attention_q8(seq, pos, 900, q))
    return w


@pytest.mark.parametrize("form", ["index", "decode", "prefill", "q8"])
def test_calls_of_two_threads_have_workspaces_of_their_own(calls, form):
    seen = []

    def during(ws):
        seen.append(ws)
        if len(seen) == 1:
            t = threading.Thread(target=calls.forms[form])
            t.start()
            t.join(20)
            assert not t.is_alive()
    calls.during = during
    calls.forms[form]()
    assert len(seen) == 2 and seen[0] != seen[1]


@pytest.mark.parametrize("form", ["index", "decode", "prefill", "q8"])
def test_a_layer_keeps_no_workspace(calls, form):
    calls.forms[form]()
    assert len(calls.made) == 1 and calls.made[0]() is None
