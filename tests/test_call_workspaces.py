"""The workspaces that attention calls make for themselves: cleared where they are read before they are
written, and not gigabytes that nothing reads (no GPU needed)."""

import ctypes
import types

import pytest
import torch

from w4_gemm_keyed_gb300 import tf


class OnDevice(torch.Tensor):
    is_cuda = True


def ones(*shape):
    return torch.ones(shape, dtype=torch.bfloat16).as_subclass(OnDevice)


@pytest.mark.parametrize("nbytes", [1 << 12, 1 << 25, (1 << 25) + 256, 1 << 27])
@pytest.mark.parametrize("op", ["tree", "batch"])
def test_no_call_clears_what_nothing_reads(monkeypatch, op, nbytes):
    seen, cleared = {}, []
    empty, zeros = torch.empty, torch.zeros

    def call(*a):
        seen["ws"], seen["bytes"] = a[-3], a[-2]
        seen["head"] = ctypes.string_at(a[-3], 256)
        return 0
    fake = types.SimpleNamespace(tf_attention_tree=call, tf_attention_batch=call,
                                 tf_attention_tree_workspace_bytes=lambda *a: nbytes,
                                 tf_attention_batch_workspace_bytes=lambda *a: nbytes)
    monkeypatch.setattr(tf, "load", lambda *a: fake)
    monkeypatch.setattr(tf, "_ptr", lambda t: None if t is None else t.data_ptr())
    cache = tf.KVBatch(2, 2, 256, device="cpu")
    q, pos, parents = ones(4, 256), torch.zeros(2, dtype=torch.int64), torch.zeros((2, 2), dtype=torch.int32)
    monkeypatch.setattr(tf, "_current_raw_stream", lambda: 0)
    monkeypatch.setattr(torch, "empty", lambda *a, **k: empty(*a, **k).fill_(3))
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: cleared.append(a[0]) or zeros(*a, **k))
    if op == "tree":
        cache.tree_attention(q, 1, pos, parents)
    else:
        cache.attention(q, 1, pos)
    assert seen["bytes"] == nbytes and seen["head"] == bytes(256)
    assert sum(cleared) <= 1 << 25
