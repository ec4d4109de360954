"""Buffers that the binding makes for a call on another stream (no GPU needed).

What a call allocates itself (outputs, the workspace with its zero fill) is made on the
stream that the call's kernels run on: a fill on the current stream would be
unordered with them, and memory freed there could be handed out again while they
still use it.  The library and the stream context are stood in for; tensors are CPU ones.
"""

import types

import pytest
import torch

from w4_gemm_keyed_gb300 import tf

D = 128


class Recorder:
    """Counts allocations inside and outside the side stream's context."""

    def __init__(self):
        self.inside, self.made, self.marked = 0, [], []

    def stream(self, s):
        rec = self

        class Context:
            def __enter__(self):
                rec.inside += 1

            def __exit__(self, *a):
                rec.inside -= 1
        assert s.cuda_stream == 77
        return Context()

    def wrap(self, f):
        def made(*a, **kw):
            t = f(*a, **kw)
            self.made.append((t, self.inside > 0))
            return t
        return made


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    lib = types.SimpleNamespace(**{name: (lambda *a: 0) for name, _, _ in tf.SIGNATURES})
    lib.tf_attention_batch_workspace_bytes = lambda *a: 1024
    monkeypatch.setattr(tf, "load", lambda *a: lib)
    monkeypatch.setattr(tf, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: "current")
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: r.marked.append((t, s)), raising=False)
    for name in ("empty", "zeros", "empty_like"):
        monkeypatch.setattr(torch, name, r.wrap(getattr(torch, name)))
    return r


SIDE = types.SimpleNamespace(cuda_stream=77)


def bf16(*shape):
    return torch.ones(shape, dtype=torch.bfloat16)


def pos(n):
    return torch.tensor([0] * n, dtype=torch.int64)


def cache(rec, fmt="e4m3"):
    c = tf.KVBatch(2, 2, 256, fmt, device="cpu")
    rec.made.clear()
    return c


def marked(rec, t):
    """Whether t's memory is known to be used on the current stream too."""
    return any(m.data_ptr() == t.data_ptr() and s == "current" for m, s in rec.marked)


def test_store(rec):
    ws = cache(rec).store(bf16(4, 256), bf16(4, 256), pos(2), stream=SIDE)
    assert rec.made and all(side for _, side in rec.made)
    assert marked(rec, ws)          # returned: read with workspace_status on whichever stream


@pytest.mark.parametrize("given", [{}, dict(k=bf16(4, 256)), dict(v=bf16(4, 256))], ids=["none", "k", "v"])
def test_load(rec, given):
    got = cache(rec).load(pos(2), 2, stream=SIDE, **given)
    assert rec.made and all(side for _, side in rec.made)
    for t in got:
        assert marked(rec, t) or any(t is g for g in given.values())


def test_attention(rec):
    out = cache(rec).attention(bf16(4, 256), 1, pos(2), stream=SIDE)
    assert len(rec.made) == 2 and all(side for _, side in rec.made)
    assert marked(rec, out)


def test_on_the_current_stream_nothing_is_switched(rec, monkeypatch):
    monkeypatch.setattr(tf, "_current_raw_stream", lambda: 0)
    c = cache(rec)
    c.store(bf16(4, 256), bf16(4, 256), pos(2))
    c.load(pos(2), 2)
    c.attention(bf16(4, 256), 1, pos(2))
    assert not any(side for _, side in rec.made) and not rec.marked


def test_rotation(rec, monkeypatch):
    class OnDevice(torch.Tensor):
        is_cuda = True
    x = torch.ones((4, 6 * D)).as_subclass(OnDevice)
    out = tf.qk_norm_rope(x, 2, 2, pos(2), stream=SIDE)
    assert rec.made and all(side for _, side in rec.made) and marked(rec, out)
