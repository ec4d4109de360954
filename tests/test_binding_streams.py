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
    monkeypatch.setattr(tf, "_check_rows_out", lambda *a: None)      # wants CUDA tensors
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


def w4(K=128, N=64):
    return tf.W4Matrix(int_(torch.uint8, 256), K, N, 64)


def f32(*shape):
    return torch.ones(shape, dtype=torch.float32)


def int_(dt, *shape):
    return torch.ones(shape, dtype=dt)


def moe():
    return tf.MoeLayer(int_(torch.uint8, 8), int_(torch.uint8, 8), 64, 64, 4, 2, 32)


def kv_cache():
    return tf.KVCache(2, 256, device="cpu")


OTHER_CALLS = dict(
    lane_gemm_w4=lambda: tf.lane_gemm_w4(w4(), bf16(2, 128), stream=SIDE),
    lane_gemm_w4_accumulate=lambda: tf.lane_gemm_w4_accumulate(w4(), bf16(2, 128), f32(2, 64), stream=SIDE),
    lane_gemm_nvfp4=lambda: tf.lane_gemm_nvfp4(tf.Nvfp4Matrix(int_(torch.uint8, 8), 128, 64, 1.0), bf16(2, 128),
                                               stream=SIDE),
    cast_bf16=lambda: tf.cast_bf16(f32(2, 64), stream=SIDE),
    rmsnorm_bf16=lambda: tf.rmsnorm_bf16(f32(2, 64), 1e-6, stream=SIDE),
    keyed_sample=lambda: tf.keyed_sample(f32(2, 100), 0.7, 20, 0.9, 1, stream=SIDE),
    lmhead_sample=lambda: tf.lmhead_sample(w4(), bf16(2, 128), 0.7, 20, 0.9, 1, stream=SIDE),
    keyed_hash=lambda: tf.keyed_hash(pos(3), pos(3), int_(torch.int32, 3), stream=SIDE),
    accept=lambda: tf.accept(int_(torch.int32, 2), int_(torch.int32, 3), stream=SIDE),
    selfcheck=lambda: tf.selfcheck_row_invariance(w4(), bf16(16, 128), stream=SIDE),
    kv_append=lambda: kv_cache().append(bf16(2, 256), bf16(2, 256), pos(1), stream=SIDE),
    kv_attention=lambda: kv_cache().attention(bf16(2, 256), 1, pos(1), stream=SIDE),
    moe_w4=lambda: tf.moe_w4(moe(), bf16(2, 64), f32(2, 4), stream=SIDE),
    pack_w4=lambda: tf.pack_w4(int_(torch.uint8, 64, 64), int_(torch.int16, 64, 2), 64, stream=SIDE).packed,
    pack_w4_affine=lambda: tf.pack_w4_affine(int_(torch.int32, 64, 16), bf16(64, 2), bf16(64, 2), 64,
                                             stream=SIDE).packed,
    pack_nvfp4=lambda: tf.pack_nvfp4(int_(torch.uint8, 64, 64), int_(torch.uint8, 64, 8), 1.0, stream=SIDE).packed,
)


@pytest.mark.parametrize("name", OTHER_CALLS)
def test_every_other_call(rec, monkeypatch, name):
    for query in [n for n, _, _ in tf.SIGNATURES if n.endswith("_bytes")]:
        setattr(tf.load(), query, lambda *a: 512)
    if name.startswith("kv_"):
        made = kv_cache()           # the caches themselves are the caller's, made on the current stream
        monkeypatch.setitem(globals(), "kv_cache", lambda: made)
        rec.made.clear()
    got = OTHER_CALLS[name]()
    assert rec.made and all(side for _, side in rec.made), name
    for t in got if isinstance(got, tuple) else [got]:
        if isinstance(t, torch.Tensor) and name != "lane_gemm_w4_accumulate":
            assert marked(rec, t), name


def test_copies_for_the_packers(rec, monkeypatch):
    inside, real = [], torch.Tensor.contiguous

    def contiguous(t):
        inside.append(rec.inside > 0)
        return real(t)
    monkeypatch.setattr(torch.Tensor, "contiguous", contiguous)
    tf.load().tf_w4_packed_bytes = lambda *a: 512
    tf.pack_w4(int_(torch.uint8, 64, 64), int_(torch.int16, 64, 2), 64, stream=SIDE)
    assert inside == [True, True]
