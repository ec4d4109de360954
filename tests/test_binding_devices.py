"""What the batch-decoding calls are given on another device than the cache, or of the
wrong rank or count, is refused before the library sees it (no GPU needed: the library
is stood in for, the cache is on the CPU, the other device is "meta")."""

import types

import pytest
import torch

from w4_gemm_keyed_gb300 import tf


@pytest.fixture
def cache(monkeypatch):
    def called(*a):
        pytest.fail("the library was called")
    lib = types.SimpleNamespace(**{name: called for name, _, _ in tf.SIGNATURES})
    lib.tf_attention_batch_workspace_bytes = lambda *a: 1024
    monkeypatch.setattr(tf, "load", lambda *a: lib)
    monkeypatch.setattr(tf, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(tf, "_current_raw_stream", lambda: 0)
    return tf.KVBatch(2, 2, 256, "e4m3", device="cpu")


def bf16(device="cpu"):
    return torch.ones((4, 256), dtype=torch.bfloat16, device=device)


POS = torch.zeros(2, dtype=torch.int64)
ELSEWHERE = torch.zeros(4096, dtype=torch.uint8, device="meta")
CASES = dict(
    store_ws=lambda c: c.store(bf16(), bf16(), POS, ws=ELSEWHERE),
    store_rows=lambda c: c.store(bf16("meta"), bf16(), POS),
    load_ws=lambda c: c.load(POS, 2, ws=ELSEWHERE),
    load_rows=lambda c: c.load(POS, 2, k=bf16(), v=bf16("meta")),
    load_pos=lambda c: c.load(POS.to("meta"), 2),
    attention_ws=lambda c: c.attention(bf16(), 1, POS, ws=ELSEWHERE),
    attention_prefix=lambda c: c.attention(bf16(), 1, POS, prefix=tf.KVBatch(1, 2, 256, "e4m3", device="meta"),
                                           prefix_len=3),
    attention_out=lambda c: c.attention(bf16(), 1, POS, out=bf16("meta")),
)


@pytest.mark.parametrize("name", CASES)
def test_another_device_is_refused(cache, name):
    with pytest.raises(tf.TFError) as e:
        CASES[name](cache)
    assert e.value.status == tf.TF_ERR_INVALID_ARG


SCALAR = torch.tensor(1.0, dtype=torch.bfloat16)
MALFORMED = dict(
    store_scalar=lambda c: c.store(SCALAR, SCALAR, POS),
    attention_scalar=lambda c: c.attention(SCALAR, 1, POS),
    attention_group=lambda c: c.attention(bf16(), -1, POS),
    store_to_none=lambda c: tf.KVBatch(0, 2, 256, device="cpu").store(bf16(), bf16(), POS),
    attention_of_none=lambda c: tf.KVBatch(0, 2, 256, device="cpu").attention(bf16(), 1, POS),
)


@pytest.mark.parametrize("name", MALFORMED)
def test_malformed_arguments_are_refused_as_others_are(cache, name):
    with pytest.raises(tf.TFError):
        MALFORMED[name](cache)
