"""Buffers that the batch-decoding calls make themselves, on the GPU."""

import pytest
import torch

from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16

pytestmark = pytest.mark.gpu
D = 128


def rows(seed, n, cols):
    return dev_bits16(inputs.bf16_normal(inputs.rng_for(seed), (n, cols)))


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_own_buffers_on_another_stream(tf, fmt):
    """Calls on a side stream, with the buffers they make themselves, while the current
    stream is busy: the results do not wait for it, nor does its next use of memory
    reach them."""
    B, R, n_kv, g, P = 100, 2, 2, 4, 300
    own, prefix = tf.KVBatch(B, n_kv, 512, fmt), tf.KVBatch(1, n_kv, 512, fmt)
    pos, start = dev_pos([b % 38 for b in range(B)]), dev_pos([0] * B)
    k, v = rows(1, B * 40, n_kv * D), rows(2, B * 40, n_kv * D)
    own.store(k, v, start)
    prefix.store(rows(3, P, n_kv * D), rows(4, P, n_kv * D), start[:1])
    q = rows(5, B * R, n_kv * g * D)
    turns = tf.rope_turns(128)
    want = [own.attention(q, g, pos, prefix=prefix, prefix_len=P), *own.load(start, 40),
            tf.qk_norm_rope(k, 1, 1, start, turns, n_v=0)]
    a = torch.ones((8192, 8192), dtype=torch.bfloat16, device="cuda")
    scratch = torch.empty_like(a)
    # blocks of the current stream's pool that hold something else than zeros
    for _ in range(8):
        torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        torch.full((own.attention_workspace_bytes(g, R, P),), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        for _ in range(40):         # some 20 ms
            torch.mm(a, a, out=scratch)
        got = [own.attention(q, g, pos, prefix=prefix, prefix_len=P, stream=side), *own.load(start, 40, stream=side),
               tf.qk_norm_rope(k, 1, 1, start, turns, n_v=0, stream=side)]
        ws = own.store(k, v, start, stream=side)
        again = [torch.full_like(t, 3.0) for t in got]      # the current stream's next use of memory
        side.synchronize()
        assert all(torch.equal(x.cpu(), y.cpu()) for x, y in zip(got, want))
        assert tf.workspace_status(ws, stream=side) == tf.TF_DEV_OK
        del got, again
        torch.cuda.synchronize()


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_load_into_one_given_strided_buffer(tf, fmt):
    c = tf.KVBatch(2, 2, 256, fmt)
    pos = dev_pos([3, 100])
    c.store(rows(1, 10, 2 * D), rows(2, 10, 2 * D), pos)
    want_k, want_v = c.load(pos, 5)
    for name in ("k", "v"):
        wide = torch.zeros((10, 3 * D), dtype=torch.bfloat16, device="cuda")
        k, v = c.load(pos, 5, **{name: wide[:, :2 * D]})
        assert (k if name == "k" else v).data_ptr() == wide.data_ptr()
        assert torch.equal(k, want_k) and torch.equal(v, want_v) and not wide[:, 2 * D:].any()
