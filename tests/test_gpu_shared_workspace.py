"""One workspace used by several operators in turn, on the GPU through the binding.

tf_attention_batch takes its items from a counter that has to start at zero: what
other operators leave in a workspace must not reach it, and what it leaves must not
reach the split-K counters of the lane GEMM.
"""

import pytest
import torch

from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16, pack

pytestmark = pytest.mark.gpu
D = 128
B, R, N_KV, GROUP, P = 100, 2, 2, 4, 300      # more own parts than SMs


def rows(seed, n, cols):
    return dev_bits16(inputs.bf16_normal(inputs.rng_for(seed), (n, cols)))


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


@pytest.fixture(params=["bf16", "e4m3"])
def batch(tf, request):
    """(call, bytes): attention of a batch on a given workspace, and the workspace it needs."""
    own, prefix = tf.KVBatch(B, N_KV, 512, request.param), tf.KVBatch(1, N_KV, 512, request.param)
    own.store(rows(1, B * 40, N_KV * D), rows(2, B * 40, N_KV * D), dev_pos([0] * B))
    prefix.store(rows(3, P, N_KV * D), rows(4, P, N_KV * D), dev_pos([0]))
    q, pos = rows(5, B * R, N_KV * GROUP * D), dev_pos([b % 38 for b in range(B)])
    need = own.attention_workspace_bytes(GROUP, R, P)
    return lambda ws: own.attention(q, GROUP, pos, prefix=prefix, prefix_len=P, ws=ws), need


def test_attention_after_the_single_sequence_attention(tf, batch):
    call, need = batch
    want = call(tf.workspace(need))
    cache = tf.KVCache(N_KV, 512)
    cache.append(rows(6, 16, N_KV * D), rows(7, 16, N_KV * D), dev_pos([0]))
    ws = tf.workspace(max(need, cache.workspace_bytes(GROUP, 16)))
    cache.attention(rows(8, 16, N_KV * GROUP * D), GROUP, dev_pos([0]), ws=ws)
    assert torch.equal(call(ws), want) and tf.workspace_status(ws) == tf.TF_DEV_OK


def test_attention_after_the_sampler(tf, batch):
    call, need = batch
    want = call(tf.workspace(need))
    V = 5000
    ws = tf.workspace(max(need, tf.keyed_sample_workspace_bytes(4, V)))
    logits = torch.randn((4, V), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    tokens = tf.keyed_sample(logits, 0.7, 20, 0.95, 7, pos=dev_pos([1, 2, 3, 4]), ws=ws).clone()
    assert torch.equal(call(ws), want) and tf.workspace_status(ws) == tf.TF_DEV_OK
    assert torch.equal(tf.keyed_sample(logits, 0.7, 20, 0.95, 7, pos=dev_pos([1, 2, 3, 4])), tokens)


def test_lane_gemm_and_attention_in_turn(tf, batch):
    call, need = batch
    want = call(tf.workspace(need))
    K, N, G = 1024, 777, 64
    W = pack(tf, *inputs.w4_weights(inputs.rng_for(9), K, N, G), G)
    x = rows(10, 5, K)
    y = tf.lane_gemm_w4(W, x)
    ws = tf.workspace(max(need, tf.lane_gemm_workspace_bytes(K, N, G)))
    for _ in range(3):
        assert torch.equal(call(ws), want)
        assert torch.equal(tf.lane_gemm_w4(W, x, ws=ws), y)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
