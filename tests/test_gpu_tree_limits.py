"""Trees of drafts at the ends of what their calls take: positions, sequences and heads."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


def dev_i32(p):
    return torch.tensor(p, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- positions next to the end of int64
FAR = [2 ** 63 - 1, 2 ** 63 - 8, 2 ** 63 - 64, 2 ** 62, 2 ** 32, 257, 256, 249, -2, -2 ** 62, -2 ** 63]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("pos", FAR)
def test_keep_takes_no_position_past_its_entries(tf, fmt, pos):
    """Position + node passes int64 for the first of these; nothing of the sequence moves."""
    cache, ws = tf.KVBatch(3, 2, 256, fmt), tf.workspace(256)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.copy_(torch.arange(t.numel(), device="cuda").view(t.shape) % 200)
    was = [t.clone() for t in (cache.k, cache.v)]
    path = [0, 7] + [-1] * 14
    cache.keep(dev_pos([10, pos, 248]), dev_i32([path] * 3), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION
    for t, w in zip((cache.k, cache.v), was):
        assert torch.equal(t[1], w[1]) and not torch.equal(t[0], w[0]) and not torch.equal(t[2], w[2])


@pytest.mark.parametrize("pos", FAR)
def test_the_other_calls_take_no_such_position_either(tf, pos):
    cache, ws = tf.KVBatch(2, 1, 256), tf.workspace(1 << 20)
    rows = torch.ones((16, 128), dtype=torch.bfloat16, device="cuda")
    cache.store(rows, rows, dev_pos([10, pos]), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and not cache.k[1].any()
    tree = dev_i32([[-1] + [0] * 7] * 2)
    out = cache.tree_attention(rows, 1, dev_pos([10, pos]), tree, ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and not out[8:].any() and out[:8].all()
