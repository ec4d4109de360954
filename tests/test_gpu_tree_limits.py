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


# ---------------------------------------------------------------- outputs beside what is read
def test_outputs_may_be_other_columns_or_rows_of_an_inputs_array(tf):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    cols, n = 8 * 128, 9

    def normal(rows, width):
        return torch.randn((rows, width), generator=gen, device="cuda").to(torch.bfloat16)
    x, starts = normal(n, 2 * cols + 512), torch.tensor([0, 4, n], device="cuda")
    q, k, v = x[:, :cols], x[:, cols:cols + 256], x[:, cols + 256:cols + 512]
    want = tf.prompt_attention(q, k, v, 2, 4, starts)
    got = tf.prompt_attention(q, k, v, 2, 4, starts, out=x[:, cols + 512:])
    assert torch.equal(got, want) and got.data_ptr() == x.data_ptr() + 2 * (cols + 512)
    rows = normal(2 * n, cols)
    rows[:n] = q
    got = tf.prompt_attention(rows[:n], k, v, 2, 4, starts, out=rows[n:])
    assert torch.equal(got, want)
    cache, pos, tree = tf.KVBatch(1, 2, 256), dev_pos([3]), dev_i32([[-1] + [0] * (n - 1)])
    cache.store(normal(20, 256), normal(20, 256), dev_pos([0]))
    want = cache.tree_attention(q, 4, pos, tree)
    assert torch.equal(cache.tree_attention(q, 4, pos, tree, out=x[:, cols + 512:]), want)
    every = torch.stack([q, torch.zeros_like(q)], 1).view(2 * n, cols)      # every other row
    assert torch.equal(cache.tree_attention(every[::2], 4, pos, tree, out=every[1::2]), want)


def test_an_output_in_an_input_is_refused(tf):
    x = torch.ones((9, 1536), dtype=torch.bfloat16, device="cuda")
    starts, cache = torch.tensor([0, 9], device="cuda"), tf.KVBatch(1, 2, 256)
    q, k, v = x[:, :1024], x[:, 1024:1280], x[:, 1280:]
    for out in (q, x[:, 512:], x[:, 8:1032]):
        with pytest.raises(tf.TFError, match="out overlaps"):
            tf.prompt_attention(q, k, v, 2, 4, starts, out=out)
        with pytest.raises(tf.TFError, match="out overlaps q"):
            cache.tree_attention(q, 4, dev_pos([0]), dev_i32([[-1] + [0] * 8]), out=out)


# ---------------------------------------------------------------- a call's own workspace
@pytest.mark.parametrize("op", ["tree", "batch"])
def test_a_calls_own_workspace_may_hold_anything(tf, op):
    """Above 32 MB it is not cleared as a whole: the same bits as on a cleared one, and no device error."""
    B, n, n_kv, g, P = 24, 8, 8, 8, 700
    cache, prefix = tf.KVBatch(B, n_kv, 8192), tf.KVBatch(1, n_kv, 768)
    size = cache.tree_attention_workspace_bytes(g, n, P) if op == "tree" else cache.attention_workspace_bytes(g, n, P)
    assert size > 32 << 20
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    for c in (cache, prefix):
        rows = [torch.randn((c.n_seq * 700, n_kv * 128), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
        c.store(*rows, dev_pos([0] * c.n_seq))
    q = torch.randn((B * n, n_kv * g * 128), generator=gen, device="cuda").to(torch.bfloat16)
    pos, parents = dev_pos([28 * b for b in range(B)]), dev_i32([[-1, *range(n - 1)]] * B)

    def call(**kw):
        if op == "tree":
            return cache.tree_attention(q, g, pos, parents, prefix=prefix, prefix_len=P, **kw)
        return cache.attention(q, g, pos, prefix=prefix, prefix_len=P, **kw)
    want, side = call(ws=tf.workspace(size)), torch.cuda.Stream()
    for stream in (None, side):
        with torch.cuda.stream(stream):
            dirty = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty       # the allocator hands its memory to the call
        got = call(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


# ---------------------------------------------------------------- many sequences, many heads
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,P,longest", [(129, 5, 0, 1500), (300, 2, 300, 1000), (1024, 3, 0, 700), (1000, 4, 600, 330)])
def test_more_sequences_than_the_table_of_own_parts(tf, B, n, P, longest, fmt):
    """Above 128 sequences an entry of that table is several of them; idle ones leave whole entries without parts.
    The bits are those of calls of 64."""
    n_kv, g = 1, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B)

    def normal(rows, heads):
        return torch.randn((rows, heads * 128), generator=gen, device="cuda").to(torch.bfloat16)
    at = [(7919 * b) % longest for b in range(B)]
    for first, count in ((0, 20), (B // 3, 40), (B - 17, 17)):      # runs of idle sequences, at both ends too
        at[first:first + count] = [-1] * count
    at[B // 2], at[B // 2 + 1], at[B // 2 + 2] = 0, 16, 17          # no far entry, and the first ones
    L = -(-(longest + n) // 256) * 256
    cache, prefix = tf.KVBatch(B, n_kv, L, fmt), tf.KVBatch(1, n_kv, 768, fmt)
    cache.store(normal(B * L, n_kv), normal(B * L, n_kv), dev_pos([0] * B))
    prefix.store(normal(768, n_kv), normal(768, n_kv), dev_pos([0]))
    q = normal(B * n, n_kv * g)
    parents = [[-1] + [(5 * b + i) % i if (b + i) % 9 else i - 1 for i in range(1, n)] for b in range(B)]
    ws = tf.workspace(cache.tree_attention_workspace_bytes(g, n, P))
    for _ in range(2):
        out = cache.tree_attention(q, g, dev_pos(at), dev_i32(parents), prefix=prefix, prefix_len=P, ws=ws).view(B, n, -1)
        assert tf.workspace_status(ws) == tf.TF_DEV_OK
    for first in range(0, B, 64):
        m = min(64, B - first)
        some = tf.KVBatch(m, n_kv, L, fmt)
        for name in ("k", "v", "k_scale", "v_scale"):
            if getattr(some, name) is not None:
                getattr(some, name).copy_(getattr(cache, name)[first:first + m])
        part = some.tree_attention(q[first * n:(first + m) * n], g, dev_pos(at[first:first + m]), dev_i32(parents[first:first + m]),
                                   prefix=prefix, prefix_len=P).view(m, n, -1)
        assert torch.equal(part, out[first:first + m]), first
    used = torch.tensor(at, device="cuda") >= 0
    assert out[used].view(int(used.sum()), -1).any(1).all() and not out[~used].any()


@pytest.mark.parametrize("n_kv,g,P", [(76, 1, 1300), (77, 2, 1300), (128, 1, 561), (128, 1, 1201)])
def test_heads_whose_prefix_is_one_part(tf, n_kv, g, P):
    """Above 76 KV heads a prefix is not split; at 76 it is."""
    from test_gpu_trees import Case
    c = Case(tf, n_kv + P, [[-1, 0, 0, 2], [-1, 0, 1, -1]], n_kv, g, P, [330, 3], "bf16")
    ws = tf.workspace(c.cache.tree_attention_workspace_bytes(g, 4, P))
    out = c.run(ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    c.check(out)
    assert torch.equal(out, c.run(ws=ws))


def test_8_bit_heads_whose_prefix_is_one_part(tf):
    from test_gpu_trees import test_large_batches_give_each_sequence_its_own_bits as same_as_16_bits
    same_as_16_bits(tf, 3, 4, 77, 1, 1300, "e4m3")


# ---------------------------------------------------------------- calls side by side, passes in a graph, far offsets
def normal_rows(gen, rows, heads):
    return torch.randn((rows, heads * 128), generator=gen, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_prompt_and_trees_at_the_same_time(tf, fmt):
    """On two streams, each with workspaces of its own: the bits of calls by themselves."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(8)
    x, starts = normal_rows(gen, 3000, 32 + 16), torch.tensor([0, 5, 1400, 3000], device="cuda")
    q, k, v = x[:, :4096], x[:, 4096:5120], x[:, 5120:]
    B, n, P = 12, 32, 5003
    cache, prefix = tf.KVBatch(B, 4, 512, fmt), tf.KVBatch(1, 4, 5120, fmt)
    cache.store(normal_rows(gen, B * 512, 4), normal_rows(gen, B * 512, 4), dev_pos([0] * B))
    prefix.store(normal_rows(gen, 5120, 4), normal_rows(gen, 5120, 4), dev_pos([0]))
    tq, pos, tree = normal_rows(gen, B * n, 32), dev_pos([37 * b for b in range(B)]), dev_i32([[-1] + [i // 2 for i in range(n - 1)]] * B)
    size = cache.tree_attention_workspace_bytes(8, n, P)

    def prompt(out, ws, stream=None):
        tf.prompt_attention(q, k, v, 8, 4, starts, out=out, ws=ws, stream=stream)

    def trees(out, ws, stream=None):
        cache.tree_attention(tq, 8, pos, tree, prefix=prefix, prefix_len=P, out=out, ws=ws, stream=stream)
    wide = torch.empty((3000, 4096), dtype=torch.bfloat16, device="cuda")
    want, two = [wide, torch.empty_like(tq)], [tf.workspace(256), tf.workspace(size)]
    prompt(want[0], two[0])
    trees(want[1], two[1])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(3):
        got = [torch.zeros_like(t) for t in want]
        torch.cuda.synchronize()
        for _ in range(5):
            prompt(got[0], two[0], streams[0])
            trees(got[1], two[1], streams[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(tf.workspace_status(ws) == tf.TF_DEV_OK for ws in two)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_captured_pass_over_trees(tf, fmt):
    """Store, attention, acceptance and the kept entries in one graph, replayed for other trees and positions: what the calls
    do one by one."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    B, n, n_kv, g, P = 3, 20, 2, 4, 700
    pair = [tf.KVBatch(B, n_kv, 512, fmt) for _ in range(2)]
    prefix = tf.KVBatch(1, n_kv, 768, fmt)
    prefix.store(normal_rows(gen, 768, n_kv), normal_rows(gen, 768, n_kv), dev_pos([0]))
    start = normal_rows(gen, B * 400, n_kv)
    for c in pair:
        c.store(start, start, dev_pos([0] * B))
    x = normal_rows(gen, B * n, n_kv * (g + 2))
    pos, ints = dev_pos([0] * B), dev_i32([[[-1] + [0] * (n - 1)] * B, [[0] * n] * B, [[0] * n] * B])
    ws = tf.workspace(pair[0].tree_attention_workspace_bytes(g, n, P))
    ko, vo = n_kv * g * 128, n_kv * (g + 1) * 128

    def step(cache, ws=None):
        cache.store(x[:, ko:vo], x[:, vo:], pos, ws=ws)
        o = cache.tree_attention(x[:, :ko], g, pos, ints[0], prefix=prefix, prefix_len=P, ws=ws)
        took = tf.tree_accept(ints[0], ints[1], ints[2], pos, ws=ws)
        cache.keep(pos, took[2], ws=ws)
        return [o, *took]
    step(pair[0], ws)
    step(pair[1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step(pair[0], ws)
    for i, at in enumerate(([400, 380, -1], [405, -1, 3], [410, 399, 200])):
        x.copy_(normal_rows(gen, B * n, n_kv * (g + 2)))
        pos.copy_(dev_pos(at))
        ints.copy_(dev_i32([[[-1] + [(7 * b + i + r) % r for r in range(1, n)] for b in range(B)],
                            [[(3 * r + b) % 2 for r in range(n)] for b in range(B)],
                            [[(r + b + i) % 2 for r in range(n)] for b in range(B)]]))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(held, step(pair[1])))
        assert torch.equal(pair[0].k, pair[1].k) and torch.equal(pair[0].v, pair[1].v)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


def test_a_prompt_past_32_bits_of_elements(tf):
    """Offsets into the rows pass 2^32 bytes and 2^31 elements."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(10)
    n, each, n_kv, g = 1024, 300, 8, 8
    x = torch.empty((n * each, (n_kv * g + 2 * n_kv) * 128), dtype=torch.bfloat16, device="cuda")
    part = normal_rows(gen, 4 * each, n_kv * (g + 2))
    for s in range(0, n, 4):
        x[s * each:(s + 4) * each] = part
    x[-each:] = normal_rows(gen, each, n_kv * (g + 2))
    assert n * each * n_kv * g * 128 > 2 ** 31

    def call(rows, starts, ws=None):
        q, k, v = rows[:, :n_kv * g * 128], rows[:, n_kv * g * 128:n_kv * (g + 1) * 128], rows[:, n_kv * (g + 1) * 128:]
        return tf.prompt_attention(q, k, v, n_kv, g, torch.tensor(starts, device="cuda"), ws=ws)
    ws = tf.workspace(256)
    out = call(x, [each * s for s in range(n + 1)], ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    for s in (0, 1, n // 2, n - 2, n - 1):
        assert torch.equal(out[s * each:(s + 1) * each], call(x[s * each:(s + 1) * each].contiguous(), [0, each]))


@pytest.mark.parametrize("pos", FAR)
def test_the_calls_of_one_cache_take_no_position_past_its_entries(tf, pos):
    cache, ws = tf.KVCache(2, 256), tf.workspace(256)
    rows = torch.ones((8, 256), dtype=torch.bfloat16, device="cuda")
    cache.append(rows, rows, dev_pos([pos]), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and not cache.k.any() and not cache.v.any()
    out, ws = torch.full((8, 256), 7.0, device="cuda"), tf.workspace(cache.workspace_bytes(1, 8))
    cache.attention(rows, 1, dev_pos([pos]), out=out, ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and (out == 7).all()
