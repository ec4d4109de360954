"""Trees of drafted tokens on the GPU through the binding: attention of their nodes,
acceptance along them and the accepted entries, against oracle/trees.py in fp64.

Attention's tolerance is that of the batch attention (one bf16 rounding of the output,
2^-8 of the value; one of the weights, 2^-8 of sum w|v|; 2^-12 of it for
scores and sums in fp32, times 1 + 2^-6 for the products of these); acceptance and entries are exact.
"""

import numpy as np
import pytest
import torch

from oracle import batch as obat
from oracle import trees as otree
from oracle.linear import bf16_to_f64
from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16

pytestmark = pytest.mark.gpu
D = 128


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


def dev_i32(p):
    return torch.tensor(p, dtype=torch.int32, device="cuda")


def random_tree(rng, used, n, back=6):
    parents, depth = [-1], [0]
    while len(parents) < used:
        p = int(rng.integers(max(0, len(parents) - back), len(parents)))
        p = 0 if depth[p] == 15 else p
        parents.append(p)
        depth.append(depth[p] + 1)
    return parents + [-1] * (n - used)


def rows_of(k):
    """[n_seq][n_kv][R][128] -> [n_seq*R][n_kv*128]."""
    n_seq, n_kv, R, _ = k.shape
    return np.ascontiguousarray(k.transpose(0, 2, 1, 3).reshape(n_seq * R, n_kv * D))


def depths(parents):
    return [len(otree.tree_path(parents, i)) - 1 for i in range(len(parents))]


class Case:
    """A batch of trees with its caches on the device and its logical arrays on the host."""

    def __init__(self, tf, seed, parents, n_kv, g, P, pos, fmt, max_len=None, q_std=2.0):
        rng = inputs.rng_for(seed)
        B, n = len(parents), len(parents[0])
        L = max_len or -(-(max(pos) + n) // 256) * 256
        self.tf, self.parents, self.pos, self.g, self.P, self.n_kv, self.fmt = tf, parents, pos, g, P, n_kv, fmt
        self.q = inputs.bf16_normal(rng, (B, n, n_kv, g, D), q_std)
        sk, sv = (inputs.bf16_normal(rng, (1, n_kv, P, D)) for _ in range(2))
        entries = min(L, max(pos) + n + 3)       # a few entries past the last node: never to be read
        self.bits = [inputs.bf16_normal(rng, (B, n_kv, entries, D)) for _ in range(2)]
        self.cache = tf.KVBatch(B, n_kv, L, fmt)
        self.cache.store(*(dev_bits16(rows_of(b)) for b in self.bits), dev_pos([0] * B))
        self.prefix = None
        if P:
            self.prefix = tf.KVBatch(1, n_kv, -(-P // 256) * 256, fmt)
            self.prefix.store(dev_bits16(rows_of(sk)), dev_bits16(rows_of(sv)), dev_pos([0]))
        self.shared = [self.values(sk)[0], self.values(sv)[0]]
        self.own = [self.values(b) for b in self.bits]

    def values(self, bits):
        x = bf16_to_f64(bits)
        if self.fmt == "bf16" or not x.size:
            return x
        flat = x.reshape(-1, D)
        return np.stack([obat.e4m3_values(*obat.e4m3_vector(v)) for v in flat]).reshape(x.shape)

    def q_dev(self):
        B, n = self.q.shape[:2]
        return dev_bits16(self.q.reshape(B * n, -1))

    def run(self, **kw):
        a = dict(parents=dev_i32(self.parents), prefix=self.prefix, prefix_len=self.P)
        return self.cache.tree_attention(self.q_dev(), self.g, dev_pos(self.pos), **{**a, **kw})

    def check(self, out):
        ref, spread = otree.attention_tree(bf16_to_f64(self.q), *self.shared, *self.own, self.pos, self.parents)
        got = out.view(torch.bfloat16).double().cpu().numpy().reshape(ref.shape)
        tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6)
        assert np.all(np.isfinite(got))
        worst = np.max(np.abs(got - ref) - tol)
        assert worst <= 0, f"off by {worst:.3e} more than allowed"
        assert np.linalg.norm(got - ref) <= 4e-3 * np.linalg.norm(ref)


def chain(n):
    return [-1] + list(range(n - 1))


def star(n):
    return [-1] + [0] * (n - 1)


def trees(seed, n, *used):
    rng = inputs.rng_for(seed)
    return [random_tree(rng, u, n) for u in used]


CASES = [  # trees, n_kv, group, prefix, pos
    ([chain(1)], 1, 1, 0, [0]),                                     # one key
    ([chain(1)], 1, 1, 1, [0]),                                     # one shared key, one own
    ([chain(16)], 1, 8, 0, [0]),                                    # the longest path, from position 0
    ([star(9), chain(9)], 2, 4, 5, [0, 30]),
    (trees(1, 24, 24, 20, 1), 2, 4, 127, [0, 128, 5]),              # unused rows
    (trees(2, 7, 7, 7, 5), 1, 5, 128, [127, 126, 250]),
    (trees(3, 33, 33, 30), 3, 3, 129, [509, 700]),                  # nodes on both sides of 512, of a warp's lanes
    (trees(4, 12, 12, 12, 12, 7), 8, 8, 300, [40, -1, 0, 513]),     # an idle sequence
    (trees(5, 64, 64, 50), 1, 16, 640, [3, 1000]),                  # the widest tree and group
    (trees(6, 64, 64), 2, 8, 0, [1300]),
    (trees(7, 40, *range(30, 39)), 1, 8, 257, [0, 5, 100, 250, 256, 3, 9, 80, 31]),
    (trees(8, 5, *[5] * 33), 1, 1, 2000, [17 * i % 90 for i in range(33)]),
    (trees(9, 16, 16, 16), 2, 8, 3333, [1234, 2]),
    (trees(10, 26, 26), 4, 7, 0, [1531]),
    (trees(11, 20, *[20] * 6), 8, 8, 4096, [511, 512, 513, 1023, 1024, 1]),
    ([chain(15) + [0], star(15) + [14]], 2, 6, 40, [15, 16]),       # positions where far entries begin
    ([chain(2), chain(2), chain(2)], 2, 2, 0, [14, 15, 16]),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("parents,n_kv,g,P,pos", CASES)
def test_attention_tree(tf, parents, n_kv, g, P, pos, fmt):
    c = Case(tf, 100 * len(pos) + len(parents[0]), parents, n_kv, g, P, pos, fmt)
    ws = tf.workspace(c.cache.tree_attention_workspace_bytes(g, len(parents[0]), P))
    out = c.run(ws=ws)
    assert out.dtype == torch.bfloat16 and tf.workspace_status(ws) == tf.TF_DEV_OK
    c.check(out)
    for _ in range(3):
        assert torch.equal(out, c.run(ws=ws))       # the same bits again, on a used workspace


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("g,P,pos", [(8, 1500, 700), (3, 130, 506), (1, 0, 3), (16, 0, 1020), (5, 20, 0)])
def test_a_node_is_its_path_decoded_one_token_a_pass(tf, fmt, g, P, pos):
    """The guarantee: a node's bits are those of serial decoding, where its ancestors were
    committed one after the other."""
    n_kv, (parents,) = 2, trees(20 + g, 40, 40)
    c = Case(tf, 77, [parents], n_kv, g, P, [pos], fmt)
    out = c.run().view(40, -1)
    q = c.q_dev().view(torch.bfloat16)
    for i in range(0, 40, 3):
        path = otree.tree_path(parents, i)
        serial = tf.KVBatch(1, n_kv, c.cache.max_len, fmt)
        at = list(range(pos)) + [pos + a for a in path]
        serial.store(*(dev_bits16(rows_of(b[:, :, at])) for b in c.bits), dev_pos([0]))
        for d, node in enumerate(path):
            one = serial.tree_attention(q[node:node + 1], g, dev_pos([pos + d]), dev_i32([[-1]]), prefix=c.prefix,
                                        prefix_len=P)
            assert torch.equal(one[0], out[node]), (i, d)
        half = len(path) // 2       # a pass that starts inside the path
        rest = serial.tree_attention(q[path[half:]], g, dev_pos([pos + half]), dev_i32([chain(len(path) - half)]),
                                     prefix=c.prefix, prefix_len=P)
        assert torch.equal(rest, out[path[half:]])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_sequences_stand_alone(tf, fmt):
    """Neither the other sequences nor the number of rows change a node's bits."""
    g, P, n_kv, pos = 4, 700, 2, [100, 600, -1, 0, 2000]
    parents = trees(31, 30, 30, 25, 30, 9, 30)
    c = Case(tf, 5, parents, n_kv, g, P, pos, fmt)
    out = c.run().view(5, 30, -1)
    assert not out[2].any() and not out[1, 25:].any()
    for b in (0, 1, 3, 4):
        cache = tf.KVBatch(1, n_kv, c.cache.max_len, fmt)
        cache.store(*(dev_bits16(rows_of(x[b:b + 1])) for x in c.bits), dev_pos([0]))
        used = 9 if b == 3 else 12
        q = c.q_dev().view(torch.bfloat16).view(5, 30, -1)[b, :used].contiguous()
        some = cache.tree_attention(q, g, dev_pos([pos[b]]), dev_i32([parents[b][:used]]), prefix=c.prefix, prefix_len=P)
        assert torch.equal(some, out[b, :used])


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("pos", [0, 500, 505, 1022])
def test_nodes_do_not_see_what_is_off_their_path(tf, fmt, bad, pos):
    """Entries of other nodes, of unused rows and past the tree may hold anything."""
    parents = trees(41, 20, 14)
    c = Case(tf, 6, parents, 2, 8, 300, [pos], fmt)
    clean = c.run()
    hit = 5
    rows = [torch.full((1, 2 * D), bad, dtype=torch.bfloat16, device="cuda")] * 2
    for slot in [hit, *range(14, 23)]:
        c.cache.store(*rows, dev_pos([pos + slot]))
    out = c.run()
    for i in range(20):
        if hit in otree.tree_path(parents[0], i):
            assert torch.isnan(out[i]).all()
        else:
            assert torch.equal(out[i], clean[i]), i


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_committed_infinities_reach_the_nodes_that_see_them(tf, fmt):
    """A committed value that is not finite reaches every node of its sequence, at any distance, and no other
    sequence."""
    for slot in (3, 590, 599):
        c = Case(tf, 8, trees(43, 20, 20, 20), 1, 4, 100, [600, 600], fmt)
        clean = c.run().view(2, 20, -1)
        k, v = (dev_bits16(rows_of(b[:, :, slot:slot + 1])).view(torch.bfloat16).clone() for b in c.bits)
        v[0, 7] = float("inf")
        c.cache.store(k, v, dev_pos([slot, slot]))
        out = c.run().view(2, 20, 4, D)
        assert torch.equal(out[1].reshape(20, -1), clean[1])
        assert not torch.isfinite(out[0, :, :, 7]).any()


BAD_TREES = [[0, 0, 0, 0], [-1, 1, 0, 0], [-1, 0, 3, 0], [-1, -1, 1, 0], [-1, 0, -2, 0], [-1, 0, 0, 99], [3, 0, 0, 0]]


@pytest.mark.parametrize("tree", BAD_TREES)
def test_parents_that_are_no_tree(tf, tree):
    c = Case(tf, 9, [tree, [-1, 0, 0, 1]], 2, 4, 30, [50, 40], "bf16")
    ws = tf.workspace(c.cache.tree_attention_workspace_bytes(4, 4, 30))
    out = c.run(ws=ws).view(2, 4, -1)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_TREE and not out[0].any()
    c.parents = [star(4), [-1, 0, 0, 1]]
    assert torch.equal(c.run(ws=ws).view(2, 4, -1)[1], out[1]) and tf.workspace_status(ws) == tf.TF_DEV_OK
    any32 = dev_i32([[1, 2, 3, 4], [5, 6, 7, 8]])
    accepted, bonus, path, committed = tf.tree_accept(dev_i32([tree, star(4)]), any32, any32, dev_pos([50, 40]), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_TREE
    assert accepted.tolist() == [-1, 0] and bonus.tolist() == [-1, 5]
    assert (path[0] == -1).all() and (committed[0] == -1).all()


def test_paths_that_are_too_long(tf):
    for parents in (chain(17), chain(64), [-1] + [0] * 10 + [10] + list(range(11, 26))):
        c = Case(tf, 9, [parents], 1, 1, 0, [50], "bf16")
        ws = tf.workspace(c.cache.tree_attention_workspace_bytes(1, len(parents), 0))
        assert not c.run(ws=ws).any() and tf.workspace_status(ws) == tf.TF_DEV_BAD_TREE


def test_bad_positions(tf):
    c = Case(tf, 9, [star(8)] * 3, 1, 4, 30, [10, 20, 30], "e4m3")
    ws = tf.workspace(c.cache.tree_attention_workspace_bytes(4, 8, 30))
    good = c.run(ws=ws).view(3, 8, -1)
    for p in (-2, 249, 1 << 40):
        c.pos = [10, p, 30]
        out = c.run(ws=ws).view(3, 8, -1)
        assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and not out[1].any()
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    c.pos = [10, 248, 30]       # the last that fits
    c.run(ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


def test_a_position_past_32_bits_of_elements(tf):
    """Offsets into the caches pass 2^32 bytes."""
    n_kv, L = 64, 1 << 18        # 64 x 2^18 x 128 two-byte elements: 4 GB in each half
    cache, small = tf.KVBatch(1, n_kv, L), tf.KVBatch(1, n_kv, 256)
    rng = inputs.rng_for(12)
    rows = [dev_bits16(inputs.bf16_normal(rng, (20, n_kv * D))) for _ in range(2)]
    q = dev_bits16(inputs.bf16_normal(rng, (8, n_kv * D), 2.0))
    tree = dev_i32(trees(51, 8, 8))
    pos = L - 8
    cache.k[:, :, :pos - 12] = 0
    cache.store(*rows, dev_pos([pos - 12]))
    ws = tf.workspace(cache.tree_attention_workspace_bytes(1, 8))
    got = cache.tree_attention(q, 1, dev_pos([pos]), tree, ws=ws).double().cpu().numpy()
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    k, v = (t.view(torch.bfloat16).double().cpu().numpy().reshape(20, n_kv, D) for t in rows)
    qn = q.view(torch.bfloat16).double().cpu().numpy().reshape(8, n_kv, D)
    parents = tree[0].tolist()
    for i in (0, 7):
        at = list(range(12)) + [12 + a for a in otree.tree_path(parents, i)]
        for j in (0, 63):        # the zero keys before: weight e^0 each, values 0
            s = np.concatenate([np.zeros(1), qn[i, j] @ k[at, j].T / np.sqrt(D)])
            top = s.max()
            w = np.exp(s - top)
            total = w[1:].sum() + w[0] * (pos - 12)
            ref = w[1:] @ v[at, j] / total
            spread = w[1:] @ np.abs(v[at, j]) / total
            tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6)
            assert np.all(np.abs(got[i].reshape(n_kv, D)[j] - ref) <= tol)


def test_strided_buffers_and_streams(tf):
    c = Case(tf, 15, trees(53, 10, 10, 8), 2, 4, 200, [60, 300], "bf16")
    ref = c.run()
    wide = torch.full((20, 8 * D + 48), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + 8 * D] = c.q_dev().view(torch.bfloat16)
    out = torch.full((20, 8 * D + 24), 5.0, dtype=torch.bfloat16, device="cuda")
    c.cache.tree_attention(wide[:, 16:16 + 8 * D], 4, dev_pos(c.pos), dev_i32(c.parents), prefix=c.prefix, prefix_len=200,
                           out=out[:, 8:8 + 8 * D])
    assert torch.equal(out[:, 8:8 + 8 * D], ref) and (out[:, :8] == 5).all() and (out[:, 8 + 8 * D:] == 5).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, ref)


def test_a_captured_pass_reads_positions_and_trees_anew(tf):
    c = Case(tf, 17, trees(55, 12, 12, 12), 2, 4, 600, [60, 900], "e4m3")
    q, pos, tree = c.q_dev(), dev_pos([0, 0]), dev_i32([chain(12), chain(12)])
    out = torch.zeros((24, 8 * D), dtype=torch.bfloat16, device="cuda")
    ws = tf.workspace(c.cache.tree_attention_workspace_bytes(4, 12, 600))

    def call():
        c.cache.tree_attention(q, 4, pos, tree, prefix=c.prefix, prefix_len=600, out=out, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for parents, at in ((c.parents, [60, 900]), ([star(12)] * 2, [700, -1]), (c.parents, [3, 4])):
        pos.copy_(dev_pos(at))
        tree.copy_(dev_i32(parents))
        graph.replay()
        c.parents, c.pos = parents, at
        assert torch.equal(out, c.run())
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


def test_a_workspace_that_batch_attention_used(tf):
    c = Case(tf, 19, [chain(8)] * 2, 2, 4, 900, [60, 300], "bf16")
    ref = c.run()
    ws = tf.workspace(max(c.cache.tree_attention_workspace_bytes(4, 8, 900), c.cache.attention_workspace_bytes(4, 8, 900)))
    for _ in range(2):
        a = c.cache.attention(c.q_dev(), 4, dev_pos(c.pos), prefix=c.prefix, prefix_len=900, ws=ws)
        assert torch.equal(c.run(ws=ws), ref)
        c.check(a)      # a chain: the same formula
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


@pytest.mark.parametrize("B,n,n_kv,g,P,fmt", [
    (57, 64, 1, 8, 700, "bf16"),        # many CTAs of the sum; two tiles an item
    (13, 64, 1, 8, 700, "e4m3"),        # fewer
    (64, 64, 2, 1, 333, "bf16"),        # one query head
    (20, 64, 2, 8, 5003, "e4m3"),       # the 8-bit prefix is expanded first
    (64, 40, 1, 16, 9001, "e4m3"),
    (9, 50, 8, 3, 1207, "bf16"),
])
def test_large_batches_give_each_sequence_its_own_bits(tf, B, n, n_kv, g, P, fmt):
    """Whatever form the size of a batch asks for, a sequence's bits are those it has alone, and an 8-bit cache's
    those of its values in 16 bits.  Twice, with other entries, on one workspace."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(B + P)
    pos = [(37 * b) % 450 - (b % 5 == 4) * 10 ** 6 for b in range(B)]
    pos = [p if p >= 0 else -1 for p in pos]
    parents = trees(71, n, *[1 + (13 * b) % n for b in range(B)])
    L = -(-(450 + n) // 256) * 256

    def normal(rows, heads, std=1.0):
        return (std * torch.randn((rows, heads * D), generator=gen, device="cuda")).to(torch.bfloat16)
    cache, prefix = tf.KVBatch(B, n_kv, L, fmt), tf.KVBatch(1, n_kv, -(-P // 256) * 256, fmt)
    ws = tf.workspace(cache.tree_attention_workspace_bytes(g, n, P))
    for _ in range(2):
        q, own, shared = normal(B * n, n_kv * g, 2.0), [normal(B * L, n_kv) for _ in range(2)], [normal(P, n_kv) for _ in range(2)]
        cache.store(*own, dev_pos([0] * B))
        prefix.store(*shared, dev_pos([0]))
        out = cache.tree_attention(q, g, dev_pos(pos), dev_i32(parents), prefix=prefix, prefix_len=P, ws=ws)
        assert tf.workspace_status(ws) == tf.TF_DEV_OK
        if fmt == "e4m3":
            wide, wide_prefix = tf.KVBatch(B, n_kv, L), tf.KVBatch(1, n_kv, prefix.max_len)
            wide.store(*cache.load(dev_pos([0] * B), L), dev_pos([0] * B))
            wide_prefix.store(*prefix.load(dev_pos([0]), P), dev_pos([0]))
            assert torch.equal(out, wide.tree_attention(q, g, dev_pos(pos), dev_i32(parents), prefix=wide_prefix, prefix_len=P))
        out = out.view(B, n, -1)
        for b in (0, B // 2, B - 1):
            one = tf.KVBatch(1, n_kv, L, fmt)
            one.store(*(x.view(B, L, -1)[b].contiguous() for x in own), dev_pos([0]))
            alone = one.tree_attention(q.view(B, n, -1)[b].contiguous(), g, dev_pos([pos[b]]), dev_i32([parents[b]]), prefix=prefix,
                                       prefix_len=P)
            assert torch.equal(alone, out[b])
            assert bool(alone.any()) == (pos[b] >= 0)


def test_two_graphs_share_a_workspace(tf):
    """One with its 8-bit prefix expanded first (four grids, two of them at once), one without."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)

    def normal(rows, heads, std=1.0):
        return (std * torch.randn((rows, heads * D), generator=gen, device="cuda")).to(torch.bfloat16)
    calls = []
    for B, n, n_kv, g, P in ((20, 64, 2, 8, 5003), (3, 10, 2, 4, 700)):
        cache, prefix = tf.KVBatch(B, n_kv, 512, "e4m3"), tf.KVBatch(1, n_kv, -(-P // 256) * 256, "e4m3")
        cache.store(normal(B * 512, n_kv), normal(B * 512, n_kv), dev_pos([0] * B))
        prefix.store(normal(P, n_kv), normal(P, n_kv), dev_pos([0]))
        q, pos = normal(B * n, n_kv * g, 2.0), dev_pos([(31 * b) % 440 for b in range(B)])
        tree, out = dev_i32(trees(81, n, *[n - b % 4 for b in range(B)])), torch.zeros((B * n, n_kv * g * D), dtype=torch.bfloat16, device="cuda")
        calls.append((cache, prefix, q, pos, tree, out, g, n, P))
    ws = tf.workspace(max(c[0].tree_attention_workspace_bytes(c[6], c[7], c[8]) for c in calls))

    def call(c, out, ws):
        c[0].tree_attention(c[2], c[6], c[3], c[4], prefix=c[1], prefix_len=c[8], out=out, ws=ws)
    graphs = []
    for c in calls:
        call(c, c[5], ws)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(c, c[5], ws)
    for i in (0, 1, 1, 0, 0, 1):
        c = calls[i]
        c[2].copy_(normal(c[2].shape[0], c[2].shape[1] // D, 2.0))
        c[5].zero_()
        graphs[i].replay()
        want = torch.empty_like(c[5])
        call(c, want, None)
        assert torch.equal(c[5], want)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


# ---------------------------------------------------------------- acceptance
@pytest.mark.parametrize("B,n,vocab", [(1, 1, 3), (1, 8, 3), (3, 33, 2), (5, 64, 4), (130, 20, 2), (1024, 64, 3)])
def test_accept(tf, B, n, vocab):
    rng = inputs.rng_for(B + n)
    parents = [random_tree(rng, int(rng.integers(1, n + 1)), n) for _ in range(B)]
    tokens, sampled = (rng.integers(0, vocab, (B, n)).tolist() for _ in range(2))
    pos = [-1 if b % 7 == 3 else int(rng.integers(0, 1 << 40)) for b in range(B)]
    ws = tf.workspace(256)
    got = tf.tree_accept(dev_i32(parents), dev_i32(tokens), dev_i32(sampled), dev_pos(pos), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    accepted, bonus, path, committed = (t.tolist() for t in got)
    for b in range(B):
        want = otree.accept_tree(parents[b], tokens[b], sampled[b]) if pos[b] >= 0 else (-1, -1, [], [])
        pad = [-1] * 16
        assert (accepted[b], bonus[b], path[b], committed[b]) == (want[0], want[1], (want[2] + pad)[:16], (want[3] + pad)[:16])


def test_accept_the_longest_path_and_a_bad_position(tf):
    ws = tf.workspace(256)
    tree, tokens = dev_i32([chain(16)] * 2), dev_i32([list(range(16))] * 2)
    sampled = dev_i32([list(range(1, 17))] * 2)
    accepted, bonus, path, committed = tf.tree_accept(tree, tokens, sampled, dev_pos([0, -5]), ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION
    assert accepted.tolist() == [15, -1] and bonus.tolist() == [16, -1]
    assert path.tolist() == [list(range(16)), [-1] * 16] and committed.tolist() == [list(range(1, 17)), [-1] * 16]


def test_accept_on_a_graph_and_a_stream(tf):
    tree, tokens, pos = dev_i32([star(6)]), dev_i32([[0, 4, 5, 5, 6, 7]]), dev_pos([9])
    sampled = dev_i32([[5, 1, 2, 3, 4, 5]])
    side, ws = torch.cuda.Stream(), tf.workspace(256)
    torch.cuda.synchronize()
    got = tf.tree_accept(tree, tokens, sampled, pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0].item() == 1 and got[1].item() == 2 and got[2][0, :3].tolist() == [0, 2, -1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = tf.tree_accept(tree, tokens, sampled, pos, ws=ws)
    sampled.copy_(dev_i32([[7, 1, 2, 3, 4, 9]]))
    graph.replay()
    assert held[0].item() == 1 and held[1].item() == 9 and held[2][0, :3].tolist() == [0, 5, -1]


# ---------------------------------------------------------------- the accepted entries
def paths(rng, B, n):
    out = []
    for b in range(B):
        m = int(rng.integers(0, min(16, n)))
        out.append([0] + sorted(rng.choice(np.arange(1, n), m, replace=False).tolist()) if n > 1 else [0])
    return out


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,n,n_kv,L", [(1, 1, 1, 256), (1, 8, 8, 256), (3, 64, 3, 512), (40, 20, 2, 256), (2, 17, 128, 256)])
def test_keep(tf, fmt, B, n, n_kv, L):
    rng = inputs.rng_for(B * n)
    cache, ws = tf.KVBatch(B, n_kv, L, fmt), tf.workspace(256)
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:       # any bits at all: they are moved as they are
            t.copy_(torch.from_numpy(rng.integers(0, 200, tuple(t.shape))).to(t.dtype))
    pos = [L - n if b % 3 == 0 else int(rng.integers(0, L - n + 1)) for b in range(B)]
    if B > 2:
        pos[1] = -1
    way = paths(rng, B, n)

    def entries():      # as stored, one sequence's entries in order
        out = []
        for t in (cache.k, cache.v):
            x = t.cpu().numpy()
            if fmt == "bf16":
                at = np.arange(L)[:, None]
                d = np.arange(D)[None]
                x = np.take_along_axis(x, np.broadcast_to(8 * ((d // 8) ^ (at % 8)) + d % 8, x.shape), axis=3)
            out.append(x.copy())
        return out + ([t.cpu().numpy().copy() for t in (cache.k_scale, cache.v_scale)] if fmt == "e4m3" else [])
    want = entries()
    for b, p in enumerate(pos):
        if p >= 0:
            for x in want:
                x[b, :, p:p + len(way[b])] = x[b][:, [p + i for i in way[b]]]
    pad = dev_i32([(w + [-1] * 16)[:16] for w in way])
    assert cache.keep(dev_pos(pos), pad, ws=ws) is ws
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    for x, y in zip(entries(), want):
        assert np.array_equal(x, y)


@pytest.mark.parametrize("path,pos,status", [
    ([1, 2], 10, "TREE"), ([0, 2, 2], 10, "TREE"), ([0, 5, 3], 10, "TREE"), ([0, -1, 3], 10, "TREE"),
    ([0, 64], 10, "TREE"), ([0, -2], 10, "TREE"), ([-1, 1], 10, "TREE"), ([0, 2], -2, "POSITION"), ([0, 8], 248, "POSITION"),
    ([0, 3], 1 << 40, "POSITION"), ([-1, -1], 10, "OK"), ([0, 8], -1, "OK")])
def test_keep_refuses_what_is_no_path(tf, path, pos, status):
    cache, ws = tf.KVBatch(2, 1, 256), tf.workspace(256)
    cache.k.copy_(torch.arange(cache.k.numel(), device="cuda").view(cache.k.shape).to(torch.int16))
    was = cache.k.clone()
    other = [0, 4] + [-1] * 14
    cache.keep(dev_pos([pos, 16]), dev_i32([path + [-1] * (16 - len(path)), other]), ws=ws)
    assert tf.workspace_status(ws) == getattr(tf, f"TF_DEV_{'BAD_' if status != 'OK' else ''}{status}")
    assert torch.equal(cache.k[0], was[0]) and not torch.equal(cache.k[1], was[1])


# ---------------------------------------------------------------- a pass as decoding runs it
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_passes_over_trees_leave_what_serial_decoding_leaves(tf, fmt):
    """Passes of rotation, store, attention, acceptance and keep; "sampling" takes a token
    from the attention's own bits, so a wrong bit anywhere changes what follows.  The tokens and
    cache entries are those of one token a pass."""
    n_kv, g, P, B, L, vocab, n = 2, 4, 150, 3, 256, 5, 20
    cols = n_kv * (g + 2) * D
    rng = inputs.rng_for(61)
    rows = dev_bits16(inputs.bf16_normal(rng, (vocab, cols), 2.0)).view(torch.bfloat16)     # a token's projection
    turns = tf.rope_turns(D, 1e4)
    shared = tf.KVBatch(1, n_kv, 256, fmt)
    start = rows[torch.from_numpy(rng.integers(0, vocab, P)).cuda()]
    shared.store(start[:, n_kv * g * D:n_kv * (g + 1) * D].contiguous(), start[:, n_kv * (g + 1) * D:].contiguous(), dev_pos([0]))
    ko, vo = n_kv * g * D, n_kv * (g + 1) * D

    def run(draft):
        cache, ws = tf.KVBatch(B, n_kv, L, fmt), tf.workspace(256)
        last, at, out = [1] * B, [0] * B, [[] for _ in range(B)]
        passes = 0
        while min(len(o) for o in out) < 40:
            parents, tokens = zip(*(draft(b, last[b], out[b]) for b in range(B)))
            tree, toks, pos, m = dev_i32(parents), dev_i32(tokens), dev_pos(at), len(parents[0])
            deep = [[max(d, 0) for d in depths(p)] for p in parents]
            where = dev_pos([a + d for a, ds in zip(at, deep) for d in ds])
            x = tf.qk_norm_rope(rows[toks.reshape(-1).long()], n_kv * g, n_kv, where, turns, pos_offset=P)
            cache.store(x[:, ko:vo], x[:, vo:], pos, ws=ws)
            o = cache.tree_attention(x[:, :ko], g, pos, tree, prefix=shared, prefix_len=P)
            bits = o.view(torch.int16).long()
            sampled = ((bits * torch.arange(1, ko + 1, device="cuda")).sum(-1) % vocab).to(torch.int32).view(B, m)
            accepted, bonus, path, committed = tf.tree_accept(tree, toks, sampled, pos, ws=ws)
            cache.keep(pos, path, ws=ws)
            assert tf.workspace_status(ws) == tf.TF_DEV_OK
            for b in range(B):
                a = accepted[b].item()
                out[b] += committed[b, :a + 1].tolist()
                last[b], at[b] = bonus[b].item(), at[b] + a + 1
            passes += 1
        kept = cache.load(dev_pos([0] * B), 40)
        return [o[:40] for o in out], passes, [t.view(B, 40, -1) for t in kept]

    def none(b, last, out):
        return [-1], [last]

    def tree(b, last, out):
        used = n - 4 * b            # the rest unused
        r = np.random.default_rng([b, len(out)])
        return random_tree(r, used, n), [last] + r.integers(0, vocab, n - 1).tolist()
    serial, many, kept = run(none)
    drafted, few, kept_too = run(tree)
    assert serial == drafted and few < many
    assert all(torch.equal(x, y) for x, y in zip(kept, kept_too))
