"""Attention of a batch of sequences over a shared prefix and their own entries, on the
GPU through the binding, against oracle/batch.py in fp64.

Tolerance, per element, with the softmax weights w: the output is rounded to bf16
once (half a step, 2^-8 of the value); the weights may be rounded to bf16 before
the product with v (2^-8 of sum w|v|); scores and sums in fp32 move a weight by
less than 2^-12 of itself for the scores here (|s| < 2^6 with fewer than 2^6
roundings of 2^-24 each).  So |got - ref| <= 2^-8 |ref| + (2^-8 + 2^-12) sum w|v|, times
1 + 2^-6 for the products of these.
"""

import math

import numpy as np
import pytest
import torch

from oracle import batch as obat
from oracle.linear import bf16_to_f64
from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16

pytestmark = pytest.mark.gpu
D = 128


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


def rows_of(k):
    """[n_seq][n_kv][R][128] -> [n_seq*R][n_kv*128]."""
    n_seq, n_kv, R, _ = k.shape
    return np.ascontiguousarray(k.transpose(0, 2, 1, 3).reshape(n_seq * R, n_kv * D))


class Case:
    """A batch with its caches on the device and its logical arrays on the host."""

    def __init__(self, tf, seed, B, R, n_kv, g, P, pos, fmt, max_len=None, q_std=2.0):
        rng = inputs.rng_for(seed)
        L = max_len or -(-(max(pos) + R) // 256) * 256
        self.tf, self.shape, self.pos, self.L = tf, (B, R, n_kv, g, P), pos, L
        self.q = inputs.bf16_normal(rng, (B, R, n_kv, g, D), q_std)
        sk, sv = (inputs.bf16_normal(rng, (1, n_kv, P, D)) for _ in range(2))
        n = min(L, max(pos) + R + 3)       # a few entries past the last row: never to be read
        ok, ov = (inputs.bf16_normal(rng, (B, n_kv, n, D)) for _ in range(2))
        self.cache = tf.KVBatch(B, n_kv, L, fmt)
        self.cache.store(dev_bits16(rows_of(ok)), dev_bits16(rows_of(ov)), dev_pos([0] * B))
        self.prefix = None
        if P:
            self.prefix = tf.KVBatch(1, n_kv, -(-P // 256) * 256, fmt)
            self.prefix.store(dev_bits16(rows_of(sk)), dev_bits16(rows_of(sv)), dev_pos([0]))
        self.held = [self.values(sk)[0], self.values(sv)[0], self.values(ok), self.values(ov)]

    def values(self, bits):
        x = bf16_to_f64(bits)
        if self.cache.fmt == "bf16" or not x.size:
            return x
        flat = x.reshape(-1, D)
        return np.stack([obat.e4m3_values(*obat.e4m3_vector(v)) for v in flat]).reshape(x.shape)

    def q_dev(self):
        B, R, n_kv, g, _ = self.shape
        return dev_bits16(self.q.reshape(B * R, n_kv * g * D))

    def run(self, **kw):
        return self.cache.attention(self.q_dev(), self.shape[3], dev_pos(self.pos), prefix=self.prefix,
                                    prefix_len=self.shape[4], **kw)

    def check(self, out):
        B, R, n_kv, g, _ = self.shape
        ref, spread = obat.attention_batch(bf16_to_f64(self.q), *self.held, self.pos)
        got = out.view(torch.bfloat16).double().cpu().numpy().reshape(ref.shape)
        tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6)
        assert np.all(np.isfinite(got))
        worst = np.max(np.abs(got - ref) - tol)
        assert worst <= 0, f"off by {worst:.3e} more than allowed"
        err = np.linalg.norm(got - ref) / max(np.linalg.norm(ref), 1e-300)
        assert err < 4e-3, err    # rms of the two roundings: sqrt(2) * 2^-8 / sqrt(3) of the spread, at most


CASES = [  # B, R, n_kv, group, prefix, pos
    (1, 1, 1, 1, 0, [0]),                           # one key
    (1, 1, 1, 1, 1, [0]),                           # one shared key, one own
    (1, 16, 1, 8, 0, [0]),                          # growing triangles, 128 query vectors
    (2, 3, 2, 4, 5, [0, 30]),
    (3, 1, 2, 4, 127, [0, 128, 5]),
    (3, 2, 1, 5, 128, [127, 126, 255]),             # rows on both sides of a 128-entry tile
    (2, 5, 3, 3, 129, [509, 700]),                  # rows on both sides of 512
    (4, 1, 8, 8, 300, [40, -1, 0, 513]),            # an idle sequence
    (2, 1, 1, 16, 640, [3, 1000]),
    (5, 7, 2, 16, 1000, [0, 1, 2, 3, 4]),           # 112 vectors a sequence
    (9, 16, 1, 8, 257, [0, 5, 100, 250, 256, 3, 9, 80, 31]),    # 1152 vectors: several tiles
    (40, 1, 2, 2, 513, list(range(0, 400, 10))),    # 80 vectors a head: part of a tile
    (33, 4, 1, 1, 2000, [17 * i % 90 for i in range(33)]),      # 132 vectors: a tile and four rows
    (2, 16, 2, 8, 3333, [1234, 2]),
    (1, 4, 4, 7, 0, [1531]),
    (6, 2, 8, 8, 4096, [511, 512, 513, 1023, 1024, 1]),
]


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("B,R,n_kv,g,P,pos", CASES)
def test_attention_batch(tf, B, R, n_kv, g, P, pos, fmt):
    c = Case(tf, 100 * B + R, B, R, n_kv, g, P, pos, fmt)
    ws = tf.workspace(c.cache.attention_workspace_bytes(g, R, P))
    out = c.run(ws=ws)
    assert out.dtype == torch.bfloat16 and tf.workspace_status(ws) == tf.TF_DEV_OK
    c.check(out)
    for _ in range(3):
        assert torch.equal(out, c.run(ws=ws))       # the same bits again, on a used workspace


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("g,P", [(8, 1500), (3, 130), (1, 0)])
def test_rows_stand_alone(tf, fmt, g, P):
    """A row's bits depend on its query, its position, and the entries it sees: not on R,
    nor on the other sequences, their number or their place."""
    n_kv, R = 2, 6
    pos = [3, 505, 127, 0, 1020]
    c = Case(tf, 77, 5, R, n_kv, g, P, pos, fmt)
    whole = c.run()
    q = c.q_dev()
    for b in range(5):
        one = tf.KVBatch(1, n_kv, c.L, fmt)
        for name in ("k", "v", "k_scale", "v_scale"):
            if getattr(one, name) is not None:
                getattr(one, name).copy_(getattr(c.cache, name)[b:b + 1])
        for r0, n in ((0, 1), (0, R), (R - 1, 1), (2, 3)):
            got = one.attention(q[b * R + r0:b * R + r0 + n], g, dev_pos([pos[b] + r0]), prefix=c.prefix, prefix_len=P)
            assert torch.equal(got, whole[b * R + r0:b * R + r0 + n]), (b, r0, n)


def test_eight_bit_entries_give_the_bits_of_their_values(tf):
    """Attention over E4M3 caches equals attention over bf16 caches holding the values."""
    pos = [700, 3, -1]
    c = Case(tf, 5, 3, 4, 2, 8, 1111, pos, "e4m3")
    own, prefix = tf.KVBatch(3, 2, c.L), tf.KVBatch(1, 2, c.prefix.max_len)
    own.store(*c.cache.load(dev_pos([0] * 3), 704), dev_pos([0] * 3))
    prefix.store(*c.prefix.load(dev_pos([0]), 1111), dev_pos([0]))
    assert torch.equal(own.attention(c.q_dev(), 8, dev_pos(pos), prefix=prefix, prefix_len=1111), c.run())


@pytest.mark.parametrize("B,R,n_kv,g,P", [(40, 2, 2, 8, 1), (23, 3, 1, 8, 127), (17, 16, 2, 2, 1300), (33, 16, 1, 1, 520),
                                          (13, 8, 3, 7, 641)])
def test_many_vectors_over_an_eight_bit_prefix(tf, B, R, n_kv, g, P):
    """Several pairs of query tiles a head: the bits are those of each sequence alone and
    of a bf16 cache of the same values."""
    pos = [(97 * b) % 600 for b in range(B)]
    pos[B // 2] = -1
    c = Case(tf, 31, B, R, n_kv, g, P, pos, "e4m3")
    ws = tf.workspace(c.cache.attention_workspace_bytes(g, R, P))
    whole = c.run(ws=ws).clone()
    c.check(whole)
    assert torch.equal(c.run(ws=ws), whole)
    own, prefix = tf.KVBatch(B, n_kv, c.L), tf.KVBatch(1, n_kv, c.prefix.max_len)
    own.store(*c.cache.load(dev_pos([0] * B), c.L), dev_pos([0] * B))
    prefix.store(*c.prefix.load(dev_pos([0]), P), dev_pos([0]))
    assert torch.equal(own.attention(c.q_dev(), g, dev_pos(pos), prefix=prefix, prefix_len=P), whole)
    q = c.q_dev()
    for b in (0, B // 2, B - 1):
        one = tf.KVBatch(1, n_kv, c.L, "e4m3")
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(one, name).copy_(getattr(c.cache, name)[b:b + 1])
        got = one.attention(q[b * R:(b + 1) * R], g, dev_pos([pos[b]]), prefix=c.prefix, prefix_len=P, ws=ws)
        assert torch.equal(got, whole[b * R:(b + 1) * R]), b
    assert torch.equal(c.run(ws=ws), whole)     # the workspace served the smaller calls in between


def test_many_vectors_over_a_prefix_with_nonfinite_entries(tf):
    """A NaN vector of the prefix reaches its head's rows and no other head's; what lies
    behind the prefix's last entry reaches none."""
    B, R, g, P = 40, 2, 8, 700
    c = Case(tf, 32, B, R, 2, g, P, [b % 5 for b in range(B)], "e4m3")
    want = c.run().clone().reshape(B * R, 2, g * D)
    c.prefix.k_scale[:, :, P:] = 255
    c.prefix.v_scale[:, :, P:] = 255
    assert torch.equal(c.run().reshape(B * R, 2, g * D), want)
    c.prefix.v_scale[0, 1, 600] = 255
    c.prefix.v[0, 1, 600] = 0
    got = c.run().reshape(B * R, 2, g * D)
    assert torch.equal(got[:, 0], want[:, 0]) and bool(got[:, 1].isnan().all())


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_entries_no_row_sees_may_hold_anything(tf, fmt):
    """NaN, infinities and garbage past every sequence's last row and past the prefix."""
    pos = [0, 130, 511, -1]
    c = Case(tf, 6, 4, 2, 2, 4, 200, pos, fmt)
    want = c.run()
    fills = [0x7FC0, 0x7F80, 0xFF80, 0x7F7F] if fmt == "bf16" else [0x7F, 0xFF, 0x55, 0x7E]
    for fill in fills:
        for cache, ends in ((c.cache, [p + 2 if p >= 0 else 0 for p in pos]), (c.prefix, [200])):
            for b, end in enumerate(ends):
                for t in (cache.k, cache.v):
                    t[b, :, end:] = fill - 65536 if fill > 0x7FFF and fmt == "bf16" else fill
                for t in (cache.k_scale, cache.v_scale):
                    if t is not None:
                        t[b, :, end:] = 255 if fill & 1 else 254
        assert torch.equal(c.run(), want), hex(fill)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_a_later_row_with_nonfinite_entries_leaves_earlier_rows_alone(tf, fmt):
    """A drafted row whose own entry holds an infinity or NaN spoils itself and the rows
    after it, in the heads it touches; the rows before it keep their bits."""
    pos, R, g = [60, 511], 5, 4
    c = Case(tf, 8, 2, R, 2, g, 300, pos, fmt)
    want = c.run().clone()
    keep = c.cache.load(dev_pos([p + 3 for p in pos]), 1)
    for which in ("k", "v"):
        rows = [t.clone() for t in keep]
        rows[which == "v"][0, 7] = math.inf
        rows[which == "v"][1, D + 9] = math.nan
        c.cache.store(*rows, dev_pos([p + 3 for p in pos]))
        got = c.run().reshape(2, R, 2, g * D)
        ref = want.reshape(2, R, 2, g * D)
        assert torch.equal(got[:, :3], ref[:, :3])
        assert torch.equal(got[0, :, 1], ref[0, :, 1]) and torch.equal(got[1, :, 0], ref[1, :, 0])
        for r in (3, 4):
            assert not got[0, r, 0].isfinite().all() and not got[1, r, 1].isfinite().all()
        if which == "v" and fmt == "bf16":     # an element stays an element: the others are finite
            assert bool(got[0, 3:, 0].reshape(2, g, D)[:, :, 7].isinf().all())
            assert int((~got[0, 3:, 0].isfinite()).sum()) == 2 * g
            assert int((~got[1, 3:, 1].isfinite()).sum()) == 2 * g
        c.cache.store(*keep, dev_pos([p + 3 for p in pos]))
    assert torch.equal(c.run(), want)


def test_visible_nonfinite_entries_spread_as_the_formula_says(tf):
    """An infinite value far inside the visible range reaches that element of every row."""
    c = Case(tf, 9, 2, 2, 1, 2, 300, [400, 3], "bf16")
    k, v = c.prefix.load(dev_pos([130]), 1)
    v[0, 17] = -math.inf
    c.prefix.store(k, v, dev_pos([130]))
    got = c.run().reshape(-1, D)
    assert bool((got[:, 17] == -math.inf).all()) and bool(got[:, :17].isfinite().all())
    assert bool(got[:, 18:].isfinite().all())


def test_extreme_scores(tf):
    """Scores far apart: one key takes all the weight; equal keys share it evenly."""
    B, n_kv, P = 1, 1, 200
    k = np.zeros((1, 1, P, D), np.float32)
    v = np.arange(P * D, dtype=np.float32).reshape(1, 1, P, D) % 97
    k[0, 0, :, 0] = np.where(np.arange(P) == 150, 300.0, -300.0)
    bits = [inputs.bf16_bits_from_f32(a) for a in (k, v)]
    prefix = tf.KVBatch(1, 1, 256)
    prefix.store(dev_bits16(rows_of(bits[0])), dev_bits16(rows_of(bits[1])), dev_pos([0]))
    own = tf.KVBatch(1, 1, 256)
    zero = torch.zeros((1, D), dtype=torch.bfloat16, device="cuda")
    own.store(zero, zero, dev_pos([0]))
    q = torch.zeros((1, D), dtype=torch.bfloat16, device="cuda")
    q[0, 0] = 1000.0
    out = own.attention(q, 1, dev_pos([0]), prefix=prefix, prefix_len=P)
    assert torch.equal(out.cpu().double(), torch.from_numpy(bf16_to_f64(bits[1][0, 0, 150:151])))
    out = own.attention(zero, 1, dev_pos([0]), prefix=prefix, prefix_len=P).double().cpu().numpy()
    mean = bf16_to_f64(bits[1][0, 0]).sum(0) / (P + 1)
    assert np.all(np.abs(out[0] - mean) <= 2.0 ** -8 * mean * (1 + 2.0 ** -6) + 1e-6)


def test_sinks_and_long_tails(tf):
    """A sink whose score is 12 above thousands of equal keys: their joint weight counts."""
    P = 6000
    k = np.zeros((1, 1, P, D), np.float32)
    k[0, 0, 0, 0] = 12.0
    v = np.ones((1, 1, P, D), np.float32)
    v[0, 0, 0] = -1.0
    prefix = tf.KVBatch(1, 1, -(-P // 256) * 256)
    prefix.store(*(dev_bits16(rows_of(inputs.bf16_bits_from_f32(a))) for a in (k, v)), dev_pos([0]))
    own = tf.KVBatch(1, 1, 256)
    q = torch.zeros((1, D), dtype=torch.bfloat16, device="cuda")
    own.store(q, q, dev_pos([0]))
    q[0, 0] = 11.3125                                  # score 12 * 11.3125 / sqrt(128) = 11.9985
    out = float(own.attention(q, 1, dev_pos([0]), prefix=prefix, prefix_len=P)[0, 5])
    e = math.exp(12 * 11.3125 / math.sqrt(128))
    want = (P - 1 - e) / (P + e)
    assert abs(out - want) <= 2.0 ** -8 * abs(want) + (2.0 ** -8 + 2.0 ** -12) * 1.02


def test_all_idle_and_bad_positions(tf):
    c = Case(tf, 10, 3, 2, 1, 2, 40, [5, 6, 7], "bf16")
    want = c.run()
    ws = tf.workspace(c.cache.attention_workspace_bytes(2, 2, 40))
    out = torch.full((6, 2 * D), 3.0, dtype=torch.bfloat16, device="cuda")
    c.cache.attention(c.q_dev(), 2, dev_pos([-1, -1, -1]), prefix=c.prefix, prefix_len=40, out=out, ws=ws)
    assert not out.any() and tf.workspace_status(ws) == tf.TF_DEV_OK
    c.cache.attention(c.q_dev(), 2, dev_pos([5, c.L - 1, -7]), prefix=c.prefix, prefix_len=40, out=out, ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION
    assert torch.equal(out[:2], want[:2]) and not out[2:].any()


def test_strides_streams_and_graphs(tf):
    c = Case(tf, 11, 4, 3, 2, 5, 777, [100, 3, 257, 40], "e4m3")
    want = c.run()
    B, R, n_kv, g, P = c.shape
    cols = n_kv * g * D
    q = torch.zeros((B * R, cols + 3 * D), dtype=torch.int16, device="cuda")
    q[:, D:D + cols] = c.q_dev()
    out = torch.zeros((B * R, cols + D), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ws = tf.workspace(c.cache.attention_workspace_bytes(g, R, P))
    pos = dev_pos(c.pos)
    s.wait_stream(torch.cuda.current_stream())
    c.cache.attention(q[:, D:D + cols], g, pos, prefix=c.prefix, prefix_len=P, out=out[:, :cols], ws=ws, stream=s)
    s.synchronize()
    assert torch.equal(out[:, :cols], want) and not out[:, cols:].any()

    # captured once, replayed with moved positions and new queries
    graph = torch.cuda.CUDAGraph()
    q1 = c.q_dev()
    out1 = torch.empty((B * R, cols), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.cache.attention(q1, g, pos, prefix=c.prefix, prefix_len=P, out=out1, ws=ws)
    graph.replay()
    assert torch.equal(out1, want)
    c.pos = [5, 0, 90, -1]
    pos.copy_(dev_pos(c.pos))
    q1.neg_()
    graph.replay()
    c.q = q1.cpu().numpy().view(np.uint16).reshape(c.q.shape)
    assert torch.equal(out1, c.run())


def test_offsets_past_32_bits(tf):
    """The last head and sequence of caches of more than 2^31 elements each."""
    n_kv, L = 3, 1 << 21
    q = dev_bits16(inputs.bf16_normal(inputs.rng_for(12), (4, n_kv * D), 2.0))
    rows = [dev_bits16(inputs.bf16_normal(inputs.rng_for(13 + i), (2 * 300, n_kv * D))) for i in range(2)]
    for fmt in ("bf16", "e4m3"):
        small, big = tf.KVBatch(2, n_kv, 512, fmt), tf.KVBatch(2, n_kv, 2 * L, fmt)
        assert big.k.numel() > 1 << 31
        outs = []
        for c in (small, big):
            c.store(*rows, dev_pos([0, 0]))
            outs.append(c.attention(q, 1, dev_pos([298, 100])))
        assert torch.equal(outs[0], outs[1])
        start = 2 * L - 300                             # the same entries at the far end, alone visible through k
        k, v = big.load(dev_pos([0, 0]), 300)
        big.store(k, v, dev_pos([start, start]))
        k2, v2 = big.load(dev_pos([start, start]), 300)
        assert torch.equal(k, k2) and torch.equal(v, v2)
        del big


def test_refusals(tf):
    c = Case(tf, 14, 2, 2, 2, 2, 40, [5, 6], "bf16")
    q, pos = c.q_dev(), dev_pos(c.pos)
    other = tf.KVBatch(1, 2, 256, "e4m3")
    wide = tf.KVBatch(1, 3, 256)
    bad = [lambda: c.cache.attention(q[:3], 2, pos), lambda: c.cache.attention(q.float(), 2, pos),
           lambda: c.cache.attention(q, 4, pos), lambda: c.cache.attention(q, 0, pos),
           lambda: c.cache.attention(q, 2, pos[:1]), lambda: c.cache.attention(q, 2, pos.cpu()),
           lambda: c.cache.attention(q, 2, pos, prefix_len=10),
           lambda: c.cache.attention(q, 2, pos, prefix=c.prefix, prefix_len=257),
           lambda: c.cache.attention(q, 2, pos, prefix=c.prefix, prefix_len=-1),
           lambda: c.cache.attention(q, 2, pos, prefix=other, prefix_len=10),
           lambda: c.cache.attention(q, 2, pos, prefix=wide, prefix_len=10),
           lambda: c.cache.attention(q, 2, pos, prefix=c.cache, prefix_len=10),
           lambda: c.cache.attention(q, 2, pos, out=q[:2]),
           lambda: c.cache.attention(q, 2, pos, ws=torch.zeros(64, dtype=torch.uint8, device="cuda"))]
    for i, f in enumerate(bad):
        with pytest.raises(tf.TFError):
            f()
            pytest.fail(f"case {i} was not refused")
