"""Causal attention of packed prompts on the GPU through the binding, against
oracle/trees.py in fp64.

Tolerance, per element, with the softmax weights w: the output is rounded to bf16
once (half a step, 2^-8 of the value); the weights may be rounded to bf16 before
the product with v (2^-8 of sum w|v|); scores and sums in fp32 move a weight by
less than 2^-12 of itself for the scores here (|s| < 2^6 with fewer than 2^6
roundings of 2^-24 each).  So |got - ref| <= 2^-8 |ref| + (2^-8 + 2^-12) sum w|v|, times
1 + 2^-6 for the products of these.
"""

import numpy as np
import pytest
import torch

from oracle import trees as otree
from oracle.linear import bf16_to_f64
from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16

pytestmark = pytest.mark.gpu
D = 128


def dev_starts(s):
    return torch.tensor(s, dtype=torch.int64, device="cuda")


class Case:
    """Rows of a projection (query, key and value heads side by side), some before and
    behind the sequences."""

    def __init__(self, seed, lengths, n_kv, g, front=0, back=0, q_std=2.0, pad=0):
        rng = inputs.rng_for(seed)
        n_q = n_kv * g
        self.n_kv, self.g, self.pad = n_kv, g, pad
        self.starts = [int(x) for x in front + np.cumsum([0] + list(lengths))]
        self.rows = self.starts[-1] + back
        q = inputs.bf16_normal(rng, (self.rows, n_q * D), q_std)
        kv = inputs.bf16_normal(rng, (self.rows, 2 * n_kv * D + pad))
        self.x = dev_bits16(np.concatenate([q, kv], axis=1)).view(torch.bfloat16)

    def views(self, x=None):
        x = self.x if x is None else x
        n_q, w = self.n_kv * self.g * D, self.n_kv * D
        return x[:, :n_q], x[:, n_q:n_q + w], x[:, n_q + w:n_q + 2 * w]

    def run(self, tf, x=None, starts=None, **kw):
        return tf.prompt_attention(*self.views(x), self.n_kv, self.g, dev_starts(starts or self.starts), **kw)

    def reference(self):
        x = self.x.double().cpu().numpy()
        q, k, v = (x[:, s] for s in (slice(0, self.n_kv * self.g * D), slice(self.n_kv * self.g * D, self.n_kv * (self.g + 1) * D),
                                     slice(self.n_kv * (self.g + 1) * D, self.n_kv * (self.g + 2) * D)))
        return otree.attention_prompt(q.reshape(self.rows, self.n_kv, self.g, D), k.reshape(self.rows, self.n_kv, D),
                                      v.reshape(self.rows, self.n_kv, D), self.starts)

    def check(self, out):
        ref, spread = self.reference()
        a, b = self.starts[0], self.starts[-1]
        got = out.double().cpu().numpy().reshape(ref.shape)[a:b]
        ref, spread = ref[a:b], spread[a:b]
        tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6)
        assert np.all(np.isfinite(got))
        worst = np.max(np.abs(got - ref) - tol)
        assert worst <= 0, f"off by {worst:.3e} more than allowed"
        err = np.linalg.norm(got - ref) / np.linalg.norm(ref)
        assert err < 4e-3, err      # rms of the two roundings: sqrt(2) * 2^-8 / sqrt(3) of the spread, at most


CASES = [  # lengths, n_kv, group
    ([1], 1, 1),
    ([1], 8, 8),
    ([2], 1, 16),
    ([16], 1, 8),                                   # one tile of 128 vectors
    ([17], 2, 8),
    ([32, 33], 2, 8),                               # two tiles, and a row more
    ([0, 1, 0, 2, 0], 2, 4),                        # empty sequences
    ([127, 128, 129], 1, 1),
    ([128], 2, 2),
    ([255, 1, 257], 1, 1),
    ([300, 0, 17, 1, 33], 2, 5),
    ([64, 200], 1, 3),
    ([43] * 9, 2, 3),
    ([513], 2, 7),
    ([700], 1, 16),
    ([30 + s for s in range(40)], 1, 2),
    ([1025, 3], 2, 4),
]


@pytest.mark.parametrize("lengths,n_kv,g", CASES)
def test_attention_prompt(tf, lengths, n_kv, g):
    c = Case(100 * len(lengths) + g, lengths, n_kv, g)
    ws = tf.workspace(256)
    out = c.run(tf, ws=ws)
    assert out.dtype == torch.bfloat16 and tf.workspace_status(ws) == tf.TF_DEV_OK
    c.check(out)
    for _ in range(3):
        assert torch.equal(out, c.run(tf, ws=ws))       # the same bits again, on a used workspace


def test_a_long_prompt_on_sampled_rows(tf):
    n, n_kv, g = 9001, 2, 4
    c = Case(3, [n], n_kv, g)
    got = c.run(tf).double().cpu().numpy().reshape(n, n_kv, g, D)
    x = c.x.double().cpu().numpy()
    q, k, v = x[:, :n_kv * g * D], x[:, n_kv * g * D:n_kv * (g + 1) * D], x[:, n_kv * (g + 1) * D:]
    for r in (0, 1, 127, 128, 1000, 4095, 4096, 8191, 8999, 9000):
        for j in range(n_kv):
            ref, spread = otree._attend(q[r].reshape(n_kv, g, D)[j], k[:r + 1].reshape(-1, n_kv, D)[:, j],
                                        v[:r + 1].reshape(-1, n_kv, D)[:, j])
            tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6)
            assert np.all(np.abs(got[r, j] - ref) <= tol), (r, j)


@pytest.mark.parametrize("g", [1, 4, 5, 16])
def test_sequences_stand_alone(tf, g):
    """A row's bits do not depend on the other sequences, on where its own lies, or on
    the rows after it."""
    c = Case(9, [70, 301, 0, 5, 140], 2, g, front=3, back=6)
    out = c.run(tf, out=torch.zeros((c.rows, 2 * g * D), dtype=torch.bfloat16, device="cuda"))
    for a, b in zip(c.starts[:-1], c.starts[1:]):
        if a < b:
            alone = c.x[a:b].contiguous()
            assert torch.equal(out[a:b], c.run(tf, x=alone, starts=[0, b - a]))
            half = (b - a + 1) // 2
            assert torch.equal(out[a:a + half], c.run(tf, x=alone, starts=[0, half])[:half])


def test_rows_outside_the_sequences_are_left_alone(tf):
    """They may hold anything, and the output keeps what it held there."""
    c = Case(5, [40, 131], 2, 4, front=7, back=30)
    clean = c.run(tf)
    x = c.x.clone()
    x[:7], x[c.starts[-1]:] = float("nan"), float("inf")
    out = torch.full((c.rows, 8 * D), 3.5, dtype=torch.bfloat16, device="cuda")
    ws = tf.workspace(256)
    c.run(tf, x=x, out=out, ws=ws)
    a, b = c.starts[0], c.starts[-1]
    assert torch.equal(out[a:b], clean[a:b]) and tf.workspace_status(ws) == tf.TF_DEV_OK
    assert (out[:a] == 3.5).all() and (out[b:] == 3.5).all()


@pytest.mark.parametrize("g", [1, 3, 8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), "lowest"])
@pytest.mark.parametrize("what", ["k", "v"])
def test_rows_before_an_infinity_do_not_see_it(tf, g, bad, what):
    """A value that is not finite reaches the rows that see it, and no other row or sequence."""
    value = torch.finfo(torch.bfloat16).min if bad == "lowest" else bad
    lengths, n_kv = [150, 300, 20], 2
    c = Case(11, lengths, n_kv, g)
    clean = c.run(tf)
    x, row, col = c.x.clone(), 150 + 201, 37
    c.views(x)[1 if what == "k" else 2][row, D + col] = value       # KV head 1
    out = c.run(tf, x=x)
    heads, was = (t.view(c.rows, n_kv, g, D) for t in (out, clean))
    assert torch.equal(heads[:, 0], was[:, 0])
    assert torch.equal(out[:row], clean[:row]) and torch.equal(out[450:], clean[450:])
    seen = heads[row:450, 1]
    if what == "v":
        others = [d for d in range(D) if d != col]
        assert torch.equal(seen[..., others], was[row:450, 1][..., others])
        if bad == "lowest":
            assert not torch.isnan(seen).any()
        else:       # a weight of zero times an infinity is not a number either
            assert not torch.isfinite(seen[..., col]).any()
            assert torch.isnan(seen[..., col]).all() if bad != bad else (seen[..., col] == value).any()
    elif bad != bad:
        assert torch.isnan(seen).all()
    # a key with an infinity or the lowest value: a score of +-inf, by the query's sign
    else:
        q = c.views()[0].view(c.rows, n_kv, g, D)[row:450, 1, :, col]
        hidden = (q * value < 0) if bad != "lowest" else (q > 1)
        assert hidden.any() and torch.isfinite(seen[hidden]).all()
        if bad != "lowest":
            assert torch.isnan(seen[(q * value) > 0]).all()


def test_one_key_takes_all(tf):
    """Scores far apart: each row returns the value of the one row it asks for, exactly."""
    n, rng = 260, inputs.rng_for(2)
    sign = np.sign(rng.standard_normal((n, D)))
    want = np.array([rng.integers(0, r + 1) for r in range(n)])
    q, k = 16.0 * sign[want], 4.0 * sign        # the row asked for scores 724, others below 400
    v = bf16_to_f64(inputs.bf16_normal(rng, (n, D)))
    q, k, v = (torch.from_numpy(a).cuda().to(torch.bfloat16) for a in (q, k, v))
    out = tf.prompt_attention(q, k, v, 1, 1, dev_starts([0, n]))
    assert torch.equal(out, v[torch.from_numpy(want).cuda()])


@pytest.mark.parametrize("std", [1e-3, 30.0])
def test_flat_and_steep_scores(tf, std):
    """Nearly equal weights, and a few large ones (|s| < 2^9: a weight moves by less than
    2^-9 of itself, so the tolerance's 2^-12 becomes 2^-9)."""
    c = Case(21, [333], 2, 4, q_std=std)
    ref, spread = c.reference()
    got = c.run(tf).double().cpu().numpy().reshape(ref.shape)
    tol = (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -9) * spread) * (1 + 2.0 ** -6)
    assert np.all(np.abs(got - ref) <= tol)


def test_strided_buffers(tf):
    c = Case(13, [50, 90], 2, 3, pad=24)
    whole = c.run(tf)
    alone = tf.prompt_attention(*(t.contiguous() for t in c.views()), 2, 3, dev_starts(c.starts))
    assert torch.equal(whole, alone)
    buf = torch.full((c.rows, 6 * D + 40), 7.0, dtype=torch.bfloat16, device="cuda")
    c.run(tf, out=buf[:, 8:8 + 6 * D])
    assert torch.equal(buf[:, 8:8 + 6 * D], whole) and (buf[:, :8] == 7).all() and (buf[:, 8 + 6 * D:] == 7).all()
    bits = [t.view(torch.int16) for t in c.views()]
    assert torch.equal(whole, tf.prompt_attention(*bits, 2, 3, dev_starts(c.starts)))


@pytest.mark.parametrize("starts", [[0, 20, 10, 30], [-1, 5, 10, 20], [0, 5, 10, 41], [0, 1 << 40, 1 << 40, 1 << 41]])
def test_bad_starts_are_reported_and_nothing_is_written(tf, starts):
    c = Case(7, [10, 10, 20], 1, 4)
    out, ws = torch.full((c.rows, 4 * D), 2.0, dtype=torch.bfloat16, device="cuda"), tf.workspace(256)
    c.run(tf, starts=starts, out=out, ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION and (out == 2).all()
    assert torch.equal(c.run(tf, ws=ws), c.run(tf)) and tf.workspace_status(ws) == tf.TF_DEV_OK


def test_nothing_but_empty_sequences(tf):
    c = Case(7, [0, 0], 1, 4, back=5)
    out = torch.full((5, 4 * D), 2.0, dtype=torch.bfloat16, device="cuda")
    c.run(tf, out=out)
    assert (out == 2).all()
    none = torch.empty((0, 4 * D), dtype=torch.bfloat16, device="cuda")
    assert tf.prompt_attention(none, none[:, :D], none[:, :D], 1, 4, dev_starts([0, 0])).shape == (0, 4 * D)


def test_many_sequences(tf):
    rng = inputs.rng_for(4)
    c = Case(4, [int(n) for n in rng.integers(0, 12, 1024)], 1, 2)
    out = c.run(tf)
    c.check(out)


@pytest.mark.parametrize("n_kv,g,longest", [(8, 8, 301), (8, 8, 20), (4, 5, 140), (8, 16, 33)])
def test_many_items_a_processor(tf, n_kv, g, longest):
    """Items of one and of two tiles, of one key tile and of several, one after the other: sequence by
    sequence the bits of calls that hold it alone."""
    rng = inputs.rng_for(longest)
    c, ws = Case(longest, [int(n) for n in rng.integers(1, longest + 1, 60)], n_kv, g), tf.workspace(256)
    out = c.run(tf, ws=ws)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    for a, b in list(zip(c.starts[:-1], c.starts[1:]))[::7]:
        assert torch.equal(out[a:b], c.run(tf, x=c.x[a:b].contiguous(), starts=[0, b - a]))
    assert torch.equal(out, c.run(tf, ws=ws)) and tf.workspace_status(ws) == tf.TF_DEV_OK


def test_graphs_share_a_workspace_and_read_the_starts_anew(tf):
    a, b = Case(31, [200, 90], 2, 4), Case(32, [40, 40, 300], 1, 8)
    ws, cases = tf.workspace(256), []
    for c in (a, b):
        starts, out = dev_starts(c.starts), torch.zeros((c.rows, c.n_kv * c.g * D), dtype=torch.bfloat16, device="cuda")
        call = (lambda c=c, starts=starts, out=out:
                tf.prompt_attention(*c.views(), c.n_kv, c.g, starts, out=out, ws=ws))
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        cases.append((c, starts, out, graph))
    for _ in range(2):
        for c, starts, out, graph in cases:
            out.zero_()
            graph.replay()
            assert torch.equal(out, c.run(tf))
    c, starts, out, graph = cases[0]
    starts.copy_(dev_starts([0, 7, 290]))
    graph.replay()
    assert torch.equal(out, c.run(tf, starts=[0, 7, 290])) and tf.workspace_status(ws) == tf.TF_DEV_OK


def test_on_another_stream(tf):
    c, side = Case(41, [120, 400], 2, 8), torch.cuda.Stream()
    ref = c.run(tf)
    starts = dev_starts(c.starts)
    torch.cuda.synchronize()
    out = tf.prompt_attention(*c.views(), 2, 8, starts, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, ref)


def test_a_workspace_that_other_operators_used(tf):
    c, ws = Case(43, [90, 260], 1, 4), tf.workspace(1 << 22)
    ref = c.run(tf)
    cache = tf.KVBatch(1, 1, 256)
    rows = c.views()[1][:40].contiguous()
    pos = torch.zeros(1, dtype=torch.int64, device="cuda")
    cache.store(rows, rows, pos, ws=ws)
    cache.attention(c.views()[0][:8].contiguous(), 4, pos, ws=ws)
    assert torch.equal(c.run(tf, ws=ws), ref)
    again = cache.attention(c.views()[0][:8].contiguous(), 4, pos, ws=ws)
    assert torch.equal(again, cache.attention(c.views()[0][:8].contiguous(), 4, pos))


@pytest.mark.parametrize("n,n_kv,g", [(3, 2, 4), (37, 1, 16), (300, 2, 3)])
def test_a_prompt_is_what_batch_attention_makes_of_it(tf, n, n_kv, g):
    """One query at a time over a cache of the same entries: another kernel, the same formula."""
    c = Case(51, [n], n_kv, g)
    q, k, v = (t.contiguous() for t in c.views())
    cache = tf.KVBatch(1, n_kv, 512)
    cache.store(k, v, dev_starts([0]))
    got = c.run(tf).double()
    for r in {0, 1, n // 2, n - 1}:
        one = cache.attention(q[r:r + 1], g, dev_starts([r])).double()
        ref, spread = otree._attend(q[r].double().cpu().numpy().reshape(n_kv, g, D)[0],
                                    k[:r + 1, :D].double().cpu().numpy(), v[:r + 1, :D].double().cpu().numpy())
        gap = (got[r] - one[0]).abs().cpu().numpy().reshape(n_kv, g, D)[0]
        assert np.all(gap <= 2 * (2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * spread) * (1 + 2.0 ** -6))
