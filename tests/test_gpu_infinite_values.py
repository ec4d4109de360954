"""Infinities and NaN in V under attention's weights, however small these are.

Every weight e^(s - m) of finite scores is above zero, so an output whose column of V holds values that are
not finite, among the entries that its row attends over, is their sum: an infinity, or NaN where they
hold a NaN or both infinities.  On the device a weight may be zero (a score 87 below the largest), and zero
times an infinity is not a number: what a row returns must not depend on which rows lie beside it.

Scores here are far apart (0 and +-724, multiples of 16 x 4 x 128 / sqrt(128)) or those of normal values.
"""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
D, INF, NAN = 128, float("inf"), float("nan")


def dev64(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


def dev32(p):
    return torch.tensor(p, dtype=torch.int32, device="cuda")


def bits(t):
    return t.view(torch.int16)


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def normal(gen, rows, heads, std=1.0):
    return (std * torch.randn((rows, heads * D), generator=gen, device="cuda")).to(torch.bfloat16)


def steep(gen, levels, n_kv, g):
    """Queries 16 u and keys 4 level u of one sign vector u a head: row t scores 724 level[t] for every query."""
    u = torch.randint(0, 2, (n_kv, D), generator=gen, device="cuda") * 2.0 - 1.0
    lv = torch.tensor(levels, device="cuda", dtype=torch.float32)[:, None, None]
    q = (16.0 * u[None, :, None, :]).expand(len(levels), n_kv, g, D).reshape(len(levels), -1)
    return q.to(torch.bfloat16).contiguous(), (4.0 * lv * u).reshape(len(levels), -1).to(torch.bfloat16)


def check(out, clean, v_seen, g):
    """One row: out, clean [n_kv * g * D] (clean: with finite values in V); v_seen [entries][n_kv * D]."""
    n_kv = v_seen.shape[1] // D
    v = v_seen.float().view(-1, n_kv, 1, D)
    x = torch.where(torch.isfinite(v), 0.0, v).sum(0).expand(n_kv, g, D)      # 0: every value is finite
    got, was = out.float().view(n_kv, g, D), clean.float().view(n_kv, g, D)
    assert torch.equal(got.isnan(), x.isnan())
    assert torch.equal(got.isinf(), x.isinf())
    assert torch.equal(got[x.isinf()], x[x.isinf()])
    assert torch.equal(got[x == 0], was[x == 0])


def spoil(v, at):
    for row, col, value in at:
        v[row, col] = value
    return v


SPOILED = [(10, 5, INF), (10, 7, -INF), (12, 7, -INF), (10, 9, INF), (12, 9, -INF), (11, 11, NAN), (17, 20, INF)]
LEVELS = {"low": lambda t: -1 if 10 <= t <= 17 else 1,          # the spoiled rows' weights are zero
          "rising": lambda t: -1 if t < 20 else (0 if t < 90 else 1),   # one first, zero when a later row outweighs them
          "flat": lambda t: 0}


# ---------------------------------------------------------------- whole prompts
@pytest.mark.parametrize("g", [1, 3, 8, 16])
@pytest.mark.parametrize("kind", [*LEVELS, "normal"])
@pytest.mark.parametrize("n", [26, 200])
def test_prompt(tf, g, kind, n):
    """Alone (items of one tile) and among 90 sequences (of two): the same bits, the formula's."""
    gen, n_kv = generator(n + g), 2
    if kind == "normal":
        q, k = normal(gen, n, n_kv * g, 16.0), normal(gen, n, n_kv)
    else:
        q, k = steep(gen, [LEVELS[kind](t) for t in range(n)], n_kv, g)
    v = normal(gen, n, n_kv)
    ws, starts = tf.workspace(256), dev64([0, n])
    clean = tf.prompt_attention(q, k, v, n_kv, g, starts, ws=ws)
    bad = spoil(v.clone(), SPOILED + [(13, D + 3, INF)])
    alone = tf.prompt_attention(q, k, bad, n_kv, g, starts, ws=ws)
    for r in range(n):
        check(alone[r], clean[r], bad[:r + 1], g)
    short = tf.prompt_attention(q[:19], k[:19], bad[:19], n_kv, g, dev64([0, 19]), ws=ws)
    assert torch.equal(bits(short), bits(alone[:19]))
    many = 90
    at = [n * i for i in range(many + 1)]
    out = tf.prompt_attention(q.repeat(many, 1), k.repeat(many, 1), bad.repeat(many, 1), n_kv, g, dev64(at), ws=ws)
    assert torch.equal(bits(out).view(many, -1), bits(alone).reshape(1, -1).expand(many, -1))
    assert tf.workspace_status(ws) == tf.TF_DEV_OK


def test_prompt_scores_that_are_not_numbers(tf):
    """They make the row NaN, whatever V holds."""
    gen, n, n_kv, g = generator(5), 120, 1, 8
    q, k, v = normal(gen, n, n_kv * g), normal(gen, n, n_kv), normal(gen, n, n_kv)
    k[30, 4], v[20, 6], v[40, 8] = NAN, INF, -INF
    out = tf.prompt_attention(q, k, v, n_kv, g, dev64([0, n])).view(n, g, D)
    assert out[30:].isnan().all() and out[:20].isfinite().all()
    assert (out[20:30, :, 6] == INF).all() and out[20:30, :, 7:].isfinite().all()


def test_a_long_prompt_of_nothing_but_infinities(tf):
    """The rows' values are looked through again where an output is not finite: in bounded time."""
    gen, n, n_kv, g = generator(6), 20001, 2, 8
    q, k, v = normal(gen, n, n_kv * g), normal(gen, n, n_kv), torch.full((n, n_kv * D), INF, device="cuda", dtype=torch.bfloat16)
    v[19000:, 3] = -INF
    ws = tf.workspace(256)
    out = tf.prompt_attention(q, k, v, n_kv, g, dev64([0, n]), ws=ws).view(n, n_kv, g, D)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    assert out[19000:, 0, :, 3].isnan().all()
    out[19000:, 0, :, 3] = INF
    assert (out == INF).all()


# ---------------------------------------------------------------- trees and batches over caches
class Cached:
    """A sequence of `own` entries behind a prefix of P, V spoiled at rows of the whole."""

    def __init__(self, tf, seed, kind, P, own, n_kv, g, spoiled, fmt="bf16"):
        gen = generator(seed)
        n = P + own
        self.tf, self.P, self.n_kv, self.g, self.own, self.fmt = tf, P, n_kv, g, own, fmt
        if kind == "normal":
            self.q, self.k = normal(gen, n, n_kv * g, 16.0), normal(gen, n, n_kv)
        else:
            self.q, self.k = steep(gen, [LEVELS[kind](t) for t in range(n)], n_kv, g)
        self.v = normal(gen, n, n_kv)
        self.bad = spoil(self.v.clone(), spoiled)

    def prefix(self, v):
        if not self.P:
            return {}
        c = self.tf.KVBatch(1, self.n_kv, -(-self.P // 256) * 256, self.fmt)
        c.store(self.k[:self.P], v[:self.P], dev64([0]))
        return dict(prefix=c, prefix_len=self.P)

    def cache(self, v, n_seq=1, rows=None):
        at = self.P + (torch.arange(self.own, device="cuda") if rows is None else torch.tensor(rows, device="cuda"))
        c = self.tf.KVBatch(n_seq, self.n_kv, 1024, self.fmt)
        c.store(self.k[at].repeat(n_seq, 1), v[at].repeat(n_seq, 1), dev64([0] * n_seq))
        return c


CASES = [  # prefix, own entries before the pass, spoiled rows of prefix + own
    (0, 12, SPOILED),                                               # near entries, of the pass and before it
    (0, 60, SPOILED),                                               # far ones
    (0, 334, [(320, 5, INF), (321, 7, -INF), (322, 7, INF), (325, 9, INF), (318, 4, NAN)]),     # mended for some nodes
    (0, 700, [(3, 5, INF), (330, 5, INF), (690, 8, -INF), (699, 9, INF)]),
    (40, 30, SPOILED + [(55, 30, INF), (60, 31, -INF)]),
    (700, 400, SPOILED + [(600, 40, INF), (650, 41, INF), (1080, 41, -INF), (1095, 42, INF)]),
]


@pytest.mark.parametrize("g", [1, 3, 8])
@pytest.mark.parametrize("kind", [*LEVELS, "normal"])
@pytest.mark.parametrize("P,pos,spoiled", CASES)
def test_tree_and_serial(tf, g, kind, P, pos, spoiled):
    """A tree of two chains, and the same nodes one a pass: the same bits, the formula's."""
    n, n_kv = 13, 2
    c = Cached(tf, P + pos + g, kind, P, pos + n, n_kv, g, spoiled + [(P + pos + 4, 50, INF), (P + pos + 9, 51, -INF)])
    parents = [-1, 0, 1, 2, 3, 4, 5, 2, 7, 8, 9, 10, 11]
    q, fixed, was = c.q[P + pos:], c.prefix(c.bad), c.prefix(c.v)
    ws = tf.workspace(c.cache(c.v).tree_attention_workspace_bytes(g, n, P))
    clean = c.cache(c.v).tree_attention(q, g, dev64([pos]), dev32([parents]), **was)
    out = c.cache(c.bad).tree_attention(q, g, dev64([pos]), dev32([parents]), ws=ws, **fixed)
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    two = c.cache(c.bad, 2).tree_attention(q.repeat(2, 1), g, dev64([pos, -1]), dev32([parents] * 2), **fixed)
    assert torch.equal(bits(two[:n]), bits(out)) and not two[n:].any()
    for leaf in (6, 12):
        path = [leaf]
        while path[0]:
            path.insert(0, parents[path[0]])
        serial = c.cache(c.bad, rows=[*range(pos), *(pos + i for i in path)])
        for d, i in enumerate(path):
            seen = c.bad[[*range(P + pos), *(P + pos + x for x in path[:d + 1])]]
            check(out[i], clean[i], seen, g)
            one = serial.tree_attention(q[i:i + 1], g, dev64([pos + d]), dev32([[-1]]), **fixed)
            assert torch.equal(bits(one[0]), bits(out[i])), (leaf, d)


@pytest.mark.parametrize("g", [1, 3, 8])
@pytest.mark.parametrize("kind", [*LEVELS, "normal"])
@pytest.mark.parametrize("P,pos,spoiled", CASES + [(0, 510, [(500, 5, INF), (505, 7, -INF), (508, 7, INF)])])
def test_batch_rows_and_one(tf, g, kind, P, pos, spoiled):
    """Several rows a pass, one, and another sequence beside them: the same bits, the formula's."""
    R, n_kv = 13, 2
    c = Cached(tf, P + pos + g, kind, P, pos + R, n_kv, g, spoiled + [(P + pos + 4, 50, INF), (P + pos + 9, 51, -INF)])
    q, fixed, was = c.q[P + pos:], c.prefix(c.bad), c.prefix(c.v)
    cache = c.cache(c.bad)
    clean = c.cache(c.v).attention(q, g, dev64([pos]), **was)
    out = cache.attention(q, g, dev64([pos]), **fixed)
    two = c.cache(c.bad, 2).attention(q.repeat(2, 1), g, dev64([-1, pos]), **fixed)
    assert torch.equal(bits(two[R:]), bits(out)) and not two[:R].any()
    for r in range(R):
        check(out[r], clean[r], c.bad[:P + pos + r + 1], g)
        one = cache.attention(q[r:r + 1], g, dev64([pos + r]), **fixed)
        assert torch.equal(bits(one[0]), bits(out[r])), r


@pytest.mark.parametrize("kind", [*LEVELS, "normal"])
def test_8_bit_entries_are_nan_whatever_their_weight(tf, kind):
    P, pos, n, n_kv, g = 700, 330, 13, 2, 8
    c = Cached(tf, 9, kind, P, pos + n, n_kv, g, [(650, 5, INF), (1015, D + 9, INF)], "e4m3")
    q, fixed, cache = c.q[P + pos:], c.prefix(c.bad), c.cache(c.bad)
    parents = [-1, *range(n - 1)]
    for out in (cache.tree_attention(q, g, dev64([pos]), dev32([parents]), **fixed), cache.attention(q, g, dev64([pos]), **fixed)):
        assert out.isnan().all()
    one = c.cache(c.bad).tree_attention(q[3:4], g, dev64([pos + 3]), dev32([[-1]]), **fixed)
    assert one.isnan().all()
