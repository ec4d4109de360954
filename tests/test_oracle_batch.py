"""Pins of oracle/batch.py, the frequencies of tf.rope_turns, and the refusals of the
batch entry points (host checks answer before any device work, so no GPU is needed)."""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import attention as oatt
from oracle import batch as obat

D = 128


# ---------------------------------------------------------------- norm and rotation
def test_norm_of_a_constant_head_is_its_gain():
    x = np.full((1, 2, D), 3.0)
    w = np.linspace(0.5, 1.5, D)
    y = obat.qk_norm_rope(x, 1, 1, w, 2 * w, 0.0, [], False, [5])
    assert np.allclose(y[0, 0], w) and np.allclose(y[0, 1], 2 * w)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_keeps_lengths_and_depends_on_the_distance_only(adjacent):
    rng = np.random.default_rng(3)
    f = [10000.0 ** (-2 * d / 64) for d in range(32)]
    q, k = rng.normal(size=(1, 1, D)), rng.normal(size=(1, 1, D))

    def at(x, p):
        return obat.qk_norm_rope(x, 1, 0, None, None, 0.0, f, adjacent, [p])[0, 0]

    assert np.allclose(np.linalg.norm(at(q, 777)), np.linalg.norm(q))
    assert np.allclose(at(q, 0), q[0, 0]) and np.array_equal(at(q, 9)[64:], q[0, 0, 64:])
    assert np.isclose(at(q, 1000) @ at(k, 990), at(q, 10) @ at(k, 0))
    assert not np.isclose(at(q, 1000) @ at(k, 990), at(q, 990) @ at(k, 1000))   # direction matters
    i0, i1 = (0, 1) if adjacent else (0, 32)      # frequency 1 radian: the first pair
    assert np.isclose(at(q, 2)[i0], q[0, 0, i0] * math.cos(2) - q[0, 0, i1] * math.sin(2))


def test_rope_turns_is_the_nearest_64_bit_fraction():
    from w4_gemm_keyed_gb300 import tf
    got = tf.rope_turns(128, 1e6, device="cpu").tolist()
    pi = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    for d in (0, 1, 31, 63):
        want = Fraction(1e6 ** (-2.0 * d / 128)) / (2 * pi) * 2 ** 64
        assert abs((got[d] % 2 ** 64) - want) <= Fraction(1, 2)
    own = tf.rope_turns(8, inv_freq=[0.0, 2 * math.pi, 1.0, -1.0], device="cpu").tolist()
    assert own[0] == 0 and abs(own[1]) < 2 ** 14 and own[2] == -own[3]    # whole turns vanish


@pytest.mark.parametrize("rot,freq", [(0, None), (12, None), (136, None), (16, [1.0] * 7), (16, [math.inf] * 8)])
def test_rope_turns_refuses(rot, freq):
    from w4_gemm_keyed_gb300 import tf
    with pytest.raises(tf.TFError):
        tf.rope_turns(rot, inv_freq=freq, device="cpu")


# ---------------------------------------------------------------- E4M3 vectors
def test_e4m3_table_is_the_format():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(obat.e4m3_table(), want, equal_nan=True)


def test_e4m3_vector_rounds_as_the_format_does():
    rng = np.random.default_rng(7)
    for scale in (1e-30, 1e-3, 1.0, 50.0):
        x = torch.tensor(rng.normal(size=D) * scale).to(torch.bfloat16).double().numpy()
        codes, s = obat.e4m3_vector(x)
        y = torch.tensor(x / 2.0 ** (s - 127))
        assert np.array_equal(codes, y.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())
        assert 224 < np.max(np.abs(y.numpy())) <= 448 or s == 7


def test_e4m3_vector_edges():
    x = np.zeros(D)
    assert obat.e4m3_vector(x)[1] == 7 and not obat.e4m3_vector(x)[0].any()
    x[3] = 448.0
    assert obat.e4m3_vector(x)[1] == 127 and obat.e4m3_vector(x)[0][3] == 0x7E
    x[3] = 450.0                                   # past 448: the next power of two
    assert obat.e4m3_vector(x)[1] == 128
    x[3] = -1e30                                   # past 448 * 2^7: saturates
    codes, s = obat.e4m3_vector(x)
    assert s == 134 and obat.e4m3_values(codes, s)[3] == -57344.0
    x[3] = math.inf
    assert obat.e4m3_vector(x)[1] == 255 and np.isnan(obat.e4m3_values(*obat.e4m3_vector(x))).all()


def test_e4m3_place_is_a_permutation_of_16_byte_groups():
    at = obat.e4m3_place(np.arange(D, dtype=np.uint8))
    assert sorted(at) == list(range(D))
    assert list(at[:16]) == [0, 2, 1, 3, 4, 6, 5, 7, 64, 66, 65, 67, 68, 70, 69, 71]


# ---------------------------------------------------------------- attention
def batch_case(rng, B, R, n_kv, g, P, L):
    def n(*shape):
        return rng.normal(size=shape)
    return n(B, R, n_kv, g, D), n(n_kv, P, D), n(n_kv, P, D), n(B, n_kv, L, D), n(B, n_kv, L, D)


def test_attention_batch_is_plain_attention_over_the_joined_entries():
    rng = np.random.default_rng(11)
    q, sk, sv, ok, ov = batch_case(rng, 3, 2, 2, 3, 5, 9)
    out, spread = obat.attention_batch(q, sk, sv, ok, ov, [0, -1, 6])
    assert not out[1].any() and np.all(spread[[0, 2]] >= np.abs(out[[0, 2]]) - 1e-15)
    for b, p in ((0, 0), (2, 6)):
        for r in range(2):
            for j in range(2):
                for h in range(3):
                    k, v = np.concatenate([sk[j], ok[b, j]]), np.concatenate([sv[j], ov[b, j]])
                    want = oatt.attention_row(q[b, r, j, h], k, v, 5 + p + r)
                    assert np.allclose(out[b, r, j, h], want, rtol=1e-12)


def test_attention_batch_planted_mistakes_are_caught():
    rng = np.random.default_rng(12)
    q, sk, sv, ok, ov = batch_case(rng, 2, 2, 1, 2, 4, 8)
    out = obat.attention_batch(q, sk, sv, ok, ov, [3, 5])[0]
    late = obat.attention_batch(q, sk, sv, ok, ov, [4, 6])[0]              # mask off by one
    none = obat.attention_batch(q, sk[:, :0], sv[:, :0], ok, ov, [3, 5])[0]    # prefix dropped
    swap = obat.attention_batch(q, sk, sv, ok[::-1], ov[::-1], [3, 5])[0]  # another sequence's entries
    for bad in (late, none, swap):
        assert np.max(np.abs(bad - out)) > 1e-2


# ---------------------------------------------------------------- refusals
@pytest.fixture(scope="module")
def lib():
    from w4_gemm_keyed_gb300 import build, tf
    build.build()
    return tf.load()


A = 4096    # a non-null, aligned stand-in for device pointers: no call below gets as far as using it


def kv(**kw):
    from w4_gemm_keyed_gb300 import tf
    d = dict(k=A, v=A, k_scale=A, v_scale=A, n_seq=2, n_kv=2, max_len=512, format=1)
    d.update(kw)
    return tf.KVBatchC(*(d[n] for n, _ in tf.KVBatchC._fields_))


BAD_BATCH = [dict(k=None), dict(v=A + 8), dict(k_scale=None), dict(v_scale=A + 4), dict(n_seq=0), dict(n_seq=1025),
             dict(n_kv=0), dict(n_kv=129), dict(max_len=0), dict(max_len=300), dict(format=2), dict(format=-1)]


@pytest.mark.parametrize("bad", BAD_BATCH, ids=str)
def test_every_call_refuses_a_bad_batch(lib, bad):
    c = kv(**bad)
    assert lib.tf_kv_store(c, A, A, 256, 1, A, A, 256, None) in (1, 2)
    assert lib.tf_kv_load(c, A, 1, A, A, 256, A, 256, None) in (1, 2)
    assert lib.tf_attention_batch(c, None, 0, 1, A, 256, 1, A, A, 256, A, 1 << 30, None) in (1, 2)
    if bad.get("n_kv") != 129:
        own = kv(n_kv=max(1, c.n_kv))
        assert lib.tf_attention_batch(own, c, 4, 1, A, 256, 1, A, A, 256, A, 1 << 30, None) in (1, 2)


@pytest.mark.parametrize("args,status", [
    (dict(R=0), 1), (dict(R=513), 1), (dict(k=None), 1), (dict(k=A + 8), 1), (dict(pos=None), 1), (dict(pos=A + 4), 1),
    (dict(ld=128), 1), (dict(ld=260), 1), (dict(ws=None), 5), (dict(ws_bytes=128), 5), (dict(ws=A + 16), 5)], ids=str)
def test_kv_rows_refusals(lib, args, status):
    a = dict(R=1, k=A, ld=256, pos=A, ws=A, ws_bytes=256)
    a.update(args)
    assert lib.tf_kv_store(kv(), a["k"], A, a["ld"], a["R"], a["pos"], a["ws"], a["ws_bytes"], None) == status
    assert lib.tf_kv_load(kv(), a["pos"], a["R"], a["k"], A, a["ld"], a["ws"], a["ws_bytes"], None) == status


@pytest.mark.parametrize("args,status", [
    (dict(group=0), 2), (dict(group=17), 2), (dict(R=0), 1), (dict(R=17), 1), (dict(R=16, group=9), 2),
    (dict(plen=-1), 1), (dict(plen=4, prefix=None), 1), (dict(plen=4, prefix=dict(n_seq=2)), 1),
    (dict(plen=4, prefix=dict(n_seq=1, n_kv=1)), 1), (dict(plen=4, prefix=dict(n_seq=1, format=0)), 1),
    (dict(plen=513, prefix=dict(n_seq=1)), 1), (dict(q=None), 1), (dict(q=A + 8), 1), (dict(ldq=255), 1),
    (dict(ldq=260), 1), (dict(out=None), 1), (dict(out=A + 2), 1), (dict(ldo=128), 1), (dict(ldo=257), 1),
    (dict(pos=None), 1), (dict(ws=None), 5), (dict(ws_bytes=0), 5)], ids=str)
def test_attention_batch_refusals(lib, args, status):
    a = dict(group=1, R=1, plen=0, prefix=None, q=A, ldq=256, out=A, ldo=256, pos=A, ws=A, ws_bytes=1 << 30)
    a.update(args)
    if a["group"] > 1:
        a["ldq"] = a["ldo"] = 256 * a["group"]
    prefix = None if a["prefix"] is None else kv(**a["prefix"])
    st = lib.tf_attention_batch(kv(), prefix, a["plen"], a["group"], a["q"], a["ldq"], a["R"], a["pos"], a["out"],
                                a["ldo"], a["ws"], a["ws_bytes"], None)
    assert st == status and lib.tf_last_error()


def test_attention_batch_workspace_query(lib):
    assert lib.tf_attention_batch_workspace_bytes(kv(), 4, 4, 1000) >= 256
    for bad in (dict(n_seq=0), dict(n_seq=1025), dict(n_kv=0), dict(max_len=100)):
        assert lib.tf_attention_batch_workspace_bytes(kv(**bad), 4, 4, 1000) == 0
    for g, R, P in ((0, 1, 0), (17, 1, 0), (1, 0, 0), (1, 17, 0), (9, 16, 0), (1, 1, -1)):
        assert lib.tf_attention_batch_workspace_bytes(kv(), g, R, P) == 0


@pytest.mark.parametrize("args,status", [
    (dict(x=None), 1), (dict(x=A + 8), 1), (dict(y=A + 8), 1), (dict(n_seq=0), 1), (dict(R=0), 1), (dict(n_q=-1), 1),
    (dict(n_q=0, n_k=0, n_v=0), 1), (dict(n_q=4097), 1), (dict(ldx=511), 1), (dict(ldx=514), 1), (dict(ldy=516), 1),
    (dict(y=A), 1), (dict(wk=None), 1), (dict(wq=A + 2), 1), (dict(eps=-1.0), 1), (dict(eps=math.nan), 1),
    (dict(rot=12), 2), (dict(rot=136), 2), (dict(rot=-8), 2), (dict(turns=None), 1), (dict(turns=A + 8), 1),
    (dict(pos=None), 1), (dict(n_seq=1 << 20, R=1 << 12), 2)], ids=str)
def test_qk_norm_rope_refusals(lib, args, status):
    a = dict(x=A, fp32=1, ldx=512, n_seq=1, R=1, n_q=2, n_k=1, n_v=1, wq=A, wk=A, eps=1e-6, turns=A, rot=64, pos=A,
             y=2 * A, ldy=512)
    a.update(args)
    st = lib.tf_qk_norm_rope(a["x"], a["fp32"], a["ldx"], a["n_seq"], a["R"], a["n_q"], a["n_k"], a["n_v"], a["wq"],
                             a["wk"], a["eps"], a["turns"], a["rot"], 0, a["pos"], 0, a["y"], a["ldy"], None)
    assert st == status and lib.tf_last_error()
