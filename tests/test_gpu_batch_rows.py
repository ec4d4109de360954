"""Per-head norm with rotation, and the batch KV caches' writes and reads, on the GPU
through the binding, against oracle/batch.py.

Tolerance of the norm and rotation: one bf16 rounding, half a step 2^-8 of the value,
plus the fp32 arithmetic before it: every element is a sum of two products whose
factors carry fewer than eight fp32 roundings (2^-24 each) and an angle off by at
most 2^-25 half turns (pi 2^-25 < 2^-23 radians), so 2^-20 of the pair's magnitude
covers it.  Cache codes, scales and values are exact.
"""

import math

import numpy as np
import pytest
import torch

from oracle import batch as obat
from oracle.linear import bf16_to_f64
from w4_gemm_keyed_gb300 import inputs
from gpu_util import dev_bits16, kv_unswizzle

pytestmark = pytest.mark.gpu
D = 128


def dev_pos(p):
    return torch.tensor(p, dtype=torch.int64, device="cuda")


def f64(t):
    return t.view(torch.bfloat16).double().cpu().numpy()


# ---------------------------------------------------------------- norm and rotation
ROPE = [  # n_seq, R, n_q, n_k, n_v, rot, adjacent, fp32, norm, positions, offset
    (1, 1, 8, 2, 2, 128, False, True, True, [0], 0),
    (1, 1, 1, 1, 0, 128, True, True, True, [1], 7),
    (3, 2, 5, 1, 1, 64, False, False, True, [10, 0, 99999], 1000),
    (2, 5, 4, 2, 2, 96, True, True, True, [1048575, 3], 0),
    (1, 37, 12, 4, 4, 8, False, True, True, [5], 0),
    (4, 1, 3, 3, 3, 128, True, False, False, [0, 1, 2, 1 << 40], 0),      # rotation only
    (2, 2, 3, 1, 1, 0, False, True, True, [0, 0], 0),                    # norm only
    (1, 3, 0, 2, 0, 32, False, True, True, [-4], 0),                     # keys alone, negative positions
    (1, 2000, 9, 1, 1, 128, False, False, True, [123456], 0),            # several heads a warp
    (1, 3, 2, 1, 1, 24, False, True, True, [2 ** 62], 0),
]


@pytest.mark.parametrize("n_seq,R,n_q,n_k,n_v,rot,adjacent,fp32,norm,pos,offset", ROPE)
def test_qk_norm_rope(tf, n_seq, R, n_q, n_k, n_v, rot, adjacent, fp32, norm, pos, offset):
    rng = np.random.default_rng(n_seq * 1000 + R * 10 + rot)
    H, rows = n_q + n_k + n_v, n_seq * R
    x = torch.tensor(rng.normal(size=(rows, H, D)) * np.exp(rng.normal(size=(rows, H, 1)) * 2), dtype=torch.float32)
    if not fp32:
        x = x.to(torch.bfloat16)
    wq, wk = (torch.tensor(1 + 0.3 * rng.normal(size=D)).to(torch.bfloat16) for _ in range(2))
    # frequencies on a 2^-16 turn grid keep the oracle's fp64 angle exact at far positions
    far = max(abs(p) for p in pos) > 1 << 30
    freq = [2 * math.pi * k / 65536 for k in range(1, rot // 2 + 1)] if far else [5e5 ** (-2 * d / max(rot, 1)) for d in
                                                                              range(rot // 2)]
    turns = tf.rope_turns(rot, inv_freq=freq) if rot else None
    if far and rot:
        turns = torch.tensor([k << 48 for k in range(1, rot // 2 + 1)], dtype=torch.int64, device="cuda")
    kw = dict(q_weight=wq.cuda(), k_weight=wk.cuda()) if norm else {}
    eps = 1e-3
    y = tf.qk_norm_rope(x.reshape(rows, -1).cuda(), n_q, n_k, dev_pos(pos), turns=turns, eps=eps, adjacent=adjacent,
                        pos_offset=offset, n_v=n_v, **kw)
    assert y.dtype == torch.bfloat16 and tuple(y.shape) == (rows, H * D)
    positions = [p + offset + r for p in pos for r in range(R)]
    seen = [p % 65536 for p in positions] if far else positions
    ref = obat.qk_norm_rope(x.double().numpy(), n_q, n_k, wq.double().numpy() if norm else None,
                            wk.double().numpy() if norm else None, eps, freq, adjacent, seen)
    got = f64(y).reshape(rows, H, D)
    size = np.max(np.abs(ref), axis=-1, keepdims=True)
    assert np.all(np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size)
    assert np.array_equal(got[:, n_q + n_k:], f64(x.to(torch.bfloat16))[:, n_q + n_k:])     # values: rounded only


def test_qk_norm_rope_rows_stand_alone(tf):
    """A row's bits do not depend on how many rows or sequences share the launch."""
    rng = np.random.default_rng(5)
    x = torch.tensor(rng.normal(size=(60, 10 * D)), dtype=torch.float32).cuda()
    turns = tf.rope_turns(128, 1e6)
    w = dev_bits16(inputs.bf16_normal(inputs.rng_for(3), (2, D)))
    pos = dev_pos([7, 400, 9, 0, 31])
    whole = tf.qk_norm_rope(x, 8, 1, pos, turns=turns, q_weight=w[0], k_weight=w[1])
    for b, r in ((0, 0), (1, 11), (4, 5)):
        one = tf.qk_norm_rope(x[b * 12 + r][None], 8, 1, pos[b:b + 1] + r, turns=turns, q_weight=w[0], k_weight=w[1])
        assert torch.equal(one[0], whole[b * 12 + r])


def test_qk_norm_rope_strides_in_place_and_streams(tf):
    rng = np.random.default_rng(6)
    x = torch.tensor(rng.normal(size=(6, 5 * D)), dtype=torch.bfloat16).cuda()
    turns = tf.rope_turns(64, 1e4)
    pos = dev_pos([3, 50])
    want = tf.qk_norm_rope(x, 3, 1, pos, turns=turns)
    wide = torch.zeros((6, 8 * D), dtype=torch.bfloat16, device="cuda")
    wide[:, :5 * D] = x
    out = torch.full((6, 6 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    tf.qk_norm_rope(wide[:, :5 * D], 3, 1, pos, turns=turns, out=out[:, :5 * D])
    assert torch.equal(out[:, :5 * D], want) and bool((out[:, 5 * D:] == 7).all())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = x.clone()
    s.wait_stream(torch.cuda.current_stream())
    tf.qk_norm_rope(again, 3, 1, pos, turns=turns, out=again, stream=s)
    s.synchronize()
    assert torch.equal(again, want)
    bits = tf.qk_norm_rope(x.view(torch.int16), 3, 1, pos, turns=turns)
    assert torch.equal(bits, want)


def test_qk_norm_rope_zero_and_nonfinite_heads(tf):
    x = torch.ones((2, 4 * D), dtype=torch.float32, device="cuda")
    x[0, :D] = 0
    x[1, D + 5] = math.nan
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    y = tf.qk_norm_rope(x, 2, 1, dev_pos([0]), turns=tf.rope_turns(128), q_weight=w, k_weight=w).float().cpu()
    assert not y[0, :D].any()                           # eps keeps a zero head finite
    assert y[1, D:2 * D].isnan().all()                  # a NaN stays in its head
    assert y[1, :D].isfinite().all() and y[1, 2 * D:].isfinite().all() and y[0].isfinite().all()


# ---------------------------------------------------------------- cache writes and reads
def rows_of(k):
    """[n_seq][n_kv][R][128] -> [n_seq*R][n_kv*128]."""
    n_seq, n_kv, R, _ = k.shape
    return np.ascontiguousarray(k.transpose(0, 2, 1, 3).reshape(n_seq * R, n_kv * D))


KV = [(1, 1, 1, [0], 256), (3, 2, 5, [0, 17, 251], 256), (2, 8, 16, [240, 3], 512), (5, 3, 1, [0, -1, 255, -1, 7], 256),
      (1, 4, 700, [68], 768)]


@pytest.mark.parametrize("n_seq,n_kv,R,pos,max_len", KV)
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_store_writes_the_documented_layout_and_load_reads_it(tf, n_seq, n_kv, R, pos, max_len, fmt):
    rng = np.random.default_rng(R + n_kv)
    size = np.exp2(rng.integers(-30, 12, size=(n_seq, n_kv, R, 1)))
    kv = [inputs.bf16_bits_from_f32((rng.normal(size=(n_seq, n_kv, R, D)) * size).astype(np.float32)) for _ in range(2)]
    kv[0][0, 0, 0] = 0                                                   # an all-zero vector
    kv[1][0, 0, R // 2, 5:9] = [0x0001, 0x8000, 0x7F7F, 0xFF7F]          # subnormal, -0, the largest values
    cache = tf.KVBatch(n_seq, n_kv, max_len, fmt)
    ws = cache.store(dev_bits16(rows_of(kv[0])), dev_bits16(rows_of(kv[1])), dev_pos(pos))
    assert tf.workspace_status(ws) == tf.TF_DEV_OK
    got = cache.load(dev_pos(pos), R, ws=ws)
    for which, (x, phys) in enumerate(zip(kv, (cache.k, cache.v))):
        phys = phys.cpu().numpy()
        scales = [cache.k_scale, cache.v_scale][which]
        back = f64(got[which]).reshape(n_seq, R, n_kv, D).transpose(0, 2, 1, 3)
        for b in range(n_seq):
            if pos[b] < 0:
                assert not phys[b].any() and not back[b].any()
                continue
            mask = np.zeros(max_len, bool)
            mask[pos[b]:pos[b] + R] = True
            if fmt == "bf16":
                plain = kv_unswizzle(phys[b].view(np.uint16))
                assert np.array_equal(plain[:, mask], x[b]) and not plain[:, ~mask].any()
                assert np.array_equal(back[b], bf16_to_f64(x[b]))
                continue
            s = scales[b].cpu().numpy()
            assert not phys[b][:, ~mask].any() and not s[:, ~mask].any()
            for j in range(n_kv):
                for r in range(R):
                    codes, sc = obat.e4m3_vector(bf16_to_f64(x[b, j, r]))
                    assert s[j, pos[b] + r] == sc
                    assert np.array_equal(phys[b, j, pos[b] + r], obat.e4m3_place(codes))
                    assert np.array_equal(back[b, j, r], obat.e4m3_values(codes, sc))


def test_e4m3_store_rounds_every_bf16_to_the_nearest_code(tf):
    """All finite bf16 patterns of one binade below 448 and all ties, each in a vector
    whose largest element pins the scale to 1."""
    bits = np.arange(0, 0x43E1, dtype=np.uint16)                          # 0 .. 448
    bits = np.concatenate([bits, bits | 0x8000])
    n = -(-len(bits) // 127)
    x = np.zeros((n, D), np.uint16)
    x[:, 0] = 0x43E0                                                      # 448
    x[:, 1:].reshape(-1)[:len(bits)] = bits
    x[:, 1:] = np.resize(bits, (n, 127))
    cache = tf.KVBatch(1, 1, -(-n // 256) * 256, "e4m3")
    cache.store(dev_bits16(x), dev_bits16(x), dev_pos([0]))
    k, v = cache.load(dev_pos([0]), n)
    want = torch.from_numpy(bf16_to_f64(x)).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(f64(k), want) and np.array_equal(f64(v), want)
    assert bool((cache.k_scale[0, 0, :n] == 127).all())


def test_e4m3_vectors_with_a_nonfinite_element_read_as_nan(tf):
    x = np.zeros((4, 2 * D), np.uint16)
    x[:] = 0x3F80
    x[0, 3], x[1, D + 100], x[2, 64] = 0x7F80, 0xFF80, 0x7FC0              # inf, -inf, NaN
    cache = tf.KVBatch(1, 2, 256, "e4m3")
    cache.store(dev_bits16(x), dev_bits16(x), dev_pos([9]))
    k, v = cache.load(dev_pos([9]), 4)
    nan = torch.zeros((4, 2), dtype=torch.bool)
    nan[0, 0] = nan[1, 1] = nan[2, 0] = True
    for t in (k, v):
        t = t.float().cpu().reshape(4, 2, D)
        assert bool(t[nan].isnan().all()) and bool((t[~nan] == 1).all())
    cache.store(dev_bits16(np.full((4, 2 * D), 0x4000, np.uint16)), dev_bits16(x), dev_pos([9]))     # rewritten: no NaN stays
    assert bool((cache.load(dev_pos([9]), 4)[0].float() == 2).all())


def test_bad_positions_are_reported_and_write_nothing(tf):
    rows = dev_bits16(inputs.bf16_normal(inputs.rng_for(9), (6, 2 * D)))
    for fmt in ("bf16", "e4m3"):
        cache = tf.KVBatch(3, 2, 256, fmt)
        ws = cache.store(rows, rows, dev_pos([255, -2, 254]))            # one past the end, negative, the last place
        assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION
        assert not cache.k[:2].any() and cache.k[2, :, 254:].any()
        k, _ = cache.load(dev_pos([255, 1 << 40, 254]), 2, ws=ws)
        assert tf.workspace_status(ws) == tf.TF_DEV_BAD_POSITION
        assert not k[:4].any() and k[4:].any()
        cache.store(rows, rows, dev_pos([-1, -1, -1]), ws=ws)
        assert tf.workspace_status(ws) == tf.TF_DEV_OK


def test_a_batch_of_one_shares_a_kvcache(tf):
    rows = dev_bits16(inputs.bf16_normal(inputs.rng_for(10), (7, 2 * D)))
    cache = tf.KVCache(2, 256)
    cache.append(rows, rows, dev_pos([30]))
    k, v = tf.KVBatch.of(cache).load(dev_pos([30]), 7)
    assert torch.equal(k.view(torch.int16), rows) and torch.equal(v.view(torch.int16), rows)


def test_strided_rows(tf):
    rows = dev_bits16(inputs.bf16_normal(inputs.rng_for(11), (4, 6 * D)))
    cache = tf.KVBatch(2, 2, 256, "e4m3")
    cache.store(rows[:, D:3 * D], rows[:, 4 * D:], dev_pos([0, 4]))
    out = torch.zeros((4, 5 * D), dtype=torch.int16, device="cuda")
    cache.load(dev_pos([0, 4]), 2, k=out[:, :2 * D], v=out[:, 3 * D:])
    dense = tf.KVBatch(2, 2, 256, "e4m3")
    dense.store(rows[:, D:3 * D].contiguous(), rows[:, 4 * D:].contiguous(), dev_pos([0, 4]))
    k, v = dense.load(dev_pos([0, 4]), 2)
    assert torch.equal(out[:, :2 * D], k.view(torch.int16)) and torch.equal(out[:, 3 * D:], v.view(torch.int16))
    assert not out[:, 2 * D:3 * D].any()


def test_binding_refusals(tf):
    rows = torch.zeros((4, 2 * D), dtype=torch.int16, device="cuda")
    cache = tf.KVBatch(2, 2, 256)
    pos = dev_pos([0, 0])
    bad = [lambda: tf.KVBatch(1, 1, 256, "int8"),
           lambda: cache.store(rows[:3], rows[:3], pos), lambda: cache.store(rows.float(), rows, pos),
           lambda: cache.store(rows, rows[:2], pos), lambda: cache.store(rows[:, :D], rows[:, :D], pos),
           lambda: cache.store(rows, rows, pos[:1]), lambda: cache.store(rows, rows, pos.int()),
           lambda: cache.store(rows, rows, pos.cpu()), lambda: cache.store(rows.t(), rows.t(), pos),
           lambda: cache.load(pos, 0), lambda: cache.load(pos, 257), lambda: cache.load(pos, 2, k=rows[:2], v=rows[:2]),
           lambda: tf.qk_norm_rope(rows.float(), 2, 1, pos), lambda: tf.qk_norm_rope(rows, 1, 0, pos, n_v=0, eps=-1.0),
           lambda: tf.qk_norm_rope(rows[:3], 1, 0, pos), lambda: tf.qk_norm_rope(rows, 1, 0, pos, turns=rows[0]),
           lambda: tf.qk_norm_rope(rows, 1, 0, pos, q_weight=rows[0, :D].contiguous()),
           lambda: tf.qk_norm_rope(rows.double(), 1, 0, pos)]
    for i, f in enumerate(bad):
        with pytest.raises(tf.TFError):
            f()
            pytest.fail(f"case {i} was not refused")
