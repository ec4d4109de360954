"""Rows of a batch of sequences that continue one prompt (test infrastructure).

* ``qk_norm_rope`` -- RMSNorm of each query / key head (Zhang & Sennrich 2019;
  per-head gain), then rotation by position (Su et al. 2021): the pair
  (a, b) of frequency f at position p becomes
  (a cos(pf) - b sin(pf), b cos(pf) + a sin(pf));
* ``e4m3_vector`` / ``e4m3_table`` -- 128-element vectors as E4M3 codes (OCP
  8-bit floating point: bias 7, subnormals, largest 448) times one power of two;
* ``attention_batch`` -- causal scaled dot-product attention of each sequence's
  rows over a shared prefix and the sequence's own entries.

Everything is evaluated in fp64; arrays are in plain layouts.
"""

from __future__ import annotations

import math

import numpy as np

HEAD_DIM = 128


def qk_norm_rope(x, n_q, n_k, wq, wk, eps, inv_freq, adjacent, positions):
    """fp64 [rows][heads][128] of x (same shape).  wq, wk: gains [128] or None (no
    norm); inv_freq: radians per position of each pair (empty: no rotation)."""
    y = np.array(x, dtype=np.float64)
    for lo, hi, w in ((0, n_q, wq), (n_q, n_q + n_k, wk)):
        if w is not None:
            h = y[:, lo:hi]
            y[:, lo:hi] = h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    out = y.copy()
    n, half = n_q + n_k, len(inv_freq)
    for i, f in enumerate(inv_freq):
        i0, i1 = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        ang = np.array([math.fmod(float(p) * float(f), 2 * math.pi) for p in positions])[:, None]
        a, b = y[:, :n, i0], y[:, :n, i1]
        out[:, :n, i0] = a * np.cos(ang) - b * np.sin(ang)
        out[:, :n, i1] = b * np.cos(ang) + a * np.sin(ang)
    return out


def e4m3_table():
    """Value of every E4M3 byte (NaN at 0x7F and 0xFF)."""
    v = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        mag = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = math.nan if e == 15 and m == 7 else (-mag if s else mag)
    return v


def e4m3_vector(x):
    """(codes uint8 [128], scale byte) of one fp64 vector: the smallest exponent e in
    [-120, 7] with max|x| <= 448 * 2^e, nearest code with ties to the even one,
    saturating; scale byte e + 127, or 255 (codes 0) where x has an infinity or NaN."""
    x = np.asarray(x, dtype=np.float64)
    if not np.all(np.isfinite(x)):
        return np.zeros(x.shape, np.uint8), 255
    peak = float(np.max(np.abs(x)))
    e = -120
    while e < 7 and peak > 448.0 * 2.0 ** e:
        e += 1
    mags = e4m3_table()[:127]                       # ascending magnitudes of codes 0..126
    a = np.minimum(np.abs(x) / 2.0 ** e, 448.0)
    hi = np.searchsorted(mags, a)                   # first code with magnitude >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | (np.signbit(x).astype(np.int64) << 7)).astype(np.uint8), e + 127


def e4m3_values(codes, scale):
    """fp64 values of a vector's codes and scale byte."""
    if scale == 255:
        return np.full(np.shape(codes), math.nan)
    return e4m3_table()[np.asarray(codes)] * 2.0 ** (int(scale) - 127)


def e4m3_place(codes):
    """A vector's codes in the order the device stores them (the rule in tf.h)."""
    out = np.empty(HEAD_DIM, np.uint8)
    for d in range(HEAD_DIM):
        i = {1: 2, 2: 1}.get(d % 4, d % 4)
        out[16 * ((d % 64) // 8) + 8 * (d // 64) + 4 * ((d % 8) // 4) + i] = codes[d]
    return out


def attention_batch(q, shared_k, shared_v, own_k, own_v, pos):
    """q [B][R][n_kv][group][128]; shared_k, shared_v [n_kv][P][128]; own_k, own_v
    [B][n_kv][L][128]; pos [B] (negative: idle).  Returns (out, spread) of q's
    shape: out = sum_t w_t v_t and spread = sum_t w_t |v_t| with the softmax weights
    w, zeros for idle sequences."""
    q = np.asarray(q, np.float64)
    B, R, n_kv, _, D = q.shape
    P = shared_k.shape[1]
    out, spread = np.zeros_like(q), np.zeros_like(q)
    for b in range(B):
        if pos[b] < 0:
            continue
        for j in range(n_kv):
            for r in range(R):
                n = int(pos[b]) + r + 1
                k = np.concatenate([shared_k[j], own_k[b, j, :n]])
                v = np.concatenate([shared_v[j], own_v[b, j, :n]])
                s = q[b, r, j] @ k.T / math.sqrt(D)
                w = np.exp(s - s.max(axis=-1, keepdims=True))
                w /= w.sum(axis=-1, keepdims=True)
                out[b, r, j] = w @ v
                spread[b, r, j] = w @ np.abs(v)
    return out, spread


def branch_logits(model, tokens, eps=1e-6):
    """fp64 logits [len(tokens)][V] of the branch decoder (decode.BranchModel) for one
    sequence of tokens at positions 0.., every row at once: per block
    n = bf16(rms(x)); q, k, v = n Wqkv; q, k normalised and turned, all three to
    bf16; o = bf16(causal attention); x += o Wo; then the MLP block.  ``model`` is
    attn_decoder's dict with, per ``attn`` entry, q_norm and k_norm (bf16 bits), and
    inv_freq, adjacent, quantise (cache vectors through E4M3)."""
    from .decoder import block_forward, final_input
    from .linear import bf16_to_f64, w4_linear
    from .numerics import bf16_bits_of, bf16_round, rms_norm
    G, n_kv, g, T = model["group"], model["n_kv"], model["attn_group"], len(tokens)
    n_q = n_kv * g
    x = bf16_to_f64(model["emb"][np.asarray(tokens)])
    for blk, att in zip(model["blocks"], model["attn"]):
        y = w4_linear(att["qkv_codes"], att["qkv_scales"], bf16_bits_of(bf16_round(rms_norm(x, eps))), G)
        y = qk_norm_rope(y.reshape(T, n_q + 2 * n_kv, HEAD_DIM), n_q, n_kv, bf16_to_f64(att["q_norm"]),
                         bf16_to_f64(att["k_norm"]), eps, model["inv_freq"], model["adjacent"], range(T))
        y = bf16_round(y)
        kv = y[:, n_q:]
        if model["quantise"]:
            kv = np.stack([e4m3_values(*e4m3_vector(v)) for v in kv.reshape(-1, HEAD_DIM)]).reshape(kv.shape)
        k, v = kv[:, :n_kv].transpose(1, 0, 2), kv[:, n_kv:].transpose(1, 0, 2)
        q = y[:, :n_q].reshape(1, T, n_kv, g, HEAD_DIM)
        o = attention_batch(q, k[:, :0], v[:, :0], k[None], v[None], [0])[0].reshape(T, n_q * HEAD_DIM)
        x = x + w4_linear(att["o_codes"], att["o_scales"], bf16_bits_of(bf16_round(o)), G)
        x = block_forward(x, blk, G)
    return w4_linear(model["lm_codes"], model["lm_scales"], final_input(x), G)
