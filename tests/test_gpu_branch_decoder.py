"""Several replies of one prompt (decode.BranchDecoder): norm and rotation, shared and
own caches, and attention over both, run together on the GPU.

* each reply's tokens are those of its branch decoding alone, one row a pass:
  neither drafts (R = 1, 4, 5), nor the number of branches, nor branches that
  finish early change them, over bf16 and E4M3 caches;
* teacher-forced logits against the fp64 oracle decoder.  Tolerance 2^-5 of the
  row's rms: both sides round the same values to bf16 at the same points (six per
  block), and where their fp32 and fp64 results fall on different sides of a
  rounding boundary, or the attention's weights are rounded, an element moves by at
  most 2^-8 of itself; 13 such steps all at their full size and independent give
  sqrt(13) 2^-8 = 2^-6.1 of the rms, and the largest of some thousand logits is
  allowed twice that.
"""

import numpy as np
import pytest
import torch

from oracle import batch as obat
from w4_gemm_keyed_gb300 import inputs

pytestmark = pytest.mark.gpu

V, H, F, G, N_KV, GROUP, ROT, THETA = 1024, 256, 512, 64, 2, 4, 64, 1e4
N_Q = N_KV * GROUP
SAMPLING = (0.7, 20, 0.95)


@pytest.fixture(scope="module")
def weights():
    rng = inputs.rng_for(91)
    blocks, attn = [], []
    for _ in range(2):
        (gc, gs), (uc, us), (dc, ds) = (inputs.w4_weights(rng, a, b, G) for a, b in ((H, F), (H, F), (F, H)))
        blocks.append(dict(gate_codes=gc, gate_scales=gs, up_codes=uc, up_scales=us, down_codes=dc, down_scales=ds))
        qc, qs = inputs.w4_weights(rng, H, (N_Q + 2 * N_KV) * 128, G)
        oc, os_ = inputs.w4_weights(rng, N_Q * 128, H, G)
        gains = inputs.bf16_bits_from_f32((1 + 0.2 * rng.normal(size=(2, 128))).astype(np.float32))
        attn.append(dict(qkv_codes=qc, qkv_scales=qs, o_codes=oc, o_scales=os_, q_norm=gains[0], k_norm=gains[1]))
    lc, ls = inputs.w4_weights(rng, H, V, G)
    return dict(emb=inputs.bf16_normal(rng, (V, H), 0.5), blocks=blocks, attn=attn, lm_codes=lc, lm_scales=ls, group=G)


@pytest.fixture(scope="module")
def model(tf, weights):
    from w4_gemm_keyed_gb300 import decode
    return decode.upload_branch_model(weights, N_KV, GROUP, THETA, ROT)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("P", [1, 150])
def test_replies_do_not_depend_on_drafts_or_on_each_other(tf, model, fmt, P):
    from w4_gemm_keyed_gb300 import decode
    rng = inputs.rng_for(92, P)
    prompt = rng.integers(0, V, P).tolist()
    lens, seeds = [40, 9, 0, 33, 40], [1234, 1235, 1236, 1237, 1234]
    one = decode.BranchDecoder(model, 1, 256, 64, fmt)
    alone = [decode.branch_decode(one, prompt, [n], 1, *SAMPLING, [s])[0] for n, s in zip(lens, seeds)]
    assert alone[0] == alone[4] and len(set(map(tuple, alone[:2] + alone[3:4]))) == 3
    dec = decode.BranchDecoder(model, 5, 256, 64, fmt)
    assert decode.branch_decode(dec, prompt, lens, 1, *SAMPLING, seeds) == alone
    for R in (4, 5):
        noisy = inputs.rng_for(93, R)

        def drafts(b, k, n):
            return inputs.noisy_drafts(noisy, np.array((alone[b] + [0] * 8)[k:k + n]), 0.75, V)

        assert decode.branch_decode(dec, prompt, lens, R, *SAMPLING, seeds, drafts) == alone
    for ws in (dec.ws_status, dec.ws_attn, dec.ws_gemm, dec.ws_sample):
        assert tf.workspace_status(ws) == tf.TF_DEV_OK


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_teacher_forced_logits(tf, model, weights, fmt):
    from w4_gemm_keyed_gb300 import decode
    rng = inputs.rng_for(94)
    prompt, P = rng.integers(0, V, 70).tolist(), 70
    replies = [rng.integers(0, V, 12).tolist() for _ in range(3)]
    dec = decode.BranchDecoder(model, 3, 256, 64, fmt)
    dec.start(prompt)
    got = [[] for _ in replies]
    for k in range(0, 12, 4):       # drafts are the replies; the position is moved as if all were accepted
        dec.last.copy_(torch.tensor([(prompt + r)[P + k - 1] for r in replies], dtype=torch.int32))
        dec.at = [k] * 3
        dec.step(4, [r[k:k + 3] for r in replies], *SAMPLING, [1, 2, 3])
        for b in range(3):
            got[b].append(dec.logits[4 * b:4 * b + 4].double().cpu().numpy())
    oracle_model = dict(weights, n_kv=N_KV, attn_group=GROUP, adjacent=False, quantise=fmt == "e4m3",
                        inv_freq=[THETA ** (-2 * d / ROT) for d in range(ROT // 2)])
    for b, reply in enumerate(replies):
        ref = obat.branch_logits(oracle_model, prompt + reply[:11])[P - 1:]
        rows = np.concatenate(got[b])
        assert rows.shape == ref.shape
        rms = np.sqrt(np.mean(ref ** 2, axis=1, keepdims=True))
        worst = np.max(np.abs(rows - ref) / rms)
        assert worst <= 2.0 ** -5, worst
