"""The edges of decode.BranchDecoder on the GPU: a reply or a prompt past the capacity
given at construction is refused, what the device reports is raised, and a model may
have as many query heads per KV head as the attention takes.

Tolerance of the logits: that of tests/test_gpu_branch_decoder.py, 2^-5 of the row's
rms, for the same number of roundings per block.
"""

import numpy as np
import pytest
import torch

from oracle import batch as obat
from w4_gemm_keyed_gb300 import inputs

pytestmark = pytest.mark.gpu

V, H, F, G, ROT, THETA = 512, 256, 256, 64, 64, 1e4
SAMPLING = (0.7, 20, 0.95)


def weights_of(n_kv, group):
    rng = inputs.rng_for(95, n_kv, group)
    n_q, blocks, attn = n_kv * group, [], []
    for _ in range(2):
        (gc, gs), (uc, us), (dc, ds) = (inputs.w4_weights(rng, a, b, G) for a, b in ((H, F), (H, F), (F, H)))
        blocks.append(dict(gate_codes=gc, gate_scales=gs, up_codes=uc, up_scales=us, down_codes=dc, down_scales=ds))
        qc, qs = inputs.w4_weights(rng, H, (n_q + 2 * n_kv) * 128, G)
        oc, os_ = inputs.w4_weights(rng, n_q * 128, H, G)
        gains = inputs.bf16_bits_from_f32((1 + 0.2 * rng.normal(size=(2, 128))).astype(np.float32))
        attn.append(dict(qkv_codes=qc, qkv_scales=qs, o_codes=oc, o_scales=os_, q_norm=gains[0], k_norm=gains[1]))
    lc, ls = inputs.w4_weights(rng, H, V, G)
    return dict(emb=inputs.bf16_normal(rng, (V, H), 0.5), blocks=blocks, attn=attn, lm_codes=lc, lm_scales=ls, group=G)


@pytest.fixture(scope="module")
def model(tf):
    from w4_gemm_keyed_gb300 import decode
    return decode.upload_branch_model(weights_of(1, 2), 1, 2, THETA, ROT)


def decoder(model, n_branch=2):
    from w4_gemm_keyed_gb300 import decode
    return decode.BranchDecoder(model, n_branch, 256, 200, max_rows=4)      # 256 own entries a branch


# ---------------------------------------------------------------- capacity
def test_a_pass_past_the_own_caches_is_refused(tf, model):
    dec = decoder(model)
    dec.start([1, 2, 3])
    dec.at = [10, 252]
    assert len(dec.step(4, [[4, 5, 6]] * 2, *SAMPLING, [1, 2])) == 2        # entries 252 .. 255: the last ones
    dec.at = [10, 253]
    with pytest.raises(ValueError):
        dec.step(4, [[4, 5, 6]] * 2, *SAMPLING, [1, 2])
    assert dec.at == [10, 253]
    dec.finish(1)                                                           # a finished branch needs no room
    assert dec.step(4, [[4, 5, 6]] * 2, *SAMPLING, [1, 2])[1] is None


def test_a_reply_longer_than_its_cache_is_refused(tf, model):
    from w4_gemm_keyed_gb300 import decode
    dec = decoder(model)
    with pytest.raises(ValueError):
        decode.branch_decode(dec, [1, 2, 3], [5, 300], 1, *SAMPLING, [1, 2])
    out = decode.branch_decode(dec, [1, 2, 3], [5, 256], 1, *SAMPLING, [1, 2])
    assert [len(o) for o in out] == [5, 256]


def test_a_prompt_longer_than_its_cache_is_refused(tf, model):
    dec = decoder(model)
    dec.start([7] * 257)            # 256 entries and the replies' first input
    assert dec.prompt_len == 256
    with pytest.raises(ValueError):
        dec.start([7] * 258)
    assert dec.prompt_len == 256


def test_rows_outside_the_decoder_are_refused(tf, model):
    dec = decoder(model)
    dec.start([1])
    for R in (0, 5):
        with pytest.raises(ValueError):
            dec.step(R, [[1] * 8] * 2, *SAMPLING, [1, 2])


# ---------------------------------------------------------------- what the device reports
def test_a_prompt_token_outside_the_vocabulary_is_refused(tf, model):
    dec = decoder(model)
    dec.start([1, 2, 3])
    want = dec.step(1, [], *SAMPLING, [1, 2])
    dec.start([1, 2, 3])
    for bad in ([1, V, 3], [1, 2, V], [-1]):
        with pytest.raises(ValueError):
            dec.start(bad)
    assert dec.step(1, [], *SAMPLING, [1, 2]) == want       # the prompt before is still there


def test_a_draft_outside_the_vocabulary_is_only_rejected(tf, model):
    dec = decoder(model)
    dec.start([1, 2, 3])
    want = dec.step(1, [], *SAMPLING, [1, 2])
    for bad in (V, -1):
        dec.start([1, 2, 3])
        got = dec.step(2, [[bad], [bad]], *SAMPLING, [1, 2])
        assert [(a, t[:1]) for a, t in got] == want


def test_nonfinite_logits_are_raised_where_they_are_committed(tf, model):
    dec = decoder(model)
    dec.start([1, 2, 3])
    want = dec.step(1, [], *SAMPLING, [1, 2])
    spoilt = next(t for t in range(10, V) if all(t != w[1][0] for w in want))
    kept = model.base.embedding[spoilt].clone()
    try:
        model.base.embedding[spoilt] = 0x7FC0           # NaN
        dec.start([1, 2, 3])
        got = dec.step(2, [[spoilt], [spoilt]], *SAMPLING, [1, 2])      # rejected: no harm done
        assert [(a, t[:1]) for a, t in got] == want
        dec.start([1, 2, spoilt])
        with pytest.raises(tf.TFError):
            dec.step(1, [], *SAMPLING, [1, 2])
    finally:
        model.base.embedding[spoilt] = kept
    dec.start([1, 2, 3])
    assert dec.step(1, [], *SAMPLING, [1, 2]) == want


@pytest.mark.parametrize("name", ["ws_attn", "ws_gemm", "ws_block"])
def test_a_reported_timeout_is_raised(tf, model, name):
    dec = decoder(model)
    dec.start([1, 2, 3])
    want = dec.step(1, [], *SAMPLING, [1, 2])

    def report():
        getattr(dec, name)[:4].view(torch.int32).fill_(tf.TF_DEV_TIMEOUT)

    dec.start([1, 2, 3])
    report()
    with pytest.raises(tf.TFError):
        dec.step(1, [], *SAMPLING, [1, 2])
    dec.start([1, 2, 3])                # the report was taken away with it
    assert dec.step(1, [], *SAMPLING, [1, 2]) == want
    report()
    with pytest.raises(tf.TFError):
        dec.start([1, 2, 3])
    dec.start([1, 2, 3])
    assert dec.step(1, [], *SAMPLING, [1, 2]) == want


# ---------------------------------------------------------------- head layouts
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
@pytest.mark.parametrize("n_kv,group", [(1, 16), (2, 11)])
def test_many_query_heads_per_kv_head(tf, fmt, n_kv, group):
    """Prompts longer than one pass of rows x group = 128 query vectors: the logits are
    the oracle's, the replies those of each branch alone."""
    from w4_gemm_keyed_gb300 import decode
    weights = weights_of(n_kv, group)
    m = decode.upload_branch_model(weights, n_kv, group, THETA, ROT)
    rng = inputs.rng_for(96, group)
    prompt = rng.integers(0, V, 45).tolist()
    replies = [rng.integers(0, V, 3).tolist() for _ in range(2)]
    dec = decode.BranchDecoder(m, 2, 256, 64, fmt)
    dec.start(prompt)
    dec.step(4, replies, *SAMPLING, [1, 2])
    oracle_model = dict(weights, n_kv=n_kv, attn_group=group, adjacent=False, quantise=fmt == "e4m3",
                        inv_freq=[THETA ** (-2 * d / ROT) for d in range(ROT // 2)])
    for b, reply in enumerate(replies):
        ref = obat.branch_logits(oracle_model, prompt + reply)[len(prompt) - 1:]
        got = dec.logits[4 * b:4 * b + 4].double().cpu().numpy()
        rms = np.sqrt(np.mean(ref ** 2, axis=1, keepdims=True))
        worst = np.max(np.abs(got - ref) / rms)
        assert worst <= 2.0 ** -5, worst
    one = decode.BranchDecoder(m, 1, 256, 64, fmt)
    alone = [decode.branch_decode(one, prompt, [12], 1, *SAMPLING, [s])[0] for s in (1234, 1235)]
    assert decode.branch_decode(dec, prompt, [12, 12], 1, *SAMPLING, [1234, 1235]) == alone


def test_drafted_rows_need_drafts(tf, model):
    from w4_gemm_keyed_gb300 import decode
    with pytest.raises(ValueError):
        decode.branch_decode(decoder(model), [1, 2], [4, 4], 2, *SAMPLING, [1, 2])
