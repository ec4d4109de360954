"""Pointers and buffers that the prompt and tree calls refuse before any device work (no GPU needed)."""

import ctypes

import pytest

from w4_gemm_keyed_gb300 import tf


@pytest.fixture(scope="module")
def lib():
    from w4_gemm_keyed_gb300 import build
    build.build()
    return tf.load()


ACCEPT = dict(parents=256, tokens=256, sampled=256, pos=256, n_seq=2, n=8, accepted=256, bonus=256, path=256,
              committed=256, ws=256, ws_bytes=256)


@pytest.mark.parametrize("name", ["parents", "tokens", "sampled", "accepted", "bonus", "path", "committed"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_accept_takes_whole_words(lib, name, off):
    """A 4-byte access at such an address would be a fault."""
    assert lib.tf_tree_accept(*{**ACCEPT, name: 256 + off}.values(), None) == tf.TF_ERR_INVALID_ARG


# ---------------------------------------------------------------- outputs that overlap what is read
# Rows of 2 x 4 heads (1,024 elements): queries 1 MB into the address space, elsewhere 16 MB.
Q, FAR = 1 << 20, 1 << 24
WITHIN = [  # output address and row stride (elements) next to queries at Q, stride 2048, 9 rows
    (Q, 2048), (Q + 16, 2048), (Q + 2 * 1016, 2048), (Q - 2 * 1016, 2048), (Q + 2 * 2048 * 8, 2048),
    (Q - 2 * 2048 * 8, 2048), (Q + 2 * (2048 * 8 + 1016), 2048), (Q + 2 * 1032, 2048), (Q, 1024), (Q + 2 * 1024, 4096)]


@pytest.mark.parametrize("out,ldo", WITHIN)
def test_a_prompt_output_lies_in_no_input(lib, out, ldo):
    here, there = dict(ld=2048, p=Q), dict(ld=2048, p=FAR)
    for which in range(3):
        q, k, v = (here if i == which else there for i in range(3))
        if which and out in (Q + 2 * 1016, Q + 2 * (2048 * 8 + 1016)):
            continue        # keys and values are 256 wide
        status = lib.tf_attention_prompt(q["p"], q["ld"], k["p"], k["ld"], v["p"], v["ld"], 9, 2, 4, 256, 1, out, ldo, 256,
                                         256, None)
        assert status == tf.TF_ERR_INVALID_ARG and b"overlaps " + b"qkv"[which:which + 1] in lib.tf_last_error()


@pytest.mark.parametrize("out,ldo", WITHIN)
def test_a_tree_output_lies_in_no_queries(lib, out, ldo):
    own = tf.KVBatchC(256, 256, 256, 256, 1, 2, 256, 0)
    status = lib.tf_attention_tree(ctypes.byref(own), None, 0, 4, Q, 2048, 9, 256, 256, out, ldo, 256, 1 << 30, None)
    assert status == tf.TF_ERR_INVALID_ARG and b"overlaps q" in lib.tf_last_error()
