"""Pointers and buffers that the prompt and tree calls refuse before any device work (no GPU needed)."""

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
