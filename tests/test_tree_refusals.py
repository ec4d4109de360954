"""What the prompt and tree calls refuse before any device work (no GPU needed)."""

import ctypes
import types

import pytest
import torch

from w4_gemm_keyed_gb300 import tf

BIG = 1 << 30
BAD, NO, WS = tf.TF_ERR_INVALID_ARG, tf.TF_ERR_UNSUPPORTED, tf.TF_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    from w4_gemm_keyed_gb300 import build
    build.build()
    return tf.load()


def batch(n_seq=2, n_kv=2, max_len=256, fmt=0, k=256):
    return tf.KVBatchC(k, 256, 256, 256, n_seq, n_kv, max_len, fmt)


PROMPT = dict(q=256, ldq=1024, k=256, ldk=256, v=256, ldv=256, rows=9, n_kv=2, group=4, starts=256, n_seq=3, out=256,
              ldo=1024, ws=256, ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), BAD), (dict(k=None), BAD), (dict(v=None), BAD), (dict(out=None), BAD), (dict(starts=None), BAD),
    (dict(q=264), BAD), (dict(k=258), BAD), (dict(out=260), BAD), (dict(starts=260), BAD),
    (dict(ldq=1023), BAD), (dict(ldq=1028), BAD), (dict(ldk=248), BAD), (dict(ldv=128), BAD), (dict(ldo=1020), BAD),
    (dict(rows=-1), BAD), (dict(rows=0x7FFFFFFF), NO), (dict(group=0), NO), (dict(group=17), NO), (dict(n_kv=0), NO),
    (dict(n_kv=129), NO), (dict(n_seq=0), NO), (dict(n_seq=1025), NO),
    (dict(ws=None), WS), (dict(ws=384), WS), (dict(ws_bytes=255), WS)])
def test_prompt(lib, change, status):
    assert lib.tf_attention_prompt(*{**PROMPT, **change}.values(), None) == status
    assert lib.tf_last_error() != b""


def test_a_prompt_of_no_rows_is_nothing_to_do(lib):
    assert lib.tf_attention_prompt(*{**PROMPT, "rows": 0, "q": None, "out": None}.values(), None) == tf.TF_OK


def tree(lib, own, prefix=None, **change):
    a = {**dict(prefix_len=0, group=4, q=256, ldq=1024, n=8, pos=256, parents=256, out=256, ldo=1024, ws=256,
                ws_bytes=BIG), **change}
    v = list(a.values())
    return lib.tf_attention_tree(ctypes.byref(own), ctypes.byref(prefix) if prefix else None, *v, None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), BAD), (dict(q=264), BAD), (dict(ldq=1016), BAD), (dict(ldq=1028), BAD), (dict(pos=None), BAD),
    (dict(pos=260), BAD), (dict(parents=None), BAD), (dict(parents=258), BAD), (dict(out=None), BAD), (dict(ldo=512), BAD),
    (dict(n=0), BAD), (dict(n=65), BAD), (dict(group=0), NO), (dict(group=17), NO), (dict(prefix_len=-1), BAD),
    (dict(prefix_len=3), BAD), (dict(ws=None), WS), (dict(ws_bytes=255), WS)])
def test_tree(lib, change, status):
    assert tree(lib, batch(), **change) == status


def test_tree_caches(lib):
    assert tree(lib, batch(n_seq=0)) == NO and tree(lib, batch(n_seq=1025)) == NO
    assert tree(lib, batch(max_len=100)) == NO and tree(lib, batch(fmt=2)) == NO and tree(lib, batch(k=258)) == BAD
    one = batch(n_seq=1)
    assert tree(lib, batch(), batch(n_seq=2), prefix_len=3) == BAD          # a prefix of two sequences
    assert tree(lib, batch(), batch(n_seq=1, fmt=1), prefix_len=3) == BAD   # of another format
    assert tree(lib, batch(), one, prefix_len=257) == BAD                   # past its entries
    assert lib.tf_attention_tree_workspace_bytes(ctypes.byref(batch()), 4, 8, 0) >= 256
    for group, n, prefix_len in ((17, 8, 0), (4, 65, 0), (4, 0, 0), (4, 8, -1)):
        assert lib.tf_attention_tree_workspace_bytes(ctypes.byref(batch()), group, n, prefix_len) == 0


ACCEPT = dict(parents=256, tokens=256, sampled=256, pos=256, n_seq=2, n=8, accepted=256, bonus=256, path=256,
              committed=256, ws=256, ws_bytes=256)


@pytest.mark.parametrize("change,status", [
    *((dict([(name, None)]), BAD) for name in ("parents", "tokens", "sampled", "pos", "accepted", "bonus", "path",
                                              "committed")),
    (dict(pos=260), BAD), (dict(n=0), BAD), (dict(n=65), BAD), (dict(n_seq=0), NO), (dict(n_seq=1025), NO),
    (dict(ws=None), WS), (dict(ws_bytes=128), WS)])
def test_accept(lib, change, status):
    assert lib.tf_tree_accept(*{**ACCEPT, **change}.values(), None) == status


def test_keep(lib):
    def keep(own, pos=256, path=256, ws=256, ws_bytes=256):
        return lib.tf_kv_keep(ctypes.byref(own), pos, path, ws, ws_bytes, None)
    assert keep(batch(n_kv=0)) == NO and keep(batch(max_len=255)) == NO and keep(batch(k=None)) == BAD
    assert keep(batch(), pos=None) == BAD and keep(batch(), path=None) == BAD and keep(batch(), path=257) == BAD
    assert keep(batch(), ws=None) == WS and keep(batch(), ws_bytes=0) == WS


# ---------------------------------------------------------------- the binding's own refusals
class OnDevice(torch.Tensor):
    is_cuda = True


def ones(*shape, dtype=torch.bfloat16, device="cpu"):
    return torch.ones(shape, dtype=dtype, device=device).as_subclass(OnDevice)


@pytest.fixture
def cache(monkeypatch):
    def called(*a):
        pytest.fail("the library was called")
    fake = types.SimpleNamespace(**{name: called for name, _, _ in tf.SIGNATURES})
    fake.tf_attention_tree_workspace_bytes = lambda *a: 1024
    monkeypatch.setattr(tf, "load", lambda *a: fake)
    monkeypatch.setattr(tf, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(tf, "_current_raw_stream", lambda: 0)
    return tf.KVBatch(2, 2, 256, "e4m3", device="cpu")


POS, ELSEWHERE = torch.zeros(2, dtype=torch.int64), torch.zeros(4096, dtype=torch.uint8, device="meta")
TREES = torch.zeros((2, 2), dtype=torch.int32)
PATHS = torch.zeros((2, tf.MAX_PATH), dtype=torch.int32)
STARTS = torch.tensor([0, 4], dtype=torch.int64)
REFUSED = dict(
    tree_parents_type=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES.long()),
    tree_parents_shape=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES[:, :1]),
    tree_parents_strided=lambda c: c.tree_attention(ones(4, 256), 1, POS, torch.zeros((2, 4), dtype=torch.int32)[:, ::2]),
    tree_parents_device=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES.to("meta")),
    tree_rows=lambda c: c.tree_attention(ones(5, 256), 1, POS, TREES),
    tree_pos=lambda c: c.tree_attention(ones(4, 256), 1, POS[:1], TREES),
    tree_group=lambda c: c.tree_attention(ones(4, 256), 0, POS, TREES),
    tree_q_type=lambda c: c.tree_attention(ones(4, 256, dtype=torch.float16), 1, POS, TREES),
    tree_q_columns=lambda c: c.tree_attention(ones(4, 256), 2, POS, TREES),
    tree_out=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES, out=ones(4, 256, device="meta")),
    tree_ws=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES, ws=ELSEWHERE),
    tree_prefix=lambda c: c.tree_attention(ones(4, 256), 1, POS, TREES, prefix=tf.KVBatch(1, 2, 256, "e4m3", "meta"),
                                           prefix_len=3),
    keep_path_shape=lambda c: c.keep(POS, PATHS[:, :8]),
    keep_path_type=lambda c: c.keep(POS, PATHS.long()),
    keep_pos=lambda c: c.keep(POS[:1], PATHS),
    keep_ws=lambda c: c.keep(POS, PATHS, ws=ELSEWHERE),
    accept_host=lambda c: tf.tree_accept(TREES, TREES, TREES, POS),
    accept_rank=lambda c: tf.tree_accept(ones(4, dtype=torch.int32), TREES, TREES, POS),
    accept_tokens=lambda c: tf.tree_accept(ones(2, 2, dtype=torch.int32), TREES[:1], TREES, POS),
    accept_sampled=lambda c: tf.tree_accept(ones(2, 2, dtype=torch.int32), TREES, TREES.long(), POS),
    accept_pos=lambda c: tf.tree_accept(ones(2, 2, dtype=torch.int32), TREES, TREES, POS[:1]),
    accept_ws=lambda c: tf.tree_accept(ones(2, 2, dtype=torch.int32), TREES, TREES, POS, ws=ELSEWHERE),
    prompt_host=lambda c: tf.prompt_attention(torch.ones(4, 256), ones(4, 256), ones(4, 256), 2, 1, STARTS),
    prompt_type=lambda c: tf.prompt_attention(ones(4, 256, dtype=torch.float32), ones(4, 256), ones(4, 256), 2, 1, STARTS),
    prompt_rows=lambda c: tf.prompt_attention(ones(4, 256), ones(3, 256), ones(4, 256), 2, 1, STARTS),
    prompt_columns=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 128), 2, 1, STARTS),
    prompt_strided=lambda c: tf.prompt_attention(ones(4, 512)[:, ::2], ones(4, 256), ones(4, 256), 2, 1, STARTS),
    prompt_heads=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 0, 1, STARTS),
    prompt_group=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 2, -1, STARTS),
    prompt_starts=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 2, 1, STARTS.int()),
    prompt_starts_device=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 2, 1, STARTS.to("meta")),
    prompt_scalar=lambda c: tf.prompt_attention(ones(), ones(4, 256), ones(4, 256), 2, 1, STARTS),
    prompt_out=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 2, 1, STARTS, out=ones(3, 256)),
    prompt_ws=lambda c: tf.prompt_attention(ones(4, 256), ones(4, 256), ones(4, 256), 2, 1, STARTS, ws=ELSEWHERE),
)


@pytest.mark.parametrize("name", REFUSED)
def test_the_binding_refuses(cache, name):
    with pytest.raises(tf.TFError) as e:
        REFUSED[name](cache)
    assert e.value.status in (BAD, NO)
