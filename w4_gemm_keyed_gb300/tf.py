"""Thin Python binding of libtf (the C ABI in include/tf.h).

Argument marshalling only: every step of the verify pass runs in the
library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  If the shared library is missing the functions raise -- there is
no CPU fallback.
"""

from __future__ import annotations

import ctypes
import math
import os
from fractions import Fraction

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtf.so")

TF_OK, TF_ERR_INVALID_ARG, TF_ERR_UNSUPPORTED, TF_ERR_CUDA, TF_ERR_TIMEOUT, TF_ERR_WORKSPACE = range(6)
TF_DEV_OK, TF_DEV_TIMEOUT, TF_DEV_NONFINITE_LOGIT, TF_DEV_BAD_TOKEN, TF_DEV_BAD_POSITION, TF_DEV_BAD_TREE = range(6)
HEAD_DIM = 128
TF_OP_LANE_GEMM, TF_OP_KEYED_SAMPLE, TF_OP_ATTENTION = 1, 2, 3
MAX_ROWS = 16
MAX_QUERIES = 128       # rows x query heads per KV head of one sequence in KVBatch.attention
MAX_NODES, MAX_PATH = 64, 16    # rows of a tree of drafts, and nodes on one of its paths, at most
MAX_TOP_K = 64
KV_FORMATS = {"bf16": 0, "e4m3": 1}

_TWO_PI = Fraction("6.28318530717958647692528676655900576839433879875021164194988918461563281257241800")

P = ctypes.c_void_p
I32 = ctypes.c_int32
SZ = ctypes.c_size_t


class TFError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"tf status {status}: {message}")
        self.status = status


class W4MatrixC(ctypes.Structure):
    _fields_ = [("packed", P), ("K", I32), ("N", I32), ("group", I32), ("affine", I32)]


class Nvfp4MatrixC(ctypes.Structure):
    _fields_ = [("packed", P), ("K", I32), ("N", I32), ("global_scale", ctypes.c_float)]


class SamplingC(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_k", I32), ("top_p", ctypes.c_float)]


class MoeLayerC(ctypes.Structure):
    _fields_ = [("gate_up", P), ("down", P), ("hidden", I32), ("ffn", I32), ("n_experts", I32),
                ("top_k", I32), ("group", I32)]


class KVCacheC(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("n_kv", I32), ("max_len", I32)]


class KVBatchC(ctypes.Structure):
    _fields_ = [("k", P), ("v", P), ("k_scale", P), ("v_scale", P), ("n_seq", I32), ("n_kv", I32), ("max_len", I32),
                ("format", I32)]


class ModelC(ctypes.Structure):
    _fields_ = [("vocab", I32), ("hidden", I32), ("ffn", I32), ("n_blocks", I32), ("group", I32),
                ("rms_eps", ctypes.c_float), ("embedding", P), ("gate_up", ctypes.POINTER(W4MatrixC)),
                ("down", ctypes.POINTER(W4MatrixC)), ("lm_head", W4MatrixC)]


# (name, restype, argtypes) of every exported symbol
SIGNATURES = [
    ("tf_last_error", ctypes.c_char_p, []),
    ("tf_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("tf_version", ctypes.c_int, []),
    ("tf_device_sm_count", I32, []),
    ("tf_workspace_status", ctypes.c_int, [P, P, ctypes.POINTER(I32)]),
    ("tf_w4_packed_bytes", SZ, [I32, I32, I32]),
    ("tf_pack_w4", ctypes.c_int, [P, P, I32, I32, I32, P, SZ, P]),
    ("tf_w4_affine_packed_bytes", SZ, [I32, I32, I32]),
    ("tf_pack_w4_affine", ctypes.c_int, [P, P, P, I32, I32, I32, P, SZ, P]),
    ("tf_pack_w4_gate_up", ctypes.c_int, [P, P, I32, I32, I32, P, SZ, P]),
    ("tf_lane_gemm_workspace_bytes", SZ, [I32, I32, I32]),
    ("tf_nvfp4_packed_bytes", SZ, [I32, I32]),
    ("tf_pack_nvfp4", ctypes.c_int, [P, P, I32, I32, P, SZ, P]),
    ("tf_lane_gemm_nvfp4_workspace_bytes", SZ, [I32, I32]),
    ("tf_lane_gemm_nvfp4", ctypes.c_int, [ctypes.POINTER(Nvfp4MatrixC), P, I32, I32, P, I32, P, SZ, P]),
    ("tf_lane_gemm_w4", ctypes.c_int, [ctypes.POINTER(W4MatrixC), P, I32, I32, P, I32, P, SZ, P]),
    ("tf_lane_gemm_w4_noalloc", ctypes.c_int, [ctypes.POINTER(W4MatrixC), P, I32, I32, P, I32, P, P]),
    ("tf_lane_gemm_w4_accumulate", ctypes.c_int, [ctypes.POINTER(W4MatrixC), P, I32, I32, P, I32, P, SZ, P]),
    ("tf_cast_bf16", ctypes.c_int, [P, I32, I32, I32, P, I32, P]),
    ("tf_keyed_sample_workspace_bytes", SZ, [I32, I32]),
    ("tf_keyed_sample", ctypes.c_int, [P, I32, I32, I32, ctypes.POINTER(SamplingC), ctypes.c_uint64, P, P, P, SZ, P]),
    ("tf_keyed_hash", ctypes.c_int, [P, P, P, ctypes.c_int64, P, P, P]),
    ("tf_lmhead_sample_workspace_bytes", SZ, [ctypes.POINTER(W4MatrixC), I32]),
    ("tf_lmhead_sample", ctypes.c_int, [ctypes.POINTER(W4MatrixC), P, I32, I32, ctypes.POINTER(SamplingC),
                                        ctypes.c_uint64, P, P, P, I32, P, P, P, P, SZ, P]),
    ("tf_accept", ctypes.c_int, [P, P, I32, P, P, P]),
    ("tf_gather_drafts", ctypes.c_int, [P, ctypes.c_int64, P, I32, P, P]),
    ("tf_commit_tokens", ctypes.c_int, [P, P, P, P, ctypes.c_int64, P]),
    ("tf_kv_append", ctypes.c_int, [ctypes.POINTER(KVCacheC), P, P, I32, I32, P, P, SZ, P]),
    ("tf_attention_workspace_bytes", SZ, [ctypes.POINTER(KVCacheC), I32, I32]),
    ("tf_attention_verify", ctypes.c_int, [ctypes.POINTER(KVCacheC), I32, P, I32, I32, P, P, I32, P, SZ, P]),
    ("tf_qk_norm_rope", ctypes.c_int, [P, I32, I32, I32, I32, I32, I32, I32, P, P, ctypes.c_float, P, I32, I32, P,
                                       ctypes.c_int64, P, I32, P]),
    ("tf_kv_store", ctypes.c_int, [ctypes.POINTER(KVBatchC), P, P, I32, I32, P, P, SZ, P]),
    ("tf_kv_load", ctypes.c_int, [ctypes.POINTER(KVBatchC), P, I32, P, P, I32, P, SZ, P]),
    ("tf_attention_batch_workspace_bytes", SZ, [ctypes.POINTER(KVBatchC), I32, I32, I32]),
    ("tf_attention_batch", ctypes.c_int, [ctypes.POINTER(KVBatchC), ctypes.POINTER(KVBatchC), I32, I32, P, I32, I32,
                                          P, P, I32, P, SZ, P]),
    ("tf_attention_prompt", ctypes.c_int, [P, I32, P, I32, P, I32, I32, I32, I32, P, I32, P, I32, P, SZ, P]),
    ("tf_attention_tree_workspace_bytes", SZ, [ctypes.POINTER(KVBatchC), I32, I32, I32]),
    ("tf_attention_tree", ctypes.c_int, [ctypes.POINTER(KVBatchC), ctypes.POINTER(KVBatchC), I32, I32, P, I32, I32,
                                         P, P, P, I32, P, SZ, P]),
    ("tf_tree_accept", ctypes.c_int, [P, P, P, P, I32, I32, P, P, P, P, P, SZ, P]),
    ("tf_kv_keep", ctypes.c_int, [ctypes.POINTER(KVBatchC), P, P, P, SZ, P]),
    ("tf_selfcheck_scratch_bytes", SZ, [I32]),
    ("tf_selfcheck_row_invariance", ctypes.c_int, [ctypes.POINTER(W4MatrixC), P, I32, P, SZ, P, SZ, P,
                                                   ctypes.POINTER(I32)]),
    ("tf_workspace_size", SZ, [I32, ctypes.POINTER(ctypes.c_int64), I32]),
    ("tf_moe_workspace_bytes", SZ, [ctypes.POINTER(MoeLayerC), I32]),
    ("tf_moe_w4", ctypes.c_int, [ctypes.POINTER(MoeLayerC), P, P, I32, P, P, SZ, P]),
    ("tf_verify_step_workspace_bytes", SZ, [ctypes.POINTER(ModelC), I32]),
    ("tf_embed_rows", ctypes.c_int, [ctypes.POINTER(ModelC), P, P, I32, P, P, P]),
    ("tf_rmsnorm_bf16", ctypes.c_int, [P, I32, I32, ctypes.c_float, P, P]),
    ("tf_decoder_block_workspace_bytes", SZ, [ctypes.POINTER(ModelC)]),
    ("tf_decoder_block", ctypes.c_int, [ctypes.POINTER(ModelC), I32, P, I32, P, P, P, SZ, P]),
    ("tf_verify_step", ctypes.c_int, [ctypes.POINTER(ModelC), I32, P, P, P, ctypes.POINTER(SamplingC),
                                      ctypes.c_uint64, P, P, P, P, SZ, P]),
]

_lib = None


def load(path: str = LIB_PATH):
    """Load libtf.so (built by ``w4_gemm_keyed_gb300.build``); raises if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(path):
            raise FileNotFoundError(f"{path} is missing: run __graft_entry__.build() first (no CPU fallback)")
        lib = ctypes.CDLL(path)
        for name, res, args in SIGNATURES:
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def _check(status: int):
    if status != TF_OK:
        raise TFError(status, load().tf_last_error().decode())


def _ptr(t):
    """Device address of a CUDA tensor (None passes NULL).  Every pointer the
    library takes is a device pointer: a host tensor, pinned or not, is refused
    here rather than handed to a kernel."""
    if t is None:
        return None
    if not t.is_cuda:
        raise TFError(TF_ERR_INVALID_ARG, f"expected a CUDA tensor, got one on {t.device}")
    return t.data_ptr()


def _current_raw_stream():
    return torch.cuda.current_stream().cuda_stream


try:  # cheaper lookup of the current stream's handle where this torch version has it
    _raw = torch._C._cuda_getCurrentRawStream

    def _current_raw_stream():  # noqa: F811
        return _raw(torch.cuda.current_device())
except AttributeError:  # pragma: no cover
    pass


def _stream(stream=None):
    return stream.cuda_stream if stream is not None else _current_raw_stream()


def workspace(nbytes: int, device="cuda", stream=None) -> torch.Tensor:
    """Zero-filled device scratch (the caching allocator aligns to >= 256 B), for calls on
    `stream` (default: the current one)."""
    if stream is None:
        return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    # filled, and handed out again once freed, in the order of the stream that uses it
    with torch.cuda.stream(stream):
        return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


_CLEARED_WHOLE = 32 << 20    # bytes that are as quickly cleared as allocated: 11 us, 14 with 256 of them; 64 MB 18, 560 MB 145


def _parts_workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """The workspace of one attention call over parts: such a call writes every result before it
    reads it, and only the status block, with its item counters, has to be zero."""
    if nbytes <= _CLEARED_WHOLE:
        return workspace(nbytes, device, stream)
    with torch.cuda.stream(stream):     # None: the current one
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        ws[:256].zero_()
    return ws


def _empty(shape, dtype, device, stream=None) -> torch.Tensor:
    """A call's own output: memory of the stream that the call runs on, so that nothing
    still queued elsewhere uses it, marked as used on the caller's stream too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _contiguous(stream, *tensors):
    """Contiguous tensors, what has to be copied copied on `stream`."""
    if stream is None:
        return [t.contiguous() for t in tensors]
    with torch.cuda.stream(stream):
        return [t.contiguous() for t in tensors]


def _status_block(device, stream=None) -> torch.Tensor:
    """The workspace of a call that returns it for its status alone."""
    ws = workspace(256, device, stream)
    if stream is not None:
        ws.record_stream(torch.cuda.current_stream(device))
    return ws


def workspace_status(ws: torch.Tensor, stream=None) -> int:
    code = I32(0)
    _check(load().tf_workspace_status(_ptr(ws), _stream(stream), ctypes.byref(code)))
    return int(code.value)


# ---------------------------------------------------------------- weights
class W4Matrix:
    """A packed W4 matrix living on the device."""

    def __init__(self, packed: torch.Tensor, K: int, N: int, group: int, gate_up: bool = False,
                 affine: bool = False):
        self.packed, self.K, self.N, self.group, self.gate_up, self.affine = packed, K, N, group, gate_up, affine
        self._c = W4MatrixC(packed.data_ptr(), K, N, group, int(affine))

    def c(self) -> W4MatrixC:
        return self._c


def packed_bytes(K: int, N: int, group: int) -> int:
    return int(load().tf_w4_packed_bytes(K, N, group))


def pack_w4(codes: torch.Tensor, scales: torch.Tensor, group: int, gate_up: bool = False,
            out: torch.Tensor = None, stream=None) -> W4Matrix:
    """codes uint8 [N][K/2] and scales fp16 (or int16/uint16 bits) [N][K/group], on the device."""
    lib = load()
    N, K2 = codes.shape
    K = 2 * K2
    nbytes = packed_bytes(K, N, group)
    if nbytes == 0:
        raise TFError(TF_ERR_UNSUPPORTED, f"unsupported shape K={K} N={N} group={group}")
    if out is None:
        out = _empty((nbytes,), torch.uint8, codes.device, stream)
    codes, scales = _contiguous(stream, codes, scales)
    if gate_up:
        _check(lib.tf_pack_w4_gate_up(_ptr(codes), _ptr(scales), K, N // 2, group, _ptr(out), nbytes, _stream(stream)))
    else:
        _check(lib.tf_pack_w4(_ptr(codes), _ptr(scales), K, N, group, _ptr(out), nbytes, _stream(stream)))
    return W4Matrix(out, K, N, group, gate_up)


def pack_w4_affine(codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor, group: int,
                   out: torch.Tensor = None, stream=None) -> W4Matrix:
    """MLX-style affine weights on the device: codes uint32 (or int32 bits) [N][K/8],
    scales and biases bf16 (or int16 bits) [N][K/group]."""
    lib = load()
    N, K8 = codes.shape
    K = 8 * K8
    nbytes = int(lib.tf_w4_affine_packed_bytes(K, N, group))
    if nbytes == 0:
        raise TFError(TF_ERR_UNSUPPORTED, f"unsupported shape K={K} N={N} group={group}")
    if out is None:
        out = _empty((nbytes,), torch.uint8, codes.device, stream)
    codes, scales, biases = _contiguous(stream, codes, scales, biases)
    _check(lib.tf_pack_w4_affine(_ptr(codes), _ptr(scales), _ptr(biases), K, N, group, _ptr(out), nbytes,
                                 _stream(stream)))
    return W4Matrix(out, K, N, group, affine=True)


# ---------------------------------------------------------------- linear
def lane_gemm_workspace_bytes(K: int, N: int, group: int) -> int:
    return int(load().tf_lane_gemm_workspace_bytes(K, N, group))


def _check_rows_in(x: torch.Tensor, K: int):
    """x: CUDA bf16 (or int16 bits) [R][>= K] with unit inner stride."""
    if x.dim() != 2 or x.dtype not in (torch.bfloat16, torch.int16):
        raise TFError(TF_ERR_INVALID_ARG, f"x must be a 2-D bf16 / int16 tensor, got {tuple(x.shape)} {x.dtype}")
    if x.stride(1) != 1 or x.shape[1] < K:
        raise TFError(TF_ERR_INVALID_ARG, f"x must have unit inner stride and >= {K} columns")


def _check_rows_out(y: torch.Tensor, R: int, N: int, device, dtype=torch.float32):
    """y: CUDA tensor of `dtype` [>= R][>= N] with unit inner stride on x's device."""
    if y.dim() != 2 or y.dtype != dtype:
        raise TFError(TF_ERR_INVALID_ARG, f"y must be a 2-D {dtype} tensor, got {tuple(y.shape)} {y.dtype}")
    if not y.is_cuda or y.device != device:
        raise TFError(TF_ERR_INVALID_ARG, f"y must be on {device}, got {y.device}")
    if y.shape[0] < R or y.shape[1] < N or y.stride(1) != 1:
        raise TFError(TF_ERR_INVALID_ARG, f"y must hold >= {R} rows of >= {N} columns with unit inner stride")


def lane_gemm_w4(W: W4Matrix, x: torch.Tensor, y: torch.Tensor = None, ws: torch.Tensor = None,
                 stream=None) -> torch.Tensor:
    """y[R][N] fp32 = W4 linear of bf16 rows x[R][K] (x may be bf16 or int16 bits)."""
    lib = load()
    _check_rows_in(x, W.K)
    R = x.shape[0]
    if y is None:
        y = _empty((R, W.N), torch.float32, x.device, stream)
    _check_rows_out(y, R, W.N, x.device)
    if ws is None:
        ws = workspace(lane_gemm_workspace_bytes(W.K, W.N, W.group), x.device, stream)
    wc = W.c()
    _check(lib.tf_lane_gemm_w4(ctypes.byref(wc), _ptr(x), x.stride(0), R, _ptr(y), y.stride(0), _ptr(ws),
                               ws.numel(), _stream(stream)))
    return y


def lane_gemm_w4_noalloc(W: W4Matrix, x: torch.Tensor, y: torch.Tensor, status: torch.Tensor = None,
                         stream=None) -> torch.Tensor:
    """lane_gemm_w4 on the library's built-in scratch: the call allocates no device
    memory, so the output y[R][N] fp32 must be given.  status: optional device int32
    (zeroed by the caller) that receives a device-side error code."""
    lib = load()
    _check_rows_in(x, W.K)
    R = x.shape[0]
    _check_rows_out(y, R, W.N, x.device)
    if status is not None and (status.dtype != torch.int32 or status.device != x.device or status.numel() < 1):
        raise TFError(TF_ERR_INVALID_ARG, "status must be a CUDA int32 tensor on x's device")
    wc = W.c()
    _check(lib.tf_lane_gemm_w4_noalloc(ctypes.byref(wc), _ptr(x), x.stride(0), R, _ptr(y), y.stride(0),
                                       _ptr(status), _stream(stream)))
    return y


# ---------------------------------------------------------------- NVFP4
class Nvfp4Matrix:
    """A packed NVFP4 matrix living on the device."""

    def __init__(self, packed: torch.Tensor, K: int, N: int, global_scale: float):
        self.packed, self.K, self.N, self.global_scale = packed, K, N, float(global_scale)
        self._c = Nvfp4MatrixC(packed.data_ptr(), K, N, float(global_scale))

    def c(self) -> Nvfp4MatrixC:
        return self._c


def nvfp4_packed_bytes(K: int, N: int) -> int:
    return int(load().tf_nvfp4_packed_bytes(K, N))


def pack_nvfp4(codes: torch.Tensor, scales: torch.Tensor, global_scale: float, out: torch.Tensor = None,
               stream=None) -> Nvfp4Matrix:
    """codes uint8 [N][K/2] (E2M1, low nibble first) and E4M3 scale bytes uint8 [N][K/16], on the device."""
    N, K2 = codes.shape
    K = 2 * K2
    nbytes = nvfp4_packed_bytes(K, N)
    if nbytes == 0:
        raise TFError(TF_ERR_UNSUPPORTED, f"unsupported shape K={K} N={N}")
    if tuple(scales.shape) != (N, K // 16) or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
        raise TFError(TF_ERR_INVALID_ARG, "codes must be uint8 [N][K/2] and scales uint8 [N][K/16]")
    if out is None:
        out = _empty((nbytes,), torch.uint8, codes.device, stream)
    codes, scales = _contiguous(stream, codes, scales)
    _check(load().tf_pack_nvfp4(_ptr(codes), _ptr(scales), K, N, _ptr(out), nbytes, _stream(stream)))
    return Nvfp4Matrix(out, K, N, global_scale)


def lane_gemm_nvfp4(W: Nvfp4Matrix, x: torch.Tensor, y: torch.Tensor = None, ws: torch.Tensor = None,
                    stream=None) -> torch.Tensor:
    """y[R][N] fp32 = NVFP4 linear of bf16 rows x[R][K] (x may be bf16 or int16 bits)."""
    lib = load()
    _check_rows_in(x, W.K)
    R = x.shape[0]
    if y is None:
        y = _empty((R, W.N), torch.float32, x.device, stream)
    _check_rows_out(y, R, W.N, x.device)
    if ws is None:
        ws = workspace(int(lib.tf_lane_gemm_nvfp4_workspace_bytes(W.K, W.N)), x.device, stream)
    _check(lib.tf_lane_gemm_nvfp4(ctypes.byref(W.c()), _ptr(x), x.stride(0), R, _ptr(y), y.stride(0), _ptr(ws),
                                  ws.numel(), _stream(stream)))
    return y


# ---------------------------------------------------------------- sampling
def lane_gemm_w4_accumulate(W: W4Matrix, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor = None,
                            stream=None) -> torch.Tensor:
    """y[R][N] (fp32, in place) += W4 linear of bf16 rows x[R][K]."""
    lib = load()
    if ws is None:
        ws = workspace(lane_gemm_workspace_bytes(W.K, W.N, W.group), x.device, stream)
    _check(lib.tf_lane_gemm_w4_accumulate(ctypes.byref(W.c()), _ptr(x), x.stride(0), x.shape[0], _ptr(y), y.stride(0),
                                          _ptr(ws), ws.numel(), _stream(stream)))
    return y


def cast_bf16(x: torch.Tensor, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """bf16 bits (int16 tensor) of the fp32 rows x [R][N], nearest-even."""
    R, N = x.shape
    if out is None:
        out = _empty((R, N), torch.int16, x.device, stream)
    _check(load().tf_cast_bf16(_ptr(x), R, N, x.stride(0), _ptr(out), out.stride(0), _stream(stream)))
    return out


def keyed_sample_workspace_bytes(R: int, V: int) -> int:
    return int(load().tf_keyed_sample_workspace_bytes(R, V))


def keyed_sample(logits: torch.Tensor, temperature: float, top_k: int, top_p: float, seed: int,
                 pos: torch.Tensor = None, tokens: torch.Tensor = None, ws: torch.Tensor = None,
                 stream=None) -> torch.Tensor:
    lib = load()
    R, V = logits.shape
    if tokens is None:
        tokens = _empty((R,), torch.int32, logits.device, stream)
    if ws is None:
        ws = workspace(keyed_sample_workspace_bytes(R, V), logits.device, stream)
    sp = SamplingC(temperature, top_k, top_p)
    _check(lib.tf_keyed_sample(_ptr(logits), logits.stride(0), R, V, ctypes.byref(sp), ctypes.c_uint64(seed & (2**64 - 1)),
                               _ptr(pos), _ptr(tokens), _ptr(ws), ws.numel(), _stream(stream)))
    return tokens


def lmhead_sample_workspace_bytes(W: W4Matrix, R: int) -> int:
    wc = W.c()
    return int(load().tf_lmhead_sample_workspace_bytes(ctypes.byref(wc), R))


def lmhead_sample(W: W4Matrix, x: torch.Tensor, temperature: float, top_k: int, top_p: float, seed: int,
                  pos: torch.Tensor = None, tokens: torch.Tensor = None, logits: torch.Tensor = None,
                  drafts: torch.Tensor = None, accepted: torch.Tensor = None, bonus: torch.Tensor = None,
                  ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """tokens[R] = keyed sample of the LM head's logits W x[R] in one call; logits
    (fp32 [R][>= N]) are also stored when given; with `accepted` (int32 [1]) the
    drafts are accepted against the tokens in the same call."""
    lib = load()
    _check_rows_in(x, W.K)
    R = x.shape[0]
    if tokens is None:
        tokens = _empty((R,), torch.int32, x.device, stream)
    if tokens.dtype != torch.int32 or tokens.numel() < R or not tokens.is_contiguous():
        raise TFError(TF_ERR_INVALID_ARG, "tokens must be a contiguous int32 tensor of >= R entries")
    if logits is not None:
        _check_rows_out(logits, R, W.N, x.device)
    if ws is None:
        ws = workspace(lmhead_sample_workspace_bytes(W, R), x.device, stream)
    wc = W.c()
    sp = SamplingC(temperature, top_k, top_p)
    _check(lib.tf_lmhead_sample(ctypes.byref(wc), _ptr(x), x.stride(0), R, ctypes.byref(sp),
                                ctypes.c_uint64(seed & (2**64 - 1)), _ptr(pos), _ptr(tokens), _ptr(logits),
                                logits.stride(0) if logits is not None else 0, _ptr(drafts), _ptr(accepted),
                                _ptr(bonus), _ptr(ws), ws.numel(), _stream(stream)))
    return tokens


def keyed_hash(seed: torch.Tensor, pos: torch.Tensor, token: torch.Tensor, stream=None):
    """(h uint64 bits as int64, g fp64) of the sampler's key and Gumbel noise for
    device triples seed (int64 holding uint64 bits), pos int64, token int32."""
    n = seed.numel()
    if pos.numel() != n or token.numel() != n:
        raise TFError(TF_ERR_INVALID_ARG, "seed, pos and token must have the same length")
    for t, dt in ((seed, torch.int64), (pos, torch.int64), (token, torch.int32)):
        if t.dtype != dt or not t.is_contiguous():
            raise TFError(TF_ERR_INVALID_ARG, f"expected a contiguous {dt} tensor, got {t.dtype}")
    h = _empty((n,), torch.int64, seed.device, stream)
    g = _empty((n,), torch.float64, seed.device, stream)
    _check(load().tf_keyed_hash(_ptr(seed), _ptr(pos), _ptr(token), n, _ptr(h), _ptr(g), _stream(stream)))
    return h, g


def accept(drafts: torch.Tensor, sampled: torch.Tensor, accepted: torch.Tensor = None,
           bonus: torch.Tensor = None, stream=None):
    lib = load()
    R = sampled.shape[0]
    dev = sampled.device
    if accepted is None:
        accepted = _empty((1,), torch.int32, dev, stream)
    if bonus is None:
        bonus = _empty((1,), torch.int32, dev, stream)
    _check(lib.tf_accept(_ptr(drafts) if R > 1 else None, _ptr(sampled), R, _ptr(accepted), _ptr(bonus),
                         _stream(stream)))
    return accepted, bonus


def gather_drafts(table: torch.Tensor, pos: torch.Tensor, R: int, drafts: torch.Tensor, stream=None):
    """drafts[i] = table[pos + i] for i < R - 1 (device int32 table, device int64 pos)."""
    _check(load().tf_gather_drafts(_ptr(table), table.numel(), _ptr(pos), R, _ptr(drafts), _stream(stream)))
    return drafts


def commit_tokens(tokens: torch.Tensor, accepted: torch.Tensor, pos: torch.Tensor, log: torch.Tensor, stream=None):
    """Write a finished pass's committed tokens into the device log (index = position - 1)."""
    _check(load().tf_commit_tokens(_ptr(tokens), _ptr(accepted), _ptr(pos), _ptr(log), log.numel(),
                                   _stream(stream)))
    return log


def selfcheck_row_invariance(W: W4Matrix, x: torch.Tensor, stream=None) -> int:
    """0 if every row of every R in 1..16 matches its one-row launch bit for bit,
    else R * 256 + row of the first mismatch.  x: bf16 [16][K] on the device."""
    lib = load()
    scratch = workspace(int(lib.tf_selfcheck_scratch_bytes(W.N)), x.device, stream)
    ws = workspace(lane_gemm_workspace_bytes(W.K, W.N, W.group), x.device, stream)
    res = I32(-1)
    _check(lib.tf_selfcheck_row_invariance(ctypes.byref(W.c()), _ptr(x), x.stride(0), _ptr(scratch), scratch.numel(),
                                           _ptr(ws), ws.numel(), _stream(stream), ctypes.byref(res)))
    return int(res.value)


def workspace_size(op: int, dims) -> int:
    arr = (ctypes.c_int64 * len(dims))(*[int(d) for d in dims])
    return int(load().tf_workspace_size(op, arr, len(dims)))


# ---------------------------------------------------------------- KV cache attention
class KVCache:
    """A KV cache on the device: k, v bf16 bits (int16) [n_kv][max_len][128] in the
    library's position-swizzled layout (tf.h), zero-filled at creation."""

    def __init__(self, n_kv: int, max_len: int, device="cuda"):
        self.k = torch.zeros((n_kv, max_len, HEAD_DIM), dtype=torch.int16, device=device)
        self.v = torch.zeros((n_kv, max_len, HEAD_DIM), dtype=torch.int16, device=device)
        self.n_kv, self.max_len = n_kv, max_len
        self._c = KVCacheC(self.k.data_ptr(), self.v.data_ptr(), n_kv, max_len)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor, ws: torch.Tensor = None,
               stream=None):
        """Entries at positions pos .. pos + R - 1 from k_new, v_new bf16 [R][n_kv*128]."""
        if ws is None:
            ws = _status_block(k_new.device, stream)
        R = k_new.shape[0]
        _check(load().tf_kv_append(ctypes.byref(self._c), _ptr(k_new), _ptr(v_new), k_new.stride(0), R, _ptr(pos),
                                   _ptr(ws), ws.numel(), _stream(stream)))
        return ws

    def workspace_bytes(self, group: int, R: int) -> int:
        return int(load().tf_attention_workspace_bytes(ctypes.byref(self._c), group, R))

    def attention(self, q: torch.Tensor, group: int, pos: torch.Tensor, out: torch.Tensor = None,
                  ws: torch.Tensor = None, stream=None) -> torch.Tensor:
        """fp32 [R][n_q*128]: rows at positions pos + r attending over entries 0..pos + r."""
        R = q.shape[0]
        n_q = self.n_kv * group
        if out is None:
            out = _empty((R, n_q * HEAD_DIM), torch.float32, q.device, stream)
        if ws is None:
            ws = workspace(self.workspace_bytes(group, R), q.device, stream)
        _check(load().tf_attention_verify(ctypes.byref(self._c), group, _ptr(q), q.stride(0), R, _ptr(pos), _ptr(out),
                                          out.stride(0), _ptr(ws), ws.numel(), _stream(stream)))
        return out


# ---------------------------------------------------------------- a batch of sequences that continue one prompt
# These calls are as short as the kernels they launch, so each tensor is looked at
# once, in few Python operations, and messages are made only on refusal.
_BITS16 = (torch.bfloat16, torch.int16)


def _refuse(message: str):
    raise TFError(TF_ERR_INVALID_ARG, message)


def _bits16(t: torch.Tensor, name: str, rows: int, cols: int, device) -> int:
    """Row stride of t: bf16 (or int16 bits) [>= rows][>= cols] with unit inner stride on `device`."""
    shape = t.shape
    ld, unit = t.stride() if len(shape) == 2 else (0, 0)
    if unit != 1 or t.dtype not in _BITS16 or shape[0] < rows or shape[1] < cols or t.device != device:
        _refuse(f"{name} must be a bf16 / int16 [>= {rows}][>= {cols}] tensor with unit inner stride on {device}, "
                f"got {tuple(shape)} {t.dtype} on {t.device}")
    return ld


def _positions(pos: torch.Tensor, device) -> int:
    if pos.dtype is not torch.int64 or pos.stride() != (1,) or pos.device != device or not pos.numel():
        _refuse(f"pos must be a contiguous 1-D int64 tensor on {device}, one per sequence")
    return pos.numel()


def _bytes(ws: torch.Tensor, device) -> int:
    if ws.device != device:
        _refuse(f"ws must be on {device}, got one on {ws.device}")
    return ws.numel()


def rope_turns(rot_dim: int, theta: float = 10000.0, inv_freq=None, device="cuda") -> torch.Tensor:
    """Frequencies of a rotation over rot_dim elements for qk_norm_rope: int64 bits of
    round(2^64 f / 2 pi) per pair, f = theta^(-2d/rot_dim) radians per position, or
    inv_freq[d] (scaled variants bring their own)."""
    if rot_dim % 8 or not 0 < rot_dim <= HEAD_DIM:
        raise TFError(TF_ERR_UNSUPPORTED, f"rot_dim={rot_dim} is not a multiple of 8 in [8, {HEAD_DIM}]")
    if inv_freq is None:
        inv_freq = [theta ** (-2.0 * d / rot_dim) for d in range(rot_dim // 2)]
    inv_freq = [float(f) for f in inv_freq]
    if len(inv_freq) != rot_dim // 2 or not all(math.isfinite(f) for f in inv_freq):
        raise TFError(TF_ERR_INVALID_ARG, f"inv_freq must hold {rot_dim // 2} finite frequencies")
    # 2 pi to 80 digits keeps the quotient's error at the frequency's own rounding
    units = [round(Fraction(f) / _TWO_PI * 2 ** 64) % 2 ** 64 for f in inv_freq]
    return torch.tensor([u - 2 ** 64 if u >= 2 ** 63 else u for u in units], dtype=torch.int64, device=device)


def qk_norm_rope(x: torch.Tensor, n_q: int, n_kv: int, pos: torch.Tensor, turns: torch.Tensor = None,
                 q_weight: torch.Tensor = None, k_weight: torch.Tensor = None, eps: float = 1e-6,
                 adjacent: bool = False, pos_offset: int = 0, n_v: int = None, out: torch.Tensor = None,
                 stream=None) -> torch.Tensor:
    """bf16 [rows][(n_q + n_kv + n_v) * 128]: the query and key heads of the projection
    rows x (fp32, or bf16 / int16 bits) normalised (where weights are given) and turned
    by their positions (where turns are), the n_v (default n_kv) value heads rounded.
    Rows are sequence-major, len(rows) / len(pos) per sequence; row r of sequence b
    turns by position pos[b] + pos_offset + r."""
    n_v = n_kv if n_v is None else n_v
    cols = (n_q + n_kv + n_v) * HEAD_DIM
    dev, shape = x.device, x.shape
    fp32 = x.dtype is torch.float32
    ldx, unit = x.stride() if len(shape) == 2 else (0, 0)
    if unit != 1 or not (fp32 or x.dtype in _BITS16) or shape[1] < cols or not x.is_cuda:
        _refuse(f"x must be a CUDA fp32 or bf16 / int16 [rows][>= {cols}] tensor with unit inner stride, got "
                f"{tuple(shape)} {x.dtype} on {dev}")
    B, rows = _positions(pos, dev), shape[0]
    if rows % B or not rows:
        _refuse(f"{rows} rows are not a positive multiple of {B} sequences")
    wq = wk = turned = None
    rot = 0
    if q_weight is not None:
        wq = _head_weight(q_weight, "q_weight", dev)
    if k_weight is not None:
        wk = _head_weight(k_weight, "k_weight", dev)
    if turns is not None:
        if turns.dtype is not torch.int64 or turns.stride() != (1,) or turns.device != dev:
            _refuse(f"turns must be a contiguous 1-D int64 tensor on {dev}")
        rot, turned = 2 * turns.numel(), turns.data_ptr()
    if out is None:
        out, ldo = _empty((rows, cols), torch.bfloat16, dev, stream), cols
    else:
        ldo = _bits16(out, "out", rows, cols, dev)
    st = load().tf_qk_norm_rope(x.data_ptr(), fp32, ldx, B, rows // B, n_q, n_kv, n_v, wq, wk, eps, turned, rot,
                                adjacent, pos.data_ptr(), pos_offset, out.data_ptr(), ldo, _stream(stream))
    if st:
        _check(st)
    return out


def _head_weight(w: torch.Tensor, name: str, device) -> int:
    if w.dtype not in _BITS16 or w.numel() != HEAD_DIM or w.stride() != (1,) or w.device != device:
        _refuse(f"{name} must be {HEAD_DIM} contiguous bf16 values on {device}")
    return w.data_ptr()


class KVBatch:
    """KV caches of n_seq sequences on the device, entries bf16 or E4M3 codes with
    one power-of-two scale per 128-element vector (layouts in tf.h)."""

    def __init__(self, n_seq: int, n_kv: int, max_len: int, fmt: str = "bf16", device="cuda"):
        if fmt not in KV_FORMATS:
            raise TFError(TF_ERR_UNSUPPORTED, f"fmt must be one of {sorted(KV_FORMATS)}, got {fmt!r}")
        shape = (n_seq, n_kv, max_len, HEAD_DIM)
        dtype = torch.int16 if fmt == "bf16" else torch.uint8
        self.k, self.v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        self.k_scale = self.v_scale = None
        if fmt == "e4m3":
            self.k_scale, self.v_scale = (torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in range(2))
        self.n_seq, self.n_kv, self.max_len, self.fmt = n_seq, n_kv, max_len, fmt
        self._bind()

    def _bind(self):
        self.device = self.k.device
        self._c = KVBatchC(_ptr(self.k), _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale), self.n_seq, self.n_kv,
                           self.max_len, KV_FORMATS[self.fmt])

    @classmethod
    def of(cls, cache: KVCache) -> "KVBatch":
        """A batch of one sequence over the memory of an existing KVCache.  Its attention
        returns bf16 and rounds the softmax weights to bf16; KVCache.attention returns fp32
        and keeps about 16 bits of them."""
        b = cls.__new__(cls)
        b.k, b.v, b.k_scale, b.v_scale = cache.k[None], cache.v[None], None, None
        b.n_seq, b.n_kv, b.max_len, b.fmt = 1, cache.n_kv, cache.max_len, "bf16"
        b._bind()
        return b

    def _rows(self, n: int) -> int:
        if not n or not self.n_seq or n % self.n_seq:
            _refuse(f"{n} rows are not a positive multiple of {self.n_seq} sequences")
        return n // self.n_seq

    def _pos(self, pos: torch.Tensor) -> int:
        if _positions(pos, self.device) != self.n_seq:
            _refuse(f"pos must hold {self.n_seq} positions")
        return pos.data_ptr()

    def store(self, k_new: torch.Tensor, v_new: torch.Tensor, pos: torch.Tensor, ws: torch.Tensor = None, stream=None):
        """Entries pos[b] + r of sequence b from rows b*R + r of k_new, v_new (bf16
        [n_seq*R][n_kv*128]); returns the workspace whose status the call sets."""
        cols, dev = self.n_kv * HEAD_DIM, self.device
        ld = _bits16(k_new, "k_new", 1, cols, dev)
        n = k_new.shape[0]
        if _bits16(v_new, "v_new", 1, cols, dev) != ld or v_new.shape[0] != n:
            _refuse("k_new and v_new must have the same rows and row stride")
        R, at = self._rows(n), self._pos(pos)
        if ws is None:
            ws = _status_block(dev, stream)
        st = load().tf_kv_store(self._c, k_new.data_ptr(), v_new.data_ptr(), ld, R, at, _ptr(ws), _bytes(ws, dev),
                                _stream(stream))
        if st:
            _check(st)
        return ws

    def load(self, pos: torch.Tensor, R: int, k: torch.Tensor = None, v: torch.Tensor = None,
             ws: torch.Tensor = None, stream=None):
        """(k, v) bf16 [n_seq*R][n_kv*128]: the values of entries pos[b] + r."""
        n, cols, dev = self.n_seq * R, self.n_kv * HEAD_DIM, self.device
        at = self._pos(pos)
        if not 0 < R <= self.max_len:
            _refuse(f"R={R} outside [1, max_len={self.max_len}]")
        if k is None and v is None:
            k, ld = _empty((n, cols), torch.bfloat16, dev, stream), cols
            v = _empty((n, cols), torch.bfloat16, dev, stream)
        else:
            ld = _bits16(v if k is None else k, "v" if k is None else "k", n, cols, dev)
            if k is None:
                k = _empty((v.shape[0], ld), v.dtype, dev, stream)[:, :v.shape[1]]
            elif v is None:
                v = _empty((k.shape[0], ld), k.dtype, dev, stream)[:, :k.shape[1]]
            elif _bits16(v, "v", n, cols, dev) != ld:
                _refuse("k and v must have the same row stride")
        if ws is None:
            ws = workspace(256, dev, stream)
        st = load().tf_kv_load(self._c, at, R, k.data_ptr(), v.data_ptr(), ld, _ptr(ws), _bytes(ws, dev),
                               _stream(stream))
        if st:
            _check(st)
        return k, v

    def attention_workspace_bytes(self, group: int, R: int, prefix_len: int = 0) -> int:
        return int(load().tf_attention_batch_workspace_bytes(self._c, group, R, prefix_len))

    def attention(self, q: torch.Tensor, group: int, pos: torch.Tensor, prefix: "KVBatch" = None,
                  prefix_len: int = 0, out: torch.Tensor = None, ws: torch.Tensor = None, stream=None) -> torch.Tensor:
        """bf16 [n_seq*R][n_kv*group*128]: rows at own positions pos[b] + r attending over
        entries 0..prefix_len-1 of the one-sequence batch `prefix` and 0..pos[b]+r of
        their own; idle sequences' rows are zeros."""
        if group < 1:
            raise TFError(TF_ERR_UNSUPPORTED, f"group={group} outside [1, 16]")
        cols, dev = self.n_kv * group * HEAD_DIM, self.device
        ldq = _bits16(q, "q", 1, cols, dev)
        n = q.shape[0]
        R, at = self._rows(n), self._pos(pos)
        if prefix is not None and prefix.device != dev:
            _refuse(f"prefix must be on {dev}, got one on {prefix.device}")
        if out is None:
            out, ldo = _empty((n, cols), torch.bfloat16, dev, stream), cols
        else:
            ldo = _bits16(out, "out", n, cols, dev)
        if ws is None:
            ws = _parts_workspace(self.attention_workspace_bytes(group, R, prefix_len), dev, stream)
        st = load().tf_attention_batch(self._c, prefix._c if prefix is not None else None, prefix_len, group,
                                       q.data_ptr(), ldq, R, at, out.data_ptr(), ldo, _ptr(ws), _bytes(ws, dev),
                                       _stream(stream))
        if st:
            _check(st)
        return out


    def tree_attention_workspace_bytes(self, group: int, n: int, prefix_len: int = 0) -> int:
        return int(load().tf_attention_tree_workspace_bytes(self._c, group, n, prefix_len))

    def tree_attention(self, q: torch.Tensor, group: int, pos: torch.Tensor, parents: torch.Tensor,
                       prefix: "KVBatch" = None, prefix_len: int = 0, out: torch.Tensor = None,
                       ws: torch.Tensor = None, stream=None) -> torch.Tensor:
        """bf16 [n_seq*n][n_kv*group*128]: node i of sequence b's tree (parents int32 [n_seq][n],
        -1 for the root, node 0, and for unused rows; entry pos[b] + i stored) attending over entries
        0..prefix_len-1 of `prefix`, own entries 0..pos[b]-1 and its path's; rows of
        idle sequences and unused rows are zeros.  A node's bits are those of its path decoded one
        token a pass by this call, not by `attention`, which adds up in another order: a run
        uses one of them throughout.  `out` does not overlap `q`."""
        if group < 1:
            raise TFError(TF_ERR_UNSUPPORTED, f"group={group} outside [1, 16]")
        cols, dev = self.n_kv * group * HEAD_DIM, self.device
        ldq = _bits16(q, "q", 1, cols, dev)
        rows, at = q.shape[0], self._pos(pos)
        n = self._rows(rows)
        tree = _int32(parents, "parents", (self.n_seq, n), dev)
        if prefix is not None and prefix.device != dev:
            _refuse(f"prefix must be on {dev}, got one on {prefix.device}")
        if out is None:
            out, ldo = _empty((rows, cols), torch.bfloat16, dev, stream), cols
        else:
            ldo = _bits16(out, "out", rows, cols, dev)
        if ws is None:
            ws = _parts_workspace(self.tree_attention_workspace_bytes(group, n, prefix_len), dev, stream)
        st = load().tf_attention_tree(self._c, prefix._c if prefix is not None else None, prefix_len, group,
                                      q.data_ptr(), ldq, n, at, tree, out.data_ptr(), ldo, _ptr(ws), _bytes(ws, dev),
                                      _stream(stream))
        if st:
            _check(st)
        return out

    def keep(self, pos: torch.Tensor, path: torch.Tensor, ws: torch.Tensor = None, stream=None):
        """Entry pos[b] + path[b][d] becomes entry pos[b] + d, for every depth of the accepted
        paths (int32 [n_seq][MAX_PATH], -1 past their ends: ``tree_accept``'s); returns the
        workspace whose status the call sets."""
        dev, at = self.device, self._pos(pos)
        way = _int32(path, "path", (self.n_seq, MAX_PATH), dev)
        if ws is None:
            ws = _status_block(dev, stream)
        st = load().tf_kv_keep(self._c, at, way, _ptr(ws), _bytes(ws, dev), _stream(stream))
        if st:
            _check(st)
        return ws


def _int32(t: torch.Tensor, name: str, shape: tuple, device) -> int:
    if t.dtype is not torch.int32 or t.shape != shape or t.device != device or not t.is_contiguous():
        _refuse(f"{name} must be a contiguous int32 {list(shape)} tensor on {device}, got {tuple(t.shape)} {t.dtype} on "
                f"{t.device}")
    return t.data_ptr()


def tree_accept(parents: torch.Tensor, tokens: torch.Tensor, sampled: torch.Tensor, pos: torch.Tensor,
                ws: torch.Tensor = None, stream=None):
    """(accepted [n_seq], bonus [n_seq], path [n_seq][MAX_PATH], committed [n_seq][MAX_PATH]), int32: the walk
    down each sequence's tree (parents, drafted tokens and the token sampled after each
    node, int32 [n_seq][n]) to the lowest-numbered child that holds the sampled token;
    -1 past a path's end and for idle sequences (pos[b] = -1)."""
    dev, shape = parents.device, parents.shape
    if not parents.is_cuda or len(shape) != 2:
        _refuse(f"parents must be a CUDA [n_seq][n] tensor, got {tuple(shape)} on {dev}")
    B, n = shape
    tree = _int32(parents, "parents", shape, dev)
    drafted, drawn = _int32(tokens, "tokens", shape, dev), _int32(sampled, "sampled", shape, dev)
    if _positions(pos, dev) != B:
        _refuse(f"pos must hold {B} positions")
    if ws is None:
        ws = workspace(256, dev, stream)
    # four calls of one path: views of one allocation took 2 us longer
    accepted = _empty((B,), torch.int32, dev, stream)
    bonus = _empty((B,), torch.int32, dev, stream)
    path = _empty((B, MAX_PATH), torch.int32, dev, stream)
    committed = _empty((B, MAX_PATH), torch.int32, dev, stream)
    st = load().tf_tree_accept(tree, drafted, drawn, pos.data_ptr(), B, n, accepted.data_ptr(), bonus.data_ptr(),
                               path.data_ptr(), committed.data_ptr(), _ptr(ws), _bytes(ws, dev), _stream(stream))
    if st:
        _check(st)
    return accepted, bonus, path, committed


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, n_kv: int, group: int, starts: torch.Tensor,
                     out: torch.Tensor = None, ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    """bf16 [rows][n_kv*group*128]: causal attention of whole prompts.  Sequence s holds rows
    starts[s] .. starts[s+1]-1 (int64 [n_seq + 1], on the device) of q [rows][n_kv*group*128]
    and of k and v [rows][n_kv*128] (bf16 / int16 bits, any row stride that is a multiple of 8:
    columns of one projection, say); rows outside every sequence are not written.  `out` overlaps
    none of the inputs.  A prompt read in passes of `KVBatch.attention` rounds otherwise: runs whose
    tokens have to agree read their prompts the same way."""
    if group < 1 or n_kv < 1:
        raise TFError(TF_ERR_UNSUPPORTED, f"n_kv={n_kv}, group={group} must be >= 1")
    dev, cols = q.device, n_kv * group * HEAD_DIM
    if not q.is_cuda:
        _refuse(f"q must be a CUDA tensor, got one on {dev}")
    ldq = _bits16(q, "q", 0, cols, dev)
    rows = q.shape[0]
    ldk, ldv = _bits16(k, "k", rows, n_kv * HEAD_DIM, dev), _bits16(v, "v", rows, n_kv * HEAD_DIM, dev)
    n = _positions(starts, dev) - 1
    if out is None:
        out, ldo = _empty((rows, cols), torch.bfloat16, dev, stream), cols
    else:
        ldo = _bits16(out, "out", rows, cols, dev)
    if ws is None:
        ws = workspace(256, dev, stream)
    st = load().tf_attention_prompt(q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, rows, n_kv, group,
                                    starts.data_ptr(), n, out.data_ptr(), ldo, _ptr(ws), _bytes(ws, dev),
                                    _stream(stream))
    if st:
        _check(st)
    return out


def rmsnorm_bf16(x: torch.Tensor, eps: float, out: torch.Tensor = None, stream=None) -> torch.Tensor:
    """bf16 bits (int16 tensor) of x / sqrt(mean(x^2) + eps), per row of fp32 x [R][H]."""
    R, H = x.shape
    if out is None:
        out = _empty((R, H), torch.int16, x.device, stream)
    _check(load().tf_rmsnorm_bf16(_ptr(x), R, H, eps, _ptr(out), _stream(stream)))
    return out


# ---------------------------------------------------------------- MoE
class MoeLayer:
    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor, hidden: int, ffn: int, n_experts: int,
                 top_k: int, group: int):
        self.gate_up, self.down = gate_up, down
        self.hidden, self.ffn, self.n_experts, self.top_k, self.group = hidden, ffn, n_experts, top_k, group

    def c(self) -> MoeLayerC:
        return MoeLayerC(self.gate_up.data_ptr(), self.down.data_ptr(), self.hidden, self.ffn, self.n_experts,
                         self.top_k, self.group)


def moe_workspace_bytes(layer: MoeLayer, R: int) -> int:
    lc = layer.c()
    return int(load().tf_moe_workspace_bytes(ctypes.byref(lc), R))


def moe_w4(layer: MoeLayer, x: torch.Tensor, router: torch.Tensor, out: torch.Tensor = None,
           ws: torch.Tensor = None, stream=None) -> torch.Tensor:
    lib = load()
    R = x.shape[0]
    if out is None:
        out = _empty((R, layer.hidden), torch.float32, x.device, stream)
    if ws is None:
        ws = workspace(moe_workspace_bytes(layer, R), x.device, stream)
    lc = layer.c()
    _check(lib.tf_moe_w4(ctypes.byref(lc), _ptr(x), _ptr(router), R, _ptr(out), _ptr(ws), ws.numel(),
                         _stream(stream)))
    return out


# ---------------------------------------------------------------- synthetic decoder
class Model:
    """Device weights of the attention-free synthetic decoder."""

    def __init__(self, embedding: torch.Tensor, gate_up, down, lm_head: W4Matrix, vocab: int, hidden: int,
                 ffn: int, group: int, rms_eps: float = 1e-6):
        self.embedding, self.gate_up, self.down, self.lm_head = embedding, list(gate_up), list(down), lm_head
        self.vocab, self.hidden, self.ffn, self.group, self.rms_eps = vocab, hidden, ffn, group, rms_eps
        n = len(self.gate_up)
        self._gu = (W4MatrixC * max(n, 1))(*[m.c() for m in self.gate_up])
        self._dn = (W4MatrixC * max(n, 1))(*[m.c() for m in self.down])
        self._c = ModelC(vocab, hidden, ffn, n, group, rms_eps, embedding.data_ptr(), self._gu, self._dn,
                         lm_head.c())

    def workspace_bytes(self, R: int) -> int:
        return int(load().tf_verify_step_workspace_bytes(ctypes.byref(self._c), R))

    def embed_rows(self, last_token, drafts, R: int, x: torch.Tensor, ws: torch.Tensor, stream=None):
        _check(load().tf_embed_rows(ctypes.byref(self._c), _ptr(last_token), _ptr(drafts) if R > 1 else None, R,
                                    _ptr(x), _ptr(ws), _stream(stream)))

    def block_workspace_bytes(self) -> int:
        return int(load().tf_decoder_block_workspace_bytes(ctypes.byref(self._c)))

    def block(self, b: int, x: torch.Tensor, n_out: torch.Tensor, h_out: torch.Tensor, ws: torch.Tensor,
              stream=None):
        """In place on the fp32 residual x [R][hidden]; n_out/h_out receive the bf16 intermediates."""
        _check(load().tf_decoder_block(ctypes.byref(self._c), b, _ptr(x), x.shape[0], _ptr(n_out), _ptr(h_out),
                                       _ptr(ws), ws.numel(), _stream(stream)))

    def verify_step(self, R: int, last_token: torch.Tensor, pos: torch.Tensor, drafts: torch.Tensor,
                    temperature: float, top_k: int, top_p: float, seed: int, tokens: torch.Tensor,
                    accepted: torch.Tensor, ws: torch.Tensor, logits: torch.Tensor = None, stream=None):
        sp = SamplingC(temperature, top_k, top_p)
        _check(load().tf_verify_step(ctypes.byref(self._c), R, _ptr(last_token), _ptr(pos),
                                     _ptr(drafts) if R > 1 else None, ctypes.byref(sp),
                                     ctypes.c_uint64(seed & (2**64 - 1)), _ptr(tokens), _ptr(accepted),
                                     _ptr(logits), _ptr(ws), ws.numel(), _stream(stream)))
