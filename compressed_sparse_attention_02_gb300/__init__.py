"""Python binding of libcsa, the GB300 (sm_103a) CSA layer hot path.

Argument marshalling only: every function below forwards to the C entry point
of the same name in ``libcsa.so`` (declared in ``include/csa.h``), passing
device pointers (``tensor.data_ptr()``), sizes, and the current CUDA stream.
All computation runs in the library's CUDA kernels; there is no fallback, and
importing this package fails if the library has not been built
(``python compressed_sparse_attention_02_gb300/build.py``).

Tensor conventions: bf16 tensors are ``torch.bfloat16``, FP8 E4M3 tensors are
``torch.float8_e4m3fn`` (or uint8 holding the same bits), positions and
indices ``torch.int32``, the sink ``torch.float32``; every tensor is
contiguous and on the current CUDA device.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libcsa.so")

if not os.path.exists(LIBRARY_PATH):
    raise ImportError(
        "libcsa.so is not built (expected at %s); run python compressed_sparse_attention_02_gb300/build.py"
        % LIBRARY_PATH)

_lib = ctypes.CDLL(LIBRARY_PATH)

CSA_OK = 0
STATUS_NAMES = {0: "CSA_OK", 1: "CSA_ERR_INVALID_ARG", 2: "CSA_ERR_UNSUPPORTED", 3: "CSA_ERR_CUDA",
                4: "CSA_ERR_TIMEOUT", 5: "CSA_ERR_INDEX_RANGE", 6: "CSA_ERR_WORKSPACE"}
(CSA_OP_COMPRESS, CSA_OP_INDEX_TOPK, CSA_OP_SPARSE_ATTN, CSA_OP_LAYER_DECODE, CSA_OP_LAYER_PREFILL,
 CSA_OP_INDEX_TOPK_POOL, CSA_OP_REINDEX_TOPK, CSA_OP_HCA_LAYER_DECODE) = range(8)
CSA_POOL_BLOCK = 8
CSA_FP4_ENTRY_BYTES = 288


class CsaParams(ctypes.Structure):
    """Mirror of ``csa_params``."""
    _fields_ = [("m", ctypes.c_int32), ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("idx_heads", ctypes.c_int32), ("idx_dim", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("swa_window", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("sm_scale", ctypes.c_float), ("inverse_rope", ctypes.c_int32),
                ("kv_format", ctypes.c_int32), ("bf16_scores", ctypes.c_int32), ("index_format", ctypes.c_int32)]


class CsaIndexKeySrc(ctypes.Structure):
    """Mirror of ``csa_index_key_src`` (device pointers)."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("CIa", "ZIa", "CIb", "ZIb", "CIb_prev", "ZIb_prev", "BIa", "BIb",
                                                "rms_wI")]


def index_key_src(CIa, ZIa, CIb, ZIb, BIa, BIb, rms_wI, CIb_prev=None, ZIb_prev=None) -> CsaIndexKeySrc:
    """A ``csa_index_key_src`` over device tensors (which the caller keeps alive)."""
    return CsaIndexKeySrc(*[None if t is None else t.data_ptr()
                            for t in (CIa, ZIa, CIb, ZIb, CIb_prev, ZIb_prev, BIa, BIb, rms_wI)])


class CsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s returned %s: %s" % (where, STATUS_NAMES.get(status, status),
                                                  csa_status_string(status)))


_vp = ctypes.c_void_p
_i32, _i64, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_P = ctypes.POINTER(CsaParams)

_lib.csa_default_params.argtypes = [_P]
_lib.csa_default_params.restype = None
_lib.csa_workspace_size.argtypes = [_i32, _P, _i32, _i32, _i64]
_lib.csa_workspace_size.restype = _sz
_lib.csa_compress.argtypes = [_P, _i32, _i32, _i64] + [_vp] * 9 + [_vp, _i64, _vp]
_lib.csa_compress_indexer_keys.argtypes = [_P, _i32, _i32, _i64] + [_vp] * 9 + [_vp, _i64, _vp]
_lib.csa_index_topk.argtypes = [_P, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _sz, _vp]
_lib.csa_index_topk_static.argtypes = [_P, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp]
_lib.csa_index_topk_static.restype = ctypes.c_int
_lib.csa_compress_single.argtypes = [_P, _i32, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
_lib.csa_compress_single.restype = ctypes.c_int
_lib.csa_compress_single_step.argtypes = [_P, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp]
_lib.csa_compress_single_step.restype = ctypes.c_int
_lib.csa_hca_layer_decode.argtypes = [_P, _i32] + [_vp] * 6 + [_vp, _i64] + [_vp] * 5 + [_vp, _sz, _vp]
_lib.csa_hca_layer_decode.restype = ctypes.c_int
_lib.csa_quantize_kv_fp4.argtypes = [_i64, _vp, _i64, _vp, _i64, _vp]
_lib.csa_quantize_kv_fp4.restype = ctypes.c_int
_lib.csa_quantize_index_keys_fp4.argtypes = [_i32, _i32, _i64, _vp, _i64, _vp, _i64, _vp]
_lib.csa_quantize_index_keys_fp4.restype = ctypes.c_int
_lib.csa_quantize_index_query_fp4.argtypes = [_i64, _vp, _vp, _vp]
_lib.csa_quantize_index_query_fp4.restype = ctypes.c_int
_lib.csa_index_topk_pool.argtypes = [_P, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _vp, _i32, _vp, _vp, _sz, _vp]
_lib.csa_index_topk_pool.restype = ctypes.c_int
_lib.csa_reindex_topk.argtypes = [_P, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _sz, _vp]
_lib.csa_reindex_topk.restype = ctypes.c_int
_lib.csa_sparse_attn.argtypes = [_P, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp,
                                 _vp, _sz, _vp]
_lib.csa_layer_decode.argtypes = [_P, _i32, _vp] + [_vp] * 7 + [_vp, _i64] + [_vp] * 9 + [_vp, _sz, _vp]
_lib.csa_layer_decode_append.argtypes = [_P, _i32, _vp] + [_vp] * 9 + [_vp, _i64] + [_vp] * 9 + [_vp, _sz, _vp]
_lib.csa_layer_prefill.argtypes = [_P, _i32, _i32, _i64] + [_vp] * 9 + [_vp, _i64] + [_vp] * 9 + [_vp, _sz, _vp]
_K = ctypes.POINTER(CsaIndexKeySrc)
_lib.csa_layer_decode_with_keys.argtypes = ([_P, _i32, _vp, _vp, _K] + [_vp] * 7 + [_vp, _i64] + [_vp] * 9 +
                                            [_vp, _sz, _vp])
_lib.csa_layer_prefill_with_keys.argtypes = ([_P, _i32, _i32, _i64] + [_vp] * 9 + [_K, _vp, _i64] + [_vp] * 9 +
                                             [_vp, _sz, _vp])
for _f in ("csa_compress", "csa_compress_indexer_keys", "csa_index_topk", "csa_sparse_attn", "csa_layer_decode",
           "csa_layer_decode_append", "csa_layer_prefill", "csa_layer_decode_with_keys",
           "csa_layer_prefill_with_keys"):
    getattr(_lib, _f).restype = ctypes.c_int
_lib.csa_set_trace_events.argtypes = [ctypes.POINTER(_vp), _i32]
_lib.csa_set_trace_events.restype = ctypes.c_int
_lib.csa_launch_count.argtypes = []
_lib.csa_launch_count.restype = ctypes.c_uint64
_lib.csa_check_status.argtypes = [_vp]
_lib.csa_check_status.restype = ctypes.c_int
_lib.csa_status_string.argtypes = [ctypes.c_int]
_lib.csa_status_string.restype = ctypes.c_char_p


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without building a torch.cuda.Stream (0.1 us
# instead of 2.9 us a call), where this torch has the call for it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream=None, device=None):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(status: int, where: str):
    if status != CSA_OK:
        raise CsaError(status, where)


def csa_default_params(**overrides) -> CsaParams:
    """The V4-Flash CSA parameters (m=4, 64x512 heads, top-k 512, window 128,
    theta 1e4, eps 1e-6, scale 1/sqrt(512)), with any field overridden."""
    p = CsaParams()
    _lib.csa_default_params(ctypes.byref(p))
    for k, v in overrides.items():
        setattr(p, k, v)
    return p


def csa_status_string(status: int) -> str:
    return _lib.csa_status_string(int(status)).decode()


def csa_workspace_size(op: int, params: CsaParams, B: int, Q: int, n_cap: int) -> int:
    return int(_lib.csa_workspace_size(op, ctypes.byref(params), B, Q, n_cap))


def workspace(op: int, params: CsaParams, B: int, Q: int, n_cap: int, device=None) -> torch.Tensor:
    """Allocates (through torch) a workspace of csa_workspace_size() bytes."""
    n = csa_workspace_size(op, params, B, Q, n_cap)
    if n == 0:
        raise CsaError(2, "csa_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def csa_compress(params, B, n_new, entry0, Ca, Za, Cb, Zb, Cb_prev, Zb_prev, Ba, Bb, rms_w, kv_out, kv_stride_b,
                 stream=None):
    _check(_lib.csa_compress(ctypes.byref(params), B, n_new, entry0, _ptr(Ca), _ptr(Za), _ptr(Cb), _ptr(Zb),
                             _ptr(Cb_prev), _ptr(Zb_prev), _ptr(Ba), _ptr(Bb), _ptr(rms_w), _ptr(kv_out),
                             kv_stride_b, _stream(stream)), "csa_compress")


def csa_compress_indexer_keys(params, B, n_new, entry0, CIa, ZIa, CIb, ZIb, CIb_prev, ZIb_prev, BIa, BIb, rms_wI,
                              kI_out, kI_stride_b, stream=None):
    _check(_lib.csa_compress_indexer_keys(ctypes.byref(params), B, n_new, entry0, _ptr(CIa), _ptr(ZIa), _ptr(CIb),
                                          _ptr(ZIb), _ptr(CIb_prev), _ptr(ZIb_prev), _ptr(BIa), _ptr(BIb),
                                          _ptr(rms_wI), _ptr(kI_out), kI_stride_b, _stream(stream)),
           "csa_compress_indexer_keys")


def csa_compress_single(params, B, n_new, entry0, C, Z, bias, rms_w, kv_out, kv_stride_b, stream=None):
    _check(_lib.csa_compress_single(ctypes.byref(params), B, n_new, entry0, _ptr(C), _ptr(Z), _ptr(bias), _ptr(rms_w),
                                    _ptr(kv_out), kv_stride_b, _stream(stream)), "csa_compress_single")


def csa_compress_single_step(params, B, q_pos, C, Z, bias, rms_w, state, kv_out, kv_stride_b, n_cap, stream=None):
    _check(_lib.csa_compress_single_step(ctypes.byref(params), B, _ptr(q_pos), _ptr(C), _ptr(Z), _ptr(bias),
                                         _ptr(rms_w), _ptr(state), _ptr(kv_out), kv_stride_b, n_cap, _stream(stream)),
           "csa_compress_single_step")


def csa_index_topk(params, B, Q, q_pos, qI, wI, kI, n_cap, idx_out, score_out, ws, stream=None):
    _check(_lib.csa_index_topk(ctypes.byref(params), B, Q, _ptr(q_pos), _ptr(qI), _ptr(wI), _ptr(kI), n_cap,
                               _ptr(idx_out), _ptr(score_out), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream(stream)), "csa_index_topk")


def csa_hca_layer_decode(params, B, q_pos, C, Z, bias, rms_w, state, kv_comp, n_cap, q, swa_ring, sink, out, lse,
                         ws, stream=None):
    _check(_lib.csa_hca_layer_decode(ctypes.byref(params), B, _ptr(q_pos), _ptr(C), _ptr(Z), _ptr(bias), _ptr(rms_w),
                                     _ptr(state), _ptr(kv_comp), n_cap, _ptr(q), _ptr(swa_ring), _ptr(sink), _ptr(out),
                                     _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "csa_hca_layer_decode")


def csa_quantize_kv_fp4(n_rows, inp, in_stride, out, out_stride, stream=None):
    _check(_lib.csa_quantize_kv_fp4(n_rows, _ptr(inp), in_stride, _ptr(out), out_stride, _stream(stream)),
           "csa_quantize_kv_fp4")


def csa_quantize_index_keys_fp4(B, n_new, entry0, inp, in_stride_b, kI, n_cap, stream=None):
    _check(_lib.csa_quantize_index_keys_fp4(B, n_new, entry0, _ptr(inp), in_stride_b, _ptr(kI), n_cap,
                                            _stream(stream)), "csa_quantize_index_keys_fp4")


def csa_quantize_index_query_fp4(n_q, inp, qI, stream=None):
    _check(_lib.csa_quantize_index_query_fp4(n_q, _ptr(inp), _ptr(qI), _stream(stream)),
           "csa_quantize_index_query_fp4")


def index_keys_fp4_bytes(B: int, n_cap: int) -> int:
    """Bytes of an FP4 indexer key cache (CSA_FP4_INDEX_KEYS_BYTES)."""
    return B * (n_cap * 64 + (n_cap + 127) // 128 * 512)


def index_query_fp4_bytes(n_q: int) -> int:
    """Bytes of n_q FP4 indexer query records (CSA_FP4_INDEX_QUERY_BYTES)."""
    return n_q * 4608


def csa_index_topk_pool(params, B, Q, q_pos, qI, wI, kI, n_cap, idx_out, score_out, pool_blocks, pool_out, ws,
                        stream=None):
    _check(_lib.csa_index_topk_pool(ctypes.byref(params), B, Q, _ptr(q_pos), _ptr(qI), _ptr(wI), _ptr(kI), n_cap,
                                    _ptr(idx_out), _ptr(score_out), pool_blocks, _ptr(pool_out), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(stream)), "csa_index_topk_pool")


def csa_reindex_topk(params, B, Q, q_pos, qI, wI, kI, n_cap, pool, pool_blocks, idx_out, score_out, ws,
                     stream=None):
    _check(_lib.csa_reindex_topk(ctypes.byref(params), B, Q, _ptr(q_pos), _ptr(qI), _ptr(wI), _ptr(kI), n_cap,
                                 _ptr(pool), pool_blocks, _ptr(idx_out), _ptr(score_out), _ptr(ws),
                                 0 if ws is None else ws.numel(), _stream(stream)), "csa_reindex_topk")


STATIC_SCRATCH_BYTES = 16 << 20


def csa_index_topk_static(params, B, Q, q_pos, qI, wI, kI, n_cap, idx_out, score_out, stream=None):
    """csa_index_topk with its scratch in libcsa's fixed 16 MiB device array
    instead of a caller-provided workspace, for callers that cannot allocate
    device memory at the call (their own pool holds the GPU's memory, or they
    must not risk cudaMalloc blocking the host and synchronising the device).
    The first call on a device should come before any stream capture; calls
    that can overlap on the GPU race on the shared array."""
    _check(_lib.csa_index_topk_static(ctypes.byref(params), B, Q, _ptr(q_pos), _ptr(qI), _ptr(wI), _ptr(kI), n_cap,
                                      _ptr(idx_out), _ptr(score_out), _stream(stream)), "csa_index_topk_static")


def csa_sparse_attn(params, B, Q, q_pos, q, kv_comp, n_cap, idx, swa, swa_mode, swa_len, swa_pos0, sink, out,
                    lse=None, ws=None, stream=None):
    _check(_lib.csa_sparse_attn(ctypes.byref(params), B, Q, _ptr(q_pos), _ptr(q), _ptr(kv_comp), n_cap, _ptr(idx),
                                _ptr(swa), swa_mode, swa_len, _ptr(swa_pos0), _ptr(sink), _ptr(out), _ptr(lse),
                                _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)), "csa_sparse_attn")


def csa_layer_decode(params, B, q_pos, ring_Ca, ring_Za, ring_Cb, ring_Zb, Ba, Bb, rms_w, kv_comp, n_cap, kI, qI,
                     wI, q, swa_ring, sink, idx_out, out, lse, ws, stream=None):
    _check(_lib.csa_layer_decode(ctypes.byref(params), B, _ptr(q_pos), _ptr(ring_Ca), _ptr(ring_Za),
                                 _ptr(ring_Cb), _ptr(ring_Zb), _ptr(Ba), _ptr(Bb), _ptr(rms_w), _ptr(kv_comp),
                                 n_cap, _ptr(kI), _ptr(qI), _ptr(wI), _ptr(q), _ptr(swa_ring), _ptr(sink),
                                 _ptr(idx_out), _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                                 _stream(stream)), "csa_layer_decode")


def csa_layer_decode_append(params, B, q_pos, swa_new, kI_new, ring_Ca, ring_Za, ring_Cb, ring_Zb, Ba, Bb, rms_w,
                            kv_comp, n_cap, kI, qI, wI, q, swa_ring, sink, idx_out, out, lse, ws, stream=None):
    _check(_lib.csa_layer_decode_append(ctypes.byref(params), B, _ptr(q_pos), _ptr(swa_new), _ptr(kI_new),
                                        _ptr(ring_Ca), _ptr(ring_Za), _ptr(ring_Cb), _ptr(ring_Zb), _ptr(Ba),
                                        _ptr(Bb), _ptr(rms_w), _ptr(kv_comp), n_cap, _ptr(kI), _ptr(qI), _ptr(wI),
                                        _ptr(q), _ptr(swa_ring), _ptr(sink), _ptr(idx_out), _ptr(out), _ptr(lse),
                                        _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "csa_layer_decode_append")


def csa_layer_decode_with_keys(params, B, q_pos, swa_new, keys, ring_Ca, ring_Za, ring_Cb, ring_Zb, Ba, Bb, rms_w,
                               kv_comp, n_cap, kI, qI, wI, q, swa_ring, sink, idx_out, out, lse, ws, stream=None):
    """``keys``: a CsaIndexKeySrc (see index_key_src) over the key compressor's staging rings."""
    _check(_lib.csa_layer_decode_with_keys(ctypes.byref(params), B, _ptr(q_pos), _ptr(swa_new),
                                           None if keys is None else ctypes.byref(keys), _ptr(ring_Ca),
                                           _ptr(ring_Za), _ptr(ring_Cb), _ptr(ring_Zb), _ptr(Ba), _ptr(Bb),
                                           _ptr(rms_w), _ptr(kv_comp), n_cap, _ptr(kI), _ptr(qI), _ptr(wI), _ptr(q),
                                           _ptr(swa_ring), _ptr(sink), _ptr(idx_out), _ptr(out), _ptr(lse),
                                           _ptr(ws), 0 if ws is None else ws.numel(), _stream(stream)),
           "csa_layer_decode_with_keys")


def csa_layer_prefill_with_keys(params, B, Q, pos0, Ca, Za, Cb, Zb, Cb_prev, Zb_prev, Ba, Bb, rms_w, keys, kv_comp,
                                n_cap, kI, qI, wI, q, swa, sink, idx_out, out, lse, ws, stream=None):
    """``keys``: a CsaIndexKeySrc (see index_key_src) over the chunk's key compressor rows."""
    _check(_lib.csa_layer_prefill_with_keys(ctypes.byref(params), B, Q, pos0, _ptr(Ca), _ptr(Za), _ptr(Cb),
                                            _ptr(Zb), _ptr(Cb_prev), _ptr(Zb_prev), _ptr(Ba), _ptr(Bb), _ptr(rms_w),
                                            None if keys is None else ctypes.byref(keys), _ptr(kv_comp), n_cap,
                                            _ptr(kI), _ptr(qI), _ptr(wI), _ptr(q), _ptr(swa), _ptr(sink),
                                            _ptr(idx_out), _ptr(out), _ptr(lse), _ptr(ws),
                                            0 if ws is None else ws.numel(), _stream(stream)),
           "csa_layer_prefill_with_keys")


def csa_layer_prefill(params, B, Q, pos0, Ca, Za, Cb, Zb, Cb_prev, Zb_prev, Ba, Bb, rms_w, kv_comp, n_cap, kI, qI,
                      wI, q, swa, sink, idx_out, out, lse, ws, stream=None):
    _check(_lib.csa_layer_prefill(ctypes.byref(params), B, Q, pos0, _ptr(Ca), _ptr(Za), _ptr(Cb), _ptr(Zb),
                                  _ptr(Cb_prev), _ptr(Zb_prev), _ptr(Ba), _ptr(Bb), _ptr(rms_w), _ptr(kv_comp),
                                  n_cap, _ptr(kI), _ptr(qI), _ptr(wI), _ptr(q), _ptr(swa), _ptr(sink),
                                  _ptr(idx_out), _ptr(out), _ptr(lse), _ptr(ws), 0 if ws is None else ws.numel(),
                                  _stream(stream)), "csa_layer_prefill")


# ---- grouped-query attention layers --------------------------------------------
# These calls take their sizes and strides from the tensors and refuse, as
# CSA_ERR_INVALID_ARG, tensors of another type, shape or device than theirs
# (the device: the current one).

(CSA_ROPE_INTERLEAVED, CSA_ROPE_HALF) = range(2)
(CSA_ROPE_UNSCALED, CSA_ROPE_LINEAR, CSA_ROPE_BY_PARTS) = range(3)


class CsaRopeParams(ctypes.Structure):
    """Mirror of ``csa_rope_params``."""
    _fields_ = [("rope_dim", ctypes.c_int32), ("offset", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("theta", ctypes.c_float), ("factor", ctypes.c_float),
                ("orig_len", ctypes.c_int32), ("beta_fast", ctypes.c_float), ("beta_slow", ctypes.c_float),
                ("mscale", ctypes.c_float)]


class CsaPagedCache(ctypes.Structure):
    """Mirror of ``csa_paged_cache`` (device pointers; see paged_cache)."""
    _fields_ = [("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("table", ctypes.c_void_p),
                ("table_stride", ctypes.c_int64)]


class CsaPageBook(ctypes.Structure):
    """Mirror of ``csa_page_book`` (device pointers; see page_book)."""
    _fields_ = [("n_seqs", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p)]


_R, _C, _K = ctypes.POINTER(CsaRopeParams), ctypes.POINTER(CsaPagedCache), ctypes.POINTER(CsaPageBook)
_lib.csa_default_rope.argtypes = [_R]
_lib.csa_default_rope.restype = None
_lib.csa_rope_table.argtypes = [_R, _vp]
_lib.csa_rope.argtypes = [_R, _vp, _i64, _i32, _i32, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _i32, _vp]
_lib.csa_kv_append.argtypes = [_C, _R, _vp, _i32, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp]
_lib.csa_paged_attn_workspace_size.argtypes = [_C, _i32, _i32]
_lib.csa_paged_attn_workspace_size.restype = _sz
_lib.csa_paged_attn.argtypes = [_C, _i32, _i32, _vp, _vp, _i64, _i64, ctypes.c_float, _i32, _vp, _vp, _vp, _vp, _sz,
                                _vp]
_lib.csa_prompt_attn.argtypes = ([_i32] * 4 + [_i64] * 2 + [_vp] * 2 + [_vp, _i64, _i64] * 3 +
                                 [ctypes.c_float, _i32, _i32] + [_vp] * 4)
_lib.csa_chunk_attn_workspace_size.argtypes = [_C, _i32]
_lib.csa_chunk_attn_workspace_size.restype = _sz
_lib.csa_chunk_attn.argtypes = [_C, _i32, _i32, _i64, _vp, _vp, _vp, _i64, _i64, ctypes.c_float, _i32, _vp, _vp, _vp,
                                _vp, _sz, _vp]
_lib.csa_pages_workspace_size.argtypes = [_K]
_lib.csa_pages_workspace_size.restype = _sz
_lib.csa_pages_resize.argtypes = [_K] + [_vp] * 5 + [_sz, _vp]
_lib.csa_pages_fork.argtypes = [_K] + [_vp] * 4 + [_sz, _vp]
_lib.csa_pages_compact.argtypes = [_K] + [_vp] * 6 + [_sz, _vp]
_lib.csa_pages_copy.argtypes = [_C, _i64, _vp, _vp, _vp]
for _f in ("csa_rope_table", "csa_rope", "csa_kv_append", "csa_paged_attn", "csa_prompt_attn", "csa_chunk_attn",
           "csa_pages_resize", "csa_pages_fork", "csa_pages_compact", "csa_pages_copy"):
    getattr(_lib, _f).restype = ctypes.c_int


_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


def _bad(where, name, t=None, expected=""):
    """Refuses an argument (the checks that lead here are written out at each call: they are most of a call's time
    on the host)."""
    if torch.is_tensor(t):
        name = "%s: %s %s, strides %s, on %s" % (name, t.dtype, tuple(t.shape), tuple(t.stride()), t.device)
    raise CsaError(1, "%s (%s%s)" % (where, name, "; expected " + expected if expected else ""))


def _flat(where, name, t, dtype, shape, dev):
    """A contiguous tensor of this type and shape on the current device: its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # no tensor
        pass
    _bad(where, name, t, "contiguous %s %s on the current device" % (dtype, tuple(shape)))


def _count(where, name, t):
    try:
        return t.numel()
    except AttributeError:
        _bad(where, name, t, "a tensor")


def _rows(where, name, t, shape, dev):
    """[rows][heads][channels] bf16 with contiguous channels on the current device: address, row and head stride (of
    a dimension of size one, whose stride has no meaning, a valid one)."""
    try:
        bad = t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev
    except AttributeError:  # no tensor
        bad = True
    if bad:
        _bad(where, name, t, "bfloat16 %s on the current device" % (tuple(shape),))
    rows, heads, dim = shape
    row, head, one = t.stride()
    if one != 1 and dim > 1:
        _bad(where, name, t, "contiguous channels")
    if heads <= 1:
        head = dim
    if rows <= 1:
        row = heads * head
    return t.data_ptr(), row, head


def _shape3(where, name, t):
    if not torch.is_tensor(t) or t.dim() != 3 or not t.is_cuda:
        _bad(where, name, t, "[rows][heads][channels] in device memory")
    return t.shape


def rope_params(**fields) -> CsaRopeParams:
    """csa_default_rope with any field overridden."""
    r = CsaRopeParams()
    _lib.csa_default_rope(ctypes.byref(r))
    for k, v in fields.items():
        if k not in dict(CsaRopeParams._fields_):
            _bad("rope_params", "no field %s" % k)
        setattr(r, k, v)
    return r


def rope_table(r: CsaRopeParams, device=None) -> torch.Tensor:
    """csa_rope_table's array in device memory (int64 bits), for csa_rope and csa_kv_append."""
    host = torch.empty(max(r.rope_dim // 2, 1), dtype=torch.int64)
    _check(_lib.csa_rope_table(ctypes.byref(r), host.data_ptr()), "csa_rope_table")
    return host.to(device or "cuda")


def csa_rope(r, turns, pos, x, out=None, inverse=False, stream=None):
    """Rotates x [rows][heads][channels] by pos [rows] (int32) into out, a new tensor where it is None; returns it."""
    w = "csa_rope"
    shape = _shape3(w, "x", x)
    dev = torch.cuda.current_device()
    if out is None:
        out = torch.empty(shape, dtype=_BF16, device=x.device)
    n, heads, dim = shape
    _check(_lib.csa_rope(ctypes.byref(r), _flat(w, "turns", turns, _I64, (r.rope_dim // 2,), dev), n, heads, dim,
                         _flat(w, "pos", pos, _I32, (n,), dev), *_rows(w, "x", x, shape, dev),
                         *_rows(w, "out", out, shape, dev), 1 if inverse else 0, _stream(stream, dev)), w)
    return out


def paged_cache(k, v, k_scale, v_scale, table) -> CsaPagedCache:
    """A ``csa_paged_cache`` over device tensors: k, v [pages][kv heads][page size][channels] E4M3 (or uint8 codes),
    k_scale, v_scale [pages][kv heads] fp32, table [sequences][pages] int32.  It keeps the tensors."""
    w = "paged_cache"
    for name, t in (("k", k), ("v", v)):
        if not torch.is_tensor(t) or t.dim() != 4 or t.dtype not in (torch.float8_e4m3fn, torch.uint8) or not t.is_cuda:
            _bad(w, name, t, "E4M3 or uint8 [pages][kv heads][page size][channels] in device memory")
    dev = torch.cuda.current_device()
    if not torch.is_tensor(table) or table.dim() != 2:
        _bad(w, "table", table, "[sequences][pages]")
    n, heads, page, dim = k.shape
    c = CsaPagedCache(heads, dim, page, n, _flat(w, "k", k, k.dtype, k.shape, dev),
                      _flat(w, "v", v, v.dtype, k.shape, dev), _flat(w, "k_scale", k_scale, _F32, (n, heads), dev),
                      _flat(w, "v_scale", v_scale, _F32, (n, heads), dev),
                      _flat(w, "table", table, _I32, table.shape, dev), table.shape[1])
    c.tensors, c.n_seqs, c.device = (k, v, k_scale, v_scale, table), table.shape[0], dev
    return c


def csa_kv_append(cache, r, turns, cu_rows, pos0, k, v, stream=None):
    """Appends rows of k and v [rows][kv heads][channels] to the cache from positions pos0 [B] on; sequence b's rows
    are cu_rows[b] .. cu_rows[b+1]-1 (cu_rows [B+1], or None: one row each).  r and turns None: keys as they are."""
    w = "csa_kv_append"
    B, shape = _count(w, "pos0", pos0), _shape3(w, "k", k)
    dev = torch.cuda.current_device()
    n, heads, dim = shape
    if heads != cache.n_kv_heads or dim != cache.head_dim or (cu_rows is None and n != B):
        _bad(w, "k", k, "[%s][%d][%d]" % (B if cu_rows is None else "rows", cache.n_kv_heads, cache.head_dim))
    if B > cache.n_seqs or cache.device != dev:
        _bad(w, "pos0", pos0, "at most %d sequences, the cache on the current device" % cache.n_seqs)
    _check(_lib.csa_kv_append(ctypes.byref(cache), None if r is None else ctypes.byref(r),
                              None if r is None else _flat(w, "turns", turns, _I64, (r.rope_dim // 2,), dev), B, n,
                              None if cu_rows is None else _flat(w, "cu_rows", cu_rows, _I32, (B + 1,), dev),
                              _flat(w, "pos0", pos0, _I32, (B,), dev), *_rows(w, "k", k, shape, dev),
                              *_rows(w, "v", v, shape, dev), _stream(stream, dev)), w)


def paged_attn_workspace(cache, B: int, n_heads: int) -> torch.Tensor:
    """Allocates (through torch) a workspace for csa_paged_attn."""
    n = int(_lib.csa_paged_attn_workspace_size(ctypes.byref(cache), B, n_heads))
    if n == 0:
        raise CsaError(2, "csa_paged_attn_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def csa_paged_attn(cache, lens, q, sm_scale, window, sink, out, lse, ws, stream=None):
    """q [B][heads][channels] over the cached tokens 0 .. lens[b]-1 into out [B][heads][channels] (and lse
    [B][heads] fp32, or None)."""
    w = "csa_paged_attn"
    shape = _shape3(w, "q", q)
    dev = torch.cuda.current_device()
    B, heads, dim = shape
    if dim != cache.head_dim or B > cache.n_seqs or cache.device != dev:
        _bad(w, "q", q, "at most %d sequences, heads of %d, the cache on the current device" %
             (cache.n_seqs, cache.head_dim))
    size = 0 if ws is None else _count(w, "ws", ws)
    _check(_lib.csa_paged_attn(ctypes.byref(cache), B, heads, _flat(w, "lens", lens, _I32, (B,), dev),
                               *_rows(w, "q", q, shape, dev), sm_scale, window,
                               None if sink is None else _flat(w, "sink", sink, _F32, (heads,), dev),
                               _flat(w, "out", out, _BF16, shape, dev),
                               None if lse is None else _flat(w, "lse", lse, _F32, (B, heads), dev),
                               None if ws is None else _flat(w, "ws", ws, torch.uint8, (size,), dev), size,
                               _stream(stream, dev)), w)


def csa_prompt_attn(cu_q, cu_k, q, k, v, sm_scale, causal, window, sink, out, lse=None, stream=None):
    """Packed sequences: q [rows][heads][channels] by cu_q [B+1], k and v [rows][kv heads][channels] by cu_k [B+1],
    into out (like q, contiguous) and lse [rows][heads] fp32 or None."""
    w = "csa_prompt_attn"
    shape, kv_shape = _shape3(w, "q", q), _shape3(w, "k", k)
    dev = torch.cuda.current_device()
    n, heads, dim = shape
    if kv_shape[2] != dim:
        _bad(w, "k", k, "heads of %d" % dim)
    B = _count(w, "cu_q", cu_q) - 1
    if B < 0:
        _bad(w, "cu_q", cu_q, "sequences + 1 offsets")
    _check(_lib.csa_prompt_attn(B, heads, kv_shape[1], dim, n, kv_shape[0],
                                _flat(w, "cu_q", cu_q, _I32, (B + 1,), dev),
                                _flat(w, "cu_k", cu_k, _I32, (B + 1,), dev), *_rows(w, "q", q, shape, dev),
                                *_rows(w, "k", k, kv_shape, dev), *_rows(w, "v", v, kv_shape, dev), sm_scale,
                                1 if causal else 0, window,
                                None if sink is None else _flat(w, "sink", sink, _F32, (heads,), dev),
                                _flat(w, "out", out, _BF16, shape, dev),
                                None if lse is None else _flat(w, "lse", lse, _F32, (n, heads), dev),
                                _stream(stream, dev)), w)


def chunk_attn_workspace(cache, n_heads: int) -> torch.Tensor:
    """Allocates (through torch) a workspace for csa_chunk_attn."""
    n = int(_lib.csa_chunk_attn_workspace_size(ctypes.byref(cache), n_heads))
    if n == 0:
        raise CsaError(2, "csa_chunk_attn_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def csa_chunk_attn(cache, cu_q, lens, q, sm_scale, window, sink, out, lse, ws, stream=None):
    """Packed queries q [rows][heads][channels] by cu_q [B+1], each sequence's at the last of its cached tokens
    0 .. lens[b]-1, into out (like q, contiguous) and lse [rows][heads] fp32 or None."""
    w = "csa_chunk_attn"
    shape, B = _shape3(w, "q", q), _count(w, "lens", lens)
    dev = torch.cuda.current_device()
    n, heads, dim = shape
    if dim != cache.head_dim or B > cache.n_seqs or cache.device != dev:
        _bad(w, "q", q, "at most %d sequences, heads of %d, the cache on the current device" %
             (cache.n_seqs, cache.head_dim))
    size = 0 if ws is None else _count(w, "ws", ws)
    _check(_lib.csa_chunk_attn(ctypes.byref(cache), B, heads, n, _flat(w, "cu_q", cu_q, _I32, (B + 1,), dev),
                               _flat(w, "lens", lens, _I32, (B,), dev), *_rows(w, "q", q, shape, dev), sm_scale,
                               window, None if sink is None else _flat(w, "sink", sink, _F32, (heads,), dev),
                               _flat(w, "out", out, _BF16, shape, dev),
                               None if lse is None else _flat(w, "lse", lse, _F32, (n, heads), dev),
                               None if ws is None else _flat(w, "ws", ws, torch.uint8, (size,), dev), size,
                               _stream(stream, dev)), w)


def page_book(table, lens, refs, page_size) -> CsaPageBook:
    """A ``csa_page_book`` over device tensors: table [sequences][pages], lens [sequences] and refs [pages of the
    pool], all int32.  It keeps the tensors."""
    w = "page_book"
    if not torch.is_tensor(table) or table.dim() != 2 or not table.is_cuda:
        _bad(w, "table", table, "[sequences][pages] in device memory")
    dev = torch.cuda.current_device()
    n = _count(w, "refs", refs)
    k = CsaPageBook(table.shape[0], page_size, n, _flat(w, "table", table, _I32, table.shape, dev), table.shape[1],
                    _flat(w, "lens", lens, _I32, (table.shape[0],), dev), _flat(w, "refs", refs, _I32, (n,), dev))
    k.tensors, k.device = (table, lens, refs), dev
    return k


def pages_workspace(book) -> torch.Tensor:
    """Allocates (through torch) a workspace for the csa_pages calls."""
    n = int(_lib.csa_pages_workspace_size(ctypes.byref(book)))
    if n == 0:
        raise CsaError(2, "csa_pages_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def _book_call(where, book, ws):
    """The current device, the book's on it, and the workspace's address and size."""
    dev = torch.cuda.current_device()
    if book.device != dev:
        _bad(where, "book: on another device than the current one")
    size = 0 if ws is None else _count(where, "ws", ws)
    return dev, None if ws is None else _flat(where, "ws", ws, torch.uint8, (size,), dev), size


def csa_pages_resize(book, target, pos0, src, dst, ws, stream=None):
    """The sequences' lengths become target [sequences] (negative: as it is); pos0 (or None) receives the length
    before of those that have grown and -1; src and dst (or None, both) the pages to copy.  All int32."""
    w, n = "csa_pages_resize", (book.n_seqs,)
    dev, at, size = _book_call(w, book, ws)
    _check(_lib.csa_pages_resize(ctypes.byref(book), _flat(w, "target", target, _I32, n, dev),
                                 *[None if t is None else _flat(w, name, t, _I32, n, dev)
                                   for name, t in (("pos0", pos0), ("src", src), ("dst", dst))],
                                 at, size, _stream(stream, dev)), w)


def csa_pages_fork(book, parent, src, dst, ws, stream=None):
    """Sequence b becomes a copy of parent[b] (negative: it is left alone); src and dst receive the pages to copy.
    All [sequences] int32."""
    w, n = "csa_pages_fork", (book.n_seqs,)
    dev, at, size = _book_call(w, book, ws)
    _check(_lib.csa_pages_fork(ctypes.byref(book), _flat(w, "parent", parent, _I32, n, dev),
                               _flat(w, "src", src, _I32, n, dev), _flat(w, "dst", dst, _I32, n, dev), at, size,
                               _stream(stream, dev)), w)


def csa_pages_compact(book, src, dst, used, table_out, refs_out, ws, stream=None):
    """New numbers for the used pages, 0 .. used-1: src and dst [pages // 2] receive the moves, table_out and refs_out
    (which may be the book's own) the table and the counts afterwards.  All int32."""
    w = "csa_pages_compact"
    dev, at, size = _book_call(w, book, ws)
    half = (book.n_pages // 2,)
    _check(_lib.csa_pages_compact(ctypes.byref(book), _flat(w, "src", src, _I32, half, dev),
                                  _flat(w, "dst", dst, _I32, half, dev), _flat(w, "used", used, _I32, (1,), dev),
                                  _flat(w, "table_out", table_out, _I32, (book.n_seqs, book.table_stride), dev),
                                  _flat(w, "refs_out", refs_out, _I32, (book.n_pages,), dev), at, size,
                                  _stream(stream, dev)), w)


def csa_pages_copy(cache, src, dst, stream=None):
    """The contents of the cache's pages src into its pages dst (int32, as many; negative: none)."""
    w = "csa_pages_copy"
    n = _count(w, "src", src)
    dev = torch.cuda.current_device()
    if cache.device != dev:
        _bad(w, "cache: on another device than the current one")
    _check(_lib.csa_pages_copy(ctypes.byref(cache), n, _flat(w, "src", src, _I32, (n,), dev),
                               _flat(w, "dst", dst, _I32, (n,), dev), _stream(stream, dev)), w)


CSA_TEST_FAULT_INDEXER, CSA_TEST_FAULT_TOPK, CSA_TEST_FAULT_ATTN = 1, 2, 4
_lib.csa_test_set_wait_fault.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
_lib.csa_test_set_wait_fault.restype = ctypes.c_int


def csa_test_set_wait_fault(wait_limit_us, faults):
    """Test-only: device wait limit (us, 0 = default) and withheld signals (CSA_TEST_FAULT_*)."""
    _check(_lib.csa_test_set_wait_fault(wait_limit_us, faults), "csa_test_set_wait_fault")


def csa_check_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status."""
    return int(_lib.csa_check_status(_stream(stream)))


def csa_set_trace_events(events) -> None:
    """Record the five stage-boundary events (torch.cuda.Event, timing
    enabled) in every following layer call; None turns tracing off."""
    if events is None:
        _check(_lib.csa_set_trace_events(None, 0), "csa_set_trace_events")
        return
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event at its first record
            e.record()
    arr = (_vp * len(events))(*[e.cuda_event for e in events])
    _check(_lib.csa_set_trace_events(arr, len(events)), "csa_set_trace_events")


def csa_launch_count() -> int:
    """Kernels launched by libcsa in this process so far."""
    return int(_lib.csa_launch_count())
