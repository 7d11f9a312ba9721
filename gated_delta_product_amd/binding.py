"""Thin ctypes binding of libgdp.so (include/gdp.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library.  torch provides device memory (outputs are allocated
with torch.empty on the inputs' device) and the current stream.  If the
library is not built this module raises; there is no fallback path.

Names follow the Megatron-Core GDP op pages: prefill_prepare
(core.ssm.ops.gdp.prepare), recompute_w_u (core.ssm.ops.gdp.wy_fast),
chunk_h and chunk_o (core.ssm.ops.gdp.chunk_o) and chunk_fwd for the three
chunk stages in order.
"""
import ctypes
import math
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libgdp.so")

GDP_OK, GDP_ERR_INVALID, GDP_ERR_UNSUPPORTED, GDP_ERR_HIP = 0, 1, 2, 3
GDP_F32, GDP_BF16 = 0, 1
CHUNK = 64
# size of the library's own scratch array used by gdp_chunk_fwd_scan_noalloc (GDP_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024

_i64, _i32, _f32, _vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_void_p


class ChunkArgs(ctypes.Structure):
    """Mirror of gdp_chunk_args (include/gdp.h)."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32),
        ("M", _i32), ("chunk_size", _i32), ("scale", _f32), ("dtype", ctypes.c_int),
        ("cu_seqlens", _vp), ("num_seqs", _i64), ("h_chunks", _i64),
        ("q", _vp), ("k", _vp), ("v", _vp), ("beta", _vp), ("g", _vp), ("k_rnorm", _vp),
        ("gcum", _vp), ("kdecay", _vp), ("w", _vp), ("u", _vp), ("v_new", _vp), ("h", _vp), ("o", _vp),
        ("h0", _vp), ("ht", _vp),
    ]


class DecodeArgs(ctypes.Structure):
    """Mirror of gdp_decode_args (include/gdp.h)."""
    _fields_ = [
        ("n", _i64), ("S", _i64), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32), ("M", _i32),
        ("scale", ctypes.c_float), ("dtype", ctypes.c_int), ("pool", _i64),
        ("q", _vp), ("k", _vp), ("v", _vp), ("beta", _vp), ("g", _vp), ("state", _vp), ("slots", _vp), ("o", _vp),
    ]


class PrepareArgs(ctypes.Structure):
    """Mirror of gdp_prepare_args (include/gdp.h)."""
    _fields_ = [
        ("x", _vp), ("x_n_stride", _i64), ("x_t_stride", _i64), ("ba", _vp), ("ba_n_stride", _i64),
        ("ba_t_stride", _i64), ("A_log", _vp), ("dt_bias", _vp), ("G", _i32),
    ]


class LinattnArgs(ctypes.Structure):
    """Mirror of gdp_linattn_args (include/gdp.h)."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32), ("scale", _f32),
        ("dtype", ctypes.c_int), ("cu_seqlens", _vp), ("num_seqs", _i64),
        ("q", _vp), ("q_b_stride", _i64), ("q_t_stride", _i64), ("k", _vp), ("k_b_stride", _i64),
        ("k_t_stride", _i64), ("v", _vp), ("v_b_stride", _i64), ("v_t_stride", _i64),
        ("g", _vp), ("g_b_stride", _i64), ("g_t_stride", _i64), ("g_head", _vp), ("h0", _vp), ("o", _vp), ("ht", _vp),
    ]


class LinattnGrads(ctypes.Structure):
    """Mirror of gdp_linattn_grads (include/gdp.h)."""
    _fields_ = [
        ("dout", _vp), ("do_b_stride", _i64), ("do_t_stride", _i64), ("dht", _vp), ("dq", _vp), ("dk", _vp),
        ("dv", _vp), ("dg", _vp), ("dg_head", _vp), ("dh0", _vp),
    ]


class LinattnDecodeArgs(ctypes.Structure):
    """Mirror of gdp_linattn_decode_args (include/gdp.h)."""
    _fields_ = [
        ("n", _i64), ("S", _i64), ("H", _i32), ("HV", _i32), ("K", _i32), ("V", _i32), ("scale", _f32),
        ("dtype", ctypes.c_int), ("pool", _i64),
        ("q", _vp), ("q_n_stride", _i64), ("q_t_stride", _i64), ("k", _vp), ("k_n_stride", _i64),
        ("k_t_stride", _i64), ("v", _vp), ("v_n_stride", _i64), ("v_t_stride", _i64),
        ("g", _vp), ("g_n_stride", _i64), ("g_t_stride", _i64), ("g_head", _vp), ("state", _vp), ("slots", _vp),
        ("o", _vp),
    ]


class GroupNormArgs(ctypes.Structure):
    """Mirror of gdp_group_norm_args (include/gdp.h)."""
    _fields_ = [
        ("n", _i64), ("T", _i64), ("groups", _i32), ("D", _i32), ("dtype", ctypes.c_int), ("activation", ctypes.c_int),
        ("centered", _i32), ("eps", _f32), ("x", _vp), ("x_n_stride", _i64), ("x_t_stride", _i64),
        ("z", _vp), ("z_n_stride", _i64), ("z_t_stride", _i64), ("w", _vp), ("b", _vp), ("y", _vp),
    ]


class GroupNormGrads(ctypes.Structure):
    """Mirror of gdp_group_norm_grads (include/gdp.h)."""
    _fields_ = [
        ("dy", _vp), ("dy_n_stride", _i64), ("dy_t_stride", _i64), ("dx", _vp), ("dz", _vp), ("dw", _vp), ("db", _vp),
    ]


class LinrecArgs(ctypes.Structure):
    """Mirror of gdp_linrec_args (include/gdp.h)."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("C", _i32), ("dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("decay", ctypes.c_int), ("complement", _i32), ("cu_seqlens", _vp), ("num_seqs", _i64),
        ("x", _vp), ("x_b_stride", _i64), ("x_t_stride", _i64), ("g", _vp), ("g_b_stride", _i64), ("g_t_stride", _i64),
        ("h0", _vp), ("y", _vp), ("ht", _vp),
    ]


class LinrecGrads(ctypes.Structure):
    """Mirror of gdp_linrec_grads (include/gdp.h)."""
    _fields_ = [
        ("dy", _vp), ("dy_b_stride", _i64), ("dy_t_stride", _i64), ("dht", _vp), ("dx", _vp), ("dg", _vp), ("dh0", _vp),
    ]


class LinrecDecodeArgs(ctypes.Structure):
    """Mirror of gdp_linrec_decode_args (include/gdp.h)."""
    _fields_ = [
        ("n", _i64), ("S", _i64), ("C", _i32), ("dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
        ("decay", ctypes.c_int), ("complement", _i32), ("pool", _i64),
        ("x", _vp), ("x_n_stride", _i64), ("x_t_stride", _i64), ("g", _vp), ("g_n_stride", _i64), ("g_t_stride", _i64),
        ("state", _vp), ("slots", _vp), ("y", _vp),
    ]


class ConvArgs(ctypes.Structure):
    """Mirror of gdp_conv_args (include/gdp.h)."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("C", _i32), ("W", _i32), ("dtype", ctypes.c_int), ("activation", ctypes.c_int),
        ("cu_seqlens", _vp), ("num_seqs", _i64), ("x", _vp), ("x_b_stride", _i64), ("x_t_stride", _i64),
        ("w", _vp), ("b", _vp), ("h0", _vp), ("y", _vp), ("ht", _vp),
    ]


class ConvGrads(ctypes.Structure):
    """Mirror of gdp_conv_grads (include/gdp.h)."""
    _fields_ = [
        ("dy", _vp), ("dy_b_stride", _i64), ("dy_t_stride", _i64), ("dht", _vp), ("dx", _vp), ("dw", _vp), ("db", _vp),
        ("dh0", _vp),
    ]


class ConvDecodeArgs(ctypes.Structure):
    """Mirror of gdp_conv_decode_args (include/gdp.h)."""
    _fields_ = [
        ("n", _i64), ("S", _i64), ("C", _i32), ("W", _i32), ("dtype", ctypes.c_int), ("activation", ctypes.c_int),
        ("pool", _i64), ("x", _vp), ("x_n_stride", _i64), ("x_t_stride", _i64), ("w", _vp), ("b", _vp),
        ("state", _vp), ("slots", _vp), ("y", _vp),
    ]


class RotaryArgs(ctypes.Structure):
    """Mirror of gdp_rotary_args (include/gdp.h)."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H", _i32), ("HK", _i32), ("D", _i32), ("R", _i32), ("dtype", ctypes.c_int),
        ("interleaved", _i32), ("inverse", _i32), ("scale", _f32), ("cu_seqlens", _vp), ("num_seqs", _i64),
        ("positions", _vp), ("pos_b_stride", _i64), ("pos_t_stride", _i64), ("offsets", _vp), ("freq", _vp),
        ("q", _vp), ("q_b_stride", _i64), ("q_t_stride", _i64), ("k", _vp), ("k_b_stride", _i64), ("k_t_stride", _i64),
        ("qo", _vp), ("qo_b_stride", _i64), ("qo_t_stride", _i64), ("ko", _vp), ("ko_b_stride", _i64),
        ("ko_t_stride", _i64),
    ]


class GdpError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__("gdp status %d: %s" % (status, msg))
        self.status = status


_lib = None


def lib():
    """Load libgdp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libgdp.so is not built; run gated_delta_product_amd.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.gdp_prefill_prepare.restype = ctypes.c_int
        L.gdp_prefill_prepare.argtypes = [
            _vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp,
            _i64, _i64, _i32, _i32, _i32, _i32, _i32, ctypes.c_int,
            _vp, _vp, _vp, _vp, _vp, _vp]
        for name in ("gdp_recompute_w_u", "gdp_chunk_h", "gdp_chunk_o", "gdp_chunk_fwd"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.POINTER(ChunkArgs), _vp]
        L.gdp_decode_prepare.restype = ctypes.c_int
        L.gdp_decode_prepare.argtypes = L.gdp_prefill_prepare.argtypes
        L.gdp_decode_update.restype = ctypes.c_int
        L.gdp_decode_update.argtypes = [ctypes.POINTER(DecodeArgs), _vp]
        L.gdp_chunk_fwd_pipelined.restype = ctypes.c_int
        L.gdp_chunk_fwd_pipelined.argtypes = [ctypes.POINTER(ChunkArgs), _i32, _vp, _vp, _vp]
        L.gdp_prefill_fwd_pipelined.restype = ctypes.c_int
        L.gdp_prefill_fwd_pipelined.argtypes = [ctypes.POINTER(PrepareArgs), ctypes.POINTER(ChunkArgs), _i32, _vp,
                                                _vp, _vp]
        L.gdp_chunk_fwd_scan.restype = ctypes.c_int
        L.gdp_chunk_fwd_scan.argtypes = [ctypes.POINTER(ChunkArgs), _i32, _vp, _i64, _vp, _vp]
        L.gdp_chunk_fwd_scan_noalloc.restype = ctypes.c_int
        L.gdp_chunk_fwd_scan_noalloc.argtypes = [ctypes.POINTER(ChunkArgs), _i32, _vp, _vp]
        L.gdp_prefill_fwd_scan.restype = ctypes.c_int
        L.gdp_prefill_fwd_scan.argtypes = [ctypes.POINTER(PrepareArgs), ctypes.POINTER(ChunkArgs), _i32, _vp, _i64,
                                           _vp, _vp]
        L.gdp_scan_segments.restype = _i32
        L.gdp_scan_segments.argtypes = [_i64, _i32]
        L.gdp_scan_workspace_bytes.restype = _i64
        L.gdp_scan_workspace_bytes.argtypes = [_i64, _i32, _i32, _i32, _i32]
        L.gdp_scan_workspace_bytes_varlen.restype = _i64
        L.gdp_scan_workspace_bytes_varlen.argtypes = [_i64, _i64, _i32, _i32, _i32, _i32]
        L.gdp_pipeline_segments.restype = _i32
        L.gdp_pipeline_segments.argtypes = [_i64, _i32]
        L.gdp_pipeline_plan.restype = _i32
        L.gdp_pipeline_plan.argtypes = [_i64, _i32, ctypes.POINTER(_i64)]
        L.gdp_num_state_chunks.restype = _i64
        L.gdp_num_state_chunks.argtypes = [ctypes.POINTER(_i32), _i64, _i64, _i64, _i32, _i32]
        L.gdp_linattn_workspace_bytes.restype = _i64
        L.gdp_linattn_workspace_bytes.argtypes = [ctypes.POINTER(LinattnArgs), _i32]
        L.gdp_linattn_fwd.restype = ctypes.c_int
        L.gdp_linattn_fwd.argtypes = [ctypes.POINTER(LinattnArgs), _vp, _i64, _vp]
        L.gdp_linattn_bwd.restype = ctypes.c_int
        L.gdp_linattn_bwd.argtypes = [ctypes.POINTER(LinattnArgs), ctypes.POINTER(LinattnGrads), _vp, _i64, _vp]
        L.gdp_linattn_decode.restype = ctypes.c_int
        L.gdp_linattn_decode.argtypes = [ctypes.POINTER(LinattnDecodeArgs), _vp]
        L.gdp_group_norm_fwd.restype = ctypes.c_int
        L.gdp_group_norm_fwd.argtypes = [ctypes.POINTER(GroupNormArgs), _vp]
        L.gdp_group_norm_workspace_bytes.restype = _i64
        L.gdp_group_norm_workspace_bytes.argtypes = [ctypes.POINTER(GroupNormArgs)]
        L.gdp_group_norm_bwd.restype = ctypes.c_int
        L.gdp_group_norm_bwd.argtypes = [ctypes.POINTER(GroupNormArgs), ctypes.POINTER(GroupNormGrads), _vp, _i64, _vp]
        L.gdp_linrec_workspace_bytes.restype = _i64
        L.gdp_linrec_workspace_bytes.argtypes = [ctypes.POINTER(LinrecArgs), _i32]
        L.gdp_linrec_fwd.restype = ctypes.c_int
        L.gdp_linrec_fwd.argtypes = [ctypes.POINTER(LinrecArgs), _vp, _i64, _vp]
        L.gdp_linrec_bwd.restype = ctypes.c_int
        L.gdp_linrec_bwd.argtypes = [ctypes.POINTER(LinrecArgs), ctypes.POINTER(LinrecGrads), _vp, _i64, _vp]
        L.gdp_linrec_decode.restype = ctypes.c_int
        L.gdp_linrec_decode.argtypes = [ctypes.POINTER(LinrecDecodeArgs), _vp]
        L.gdp_conv_fwd.restype = ctypes.c_int
        L.gdp_conv_fwd.argtypes = [ctypes.POINTER(ConvArgs), _vp]
        L.gdp_conv_workspace_bytes.restype = _i64
        L.gdp_conv_workspace_bytes.argtypes = [ctypes.POINTER(ConvArgs)]
        L.gdp_conv_bwd.restype = ctypes.c_int
        L.gdp_conv_bwd.argtypes = [ctypes.POINTER(ConvArgs), ctypes.POINTER(ConvGrads), _vp, _i64, _vp]
        L.gdp_conv_decode.restype = ctypes.c_int
        L.gdp_conv_decode.argtypes = [ctypes.POINTER(ConvDecodeArgs), _vp]
        L.gdp_rotary.restype = ctypes.c_int
        L.gdp_rotary.argtypes = [ctypes.POINTER(RotaryArgs), _vp]
        L.gdp_last_error.restype = ctypes.c_char_p
        L.gdp_last_error.argtypes = []
        L.gdp_version.restype = ctypes.c_char_p
        L.gdp_version.argtypes = []
        _lib = L
    return _lib


def _check(status):
    if status != GDP_OK:
        raise GdpError(status, lib().gdp_last_error().decode())


def _dtype_code(t):
    if t == torch.bfloat16:
        return GDP_BF16
    if t == torch.float32:
        return GDP_F32
    raise TypeError("unsupported dtype %s (bf16 or f32)" % t)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*ts):
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("tensors must be on a GPU")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError("tensors on different devices")
    return dev


def _contig(t, name):
    if t is not None and not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


# ------------------------------------------------------------------ prepare

def prefill_prepare(x, ba, A_log, dt_bias, num_householder, num_heads, num_groups, head_dim, state_dim,
                    out=None):
    """Split, GQA-expand, Householder-fold and gate a prefill step.

    x [n, T, M*H*P + M*G*N + G*N] and ba [n, T, M*H + H] (bf16 or f32, last
    dim contiguous, rows may be strided); A_log, dt_bias [H] float32.
    Returns (q [n,T,H,N], k [n,T*M,H,N], v [n,T*M,H,P], beta [n,T*M,H] f32,
    g [n,T,H] f32).  ``out`` may hold preallocated (q, k, v, beta, g).
    """
    M, H, G, P, N = num_householder, num_heads, num_groups, head_dim, state_dim
    dev = _need_cuda(x, ba, A_log, dt_bias)
    if x.dim() != 3 or ba.dim() != 3:
        raise ValueError("x and ba must be 3-D [n, T, ...]")
    if x.stride(-1) != 1 or ba.stride(-1) != 1:
        raise ValueError("the last dimension of x and ba must be contiguous")
    if ba.dtype != x.dtype:
        raise ValueError("x and ba must share a dtype")
    if A_log.dtype != torch.float32 or dt_bias.dtype != torch.float32:
        raise ValueError("A_log and dt_bias must be float32")
    _contig(A_log, "A_log")
    _contig(dt_bias, "dt_bias")
    n, T = x.shape[0], x.shape[1]
    shapes = [((n, T, H, N), x.dtype), ((n, T * M, H, N), x.dtype), ((n, T * M, H, P), x.dtype),
              ((n, T * M, H), torch.float32), ((n, T, H), torch.float32)]
    if out is None:
        out = [torch.empty(s, dtype=d, device=dev) for s, d in shapes]
    for t, (s, d) in zip(out, shapes):
        if tuple(t.shape) != s or t.dtype != d or not t.is_contiguous() or t.device != dev:
            raise ValueError("out tensor mismatch: want %s %s" % (s, d))
    q, k, v, beta, g = out
    if x.shape[2] != M * H * P + M * G * N + G * N:
        raise ValueError("x last dim %d != M*H*P + M*G*N + G*N" % x.shape[2])
    if tuple(ba.shape) != (n, T, M * H + H):
        raise ValueError("ba must be [n, T, M*H + H]")
    _check(lib().gdp_prefill_prepare(
        _ptr(x), x.stride(0), x.stride(1), _ptr(ba), ba.stride(0), ba.stride(1),
        _ptr(A_log), _ptr(dt_bias), n, T, M, H, G, P, N, _dtype_code(x.dtype),
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _stream(dev)))
    return q, k, v, beta, g


# ------------------------------------------------------------------ chunk stages

def pipeline_segments(T, num_segments):
    """Segments gdp_chunk_fwd_pipelined runs for T tokens."""
    return int(lib().gdp_pipeline_segments(int(T), int(num_segments)))


def pipeline_plan(T, num_segments):
    """Token offsets where those segments start, then T (a list of n + 1)."""
    buf = (_i64 * (max(int(num_segments), 0) + 1))()
    n = lib().gdp_pipeline_plan(int(T), int(num_segments), buf)
    if n < 0:
        raise GdpError(GDP_ERR_INVALID, "bad arguments to gdp_pipeline_plan")
    return [int(buf[i]) for i in range(n + 1)]


def scan_segments(T, num_segments):
    """Segments gdp_chunk_fwd_scan runs for T tokens."""
    n = lib().gdp_scan_segments(int(T), int(num_segments))
    if n < 0:
        raise ValueError("bad arguments")
    return n


def num_state_chunks(T, M, B=1, cu_seqlens_host=None):
    """Chunks h must hold (sum over sequences of ceil(len*M/64))."""
    if cu_seqlens_host is None:
        return B * math.ceil(T * M / CHUNK)
    cu = torch.as_tensor(cu_seqlens_host, dtype=torch.int32).contiguous()
    n = cu.numel() - 1
    arr = (_i32 * (n + 1))(*cu.tolist())
    return int(lib().gdp_num_state_chunks(arr, n, 1, T, M, CHUNK))


class ChunkBuffers:
    """All tensors of one chunk forward (inputs, scratch and outputs)."""

    def __init__(self, q, k, v, beta, g, cu_seqlens=None, scale=None, h_chunks=None,
                 cu_seqlens_host=None, num_householder=None, initial_state=None, output_final_state=False):
        dev = _need_cuda(q, k, v, beta, g, cu_seqlens, initial_state)
        for t, nm in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (g, "g"), (initial_state, "initial_state")):
            if t is not None:
                _contig(t, nm)
        if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
            raise ValueError("q, k, v must be 4-D")
        B, T, H, K = q.shape
        M = num_householder if num_householder is not None else k.shape[1] // max(T, 1)
        HV, V = v.shape[2], v.shape[3]
        if tuple(k.shape) != (B, T * M, H, K):
            raise ValueError("k must be [B, T*M, H, K] = %s, got %s" % ((B, T * M, H, K), tuple(k.shape)))
        if tuple(v.shape[:2]) != (B, T * M):
            raise ValueError("v must be [B, T*M, HV, V]")
        if tuple(beta.shape) != (B, T * M, HV) or beta.dtype != torch.float32:
            raise ValueError("beta must be float32 [B, T*M, HV]")
        if g is not None and (tuple(g.shape) != (B, T, HV) or g.dtype != torch.float32):
            raise ValueError("g must be float32 [B, T, HV] (or None: ungated)")
        if k.dtype != q.dtype or v.dtype != q.dtype:
            raise ValueError("q, k, v must share a dtype")
        nseq = B
        if cu_seqlens is not None:
            if cu_seqlens.dtype != torch.int32:
                raise ValueError("cu_seqlens must be int32")
            _contig(cu_seqlens, "cu_seqlens")
            nseq = cu_seqlens.numel() - 1
        if h_chunks is None:
            if cu_seqlens is None:
                h_chunks = num_state_chunks(T, M, B)
            elif cu_seqlens_host is not None:
                h_chunks = num_state_chunks(T, M, 1, cu_seqlens_host)
            else:
                h_chunks = math.ceil(T * M / CHUNK) + nseq
        if initial_state is not None and (tuple(initial_state.shape) != (nseq, HV, V, K)
                                          or initial_state.dtype != torch.float32):
            raise ValueError("initial_state must be float32 [nseq, HV, V, K] = %s" % ((nseq, HV, V, K),))
        dt = q.dtype
        self.dims = dict(B=B, T=T, H=H, HV=HV, K=K, V=V, M=M, nseq=nseq)
        self.h0 = initial_state
        self.ht = torch.empty((nseq, HV, V, K), dtype=torch.float32, device=dev) if output_final_state else None
        self.q, self.k, self.v, self.beta, self.g = q, k, v, beta, g
        self.cu_seqlens = cu_seqlens
        self.k_rnorm = torch.empty((B, H, T * M), dtype=torch.float32, device=dev)
        self.gcum = torch.empty((B, HV, T * M), dtype=torch.float32, device=dev)
        self.kdecay = torch.empty((B, HV, T * M), dtype=torch.float32, device=dev)
        self.w = torch.empty((B, T * M, HV, K), dtype=dt, device=dev)
        # u and v_new are stored as 16-column slices [B, HV, V/16, T*M, 16]
        # (slices_to_rows gives the [B, T*M, HV, V] view)
        self.u = torch.empty((B, HV, V // 16, T * M, 16), dtype=dt, device=dev)
        self.v_new = torch.empty((B, HV, V // 16, T * M, 16), dtype=dt, device=dev)
        self.h = torch.empty((h_chunks, HV, V, K), dtype=dt, device=dev)
        self.o = torch.empty((B, T, HV, V), dtype=dt, device=dev)
        self.device = dev
        self.args = ChunkArgs(
            B=B, T=T, H=H, HV=HV, K=K, V=V, M=M, chunk_size=CHUNK,
            scale=float(scale) if scale is not None else 0.0, dtype=_dtype_code(dt),
            cu_seqlens=None if cu_seqlens is None else cu_seqlens.data_ptr(),
            num_seqs=nseq, h_chunks=h_chunks,
            q=q.data_ptr(), k=k.data_ptr(), v=v.data_ptr(), beta=beta.data_ptr(),
            g=None if g is None else g.data_ptr(),
            k_rnorm=self.k_rnorm.data_ptr(), gcum=self.gcum.data_ptr(), kdecay=self.kdecay.data_ptr(), w=self.w.data_ptr(), u=self.u.data_ptr(),
            v_new=self.v_new.data_ptr(), h=self.h.data_ptr(), o=self.o.data_ptr(),
            h0=None if initial_state is None else initial_state.data_ptr(),
            ht=None if self.ht is None else self.ht.data_ptr())

    def set(self, **tensors):
        """Point a slot (e.g. h, v_new) at another tensor of the same shape."""
        for name, t in tensors.items():
            cur = getattr(self, name)
            if tuple(t.shape) != tuple(cur.shape) or t.dtype != cur.dtype or not t.is_contiguous():
                raise ValueError("%s: shape/dtype mismatch" % name)
            setattr(self, name, t)
            setattr(self.args, name, t.data_ptr())

    def _call(self, fn, stream=None):
        s = stream if stream is not None else _stream(self.device)
        _check(fn(ctypes.byref(self.args), s))

    def recompute_w_u(self, stream=None):
        self._call(lib().gdp_recompute_w_u, stream)

    def chunk_h(self, stream=None):
        self._call(lib().gdp_chunk_h, stream)

    def chunk_o(self, stream=None):
        self._call(lib().gdp_chunk_o, stream)

    def forward(self, stream=None, store_vnew_h=True):
        """gdp_chunk_fwd.  store_vnew_h=False passes v_new and h as NULL:
        chunk_h and chunk_o then run as one pass that stores neither (bf16,
        M >= 2)."""
        if store_vnew_h:
            self._call(lib().gdp_chunk_fwd, stream)
        else:
            s = stream if stream is not None else _stream(self.device)
            _check(lib().gdp_chunk_fwd(ctypes.byref(self._args_without("v_new", "h")), s))
        return self.o

    def prefill_pipelined(self, x, ba, A_log, dt_bias, num_groups, num_segments, stream=None, chunk_h_events=None):
        """gdp_prefill_fwd_pipelined: prepare x / ba into this buffer's q, k,
        v, beta, g (allocated with the prepare shapes) and run the pipelined
        chunk forward, each segment's prepare overlapped with the serial
        stage.  Arguments as prefill_prepare and forward_pipelined."""
        _need_cuda(x, ba, A_log, dt_bias)
        d = self.dims
        if x.dim() != 3 or x.stride(2) != 1 or ba.dim() != 3 or ba.stride(2) != 1:
            raise ValueError("x and ba must be 3-D with a contiguous last dimension")
        if x.shape[:2] != (d["B"], d["T"]) or ba.shape[:2] != (d["B"], d["T"]) or x.dtype != self.q.dtype:
            raise ValueError("x / ba do not match the buffers")
        pa = PrepareArgs(x=x.data_ptr(), x_n_stride=x.stride(0), x_t_stride=x.stride(1), ba=ba.data_ptr(),
                         ba_n_stride=ba.stride(0), ba_t_stride=ba.stride(1), A_log=A_log.data_ptr(),
                         dt_bias=dt_bias.data_ptr(), G=int(num_groups))
        return self._pipelined(lambda ws, ev, s: lib().gdp_prefill_fwd_pipelined(
            ctypes.byref(pa), ctypes.byref(self.args), int(num_segments), ws, ev, s), num_segments, stream,
            chunk_h_events)

    def forward_pipelined(self, num_segments, stream=None, chunk_h_events=None):
        """gdp_chunk_fwd_pipelined: the same results for B == 1 without
        cu_seqlens, with the parallel stages of neighbouring segments
        overlapping the serial one.  chunk_h_events: optional list of
        2 * pipeline_segments(T, num_segments) torch.cuda.Event (timing
        enabled, recorded at least once) marking each segment's chunk_h."""
        return self._pipelined(lambda ws, ev, s: lib().gdp_chunk_fwd_pipelined(
            ctypes.byref(self.args), int(num_segments), ws, ev, s), num_segments, stream, chunk_h_events)

    def _args_without(self, *names):
        """A copy of the argument struct with the named tensors set to NULL."""
        args = type(self.args).from_buffer_copy(self.args)
        for nm in names:
            setattr(args, nm, None)
        return args

    def prefill_scan(self, x, ba, A_log, dt_bias, num_groups, num_segments, stream=None, stage_events=None,
                     store_v_beta=True, store_vnew_h=True, store_qk=True):
        """gdp_prefill_fwd_scan: prepare x / ba into this buffer's q, k, v,
        beta, g (allocated with the prepare shapes) inside the WY stage of the
        segment-parallel forward.  Arguments as prefill_prepare and
        forward_scan.  store_v_beta=False passes v and beta as NULL: nothing
        after the WY stage reads them, and they are left untouched.
        store_vnew_h=False as for forward_scan.  store_qk=False (with
        store_vnew_h=False) passes q and k as NULL: the later stages read their
        rows from x, and q and k are left untouched."""
        _need_cuda(x, ba, A_log, dt_bias)
        d = self.dims
        if x.dim() != 3 or x.stride(2) != 1 or ba.dim() != 3 or ba.stride(2) != 1:
            raise ValueError("x and ba must be 3-D with a contiguous last dimension")
        if x.shape[:2] != (d["B"], d["T"]) or ba.shape[:2] != (d["B"], d["T"]) or x.dtype != self.q.dtype:
            raise ValueError("x / ba do not match the buffers")
        pa = PrepareArgs(x=x.data_ptr(), x_n_stride=x.stride(0), x_t_stride=x.stride(1), ba=ba.data_ptr(),
                         ba_n_stride=ba.stride(0), ba_t_stride=ba.stride(1), A_log=A_log.data_ptr(),
                         dt_bias=dt_bias.data_ptr(), G=int(num_groups))
        args = self._args_without(*((() if store_v_beta else ("v", "beta")) +
                                    (() if store_vnew_h else ("v_new", "h")) +
                                    (() if store_qk else ("q", "k"))))
        return self._scan(lambda ws, nb, ev, s: lib().gdp_prefill_fwd_scan(
            ctypes.byref(pa), ctypes.byref(args), int(num_segments), ws, nb, ev, s), num_segments, stream,
            stage_events)

    def forward_scan(self, num_segments, stream=None, stage_events=None, store_vnew_h=True):
        """gdp_chunk_fwd_scan: the results of forward() for B == 1, one
        sequence or packed requests (cu_seqlens), to rounding past the first
        segment of each sequence, with every long serial chunk_h chain cut
        into segments run in parallel from the states a scan over the
        segments' composed maps gives.  Of h only the states entering chunks
        i*M (the ones chunk_o reads) are written; the other slots keep what
        they held.
        stage_events: optional 5 events with a cuda_event handle (timing
        enabled, recorded at least once), recorded after the WY stage, the
        segment maps, the scan, chunk_h and chunk_o.
        store_vnew_h=False passes v_new and h as NULL: chunk_h and chunk_o
        then run as one pass that stores neither (M >= 2), and they keep
        what they held."""
        args = self.args if store_vnew_h else self._args_without("v_new", "h")
        return self._scan(lambda ws, nb, ev, s: lib().gdp_chunk_fwd_scan(
            ctypes.byref(args), int(num_segments), ws, nb, ev, s), num_segments, stream, stage_events)

    def forward_scan_noalloc(self, num_segments, stream=None, stage_events=None, store_vnew_h=True):
        """gdp_chunk_fwd_scan_noalloc: forward_scan with the workspace taken
        from the library's own device scratch array (GDP_NOALLOC_SCRATCH_BYTES)
        instead of a tensor; nothing is allocated by the call.  Calls that
        overlap on one GPU share that array."""
        ev = _stage_events(stage_events)
        s = stream if stream is not None else _stream(self.device)
        args = self.args if store_vnew_h else self._args_without("v_new", "h")
        _check(lib().gdp_chunk_fwd_scan_noalloc(ctypes.byref(args), int(num_segments), ev, s))
        return self.o

    def scan_workspace_bytes(self, num_segments):
        """Workspace bytes gdp_chunk_fwd_scan needs for these buffers."""
        d = self.dims
        if self.cu_seqlens is not None:
            return lib().gdp_scan_workspace_bytes_varlen(d["T"], d["nseq"], d["HV"], d["K"], d["V"],
                                                         int(num_segments))
        return lib().gdp_scan_workspace_bytes(d["T"], d["HV"], d["K"], d["V"], int(num_segments))

    def _scan(self, call, num_segments, stream, stage_events):
        need = self.scan_workspace_bytes(num_segments)
        if need < 0:
            raise ValueError("num_segments %r out of range" % (num_segments,))
        ws = getattr(self, "_scan_ws", None)
        if ws is None or ws.numel() < need:
            # torch's caching allocator returns 512-byte aligned blocks
            self._scan_ws = ws = torch.empty(max(need, 256), dtype=torch.uint8, device=self.device)
        ev = _stage_events(stage_events)
        s = stream if stream is not None else _stream(self.device)
        _check(call(ws.data_ptr(), ws.numel(), ev, s))
        return self.o

    def _pipelined(self, call, num_segments, stream, chunk_h_events):
        d = self.dims
        if getattr(self, "_ws", None) is None:
            self._ws = torch.empty((2, d["HV"], d["V"], d["K"]), dtype=torch.float32, device=self.device)
        ev = None
        if chunk_h_events is not None:
            n = pipeline_segments(d["T"], num_segments)
            if len(chunk_h_events) != 2 * n:
                raise ValueError("need %d events" % (2 * n))
            ev = (_vp * (2 * n))(*[e.cuda_event for e in chunk_h_events])
        s = stream if stream is not None else _stream(self.device)
        _check(call(self._ws.data_ptr(), ev, s))
        return self.o


def _stage_events(events):
    """The 5 stage events of the segment-parallel forward as a C array."""
    if events is None:
        return None
    if len(events) != 5:
        raise ValueError("need 5 events")
    return (_vp * 5)(*[e.cuda_event for e in events])


def slices_to_rows(t):
    """A slice-major u / v_new [B, HV, V/16, T*M, 16] as [B, T*M, HV, V] (a copy)."""
    B, HV, S, TM, _ = t.shape
    return t.permute(0, 3, 1, 2, 4).reshape(B, TM, HV, S * 16)


def rows_to_slices(t):
    """[B, T*M, HV, V] -> the slice-major [B, HV, V/16, T*M, 16] layout of u / v_new."""
    B, TM, HV, V = t.shape
    return t.reshape(B, TM, HV, V // 16, 16).permute(0, 2, 3, 1, 4).contiguous()


def chunk_fwd(q, k, v, beta, g, scale=None, cu_seqlens=None, cu_seqlens_host=None, initial_state=None,
              output_final_state=False):
    """Chunked GDP forward.  q [B,T,H,K]; k [B,T*M,H,K]; v [B,T*M,HV,V];
    beta [B,T*M,HV] f32; g [B,T,HV] f32 natural-log decay per token, or None
    (ungated); initial_state [nseq,HV,V,K] f32 or None.
    Returns the ChunkBuffers holding o, the intermediates (w, u, v_new, h) and,
    if output_final_state, ht [nseq,HV,V,K] f32."""
    buf = ChunkBuffers(q, k, v, beta, g, cu_seqlens=cu_seqlens, scale=scale, cu_seqlens_host=cu_seqlens_host,
                       initial_state=initial_state, output_final_state=output_final_state)
    buf.forward()
    return buf


def version():
    return lib().gdp_version().decode()


# ------------------------------------------------------------------ decode

def decode_prepare(x, ba, A_log, dt_bias, M, H, G, P, N, out=None):
    """gdp_decode_prepare: x [n, S, M*H*P + M*G*N + G*N], ba [n, S, M*H + H]
    (last dimensions contiguous).  Returns (q [n,S*M,H,N] with the query on
    each token's last copy, k [n,S*M,H,N], v [n,S*M,H,P], beta [n,S*M,H]
    f32, g [n,S*M,H] f32 with the decay on each token's first copy)."""
    dev = _need_cuda(x, ba, A_log, dt_bias)
    n, S, width = x.shape
    if width != M * H * P + M * G * N + G * N or x.stride(2) != 1:
        raise ValueError("x must be [n, S, M*H*P + M*G*N + G*N] with a contiguous last dimension")
    if tuple(ba.shape) != (n, S, M * H + H) or ba.stride(2) != 1:
        raise ValueError("ba must be [n, S, M*H + H]")
    if out is None:
        dt = x.dtype
        out = (torch.empty((n, S * M, H, N), dtype=dt, device=dev), torch.empty((n, S * M, H, N), dtype=dt, device=dev),
               torch.empty((n, S * M, H, P), dtype=dt, device=dev),
               torch.empty((n, S * M, H), dtype=torch.float32, device=dev),
               torch.empty((n, S * M, H), dtype=torch.float32, device=dev))
    q, k, v, beta, g = out
    _check(lib().gdp_decode_prepare(
        _ptr(x), x.stride(0), x.stride(1), _ptr(ba), ba.stride(0), ba.stride(1),
        _ptr(A_log), _ptr(dt_bias), n, S, M, H, G, P, N, _dtype_code(x.dtype),
        _ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(g), _stream(dev)))
    return out


def decode_update(q, k, v, beta, g, state, M, slots=None, scale=None, o=None):
    """gdp_decode_update: one decode step over rows from decode_prepare.
    q, k [n, S*M, H, K]; v [n, S*M, HV, V]; beta, g [n, S*M, HV] f32 (g may
    be None); state [pool, HV, V, K] f32 updated in place; slots int32 [n]
    or None.  Returns o [n, S*M, HV, V]."""
    dev = _need_cuda(q, k, v, beta, g, state, slots)
    for t, nm in ((q, "q"), (k, "k"), (v, "v"), (beta, "beta"), (g, "g"), (state, "state"), (slots, "slots")):
        if t is not None:
            _contig(t, nm)
    n, L, H, K = q.shape
    HV, V = v.shape[2], v.shape[3]
    if L % M:
        raise ValueError("rows per request must be a multiple of M")
    if tuple(k.shape) != (n, L, H, K) or tuple(v.shape[:2]) != (n, L) or tuple(beta.shape) != (n, L, HV):
        raise ValueError("q, k, v, beta shapes disagree")
    if g is not None and tuple(g.shape) != (n, L, HV):
        raise ValueError("g must be [n, S*M, HV]")
    if state.dtype != torch.float32 or tuple(state.shape[1:]) != (HV, V, K):
        raise ValueError("state must be float32 [pool, HV, V, K]")
    if slots is not None and (slots.dtype != torch.int32 or tuple(slots.shape) != (n,)):
        raise ValueError("slots must be int32 [n]")
    if o is None:
        o = torch.empty((n, L, HV, V), dtype=q.dtype, device=dev)
    a = DecodeArgs(n=n, S=L // M, H=H, HV=HV, K=K, V=V, M=M, scale=float(scale) if scale is not None else 0.0,
                   dtype=_dtype_code(q.dtype), pool=state.shape[0], q=_ptr(q), k=_ptr(k), v=_ptr(v),
                   beta=_ptr(beta), g=None if g is None else _ptr(g), state=_ptr(state),
                   slots=None if slots is None else _ptr(slots), o=_ptr(o))
    _check(lib().gdp_decode_update(ctypes.byref(a), _stream(dev)))
    return o


# ------------------------------------------------------------------ linear attention
#
# These calls are made once a layer and token in decoding, where the host sets
# the pace: pointers go over as plain integers and every attribute of a tensor
# is asked for once.
#
# Like every call of this module they record nothing for autograd: results
# have no graph, also where an input requires gradients, which the _bwd calls give.

def _call(dev, fn, *args):
    """fn(*args, stream) on the tensors' device and its current stream."""
    i = dev.index
    if torch._C._cuda_getDevice() == i:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(i):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status != GDP_OK:
        raise GdpError(status, lib().gdp_last_error().decode())


def _at(t):
    return None if t is None else t.data_ptr()


def _rows(t, name, shape, dtype):
    """Checks a [n, T, heads, D] tensor whose rows [heads, D] are contiguous; its batch and token strides."""
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype != dtype:
        raise ValueError("q, k, v and %s must share a dtype" % name)
    s = t.stride()
    if (s[3] != 1 and shape[3] > 1) or (s[2] != shape[3] and shape[2] > 1):
        raise ValueError("the heads of %s must be contiguous" % name)
    return s[0], s[1]


def _decay(g, n, T, HV):
    """(g, batch stride, token stride, g_head) of a decay per token [n, T, HV], per head [HV], or None."""
    if g is None:
        return None, 0, 0, None
    if g.dtype != torch.float32:
        raise ValueError("g must be float32")
    if g.dim() == 1:
        if g.shape[0] != HV or not g.is_contiguous():
            raise ValueError("a decay per head must be a contiguous [HV]")
        return None, 0, 0, g.data_ptr()
    s = g.stride()
    if g.shape != (n, T, HV) or (HV > 1 and s[2] != 1):
        raise ValueError("g must be [n, T, HV] with a contiguous last dimension, or [HV]")
    return g.data_ptr(), s[0], s[1], None


def _qkv(q, k, v):
    if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be 4-D")
    shape = q.shape
    n, T, H, K = shape
    HV, V = v.shape[2:]
    dt = q.dtype
    return (n, T, H, HV, K, V, _dtype_code(dt), _rows(q, "q", shape, dt), _rows(k, "k", shape, dt),
            _rows(v, "v", (n, T, HV, V), dt))


def _state(t, name, shape):
    if t is not None and (t.shape != shape or t.dtype != torch.float32 or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous float32 %s" % (name, list(shape)))


def _output(t, name, shape, dtype, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s %s" % (name, dtype, list(shape)))
    return t


def _lin_args(q, k, v, g, scale, cu_seqlens, initial_state):
    B, T, H, HV, K, V, code, qs, ks, vs = _qkv(q, k, v)
    nseq = B
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
            raise ValueError("cu_seqlens must be int32 [num_seqs + 1]")
        _contig(cu_seqlens, "cu_seqlens")
        nseq = cu_seqlens.numel() - 1
    _state(initial_state, "initial_state", (nseq, HV, V, K))
    gp, gb, gt, gh = _decay(g, B, T, HV)
    return nseq, LinattnArgs(B, T, H, HV, K, V, 0.0 if scale is None else scale, code, _at(cu_seqlens), nseq,
                             q.data_ptr(), qs[0], qs[1], k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
                             gp, gb, gt, gh, _at(initial_state))


def _workspace(need, dev):
    # torch's caching allocator returns 512-byte aligned blocks.  Sizes that are
    # refused (need < 0) get none: the call itself then says so, with its status.
    return torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None


def linattn_fwd(q, k, v, g=None, scale=None, cu_seqlens=None, initial_state=None, output_final_state=False, o=None):
    """gdp_linattn_fwd: linear attention with a decay for each head,
    S_t = exp(g_t) S_{t-1} + v_t k_t^T and o_t = scale S_t q_t.

    q, k [B, T, H, K], v [B, T, HV, V] (bf16 or f32; heads contiguous, tokens
    and batch rows may be strided); g float32 [B, T, HV] natural-log decay per
    token, [HV] per head, or None; cu_seqlens int32 [num_seqs + 1] (B == 1) or
    None; initial_state [nseq, HV, V, K] float32 or None.  ``o`` may hold a
    preallocated contiguous output.  scale None, or any that is not above zero,
    is 1/sqrt(K).  Returns (o [B, T, HV, V], ht [nseq, HV, V, K] float32 or
    None).  Rows of o outside every request are not written: they keep what
    ``o`` held, or are uninitialised.  Nothing is recorded for autograd; the
    gradients come from linattn_bwd."""
    dev = _need_cuda(q, k, v, g, cu_seqlens, initial_state, o)
    nseq, a = _lin_args(q, k, v, g, scale, cu_seqlens, initial_state)
    o = _output(o, "o", (a.B, a.T, a.HV, a.V), q.dtype, dev)
    a.o = o.data_ptr()
    ht = None
    if output_final_state:
        ht = torch.empty((nseq, a.HV, a.V, a.K), dtype=torch.float32, device=dev)
        a.ht = ht.data_ptr()
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_linattn_workspace_bytes(pa, 0)
    ws = _workspace(need, dev)
    _call(dev, L.gdp_linattn_fwd, pa, _at(ws), need)
    return o, ht


def linattn_bwd(do, q, k, v, g=None, scale=None, cu_seqlens=None, initial_state=None, dht=None):
    """gdp_linattn_bwd: the gradients of linattn_fwd for those of o (do
    [B, T, HV, V], strided like v) and of ht (dht, or None).  Returns (dq, dk,
    dv, dg, dh0): dq, dk [B, T, H, K], summed over the value heads of a key
    head, dv [B, T, HV, V], dg shaped as g (None without g), dh0
    [nseq, HV, V, K] float32 (None without initial_state).  Rows of tokens
    outside every request hold zeros, and those of do are not read.  scale as
    in linattn_fwd."""
    dev = _need_cuda(q, k, v, g, cu_seqlens, initial_state, do, dht)
    nseq, a = _lin_args(q, k, v, g, scale, cu_seqlens, initial_state)
    ds = _rows(do, "do", v.shape, q.dtype)
    _state(dht, "dht", (nseq, a.HV, a.V, a.K))
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dk = torch.empty(q.shape, dtype=q.dtype, device=dev)
    dv = torch.empty(v.shape, dtype=q.dtype, device=dev)
    per_head = g is not None and g.dim() == 1
    dg = None if g is None else torch.empty(g.shape, dtype=torch.float32, device=dev)
    dh0 = None if initial_state is None else torch.empty_like(initial_state)
    d = LinattnGrads(do.data_ptr(), ds[0], ds[1], _at(dht), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                     None if per_head else _at(dg), _at(dg) if per_head else None, _at(dh0))
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_linattn_workspace_bytes(pa, 1)
    ws = _workspace(need, dev)
    _call(dev, L.gdp_linattn_bwd, pa, ctypes.byref(d), _at(ws), need)
    return dq, dk, dv, dg, dh0


def linattn_decode(q, k, v, state, g=None, slots=None, scale=None, o=None):
    """gdp_linattn_decode: S new tokens of each request through the recurrence
    of linattn_fwd.  q, k [n, S, H, K], v [n, S, HV, V] (strided as there); g
    float32 [n, S, HV], [HV] or None; state [pool, HV, V, K] float32, updated
    in place; slots int32 [n] (outside [0, pool): skipped, its o rows zero) or
    None; scale as there.  Returns o [n, S, HV, V].  It has no gradients."""
    dev = _need_cuda(q, k, v, g, state, slots, o)
    n, S, H, HV, K, V, code, qs, ks, vs = _qkv(q, k, v)
    pool = state.shape[0] if state.dim() else 0
    _state(state, "state", (pool, HV, V, K))
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (n,) or not slots.is_contiguous()):
        raise ValueError("slots must be a contiguous int32 [n]")
    o = _output(o, "o", (n, S, HV, V), q.dtype, dev)
    gp, gb, gt, gh = _decay(g, n, S, HV)
    a = LinattnDecodeArgs(n, S, H, HV, K, V, 0.0 if scale is None else scale, code, pool, q.data_ptr(), qs[0], qs[1],
                          k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], gp, gb, gt, gh, state.data_ptr(),
                          _at(slots), o.data_ptr())
    _call(dev, lib().gdp_linattn_decode, ctypes.byref(a))
    return o


# ------------------------------------------------------------------ group norm

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "sigmoid": 2}


def _token_rows(t, name):
    """[..., C] with a contiguous last dimension as (n, T, n stride, t stride): leading dimensions beyond two
    have to fold into the first."""
    shape, strides = t.shape, t.stride()
    if len(shape) < 1 or (strides[-1] != 1 and shape[-1] > 1):
        raise ValueError("the last dimension of %s must be contiguous" % name)
    if len(shape) == 2:
        return 1, shape[0], 0, strides[0]
    lead, strides = list(shape[:-1]), list(strides[:-1])
    while len(lead) < 2:
        lead.insert(0, 1)
        strides.insert(0, 0)
    while len(lead) > 2:
        if strides[0] != strides[1] * lead[1] and lead[0] > 1 and lead[1] > 1:
            raise ValueError("the leading dimensions of %s must fold into [n, T]" % name)
        lead[:2], strides[:2] = [lead[0] * lead[1]], [strides[1] if lead[1] > 1 else strides[0]]
    return lead[0], lead[1], strides[0], strides[1]


def _like(t, name, x):
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError("%s must match x: %s %s" % (name, x.dtype, list(x.shape)))
    return _token_rows(t, name)[2:]


def _norm_args(x, groups, weight, bias, gate, activation, centered, eps):
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError("activation must be one of %s" % sorted(k for k in ACTIVATIONS if k))
    n, T, ns, ts = _token_rows(x, "x")
    C = x.shape[-1]
    if groups < 1 or C < 1 or C % groups:
        raise ValueError("the %d channels do not split into %d groups" % (C, groups))
    for t, nm in ((weight, "weight"), (bias, "bias")):
        if t is not None and (t.dtype != torch.float32 or t.shape != (C,) or not t.is_contiguous()):
            raise ValueError("%s must be a contiguous float32 [C]" % nm)
    zs = (0, 0) if gate is None else _like(gate, "gate", x)
    return GroupNormArgs(n, T, groups, C // groups, _dtype_code(x.dtype), act, 1 if centered else 0, eps,
                         x.data_ptr(), ns, ts, _at(gate), zs[0], zs[1], _at(weight), _at(bias))


def group_norm_fwd(x, groups, weight=None, bias=None, gate=None, activation="silu", centered=True, eps=1e-5, out=None):
    """gdp_group_norm_fwd: x [..., C] (bf16 or f32, channels last) normalised per token in ``groups`` groups of
    neighbouring channels (centered=False: by the root of the mean square alone), times weight plus bias ([C]
    float32 or None), then times activation(gate), or without a gate through the activation ("silu", "sigmoid",
    "none").  gate is shaped as x; both may be slices of wider rows.  Returns y, contiguous (``out`` if given; it
    may be x or gate).  Nothing is recorded for autograd; the gradients come from group_norm_bwd."""
    dev = _need_cuda(x, weight, bias, gate, out)
    a = _norm_args(x, groups, weight, bias, gate, activation, centered, eps)
    out = _output(out, "out", x.shape, x.dtype, dev)
    a.y = out.data_ptr()
    _call(dev, lib().gdp_group_norm_fwd, ctypes.byref(a))
    return out


def group_norm_bwd(dy, x, groups, weight=None, bias=None, gate=None, activation="silu", centered=True, eps=1e-5):
    """gdp_group_norm_bwd: the gradients of group_norm_fwd for that of y (dy, shaped as x).  Returns (dx, dz,
    dweight, dbias): dx and dz as x (dz None without a gate), dweight and dbias [C] float32 (None where there is
    none)."""
    dev = _need_cuda(x, weight, bias, gate, dy)
    a = _norm_args(x, groups, weight, bias, gate, activation, centered, eps)
    ds = _like(dy, "dy", x)
    dx = torch.empty(x.shape, dtype=x.dtype, device=dev)
    dz = None if gate is None else torch.empty(x.shape, dtype=x.dtype, device=dev)
    dw = None if weight is None else torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    d = GroupNormGrads(dy.data_ptr(), ds[0], ds[1], dx.data_ptr(), _at(dz), _at(dw), _at(db))
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_group_norm_workspace_bytes(pa) if dw is not None or db is not None else 0
    ws = _workspace(need, dev)
    _call(dev, L.gdp_group_norm_bwd, pa, ctypes.byref(d), _at(ws), need)
    return dx, dz, dw, db


# ------------------------------------------------------------------ gated linear recurrence

DECAYS = {"log": 0, "sigmoid": 1}


def _channels(t, name, shape, dtypes):
    """Checks a [n, T, C] tensor with a contiguous last dimension; its batch and token strides."""
    if t.shape != shape:
        raise ValueError("%s must be %s, got %s" % (name, list(shape), list(t.shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s is %s, expected %s" % (name, t.dtype, " or ".join(str(d) for d in dtypes)))
    s = t.stride()
    if s[2] != 1 and shape[2] > 1:
        raise ValueError("the last dimension of %s must be contiguous" % name)
    return s[0], s[1]


def _new_like(t, dev):
    """A contiguous tensor of t's shape and dtype (empty_like takes half of empty's time on the host)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=dev)


def _out_like(y, name, t, dev):
    return _new_like(t, dev) if y is None else _output(y, name, t.shape, t.dtype, dev)


def _sequences(cu_seqlens, B):
    if cu_seqlens is None:
        return B
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be int32 [num_seqs + 1]")
    _contig(cu_seqlens, "cu_seqlens")
    return cu_seqlens.numel() - 1


def _state_of(t, name, shape, dtype):
    if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous()):
        raise ValueError("%s must be a contiguous %s %s" % (name, dtype, list(shape)))


def _slots_of(slots, n):
    if slots is not None and (slots.dtype != torch.int32 or slots.shape != (n,) or not slots.is_contiguous()):
        raise ValueError("slots must be a contiguous int32 [n]")


def _rec_input(x, g, decay):
    if x.dim() != 3:
        raise ValueError("x must be 3-D")
    if decay not in DECAYS:
        raise ValueError("decay must be one of %s" % sorted(DECAYS))
    code = _dtype_code(x.dtype)
    return code, _channels(x, "x", x.shape, (x.dtype,)), _channels(g, "g", x.shape, (x.dtype, torch.float32))


def _rec_args(x, g, decay, complement, cu_seqlens, initial_state):
    code, xs, gs = _rec_input(x, g, decay)
    B, T, C = x.shape
    nseq = _sequences(cu_seqlens, B)
    _state_of(initial_state, "initial_state", (nseq, C), torch.float32)
    return nseq, LinrecArgs(B, T, C, code, _dtype_code(g.dtype), DECAYS[decay], 1 if complement else 0,
                            _at(cu_seqlens), nseq, x.data_ptr(), xs[0], xs[1], g.data_ptr(), gs[0], gs[1],
                            _at(initial_state))


def linrec_fwd(x, g, decay="log", complement=False, cu_seqlens=None, initial_state=None, output_final_state=False,
               y=None):
    """gdp_linrec_fwd: the gated linear recurrence h_t = a_t h_{t-1} + c_t x_t, y_t = h_t, a state of one number per
    channel.

    x [B, T, C] (bf16 or f32; tokens and batch rows may be strided); g [B, T, C] of that dtype or float32: a = e^g
    (decay="log") or 1 / (1 + e^-g) (decay="sigmoid"); c is 1, or 1 - a with complement=True; cu_seqlens int32
    [num_seqs + 1] (B == 1) or None; initial_state [nseq, C] float32 or None.  ``y`` may hold a preallocated contiguous
    output, also x itself, or g.  Returns (y [B, T, C], ht [nseq, C] float32 or None).  Rows of y outside every request
    are not written: they keep what ``y`` held, or are uninitialised.  Nothing is recorded for autograd; the gradients
    come from linrec_bwd."""
    dev = _need_cuda(x, g, cu_seqlens, initial_state, y)
    nseq, a = _rec_args(x, g, decay, complement, cu_seqlens, initial_state)
    y = _out_like(y, "y", x, dev)
    a.y = y.data_ptr()
    ht = None
    if output_final_state:
        ht = torch.empty((nseq, a.C), dtype=torch.float32, device=dev)
        a.ht = ht.data_ptr()
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_linrec_workspace_bytes(pa, 0)
    ws = _workspace(need, dev)
    _call(dev, L.gdp_linrec_fwd, pa, _at(ws), need)
    return y, ht


def linrec_bwd(dy, x, g, decay="log", complement=False, cu_seqlens=None, initial_state=None, dht=None):
    """gdp_linrec_bwd: the gradients of linrec_fwd for those of y (dy, shaped as x, strided) and of ht (dht, or None).
    Returns (dx, dg, dh0): dx and dg as x and g, contiguous, zero in rows outside every request; dh0 [nseq, C] float32
    (None without initial_state)."""
    dev = _need_cuda(x, g, cu_seqlens, initial_state, dy, dht)
    nseq, a = _rec_args(x, g, decay, complement, cu_seqlens, initial_state)
    ds = _channels(dy, "dy", x.shape, (x.dtype,))
    _state_of(dht, "dht", (nseq, a.C), torch.float32)
    dx = _new_like(x, dev)
    dg = _new_like(g, dev)
    dh0 = None if initial_state is None else torch.empty_like(initial_state)
    d = LinrecGrads(dy.data_ptr(), ds[0], ds[1], _at(dht), dx.data_ptr(), dg.data_ptr(), _at(dh0))
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_linrec_workspace_bytes(pa, 1)
    ws = _workspace(need, dev)
    _call(dev, L.gdp_linrec_bwd, pa, ctypes.byref(d), _at(ws), need)
    return dx, dg, dh0


def linrec_decode(x, g, state, decay="log", complement=False, slots=None, y=None):
    """gdp_linrec_decode: S new tokens of each request through the recurrence of linrec_fwd.  x, g [n, S, C] (strided
    as there); state [pool, C] float32, updated in place; slots int32 [n] (outside [0, pool): skipped, its y rows zero)
    or None.  Returns y [n, S, C] (``y`` may be x or g, as there).  It has no gradients."""
    dev = _need_cuda(x, g, state, slots, y)
    code, xs, gs = _rec_input(x, g, decay)
    n, S, C = x.shape
    pool = state.shape[0] if state.dim() else 0
    _state_of(state, "state", (pool, C), torch.float32)
    _slots_of(slots, n)
    y = _out_like(y, "y", x, dev)
    a = LinrecDecodeArgs(n, S, C, code, _dtype_code(g.dtype), DECAYS[decay], 1 if complement else 0, pool, x.data_ptr(),
                         xs[0], xs[1], g.data_ptr(), gs[0], gs[1], state.data_ptr(), _at(slots), y.data_ptr())
    _call(dev, lib().gdp_linrec_decode, ctypes.byref(a))
    return y


# ------------------------------------------------------------------ short causal convolution

def _taps(weight, bias, C):
    if weight.dim() != 2 or weight.shape[0] != C or weight.dtype != torch.float32 or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous float32 [C, W]")
    if bias is not None and (bias.shape != (C,) or bias.dtype != torch.float32 or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous float32 [C]")
    return weight.shape[1]


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError("activation must be one of %s" % sorted(k for k in ACTIVATIONS if k))
    return act


def _conv_args(x, weight, bias, activation, cu_seqlens, initial_state):
    if x.dim() != 3:
        raise ValueError("x must be 3-D")
    B, T, C = x.shape
    act, W = _activation(activation), _taps(weight, bias, C)
    xs = _channels(x, "x", x.shape, (x.dtype,))
    nseq = _sequences(cu_seqlens, B)
    _state_of(initial_state, "initial_state", (nseq, W - 1, C), x.dtype)
    return nseq, ConvArgs(B, T, C, W, _dtype_code(x.dtype), act, _at(cu_seqlens), nseq, x.data_ptr(), xs[0], xs[1],
                          weight.data_ptr(), _at(bias), _at(initial_state))


def conv_fwd(x, weight, bias=None, activation="silu", cu_seqlens=None, initial_state=None, output_final_state=False,
             y=None):
    """gdp_conv_fwd: the short causal convolution in front of a mixer, y_t = act(bias + sum_j weight[:, j]
    x_{t-W+1+j}), depthwise and channels last.

    x [B, T, C] (bf16 or f32; tokens and batch rows may be strided); weight [C, W] float32, W 2 to 4; bias [C] float32
    or None; activation "silu", "sigmoid" or "none"; cu_seqlens int32 [num_seqs + 1] (B == 1) or None; initial_state
    [nseq, W - 1, C] of x's dtype, the inputs before each sequence, oldest first, or None (zeros).  ``y`` may hold a
    preallocated contiguous output that does not overlap x.  Returns (y [B, T, C], ht [nseq, W - 1, C] or None); rows of
    y outside every request are not written.  Nothing is recorded for autograd; the gradients come from conv_bwd."""
    dev = _need_cuda(x, weight, bias, cu_seqlens, initial_state, y)
    nseq, a = _conv_args(x, weight, bias, activation, cu_seqlens, initial_state)
    y = _out_like(y, "y", x, dev)
    a.y = y.data_ptr()
    ht = None
    if output_final_state:
        ht = torch.empty((nseq, max(a.W - 1, 0), a.C), dtype=x.dtype, device=dev)
        a.ht = ht.data_ptr()
    _call(dev, lib().gdp_conv_fwd, ctypes.byref(a))
    return y, ht


def conv_bwd(dy, x, weight, bias=None, activation="silu", cu_seqlens=None, initial_state=None, dht=None):
    """gdp_conv_bwd: the gradients of conv_fwd for those of y (dy, shaped as x, strided) and of ht (dht, or None).
    Returns (dx, dweight, dbias, dh0): dx as x, contiguous, zero in rows outside every request; dweight [C, W] and dbias
    [C] float32 (None without bias); dh0 [nseq, W - 1, C] (None without initial_state)."""
    dev = _need_cuda(x, weight, bias, cu_seqlens, initial_state, dy, dht)
    nseq, a = _conv_args(x, weight, bias, activation, cu_seqlens, initial_state)
    ds = _channels(dy, "dy", x.shape, (x.dtype,))
    _state_of(dht, "dht", (nseq, a.W - 1, a.C), x.dtype)
    dx = _new_like(x, dev)
    dw = torch.empty_like(weight)
    db = None if bias is None else torch.empty_like(bias)
    dh0 = None if initial_state is None else torch.empty_like(initial_state)
    d = ConvGrads(dy.data_ptr(), ds[0], ds[1], _at(dht), dx.data_ptr(), dw.data_ptr(), _at(db), _at(dh0))
    L, pa = lib(), ctypes.byref(a)
    need = L.gdp_conv_workspace_bytes(pa)
    ws = _workspace(need, dev)
    _call(dev, L.gdp_conv_bwd, pa, ctypes.byref(d), _at(ws), need)
    return dx, dw, db, dh0


def conv_decode(x, state, weight, bias=None, activation="silu", slots=None, y=None):
    """gdp_conv_decode: S new tokens of each request through the convolution of conv_fwd.  x [n, S, C] (strided as
    there); state [pool, W - 1, C] of x's dtype, updated in place; slots int32 [n] (outside [0, pool): skipped, its y
    rows zero) or None.  Returns y [n, S, C] (``y`` may be x).  It has no gradients."""
    dev = _need_cuda(x, weight, bias, state, slots, y)
    if x.dim() != 3:
        raise ValueError("x must be 3-D")
    n, S, C = x.shape
    act, W = _activation(activation), _taps(weight, bias, C)
    xs = _channels(x, "x", x.shape, (x.dtype,))
    pool = state.shape[0] if state.dim() else 0
    _state_of(state, "state", (pool, W - 1, C), x.dtype)
    _slots_of(slots, n)
    y = _out_like(y, "y", x, dev)
    a = ConvDecodeArgs(n, S, C, W, _dtype_code(x.dtype), act, pool, x.data_ptr(), xs[0], xs[1], weight.data_ptr(),
                       _at(bias), state.data_ptr(), _at(slots), y.data_ptr())
    _call(dev, lib().gdp_conv_decode, ctypes.byref(a))
    return y


# ------------------------------------------------------------------ rotary positions

def rotary_freq(rotated, base=10000.0, scaling=None, factor=1.0, original_length=None, fast=32.0, slow=1.0,
                device=None):
    """Frequencies of rotary positions: (freq [rotated / 2] float64 in radians per position, scale of the outputs).

    freq[i] = base^(-2i / rotated), for contexts of ``factor`` times the trained length changed by ``scaling``:
      None      not at all
      "linear"  positions pressed together: freq / factor
      "base"    a larger base, so that the slowest pair is slowed by factor and the fastest not at all
      "parts"   by what a pair turns over original_length positions: more than ``fast`` times stays, less than ``slow``
                times is divided by factor, linear in the pair's index between; the scale is 0.1 ln(factor) + 1."""
    if rotated < 2 or rotated % 2:
        raise ValueError("rotated must be even and at least 2")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be above 0 and factor at least 1")
    half = rotated // 2
    i = torch.arange(half, dtype=torch.float64)
    scale = 1.0
    if scaling == "base" and half > 1:
        base = base * factor ** (rotated / (rotated - 2))
    freq = torch.exp(i * (-2.0 / rotated) * math.log(base))
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "parts":
        if not original_length or not fast > slow > 0:
            raise ValueError("scaling by parts needs original_length and fast > slow > 0")

        def index(turns):  # of the pair that turns so often over the original length
            if base == 1:
                raise ValueError("scaling by parts needs a base other than 1")
            return rotated * math.log(original_length / (2 * math.pi * turns)) / (2 * math.log(base))

        lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rotated - 1)
        part = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        freq = freq * (1 - part) + freq / factor * part
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    return freq.to(device) if device is not None else freq, scale


def rotary(q, k, freq, positions=None, offsets=None, cu_seqlens=None, interleaved=False, scale=1.0, inverse=False,
           out=None):
    """gdp_rotary: rotary positions of q [B, T, H, D] and k [B, T, HK, D] (k may be None; bf16 or f32, heads contiguous,
    tokens and batch rows may be strided).  The first 2 len(freq) elements of a head are pairs, (i, i + len(freq)) or,
    interleaved, (2i, 2i + 1), and pair i turns by position * freq[i] (freq float64, radians; see rotary_freq), times
    scale.  A token's position is positions[b, t] (int32), or its place in its row or request of cu_seqlens plus
    offsets[sequence] (int32 [nseq], or None: 0).  inverse=True turns back: given the gradients of the outputs it
    returns those of q and k.  ``out`` may be (q', k') to write to, strided likewise without rows that overlap, also
    (q, k) themselves.  Returns (q', k'); rows outside every request are not written."""
    dev = _need_cuda(q, k, freq, positions, offsets, cu_seqlens, *(out or ()))
    if q.dim() != 4 or (k is not None and k.dim() != 4):
        raise ValueError("q and k must be 4-D")
    B, T, H, D = q.shape
    qs = _rows(q, "q", q.shape, q.dtype)
    HK = 0 if k is None else k.shape[2]
    ks = (0, 0) if k is None else _rows(k, "k", (B, T, HK, D), q.dtype)
    if freq.dim() != 1 or freq.dtype != torch.float64 or not freq.is_contiguous():
        raise ValueError("freq must be a contiguous float64 [R / 2]")
    nseq = _sequences(cu_seqlens, B)
    ps = (0, 0)
    if positions is not None:
        if positions.dtype != torch.int32 or positions.shape != (B, T):
            raise ValueError("positions must be int32 [B, T]")
        ps = positions.stride()
    if offsets is not None and (offsets.dtype != torch.int32 or offsets.shape != (nseq,) or not offsets.is_contiguous()):
        raise ValueError("offsets must be a contiguous int32 [nseq]")
    if out is None:
        qo = _new_like(q, dev)
        ko = None if k is None else _new_like(k, dev)
    else:
        qo, ko = out
        if (k is None) != (ko is None):
            raise ValueError("out must hold an output for each input")
    qos = _rows(qo, "out", q.shape, q.dtype)
    kos = (0, 0) if k is None else _rows(ko, "out", k.shape, q.dtype)
    a = RotaryArgs(B, T, H, HK, D, 2 * freq.shape[0], _dtype_code(q.dtype), 1 if interleaved else 0,
                   1 if inverse else 0, scale, _at(cu_seqlens), nseq, _at(positions), ps[0], ps[1], _at(offsets),
                   freq.data_ptr(), q.data_ptr(), qs[0], qs[1], _at(k), ks[0], ks[1], qo.data_ptr(), qos[0], qos[1],
                   _at(ko), kos[0], kos[1])
    _call(dev, lib().gdp_rotary, ctypes.byref(a))
    return qo, ko
