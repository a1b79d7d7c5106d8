"""Thin Python binding of libbiloco_hip (ctypes).

Argument marshalling only: every step runs in the library's HIP kernels.
Functions carry the C ABI's names; array arguments are torch tensors on the
GPU (device memory), passed by pointer, and calls are enqueued on torch's
current stream.  A missing library is an error: there is no other path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# another build of the same library (the host-sanitized one the tests load)
# can be named with BILOCO_HIP_LIB
LIB_PATH = os.environ.get("BILOCO_HIP_LIB") or os.path.join(_PKG, "libbiloco_hip.so")

BILOCO_OK = 0
BILOCO_ERR_INVALID_VALUE = 1
BILOCO_ERR_UNSUPPORTED = 2
BILOCO_ERR_HIP = 3
BILOCO_ERR_WORKSPACE_TOO_SMALL = 4

BILOCO_SCHED_AUTO = 0
BILOCO_SCHED_UNFUSED = 1
BILOCO_SCHED_FUSED_GEMV = 2
BILOCO_SCHED_FUSED_MFMA = 3
BILOCO_SCHED_COMPOSED = 4
BILOCO_SCHED_COMPOSED_MFMA = 5
BILOCO_SCHED_MFMA_ALLWG = 6
BILOCO_SCHED_MFMA_SIDE = 7
BILOCO_SCHED_MFMA_ZEPI = 8

EXPORTED = ["biloco_status_string", "biloco_pack_signs", "biloco_quant_act_fp4",
            "biloco_gemm_workspace_bytes", "biloco_gemm_lowrank", "biloco_gemm_lowrank_sched",
            "biloco_gemm_check", "biloco_default_schedule", "biloco_schedules_for",
            "biloco_quant_weight_nvfp4", "biloco_quant_weight_workspace_bytes",
            "biloco_peel_decompose", "biloco_peel_workspace_bytes", "biloco_gemm_lowrank_quant",
            "biloco_gemm_lowrank_quant_noalloc", "biloco_kv_append", "biloco_attn_paged",
            "biloco_attn_workspace_bytes", "biloco_norm_gate_residual"]

# size of the device array biloco_gemm_lowrank_quant_noalloc works in
BILOCO_NOALLOC_SCRATCH_BYTES = 16 << 20

_lib = None
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


class BilocoError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_name(status)} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m bit_weight_gemm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        p, i32, i64, sz, st = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t,
                               ctypes.c_int32)
        L.biloco_status_string.restype = ctypes.c_char_p
        L.biloco_status_string.argtypes = [st]
        L.biloco_pack_signs.restype = st
        L.biloco_pack_signs.argtypes = [p, i64, i64, p, p]
        L.biloco_quant_act_fp4.restype = st
        L.biloco_quant_act_fp4.argtypes = [p, i32, i32, p, p, p]
        L.biloco_quant_weight_nvfp4.restype = st
        L.biloco_quant_weight_nvfp4.argtypes = [p, i64, i64, p, p, p, p, sz, p]
        L.biloco_quant_weight_workspace_bytes.restype = st
        L.biloco_quant_weight_workspace_bytes.argtypes = [i64, i64, ctypes.POINTER(sz)]
        L.biloco_peel_decompose.restype = st
        L.biloco_peel_decompose.argtypes = [p, i64, i64, i32, i32, p, p, p, p, p, p, p, sz, p]
        L.biloco_peel_workspace_bytes.restype = st
        L.biloco_peel_workspace_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(sz)]
        L.biloco_gemm_workspace_bytes.restype = st
        L.biloco_gemm_workspace_bytes.argtypes = [i32, i32, i32, i32, ctypes.POINTER(sz)]
        gemm = [p, p, p, p, p, ctypes.c_float, p, p, p, i32, i32, i32, i32, p, p, sz]
        L.biloco_gemm_lowrank.restype = st
        L.biloco_gemm_lowrank.argtypes = gemm + [p]
        L.biloco_gemm_lowrank_sched.restype = st
        L.biloco_gemm_lowrank_sched.argtypes = gemm + [i32, p]
        L.biloco_gemm_lowrank_quant.restype = st
        L.biloco_gemm_lowrank_quant.argtypes = [p, p, p, p, p, ctypes.c_float, p, p, p, i32, i32, i32,
                                                i32, p, p, sz, i32, p]
        L.biloco_gemm_lowrank_quant_noalloc.restype = st
        L.biloco_gemm_lowrank_quant_noalloc.argtypes = [p, p, p, p, p, ctypes.c_float, p, p, p, i32,
                                                        i32, i32, i32, p, i32, p]
        L.biloco_gemm_check.restype = st
        L.biloco_gemm_check.argtypes = [p, p, p, p, p, p, p, p, i32, i32, i32, i32, p, p, sz, i32]
        L.biloco_default_schedule.restype = i32
        L.biloco_default_schedule.argtypes = [i32, i32, i32, i32]
        L.biloco_schedules_for.restype = i32
        L.biloco_schedules_for.argtypes = [i32, i32, i32, i32, ctypes.POINTER(i32), i32]
        f32 = ctypes.c_float
        cache = [p, p, p, p, i32, i32, i32, i32]
        ragged = [p, p, p, i32, i32, i32, i32]
        L.biloco_kv_append.restype = st
        L.biloco_kv_append.argtypes = cache + [p, i64, p, i64, p, i64, i32, p, i32, ctypes.c_char_p, p, i32,
                                               i32, i32] + ragged + [p, i64, p]
        L.biloco_attn_paged.restype = st
        L.biloco_attn_paged.argtypes = cache + [p, i64, i32] + ragged + [i32, f32, i32, i32, p, i64, p, p,
                                                                         sz, p]
        L.biloco_attn_workspace_bytes.restype = st
        L.biloco_attn_workspace_bytes.argtypes = [i32] * 7 + [ctypes.POINTER(sz)]
        L.biloco_norm_gate_residual.restype = st
        L.biloco_norm_gate_residual.argtypes = [p, i64, p, p, i64, f32, p, i64, i32, p, f32, f32, i32, i32, p,
                                                i64, p, i64, p, p, p]
        _lib = L
    return _lib


def status_name(s: int) -> str:
    return lib().biloco_status_string(int(s)).decode()


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # the current device's current stream, without building a Stream object
        # (0.2 us instead of 2.9)
        if torch.cuda.is_initialized():
            return _raw_stream(_current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(status: int, what: str):
    if status != BILOCO_OK:
        raise BilocoError(status, what)


def biloco_status_string(s: int) -> str:
    return status_name(s)


def biloco_pack_signs(signs: torch.Tensor, packed: torch.Tensor | None = None, stream=None):
    """signs int8 [rows][cols] (pass V.T / U.T) -> int32 words [ceil(rows/32)][cols]."""
    rows, cols = signs.shape
    if packed is None:
        packed = torch.empty(((rows + 31) // 32, cols), dtype=torch.int32, device=signs.device)
    _ok(lib().biloco_pack_signs(_p(signs), rows, cols, _p(packed), _stream(stream)),
        "biloco_pack_signs")
    return packed


def biloco_quant_act_fp4(x_bf16: torch.Tensor, codes=None, scales=None, stream=None):
    """x bf16 [M][K] -> (codes uint8 [M][K/2], scales uint8 [M][K/16])."""
    M, K = x_bf16.shape
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x_bf16.device)
    if scales is None:
        scales = torch.empty((M, K // 16), dtype=torch.uint8, device=x_bf16.device)
    _ok(lib().biloco_quant_act_fp4(_p(x_bf16), M, K, _p(codes), _p(scales), _stream(stream)),
        "biloco_quant_act_fp4")
    return codes, scales


def biloco_quant_weight_workspace_bytes(N: int, K: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().biloco_quant_weight_workspace_bytes(N, K, ctypes.byref(out)),
        "biloco_quant_weight_workspace_bytes")
    return int(out.value)


def biloco_quant_weight_nvfp4(w: torch.Tensor, codes=None, scales=None, g=None, workspace=None,
                              stream=None):
    """w fp32 [N][K] -> (codes uint8 [N][K/2], scales uint8 [N][K/16], g fp32 [1]), all on w's device."""
    N, K = w.shape
    dev = w.device
    if codes is None:
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((N, K // 16), dtype=torch.uint8, device=dev)
    if g is None:
        g = torch.empty(4, dtype=torch.float32, device=dev)[:1]
    nws = biloco_quant_weight_workspace_bytes(N, K)
    if workspace is None:
        workspace = torch.empty(nws, dtype=torch.uint8, device=dev)
    _ok(lib().biloco_quant_weight_nvfp4(_p(w), N, K, _p(codes), _p(scales), _p(g), _p(workspace),
                                        workspace.numel() * workspace.element_size(),
                                        _stream(stream)),
        "biloco_quant_weight_nvfp4")
    return codes, scales, g


def biloco_peel_workspace_bytes(m: int, n: int, r: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().biloco_peel_workspace_bytes(m, n, r, ctypes.byref(out)),
        "biloco_peel_workspace_bytes")
    return int(out.value)


def biloco_peel_decompose(W: torch.Tensor, r: int, T: int, v_init: torch.Tensor,
                          want_residual: bool = True, workspace=None, stream=None):
    """W fp32 [m][n], v_init int32 words [r][ceil(n/32)] (bit set = -1) ->
    dict(u_packed [ceil(r/32)][m], v_packed [ceil(r/32)][n] (int32 words),
    alpha [r], alpha_greedy [r], R [m][n] or None), all on W's device."""
    m, n = W.shape
    dev = W.device
    RW = (r + 31) // 32
    out = {"u_packed": torch.empty((RW, m), dtype=torch.int32, device=dev),
           "v_packed": torch.empty((RW, n), dtype=torch.int32, device=dev),
           "alpha": torch.empty(r, dtype=torch.float32, device=dev),
           "alpha_greedy": torch.empty(r, dtype=torch.float32, device=dev),
           "R": torch.empty((m, n), dtype=torch.float32, device=dev) if want_residual else None}
    if workspace is None:
        workspace = torch.empty(biloco_peel_workspace_bytes(m, n, r), dtype=torch.uint8, device=dev)
    _ok(lib().biloco_peel_decompose(_p(W), m, n, r, T, _p(v_init), _p(out["u_packed"]),
                                    _p(out["v_packed"]), _p(out["alpha"]), _p(out["alpha_greedy"]),
                                    _p(out["R"]), _p(workspace),
                                    workspace.numel() * workspace.element_size(), _stream(stream)),
        "biloco_peel_decompose")
    return out


def biloco_gemm_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().biloco_gemm_workspace_bytes(M, N, K, r, ctypes.byref(out)),
        "biloco_gemm_workspace_bytes")
    return int(out.value)


def biloco_gemm_lowrank_sched(a_codes, a_scales, x_bf16, w_codes, w_scales, w_global_scale,
                              v_packed, u_packed, alpha_bf16, M, N, K, r, y, workspace,
                              workspace_bytes, schedule=BILOCO_SCHED_AUTO, stream=None):
    st = lib().biloco_gemm_lowrank_sched(
        _p(a_codes), _p(a_scales), _p(x_bf16), _p(w_codes), _p(w_scales), float(w_global_scale),
        _p(v_packed), _p(u_packed), _p(alpha_bf16), M, N, K, r, _p(y), _p(workspace),
        int(workspace_bytes), int(schedule), _stream(stream))
    _ok(st, "biloco_gemm_lowrank_sched")
    return y


def biloco_gemm_lowrank(a_codes, a_scales, x_bf16, w_codes, w_scales, w_global_scale, v_packed,
                        u_packed, alpha_bf16, M, N, K, r, y, workspace, workspace_bytes,
                        stream=None):
    st = lib().biloco_gemm_lowrank(
        _p(a_codes), _p(a_scales), _p(x_bf16), _p(w_codes), _p(w_scales), float(w_global_scale),
        _p(v_packed), _p(u_packed), _p(alpha_bf16), M, N, K, r, _p(y), _p(workspace),
        int(workspace_bytes), _stream(stream))
    _ok(st, "biloco_gemm_lowrank")
    return y


def biloco_gemm_lowrank_quant_noalloc(x_bf16, a_codes, a_scales, w_codes, w_scales,
                                      w_global_scale, v_packed, u_packed, alpha_bf16, M, N, K, r, y,
                                      schedule=BILOCO_SCHED_AUTO, stream=None):
    """biloco_gemm_lowrank_quant in the library's own per-GPU scratch array
    (no workspace argument; nothing is allocated)."""
    st = lib().biloco_gemm_lowrank_quant_noalloc(
        _p(x_bf16), _p(a_codes), _p(a_scales), _p(w_codes), _p(w_scales), float(w_global_scale),
        _p(v_packed), _p(u_packed), _p(alpha_bf16), M, N, K, r, _p(y), int(schedule),
        _stream(stream))
    _ok(st, "biloco_gemm_lowrank_quant_noalloc")
    return y


def biloco_gemm_lowrank_quant(x_bf16, a_codes, a_scales, w_codes, w_scales, w_global_scale,
                              v_packed, u_packed, alpha_bf16, M, N, K, r, y, workspace,
                              workspace_bytes, schedule=BILOCO_SCHED_AUTO, stream=None):
    """Quantise x into a_codes / a_scales (outputs) and compute y, in one call."""
    st = lib().biloco_gemm_lowrank_quant(
        _p(x_bf16), _p(a_codes), _p(a_scales), _p(w_codes), _p(w_scales), float(w_global_scale),
        _p(v_packed), _p(u_packed), _p(alpha_bf16), M, N, K, r, _p(y), _p(workspace),
        int(workspace_bytes), int(schedule), _stream(stream))
    _ok(st, "biloco_gemm_lowrank_quant")
    return y


def biloco_gemm_check(a_codes, a_scales, x_bf16, w_codes, w_scales, v_packed, u_packed,
                      alpha_bf16, M, N, K, r, y, workspace, workspace_bytes,
                      schedule=BILOCO_SCHED_AUTO) -> int:
    """Host-only argument check; returns the status code (no GPU needed)."""
    return int(lib().biloco_gemm_check(
        _p(a_codes), _p(a_scales), _p(x_bf16), _p(w_codes), _p(w_scales), _p(v_packed),
        _p(u_packed), _p(alpha_bf16), M, N, K, r, _p(y), _p(workspace), int(workspace_bytes),
        int(schedule)))


def biloco_default_schedule(M: int, N: int, K: int, r: int) -> int:
    return int(lib().biloco_default_schedule(M, N, K, r))


def biloco_schedules_for(M: int, N: int, K: int, r: int) -> list:
    buf = (ctypes.c_int32 * 8)()
    n = lib().biloco_schedules_for(M, N, K, r, buf, 8)
    return [int(buf[i]) for i in range(min(n, 8))]


# ---------------------------------------------------------------- decoder-layer operators
_bf16, _fp32, _int32, _uint8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8

# `cache` is the tuple (k_codes [pages][kv_heads][page][dim], v_codes
# [pages][kv_heads][page/8][dim][8], k_scales [pages][kv_heads], v_scales
# likewise), uint8, contiguous.  q, k, v and o are bf16 [tokens][heads][dim] whose
# heads and channels are contiguous; their token strides are free.

def biloco_kv_cache(num_pages: int, kv_heads: int, page_size: int, head_dim: int, device="cuda") -> tuple:
    """Uninitialised cache arrays in the layouts above (plain allocation)."""
    def new(*shape):
        return torch.empty(shape, dtype=torch.uint8, device=device)
    return (new(num_pages, kv_heads, page_size, head_dim),
            new(num_pages, kv_heads, page_size // 8, head_dim, 8),
            new(num_pages, kv_heads), new(num_pages, kv_heads))


# The checks below run on every call of a decode step: plain comparisons of
# attributes, no helper objects.

def _cache_args(cache):
    k, v, ks, vs = cache
    shape = k.shape
    pages, kv_heads, page, dim = shape
    if v.shape != (pages, kv_heads, page // 8, dim, 8) or ks.shape != (pages, kv_heads) or \
            vs.shape != (pages, kv_heads):
        raise ValueError("cache arrays of different shapes")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("cache arrays must be contiguous")
    return k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr(), pages, kv_heads, page, dim


def _rows(t, shape, what):
    """Token stride of a bf16 tensor [tokens][heads][dim] whose heads are contiguous."""
    a, b, c = t.stride()
    if t.shape != shape or t.dtype is not _bf16 or c != 1 or (b != shape[2] and shape[1] > 1):
        raise ValueError(f"{what}: bf16 {list(shape)} with contiguous heads expected")
    return a if shape[0] > 1 else shape[1] * shape[2]


def _ints(t, shape, what):
    if t.shape != shape or t.dtype is not _int32 or not t.is_contiguous():
        raise ValueError(f"{what}: contiguous int32 {list(shape)} expected")
    return t.data_ptr()


def biloco_kv_append(cache, q, k, v, positions, cos_sin, q_start, kv_len, block_table, max_q_len: int,
                     q_out=None, pair_axis: bytes | None = None, interleaved: bool = False, stream=None):
    """Rotate q and k, quantise and append k and v; returns q_out (None without q).
    positions int32 [axes][T]; cos_sin fp32 [n_pos][rot_dim] (None: no rotation);
    pair_axis: one byte per pair, the axis it turns by."""
    ck, cv, cks, cvs, pages, kv_heads, page, dim = _cache_args(cache)
    T, (B, max_pages) = k.shape[0], block_table.shape
    rot = n_pos = axes = heads = sq = so = 0
    pos = table = pq = po = None
    if cos_sin is not None:
        (n_pos, rot), axes = cos_sin.shape, positions.shape[0]
        if cos_sin.dtype is not _fp32 or not cos_sin.is_contiguous():
            raise ValueError("cos_sin: contiguous fp32 expected")
        pos, table = _ints(positions, (axes, T), "positions"), cos_sin.data_ptr()
    if pair_axis is not None and len(pair_axis) != rot // 2:
        raise ValueError("pair_axis has one byte per pair")
    if T == 0 or B == 0:      # empty tensors have no addresses
        return q_out if q is None or q_out is not None else torch.empty_like(q)
    kv = (T, kv_heads, dim)
    sk, sv = _rows(k, kv, "k"), _rows(v, kv, "v")
    if q is not None:
        heads = q.shape[1]
        qs = (T, heads, dim)
        if q_out is None:
            q_out = torch.empty(qs, dtype=_bf16, device=q.device)
        sq, so = _rows(q, qs, "q"), _rows(q_out, qs, "q_out")
        pq, po = q.data_ptr(), q_out.data_ptr()
    st = lib().biloco_kv_append(
        ck, cv, cks, cvs, pages, kv_heads, page, dim, pq, sq, k.data_ptr(), sk, v.data_ptr(), sv, heads, pos, axes,
        pair_axis, table, n_pos, rot, interleaved, _ints(q_start, (B + 1,), "q_start"), _ints(kv_len, (B,), "kv_len"),
        _ints(block_table, (B, max_pages), "block_table"), max_pages, B, T, max_q_len, po, so, _stream(stream))
    if st:
        _ok(st, "biloco_kv_append")
    return q_out


def biloco_attn_workspace_bytes(B: int, T: int, q_heads: int, kv_heads: int, head_dim: int, max_q_len: int,
                                max_kv_len: int) -> int:
    out = ctypes.c_size_t(0)
    _ok(lib().biloco_attn_workspace_bytes(B, T, q_heads, kv_heads, head_dim, max_q_len, max_kv_len,
                                          ctypes.byref(out)), "biloco_attn_workspace_bytes")
    return int(out.value)


def biloco_attn_paged(cache, q, q_start, kv_len, block_table, max_q_len: int, max_kv_len: int, scale: float,
                      window: int = 0, sinks: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of the new tokens q over the cache; returns out."""
    ck, cv, cks, cvs, pages, kv_heads, page, dim = _cache_args(cache)
    shape = q.shape
    T, heads, _ = shape
    B, max_pages = block_table.shape
    if out is None:
        out = torch.empty((T, heads, dim), dtype=_bf16, device=q.device)
    if lse is not None and (lse.shape != (T, heads) or lse.dtype is not _fp32 or not lse.is_contiguous()):
        raise ValueError("lse: contiguous fp32 [tokens][heads] expected")
    if T == 0 or B == 0:      # empty tensors have no addresses
        return out
    shape = (T, heads, dim)
    sq, so = _rows(q, shape, "q"), _rows(out, shape, "out")
    if workspace is None:
        n = biloco_attn_workspace_bytes(B, T, heads, kv_heads, dim, max_q_len, max_kv_len)
        workspace = torch.empty(max(n, 16), dtype=_uint8, device=q.device)
    st = lib().biloco_attn_paged(
        ck, cv, cks, cvs, pages, kv_heads, page, dim, q.data_ptr(), sq, heads, _ints(q_start, (B + 1,), "q_start"),
        _ints(kv_len, (B,), "kv_len"), _ints(block_table, (B, max_pages), "block_table"), max_pages, B, T, max_q_len,
        max_kv_len, scale, window, sinks, out.data_ptr(), so, None if lse is None else lse.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if st:
        _ok(st, "biloco_attn_paged")
    return out


def _row_stride(t, T, C, dtype, what):
    a, b = t.stride()
    if t.shape != (T, C) or t.dtype is not dtype or (b != 1 and C > 1):
        raise ValueError(f"{what}: {dtype} [{T}][{C}] with contiguous rows expected")
    return a if T > 1 else C


def _vector(w, C, what):
    if w.shape != (C,) or w.dtype is not _bf16 or not w.is_contiguous():
        raise ValueError(f"{what}: contiguous bf16 [{C}] expected")
    return w.data_ptr()


def biloco_norm_gate_residual(x, res, pre_w, post_w=None, gate=None, res_scale: float = 1.0, eps: float = 1e-6,
                              w_offset: float = 0.0, res_out=None, h=None, a_codes=None, a_scales=None,
                              stream=None):
    """r' = res + res_scale * gate * norm(x), h = norm(r'); returns (r', h).
    gate [1][C] (every token) or [T][C].  a_codes and a_scales: h's FP4
    quantisation (outputs)."""
    T, C = x.shape
    kind = res.dtype
    if kind is not _fp32 and kind is not _bf16:
        raise ValueError("res: bf16 or fp32 expected")
    if res_out is None:
        res_out = torch.empty((T, C), dtype=kind, device=x.device)
    if h is None:
        h = torch.empty((T, C), dtype=_bf16, device=x.device)
    if T == 0:      # empty tensors have no addresses
        return res_out, h
    gate_stride, pg, pc, ps = 0, None, None, None
    if gate is not None:
        one = gate.shape[0] == 1
        gate_stride = _row_stride(gate, 1 if one else T, C, _bf16, "gate")
        if one and T > 1:
            gate_stride = 0
        pg = gate.data_ptr()
    if a_codes is not None:
        if a_codes.shape != (T, C // 2) or a_codes.dtype is not _uint8 or not a_codes.is_contiguous():
            raise ValueError("a_codes: contiguous uint8 [tokens][C/2] expected")
        pc = a_codes.data_ptr()
    if a_scales is not None:
        if a_scales.shape != (T, C // 16) or a_scales.dtype is not _uint8 or not a_scales.is_contiguous():
            raise ValueError("a_scales: contiguous uint8 [tokens][C/16] expected")
        ps = a_scales.data_ptr()
    st = lib().biloco_norm_gate_residual(
        x.data_ptr(), _row_stride(x, T, C, _bf16, "x"), None if post_w is None else _vector(post_w, C, "post_w"), pg,
        gate_stride, res_scale, res.data_ptr(), _row_stride(res, T, C, kind, "res"), kind is _fp32,
        _vector(pre_w, C, "pre_w"), eps, w_offset, T, C, res_out.data_ptr(),
        _row_stride(res_out, T, C, kind, "res_out"), h.data_ptr(), _row_stride(h, T, C, _bf16, "h"), pc, ps,
        _stream(stream))
    if st:
        _ok(st, "biloco_norm_gate_residual")
    return res_out, h
