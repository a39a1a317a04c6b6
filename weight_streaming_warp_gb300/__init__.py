"""weight_streaming_warp_gb300 -- Python binding of libwsw.so, the GB300 (sm_103a)
decode-time weight-streaming hot path.

Every function marshals torch tensors into the C ABI declared in include/wsw.h and
launches the library's CUDA kernels on the current torch stream.  Nothing here
computes: outputs are allocated with torch (device memory) and filled by the
kernels.  The shared library is built in-tree by ``weight_streaming_warp_gb300.build``
(or ``__graft_entry__.build()``); if it is missing, every call raises.  There is no
CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import NamedTuple, Optional

import torch

__all__ = [
    "LaunchOpts", "WswError", "library_path", "load", "quantize_q8", "gemv_bf16",
    "gemv_bf16_chain", "gemv_q8_0", "quantize_gemv_q8_0", "moe_gemv_q8_0", "dequant_q8_0_kv", "gemm_bf16",
    "upload_padded", "status_string", "abi_version", "moe_workspace_bytes", "gemv_bf16_plan",
    "bounded_wait_check", "attn_decode_f16", "attn_decode_workspace_bytes", "attn_prefill_f16",
    "attn_prefill_q8_0", "attn_prefill_q8_0_workspace_bytes", "PagedKV", "KvPlan", "kv_page_plan", "RopeTable",
    "rope_table", "rope_kv_write", "attn_paged_decode", "attn_paged_decode_workspace_bytes", "TokenLogprobs",
    "token_logprobs", "token_logprobs_out", "token_logprobs_workspace_bytes", "PageCopies", "KvFork", "kv_page_fork",
    "kv_page_copy", "KvCompact", "kv_page_compact", "kv_page_compact_workspace_bytes", "BeamStep", "beam_select",
    "beam_select_out", "beam_select_workspace_bytes", "attn_paged_prefix", "attn_paged_prefix_workspace_bytes",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libwsw.so")
_lib = None

_current_device = getattr(torch._C, "_cuda_getDevice", None)  # none in a torch without CUDA
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_i64, _i32, _p, _f32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class WswError(RuntimeError):
    pass


class _COpts(ctypes.Structure):
    _fields_ = [("rows_per_warp", ctypes.c_int32), ("load_bytes", ctypes.c_int32),
                ("pdl", ctypes.c_int32), ("ctas_per_sm", ctypes.c_int32),
                ("l2_prefetch_steps", ctypes.c_int32)]


class _CLink(ctypes.Structure):
    _fields_ = [("W", ctypes.c_void_p), ("M", ctypes.c_int64), ("K", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("x", ctypes.c_void_p), ("alpha", ctypes.c_float),
                ("y", ctypes.c_void_p)]


class _CPlan(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("load_bytes", "rows_per_warp", "pdl", "ctas", "threads",
                                               "log2_segments", "x_in_smem", "l2_prefetch_steps")]


class _CKv(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k", "v", "kd", "vd")]
                + [(n, ctypes.c_int64) for n in ("num_pages", "page_size", "heads", "head_dim", "page_stride",
                                                 "pos_stride", "head_stride", "d_page_stride", "d_pos_stride",
                                                 "d_head_stride")]
                + [("dtype", ctypes.c_int32)])


@dataclass
class LaunchOpts:
    """Launch knobs (0 = library default).  None of them changes a result bit."""
    rows_per_warp: int = 0
    load_bytes: int = 0
    pdl: int = 0
    ctas_per_sm: int = 0
    l2_prefetch_steps: int = 0  # chain only: -1 = off

    def _c(self):
        return _COpts(self.rows_per_warp, self.load_bytes, self.pdl, self.ctas_per_sm, self.l2_prefetch_steps)


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load libwsw.so (once).  Raises WswError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise WswError("libwsw.so is not built (%s); run python -m weight_streaming_warp_gb300.build"
                       % _LIB_PATH)
    L = ctypes.CDLL(_LIB_PATH)
    L.wsw_status_string.argtypes = [ctypes.c_int]
    L.wsw_status_string.restype = ctypes.c_char_p
    L.wsw_abi_version.argtypes = []
    L.wsw_abi_version.restype = ctypes.c_int
    L.wsw_quantize_q8.argtypes = [_p, _i64, _i64, _i64, _i32, _p, _p, _p, _p]
    L.wsw_gemv_bf16.argtypes = [_p, _i64, _i64, _i64, _p, _f32, _p, _p, _p]
    L.wsw_gemv_bf16_chain.argtypes = [_i64, _p, _p, _p]
    L.wsw_gemv_q8_0.argtypes = [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p]
    L.wsw_quantize_gemv_q8_0.argtypes = [_p, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p]
    L.wsw_moe_gemv_q8_0.argtypes = [_p, _p, _i64, _i64, _i64, _p, _p, _p, _i64, _p, _p, _p, ctypes.c_size_t, _p, _p]
    L.wsw_moe_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.wsw_moe_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_dequant_q8_0_kv.argtypes = [_p, _p, _i64, _i64, _i64, _p, _p, _p]
    L.wsw_gemm_bf16.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _i64, _p, _p, _p]
    L.wsw_gemv_bf16_plan.argtypes = [_p, _i64, _i64, _i64, _i32, _i32, _p, _p]
    L.wsw_bounded_wait_check.argtypes = [_i32, _p, _p]
    L.wsw_attn_decode_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.wsw_attn_decode_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_attn_decode_f16.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _f32, _p, _p,
                                      ctypes.c_size_t, _p, _p]
    L.wsw_attn_prefill_f16.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _f32,
                                       _p, _p, _p]
    L.wsw_attn_prefill_q8_0_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64]
    L.wsw_attn_prefill_q8_0_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_attn_prefill_q8_0.argtypes = [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _i64, _f32, _i64, _p,
                                        ctypes.c_size_t, _p, _p, _p]
    L.wsw_attn_prefill_q8_0.restype = ctypes.c_int
    L.wsw_kv_page_plan.argtypes = [_p, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i64, _i64, _p, _p, _p, _p, _p, _p, _p,
                                   _p]
    L.wsw_rope_table.argtypes = [_i64, ctypes.c_double, _i32, ctypes.c_double, _i64, _p, _p, _p]
    L.wsw_rope_kv_write.argtypes = [_p, _p, _p, _i32, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _i64, _p, _i64, _f32,
                                    _i32, _p, _p, _p, _p, _p, _p, _p]
    L.wsw_attn_paged_decode_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64]
    L.wsw_attn_paged_decode_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_attn_paged_decode.argtypes = [_p, _i32, _i64, _i64, _p, _p, _i64, _i64, _p, _f32, _f32, _i64, _p, _p, _p, _p,
                                        _p, ctypes.c_size_t, _p, _p]
    L.wsw_token_logprobs_workspace_bytes.argtypes = [_i64, _i64, _i64]
    L.wsw_token_logprobs_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_token_logprobs.argtypes = [_p, _i32, _i64, _i64, _i64, _p, _f32, _i32, _p, _p, _p, _p, _p, _p, _p,
                                     ctypes.c_size_t, _p, _p]
    L.wsw_kv_page_fork.argtypes = [_p, _i64, _p, _i64, _p, _i64, _p, _i64, _p, _i64, _i64, _p, _i64, _p, _p, _p, _p, _p,
                                   _p, _p, _p, _p]
    L.wsw_kv_page_copy.argtypes = [_p, _p, _p, _p, _i64, _p, _i64, _p, _p, _p]
    L.wsw_kv_page_compact_workspace_bytes.argtypes = [_i64]
    L.wsw_kv_page_compact_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_kv_page_compact.argtypes = [_p, _i64, _p, _i64, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _p, _p, _p, _p,
                                      _p, ctypes.c_size_t, _p, _p]
    L.wsw_beam_select_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64]
    L.wsw_beam_select_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_beam_select.argtypes = [_p, _i32, _i64, _i64, _i64, _i64, _p, _p, _i64, _f32, _p, _p, _p, _p, _p, _p, _p,
                                  ctypes.c_size_t, _p, _p]
    L.wsw_attn_paged_prefix_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64, _i64]
    L.wsw_attn_paged_prefix_workspace_bytes.restype = ctypes.c_size_t
    L.wsw_attn_paged_prefix.argtypes = [_p, _i32, _i64, _i64, _p, _p, _i64, _i64, _p, _p, _i64, _p, _i32, _f32, _f32, _p,
                                        _p, _p, _p, _p, ctypes.c_size_t, _p, _p]
    for f in ("wsw_attn_paged_prefix", "wsw_beam_select", "wsw_kv_page_fork", "wsw_kv_page_copy", "wsw_kv_page_compact", "wsw_kv_page_plan", "wsw_rope_table", "wsw_rope_kv_write", "wsw_attn_paged_decode",
              "wsw_token_logprobs"):
        getattr(L, f).restype = ctypes.c_int
    for f in ("wsw_quantize_q8", "wsw_gemv_bf16", "wsw_gemv_bf16_chain", "wsw_gemv_q8_0", "wsw_quantize_gemv_q8_0",
              "wsw_moe_gemv_q8_0", "wsw_dequant_q8_0_kv", "wsw_gemm_bf16", "wsw_gemv_bf16_plan",
              "wsw_bounded_wait_check", "wsw_attn_decode_f16", "wsw_attn_prefill_f16"):
        getattr(L, f).restype = ctypes.c_int
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().wsw_status_string(code).decode()


def abi_version() -> int:
    return load().wsw_abi_version()


def _check(code: int, what: str):
    if code != 0:
        raise WswError("%s failed: %s" % (what, status_string(code)))


def _opts(opts):
    if opts is None:
        return None
    if isinstance(opts, dict):
        opts = LaunchOpts(**opts)
    return ctypes.byref(opts._c())


def _stream():
    """The current stream's handle (torch's raw accessor: a Stream object costs 3 us to make)."""
    return _raw_stream(_current_device())


def _dev(t: torch.Tensor, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise WswError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise WswError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _rowmajor(t: torch.Tensor, name):
    """(rows, cols, row stride) of a 2-D tensor whose last dim is contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise WswError("%s must be 2-D with unit stride in the last dimension" % name)
    return t.shape[0], t.shape[1], (t.stride(0) if t.shape[0] > 1 else max(t.shape[1], t.stride(0)))


# ---------------------------------------------------------------- calls ----

def quantize_q8(x: torch.Tensor, block: int = 32, out=None, opts=None):
    """x fp32 [rows][n] (or [n]) -> (q int8 [rows][n], scales).  Scales are fp16
    [rows][n/32] for block 32 and fp32 [rows][n/256] for block 256."""
    _dev(x, torch.float32, "x")
    squeeze = x.dim() == 1
    x2 = x.view(1, -1) if squeeze else x
    rows, n, ldx = _rowmajor(x2, "x")
    if out is None:
        q = torch.empty((rows, n), dtype=torch.int8, device=x.device)
        sc = torch.empty((rows, n // block), dtype=torch.float16 if block == 32 else torch.float32,
                         device=x.device)
    else:
        q, sc = out
    _check(load().wsw_quantize_q8(x2.data_ptr(), rows, n, ldx, block, q.data_ptr(), sc.data_ptr(),
                                  _stream(), _opts(opts)), "quantize_q8")
    return (q.view(-1), sc.view(-1)) if squeeze else (q, sc)


def gemv_bf16(W: torch.Tensor, x: torch.Tensor, alpha: float = 1.0, K=None, out=None, opts=None):
    """y fp32 [M] = alpha * W[:, :K] . x with W bf16 [M][ld] (row stride ld >= K)."""
    _dev(W, torch.bfloat16, "W")
    _dev(x, torch.float32, "x")
    M, cols, ld = _rowmajor(W, "W")
    K = cols if K is None else int(K)
    y = torch.empty(M, dtype=torch.float32, device=W.device) if out is None else out
    _check(load().wsw_gemv_bf16(W.data_ptr(), M, K, ld, x.data_ptr(), float(alpha), y.data_ptr(),
                                _stream(), _opts(opts)), "gemv_bf16")
    return y


def gemv_bf16_chain(links, opts=None):
    """links: iterable of (W, K, x, alpha, y) with W bf16 [M][ld] and x/y fp32 device
    tensors (x may be a view of an earlier link's y).  Launches every link back to
    back on the current stream, PDL-linked unless opts.pdl == 0 is given."""
    arr = (_CLink * len(links))()
    keep = []
    for i, (W, K, x, alpha, y) in enumerate(links):
        _dev(W, torch.bfloat16, "W")
        M, cols, ld = _rowmajor(W, "W")
        arr[i] = _CLink(W.data_ptr(), M, cols if K is None else int(K), ld, x.data_ptr(), float(alpha),
                        y.data_ptr())
        keep.append((W, x, y))
    _check(load().wsw_gemv_bf16_chain(len(links), ctypes.cast(arr, ctypes.c_void_p), _stream(),
                                      _opts(opts)), "gemv_bf16_chain")


def gemv_q8_0(Wq, Wd, xq, xd, K=None, out=None, opts=None):
    """y fp32 [M] from q8_0 weights (Wq int8 [M][ldq], Wd fp16 [M][K/32]) and a q8_0
    activation (xq int8 [K], xd fp16 [K/32])."""
    _dev(Wq, torch.int8, "Wq")
    _dev(Wd, torch.float16, "Wd")
    _dev(xq, torch.int8, "xq")
    _dev(xd, torch.float16, "xd")
    M, cols, ldq = _rowmajor(Wq, "Wq")
    K = cols if K is None else int(K)
    y = torch.empty(M, dtype=torch.float32, device=Wq.device) if out is None else out
    _check(load().wsw_gemv_q8_0(Wq.data_ptr(), Wd.data_ptr(), M, K, ldq, xq.data_ptr(), xd.data_ptr(),
                                y.data_ptr(), _stream(), _opts(opts)), "gemv_q8_0")
    return y


def quantize_gemv_q8_0(Wq, Wd, x, K=None, out=None, x_out=None, opts=None):
    """y fp32 [M] from q8_0 weights and the fp32 activation x [K], quantized to q8_0
    (block 32) inside the same launch; equals gemv_q8_0(Wq, Wd, *quantize_q8(x, 32))
    bit for bit.  x_out = (xq int8 [K], xd fp16 [K/32]) receives the quantized x."""
    _dev(Wq, torch.int8, "Wq")
    _dev(Wd, torch.float16, "Wd")
    _dev(x, torch.float32, "x")
    M, cols, ldq = _rowmajor(Wq, "Wq")
    K = cols if K is None else int(K)
    y = torch.empty(M, dtype=torch.float32, device=Wq.device) if out is None else out
    xq_p = xd_p = None
    if x_out is not None:
        _dev(x_out[0], torch.int8, "xq_out")
        _dev(x_out[1], torch.float16, "xd_out")
        xq_p, xd_p = x_out[0].data_ptr(), x_out[1].data_ptr()
    _check(load().wsw_quantize_gemv_q8_0(Wq.data_ptr(), Wd.data_ptr(), M, K, ldq, x.data_ptr(), xq_p, xd_p,
                                         y.data_ptr(), _stream(), _opts(opts)), "quantize_gemv_q8_0")
    return y


def moe_workspace_bytes(E, K, R) -> int:
    """Device workspace bytes that moe_gemv_q8_0 can use for these sizes (0: none)."""
    return int(load().wsw_moe_workspace_bytes(E, K, R))


def moe_gemv_q8_0(Wq, Wd, xq, xd, ids, out=None, err_flag=None, opts=None, ws=None):
    """Grouped q8_0 mat-vec.  Wq int8 [E][Mo][K], Wd fp16 [E][Mo][K/32], xq int8 [R][K],
    xd fp16 [R][K/32], ids int32 [R] -> y fp32 [R][Mo].  Rows with an id outside
    [0, E) are skipped and set err_flag (an int32 device tensor) nonzero.  ws: a uint8
    device tensor of at least moe_workspace_bytes(E, K, R) bytes; by default one is
    allocated when the call can use it, ws=False runs without one."""
    _dev(Wq, torch.int8, "Wq")
    _dev(Wd, torch.float16, "Wd")
    _dev(xq, torch.int8, "xq")
    _dev(xd, torch.float16, "xd")
    _dev(ids, torch.int32, "ids")
    E, Mo, K = Wq.shape
    R = ids.shape[0]
    for t, nm in ((Wq, "Wq"), (Wd, "Wd"), (xq, "xq"), (xd, "xd"), (ids, "ids")):
        if not t.is_contiguous():
            raise WswError("%s must be contiguous" % nm)
    y = torch.empty((R, Mo), dtype=torch.float32, device=Wq.device) if out is None else out
    errp = err_flag.data_ptr() if err_flag is not None else None
    if ws is None:
        nbytes = moe_workspace_bytes(E, K, R)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=Wq.device) if nbytes else False
    wsp, wsn = (ws.data_ptr(), ws.numel()) if ws is not False else (None, 0)
    _check(load().wsw_moe_gemv_q8_0(Wq.data_ptr(), Wd.data_ptr(), E, Mo, K, xq.data_ptr(),
                                    xd.data_ptr(), ids.data_ptr(), R, y.data_ptr(), errp, wsp, wsn,
                                    _stream(), _opts(opts)), "moe_gemv_q8_0")
    return y


def dequant_q8_0_kv(q, d, out=None, opts=None):
    """q int8 [depth][heads][head_dim], d fp16 [depth][heads][head_dim/32] ->
    fp16 [heads][depth][head_dim]."""
    _dev(q, torch.int8, "q")
    _dev(d, torch.float16, "d")
    if not (q.is_contiguous() and d.is_contiguous()):
        raise WswError("q and d must be contiguous")
    depth, heads, hd = q.shape
    o = torch.empty((heads, depth, hd), dtype=torch.float16, device=q.device) if out is None else out
    _check(load().wsw_dequant_q8_0_kv(q.data_ptr(), d.data_ptr(), depth, heads, hd, o.data_ptr(),
                                      _stream(), _opts(opts)), "dequant_q8_0_kv")
    return o


def gemm_bf16(W, X, K=None, out=None, opts=None):
    """Y fp32 [N][M] = X[:, :K] . W[:, :K]^T with W bf16 [M][ld], X bf16 [N][ldx]."""
    _dev(W, torch.bfloat16, "W")
    _dev(X, torch.bfloat16, "X")
    M, wc, ld = _rowmajor(W, "W")
    N, xc, ldx = _rowmajor(X, "X")
    K = min(wc, xc) if K is None else int(K)
    Y = torch.empty((N, M), dtype=torch.float32, device=W.device) if out is None else out
    _check(load().wsw_gemm_bf16(W.data_ptr(), M, K, ld, X.data_ptr(), N, ldx, Y.data_ptr(),
                                _stream(), _opts(opts)), "gemm_bf16")
    return Y


def gemv_bf16_plan(W_addr: int, M: int, K: int, ld: int, sm_count: int = 152, chain: bool = False,
                   opts=None) -> dict:
    """The launch that gemv_bf16 (chain=False) or a link of gemv_bf16_chain (chain=True)
    makes for a weight matrix at device address W_addr (only its alignment matters),
    as a dict of the wsw_gemv_plan fields.  Host only: no CUDA call."""
    p = _CPlan()
    _check(load().wsw_gemv_bf16_plan(ctypes.c_void_p(W_addr), M, K, ld, sm_count, int(bool(chain)),
                                      _opts(opts), ctypes.byref(p)), "wsw_gemv_bf16_plan")
    return {n: getattr(p, n) for n, _ in _CPlan._fields_}


def bounded_wait_check(arrive: bool) -> torch.Tensor:
    """Run the tensor-core kernels' bounded wait on its own; returns the int32 device
    status it writes (0 = WSW_OK after an arrival, 6 = WSW_ERR_TIMEOUT after about a
    second without one)."""
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    _check(load().wsw_bounded_wait_check(int(bool(arrive)), status.data_ptr(), _stream()),
           "wsw_bounded_wait_check")
    return status


def attn_decode_workspace_bytes(depth, heads, group) -> int:
    return int(load().wsw_attn_decode_workspace_bytes(depth, heads, group))


def attn_decode_f16(q, k, v, scale=None, out=None, ws=None, opts=None):
    """One decoding step of attention.  q fp32 [heads][group][head_dim]; k and v fp16
    views indexed [head][position][dim] with unit stride in dim and any head and
    position strides (the per-head-contiguous scratch as is, the position-major cache
    as cache.permute(1, 0, 2)).  scale defaults to 1/sqrt(head_dim).  Returns out fp32
    [heads][group][head_dim].  ws: a uint8 device tensor of at least
    attn_decode_workspace_bytes(depth, heads, group) bytes, zero-filled before its first
    use (every call leaves it ready for the next), allocated if None."""
    _dev(q, torch.float32, "q")
    _dev(k, torch.float16, "k")
    _dev(v, torch.float16, "v")
    if q.dim() != 3 or not q.is_contiguous():
        raise WswError("q must be a contiguous [heads][group][head_dim] tensor")
    heads, group, hd = q.shape
    for t, n in ((k, "k"), (v, "v")):
        if t.dim() != 3 or t.shape[0] != heads or t.shape[2] != hd or t.shape[1] != k.shape[1] or t.stride(2) != 1:
            raise WswError("%s must be a [heads][depth][head_dim] view with unit stride in head_dim" % n)
    depth = k.shape[1]
    if scale is None:
        scale = 1.0 / float(hd) ** 0.5
    y = out if out is not None else torch.empty((heads, group, hd), dtype=torch.float32, device=q.device)
    need = attn_decode_workspace_bytes(depth, heads, group)
    if ws is None:
        ws = torch.zeros(max(need, 1), dtype=torch.uint8, device=q.device)
    _check(load().wsw_attn_decode_f16(q.data_ptr(), k.data_ptr(), v.data_ptr(), depth, heads, group, hd,
                                      k.stride(1), k.stride(0), v.stride(1), v.stride(0), float(scale),
                                      y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(), _opts(opts)),
           "attn_decode_f16")
    return y


def attn_prefill_f16(q, k, v, scale=None, out=None, opts=None):
    """Causal prefill attention on the tensor cores.  q fp16 [heads][group][nq][head_dim]
    (contiguous); k and v fp16 views indexed [head][position][dim] with unit stride in
    dim and any head and position strides (multiples of 8).  Query i sits at position
    depth - nq + i and sees positions 0 .. depth - nq + i.  scale defaults to
    1/sqrt(head_dim).  Returns out fp32 [heads][group][nq][head_dim]."""
    _dev(q, torch.float16, "q")
    _dev(k, torch.float16, "k")
    _dev(v, torch.float16, "v")
    if q.dim() != 4 or not q.is_contiguous():
        raise WswError("q must be a contiguous [heads][group][nq][head_dim] tensor")
    heads, group, nq, hd = q.shape
    for t, n in ((k, "k"), (v, "v")):
        if t.dim() != 3 or t.shape[0] != heads or t.shape[2] != hd or t.shape[1] != k.shape[1] or t.stride(2) != 1:
            raise WswError("%s must be a [heads][depth][head_dim] view with unit stride in head_dim" % n)
    depth = k.shape[1]
    if scale is None:
        scale = 1.0 / float(hd) ** 0.5
    y = out if out is not None else torch.empty((heads, group, nq, hd), dtype=torch.float32, device=q.device)
    _check(load().wsw_attn_prefill_f16(q.data_ptr(), k.data_ptr(), v.data_ptr(), depth, heads, group, nq, hd,
                                       k.stride(1), k.stride(0), v.stride(1), v.stride(0), float(scale),
                                       y.data_ptr(), _stream(), _opts(opts)), "attn_prefill_f16")
    return y


def attn_prefill_q8_0_workspace_bytes(depth, heads, group, nq, window) -> int:
    return int(load().wsw_attn_prefill_q8_0_workspace_bytes(depth, heads, group, nq, window))


def attn_prefill_q8_0(q, kq, kd, vq, vd, window, scale=None, out=None, ws=None, opts=None):
    """Causal prefill attention over a q8_0 KV cache, dequantized and attended one window
    of `window` positions at a time (a multiple of 128), so the binary16 scratch holds one
    window of K and V.  q fp16 [heads][group][nq][head_dim]; kq, vq int8
    [depth][heads][head_dim]; kd, vd fp16 [depth][heads][head_dim/32].  ws: a uint8 device
    tensor of at least attn_prefill_q8_0_workspace_bytes(...) bytes, allocated if None.
    Returns out fp32 [heads][group][nq][head_dim]."""
    _dev(q, torch.float16, "q")
    for t, n, dt in ((kq, "kq", torch.int8), (vq, "vq", torch.int8), (kd, "kd", torch.float16),
                     (vd, "vd", torch.float16)):
        _dev(t, dt, n)
        if not t.is_contiguous():
            raise WswError("%s must be contiguous" % n)
    if q.dim() != 4 or not q.is_contiguous():
        raise WswError("q must be a contiguous [heads][group][nq][head_dim] tensor")
    heads, group, nq, hd = q.shape
    depth = kq.shape[0]
    if scale is None:
        scale = 1.0 / float(hd) ** 0.5
    y = out if out is not None else torch.empty((heads, group, nq, hd), dtype=torch.float32, device=q.device)
    if ws is None:
        ws = torch.empty(max(attn_prefill_q8_0_workspace_bytes(depth, heads, group, nq, window), 1),
                         dtype=torch.uint8, device=q.device)
    _check(load().wsw_attn_prefill_q8_0(q.data_ptr(), kq.data_ptr(), kd.data_ptr(), vq.data_ptr(), vd.data_ptr(),
                                        depth, heads, group, nq, hd, float(scale), int(window), ws.data_ptr(),
                                        ws.numel(), y.data_ptr(), _stream(), _opts(opts)), "attn_prefill_q8_0")
    return y


# ------------------------------------------------- a step around a paged KV cache ----

_FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # wsw_dtype
_I32, _I64, _F32, _U8, _Tensor = torch.int32, torch.int64, torch.float32, torch.uint8, torch.Tensor
_CACHES = {torch.float16: 1, torch.bfloat16: 2, torch.int8: 3}


def _home(t, name):
    """The device index of a call's first tensor.  It is the current device, whose stream the launch
    takes; the call's other tensors have to lie there, too."""
    dev = t.get_device() if isinstance(t, _Tensor) else -1
    if dev < 0:
        raise WswError("%s must be a CUDA tensor" % name)
    if dev == _current_device():
        return dev
    raise WswError("%s is on cuda:%d, which is not the current device" % (name, dev))


def _float_dev(t, name):
    """(type code, device index) of a call's first tensor."""
    code = _FLOATS.get(t.dtype) if isinstance(t, _Tensor) else None
    if code is None or not t.is_cuda:
        raise WswError("%s must be a CUDA tensor of float32, float16 or bfloat16" % name)
    dev = t.get_device()
    return code, dev if dev == _current_device() else _home(t, name)


def _on(t, dtype, name, dev):
    """What is wrong with a tensor that is not `dtype` on device `dev`."""
    _dev(t, dtype, name)
    if t.get_device() != dev:
        raise WswError("%s is on cuda:%d, the call's device is cuda:%d" % (name, t.get_device(), dev))


def _packed(t, dtype, name, dev, shape=None):
    """The address of a contiguous tensor of device `dev`."""
    if (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t.data_ptr()
    _on(t, dtype, name, dev)
    raise WswError("%s must be contiguous%s" % (name, "" if shape is None else " of shape %s" % (shape,)))


def _table(t, n, dev):
    """(address, pages per row, row stride) of a block table of n requests."""
    if not (isinstance(t, _Tensor) and t.dtype is _I32 and t.get_device() == dev):
        _on(t, _I32, "table", dev)
    shape = t.shape
    if len(shape) != 2 or shape[0] != n:
        raise WswError("table must be [requests][max_pages]")
    width = shape[1]
    if t.is_contiguous():
        return t.data_ptr(), width, width
    row, unit = t.stride()
    if (width > 1 and unit != 1) or (n > 1 and row < width):
        raise WswError("table must have unit stride in max_pages and rows that do not overlap")
    return t.data_ptr(), width, max(row, width)


def _elsewhere(kv, dev):
    raise WswError("the cache is on cuda:%d, the call's device is cuda:%d" % (kv._device, dev))


class PagedKV:
    """A paged KV cache of one layer: pages shared by all requests.  k and v: fp16, bf16 or
    (q8_0) int8, [pages][page_size][heads][head_dim] (layout "nhd") or
    [pages][heads][page_size][head_dim] ("hnd"), any strides but unit in head_dim and the
    same for both; kd and vd: the q8_0 scales, fp16, head_dim / 32 in the last dimension.
    page_size a power of two, head_dim 64, 128 or 256, all on one device.  The object holds the tensors."""

    def __init__(self, k, v, kd=None, vd=None, layout="nhd"):
        if layout not in ("nhd", "hnd"):
            raise WswError("layout must be 'nhd' or 'hnd'")
        dtype = _CACHES.get(k.dtype) if isinstance(k, torch.Tensor) and k.is_cuda else None
        if dtype is None:
            raise WswError("k must be a CUDA tensor of float16, bfloat16 or int8")
        _dev(v, k.dtype, "v")
        if k.dim() != 4 or k.stride(3) != 1 or k.shape != v.shape or k.stride() != v.stride():
            raise WswError("k and v must be 4-D views of equal shape and strides, unit in head_dim")
        pos, head = (1, 2) if layout == "nhd" else (2, 1)
        c = _CKv(k.data_ptr(), v.data_ptr(), None, None, k.shape[0], k.shape[pos], k.shape[head], k.shape[3],
                 k.stride(0), k.stride(pos), k.stride(head), 0, 0, 0, dtype)
        if dtype == 3:
            _dev(kd, torch.float16, "kd")
            _dev(vd, torch.float16, "vd")
            if (tuple(kd.shape) != tuple(k.shape[:3]) + (k.shape[3] // 32,) or kd.shape != vd.shape
                    or kd.stride() != vd.stride() or kd.stride(3) != 1):
                raise WswError("kd and vd must be [..][head_dim / 32] views with equal strides, unit in the last")
            c.kd, c.vd = kd.data_ptr(), vd.data_ptr()
            c.d_page_stride, c.d_pos_stride, c.d_head_stride = kd.stride(0), kd.stride(pos), kd.stride(head)
        elif kd is not None or vd is not None:
            raise WswError("kd and vd belong to an int8 cache")
        self.k, self.v, self.kd, self.vd, self.layout = k, v, kd, vd, layout
        self.num_pages, self.page_size, self.heads, self.head_dim = k.shape[0], k.shape[pos], k.shape[head], k.shape[3]
        self._device = k.get_device()
        for t, name in ((v, "v"), (kd, "kd"), (vd, "vd")):
            if t is not None and t.get_device() != self._device:
                raise WswError("%s must be on k's device" % name)
        self._c = c
        self._ref = ctypes.addressof(c)


class KvPlan(NamedTuple):
    positions: torch.Tensor  # int32 [tokens]
    slots: torch.Tensor      # int64 [tokens]
    cu: torch.Tensor         # int32 [requests + 1]
    seq_len: torch.Tensor    # int32 [requests], with the new tokens
    head: torch.Tensor       # int32 [1]


def kv_page_plan(seq_len, new_len, free_pages, head, table, page_size, tokens, out=None, err_flag=None, opts=None):
    """Pages, positions and cache slots of a step's new tokens, on the device.  Request r
    has seq_len[r] cached tokens and adds new_len[r]; the pages that it opens are taken
    from free_pages[head ..] and written into its row of table (int32 [requests][max_pages],
    updated in place).  `tokens` is the room for the step's tokens: rows beyond their sum
    get position and slot -1, as do the tokens of a request that does not fit (err_flag,
    an int32 device tensor, tells why: wsw.h).  Returns a KvPlan; out = such a tuple of
    tensors to fill, in which seq_len and head may be the arguments themselves."""
    dev = _home(seq_len, "seq_len")
    sp = _packed(seq_len, _I32, "seq_len", dev)
    n = seq_len.numel()
    tp, width, row = _table(table, n, dev)
    if out is None:
        where = seq_len.device
        out = KvPlan(torch.empty(tokens, dtype=torch.int32, device=where),
                     torch.empty(tokens, dtype=torch.int64, device=where),
                     torch.empty(n + 1, dtype=torch.int32, device=where), torch.empty_like(seq_len),
                     torch.empty_like(head))
    elif type(out) is not KvPlan:
        out = KvPlan(*out)
    positions, slots, cu, lens, head_out = out
    _check(load().wsw_kv_page_plan(
        sp, _packed(new_len, _I32, "new_len", dev, (n,)), n,
        _packed(free_pages, _I32, "free_pages", dev), free_pages.numel(),
        _packed(head, _I32, "head", dev, (1,)), page_size, tp, width, row, tokens,
        _packed(positions, _I32, "positions", dev, (tokens,)),
        _packed(slots, _I64, "slots", dev, (tokens,)), _packed(cu, _I32, "cu", dev, (n + 1,)),
        _packed(lens, _I32, "seq_len (out)", dev, (n,)), _packed(head_out, _I32, "head (out)", dev, (1,)),
        None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev), _raw_stream(dev), _opts(opts)),
        "kv_page_plan")
    return out


class RopeTable(NamedTuple):
    turns: torch.Tensor  # int64 (the bits of uint64) [rot_dim / 2]: turns per position, times 2^64
    mscale: float
    rot_dim: int


_ROPE_SCALING = {None: 0, "linear": 1, "ntk": 2, "by_parts": 3}


def rope_table(rot_dim, theta=10000.0, scaling=None, factor=1.0, original=0, freqs=None, device="cuda"):
    """The frequencies of rope_kv_write, made once per model: theta^(-2 i / rot_dim), scaled
    for contexts `factor` times the `original` length by "linear", "ntk" or "by_parts"
    (wsw.h), or freqs, the caller's own rot_dim / 2 radians per position."""
    if scaling not in _ROPE_SCALING:
        raise WswError("scaling must be one of None, 'linear', 'ntk', 'by_parts'")
    turns = (ctypes.c_uint64 * max(rot_dim // 2, 1))()
    mscale = ctypes.c_float()
    arr = None
    if freqs is not None:
        freqs = [float(f) for f in freqs]
        if len(freqs) != rot_dim // 2:
            raise WswError("freqs must have rot_dim / 2 values")
        arr = (ctypes.c_double * len(freqs))(*freqs)
    _check(load().wsw_rope_table(rot_dim, theta, _ROPE_SCALING[scaling], factor, original, arr, turns,
                                 ctypes.byref(mscale)), "rope_table")
    t = torch.tensor([v - (1 << 64) if v >> 63 else v for v in turns], dtype=torch.int64)
    return RopeTable(t.to(device), mscale.value, rot_dim)


def _rows3(t, dtype, name, dev, shape):
    """(address, token stride, head stride) of a [tokens][heads][head_dim] view."""
    if not (isinstance(t, _Tensor) and t.dtype is dtype and t.get_device() == dev):
        _on(t, dtype, name, dev)
    if t.shape != shape:
        raise WswError("%s must have shape %s" % (name, shape))
    tok, head, unit = t.stride()
    if unit != 1:
        raise WswError("%s must have unit stride in head_dim" % name)
    return t.data_ptr(), tok, head


def rope_kv_write(q, k, v, rope, positions, slots, kv, interleaved=False, out=None, err_flag=None, opts=None):
    """Rotates q [tokens][q_heads][head_dim] and k [tokens][kv_heads][head_dim] by their
    positions and writes k and v into the cache at their slots, in one pass; returns the
    rotated q (packed, q's dtype; out = the tensor to fill).  q, k, v: fp32, fp16 or bf16
    views with any token and head strides, for instance of one fused QKV row.  rope: a
    RopeTable; positions int32 and slots int64 [tokens], as kv_page_plan gives them.
    interleaved: pairs (2 i, 2 i + 1) instead of (i, i + rot_dim / 2)."""
    code, dev = _float_dev(q, "q")
    if q.dim() != 3:
        raise WswError("q must be a [tokens][q_heads][head_dim] view")
    dtype, shape = q.dtype, q.shape
    n, heads, hd = shape
    if hd != kv.head_dim:
        raise WswError("q must have the cache's head_dim")
    qt, qh, unit = q.stride()
    if unit != 1:
        raise WswError("q must have unit stride in head_dim")
    kp, kt, kh = _rows3(k, dtype, "k", dev, (n, kv.heads, hd))
    vp, vt, vh = _rows3(v, dtype, "v", dev, (n, kv.heads, hd))
    if out is None:
        out = torch.empty((n, heads, hd), dtype=dtype, device=q.device)
    rot = rope.rot_dim
    _check(load().wsw_rope_kv_write(
        q.data_ptr(), kp, vp, code, n, heads, qt, qh, kt, kh, vt, vh,
        _packed(rope.turns, _I64, "rope.turns", dev, (rot // 2,)), rot, rope.mscale, 1 if interleaved else 0,
        _packed(positions, _I32, "positions", dev, (n,)), _packed(slots, _I64, "slots", dev, (n,)),
        _packed(out, dtype, "out", dev, shape), kv._ref if kv._device == dev else _elsewhere(kv, dev),
        None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev), _raw_stream(dev), _opts(opts)),
        "rope_kv_write")
    return out


def attn_paged_decode_workspace_bytes(requests, q_heads, kv_heads, head_dim) -> int:
    return int(load().wsw_attn_paged_decode_workspace_bytes(requests, q_heads, kv_heads, head_dim))


def attn_paged_decode(q, kv, table, lens, scale=None, softcap=0.0, window=0, slopes=None, out=None, lse=None,
                      err_flag=None, ws=None, opts=None):
    """Attention of one new token per request over the paged cache kv (a PagedKV).
    q [requests][q_heads][head_dim] (contiguous, fp32, fp16 or bf16; q_heads a multiple of
    the cache's heads); table int32 [requests][max_pages]; lens int32 [requests], the
    cached tokens with the new one.  scale defaults to 1 / sqrt(head_dim); softcap > 0
    caps the scores by softcap * tanh(score / softcap); window > 0 shows only the last
    `window` positions; slopes fp32 [q_heads] subtracts slope * distance.  Returns out
    (q's dtype); lse, an fp32 [requests][q_heads] tensor, receives the log of the sum of
    exponentials.  A request of length 0 gives zeros and -inf.  ws: a uint8 device tensor
    of at least attn_paged_decode_workspace_bytes(...) bytes, zero-filled before its first
    use (every call leaves it ready for the next), allocated if None."""
    code, dev = _float_dev(q, "q")
    if q.dim() != 3 or not q.is_contiguous():
        raise WswError("q must be a contiguous [requests][q_heads][head_dim] tensor")
    shape = q.shape
    n, heads, hd = shape
    if hd != kv.head_dim or heads % kv.heads != 0:
        raise WswError("q must have the cache's head_dim and a multiple of its heads")
    tp, width, row = _table(table, n, dev)
    if scale is None:
        scale = 1.0 / float(hd) ** 0.5
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = torch.zeros(attn_paged_decode_workspace_bytes(n, heads, kv.heads, hd), dtype=torch.uint8,
                         device=q.device)
    _check(load().wsw_attn_paged_decode(
        q.data_ptr(), code, n, heads, kv._ref if kv._device == dev else _elsewhere(kv, dev), tp, width, row,
        _packed(lens, _I32, "lens", dev, (n,)), scale, softcap, window,
        None if slopes is None else _packed(slopes, _F32, "slopes", dev, (heads,)),
        _packed(out, q.dtype, "out", dev, shape),
        None if lse is None else _packed(lse, _F32, "lse", dev, (n, heads)),
        None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev),
        _packed(ws, _U8, "ws", dev), ws.numel(), _raw_stream(dev), _opts(opts)), "attn_paged_decode")
    return out


class TokenLogprobs(NamedTuple):
    logprob: Optional[torch.Tensor]  # fp32 [rows] (None without tokens)
    rank: Optional[torch.Tensor]     # int32 [rows]
    lse: torch.Tensor                # fp32 [rows]
    entropy: torch.Tensor            # fp32 [rows]
    top_logprob: torch.Tensor        # fp32 [rows][top]
    top_id: torch.Tensor             # int32 [rows][top]


def token_logprobs_workspace_bytes(rows, vocab, top) -> int:
    return int(load().wsw_token_logprobs_workspace_bytes(rows, vocab, top))


def token_logprobs_out(rows, top, tokens=True, device="cuda") -> TokenLogprobs:
    """Tensors for token_logprobs to fill."""
    f = lambda *s: torch.empty(s, dtype=torch.float32, device=device)  # noqa: E731
    i = lambda *s: torch.empty(s, dtype=torch.int32, device=device)  # noqa: E731
    return TokenLogprobs(f(rows) if tokens else None, i(rows) if tokens else None, f(rows), f(rows), f(rows, top),
                         i(rows, top))


def token_logprobs(logits, tokens=None, top=0, scale=1.0, out=None, ws=None, opts=None):
    """Per row of logits [rows][vocab] (fp32, fp16 or bf16, any row stride), with y = scale *
    logits: the log probability and rank of its token (int32 [rows], or None), the log of
    the sum of exponentials, the entropy, and the `top` (at most 32) most likely tokens
    with their log probabilities, equal ones by the lower id.  Returns a TokenLogprobs
    (out = one to fill).  ws: a uint8 device tensor of at least
    token_logprobs_workspace_bytes(...) bytes, zero-filled before its first use, allocated
    if None."""
    code, dev = _float_dev(logits, "logits")
    rows, vocab, ld = _rowmajor(logits, "logits")
    if out is None:
        out = token_logprobs_out(rows, top, tokens is not None, logits.device)
    logprob, rank, lse, entropy, top_logprob, top_id = out
    tp = lp = rp = bp = ip = wp = None
    if tokens is not None:
        tp = _packed(tokens, _I32, "tokens", dev, (rows,))
        lp = _packed(logprob, _F32, "logprob", dev, (rows,))
        rp = _packed(rank, _I32, "rank", dev, (rows,))
    if top:
        bp = _packed(top_logprob, _F32, "top_logprob", dev, (rows, top))
        ip = _packed(top_id, _I32, "top_id", dev, (rows, top))
    if ws is None:
        need = token_logprobs_workspace_bytes(rows, vocab, top)
        if need:
            ws = torch.zeros(need, dtype=torch.uint8, device=logits.device)
    if ws is not None:
        wp = _packed(ws, _U8, "ws", dev)
    _check(load().wsw_token_logprobs(
        logits.data_ptr(), code, rows, vocab, ld, tp, scale, top, lp, rp,
        _packed(lse, _F32, "lse", dev, (rows,)), _packed(entropy, _F32, "entropy", dev, (rows,)), bp, ip,
        wp, 0 if wp is None else ws.numel(), _raw_stream(dev), _opts(opts)), "token_logprobs")
    return out


# ------------------------------------------------------ rows that continue one prompt ----

class _Held:
    """Tensors that a program makes once and passes to call after call: checked here, held by the
    object, their addresses kept."""
    __slots__ = ("_device", "_at")
    _names = ()

    def __iter__(self):
        return iter([getattr(self, n) for n in self._names])

    def __setattr__(self, name, value):
        if name in self._names and hasattr(self, name):
            raise AttributeError("the tensors of a %s stay those that it was made with" % type(self).__name__)
        object.__setattr__(self, name, value)

    def _hold(self, first, checks):
        """checks: (tensor, type, name, shape) of each, all on the first one's device."""
        if not isinstance(first, _Tensor) or not first.is_cuda:
            raise WswError("%s must be a CUDA tensor" % checks[0][2])
        self._device = first.get_device()
        self._at = tuple([None if t is None else _packed(t, d, n, self._device, s) for t, d, n, s in checks])

    def _on_device(self, dev):
        if self._device != dev:
            raise WswError("the %s is on cuda:%d, the call's device is cuda:%d" % (type(self).__name__, self._device, dev))
        return self._at


class PageCopies(_Held):
    """Copies of pages for kv_page_copy: the first `count` (int32 [1]) of src and dst (int32 [most]) are
    there, of fill (int32 [most], or None: whole pages) positions each."""
    __slots__ = ("src", "dst", "fill", "count", "most")
    _names = ("src", "dst", "fill", "count")

    def __init__(self, src, dst, fill, count):
        self.src, self.dst, self.fill, self.count = src, dst, fill, count
        self.most = src.numel() if isinstance(src, _Tensor) else 0
        n = (self.most,)
        self._hold(src, [(src, _I32, "copies.src", n), (dst, _I32, "copies.dst", n), (fill, _I32, "copies.fill", n),
                         (count, _I32, "copies.count", (1,))])


class KvFork(_Held):
    """What kv_page_fork fills: table int32 [children][max_pages], seq_len int32 [children], head int32
    [1], copies (a PageCopies with room for one of each child)."""
    __slots__ = ("table", "seq_len", "head", "copies", "_table")
    _names = ("table", "seq_len", "head", "copies")

    def __init__(self, table, seq_len, head, copies):
        self.table, self.seq_len, self.head, self.copies = table, seq_len, head, copies
        self._hold(seq_len, [(seq_len, _I32, "seq_len (out)", None), (head, _I32, "head (out)", (1,))])
        self._table = _table(table, seq_len.numel(), self._device)
        if copies.fill is None or copies.most != seq_len.numel():
            raise WswError("copies must have room for one copy of each child")
        self._at += copies._on_device(self._device)


def _page_copies(n, device, fill):
    i = lambda m: torch.empty(m, dtype=torch.int32, device=device)  # noqa: E731
    return PageCopies(i(n), i(n), i(n) if fill else None, i(1))


def kv_page_fork(parent, seq_len, free_pages, head, table, page_size, out=None, err_flag=None, opts=None):
    """Block table rows of children (beams, samples) from their parents' rows: row i continues
    row parent[i] (int32 [children]; -1: an empty row) of table, whose lengths are seq_len.
    Full pages are shared; all but a row's lowest child get a page from free_pages[head ..]
    for a partly filled last page, and an entry in copies, which kv_page_copy carries out
    before the next tokens are written.  Returns a KvFork; out = one to fill, in which table,
    seq_len and head may be the arguments themselves.  err_flag: wsw.h."""
    dev = _home(parent, "parent")
    pp = _packed(parent, _I32, "parent", dev)
    n = parent.numel()
    sp = _packed(seq_len, _I32, "seq_len", dev)
    rows = seq_len.numel()
    tp, width, row = _table(table, rows, dev)
    if out is None:
        out = KvFork(table.new_full((n, width), -1), parent.new_empty(n), torch.empty_like(head),
                     _page_copies(n, parent.device, True))
    lens_out, head_out, src, dst, fill, count = out._on_device(dev)
    op, out_width, out_row = out._table
    if out_width != width or out.copies.most != n:
        raise WswError("the new table must be [children][max_pages], with the old one's max_pages")
    _check(load().wsw_kv_page_fork(
        pp, n, sp, rows, _packed(free_pages, _I32, "free_pages", dev), free_pages.numel(),
        _packed(head, _I32, "head", dev, (1,)), page_size, tp, width, row, op, out_row, lens_out, head_out, src, dst, fill,
        count, None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev), _raw_stream(dev), _opts(opts)),
        "kv_page_fork")
    return out


def kv_page_copy(copies, caches, err_flag=None, opts=None):
    """Carries out copies (a PageCopies, as kv_page_fork and kv_page_compact give them) in each
    of caches, the PagedKV of every layer that shares the block table, in one launch for up to 32
    of them.  A copy that names a page outside a cache is left out there (err_flag, bit 0)."""
    dev = copies._device
    if dev != _current_device():
        _home(copies.src, "copies.src")
    src, dst, fill, count = copies._at
    caches = (caches,) if isinstance(caches, PagedKV) else caches
    for kv in caches:
        if kv._device != dev:
            _elsewhere(kv, dev)
    refs = (_p * max(len(caches), 1))(*[kv._ref for kv in caches])
    _check(load().wsw_kv_page_copy(
        src, dst, fill, count, copies.most, refs, len(caches),
        None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev), _raw_stream(dev), _opts(opts)),
        "kv_page_copy")


class KvCompact(_Held):
    """What kv_page_compact fills: table int32 [requests][max_pages], free_pages int32 [num_pages] (the free
    ones from head, int32 [1], on), copies (a PageCopies with room for max_moves whole pages)."""
    __slots__ = ("table", "free_pages", "head", "copies", "_table")
    _names = ("table", "free_pages", "head", "copies")

    def __init__(self, table, free_pages, head, copies):
        self.table, self.free_pages, self.head, self.copies = table, free_pages, head, copies
        self._hold(free_pages, [(free_pages, _I32, "free_pages", None), (head, _I32, "head", (1,))])
        self._table = _table(table, table.shape[0] if isinstance(table, _Tensor) and table.dim() == 2 else -1, self._device)
        if copies.fill is not None:
            raise WswError("whole pages move: copies.fill must be None")
        self._at += copies._on_device(self._device)


def kv_page_compact_workspace_bytes(num_pages) -> int:
    return int(load().wsw_kv_page_compact_workspace_bytes(num_pages))


def kv_page_compact(seq_len, table, page_size, num_pages, held=None, max_moves=0, out=None, err_flag=None, ws=None,
                    opts=None):
    """The free list of a pool of num_pages pages from what the rows of table list (and held,
    uint8 [num_pages], marks): with max_moves = 0 it only frees what no row lists any more; else
    up to max_moves live pages behind the others also move into the gaps, the table follows and
    copies names the pages, which kv_page_copy has to copy before the cache is used again.
    Returns a KvCompact, whose table is `table` itself, updated in place; out = one to fill, in
    which table may lie elsewhere (it is written when max_moves is not 0).  ws: a uint8 device tensor of at least
    kv_page_compact_workspace_bytes(num_pages) bytes, allocated if None."""
    dev = _home(seq_len, "seq_len")
    sp = _packed(seq_len, _I32, "seq_len", dev)
    n = seq_len.numel()
    tp, width, row = _table(table, n, dev)
    if out is None:
        out = KvCompact(table, torch.full((num_pages,), -1, dtype=torch.int32, device=seq_len.device),
                        torch.empty(1, dtype=torch.int32, device=seq_len.device),
                        _page_copies(max_moves, seq_len.device, False))
    free_pages, head, src, dst, _, count = out._on_device(dev)
    op, out_width, out_row = out._table
    if out_width != width or out.table.shape[0] != n or out.free_pages.numel() != num_pages or out.copies.most != max_moves:
        raise WswError("out must have a table of the old one's shape, num_pages free pages and max_moves copies")
    if ws is None:
        ws = torch.empty(kv_page_compact_workspace_bytes(num_pages), dtype=torch.uint8, device=seq_len.device)
    _check(load().wsw_kv_page_compact(
        sp, n, tp, width, row, page_size, num_pages,
        None if held is None else _packed(held, _U8, "held", dev, (num_pages,)), max_moves, op, out_row, free_pages, head,
        src, dst, count, None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev),
        _packed(ws, _U8, "ws", dev), ws.numel(), _raw_stream(dev), _opts(opts)), "kv_page_compact")
    return out


class BeamStep(_Held):
    """What beam_select fills, each [requests][beams]: parent int32 (rows of the logits), token int32 and
    score fp32 of the next beams, and the same of the candidates that end."""
    __slots__ = ("parent", "token", "score", "end_parent", "end_token", "end_score", "_shape")
    _names = ("parent", "token", "score", "end_parent", "end_token", "end_score")

    def __init__(self, parent, token, score, end_parent, end_token, end_score):
        self.parent, self.token, self.score = parent, token, score
        self.end_parent, self.end_token, self.end_score = end_parent, end_token, end_score
        self._shape = parent.shape if isinstance(parent, _Tensor) else None
        self._hold(parent, [(t, _F32 if n.endswith("score") else _I32, n, self._shape) for n, t in zip(self._names, self)])


def beam_select_workspace_bytes(requests, beams, vocab, ends=0) -> int:
    return int(load().wsw_beam_select_workspace_bytes(requests, beams, vocab, ends))


def beam_select_out(requests, beams, device="cuda") -> BeamStep:
    """Tensors for beam_select to fill."""
    return BeamStep(*[torch.empty((requests, beams), dtype=t, device=device) for t in (_I32, _I32, _F32) * 2])


def beam_select(logits, scores, end_tokens=(), scale=1.0, out=None, ws=None, opts=None):
    """The next beams of every request.  logits [requests * beams][vocab] (fp32, fp16 or bf16, any
    row stride), scores fp32 [requests][beams] the beams' log probabilities so far (-inf: no
    beam).  Of all candidates (beam, token), ranked by score + log softmax(scale * logits), the first
    `beams` whose token is not one of end_tokens (at most 8) are the next beams; those that
    end and have fewer than `beams` before them are reported beside them.  beams * (1 + number of
    end tokens) <= 32.  Returns a BeamStep (out = one to fill), -1 and -inf where there are fewer
    candidates; its parent, flattened, is kv_page_fork's.  ws: a uint8 device tensor of at
    least beam_select_workspace_bytes(...) bytes, zero-filled before its first use, allocated if
    None."""
    code, dev = _float_dev(logits, "logits")
    rows, vocab, ld = _rowmajor(logits, "logits")
    sp = _packed(scores, _F32, "scores", dev)
    shape = scores.shape
    if len(shape) != 2 or shape[0] * shape[1] != rows:
        raise WswError("scores must be [requests][beams], logits [requests * beams][vocab]")
    n, beams = shape
    ends = (_i32 * len(end_tokens))(*end_tokens) if end_tokens else None
    if ends and ends[:] != list(end_tokens):
        raise WswError("end tokens must fit into 32 bits")
    if out is None:
        out = beam_select_out(n, beams, logits.device)
    if ws is None:
        ws = torch.zeros(beam_select_workspace_bytes(n, beams, vocab, len(end_tokens)), dtype=torch.uint8,
                         device=logits.device)
    at = out._on_device(dev)
    if out._shape != shape:
        raise WswError("out must be [requests][beams] as scores")
    _check(load().wsw_beam_select(
        logits.data_ptr(), code, n, beams, vocab, ld, sp, ends, len(end_tokens), scale, *at,
        _packed(ws, _U8, "ws", dev), ws.numel(), _raw_stream(dev), _opts(opts)), "beam_select")
    return out


def attn_paged_prefix_workspace_bytes(requests, groups, q_heads, kv_heads, head_dim) -> int:
    return int(load().wsw_attn_paged_prefix_workspace_bytes(requests, groups, q_heads, kv_heads, head_dim))


def attn_paged_prefix(q, kv, table, lens, groups, prefix, scale=None, softcap=0.0, slopes=None, out=None, lse=None,
                      err_flag=None, ws=None, share=False, opts=None):
    """attn_paged_decode for a batch in which groups of requests share a prefix, read once for each
    group: requests groups[g] .. groups[g + 1] - 1 (int32 [n + 1], ascending) have the same keys
    and values at their first prefix[g] (int32 [n]) positions.  head_dim 64 or 128, no window; the
    other arguments and the result are attn_paged_decode's.  Small batches (128 MB of cached
    positions by the table's size) go attn_paged_decode's way unless share is true.  ws: a uint8
    device tensor of at least attn_paged_prefix_workspace_bytes(...) bytes, zero-filled before its
    first use (every call leaves it ready for the next), allocated if None."""
    code, dev = _float_dev(q, "q")
    if q.dim() != 3 or not q.is_contiguous():
        raise WswError("q must be a contiguous [requests][q_heads][head_dim] tensor")
    shape = q.shape
    n, heads, hd = shape
    if hd != kv.head_dim or heads % kv.heads != 0:
        raise WswError("q must have the cache's head_dim and a multiple of its heads")
    tp, width, row = _table(table, n, dev)
    pp = _packed(prefix, _I32, "prefix", dev)
    count = prefix.numel()
    if scale is None:
        scale = 1.0 / float(hd) ** 0.5
    if out is None:
        out = torch.empty_like(q)
    if ws is None:
        ws = torch.zeros(attn_paged_prefix_workspace_bytes(n, count, heads, kv.heads, hd), dtype=torch.uint8,
                         device=q.device)
    _check(load().wsw_attn_paged_prefix(
        q.data_ptr(), code, n, heads, kv._ref if kv._device == dev else _elsewhere(kv, dev), tp, width, row,
        _packed(lens, _I32, "lens", dev, (n,)), _packed(groups, _I32, "groups", dev, (count + 1,)), count, pp,
        1 if share else 0, scale, softcap, None if slopes is None else _packed(slopes, _F32, "slopes", dev, (heads,)),
        _packed(out, q.dtype, "out", dev, shape),
        None if lse is None else _packed(lse, _F32, "lse", dev, (n, heads)),
        None if err_flag is None else _packed(err_flag, _I32, "err_flag", dev),
        _packed(ws, _U8, "ws", dev), ws.numel(), _raw_stream(dev), _opts(opts)), "attn_paged_prefix")
    return out


def upload_padded(W: torch.Tensor, ld: int, device=None) -> torch.Tensor:
    """Copy a [M][K] weight into a new [M][ld] device buffer whose pad columns are
    zero (so they can never hold NaNs) and return the [M][K] view with row stride ld.
    Padding the row stride by one cache line breaks cache-set aliasing of rows whose
    byte length is a multiple of the set stride."""
    M, K = W.shape
    if ld < K:
        raise WswError("ld must be >= K")
    dev = device if device is not None else (W.device if W.is_cuda else torch.device("cuda"))
    buf = torch.zeros((M, ld), dtype=W.dtype, device=dev)
    buf[:, :K].copy_(W, non_blocking=True)
    return buf[:, :K]
