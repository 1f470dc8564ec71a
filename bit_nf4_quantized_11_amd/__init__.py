"""Python binding of libqlora (QLoRA linear layer on MI355X / gfx950).

Thin argument marshalling over the C ABI in include/qlora.h: each function has
the name of the C entry point it calls.  torch is used for device memory and
streams only; every computation runs in the library's HIP kernels.  There is no
CPU fallback: without the built library or a GPU the calls raise.
"""
from __future__ import annotations

import ctypes as C
import struct
from dataclasses import dataclass

import torch

from . import _lib

__all__ = [
    "NF4Weight", "QLoRAError", "nf4_alloc", "qlora_nf4_codebook", "qlora_codebook_table", "qlora_nf4_sizes",
    "CODEBOOK_NF4", "CODEBOOK_FP4", "CODEBOOK_INT4", "CODEBOOKS", "qlora_quantize_workspace",
    "qlora_fwd_workspace", "qlora_bwd_workspace", "qlora_quantize_nf4", "qlora_dequant", "qlora_linear_fwd",
    "qlora_linear_bwd", "qlora_merge_adapter", "qlora_adamw_step", "qlora_profile_enable", "qlora_profile_read", "lib",
    "KVCache", "KVBatch", "kv_alloc", "qlora_qk_norm_rope", "qlora_qk_norm_rope_bwd_workspace",
    "qlora_qk_norm_rope_bwd", "qlora_kv_sizes", "qlora_kv_write", "qlora_kv_read", "qlora_kv_attn_workspace",
    "qlora_kv_attn", "qlora_rms_norm", "qlora_rms_norm_bwd_workspace", "qlora_rms_norm_bwd", "ACTIVATIONS",
    "qlora_gated_workspace", "qlora_gated_fwd", "qlora_gated_bwd", "qlora_token_logprob_workspace", "qlora_token_logprob",
    "qlora_token_logprob_bwd",
]


class QLoRAError(RuntimeError):
    pass


# qlora_codebook values: the 16-entry table a quantized weight's codes index
CODEBOOK_NF4, CODEBOOK_FP4, CODEBOOK_INT4 = 0, 1, 2
CODEBOOKS = {"nf4": CODEBOOK_NF4, "fp4": CODEBOOK_FP4, "int4": CODEBOOK_INT4}


def lib():
    return _lib.load()


def _check(status: int, what: str):
    if status != 0:
        msg = lib().qlora_status_str(status).decode()
        raise QLoRAError(f"{what}: {_lib.STATUS.get(status, status)} ({msg})")


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _bf16(t, name):
    if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
        raise QLoRAError(f"{name} must be a contiguous bf16 tensor on the GPU")
    return t


@dataclass
class NF4Weight:
    """A quantized [rows][cols] weight: caller-owned device buffers (torch tensors)."""
    rows: int
    cols: int
    double_quant: bool
    codes: torch.Tensor      # uint8 [32 per 64 weights, padded to whole blocks]
    absmax: torch.Tensor     # uint8 [nblk] (double quant) or float32 [nblk]
    c1: torch.Tensor | None  # float32 [nsup]
    mu: torch.Tensor | None  # float32 [1]
    codebook: int = CODEBOOK_NF4
    block: int = 64          # weights per constant: 32, 64, 128 or 256

    def desc(self) -> _lib.qlora_nf4:
        return _lib.qlora_nf4(self.rows, self.cols, int(self.double_quant), int(self.codebook), int(self.block), 0,
                              self.codes.data_ptr(), self.absmax.data_ptr(),
                              self.c1.data_ptr() if self.c1 is not None else None,
                              self.mu.data_ptr() if self.mu is not None else None)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.absmax, self.c1, self.mu) if t is not None)


def qlora_nf4_codebook():
    """(levels[16], thresholds[15]) as Python floats, computed by the library."""
    lv = (C.c_float * 16)()
    th = (C.c_float * 15)()
    _check(lib().qlora_nf4_codebook(lv, th), "qlora_nf4_codebook")
    return list(lv), list(th)


def qlora_codebook_table(codebook: int = CODEBOOK_NF4):
    """(levels[16], thresholds[15]) of any codebook, computed by the library."""
    lv = (C.c_float * 16)()
    th = (C.c_float * 15)()
    _check(lib().qlora_codebook_table(int(codebook), lv, th), "qlora_codebook_table")
    return list(lv), list(th)


def qlora_nf4_sizes(rows: int, cols: int, double_quant: bool = True, block: int = 64):
    out = [C.c_size_t() for _ in range(4)]
    _check(lib().qlora_nf4_sizes(rows, cols, int(double_quant), int(block), *[C.byref(o) for o in out]),
           "qlora_nf4_sizes")
    return tuple(o.value for o in out)


def qlora_quantize_workspace(rows: int, cols: int, double_quant: bool = True, block: int = 64) -> int:
    return lib().qlora_quantize_workspace(rows, cols, int(double_quant), int(block))


def qlora_fwd_workspace(M: int, d_in: int, d_out: int, r: int) -> int:
    return lib().qlora_fwd_workspace(M, d_in, d_out, r)


def qlora_bwd_workspace(M: int, d_in: int, d_out: int, r: int) -> int:
    return lib().qlora_bwd_workspace(M, d_in, d_out, r)


def _workspace(nbytes: int, device, ws):
    if nbytes == 0:
        return None
    if ws is not None and ws.numel() * ws.element_size() >= nbytes:
        return ws
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def nf4_alloc(rows: int, cols: int, double_quant: bool = True, device="cuda", codebook: int = CODEBOOK_NF4,
              block: int = 64) -> NF4Weight:
    cb, ab, c1b, mub = qlora_nf4_sizes(rows, cols, double_quant, block)
    codes = torch.empty(cb, dtype=torch.uint8, device=device)
    if double_quant:
        absmax = torch.empty(ab, dtype=torch.uint8, device=device)
        c1 = torch.empty(c1b // 4, dtype=torch.float32, device=device)
        mu = torch.empty(1, dtype=torch.float32, device=device)
    else:
        absmax = torch.empty(ab // 4, dtype=torch.float32, device=device)
        c1 = mu = None
    return NF4Weight(rows, cols, double_quant, codes, absmax, c1, mu, codebook, block)


def qlora_quantize_nf4(W: torch.Tensor, double_quant: bool = True, out: NF4Weight | None = None,
                       workspace: torch.Tensor | None = None, stream=None, codebook: int = CODEBOOK_NF4,
                       block: int = 64) -> NF4Weight:
    """Quantize a bf16 [rows][cols] weight (any 2-D shape) to 4-bit codes of `codebook`
    (NF4 by default) with one absmax per `block` weights (+ double quantization).  With
    `out` given, its own codebook and block size are used."""
    _bf16(W, "W")
    rows, cols = (W.shape[0], W.shape[1]) if W.dim() == 2 else (1, W.numel())
    if out is None:
        out = nf4_alloc(rows, cols, double_quant, W.device, codebook, block)
    ws = _workspace(qlora_quantize_workspace(rows, cols, out.double_quant, out.block), W.device, workspace)
    d = out.desc()
    _check(lib().qlora_quantize_nf4(_ptr(W), rows, cols, C.byref(d), _ptr(ws),
                                    0 if ws is None else ws.numel(), _stream(stream)), "qlora_quantize_nf4")
    return out


def qlora_dequant(w: NF4Weight, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.bfloat16, device=w.codes.device)
    d = w.desc()
    _check(lib().qlora_dequant(C.byref(d), _ptr(out), _stream(stream)), "qlora_dequant")
    return out


def qlora_linear_fwd(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: float,
                     Y: torch.Tensor | None = None, save_T: bool = True, T_save: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Y = X deq(W)^T + scale (X A) B.  Returns (Y, T) with T = bf16(X A) or None."""
    _bf16(X, "X"); _bf16(A, "A"); _bf16(B, "B")
    M = X.shape[0]
    r = A.shape[1]
    if Y is None:
        Y = torch.empty((M, w.rows), dtype=torch.bfloat16, device=X.device)
    if save_T and T_save is None:
        T_save = torch.empty((M, r), dtype=torch.bfloat16, device=X.device)
    ws = _workspace(qlora_fwd_workspace(M, w.cols, w.rows, r), X.device, workspace)
    d = w.desc()
    _check(lib().qlora_linear_fwd(_ptr(X), M, C.byref(d), _ptr(A), _ptr(B), r, float(scale), _ptr(Y),
                                  _ptr(T_save if save_T else None), _ptr(ws), 0 if ws is None else ws.numel(),
                                  _stream(stream)), "qlora_linear_fwd")
    return Y, (T_save if save_T else None)


def qlora_linear_fwd_noalloc(X: torch.Tensor, w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: float,
                             Y: torch.Tensor, T_save: torch.Tensor | None = None, stream=None):
    """The forward with the library's own scratch array (no workspace, nothing allocated);
    Y (and T_save, if given) must be allocated by the caller.  Returns (Y, T_save)."""
    _bf16(X, "X"); _bf16(A, "A"); _bf16(B, "B")
    d = w.desc()
    _check(lib().qlora_linear_fwd_noalloc(_ptr(X), X.shape[0], C.byref(d), _ptr(A), _ptr(B), A.shape[1],
                                          float(scale), _ptr(Y), _ptr(T_save), _stream(stream)),
           "qlora_linear_fwd_noalloc")
    return Y, T_save


def qlora_linear_bwd(dY: torch.Tensor, X: torch.Tensor, T_saved: torch.Tensor | None, w: NF4Weight,
                     A: torch.Tensor, B: torch.Tensor, scale: float, need_dX: bool = True,
                     dX: torch.Tensor | None = None, dA: torch.Tensor | None = None, dB: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream=None):
    """Returns (dX or None, dA fp32 [in][r], dB fp32 [r][out]); no gradient for W."""
    _bf16(dY, "dY"); _bf16(X, "X"); _bf16(A, "A"); _bf16(B, "B")
    M = X.shape[0]
    r = A.shape[1]
    dev = X.device
    if need_dX and dX is None:
        dX = torch.empty((M, w.cols), dtype=torch.bfloat16, device=dev)
    if dA is None:
        dA = torch.empty((w.cols, r), dtype=torch.float32, device=dev)
    if dB is None:
        dB = torch.empty((r, w.rows), dtype=torch.float32, device=dev)
    ws = _workspace(qlora_bwd_workspace(M, w.cols, w.rows, r), dev, workspace)
    d = w.desc()
    _check(lib().qlora_linear_bwd(_ptr(dY), _ptr(X), _ptr(T_saved), M, C.byref(d), _ptr(A), _ptr(B), r,
                                  float(scale), _ptr(dX if need_dX else None), _ptr(dA), _ptr(dB), _ptr(ws),
                                  0 if ws is None else ws.numel(), _stream(stream)), "qlora_linear_bwd")
    return (dX if need_dX else None), dA, dB


def qlora_merge_adapter(w: NF4Weight, A: torch.Tensor, B: torch.Tensor, scale: float,
                        out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 [rows][cols] weight deq(W) + scale (A B)^T (requantize it with qlora_quantize_nf4)."""
    _bf16(A, "A"); _bf16(B, "B")
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.bfloat16, device=A.device)
    d = w.desc()
    _check(lib().qlora_merge_adapter(C.byref(d), _ptr(A), _ptr(B), A.shape[1], float(scale), _ptr(out),
                                     _stream(stream)), "qlora_merge_adapter")
    return out


def qlora_adamw_step(param: torch.Tensor, grad: torch.Tensor, m: torch.Tensor, v: torch.Tensor, step: int,
                     lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                     weight_decay: float = 0.0, param_bf16: torch.Tensor | None = None, stream=None):
    """One AdamW step in place on fp32 `param`, `m`, `v` (same number of elements as the
    fp32 `grad`); writes bf16(param) into `param_bf16` when given."""
    n = param.numel()
    for t, name in ((param, "param"), (grad, "grad"), (m, "m"), (v, "v")):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n:
            raise QLoRAError(f"{name} must be a contiguous float32 tensor of {n} elements")
    if param_bf16 is not None and (param_bf16.dtype != torch.bfloat16 or param_bf16.numel() != n
                                   or not param_bf16.is_contiguous()):
        raise QLoRAError("param_bf16 must be a contiguous bf16 tensor of the same size")
    _check(lib().qlora_adamw_step(_ptr(param), _ptr(param_bf16), _ptr(grad), _ptr(m), _ptr(v), n, int(step),
                                  float(lr), float(beta1), float(beta2), float(eps), float(weight_decay),
                                  _stream(stream)), "qlora_adamw_step")


def _page_args(dev: torch.Tensor, host: torch.Tensor):
    if not dev.is_cuda or host.is_cuda or not host.is_pinned():
        raise QLoRAError("paging copies between a device tensor and a pinned host tensor")
    if not dev.is_contiguous() or not host.is_contiguous() or dev.nbytes != host.nbytes:
        raise QLoRAError("paging needs two contiguous tensors of the same size")


def qlora_state_page_out(dev: torch.Tensor, host: torch.Tensor, stream=None) -> torch.Tensor:
    """Copy optimizer state from device memory into a pinned host tensor (asynchronous on the
    stream).  Returns `host`."""
    _page_args(dev, host)
    _check(lib().qlora_state_page_out(_ptr(dev), _ptr(host), dev.nbytes, _stream(stream)), "qlora_state_page_out")
    return host


def qlora_state_page_in(host: torch.Tensor, dev: torch.Tensor, stream=None) -> torch.Tensor:
    """Copy optimizer state from a pinned host tensor back into device memory (asynchronous
    on the stream).  Returns `dev`."""
    _page_args(dev, host)
    _check(lib().qlora_state_page_in(_ptr(host), _ptr(dev), dev.nbytes, _stream(stream)), "qlora_state_page_in")
    return dev


# ---- between the projections: head norms and rotation, the 4-bit key/value cache, its attention --------
# These calls' kernels can take less time than a few lines of Python, so what every call does is kept short: the
# stream's handle alone (a torch Stream object costs 2 us to make), no context where none is needed, and the views of
# head tensors (qlora_heads) packed as bytes rather than made as ctypes structures.
_view = struct.Struct("<Qqqii").pack   # data, row_stride, head_stride, heads, reserved


def _launch(t: torch.Tensor, stream, run):
    """run(handle of the stream), with the tensor's device current and, where the caller named a stream, that
    stream current too, so that what `run` allocates belongs to it and is not reused before its kernels are done."""
    dev = t.device
    index = dev.index
    if stream is None and index == torch._C._cuda_getDevice():
        return run(torch._C._cuda_getCurrentRawStream(index))
    if stream is not None and stream.device != dev:
        raise QLoRAError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev), torch.cuda.stream(stream):
        return run(torch._C._cuda_getCurrentRawStream(index))


def _need(t, dtype, device, name, shape=None):
    """A contiguous tensor of `dtype` on `device` (and of `shape`)."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise QLoRAError(f"{name} must be a contiguous {dtype} tensor on {device}")
    if shape is not None and t.shape != shape:
        raise QLoRAError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return t


def _heads(t: torch.Tensor, name: str, device=None, shape=None) -> bytes:
    """The view of a bf16 [rows][heads][head_dim] tensor, any strides with a dense last dimension."""
    strides = t.stride()
    if t.dtype is not torch.bfloat16 or len(strides) != 3 or strides[2] != 1 or not t.is_cuda:
        raise QLoRAError(f"{name} must be a bf16 [rows][heads][head_dim] tensor on the GPU, dense along head_dim")
    if device is not None and t.device != device:
        raise QLoRAError(f"{name} must be on {device}")
    if shape is not None and t.shape != shape:
        raise QLoRAError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return _view(t.data_ptr(), strides[0], strides[1], t.size(1), 0)


def _out(given, name: str, device, rows: int, heads: int, dim: int):
    """An output and its view: the caller's, checked, or a new contiguous one."""
    if given is not None:
        return given, _heads(given, name, device, (rows, heads, dim))
    t = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device=device)
    return t, _view(t.data_ptr(), heads * dim, dim, heads, 0)


def _at(t):
    return None if t is None else t.data_ptr()


def _bytes(ws, device, need):
    """The caller's workspace, checked, or a new one of need() bytes."""
    if ws is None:
        return torch.empty(max(need(), 1), dtype=torch.uint8, device=device)
    if ws.device != device or not ws.is_contiguous():
        raise QLoRAError(f"workspace must be a contiguous tensor on {device}")
    return ws


@dataclass(frozen=True)
class KVCache:
    """A key/value cache in 4 bits: caller-owned device buffers, laid out as include/qlora.h says.  Their addresses are
    taken when it is made: a tensor is not to be given other storage (resize_, set_, .data) while it lives."""
    k_codes: torch.Tensor    # uint8 [pages][heads][page_size][head_dim / 2]
    k_scale: torch.Tensor    # bf16 [pages][heads][page_size][head_dim / block]
    v_codes: torch.Tensor
    v_scale: torch.Tensor
    block: int = 64          # elements per scale: 32, 64 or 128
    codebook: int = CODEBOOK_NF4

    def __post_init__(self):
        c = self.k_codes
        if c.dim() != 4 or not c.is_cuda or c.dtype != torch.uint8:
            raise QLoRAError("k_codes must be a uint8 [pages][heads][page_size][head_dim / 2] tensor on the GPU")
        pages, heads, page_size, half = c.shape
        if self.block not in (32, 64, 128) or 2 * half % self.block:
            raise QLoRAError(f"block must be 32, 64 or 128 and divide head_dim, not {self.block}")
        scales = (pages, heads, page_size, 2 * half // self.block)
        _need(c, torch.uint8, c.device, "k_codes")
        _need(self.v_codes, torch.uint8, c.device, "v_codes", tuple(c.shape))
        _need(self.k_scale, torch.bfloat16, c.device, "k_scale", scales)
        _need(self.v_scale, torch.bfloat16, c.device, "v_scale", scales)
        # the fields are frozen, so the descriptor (as an argument) and the sizes are taken once
        for name, value in (("pages", pages), ("heads", heads), ("page_size", page_size), ("head_dim", 2 * half),
                            ("device", c.device)):
            object.__setattr__(self, name, value)
        object.__setattr__(self, "arg", C.byref(_lib.qlora_kv_cache(
            pages, page_size, heads, 2 * half, int(self.block), int(self.codebook), 0, self.k_codes.data_ptr(),
            self.k_scale.data_ptr(), self.v_codes.data_ptr(), self.v_scale.data_ptr())))

    def __reduce__(self):   # copies and pickles: made anew from the fields, the descriptor points at their own buffers
        return KVCache, (self.k_codes, self.k_scale, self.v_codes, self.v_scale, self.block, self.codebook)

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k_codes, self.k_scale, self.v_codes, self.v_scale))


def qlora_kv_sizes(pages: int, page_size: int, heads: int, head_dim: int, block: int = 64):
    """(bytes of one codes buffer, bytes of one scale buffer) of a cache."""
    d = _lib.qlora_kv_cache(pages, page_size, heads, head_dim, int(block), 0, 0, None, None, None, None)
    out = [C.c_size_t(), C.c_size_t()]
    _check(lib().qlora_kv_sizes(C.byref(d), *[C.byref(o) for o in out]), "qlora_kv_sizes")
    return tuple(o.value for o in out)


def kv_alloc(pages: int, page_size: int, heads: int, head_dim: int, block: int = 64, codebook: int = CODEBOOK_NF4,
             device="cuda") -> KVCache:
    """An empty cache (its contents are undefined until written)."""
    qlora_kv_sizes(pages, page_size, heads, head_dim, block)   # checks the sizes
    bufs = []
    for _ in range(2):
        bufs.append(torch.empty((pages, heads, page_size, head_dim // 2), dtype=torch.uint8, device=device))
        bufs.append(torch.empty((pages, heads, page_size, head_dim // block), dtype=torch.bfloat16, device=device))
    return KVCache(*bufs, block, codebook)


@dataclass(frozen=True)
class KVBatch:
    """The tokens a call is about: rows start[b] .. start[b + 1] - 1 are the last ones of sequence b, whose
    length[b] tokens lie in the pages table[b].  Device tensors that the kernels read, so their contents may
    change between calls (and between replays of a captured call), but not their storage, as that of a cache."""
    start: torch.Tensor               # int32 [batch + 1]
    length: torch.Tensor              # int32 [batch]
    table: torch.Tensor               # int32 [batch][max_pages]
    fault: torch.Tensor | None = None   # int32 [1]: bits of wrong entries are OR-ed in (see include/qlora.h)

    def __post_init__(self):
        n, dev = self.length.numel(), self.length.device
        if not self.length.is_cuda or self.table.dim() != 2:
            raise QLoRAError("start, length and table must be on the GPU, table [batch][max_pages]")
        _need(self.length, torch.int32, dev, "length", (n,))
        _need(self.start, torch.int32, dev, "start", (n + 1,))
        _need(self.table, torch.int32, dev, "table", (n, self.table.shape[1]))
        if self.fault is not None:
            _need(self.fault, torch.int32, dev, "fault", (1,))
        object.__setattr__(self, "device", dev)
        object.__setattr__(self, "arg", C.byref(_lib.qlora_kv_batch(
            n, self.table.shape[1], self.start.data_ptr(), self.length.data_ptr(), self.table.data_ptr(),
            None if self.fault is None else self.fault.data_ptr())))

    def __reduce__(self):   # (as of a cache)
        return KVBatch, (self.start, self.length, self.table, self.fault)


def _same_device(cache: KVCache, batch: KVBatch):
    if cache.device != batch.device:
        raise QLoRAError("the cache and the batch must be on one device")
    return cache.device


def _keys(k, name: str, device, rows: int, dim: int):
    """(view, heads) of k, or (None, 0): any number of heads, otherwise like q."""
    if k is None:
        return None, 0
    view = _heads(k, name, device)
    n, heads, d = k.shape
    if n != rows or d != dim:
        raise QLoRAError(f"{name} must have {rows} rows of head_dim {dim}, not {tuple(k.shape)}")
    return view, heads


def _qk_inputs(k, dev, rows, dim, positions, inv_freq, q_weight, k_weight) -> int:
    """Checks what both directions take; the rotated elements of a head."""
    rot = 0
    if inv_freq is not None:
        half = inv_freq.numel()
        rot = 2 * half
        _need(inv_freq, torch.float32, dev, "inv_freq", (half,))
    if rot:
        if positions is None:
            raise QLoRAError("inv_freq needs positions")
        _need(positions, torch.int64, dev, "positions", (rows,))
    if k is None and k_weight is not None:
        raise QLoRAError("k_weight needs k")
    if q_weight is not None:
        _need(q_weight, torch.bfloat16, dev, "q_weight", (dim,))
    if k_weight is not None:
        _need(k_weight, torch.bfloat16, dev, "k_weight", (dim,))
    return rot


def qlora_qk_norm_rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None,
                       inv_freq: torch.Tensor | None, q_weight: torch.Tensor | None = None,
                       k_weight: torch.Tensor | None = None, eps: float = 1e-6, interleaved: bool = False,
                       q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None, stream=None):
    """Norm of each head (where its weight is given) and rotation by positions [rows] (int64) * inv_freq
    [rot_dim / 2] (fp32) of q, k [rows][heads][head_dim] bf16, any strides.  The outputs may be the inputs.
    Returns (q_out, k_out or None)."""
    hq, dev = _heads(q, "q"), q.device
    rows, q_heads, dim = q.shape
    hk, k_heads = _keys(k, "k", dev, rows, dim)
    rot = _qk_inputs(k, dev, rows, dim, positions, inv_freq, q_weight, k_weight)
    if k is None and k_out is not None:
        raise QLoRAError("k_out needs k")

    def run(stream):
        qo, oq = _out(q_out, "q_out", dev, rows, q_heads, dim)
        ko, ok = (None, None) if k is None else _out(k_out, "k_out", dev, rows, k_heads, dim)
        _check(lib().qlora_qk_norm_rope(hq, hk, rows, dim, _at(q_weight), _at(k_weight), eps,
                                        _at(positions), _at(inv_freq), rot, interleaved, oq, ok, stream),
               "qlora_qk_norm_rope")
        return qo, ko

    return _launch(q, stream, run)


def qlora_qk_norm_rope_bwd_workspace(rows: int, q_heads: int, k_heads: int, head_dim: int) -> int:
    return lib().qlora_qk_norm_rope_bwd_workspace(rows, q_heads, k_heads, head_dim)


def qlora_qk_norm_rope_bwd(dq_out: torch.Tensor, dk_out: torch.Tensor | None, q: torch.Tensor | None,
                           k: torch.Tensor | None, positions: torch.Tensor | None, inv_freq: torch.Tensor | None,
                           q_weight: torch.Tensor | None = None, k_weight: torch.Tensor | None = None,
                           eps: float = 1e-6, interleaved: bool = False, dq: torch.Tensor | None = None,
                           dk: torch.Tensor | None = None, dq_weight: torch.Tensor | None = None,
                           dk_weight: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of qlora_qk_norm_rope's inputs from those of its outputs; q, k are the forward's inputs
    (needed where there is a weight).  dq may be dq_out and dk may be dk_out.  Returns (dq, dk or None,
    dq_weight or None, dk_weight or None), the weights' fp32 [head_dim]."""
    gq, dev = _heads(dq_out, "dq_out"), dq_out.device
    rows, q_heads, dim = dq_out.shape
    gk, k_heads = _keys(dk_out, "dk_out", dev, rows, dim)
    rot = _qk_inputs(dk_out, dev, rows, dim, positions, inv_freq, q_weight, k_weight)
    if (q_weight is not None and q is None) or (k_weight is not None and k is None):
        raise QLoRAError("a weight's gradient needs the forward's input")
    xq = _heads(q, "q", dev, (rows, q_heads, dim)) if q_weight is not None else None
    xk = _heads(k, "k", dev, (rows, k_heads, dim)) if k_weight is not None else None
    if dk_out is None and dk is not None:
        raise QLoRAError("dk needs dk_out")
    if (q_weight is None and dq_weight is not None) or (k_weight is None and dk_weight is not None):
        raise QLoRAError("a weight's gradient needs the weight")

    def run(stream):
        oq, hq = _out(dq, "dq", dev, rows, q_heads, dim)
        ok, hk = (None, None) if dk_out is None else _out(dk, "dk", dev, rows, k_heads, dim)
        gwq, gwk = dq_weight, dk_weight
        if q_weight is not None:
            gwq = torch.empty(dim, dtype=torch.float32, device=dev) if gwq is None else \
                _need(gwq, torch.float32, dev, "dq_weight", (dim,))
        if k_weight is not None:
            gwk = torch.empty(dim, dtype=torch.float32, device=dev) if gwk is None else \
                _need(gwk, torch.float32, dev, "dk_weight", (dim,))
        ws = None
        if q_weight is not None or k_weight is not None:
            ws = _bytes(workspace, dev, lambda: qlora_qk_norm_rope_bwd_workspace(rows, q_heads, k_heads, dim))
        _check(lib().qlora_qk_norm_rope_bwd(gq, gk, xq, xk, rows, dim, _at(q_weight),
                                            _at(k_weight), eps, _at(positions), _at(inv_freq), rot, interleaved,
                                            hq, hk, _at(gwq), _at(gwk), _at(ws),
                                            0 if ws is None else ws.nbytes, stream), "qlora_qk_norm_rope_bwd")
        return oq, ok, gwq, gwk

    return _launch(dq_out, stream, run)


def qlora_kv_write(k: torch.Tensor, v: torch.Tensor, cache: KVCache, batch: KVBatch, stream=None):
    """Quantize the rows k, v [rows][heads][head_dim] (bf16, any strides) into the cache."""
    dev = _same_device(cache, batch)
    shape = (len(k) if k.dim() else 0, cache.heads, cache.head_dim)
    hk, hv = _heads(k, "k", dev, shape), _heads(v, "v", dev, shape)
    _launch(k, stream, lambda stream: _check(
        lib().qlora_kv_write(hk, hv, shape[0], cache.arg, batch.arg, stream),
        "qlora_kv_write"))


def qlora_kv_read(cache: KVCache, batch: KVBatch, rows: int, k: torch.Tensor | None = None,
                  v: torch.Tensor | None = None, stream=None):
    """The batch's rows read back from the cache: (k, v) [rows][heads][head_dim] bf16.  Rows of no sequence
    keep what k and v hold (undefined if they are not given)."""
    dev = _same_device(cache, batch)

    def run(stream):
        ko, hk = _out(k, "k", dev, rows, cache.heads, cache.head_dim)
        vo, hv = _out(v, "v", dev, rows, cache.heads, cache.head_dim)
        _check(lib().qlora_kv_read(cache.arg, batch.arg, rows, hk, hv, stream),
               "qlora_kv_read")
        return ko, vo

    return _launch(cache.k_codes, stream, run)


def qlora_kv_attn_workspace(cache: KVCache, batch: KVBatch, rows: int, q_heads: int) -> int:
    return lib().qlora_kv_attn_workspace(cache.arg, batch.arg, rows, q_heads)


def qlora_kv_attn(q: torch.Tensor, cache: KVCache, batch: KVBatch, scale: float | None = None, causal: bool = True,
                  window: int = 0, out: torch.Tensor | None = None, lse: torch.Tensor | bool = False,
                  workspace: torch.Tensor | None = None, stream=None):
    """Attention of q [rows][q_heads][head_dim] (bf16, any strides) over the cache; scale defaults to
    head_dim ** -0.5.  lse: True for a new fp32 [rows][q_heads], or a tensor to fill.  Returns (out, lse or
    None).  Rows of no sequence keep what out and lse hold (undefined if they are not given)."""
    dev = _same_device(cache, batch)
    hq = _heads(q, "q", dev)
    rows, heads, dim = q.shape
    if dim != cache.head_dim:
        raise QLoRAError(f"q must have the cache's head_dim {cache.head_dim}, not {dim}")
    if window < 0:
        raise QLoRAError("window must be 0 (none) or positive")
    window = min(window, 2 ** 31 - 1)   # (past every cache's length, where a window is none)

    def run(stream):
        o, ho = _out(out, "out", dev, rows, heads, dim)
        sums = None
        if lse is True:
            sums = torch.empty((rows, heads), dtype=torch.float32, device=dev)
        elif lse is not False and lse is not None:
            sums = _need(lse, torch.float32, dev, "lse", (rows, heads))
        ws = _bytes(workspace, dev, lambda: qlora_kv_attn_workspace(cache, batch, rows, heads))
        _check(lib().qlora_kv_attn(hq, rows, cache.arg, batch.arg,
                                   cache.head_dim ** -0.5 if scale is None else scale, causal, window, ho,
                                   _at(sums), _at(ws), ws.nbytes, stream), "qlora_kv_attn")
        return o, sums

    return _launch(q, stream, run)


# ---- around the projections: the residual's norm, the gated block, log probabilities ---------------------------
_I32 = 2 ** 31 - 1


def _i32(n: int) -> int:
    """n, or the end of 32 bits that it lies past: the library refuses these, where ctypes would drop n's upper bits."""
    return max(-_I32, min(n, _I32))


def _rows(t: torch.Tensor, name: str, device=None, shape=None):
    """(address, row stride) of a bf16 [rows][dim] tensor, any row stride with dense rows."""
    strides = t.stride()
    if t.dtype is not torch.bfloat16 or len(strides) != 2 or strides[1] != 1 or not t.is_cuda:
        raise QLoRAError(f"{name} must be a bf16 [rows][dim] tensor on the GPU, dense along dim")
    if device is not None and t.device != device:
        raise QLoRAError(f"{name} must be on {device}")
    if shape is not None and t.shape != shape:
        raise QLoRAError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    return t.data_ptr(), strides[0]


def _new_rows(given, name: str, device, like):
    """An output like the tensor `like` and its (address, row stride): the caller's, checked, or a new contiguous one."""
    if given is not None:
        return given, _rows(given, name, device, like.shape)
    t = torch.empty_like(like, memory_format=torch.contiguous_format)   # (less than half the cost of torch.empty's arguments)
    return t, (t.data_ptr(), like.size(1))


def qlora_rms_norm(x: torch.Tensor, weight: torch.Tensor | None, residual: torch.Tensor | None = None,
                   eps: float = 1e-6, out: torch.Tensor | None = None, sum_out: torch.Tensor | None = None, stream=None):
    """Residual addition and root-mean-square norm of x [rows][dim] (bf16, any row stride): h = bf16(x + residual),
    out = bf16(h weight / sqrt(mean(h^2) + eps)).  out and sum_out may be x or residual.  Returns (out, h), h being x
    without a residual."""
    dev = x.device
    px, sx = _rows(x, "x")
    shape = x.shape
    pr, sr = (None, 0) if residual is None else _rows(residual, "residual", dev, shape)
    if weight is not None:
        _need(weight, torch.bfloat16, dev, "weight", (shape[1],))
    if residual is None and sum_out is not None:
        raise QLoRAError("sum_out needs a residual")

    def run(stream):
        y, (py, sy) = _new_rows(out, "out", dev, x)
        h, (ph, sh) = (x, (None, 0)) if residual is None else _new_rows(sum_out, "sum_out", dev, x)
        _check(lib().qlora_rms_norm(px, sx, pr, sr, shape[0], min(shape[1], _I32), _at(weight), eps, py, sy, ph, sh, stream),
               "qlora_rms_norm")
        return y, h

    return _launch(x, stream, run)


def qlora_rms_norm_bwd_workspace(rows: int, dim: int) -> int:
    return lib().qlora_rms_norm_bwd_workspace(rows, _i32(dim))


def qlora_rms_norm_bwd(dy: torch.Tensor, h: torch.Tensor, weight: torch.Tensor | None, dh: torch.Tensor | None = None,
                       eps: float = 1e-6, weight_grad: bool = True, dx: torch.Tensor | None = None,
                       dweight: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of qlora_rms_norm from that of its output, its h and (where h goes on beside the norm) the gradient dh
    of h.  dx, the gradient of x and of the residual, may be dy, h or dh.  Returns (dx, dweight fp32 [dim] or None:
    without a weight, or with weight_grad=False)."""
    dev = dy.device
    pg, sg = _rows(dy, "dy")
    shape = dy.shape
    ph, sh = _rows(h, "h", dev, shape)
    pd, sd = (None, 0) if dh is None else _rows(dh, "dh", dev, shape)
    if weight is not None:
        _need(weight, torch.bfloat16, dev, "weight", (shape[1],))
    if weight is None or not weight_grad:
        if dweight is not None:
            raise QLoRAError("dweight needs the weight, and weight_grad")
        weight_grad = False
    elif dweight is not None:
        _need(dweight, torch.float32, dev, "dweight", (shape[1],))

    def run(stream):
        out, (px, sx) = _new_rows(dx, "dx", dev, dy)
        gw, ws = None, None
        if weight_grad:
            gw = torch.empty(shape[1], dtype=torch.float32, device=dev) if dweight is None else dweight
            ws = _bytes(workspace, dev, lambda: qlora_rms_norm_bwd_workspace(shape[0], shape[1]))
        _check(lib().qlora_rms_norm_bwd(pg, sg, ph, sh, pd, sd, shape[0], min(shape[1], _I32), _at(weight), eps, px, sx,
                                        _at(gw), _at(ws), 0 if ws is None else ws.nbytes, stream), "qlora_rms_norm_bwd")
        return out, gw

    return _launch(dy, stream, run)


# qlora_activation values
ACTIVATIONS = {"silu": 0, "gelu": 1}


def _activation(name: str) -> int:
    if name not in ACTIVATIONS:
        raise QLoRAError(f"activation must be one of {sorted(ACTIVATIONS)}, not {name!r}")
    return ACTIVATIONS[name]


def qlora_gated_workspace(M: int, d_in: int, d_out: int, r: int) -> int:
    return lib().qlora_gated_workspace(M, d_in, d_out, _i32(r))


def qlora_gated_fwd(X: torch.Tensor, gate: NF4Weight, up: NF4Weight, A_gate: torch.Tensor, B_gate: torch.Tensor,
                    A_up: torch.Tensor, B_up: torch.Tensor, scale: float, activation: str = "silu", save: bool = True,
                    H: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """H = act(G) U with G = X deq(gate)^T + scale (X A_gate) B_gate and U likewise, X [M][in] bf16 (fp32 up to the activation,
    but for bf16 of scale X A, as in qlora_linear_fwd).  save: also bf16 of G
    and U, and of X A of each, for the backward.  Returns (H, G, U, T_gate, T_up), the last four None without save."""
    dev, kind = X.device, _activation(activation)
    if X.dim() != 2 or X.shape[1] != gate.cols or not X.is_cuda:
        raise QLoRAError(f"X must be [M][{gate.cols}] on the GPU")
    M, d_in, d_out = X.shape[0], gate.cols, gate.rows
    _need(X, torch.bfloat16, dev, "X")
    if A_gate.dim() != 2:
        raise QLoRAError("A_gate must be [in][r]")
    r = A_gate.shape[1]
    for t, name, shape in ((A_gate, "A_gate", (d_in, r)), (A_up, "A_up", (d_in, r)), (B_gate, "B_gate", (r, d_out)),
                           (B_up, "B_up", (r, d_out))):
        _need(t, torch.bfloat16, dev, name, shape)
    for w, name in ((gate, "gate"), (up, "up")):
        if w.codes.device != dev:
            raise QLoRAError(f"{name} must be on {dev}")
    if H is not None:
        _need(H, torch.bfloat16, dev, "H", (M, d_out))

    def run(stream):
        new = X.new_empty
        out = new((M, d_out)) if H is None else H
        saved = (None,) * 4
        if save:
            T = new((M, r))
            saved = (torch.empty_like(out), torch.empty_like(out), T, torch.empty_like(T))
        ws = _bytes(workspace, dev, lambda: qlora_gated_workspace(M, d_in, d_out, r))
        g, u = gate.desc(), up.desc()
        _check(lib().qlora_gated_fwd(X.data_ptr(), M, C.byref(g), C.byref(u), A_gate.data_ptr(), B_gate.data_ptr(),
                                     A_up.data_ptr(), B_up.data_ptr(), r, scale, kind, out.data_ptr(),
                                     *[_at(t) for t in saved], ws.data_ptr(), ws.nbytes, stream), "qlora_gated_fwd")
        return out, *saved

    return _launch(X, stream, run)


def qlora_gated_bwd(dH: torch.Tensor | None, G: torch.Tensor, U: torch.Tensor, activation: str = "silu",
                    H: torch.Tensor | bool = False, dG: torch.Tensor | None = None, dU: torch.Tensor | None = None,
                    stream=None):
    """Gradients of the gated block's G and U from that of H = act(G) U and the saved G, U [M][out]; qlora_linear_bwd of each
    projection goes on from them.  H: True for H itself in a new tensor, or a tensor to fill.  dH None: H alone (which the
    last projection's backward needs), in place of a kept one.  Outputs may be the inputs, one each.  Returns (dG, dU,
    H or None)."""
    dev, kind = G.device, _activation(activation)
    if G.dim() != 2 or not G.is_cuda:
        raise QLoRAError("G must be [M][out] on the GPU")
    shape = G.shape
    if dH is None and (H is False or dG is not None or dU is not None):
        raise QLoRAError("without dH there is H alone")
    for t, name in ((dH, "dH"), (G, "G"), (U, "U"), (dG, "dG"), (dU, "dU"), (H, "H")):
        if isinstance(t, torch.Tensor):
            _need(t, torch.bfloat16, dev, name, shape)

    def run(stream):
        new = lambda: torch.empty_like(G)
        g = new() if dG is None and dH is not None else dG
        u = new() if dU is None and dH is not None else dU
        h = new() if H is True else H if isinstance(H, torch.Tensor) else None
        _check(lib().qlora_gated_bwd(_at(dH), G.data_ptr(), U.data_ptr(), shape[0], shape[1], kind, _at(g), _at(u), _at(h),
                                     stream), "qlora_gated_bwd")
        return g, u, h

    return _launch(G, stream, run)


_LOGIT_TYPES = {torch.bfloat16: 0, torch.float32: 1}   # qlora_dtype values


def _logits(t: torch.Tensor, name: str, device=None, like=None):
    """(address, row stride, qlora_dtype) of [rows][vocab] logits, any row stride with dense rows."""
    strides = t.stride()
    kind = _LOGIT_TYPES.get(t.dtype)
    if kind is None or len(strides) != 2 or strides[1] != 1 and t.shape[1] != 1 or not t.is_cuda:
        raise QLoRAError(f"{name} must be a bf16 or float32 [rows][vocab] tensor on the GPU, dense along vocab")
    if like is not None and (t.device != device or t.shape != like.shape or t.dtype != like.dtype):
        raise QLoRAError(f"{name} must be like the logits")
    return t.data_ptr(), strides[0], kind


def qlora_token_logprob_workspace(rows: int, vocab: int, top: int = 0) -> int:
    return lib().qlora_token_logprob_workspace(rows, vocab, _i32(top))


def qlora_token_logprob(logits: torch.Tensor, token: torch.Tensor | None, scale: float = 1.0, entropy: bool = False,
                        top: int = 0, workspace: torch.Tensor | None = None, stream=None):
    """Log probabilities of the tokens [rows] (int64; negative: none) under the softmax of scale * logits [rows][vocab]
    (bf16 or fp32, any row stride).  Returns (logprob [rows] or None without tokens, stats [rows][2] = largest scaled logit
    and sum of exponentials from it, entropy [rows] or None, top_logprob and top_index [rows][top] or None), all
    fp32 but the indices (int64)."""
    dev = logits.device
    px, sx, kind = _logits(logits, "logits")
    rows, vocab = logits.shape
    if token is not None:
        _need(token, torch.int64, dev, "token", (rows,))

    def run(stream):
        new, f32 = logits.new_empty, torch.float32
        lp = None if token is None else new((rows,), dtype=f32)
        stats = new((rows, 2), dtype=f32)
        ent = new((rows,), dtype=f32) if entropy else None
        tlp = new((rows, top), dtype=f32) if top else None
        tix = new((rows, top), dtype=torch.int64) if top else None
        need = qlora_token_logprob_workspace(rows, vocab, top)   # 0: none (an allocation less is 1.4 us)
        ws = _bytes(workspace, dev, lambda: need) if need or workspace is not None else None
        _check(lib().qlora_token_logprob(px, sx, rows, vocab, kind, _at(token), scale, top, _at(lp), stats.data_ptr(),
                                         _at(ent), _at(tlp), _at(tix), _at(ws), 0 if ws is None else ws.nbytes, stream),
               "qlora_token_logprob")
        return lp, stats, ent, tlp, tix

    if not 0 <= top <= vocab:
        raise QLoRAError(f"top must be 0 (none) to {vocab}, the number of logits")
    return _launch(logits, stream, run)


def qlora_token_logprob_bwd(logits: torch.Tensor, token: torch.Tensor | None, stats: torch.Tensor,
                            dlogprob: torch.Tensor | None, entropy: torch.Tensor | None = None,
                            dentropy: torch.Tensor | None = None, scale: float = 1.0, out: torch.Tensor | None = None,
                            stream=None):
    """Gradient of the logits from those of qlora_token_logprob's logprob and entropy (fp32 [rows], either may be None), its
    stats and, with dentropy, its entropy.  out may be the logits.  Returns it, in the logits' type."""
    dev = logits.device
    px, sx, kind = _logits(logits, "logits")
    rows, vocab = logits.shape
    if dlogprob is not None and token is None:
        raise QLoRAError("dlogprob needs the tokens")
    if dentropy is not None and entropy is None:
        raise QLoRAError("dentropy needs the entropy")
    if token is not None:
        _need(token, torch.int64, dev, "token", (rows,))
    _need(stats, torch.float32, dev, "stats", (rows, 2))
    for t, name in ((dlogprob, "dlogprob"), (entropy, "entropy"), (dentropy, "dentropy")):
        if t is not None:
            _need(t, torch.float32, dev, name, (rows,))

    def run(stream):
        d = torch.empty_like(logits, memory_format=torch.contiguous_format) if out is None else out
        pd, sd, _ = _logits(d, "out", dev, logits)
        _check(lib().qlora_token_logprob_bwd(px, sx, rows, vocab, kind, _at(token), scale, stats.data_ptr(), _at(dlogprob),
                                             _at(entropy), _at(dentropy), pd, sd, stream), "qlora_token_logprob_bwd")
        return d

    return _launch(logits, stream, run)


def qlora_profile_enable(enable: bool = True):
    _check(lib().qlora_profile_enable(int(enable)), "qlora_profile_enable")


def qlora_profile_read(reset: bool = True) -> dict:
    """{kernel name: (launches, total_ms)} since the last reset (synchronizes the recorded events)."""
    buf = (_lib.qlora_kernel_time * 64)()
    n = lib().qlora_profile_read(buf, 64, int(reset))
    return {buf[i].name.decode(): (buf[i].launches, buf[i].total_ms) for i in range(n)}
