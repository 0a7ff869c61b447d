"""MI355X-native Hessian-weighted sequential layer quantization.

GPTQ read as Babai's nearest-plane algorithm ("The Geometry of LLM
Quantization: GPTQ as Babai's Nearest Plane Algorithm", technical summary
2.1-2.3) and its successive-interference-cancellation form with per-column
spacing ("WaterSIC: information-theoretically (near) optimal linear layer
quantization", technical summary 2), behind the C ABI of ``libpwq.so``
(``include/pwq.h``; ``include/pwq_serve.h`` and ``include/pwq_cache.h`` for
running quantized layers and the cache between them).  These wrappers only marshal torch tensors (device
memory) and the current stream into that ABI; the HIP kernels do all the
work and there is no CPU fallback.
"""
import ctypes
import functools
import struct
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import PwqError, check, lib, make_grid, parse_result

__all__ = ["Grid", "hessian_accum", "damp_cholesky", "damp_cholesky_static", "grid_steps", "babai_sweep",
           "quant_layer", "column_entropy", "read_result", "PwqError", "KernelTimer",
           "HessianTileTimer", "overflow_entries", "ssqr_quant_layer", "pack_weights", "rms_norm",
           "packed_linear", "new_cache", "cache_write", "cache_read", "cached_attention"]


@dataclass(frozen=True)
class Grid:
    kind: str = "sym"       # "sym" | "asym" | "colspacing"
    bits: int = 4
    group: int = 0          # 0 = one step per row
    c: float = 0.0          # colspacing constant (alpha_k = c / l_kk); colspacing only
    kappa: float = 0.0      # step multiplier (0 = none); sym / asym only

    def c_struct(self):
        return make_grid(self.kind, self.bits, self.group, self.c, self.kappa)


def _stream():
    return torch.cuda.current_stream().cuda_stream or None


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return _lib.PWQ_F32
    if t.dtype == torch.bfloat16:
        return _lib.PWQ_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def _prec(prec: str) -> int:
    return {"f32": _lib.PWQ_F32, "f64": _lib.PWQ_F64}[prec]


def _tdt(prec: str):
    return torch.float64 if prec == "f64" else torch.float32


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on the GPU")


def _row_major(t: torch.Tensor) -> int:
    """Row stride (elements) of a 2-D row-major tensor.  A single row may
    carry any stride in torch; its row stride is then its length."""
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1):
        raise ValueError("expected a 2-D tensor with unit column stride")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _check(t: Optional[torch.Tensor], name: str, shape, dtypes):
    """A tensor handed to the library as a raw pointer must have exactly the
    shape, element type and (contiguous, row-major) layout the C ABI reads."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_F32 = (torch.float32,)
_I32 = (torch.int32,)


def _check_result(res: Optional[torch.Tensor]):
    if res is None:
        return
    if res.dtype != torch.uint8 or res.numel() < _lib.RESULT_BYTES or not res.is_contiguous():
        raise ValueError(f"result must be a contiguous uint8 tensor of >= {_lib.RESULT_BYTES} "
                         "bytes (see new_result)")


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def new_result(device) -> torch.Tensor:
    return torch.zeros(_lib.RESULT_BYTES, dtype=torch.uint8, device=device)


def read_result(res: torch.Tensor) -> dict:
    """Synchronising read of a device result record."""
    return parse_result(bytes(res.cpu().numpy().tobytes()))


def _x_args(X: torch.Tensor, x_layout: str):
    """(n, ntok, ldx, xdtype) of activations X: ``x_layout`` "channels" for
    X [n, ntok], "tokens" for X [ntok, n] (one row per token)."""
    ldx = _row_major(X)
    if x_layout == "channels":
        n, ntok = X.shape
        return n, ntok, ldx, _dtype_code(X)
    if x_layout == "tokens":
        ntok, n = X.shape
        return n, ntok, ldx, _dtype_code(X) | _lib.PWQ_X_TOKEN_MAJOR
    raise ValueError(f"x_layout must be 'channels' or 'tokens', not {x_layout!r}")


def hessian_accum(X: torch.Tensor, H: Optional[torch.Tensor] = None,
                  accumulate: bool = False, x_layout: str = "channels") -> torch.Tensor:
    """H (+)= 2 X X^T for activations X (bf16 or fp32) stored [n, ntok]
    (``x_layout="channels"``) or [ntok, n] (``x_layout="tokens"``)."""
    _require_cuda(X, H)
    n, ntok, ldx, xdt = _x_args(X, x_layout)
    _check(H, "H", (n, n), _F32)
    if H is None:
        H = torch.empty((n, n), dtype=torch.float32, device=X.device)
    L = lib()
    wsb = L.pwq_hessian_workspace_size(n, ntok)
    ws = _workspace(wsb, X.device)
    check(L.pwq_hessian_accum(H.data_ptr(), n, X.data_ptr(), xdt, ntok, ldx,
                              int(accumulate), ws.data_ptr(), ws.numel(), _stream()))
    return H


def damp_cholesky(H: torch.Tensor, damp: float = 0.01, prec: str = "f32"):
    """(L, dead, result) for H_d = H' + lambda I (lower factor)."""
    _require_cuda(H)
    n = H.shape[0]
    _check(H, "H", (n, n), _F32)
    L_ = lib()
    Lt = torch.empty((n, n), dtype=_tdt(prec), device=H.device)
    dead = torch.empty(n, dtype=torch.int32, device=H.device)
    res = new_result(H.device)
    ws = _workspace(L_.pwq_cholesky_workspace_size(n, _prec(prec)), H.device)
    check(L_.pwq_damp_cholesky(H.data_ptr(), n, float(damp), _prec(prec), Lt.data_ptr(),
                               dead.data_ptr(), res.data_ptr(), ws.data_ptr(), ws.numel(),
                               _stream()))
    return Lt, dead, res


def damp_cholesky_static(H: torch.Tensor, damp: float = 0.01, prec: str = "f32",
                         out: Optional[tuple] = None):
    """damp_cholesky through pwq_damp_cholesky_static: no workspace (the
    library's static device scratch; calls overlapping on one GPU race).
    ``out`` may pass preallocated (L, dead, result) so that the call itself
    allocates nothing."""
    _require_cuda(H)
    n = H.shape[0]
    _check(H, "H", (n, n), _F32)
    if out is None:
        out = (torch.empty((n, n), dtype=_tdt(prec), device=H.device),
               torch.empty(n, dtype=torch.int32, device=H.device), new_result(H.device))
    Lt, dead, res = out
    _require_cuda(Lt, dead, res)
    _check(Lt, "L", (n, n), (_tdt(prec),))
    _check(dead, "dead", (n,), _I32)
    _check_result(res)
    check(lib().pwq_damp_cholesky_static(H.data_ptr(), n, float(damp), _prec(prec),
                                         Lt.data_ptr(), dead.data_ptr(), res.data_ptr(),
                                         _stream()))
    return Lt, dead, res


def min_pivot_order(H: torch.Tensor, damp: float = 0.01, want_pivots: bool = False):
    """Min-pivot order of H_d = H' + lambda I: (perm, pivots or None, result).
    perm[k] (int32) is the column at position k (position 0 is processed
    last); pivots (float64) are the LDL pivots D_kk of the permuted matrix."""
    _require_cuda(H)
    n = H.shape[0]
    if H.dim() != 2 or H.shape[1] != n or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be a contiguous float32 [n, n] tensor")
    L_ = lib()
    perm = torch.empty(n, dtype=torch.int32, device=H.device)
    piv = torch.empty(n, dtype=torch.float64, device=H.device) if want_pivots else None
    res = new_result(H.device)
    ws = _workspace(L_.pwq_min_pivot_workspace_size(n), H.device)
    check(L_.pwq_min_pivot_order(H.data_ptr(), n, float(damp), perm.data_ptr(), _ptr(piv),
                                 res.data_ptr(), ws.data_ptr(), ws.numel(), _stream()))
    return perm, piv, res


def oaem_init(W: torch.Tensor, H: torch.Tensor, seeds: torch.Tensor, g: int = 8,
              iters: int = 10, damp: float = 0.01, want_objective: bool = True):
    """OA-EM codebook initialisation.  seeds: int64 [M, K] group indices
    r (n/g) + i.  Returns (codebooks float64 [M, K, g], codes int32
    [M, m, n/g], objective float64 [M] or None, result)."""
    _require_cuda(W, H, seeds)
    m, n = W.shape
    if H.shape != (n, n) or H.dtype != torch.float32 or not H.is_contiguous():
        raise ValueError("H must be a contiguous float32 [n, n] tensor")
    if seeds.dim() != 2 or seeds.dtype != torch.int64 or not seeds.is_contiguous():
        raise ValueError("seeds must be a contiguous int64 [M, K] tensor")
    M, K = seeds.shape
    if g <= 0 or n % g:
        raise ValueError("g must divide n")
    dev = W.device
    L_ = lib()
    books = torch.empty((M, K, g), dtype=torch.float64, device=dev)
    codes = torch.empty((M, m, n // g), dtype=torch.int32, device=dev)
    obj = torch.empty(M, dtype=torch.float64, device=dev) if want_objective else None
    res = new_result(dev)
    nb = L_.pwq_oaem_workspace_size(m, n, g, K)
    ws = _workspace(nb, dev) if nb else None
    check(L_.pwq_oaem_init(W.data_ptr(), _dtype_code(W), m, n, _row_major(W), H.data_ptr(),
                           float(damp), int(g), int(K), int(M), int(iters), seeds.data_ptr(),
                           books.data_ptr(), codes.data_ptr(), _ptr(obj), res.data_ptr(),
                           _ptr(ws), 0 if ws is None else ws.numel(), _stream()))
    return books, codes, obj, res


def grid_steps(W: torch.Tensor, grid: Grid, dead: Optional[torch.Tensor] = None):
    """(scales [m, n/G], zeros [m, n/G] or None) for SYM / ASYM grids."""
    _require_cuda(W, dead)
    m, n = W.shape
    _check(dead, "dead", (n,), _I32)
    if grid.group and n % grid.group:
        raise ValueError(f"group {grid.group} does not divide n = {n}")
    G = grid.group or n
    scales = torch.empty((m, n // G), dtype=torch.float32, device=W.device)
    zeros = (torch.empty((m, n // G), dtype=torch.int32, device=W.device)
             if grid.kind == "asym" else None)
    g = grid.c_struct()
    check(lib().pwq_grid_steps(W.data_ptr(), _dtype_code(W), m, n, _row_major(W), _ptr(dead),
                               g, scales.data_ptr(), _ptr(zeros), _stream()))
    return scales, zeros


def babai_sweep(W: torch.Tensor, L: torch.Tensor, grid: Grid, scales=None, zeros=None,
                dead=None, block: int = 128, result: Optional[torch.Tensor] = None):
    """Nearest-plane sweep given a factor L (natural order).  Returns
    (codes, scales, result)."""
    _require_cuda(W, L, scales, zeros, dead)
    m, n = W.shape
    _check(L, "L", (n, n), (torch.float32, torch.float64))
    prec = "f64" if L.dtype == torch.float64 else "f32"
    _check(dead, "dead", (n,), _I32)
    _check_result(result)
    if grid.kind == "colspacing":
        scales = torch.empty(n, dtype=torch.float32, device=W.device)
    elif scales is None:
        raise ValueError("SYM/ASYM sweeps need scales (see grid_steps)")
    else:
        if grid.group and n % grid.group:
            raise ValueError(f"group {grid.group} does not divide n = {n}")
        ng = n // (grid.group or n)
        _check(scales, "scales", (m, ng), _F32)
        _check(zeros, "zeros", (m, ng), _I32)
    codes = torch.empty((m, n), dtype=torch.int32, device=W.device)
    res = new_result(W.device) if result is None else result
    L_ = lib()
    ws = _workspace(L_.pwq_sweep_workspace_size(m, n, block, _prec(prec)), W.device)
    g = grid.c_struct()
    check(L_.pwq_babai_sweep(W.data_ptr(), _dtype_code(W), m, n, _row_major(W), L.data_ptr(),
                             _prec(prec), _ptr(dead), g, scales.data_ptr(), _ptr(zeros),
                             block, codes.data_ptr(), res.data_ptr(), ws.data_ptr(),
                             ws.numel(), _stream()))
    return codes, scales, res


def workspace_for_layer(m, n, ntok, has_x, order, block, prec, device) -> torch.Tensor:
    nb = lib().pwq_quant_layer_workspace_size(m, n, ntok, int(has_x), _lib.ORDERS[order],
                                             block, _prec(prec))
    return _workspace(nb, device)


def quant_layer(W: torch.Tensor, X: Optional[torch.Tensor] = None,
                H: Optional[torch.Tensor] = None, grid: Grid = Grid(),
                order: str = "back_to_front", perm: Optional[torch.Tensor] = None,
                damp: float = 0.01, block: int = 128, prec: str = "f32",
                want_H: bool = False, want_L: bool = False,
                workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                x_layout: str = "channels"):
    """quant_layer(W, X or H, grid, order, damp) -> dict(codes, scales, zeros,
    result[, H, L]).  ``out`` may pass preallocated outputs (same keys);
    ``x_layout`` as for hessian_accum."""
    _require_cuda(W, X, H, perm, workspace)
    m, n = W.shape
    dev = W.device
    ntok, ldx, xdt = 0, 0, 0
    if X is not None:
        nx, ntok, ldx, xdt = _x_args(X, x_layout)
        if nx != n:
            raise ValueError(f"X has {nx} channels, W has {n} columns")
    _check(H, "H", (n, n), _F32)
    _check(perm, "perm", (n,), _I32)
    if grid.kind != "colspacing" and grid.group and n % grid.group:
        raise ValueError(f"group {grid.group} does not divide n = {n}")
    G = n if grid.kind == "colspacing" else (grid.group or n)
    for k, t in (out or {}).items():
        _require_cuda(t)
    if out:
        ng = n // G
        _check(out.get("codes"), "out['codes']", (m, n), _I32)
        _check(out.get("scales"), "out['scales']",
               (n,) if grid.kind == "colspacing" else (m, ng), _F32)
        if grid.kind == "asym":
            _check(out.get("zeros"), "out['zeros']", (m, ng), _I32)
        _check_result(out.get("result"))
        _check(out.get("H"), "out['H']", (n, n), _F32)
        _check(out.get("L"), "out['L']", (n, n), (_tdt(prec),))
    o = dict(out or {})
    if "codes" not in o:
        o["codes"] = torch.empty((m, n), dtype=torch.int32, device=dev)
    if "scales" not in o:
        o["scales"] = (torch.empty(n, dtype=torch.float32, device=dev)
                       if grid.kind == "colspacing"
                       else torch.empty((m, n // G), dtype=torch.float32, device=dev))
    if "zeros" not in o:
        o["zeros"] = (torch.empty((m, n // G), dtype=torch.int32, device=dev)
                      if grid.kind == "asym" else None)
    if "result" not in o:
        o["result"] = new_result(dev)
    if want_H and X is not None and o.get("H") is None:
        o["H"] = torch.empty((n, n), dtype=torch.float32, device=dev)
    if want_L and o.get("L") is None:
        o["L"] = torch.empty((n, n), dtype=_tdt(prec), device=dev)
    ws = workspace if workspace is not None else workspace_for_layer(
        m, n, ntok, X is not None, order, block, prec, dev)
    g = grid.c_struct()
    check(lib().pwq_quant_layer(
        W.data_ptr(), _dtype_code(W), m, n, _row_major(W),
        _ptr(X), xdt, ntok, ldx, _ptr(H), g,
        _lib.ORDERS[order], _ptr(perm), float(damp), int(block), _prec(prec),
        o["codes"].data_ptr(), o["scales"].data_ptr(), _ptr(o["zeros"]),
        o["result"].data_ptr(), _ptr(o.get("H")), _ptr(o.get("L")), ws.data_ptr(),
        ws.numel(), _stream()))
    return o


def column_entropy(codes: torch.Tensor, huffman: bool = False):
    """Per-column empirical entropy (bits) of int32 codes [m, n] and its mean
    over the columns: (bits [n] float64, mean [] float64), both on the GPU;
    with ``huffman`` also each column's Huffman-coded length in bits
    ([n] int64, -1 where not computed) as a third element."""
    _require_cuda(codes)
    if codes.dtype != torch.int32:
        raise TypeError("codes must be int32")
    m, n = codes.shape
    ldc = _row_major(codes) if m > 0 else n
    bits = torch.empty(n, dtype=torch.float64, device=codes.device)
    mean = torch.empty((), dtype=torch.float64, device=codes.device)
    huff = torch.empty(n, dtype=torch.int64, device=codes.device) if huffman else None
    L_ = lib()
    ws = _workspace(L_.pwq_rate_workspace_size(n), codes.device)
    check(L_.pwq_column_entropy(codes.data_ptr(), m, n, ldc, bits.data_ptr(), mean.data_ptr(),
                                _ptr(huff), ws.data_ptr(), ws.numel(), _stream()))
    return (bits, mean, huff) if huffman else (bits, mean)


class KernelTimer:
    """Times one of the library's kernels (pwq_kernel_timer_attach):
    inside the ``with`` block, its first ``capacity`` launches record a pair
    of HIP events on the stream they run on.  ``kernel`` is "hessian_tiles"
    (the SYRK tiles), "lazy_update" (one lazy block update of the sweep) or
    "sweep_block" (one block of the column sweep).  Measurement only."""

    def __init__(self, kernel: str, capacity: int):
        self.kernel = _lib.TIMED_KERNELS[kernel]
        self.starts = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        self.stops = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.starts + self.stops:
            e.record()          # torch creates the HIP event on its first record
        arr = ctypes.c_void_p * max(capacity, 1)
        self._s = arr(*[e.cuda_event for e in self.starts])
        self._e = arr(*[e.cuda_event for e in self.stops])
        self.capacity = capacity
        self.count = 0

    def __enter__(self):
        check(lib().pwq_kernel_timer_attach(self.kernel, self._s, self._e, self.capacity))
        return self

    def __exit__(self, *exc):
        self.count = int(lib().pwq_kernel_timer_count(self.kernel))
        check(lib().pwq_kernel_timer_attach(self.kernel, None, None, 0))
        return False

    def durations_ms(self):
        """Per-launch durations (synchronises)."""
        torch.cuda.synchronize()
        return [a.elapsed_time(b) for a, b in zip(self.starts[:self.count],
                                                  self.stops[:self.count])]


class HessianTileTimer(KernelTimer):
    """KernelTimer of the Hessian product kernel."""

    def __init__(self, capacity: int):
        super().__init__("hessian_tiles", capacity)


def overflow_entries(codes: torch.Tensor, scales: torch.Tensor, grid: Grid,
                     zeros: Optional[torch.Tensor] = None, max_out: Optional[int] = None):
    """Overflow entries of int32 codes [m, n] for a SYM/ASYM grid (SSQR):
    (rows, cols, vals, count) -- the first min(count, max_out) entries of the
    (row, column)-sorted list, and the device int64 count."""
    _require_cuda(codes, scales, zeros)
    if codes.dtype != torch.int32:
        raise TypeError("codes must be int32")
    m, n = codes.shape
    if grid.group and n % grid.group:
        raise ValueError(f"group {grid.group} does not divide n = {n}")
    ng = n // (grid.group or n)
    _check(scales, "scales", (m, ng), _F32)
    _check(zeros, "zeros", (m, ng), _I32)
    ldc = _row_major(codes) if m > 0 else n
    cap = m * n if max_out is None else int(max_out)
    dev = codes.device
    rows = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    cols = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    vals = torch.empty(max(cap, 1), dtype=torch.float32, device=dev)
    count = torch.zeros((), dtype=torch.int64, device=dev)
    L_ = lib()
    ws = _workspace(L_.pwq_overflow_workspace_size(m), dev)
    g = grid.c_struct()
    check(L_.pwq_overflow_entries(codes.data_ptr(), m, n, ldc, g, scales.data_ptr(),
                                  _ptr(zeros), cap, rows.data_ptr(), cols.data_ptr(),
                                  vals.data_ptr(), count.data_ptr(), ws.data_ptr(), ws.numel(),
                                  _stream()))
    return rows, cols, vals, count


def ssqr_quant_layer(W: torch.Tensor, X: Optional[torch.Tensor] = None,
                     H: Optional[torch.Tensor] = None, grid: Grid = Grid(),
                     damp: float = 0.01, block: int = 128, prec: str = "f32",
                     density: float = 0.01, iters: int = 12, log2_lo: float = -8.0,
                     max_outliers: Optional[int] = None, x_layout: str = "channels"):
    """Overflow-tolerant quantization (SSQR): the step multiplier kappa is
    bisected in log2 for at most ``density`` m n outlier codes.  Returns a
    dict: codes, scales, zeros, result, kappa, n_outliers and the outlier
    list rows / cols / vals (trimmed to min(n_outliers, max_outliers)).
    Synchronous."""
    _require_cuda(W, X, H)
    m, n = W.shape
    dev = W.device
    ntok, ldx, xdt = 0, 0, 0
    if X is not None:
        nx, ntok, ldx, xdt = _x_args(X, x_layout)
        if nx != n:
            raise ValueError(f"X has {nx} channels, W has {n} columns")
    _check(H, "H", (n, n), _F32)
    if grid.group and n % grid.group:
        raise ValueError(f"group {grid.group} does not divide n = {n}")
    G = grid.group or n
    cap = m * n if max_outliers is None else int(max_outliers)
    o = {"codes": torch.empty((m, n), dtype=torch.int32, device=dev),
         "scales": torch.empty((m, n // G), dtype=torch.float32, device=dev),
         "zeros": (torch.empty((m, n // G), dtype=torch.int32, device=dev)
                   if grid.kind == "asym" else None),
         "result": new_result(dev)}
    rows = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    cols = torch.empty(max(cap, 1), dtype=torch.int32, device=dev)
    vals = torch.empty(max(cap, 1), dtype=torch.float32, device=dev)
    n_out = ctypes.c_int64(0)
    kappa = ctypes.c_double(0.0)
    L_ = lib()
    ws = _workspace(L_.pwq_ssqr_workspace_size(m, n, ntok, int(X is not None), block,
                                               _prec(prec)), dev)
    g = grid.c_struct()
    check(L_.pwq_ssqr_quant_layer(
        W.data_ptr(), _dtype_code(W), m, n, _row_major(W), _ptr(X), xdt, ntok, ldx, _ptr(H),
        g, float(damp), int(block), _prec(prec), float(density), int(iters), float(log2_lo),
        o["codes"].data_ptr(), o["scales"].data_ptr(), _ptr(o["zeros"]),
        o["result"].data_ptr(), cap, rows.data_ptr(), cols.data_ptr(), vals.data_ptr(),
        ctypes.byref(n_out), ctypes.byref(kappa), ws.data_ptr(), ws.numel(), _stream()))
    k = min(int(n_out.value), cap)
    o.update(kappa=float(kappa.value), n_outliers=int(n_out.value), rows=rows[:k],
             cols=cols[:k], vals=vals[:k])
    return o


# ------------------------------------------------------------ running a packed layer

# A serving step calls these once per layer, so they check with plain
# comparisons and ask for a workspace only where the library wants one.

_DTYPES = {torch.float32: _lib.PWQ_F32, torch.bfloat16: _lib.PWQ_BF16, torch.int8: _lib.PWQ_I8}


def _rows(t: torch.Tensor, name: str, device: int) -> int:
    """Row stride of a 2-D tensor with unit column stride on this GPU."""
    if t.get_device() != device:
        raise ValueError(f"{name} must be on x's GPU")
    return t.shape[1] if t.dim() == 2 and t.is_contiguous() else _row_major(t)


def _expect(t: torch.Tensor, name: str, shape: tuple, dtype: torch.dtype, device: int) -> int:
    """Address of a contiguous tensor of this shape and type on this GPU."""
    if t.get_device() != device:
        raise ValueError(f"{name} must be on x's GPU")
    if t.shape != shape or t.dtype is not dtype or not t.is_contiguous():
        _check(t, name, shape, (dtype,))
    return t.data_ptr()


def _on_device(device: int):
    """The context of a call whose input is not on the current GPU."""
    if device < 0:
        raise ValueError("x must be on the GPU")
    return torch.cuda.device(device)


def _no_gradient(*ts):
    for t in ts:
        if t is not None and t.requires_grad:
            raise ValueError("a tensor requires a gradient, which this call does not give: "
                             "call it under torch.no_grad(), or detach the tensor")


def pack_weights(codes: torch.Tensor, scales: torch.Tensor, grid: Grid,
                 zeros: Optional[torch.Tensor] = None) -> dict:
    """Codes [m, n] int32, steps and zero points of a SYM / ASYM grid of at
    most 4 bits (as returned by quant_layer or ssqr_quant_layer) -> the packed
    layer that packed_linear reads: dict(qweight, scales, zeros, n, group,
    outlier_off, outliers).  Codes outside 4 bits go into the overflow list,
    so nothing is clipped.  Raises ValueError where a lattice step exceeds
    127.  Synchronous (the list's length is read on the host); runs on codes'
    GPU, on its current stream."""
    _require_cuda(codes, scales, zeros)
    index = codes.get_device()
    if any(t is not None and t.get_device() != index for t in (scales, zeros)):
        raise ValueError("scales and zeros must be on codes' GPU")
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return pack_weights(codes, scales, grid, zeros)
    if codes.dtype != torch.int32:
        raise TypeError("codes must be int32")
    m, n = codes.shape
    if grid.kind not in ("sym", "asym"):
        raise ValueError("a packed layer has group steps: grid kind sym or asym")
    if grid.group and n % grid.group:
        raise ValueError(f"group {grid.group} does not divide n = {n}")
    ng = n // (grid.group or n)
    asym = grid.kind == "asym"
    _check(scales, "scales", (m, ng), _F32)
    _check(zeros, "zeros", (m, ng), _I32)
    if asym and zeros is None:
        raise ValueError("an asym grid needs zeros")
    ldc = _row_major(codes) if m > 0 else n
    dev = codes.device
    L_ = lib()
    g = grid.c_struct()
    qweight = torch.empty((m, L_.pwq_packed_row_bytes(n)), dtype=torch.uint8, device=dev)
    zeros8 = torch.empty((m, ng), dtype=torch.uint8, device=dev) if asym else None
    off = torch.empty(L_.pwq_pack_tiles(m, n) + 1, dtype=torch.int32, device=dev)
    info = torch.empty(2, dtype=torch.int32, device=dev)
    check(L_.pwq_pack_codes(codes.data_ptr(), m, n, ldc, g, _ptr(zeros) if asym else None,
                            qweight.data_ptr(), _ptr(zeros8), off.data_ptr(), info.data_ptr(),
                            _stream()))
    count, wide, bad = torch.cat((off[-1:], info)).tolist()
    if wide or bad:
        raise ValueError(f"{wide} codes are more than 127 steps from zero and {bad} zero points "
                         "lie outside 0 .. 127: the layer cannot be packed")
    outliers = None
    if count:
        outliers = torch.empty(count, dtype=torch.int32, device=dev)
        check(L_.pwq_pack_overflow(codes.data_ptr(), m, n, ldc, g, off.data_ptr(),
                                   outliers.data_ptr(), count, _stream()))
    return {"qweight": qweight, "scales": scales, "zeros": zeros8, "n": n,
            "group": grid.group or n, "outlier_off": off if count else None,
            "outliers": outliers}


def rms_norm(x: torch.Tensor, weight: torch.Tensor, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-6, out_dtype: Optional[torch.dtype] = None,
             sum_out: Optional[torch.Tensor] = None):
    """Root-mean-square norm of x (+ residual), [tokens, n] bf16 or fp32, per
    token: (y, scales or None, sum or None).  ``out_dtype`` is bf16, fp32
    (default: x's) or int8, which comes with a step per token (scales [tokens]
    fp32, y = codes).  ``sum`` is x + residual in x's type, written to
    ``sum_out`` where given (x or residual itself for in place).  Runs on x's
    GPU, on its current stream.  Gives no gradients, and refuses tensors that
    require one unless they are off (torch.no_grad())."""
    dev = x.get_device()
    if dev != torch._C._cuda_getDevice():
        with _on_device(dev):
            return rms_norm(x, weight, residual, eps, out_dtype, sum_out)
    if torch.is_grad_enabled():
        _no_gradient(x, weight, residual, sum_out)
    ldx = _rows(x, "x", dev)
    ntok, n = x.shape
    xdt = _dtype_code(x)
    wdt = _dtype_code(weight)
    wp = _expect(weight, "weight", (n,), weight.dtype, dev)
    odt = x.dtype if out_dtype is None else out_dtype
    ydt = _DTYPES.get(odt)
    if ydt is None:
        raise TypeError(f"unsupported output dtype {odt}")
    total, rp, ldr, tp, lds = sum_out, None, 0, None, 0
    if residual is not None:
        if residual.shape != x.shape or residual.dtype is not x.dtype:
            raise ValueError("residual must have x's shape and type")
        rp, ldr = residual.data_ptr(), _rows(residual, "residual", dev)
        if total is None:
            total, lds = torch.empty_like(x, memory_format=torch.contiguous_format), n
        elif total.shape != x.shape or total.dtype is not x.dtype:
            raise ValueError("sum_out must have x's shape and type")
        else:
            lds = _rows(total, "sum_out", dev)
        tp = total.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out goes with a residual")
    y = torch.empty_like(x, dtype=odt, memory_format=torch.contiguous_format)
    scales, sp = None, None
    if ydt == _lib.PWQ_I8:
        scales = x.new_empty(ntok, dtype=torch.float32)
        sp = scales.data_ptr()
    status = lib().pwq_rms_norm(x.data_ptr(), xdt, ntok, n, ldx, rp, ldr, wp, wdt, eps, tp, lds,
                                y.data_ptr(), ydt, n, sp, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        check(status)
    return y, scales, total


def packed_linear(x: torch.Tensor, packed: dict, x_scales: Optional[torch.Tensor] = None,
                  out_dtype: Optional[torch.dtype] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [tokens, m] = x [tokens, n] times a packed layer (pack_weights).  x is
    bf16, fp32, or int8 with a step per token (``x_scales`` [tokens] fp32, as
    from rms_norm).  ``out_dtype`` is bf16 or fp32 (default: x's; bf16 for
    int8); ``out`` may pass the result's memory.  Runs on x's GPU, on its
    current stream.  Gives no gradients, and refuses tensors that require one
    unless they are off (torch.no_grad())."""
    dev = x.get_device()
    if dev != torch._C._cuda_getDevice():
        with _on_device(dev):
            return packed_linear(x, packed, x_scales, out_dtype, out)
    if torch.is_grad_enabled():
        _no_gradient(x, x_scales, packed["scales"], out)
    q, zeros, outliers = packed["qweight"], packed["zeros"], packed["outliers"]
    n, group = packed["n"], packed["group"]
    ldx = _rows(x, "x", dev)
    ntok, cols = x.shape
    m = q.shape[0]
    if cols != n:
        raise ValueError(f"x has {cols} columns, the layer {n}")
    xdt = _DTYPES.get(x.dtype)
    if xdt is None:
        raise TypeError(f"unsupported dtype {x.dtype}")
    if group <= 0 or n % group:
        raise ValueError(f"group {group} does not divide n = {n}")
    qp = _expect(q, "qweight", (m, (n + 31) // 32 * 16), torch.uint8, dev)
    sp = _expect(packed["scales"], "scales", (m, n // group), torch.float32, dev)
    zp = offp = outp = xsp = None
    n_out = 0
    if zeros is not None:
        zp = _expect(zeros, "zeros", (m, n // group), torch.uint8, dev)
    if outliers is not None:
        n_out = outliers.shape[0]
        outp = _expect(outliers, "outliers", (n_out,), torch.int32, dev)
        offp = _expect(packed["outlier_off"], "outlier_off",
                       ((m + 15) // 16 * ((n + 127) // 128) + 1,), torch.int32, dev)
    if x_scales is not None:
        xsp = _expect(x_scales, "x_scales", (ntok,), torch.float32, dev)
    if (xdt == _lib.PWQ_I8) != (x_scales is not None):
        raise ValueError("x_scales goes with int8 x, and only with it")
    odt = out_dtype
    if odt is None:
        odt = out.dtype if out is not None else (torch.bfloat16 if xdt == _lib.PWQ_I8
                                                 else x.dtype)
    if odt is not torch.bfloat16 and odt is not torch.float32:
        raise TypeError(f"unsupported output dtype {odt}")
    if out is None:
        out, ldy = x.new_empty((ntok, m), dtype=odt), m
    else:
        if out.shape != (ntok, m) or out.dtype is not odt:
            raise ValueError(f"out must be [{ntok}, {m}] {odt}")
        ldy = _rows(out, "out", dev) if ntok and m else m
    L_, stream = lib(), torch._C._cuda_getCurrentRawStream(dev)
    ws, nb = None, 0
    while True:
        status = L_.pwq_packed_linear(x.data_ptr(), xdt, ntok, ldx, xsp, qp, m, n, sp, zp, group,
                                      offp, outp, n_out, out.data_ptr(), _DTYPES[odt], ldy,
                                      None if ws is None else ws.data_ptr(), nb, stream)
        if status != _lib.PWQ_ERR_WORKSPACE or ws is not None:
            break
        ws = _workspace(L_.pwq_packed_linear_workspace_size(x.data_ptr(), xdt, ntok, ldx, m, n,
                                                            group, n_out), x.device)
        nb = ws.numel()
    if status:
        check(status)
    return out


# ------------------------------------------------------------ the key-value cache

def new_cache(pages: int, kv_heads: int, head_dim: int, bits: int = 8, page: int = 64,
              device="cuda") -> dict:
    """An empty key-value cache of ``pages`` pages of ``page`` tokens (a power of
    two, 32 .. 4096), for heads of 64, 128 or 256 channels in 8 or 4 bits:
    dict(records [pages, kv_heads, page / 32, bytes of a record] uint8, bits,
    head_dim, page)."""
    size = lib().pwq_cache_record_bytes(head_dim, bits)
    if not size:
        raise ValueError("a cache has head_dim 64, 128 or 256 and 4 or 8 bits")
    if page < 32 or page > 4096 or page & (page - 1):
        raise ValueError("page must be a power of two in 32 .. 4096")
    if pages < 0 or kv_heads < 1:
        raise ValueError("need pages >= 0 and kv_heads >= 1")
    records = torch.zeros((pages, kv_heads, page // 32, size), dtype=torch.uint8, device=device)
    return {"records": records, "bits": bits, "head_dim": head_dim, "page": page}


# pwq_cache and pwq_batch of include/pwq_cache.h, packed (half the time of filling
# ctypes structures)
_PACK_CACHE = struct.Struct("@Pqiiii").pack
_PACK_BATCH = struct.Struct("@PPPqii").pack


def _cache_args(cache: dict, starts, lengths, table, device: int):
    """(pwq_cache, pwq_batch, kv_heads, head_dim, sizes that the workspace goes by) of
    tensors on this GPU."""
    records, page, bits, dim = cache["records"], cache["page"], cache["bits"], cache["head_dim"]
    rs, ts = records.shape, table.shape
    if len(rs) != 4 or records.dtype is not torch.uint8 or not records.is_contiguous():
        raise ValueError("records must be a contiguous 4-D uint8 tensor")
    pages, heads, blocks, size = rs
    if blocks * 32 != page or size != 8 * dim * bits + 256:
        raise ValueError(f"records of {tuple(rs)} do not fit pages of {page} tokens, "
                         f"{dim} channels and {bits} bits")
    if len(ts) != 2 or table.dtype is not torch.int32:
        raise ValueError("table must be a 2-D int32 tensor")
    nseq, width = ts
    if not (records.get_device() == table.get_device() == device):
        raise ValueError("the cache and the table must be on the tensors' GPU")
    ld = width
    if not table.is_contiguous():
        ld = table.stride(0)
        if width > 1 and table.stride(1) != 1 or nseq > 1 and ld < width:
            raise ValueError("table must be row-major")
        ld = max(ld, width)
    return (_PACK_CACHE(records.data_ptr(), pages, heads, dim, bits, page),
            _PACK_BATCH(_expect(starts, "starts", (nseq + 1,), torch.int32, device),
                        _expect(lengths, "lengths", (nseq,), torch.int32, device),
                        table.data_ptr(), ld, nseq, width),
            heads, dim, (pages, heads, dim, bits, page, nseq, width))


@functools.lru_cache(maxsize=256)
def _attention_workspace(sizes, prefix_width, heads, dtype, tokens) -> int:
    pages, kv_heads, dim, bits, page, nseq, width = sizes
    p = None if prefix_width < 0 else _PACK_BATCH(0, 0, 0, prefix_width, 1, prefix_width)
    return lib().pwq_cached_attention_workspace_size(
        _PACK_CACHE(0, pages, kv_heads, dim, bits, page),
        _PACK_BATCH(0, 0, 0, width, nseq, width), p, heads, dtype, tokens)


def _heads(t: torch.Tensor, name: str, shape: tuple, dtype, device: int):
    """Strides of a [tokens, heads, head_dim] tensor with unit channel stride."""
    if t.get_device() != device or t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be {list(shape)} {dtype} on the cache's GPU")
    ts, hs, ds = t.stride()
    if ds != 1:
        raise ValueError(f"{name} must have unit channel stride")
    return ts, hs


def cache_write(k: torch.Tensor, v: torch.Tensor, cache: dict, starts: torch.Tensor,
                lengths: torch.Tensor, table: torch.Tensor) -> None:
    """Quantizes keys and values [tokens, kv_heads, head_dim] (bf16 or fp32, any
    token and head stride) into a cache, one step and zero point per token and
    head.  The batch is ragged: rows starts[i] .. starts[i + 1] - 1 are the last
    of the lengths[i] tokens of sequence i (these rows included), whose token p
    lies in page table[i, p // page].  ``starts`` [n + 1], ``lengths`` [n] and
    ``table`` [n, width] are int32 on the GPU; a captured call reads them anew on
    every replay.  Rows of no sequence, and tokens whose page is none of the
    cache's (-1, say), are left out.  Runs on k's GPU, on its current stream.
    Gives no gradients, and refuses tensors that require one unless they are off
    (torch.no_grad())."""
    dev = k.get_device()
    if dev != torch._C._cuda_getDevice():
        with _on_device(dev):
            return cache_write(k, v, cache, starts, lengths, table)
    if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
        _no_gradient(k, v)
    c, b, heads, dim, _ = _cache_args(cache, starts, lengths, table, dev)
    shape = (*k.shape[:1], heads, dim)
    kts, khs = _heads(k, "k", shape, k.dtype, dev)
    vts, vhs = _heads(v, "v", shape, k.dtype, dev)
    status = lib().pwq_cache_write(c, b, k.data_ptr(), kts, khs, v.data_ptr(), vts, vhs,
                                   _dtype_code(k), shape[0],
                                   torch._C._cuda_getCurrentRawStream(dev))
    if status:
        check(status)


def cache_read(cache: dict, starts: torch.Tensor, lengths: torch.Tensor, table: torch.Tensor,
               tokens: int, dtype: torch.dtype = torch.bfloat16, out: Optional[tuple] = None):
    """(k, v) [tokens, kv_heads, head_dim] that a cache holds for the rows of a
    batch as for cache_write (for whole sequences: starts that count all of their
    tokens); fp32 is exact, bf16 rounded once.  Tokens of pages that are none of
    the cache's read as 0.  ``out`` may pass (k, v); their rows of no sequence
    keep what was there, and are unspecified where the call allocates.  Runs on
    the cache's GPU, on its current stream."""
    dev = cache["records"].get_device()
    if dev != torch._C._cuda_getDevice():
        with _on_device(dev):
            return cache_read(cache, starts, lengths, table, tokens, dtype, out)
    c, b, heads, dim, _ = _cache_args(cache, starts, lengths, table, dev)
    shape = (tokens, heads, dim)
    if out is None:
        k = cache["records"].new_empty(shape, dtype=dtype)
        v = torch.empty_like(k)
        kts = vts = heads * dim
        khs = vhs = dim
    else:
        k, v = out
        if (k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
            _no_gradient(k, v)
        kts, khs = _heads(k, "k", shape, k.dtype, dev)
        vts, vhs = _heads(v, "v", shape, k.dtype, dev)
    status = lib().pwq_cache_read(c, b, k.data_ptr(), kts, khs, v.data_ptr(), vts, vhs,
                                  _dtype_code(k), tokens, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        check(status)
    return k, v


def cached_attention(q: torch.Tensor, cache: dict, starts: torch.Tensor, lengths: torch.Tensor,
                     table: torch.Tensor, scale: Optional[float] = None, causal: bool = True,
                     prefix: Optional[tuple] = None,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of q [tokens, heads, head_dim] (bf16 or fp32, any token and head
    stride; heads a multiple of the cache's) over a cache, for a batch as for
    cache_write; query head h reads key head h // (heads / kv_heads).  A row sees
    its sequence's tokens up to its own (``causal``), which have to be written, or
    all of them.  ``scale`` defaults to head_dim ** -0.5.  ``prefix`` = (pages
    int32 [n], length int32 [1], both on the GPU) names tokens of the cache that
    come before those of every sequence: they are read once for the whole batch,
    and neither ``table`` nor ``lengths`` counts them.  A row that sees no token
    gives 0.  ``out`` may pass the result's memory (q's shape and type; must not
    overlap q); rows of no sequence keep what was there, and are unspecified
    where the call allocates.  Runs on q's GPU, on its current stream.  Gives no
    gradients, and refuses tensors that require one unless they are off
    (torch.no_grad())."""
    dev = q.get_device()
    if dev != torch._C._cuda_getDevice():
        with _on_device(dev):
            return cached_attention(q, cache, starts, lengths, table, scale, causal, prefix, out)
    if (q.requires_grad or out is not None and out.requires_grad) and torch.is_grad_enabled():
        _no_gradient(q, out)
    c, b, _, dim, sizes = _cache_args(cache, starts, lengths, table, dev)
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    tokens, heads, _ = shape
    qts, qhs = _heads(q, "q", (tokens, heads, dim), q.dtype, dev)
    dtype = _dtype_code(q)
    if out is None:
        out, ots, ohs = q.new_empty(shape), heads * dim, dim
    else:
        ots, ohs = _heads(out, "out", shape, q.dtype, dev)
    p, n = None, -1
    if prefix is not None:
        pages, length = prefix
        n = pages.shape[0] if pages.dim() == 1 else -1
        p = _PACK_BATCH(0, _expect(length, "the prefix's length", (1,), torch.int32, dev),
                        _expect(pages, "the prefix's pages", (n,), torch.int32, dev), n, 1, n)
    ws, nb = None, _attention_workspace(sizes, n, heads, dtype, tokens)
    if nb:
        ws = q.new_empty(nb, dtype=torch.uint8)
    status = lib().pwq_cached_attention(
        c, b, p, q.data_ptr(), qts, qhs, out.data_ptr(), ots, ohs, heads, dtype, tokens,
        dim ** -0.5 if scale is None else scale, causal, None if ws is None else ws.data_ptr(),
        nb, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        check(status)
    return out
