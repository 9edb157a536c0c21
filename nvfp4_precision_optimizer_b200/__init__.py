"""Direct NVFP4 Newton-Schulz orthogonalisation (the Q-Root step of "Full-Stack
FP4", arXiv 2607.04422, Section 3.4), MXFP4 quantisation and products, and the Muon
step on NVIDIA B200.

Every step runs in the sm_100a kernels of libfs4.so behind the C ABI declared
in include/fs4.h; this module only marshals torch tensors (device memory and
streams) into those calls.  There is no CPU or fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Sequence

import torch

from . import _lib
from ._lib import (FS4_AXIS_COL, FS4_AXIS_ROW, FS4_LAYOUT_TILED, FS4_NS_ADAPTIVE46, FS4_NS_CLIP_QUANTILE, FS4_NS_RHT,
                   FS4_SG_AMAX, FS4_TEST_STALL, Fs4Error, NsDesc, NsLayout, check, stop_after)

MUON_COEFFS = (3.4445, -4.7750, 2.0315)

__all__ = [
    "quantize", "quantize_batched", "dequantize", "gemm", "root_ns", "root_ns_batched", "ns_workspace_size",
    "ns_batched_workspace_size", "ns_layout", "device_status", "tiled_shape", "Fs4Error",
    "momentum_nvfp4", "root_ns_batched_nvfp4", "root_ns_bf16_batched", "ns_bf16_batched_workspace_size",
    "ns_bf16_layout",
    "mxfp4_quantize", "mxfp4_quantize_both", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_linear",
    "mxfp4_linear_workspace_size", "mxfp4_tiled_shape",
    "muon_orthogonalize", "muon_step", "muon_workspace_size",
    "MUON_COEFFS", "stop_after", "FS4_AXIS_ROW", "FS4_AXIS_COL", "FS4_TEST_STALL",
    "FS4_NS_RHT", "FS4_NS_ADAPTIVE46", "FS4_NS_CLIP_QUANTILE",
]


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check_f32_matrix(x: torch.Tensor, name: str) -> None:
    if not x.is_cuda or x.dtype != torch.float32 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be a CUDA float32 matrix with unit column stride")


def _round_up(v: int, a: int) -> int:
    return (v + a - 1) // a * a


def tiled_shape(rows: int, cols: int) -> tuple[int, int]:
    """(codes bytes, scales bytes) of a rows x cols matrix in the TILED layout."""
    rp, cp = _round_up(rows, 128), _round_up(cols, 256)
    return rp * cp // 2, rp * cp // 16


def quantize(x: torch.Tensor, axis: int = FS4_AXIS_ROW, tiled: bool = False,
             sg_mode: str = "pow2", workspace: torch.Tensor | None = None, stream=None,
             flags: int = 0):
    """NVFP4-quantise x (fs4_nvfp4_quantize).  Returns (codes, scales, s_g).
    flags: extra call flags (FS4_TEST_STALL for the timeout test)."""
    _check_f32_matrix(x, "x")
    rows, cols = x.shape
    R, C = (rows, cols) if axis == FS4_AXIS_ROW else (cols, rows)
    if tiled:
        ncode, nscale = tiled_shape(R, C)
        codes = torch.empty(ncode, dtype=torch.uint8, device=x.device)
        scales = torch.empty(nscale, dtype=torch.uint8, device=x.device)
    else:
        codes = torch.empty((R, C // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((R, max(C // 16, 1)), dtype=torch.uint8, device=x.device)
    s_g = torch.empty(1, dtype=torch.float32, device=x.device)
    ws_bytes = _lib.lib().fs4_nvfp4_quantize_workspace_size()
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=x.device)
    flags |= (FS4_LAYOUT_TILED if tiled else 0) | (FS4_SG_AMAX if sg_mode == "amax" else 0)
    ld = x.stride(0) if rows > 1 else cols
    check(_lib.lib().fs4_nvfp4_quantize(x.data_ptr(), rows, cols, ld, axis,
                                        codes.data_ptr(), scales.data_ptr(), s_g.data_ptr(), flags,
                                        workspace.data_ptr(), workspace.numel(), _stream(stream)),
          "fs4_nvfp4_quantize")
    return codes, scales, s_g


def quantize_batched(xs: Sequence[torch.Tensor], axis: int = FS4_AXIS_ROW, tiled: bool = False,
                     sg_mode: str = "pow2", workspace: torch.Tensor | None = None, stream=None,
                     flags: int = 0):
    """fs4_nvfp4_quantize on every matrix of xs in one launch
    (fs4_nvfp4_quantize_batched).  Returns a list of (codes, scales, s_g)."""
    outs = []
    arr = (_lib.QuantDesc * len(xs))()
    for i, x in enumerate(xs):
        _check_f32_matrix(x, "x")
        rows, cols = x.shape
        R, C = (rows, cols) if axis == FS4_AXIS_ROW else (cols, rows)
        if tiled:
            ncode, nscale = tiled_shape(R, C)
            codes = torch.empty(ncode, dtype=torch.uint8, device=x.device)
            scales = torch.empty(nscale, dtype=torch.uint8, device=x.device)
        else:
            codes = torch.empty((R, C // 2), dtype=torch.uint8, device=x.device)
            scales = torch.empty((R, max(C // 16, 1)), dtype=torch.uint8, device=x.device)
        s_g = torch.empty(1, dtype=torch.float32, device=x.device)
        ld = x.stride(0) if rows > 1 else cols
        arr[i] = _lib.QuantDesc(x.data_ptr(), rows, cols, ld, axis, codes.data_ptr(), scales.data_ptr(),
                                s_g.data_ptr())
        outs.append((codes, scales, s_g))
    need = int(_lib.lib().fs4_nvfp4_quantize_batched_workspace_size(len(xs)))
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=xs[0].device)
    flags |= (FS4_LAYOUT_TILED if tiled else 0) | (FS4_SG_AMAX if sg_mode == "amax" else 0)
    check(_lib.lib().fs4_nvfp4_quantize_batched(len(xs), arr, flags, workspace.data_ptr(),
                                                workspace.numel(), _stream(stream)),
          "fs4_nvfp4_quantize_batched")
    return outs


def dequantize(codes: torch.Tensor, scales: torch.Tensor, s_g: torch.Tensor, rows: int, cols: int,
               tiled: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """FP32 rows x cols matrix from an NVFP4 one (fs4_nvfp4_dequantize); `out`, if
    given, is a rows x cols FP32 view with unit column stride (any row stride)."""
    if out is None:
        y = torch.empty((rows, cols), dtype=torch.float32, device=codes.device)
    else:
        _check_f32_matrix(out, "out")
        if tuple(out.shape) != (rows, cols):
            raise ValueError(f"out must be {rows} x {cols}, got {tuple(out.shape)}")
        y = out
    check(_lib.lib().fs4_nvfp4_dequantize(codes.data_ptr(), scales.data_ptr(), s_g.data_ptr(),
                                          rows, cols, y.data_ptr(), _ld(y),
                                          FS4_LAYOUT_TILED if tiled else 0, _stream(stream)),
          "fs4_nvfp4_dequantize")
    return y


def momentum_nvfp4(g: torch.Tensor, beta: float, state=None, prev_mask: int = 0, mask: int = 0,
                   seed: int = 0, want_m: bool = True, out_state=None,
                   workspace: torch.Tensor | None = None, stream=None):
    """One step of the NVFP4-stored first moment (fs4_momentum_nvfp4).  state / out_state
    are (codes, scales, s_g) triples in the PLAIN layout (out_state may be `state` for an
    in-place step).  Returns (m_t FP32 or None, new state)."""
    _check_f32_matrix(g, "g")
    rows, cols = g.shape
    dev = g.device
    if out_state is None:
        out_state = (torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev),
                     torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev),
                     torch.empty(1, dtype=torch.float32, device=dev))
    m_out = torch.empty_like(g) if want_m else None
    if workspace is None:
        workspace = torch.empty(_lib.lib().fs4_momentum_workspace_size(), dtype=torch.uint8, device=dev)
    prev = (None, None, None) if state is None else tuple(t.data_ptr() for t in state)
    check(_lib.lib().fs4_momentum_nvfp4(g.data_ptr(), rows, cols, _ld(g), beta, prev[0], prev[1],
                                        prev[2], prev_mask, out_state[0].data_ptr(),
                                        out_state[1].data_ptr(), out_state[2].data_ptr(), mask,
                                        seed, _ptr(m_out), _ld(m_out) if want_m else cols,
                                        workspace.data_ptr(), workspace.numel(), _stream(stream)),
          "fs4_momentum_nvfp4")
    return m_out, out_state


def gemm(a, b, M: int, N: int, K: int, out: torch.Tensor | None = None,
         workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """D = deq(A) deq(B)^T on the tensor cores (fs4_nvfp4_gemm); a, b are
    (codes, scales, s_g) triples in the TILED layout, A M x K and B N x K."""
    dev = a[0].device
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(256, dtype=torch.uint8, device=dev)
    check(_lib.lib().fs4_nvfp4_gemm(a[0].data_ptr(), a[1].data_ptr(), a[2].data_ptr(),
                                    b[0].data_ptr(), b[1].data_ptr(), b[2].data_ptr(), M, N, K,
                                    out.data_ptr(), _ld(out), workspace.data_ptr(),
                                    workspace.numel(), _stream(stream)),
          "fs4_nvfp4_gemm")
    return out


_DTYPES = {torch.float32: _lib.FS4_F32, torch.bfloat16: _lib.FS4_BF16, torch.float16: _lib.FS4_F16}


def _check_matrix(x: torch.Tensor, name: str, device: torch.device | None = None) -> None:
    if not x.is_cuda or x.dtype not in _DTYPES or x.dim() != 2 or (x.stride(1) != 1 and x.shape[1] > 1):
        raise ValueError(f"{name} must be a CUDA float32, bfloat16 or float16 matrix with unit column stride")
    if device is not None and x.device != device:
        raise ValueError(f"{name} is on {x.device}, not on {device}")


def _check_bytes(t: torch.Tensor, need: int, name: str, device: torch.device) -> None:
    if t.dtype is not torch.uint8 or t.numel() < need or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 tensor of at least {need} bytes on {device}")


def _here(device: torch.device, stream) -> bool:
    """Whether a call can go to the current stream of the current device."""
    return stream is None and device.index == torch._C._cuda_getDevice()


def _handle(device: torch.device) -> int:
    return torch._C._cuda_getCurrentRawStream(device.index)


@contextlib.contextmanager
def _at(device: torch.device, stream):
    """Makes `device` and `stream` (None: the device's current one) current, so that what a call
    allocates or zeroes belongs to the stream it runs on."""
    if stream is not None and stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


# Where MXFP4 and Muon calls without a workspace of the caller's report: 256 bytes for each stream,
# zero at first and after device_status() has read them.
_status_words: dict[tuple[int, int], torch.Tensor] = {}


def _status_word(device: torch.device) -> torch.Tensor:
    key = (device.index, _handle(device))
    word = _status_words.get(key)
    if word is None:
        word = torch.zeros(256, dtype=torch.uint8, device=device)
        if not torch.cuda.is_current_stream_capturing():     # (a graph's memory is not ours to keep)
            word = _status_words.setdefault(key, word)
    return word


def mxfp4_tiled_shape(rows: int, cols: int) -> tuple[int, int]:
    """(codes bytes, scales bytes) of a rows x cols MXFP4 matrix in the TILED layout."""
    padded = (rows + 127) // 128 * 128 * ((cols + 255) // 256 * 256)
    return padded // 2, padded // 32


def _mx_sizes(rows: int, cols: int, tiled: bool) -> tuple[int, int]:
    return mxfp4_tiled_shape(rows, cols) if tiled else (rows * ((cols + 1) // 2), rows * ((cols + 31) // 32))


def _mx_check(op, rows: int, cols: int, tiled: bool, name: str, device) -> None:
    """(codes, scales) of a rows x cols view."""
    codes, scales = op
    n_codes, n_scales = _mx_sizes(rows, cols, tiled)
    _check_bytes(codes, n_codes, name, device)
    _check_bytes(scales, n_scales, name, device)


def _mx_view(rows: int, cols: int, tiled: bool, device, out):
    if out is not None:
        _mx_check(out, rows, cols, tiled, "out", device)
        return out
    if tiled:
        a, b = mxfp4_tiled_shape(rows, cols)
        return (torch.empty(a, dtype=torch.uint8, device=device), torch.empty(b, dtype=torch.uint8, device=device))
    return (torch.empty((rows, (cols + 1) // 2), dtype=torch.uint8, device=device),
            torch.empty((rows, (cols + 31) // 32), dtype=torch.uint8, device=device))


def _mx_scale_flag(scale_rule: str) -> int:
    if scale_rule == "floor":
        return 0
    if scale_rule != "ceil":
        raise ValueError(f"scale_rule must be 'floor' or 'ceil', not {scale_rule!r}")
    return _lib.FS4_MX_SCALE_CEIL


def _mx_quantize(x, row, col, tiled, scale_rule, seed):
    flags = _mx_scale_flag(scale_rule) | (FS4_LAYOUT_TILED if tiled else 0)
    if x.numel() == 0:           # as an expert without tokens has; the views are empty too
        return
    if seed is None:
        seed = 0
    else:
        flags |= _lib.FS4_MX_STOCHASTIC
        seed = int(seed) & 0xFFFFFFFFFFFFFFFF
    rows, cols = x.shape
    rc, rs = (None, None) if row is None else (row[0].data_ptr(), row[1].data_ptr())
    cc, cs = (None, None) if col is None else (col[0].data_ptr(), col[1].data_ptr())
    check(_lib.lib().fs4_mxfp4_quantize(x.data_ptr(), _DTYPES[x.dtype], rows, cols, _ld(x), rc, rs, cc, cs, flags, seed,
                                        _handle(x.device)),
          "fs4_mxfp4_quantize")


def mxfp4_quantize(x: torch.Tensor, axis: int = FS4_AXIS_ROW, tiled: bool = False, scale_rule: str = "floor",
                   seed: int | None = None, out=None, stream=None):
    """MXFP4-quantise an FP32, BF16 or FP16 matrix (fs4_mxfp4_quantize): its row view, or with
    FS4_AXIS_COL the row view of x^T.  scale_rule "floor" is the MX specification's, "ceil"
    saturates nothing; a seed rounds stochastically.  Returns (codes, scales); `out` is such
    a pair to write into."""
    _check_matrix(x, "x")
    dev = x.device
    if not _here(dev, stream):
        with _at(dev, stream):
            return mxfp4_quantize(x, axis, tiled, scale_rule, seed, out)
    rows, cols = x.shape
    if axis == FS4_AXIS_ROW:
        view = _mx_view(rows, cols, tiled, dev, out)
        _mx_quantize(x, view, None, tiled, scale_rule, seed)
    elif axis == FS4_AXIS_COL:
        view = _mx_view(cols, rows, tiled, dev, out)
        _mx_quantize(x, None, view, tiled, scale_rule, seed)
    else:
        raise ValueError(f"axis must be FS4_AXIS_ROW or FS4_AXIS_COL, not {axis}")
    return view


def mxfp4_quantize_both(x: torch.Tensor, tiled: bool = False, scale_rule: str = "floor", seed: int | None = None,
                        out=None, stream=None):
    """The row view and the column view of x in one pass over it (fs4_mxfp4_quantize), as a
    training step needs them.  Returns ((codes, scales) of x, (codes, scales) of x^T)."""
    _check_matrix(x, "x")
    dev = x.device
    if not _here(dev, stream):
        with _at(dev, stream):
            return mxfp4_quantize_both(x, tiled, scale_rule, seed, out)
    rows, cols = x.shape
    row = _mx_view(rows, cols, tiled, dev, None if out is None else out[0])
    col = _mx_view(cols, rows, tiled, dev, None if out is None else out[1])
    _mx_quantize(x, row, col, tiled, scale_rule, seed)
    return row, col


def _mx_out(out, rows: int, cols: int, dtype, device):
    if out is None:
        if dtype not in _DTYPES:
            raise ValueError(f"dtype must be float32, bfloat16 or float16, not {dtype}")
        return torch.empty((rows, cols), dtype=dtype, device=device)
    _check_matrix(out, "out", device)
    if out.shape[0] != rows or out.shape[1] != cols:
        raise ValueError(f"out must be {rows} x {cols}, got {tuple(out.shape)}")
    return out


def _mx_empty(d, K: int, accumulate: bool) -> bool:
    """Whether a product has no rows, columns or terms; without terms D is 0, or stays."""
    if K == 0 and not accumulate:
        d.zero_()
    return K == 0 or d.numel() == 0


def mxfp4_dequantize(codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, tiled: bool = False,
                     dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values of a rows x cols MXFP4 matrix (fs4_mxfp4_dequantize) in `dtype`, or in `out`."""
    dev = codes.device
    _mx_check((codes, scales), rows, cols, tiled, "codes and scales", dev)
    if not _here(dev, stream):
        with _at(dev, stream):
            return mxfp4_dequantize(codes, scales, rows, cols, tiled, dtype, out)
    y = _mx_out(out, rows, cols, dtype, dev)
    if y.numel() == 0:
        return y
    check(_lib.lib().fs4_mxfp4_dequantize(codes.data_ptr(), scales.data_ptr(), rows, cols, y.data_ptr(), _DTYPES[y.dtype],
                                          _ld(y), FS4_LAYOUT_TILED if tiled else 0, _handle(dev)),
          "fs4_mxfp4_dequantize")
    return y


def mxfp4_gemm(a, b, M: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               accumulate: bool = False, workspace: torch.Tensor | None = None, stream=None, flags: int = 0) -> torch.Tensor:
    """D = deq(A) deq(B)^T, or D += with accumulate (fs4_mxfp4_gemm); a and b are (codes,
    scales) in the TILED layout, A M x K and B N x K.  M, N or K may be 0, as for an expert
    without tokens.  A workspace of the caller's is zeroed once, before its first call.
    flags: extra call flags (FS4_TEST_STALL for the timeout test)."""
    dev = a[0].device
    _mx_check(a, M, K, True, "a", dev)
    _mx_check(b, N, K, True, "b", dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if not _here(dev, stream):
        with _at(dev, stream):
            return mxfp4_gemm(a, b, M, N, K, dtype, out, accumulate, workspace, None, flags)
    d = _mx_out(out, M, N, dtype, dev)
    if _mx_empty(d, K, accumulate):
        return d
    if workspace is None:
        workspace = _status_word(dev)
    else:
        _check_bytes(workspace, 256, "workspace", dev)
    check(_lib.lib().fs4_mxfp4_gemm(a[0].data_ptr(), a[1].data_ptr(), b[0].data_ptr(), b[1].data_ptr(), M, N, K, d.data_ptr(),
                                    _DTYPES[d.dtype], _ld(d), flags | (_lib.FS4_MX_ACCUMULATE if accumulate else 0),
                                    workspace.data_ptr(), workspace.numel(), _handle(dev)),
          "fs4_mxfp4_gemm")
    return d


def mxfp4_linear_workspace_size(M: int, K: int) -> int:
    return int(_lib.lib().fs4_mxfp4_linear_workspace_size(M, K))


def mxfp4_linear(x: torch.Tensor, w, N: int, dtype: torch.dtype | None = None, scale_rule: str = "floor",
                 out: torch.Tensor | None = None, accumulate: bool = False, workspace: torch.Tensor | None = None,
                 stream=None, flags: int = 0) -> torch.Tensor:
    """Q(x) deq(W)^T for an FP32, BF16 or FP16 x (M x K) and TILED MXFP4 weights w = (codes,
    scales), N x K (fs4_mxfp4_linear); in x's type unless dtype or out says otherwise.
    flags as mxfp4_gemm."""
    _check_matrix(x, "x")
    M, K = x.shape
    dev = x.device
    _mx_check(w, N, K, True, "w", dev)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    if not _here(dev, stream):
        with _at(dev, stream):
            return mxfp4_linear(x, w, N, dtype, scale_rule, out, accumulate, workspace, None, flags)
    d = _mx_out(out, M, N, x.dtype if dtype is None else dtype, dev)
    if _mx_empty(d, K, accumulate):
        return d
    need = 256 + 17 * mxfp4_tiled_shape(M, K)[1]             # mxfp4_linear_workspace_size(M, K)
    if workspace is None:
        workspace, status = torch.empty(need, dtype=torch.uint8, device=dev), _status_word(dev)
    else:
        _check_bytes(workspace, need, "workspace", dev)
        status = workspace
    check(_lib.lib().fs4_mxfp4_linear_ex(x.data_ptr(), _DTYPES[x.dtype], M, K, _ld(x), w[0].data_ptr(), w[1].data_ptr(), N,
                                         d.data_ptr(), _DTYPES[d.dtype], _ld(d),
                                         flags | _mx_scale_flag(scale_rule) | (_lib.FS4_MX_ACCUMULATE if accumulate else 0),
                                         workspace.data_ptr(), workspace.numel(), status.data_ptr(), _handle(dev)),
          "fs4_mxfp4_linear")
    return d


def muon_workspace_size(shapes: Sequence[tuple[int, int]]) -> int:
    """Workspace bytes of muon_orthogonalize and muon_step on matrices of these shapes."""
    n = len(shapes)
    rows, cols = (c_i64s(*(int(s[i]) for s in shapes)) for i, c_i64s in ((0, ctypes.c_int64 * n), (1, ctypes.c_int64 * n)))
    return int(_lib.lib().fs4_muon_workspace_size(n, rows, cols))


def _muon_coeffs(coeffs, K: int):
    """(ctypes array of (a, b, c) triples, their number): one triple, or one per iteration."""
    flat = [float(v) for v in coeffs] if not hasattr(coeffs[0], "__len__") else [float(v) for t in coeffs for v in t]
    if len(flat) not in (3, 3 * K):
        raise ValueError(f"coeffs must be one (a, b, c) or K = {K} of them")
    return (ctypes.c_float * len(flat))(*flat), len(flat) // 3


def _muon_call(ws_list, gs, ms, scales, K, coeffs, workspace, step):
    n, dev = len(gs), gs[0].device
    arr = (_lib.MuonDesc * n)()
    for d, w, g, m, scale in zip(arr, ws_list, gs, ms, scales):
        d.w, d.g, d.scale = w.data_ptr(), g.data_ptr(), scale
        d.rows, d.cols = g.shape
        d.ld_w, d.ld_g, d.w_dtype, d.g_dtype = _ld(w), _ld(g), _DTYPES[w.dtype], _DTYPES[g.dtype]
        if m is not None:
            d.m, d.ld_m, d.m_dtype = m.data_ptr(), _ld(m), _DTYPES[m.dtype]
    c, nc = _muon_coeffs(coeffs, K)
    own = workspace is None
    if own:
        workspace = torch.empty(max(muon_workspace_size([g.shape for g in gs]), 1), dtype=torch.uint8, device=dev)
    else:      # the call itself checks its size
        _check_bytes(workspace, 1, "workspace", dev)
    if step is None:
        check(_lib.lib().fs4_muon_orthogonalize(n, arr, K, c, nc, workspace.data_ptr(), workspace.numel(), _handle(dev)),
              "fs4_muon_orthogonalize")
    else:
        check(_lib.lib().fs4_muon_step(n, arr, K, c, nc, *step, workspace.data_ptr(), workspace.numel(), _handle(dev)),
              "fs4_muon_step")
    if own:       # each call resets the word in its workspace
        _status_word(dev)[:4].view(torch.int32).bitwise_or_(workspace[:4].view(torch.int32))


def muon_orthogonalize(Gs: Sequence[torch.Tensor], K: int = 5, coeffs=MUON_COEFFS, dtype: torch.dtype = torch.bfloat16,
                       outs: Sequence[torch.Tensor] | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Orthogonalise a list of FP32, BF16 or FP16 matrices of any sizes by K Newton-Schulz
    iterations (fs4_muon_orthogonalize), in `dtype` or into `outs`.  coeffs is one (a, b, c)
    or one per iteration.  About 1e-3 from the exact iteration, at most 2e-3 but for dominant
    directions of equal elements (include/fs4.h)."""
    if not Gs:
        return []
    dev = Gs[0].device
    for i, G in enumerate(Gs):
        _check_matrix(G, f"Gs[{i}]", dev)
    if outs is not None and len(outs) != len(Gs):
        raise ValueError(f"{len(outs)} outs for {len(Gs)} matrices")
    if not _here(dev, stream):
        with _at(dev, stream):
            return muon_orthogonalize(Gs, K, coeffs, dtype, outs, workspace)
    outs = [_mx_out(None if outs is None else outs[i], *G.shape, dtype, dev) for i, G in enumerate(Gs)]
    _muon_call(outs, Gs, [None] * len(Gs), [1.0] * len(Gs), K, coeffs, workspace, None)
    return outs


def _muon_scale(scale, rows: int, cols: int) -> float:
    if scale == "rms":
        return 0.2 * max(rows, cols) ** 0.5
    if scale == "spectral":
        return max(1.0, rows / cols) ** 0.5
    return float(scale)


def muon_step(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor], momenta: Sequence[torch.Tensor], lr: float,
              beta: float = 0.95, nesterov: bool = True, weight_decay: float = 0.0, K: int = 5, coeffs=MUON_COEFFS,
              scale="rms", workspace: torch.Tensor | None = None, stream=None, flags: int = 0) -> None:
    """One Muon step on every matrix, in place (fs4_muon_step): momentum, orthogonalised
    direction, decoupled weight decay, weights.  Each tensor is FP32, BF16 or FP16.  scale:
    "rms" multiplies the direction by 0.2 sqrt(max(rows, cols)), "spectral" by
    sqrt(max(1, rows / cols)); or a number.  flags as mxfp4_gemm."""
    if not (len(params) == len(grads) == len(momenta)):
        raise ValueError("params, grads and momenta must be lists of one length")
    if not params:
        return
    dev = params[0].device
    for i, ts in enumerate(zip(params, grads, momenta)):
        for t, name in zip(ts, ("params", "grads", "momenta")):
            _check_matrix(t, f"{name}[{i}]", dev)
            if t.shape != ts[0].shape:
                raise ValueError(f"{name}[{i}] must have the shape of params[{i}], {tuple(ts[0].shape)}")
    if not _here(dev, stream):
        with _at(dev, stream):
            return muon_step(params, grads, momenta, lr, beta, nesterov, weight_decay, K, coeffs, scale, workspace,
                             None, flags)
    _muon_call(params, grads, momenta, [_muon_scale(scale, *p.shape) for p in params], K, coeffs, workspace,
               (lr, beta, weight_decay, flags | (_lib.FS4_MUON_NESTEROV if nesterov else 0)))


def _ld(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _descs(Gs: Sequence[torch.Tensor], outs: Sequence[torch.Tensor], coeffs) -> ctypes.Array:
    arr = (NsDesc * len(Gs))()
    for i, (G, o) in enumerate(zip(Gs, outs)):
        a, b, c = coeffs[i]
        arr[i] = NsDesc(G.data_ptr(), o.data_ptr(), G.shape[0], G.shape[1], _ld(G), _ld(o), a, b, c)
    return arr


def ns_workspace_size(m: int, n: int) -> int:
    return int(_lib.lib().fs4_root_ns_workspace_size(m, n))


def _shape_descs(shapes: Sequence[tuple[int, int]]) -> ctypes.Array:
    """Descriptors for size/layout queries: disjoint placeholder address ranges
    (never dereferenced) so that the overlap checks pass."""
    arr = (NsDesc * len(shapes))()
    for i, (m, n) in enumerate(shapes):
        arr[i] = NsDesc((2 * i + 1) << 36, (2 * i + 2) << 36, m, n, n, n, 1.0, 0.0, 0.0)
    return arr


def ns_batched_workspace_size(shapes: Sequence[tuple[int, int]]) -> int:
    return int(_lib.lib().fs4_root_ns_batched_workspace_size(len(shapes), _shape_descs(shapes)))


def _masks(rht_masks, K):
    """Host uint16 array of the 3K H16^r sign masks (or None)."""
    if rht_masks is None:
        return None
    masks = [int(v) & 0xFFFF for v in rht_masks]
    if len(masks) < 3 * K:
        raise ValueError(f"need 3K = {3 * K} sign masks, got {len(masks)}")
    return (ctypes.c_uint16 * len(masks))(*masks)


def root_ns(G: torch.Tensor, K: int = 5, a: float = MUON_COEFFS[0], b: float = MUON_COEFFS[1],
            c: float = MUON_COEFFS[2], clip_k: float = 3.0, out: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, flags: int = 0, stream=None,
            rht_masks=None, adaptive46: bool = False,
            clip_quantile: float | None = None) -> torch.Tensor:
    """Direct NVFP4 Newton-Schulz step on one FP32 matrix (fs4_root_ns; with
    rht_masks (3K sign masks of H16^r) or adaptive46, fs4_root_ns_batched_ex).
    clip_quantile = q clips at the q-quantile of |X_0| (FS4_NS_CLIP_QUANTILE)
    instead of clip_k * RMS."""
    _check_f32_matrix(G, "G")
    if clip_quantile is not None:
        flags |= FS4_NS_CLIP_QUANTILE
        clip_k = clip_quantile
    if out is None:
        out = torch.empty_like(G)
    m, n = G.shape
    if workspace is None:
        workspace = torch.empty(ns_workspace_size(m, n), dtype=torch.uint8, device=G.device)
    if rht_masks is None and not adaptive46:
        check(_lib.lib().fs4_root_ns(G.data_ptr(), m, n, _ld(G), out.data_ptr(), _ld(out), K,
                                     a, b, c, clip_k, flags, workspace.data_ptr(), workspace.numel(),
                                     _stream(stream)),
              "fs4_root_ns")
        return out
    root_ns_batched([G], K, [(a, b, c)], clip_k, [out], workspace, flags, stream, rht_masks,
                    adaptive46)
    return out


def root_ns_batched(Gs: Sequence[torch.Tensor], K: int = 5, coeffs=None, clip_k: float = 3.0,
                    outs: Sequence[torch.Tensor] | None = None,
                    workspace: torch.Tensor | None = None, flags: int = 0, stream=None,
                    rht_masks=None, adaptive46: bool = False,
                    clip_quantile: float | None = None):
    """Direct NVFP4 Newton-Schulz step on a list of matrices in one grouped call
    (fs4_root_ns_batched); coeffs is a list of per-matrix (a, b, c).  rht_masks
    (3K sign masks of H16^r) and adaptive46 select the Section 3.4 quantiser
    options (fs4_root_ns_batched_ex); clip_quantile = q clips at the q-quantile
    of |X_0| (FS4_NS_CLIP_QUANTILE) instead of clip_k * RMS."""
    if clip_quantile is not None:
        flags |= FS4_NS_CLIP_QUANTILE
        clip_k = clip_quantile
    for G in Gs:
        _check_f32_matrix(G, "G")
    if coeffs is None:
        coeffs = [MUON_COEFFS] * len(Gs)
    if outs is None:
        outs = [torch.empty_like(G) for G in Gs]
    arr = _descs(Gs, outs, coeffs)
    need = int(_lib.lib().fs4_root_ns_batched_workspace_size(len(Gs), arr))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=Gs[0].device)
    if rht_masks is None and not adaptive46:
        check(_lib.lib().fs4_root_ns_batched(len(Gs), arr, K, clip_k, flags, workspace.data_ptr(),
                                             workspace.numel(), _stream(stream)),
              "fs4_root_ns_batched")
        return outs
    flags |= (FS4_NS_RHT if rht_masks is not None else 0) | (FS4_NS_ADAPTIVE46 if adaptive46 else 0)
    masks = _masks(rht_masks, K)
    check(_lib.lib().fs4_root_ns_batched_ex(len(Gs), arr, K, clip_k, flags,
                                            ctypes.cast(masks, ctypes.c_void_p) if masks else None,
                                            workspace.data_ptr(), workspace.numel(),
                                            _stream(stream)),
          "fs4_root_ns_batched_ex")
    return outs


def root_ns_batched_nvfp4(states, K: int = 5, coeffs=None, clip_k: float = 3.0,
                          outs: Sequence[torch.Tensor] | None = None,
                          workspace: torch.Tensor | None = None, flags: int = 0, stream=None,
                          rht_masks=None, adaptive46: bool = False,
                          clip_quantile: float | None = None):
    """The Newton-Schulz step on matrices given as NVFP4 first-moment states
    (fs4_root_ns_batched_nvfp4): each state is (codes, scales, s_g, mask) as
    momentum_nvfp4 returns it (plus the mask it was stored with); the matrix is
    codes.shape[0] x 2 * codes.shape[1].  Other arguments as root_ns_batched."""
    if clip_quantile is not None:
        flags |= FS4_NS_CLIP_QUANTILE
        clip_k = clip_quantile
    shapes = [(int(st[0].shape[0]), int(st[0].shape[1]) * 2) for st in states]
    dev = states[0][0].device
    if coeffs is None:
        coeffs = [MUON_COEFFS] * len(states)
    if outs is None:
        outs = [torch.empty(sh, dtype=torch.float32, device=dev) for sh in shapes]
    arr = (NsDesc * len(states))()
    sts = (_lib.Nvfp4State * len(states))()
    for i, (st, o, sh) in enumerate(zip(states, outs, shapes)):
        a, b, c = coeffs[i]
        arr[i] = NsDesc(None, o.data_ptr(), sh[0], sh[1], sh[1], _ld(o), a, b, c)
        sts[i] = _lib.Nvfp4State(st[0].data_ptr(), st[1].data_ptr(), st[2].data_ptr(), int(st[3]))
    need = int(_lib.lib().fs4_root_ns_batched_workspace_size(len(states), arr))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    flags |= (FS4_NS_RHT if rht_masks is not None else 0) | (FS4_NS_ADAPTIVE46 if adaptive46 else 0)
    masks = _masks(rht_masks, K)
    check(_lib.lib().fs4_root_ns_batched_nvfp4(len(states), arr, sts, K, clip_k, flags,
                                               ctypes.cast(masks, ctypes.c_void_p) if masks else None,
                                               workspace.data_ptr(), workspace.numel(),
                                               _stream(stream)),
          "fs4_root_ns_batched_nvfp4")
    return outs


def root_ns_bf16_batched(Gs: Sequence[torch.Tensor], K: int = 5, coeffs=None, clip_k: float = 3.0,
                         outs: Sequence[torch.Tensor] | None = None,
                         workspace: torch.Tensor | None = None, flags: int = 0, stream=None,
                         clip_quantile: float | None = None):
    """The BF16 comparison step (fs4_root_ns_bf16_batched): the same Newton-Schulz
    iteration with BF16 operands on the tensor cores instead of NVFP4.  Arguments as
    root_ns_batched (no quantiser options)."""
    if clip_quantile is not None:
        flags |= FS4_NS_CLIP_QUANTILE
        clip_k = clip_quantile
    for G in Gs:
        _check_f32_matrix(G, "G")
    if coeffs is None:
        coeffs = [MUON_COEFFS] * len(Gs)
    if outs is None:
        outs = [torch.empty_like(G) for G in Gs]
    arr = _descs(Gs, outs, coeffs)
    need = int(_lib.lib().fs4_root_ns_bf16_batched_workspace_size(len(Gs), arr))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=Gs[0].device)
    check(_lib.lib().fs4_root_ns_bf16_batched(len(Gs), arr, K, clip_k, flags, workspace.data_ptr(),
                                              workspace.numel(), _stream(stream)),
          "fs4_root_ns_bf16_batched")
    return outs


def ns_bf16_batched_workspace_size(shapes: Sequence[tuple[int, int]]) -> int:
    return int(_lib.lib().fs4_root_ns_bf16_batched_workspace_size(len(shapes), _shape_descs(shapes)))


def ns_bf16_layout(shapes: Sequence[tuple[int, int]], index: int = 0) -> NsLayout:
    """Workspace offsets of matrix `index` of a BF16 step on matrices of these shapes."""
    arr = _shape_descs(shapes)
    lay = NsLayout()
    check(_lib.lib().fs4_root_ns_bf16_layout(len(shapes), arr, index, ctypes.byref(lay)),
          "fs4_root_ns_bf16_layout")
    return lay


def ns_layout(shapes: Sequence[tuple[int, int]], index: int = 0) -> NsLayout:
    """Offsets of the internal tensors of matrix `index` (of a batched call on
    matrices of these shapes) in the workspace."""
    arr = _shape_descs(shapes)
    lay = NsLayout()
    check(_lib.lib().fs4_root_ns_layout(len(shapes), arr, index, ctypes.byref(lay)),
          "fs4_root_ns_layout")
    return lay


def device_status(workspace: torch.Tensor | None = None, stream=None) -> int:
    """Synchronise and return the device status word of the last call (0 = FS4_OK).  Without a
    workspace: that of all mxfp4_* and muon_* calls since the last such query, on any stream of
    any device, that were not given one (calls captured into a graph should be: their status is
    kept only where their stream has made such a call outside the capture)."""
    if workspace is not None:
        return int(_lib.lib().fs4_device_status(workspace.data_ptr(), _stream(stream)))
    worst = 0
    for device in {word.device for word in list(_status_words.values())}:
        with torch.cuda.device(device):
            torch.cuda.synchronize()
            for word in [w for w in list(_status_words.values()) if w.device == device]:
                status = int(_lib.lib().fs4_device_status(word.data_ptr(), None))
                if status != 0:
                    word.zero_()
                worst = min(worst, status)
            torch.cuda.synchronize()
    return worst


GEMM_SOURCES = ("gemm.cu", "fs4_device.cuh", "fs4_internal.h")
ELEMENTWISE_SOURCES = ("kernels.cu", "fs4_device.cuh", "fs4_internal.h")


def _source_digest(files=GEMM_SOURCES) -> str:
    """Short hash of the CUDA sources that define a kernel (ties stored ncu counters
    to the code they measured)."""
    import hashlib
    import os
    csrc = os.path.join(os.path.dirname(os.path.abspath(__file__)), "csrc")
    h = hashlib.sha256()
    for name in sorted(files):
        with open(os.path.join(csrc, name), "rb") as f:
            h.update(name.encode() + f.read())
    return h.hexdigest()[:16]
