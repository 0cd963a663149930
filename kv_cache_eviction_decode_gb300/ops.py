"""Operators around the decode step (include/kvevict_ops.h): argument checks
and marshalling only, every step runs in the library's kernels.

Work is queued on the current stream of the tensors' device. Nothing here
waits for the GPU, and every call can be captured in a CUDA graph. All of them
are forward only: tensors that require gradients are refused where gradients
are enabled (the gradient of rotary() is rotary() with inverse=True).
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from ._lib import BF16, ERR_DEVICE, F32, OK, check, lib

_INT_MAX = 2**31 - 1
_DT = {torch.float32: F32, torch.bfloat16: BF16}

# The argument structs of include/kvevict_ops.h, as their fields in order.
_ATTN = struct.Struct("@9if2q5P12q4PPNP")
_SHARED = struct.Struct("@9if2q5P12q4PPNP2P5q")
_ROT = struct.Struct("@8i2q4P12qP3qPf4x")
# ... and in pieces: shapes, addresses, strides, addresses (all multiples of 8 bytes).
_HEAD, _PTRS, _Q9, _Q3, _TAIL = (struct.Struct("@" + f) for f in ("9if2q", "5P", "9q", "3q", "4PPNP"))
_ROT_HEAD, _Q12, _ROT_TAIL, _P2, _P4 = (struct.Struct("@" + f) for f in ("8i2q", "12q", "P3qPf4x", "2P", "4P"))

# The handle of a device's current stream as a number (torch.cuda.current_stream
# builds a Stream object first, ten times the cost), where torch has it.
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _dtype(t: torch.Tensor, name: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name}: need float32 or bfloat16, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: need a CUDA tensor, got one on {t.device}")
    return dt


def _like(t: torch.Tensor, q: torch.Tensor, dims: int, name: str, shape=None) -> None:
    """t goes with q: its type, device, `dims` axes (or the whole shape), the last one contiguous."""
    if t.dtype is q.dtype and t.get_device() == q.get_device() and (t.dim() == dims if shape is None else t.shape == shape) \
            and (t.stride(-1) == 1 or t.shape[-1] <= 1):
        return
    if t.dtype != q.dtype or t.device != q.device or t.dim() != dims or (shape is not None and t.shape != shape):
        raise ValueError(f"{name}: need a {q.dtype} tensor of {dims if shape is None else tuple(shape)} "
                         f"{'axes' if shape is None else ''} on {q.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    raise ValueError(f"{name}: the last axis must be contiguous")


def _strides(t: torch.Tensor, name: str, least: int = 1) -> None:
    """Over axes of several entries the strides are positive (0 for tensors that are only read by rotary) multiples of
    16 bytes."""
    for size, stride in zip(t.shape[:-1], t.stride()):
        if size > 1 and (stride < least or stride * t.element_size() % 16) and t.numel() > 0:
            raise ValueError(f"{name}: need strides that are {'positive ' if least else ''}multiples of 16 bytes, got {stride} elements over "
                             f"an axis of {size} (expanded tensors and rows off 16-byte boundaries have to be made contiguous)")


def _forward_only(name: str, *tensors) -> None:
    """Refuses tensors whose gradient would be lost: the operators have no backward pass."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in tensors):
        raise ValueError(f"{name}: forward only, there is no backward pass: detach the tensors that require gradients, or call "
                         f"it under torch.no_grad()")


def _ints(t, n: int, q: torch.Tensor, name: str) -> int:
    if t is None:
        return 0
    if t.dtype is not torch.int32 or t.get_device() != q.get_device() or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous int32 tensor of {n} on {q.device}, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _scale(scale) -> float:
    if scale is None:
        return 0.0
    if not (scale > 0 and math.isfinite(scale)):
        raise ValueError("scale: need a positive finite number")
    return float(scale)


def _outputs(q, out, lse, return_lse, lse_shape):
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    else:
        _like(out, q, q.dim(), "out", q.shape)
        _strides(out, "out")
    if lse is None:
        if return_lse:
            lse = torch.empty(lse_shape, dtype=torch.float32, device=q.device)
    elif lse.dtype != torch.float32 or lse.device != q.device or lse.shape != lse_shape or not lse.is_contiguous():
        raise ValueError(f"lse: need a contiguous float32 tensor of {tuple(lse_shape)} on {q.device}")
    return out, lse


def _workspace(workspace, need: int, q: torch.Tensor):
    if need == 0:
        return None, 0, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    size = workspace.numel() * workspace.element_size()
    if workspace.device != q.device or not workspace.is_contiguous() or size < need:
        raise ValueError(f"workspace: need {need} contiguous bytes on {q.device}")
    return workspace, workspace.data_ptr(), size


def _error_word(t, q: torch.Tensor) -> int:
    if t is None:
        return 0
    if t.dtype != torch.int32 or t.device != q.device or t.numel() < 1:
        raise ValueError(f"error_word: need an int32 tensor on {q.device}")
    return t.data_ptr()


def operator_errors(device=None) -> int:
    """Waits for the device (None: the current one); returns the error bits that calls without an error_word have set
    on it since the last time (0: clean; DEV_BAD_LENGTH, DEV_WAIT_TIMEOUT), and clears them."""
    if device is not None and torch.device(device).type != "cuda":
        raise ValueError(f"operator_errors: need a CUDA device, got {device}")
    w = ctypes.c_uint32(0)
    with torch.cuda.device(device):
        rc = lib().kvevict_operator_errors(w)
    if rc not in (OK, ERR_DEVICE):
        check(rc, "kvevict_operator_errors")
    return w.value


_entry = {}  # the library's entry points, looked up once


def _call(name: str, dev: int, args: bytes) -> None:
    """The entry point on the current stream of device `dev`, with that device current."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    if dev == _current_device():
        rc = fn(args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(args, _raw_stream(dev))
    if rc != OK:
        check(rc, name)


def _workspace_need(name: str, args: bytes) -> int:
    n = ctypes.c_size_t(0)
    check(getattr(lib(), name + "_workspace_bytes")(args, n), name + "_workspace_bytes")
    return n.value


class _Layout:
    """What a call's argument struct holds besides addresses, checked and packed once per shapes, strides, types and
    options: the checks and the packing cost more than the launch."""

    __slots__ = ("head", "strides", "out_strides", "need", "out_shape", "lse_shape", "batch", "tail")


_layouts: dict = {}


def _remember(key, layout: _Layout) -> _Layout:
    if len(_layouts) >= 4096:
        _layouts.clear()
    _layouts[key] = layout
    return layout


def window_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *, n_sink: int = 0, window: int | None = None,
                     scale: float | None = None, q_starts: torch.Tensor | None = None,
                     k_starts: torch.Tensor | None = None, max_q: int | None = None, max_k: int | None = None,
                     q_lens: torch.Tensor | None = None, kv_lens: torch.Tensor | None = None,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = False,
                     workspace: torch.Tensor | None = None, error_word: torch.Tensor | None = None):
    """Attention in which a query at position p sees the keys up to p that are
    among the first n_sink or the newest `window` (None: all of them). The
    queries are the last rows of their sequence: whole prompts, chunks of one,
    or single tokens.

    Padded: q [B][Hq][N][d], k and v [B][Hkv][M][d]; q_lens and kv_lens (int32
    [B] on the device) say how many rows are real. Packed (q_starts and
    k_starts, int32 [B + 1] on the device, with max_q and max_k the longest
    sequences): q [T][Hq][d], k and v [S][Hkv][d]. d is contiguous, the other
    axes have any strides that are positive multiples of 16 bytes (so no expanded
    tensors); out overlaps no input.
    Returns out (as q), or (out, lse) with return_lse or an lse tensor: fp32
    [B][Hq][N], or [T][Hq] packed. A row that sees nothing gives 0 and -inf.
    Rows behind q_lens, outside the starts or beyond max_q are not written (in
    an output made here they hold anything). Lengths and starts out of range are
    clamped and set DEV_BAD_LENGTH in error_word (int32 on the device; None: see
    operator_errors).
    """
    if q.requires_grad or k.requires_grad or v.requires_grad or (out is not None and out.requires_grad):
        _forward_only("window_attention", q, k, v, out)
    packed = q_starts is not None
    key = (q.dtype, k.dtype, v.dtype, q.get_device(), k.get_device(), v.get_device(), q.shape, k.shape, v.shape, q.stride(),
           k.stride(), v.stride(), n_sink, window, scale, max_q, max_k, q_starts.shape if packed else None)
    lay = _layouts.get(key) or _remember(key, _window_layout(q, k, v, n_sink, window, scale, q_starts, max_q, max_k))
    if packed:
        if k_starts is None or q_lens is not None or kv_lens is not None:
            raise ValueError("packed: give q_starts, k_starts, max_q and max_k, and no lengths")
        starts = (_ints(q_starts, lay.batch + 1, q, "q_starts"), _ints(k_starts, lay.batch + 1, q, "k_starts"), 0, 0)
    else:
        if k_starts is not None:
            raise ValueError("k_starts: goes with q_starts")
        starts = (0, 0, _ints(q_lens, lay.batch, q, "q_lens"), _ints(kv_lens, lay.batch, q, "kv_lens"))
    given = out is not None
    out, lse = _outputs(q, out, lse, return_lse, lay.lse_shape)
    if not given:
        out_strides = lay.out_strides
    else:
        out_strides = _Q3.pack(*((0, out.stride(1), out.stride(0)) if packed else out.stride()[:3]))
    workspace, wp, wn = _workspace(workspace, lay.need, q)
    _call("kvevict_window_attention", q.get_device(), b"".join((
        lay.head, _PTRS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr()),
        lay.strides, out_strides, _TAIL.pack(*starts, wp, wn, _error_word(error_word, q)))))
    return out if lse is None else (out, lse)


def _window_layout(q, k, v, n_sink, window, scale, q_starts, max_q, max_k) -> _Layout:
    dt = _dtype(q, "q")
    packed = q_starts is not None
    dims = 3 if packed else 4
    _like(q, q, dims, "q")
    _like(k, q, dims, "k")
    _like(v, q, dims, "v", k.shape)
    if q.numel() > 0:  # (else nothing is read)
        for t, name in ((q, "q"), (k, "k"), (v, "v")):
            _strides(t, name)
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window: need at least 1, or None for no window")
    if n_sink < 0:
        raise ValueError("n_sink: need 0 or more")
    d = q.shape[-1]
    if k.shape[-1] != d:
        raise ValueError(f"k: head_dim {k.shape[-1]}, q has {d}")
    lay = _Layout()
    if packed:
        if max_q is None or max_k is None:
            raise ValueError("packed: give q_starts, k_starts, max_q and max_k, and no lengths")
        if max_q < 0 or max_k < 0:
            raise ValueError("max_q, max_k: need 0 or more")
        max_q, max_k = min(max_q, _INT_MAX), min(max_k, _INT_MAX)
        B = q_starts.shape[0] - 1
        N, Hq, M, Hkv = q.shape[0], q.shape[1], k.shape[0], k.shape[1]
        strides = [(0, t.stride(1), t.stride(0)) for t in (q, k, v)]
        dense = (0, d, Hq * d)
        lay.lse_shape = q.shape[:2]
    else:
        B, Hq, N = q.shape[:3]
        if k.shape[0] != B:
            raise ValueError(f"k: {k.shape[0]} sequences, q has {B}")
        Hkv, M = k.shape[1], k.shape[2]
        strides = [t.stride()[:3] for t in (q, k, v)]
        dense = (Hq * N * d, N * d, d)
        max_q = max_k = 0
        lay.lse_shape = q.shape[:3]
    shape = (dt, d, Hq, Hkv, B, min(n_sink, _INT_MAX), min(window, _INT_MAX), max_q, max_k, _scale(scale), N, M)
    lay.batch = B
    lay.head = _HEAD.pack(*shape)
    lay.strides = _Q9.pack(*strides[0], *strides[1], *strides[2])
    lay.out_strides = _Q3.pack(*dense)
    # (of the starts only their presence counts for the size)
    lay.need = _workspace_need("kvevict_window_attention", _ATTN.pack(*shape, *(0,) * 17, *((16, 16) if packed else (0, 0)), 0, 0, 0, 0, 0))
    return lay


def shared_prefix_attention(q: torch.Tensor, k_prefix: torch.Tensor, v_prefix: torch.Tensor, k: torch.Tensor,
                            v: torch.Tensor, kv_lens: torch.Tensor | None = None, *, scale: float | None = None,
                            out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = False,
                            workspace: torch.Tensor | None = None, error_word: torch.Tensor | None = None):
    """One token of every sequence, q [B][Hq][d], over a prefix that all share,
    k_prefix and v_prefix [Hkv][P][d], and a suffix of its own, k and v
    [B][Hkv][M][d], of kv_lens rows (int32 [B] on the device; None: M). The
    prefix is read once for the batch. P and M may be 0. Returns out (as q), or
    (out, lse [B][Hq])."""
    if q.requires_grad or k_prefix.requires_grad or v_prefix.requires_grad or k.requires_grad or v.requires_grad or \
            (out is not None and out.requires_grad):
        _forward_only("shared_prefix_attention", q, k_prefix, v_prefix, k, v, out)
    key = (q.dtype, k.dtype, v.dtype, k_prefix.dtype, v_prefix.dtype, q.get_device(), k.get_device(), v.get_device(),
           k_prefix.get_device(), v_prefix.get_device(), q.shape, k.shape, v.shape, k_prefix.shape, v_prefix.shape, q.stride(),
           k.stride(), v.stride(), k_prefix.stride(), v_prefix.stride(), scale)
    lay = _layouts.get(key) or _remember(key, _shared_layout(q, k_prefix, v_prefix, k, v, scale))
    given = out is not None
    out, lse = _outputs(q, out, lse, return_lse, lay.lse_shape)
    out_strides = _Q3.pack(out.stride(0), out.stride(1), 0) if given else lay.out_strides
    workspace, wp, wn = _workspace(workspace, lay.need, q)
    _call("kvevict_shared_prefix_attention", q.get_device(), b"".join((
        lay.head, _PTRS.pack(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr()),
        lay.strides, out_strides, _TAIL.pack(0, 0, 0, _ints(kv_lens, lay.batch, q, "kv_lens"), wp, wn, _error_word(error_word, q)),
        _P2.pack(k_prefix.data_ptr(), v_prefix.data_ptr()), lay.tail)))
    return out if lse is None else (out, lse)


def _shared_layout(q, k_prefix, v_prefix, k, v, scale) -> _Layout:
    dt = _dtype(q, "q")
    _like(q, q, 3, "q")
    _like(k_prefix, q, 3, "k_prefix")
    _like(v_prefix, q, 3, "v_prefix", k_prefix.shape)
    _like(k, q, 4, "k")
    _like(v, q, 4, "v", k.shape)
    if q.numel() > 0:  # (else nothing is read)
        for t, name in ((q, "q"), (k_prefix, "k_prefix"), (v_prefix, "v_prefix"), (k, "k"), (v, "v")):
            _strides(t, name)
    B, Hq, d = q.shape
    Hkv, M = k.shape[1], k.shape[2]
    if k.shape[0] != B or k.shape[3] != d or k_prefix.shape[0] != Hkv or k_prefix.shape[2] != d:
        raise ValueError(f"k, k_prefix: need [{B}][Hkv][M][{d}] and [Hkv][P][{d}], got {tuple(k.shape)} and {tuple(k_prefix.shape)}")
    P = k_prefix.shape[1]
    shape = (dt, d, Hq, Hkv, B, 0, 0, 0, 0, _scale(scale), 1, M)
    lay = _Layout()
    lay.batch = B
    lay.lse_shape = q.shape[:2]
    lay.head = _HEAD.pack(*shape)
    lay.strides = _Q9.pack(q.stride(0), q.stride(1), 0, *k.stride()[:3], *v.stride()[:3])
    lay.out_strides = _Q3.pack(Hq * d, d, 0)
    tail = (*k_prefix.stride()[:2], *v_prefix.stride()[:2], P)
    lay.tail = struct.pack("@5q", *tail)
    lay.need = _workspace_need("kvevict_shared_prefix_attention", _SHARED.pack(*shape, *(0,) * 24, 0, 0, *tail))
    return lay


def rotary_frequencies(rotary_dim: int, *, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                       original_context: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0,
                       device=None) -> tuple[torch.Tensor, float]:
    """The angles per position of a head's pairs, fp64 [rotary_dim / 2], and the
    factor on cosines and sines, for rotary(). inv_freq_i = base^(-2 i /
    rotary_dim), changed for longer contexts by `scaling`:
    "linear": every frequency / factor (positions interpolated);
    "ntk": base * factor^(rotary_dim / (rotary_dim - 2)), which slows the
    slowest pair by `factor` and leaves the fastest;
    "yarn": pairs that turn more than beta_fast times over original_context
    positions stay, those that turn less than beta_slow times are slowed by
    `factor`, a linear ramp over the pair index between; the factor on the
    result is 0.1 ln(factor) + 1."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim: need an even number of at least 2")
    if not (base > 1 and factor >= 1):
        raise ValueError("base: above 1; factor: at least 1")
    i = torch.arange(rotary_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "ntk":
        if rotary_dim == 2:
            raise ValueError("ntk: needs a rotary_dim above 2")
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-2.0 * i / rotary_dim)
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        def pair_of(turns):
            return rotary_dim * math.log(original_context / (turns * 2 * math.pi)) / (2 * math.log(base))
        low, high = max(math.floor(pair_of(beta_fast)), 0), min(math.ceil(pair_of(beta_slow)), rotary_dim - 1)
        slow = ((i - low) / max(high - low, 1e-3)).clamp(0, 1)
        f = f / factor * slow + f * (1 - slow)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling: None, 'linear', 'ntk' or 'yarn', got {scaling!r}")
    return f.to(device if device is not None else "cuda"), scale


def rotary(q: torch.Tensor, k: torch.Tensor | None, positions, inv_freq: torch.Tensor, *, interleaved: bool = False,
           scale: float = 1.0, inverse: bool = False, q_out: torch.Tensor | None = None,
           k_out: torch.Tensor | None = None):
    """Rotary positions of queries and keys in one launch: the first
    2 * len(inv_freq) elements of every head turn by positions * inv_freq,
    pairs (i, i + half) or, interleaved, (2 i, 2 i + 1); the rest is copied.

    q [T][Hq][d] with positions [T], or q [B][Hq][N][d] with positions [B][N]
    (or [N], the same for every sequence); k alike with its own heads, or None.
    positions: an int32 or int64 tensor on the device, or an int, the first
    token's position. inv_freq: fp64 on the device (rotary_frequencies).
    q_out / k_out may be q / k: in place. inverse: by the negative angle, the
    gradient of the forward call. Returns (q_out, k_out), or q_out without k."""
    if q.requires_grad or (k is not None and k.requires_grad) or q_out is not None or k_out is not None:
        _forward_only("rotary", q, k, q_out, k_out)
    key = (q.dtype, q.get_device(), q.shape, q.stride(), None if k is None else (k.dtype, k.get_device(), k.shape, k.stride()),
           None if isinstance(positions, int) else (positions.dtype, positions.get_device(), positions.shape, positions.stride()),
           inv_freq.shape, interleaved, inverse)
    lay = _layouts.get(key) or _remember(key, _rotary_layout(q, k, positions, inv_freq, interleaved, inverse))
    if q_out is None and k_out is None:
        q_out, strides = torch.empty(q.shape, dtype=q.dtype, device=q.device), lay.strides
        if k is not None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
    else:
        dims = q.dim()
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _like(q_out, q, dims, "q_out", q.shape)
        _strides(q_out, "q_out")
        if k is not None:
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
            _like(k_out, q, dims, "k_out", k.shape)
            _strides(k_out, "k_out")
        strides = _Q12.pack(*_heads(q), *_heads(q_out), *((0,) * 6 if k is None else (*_heads(k), *_heads(k_out))))
    if inv_freq.dtype is not torch.float64 or inv_freq.get_device() != q.get_device() or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq: need a contiguous float64 vector on {q.device}")
    pp, start = (0, positions) if isinstance(positions, int) else (positions.data_ptr(), 0)
    kp, kop = (0, 0) if k is None else (k.data_ptr(), k_out.data_ptr())
    _call("kvevict_rotary", q.get_device(), b"".join((
        lay.head, _P4.pack(q.data_ptr(), kp, q_out.data_ptr(), kop), strides,
        _ROT_TAIL.pack(pp, *lay.tail, start, inv_freq.data_ptr(), scale))))
    return q_out if k is None else (q_out, k_out)


def _heads(t: torch.Tensor) -> tuple:
    """Strides of sequence, head, token."""
    return (0, t.stride(1), t.stride(0)) if t.dim() == 3 else t.stride()[:3]


def _rotary_layout(q, k, positions, inv_freq, interleaved, inverse) -> _Layout:
    dt = _dtype(q, "q")
    dims = q.dim()
    if dims not in (3, 4):
        raise ValueError(f"q: need [T][H][d] or [B][H][N][d], got {tuple(q.shape)}")
    _like(q, q, dims, "q")
    _strides(q, "q", 0)
    d = q.shape[-1]
    if dims == 3:
        B, N, Hq = 1, q.shape[0], q.shape[1]
        dense = [(0, d, Hq * d)]
    else:
        B, Hq, N = q.shape[:3]
        dense = [(Hq * N * d, N * d, d)]
    Hk = 0
    if k is not None:
        _like(k, q, dims, "k")
        _strides(k, "k", 0)
        Hk = k.shape[1]
        if k.shape[-1] != d or k.shape[0] != q.shape[0] or (dims == 4 and k.shape[2] != N):
            raise ValueError(f"k: {tuple(k.shape)} does not go with q {tuple(q.shape)}")
        dense.append((0, d, Hk * d) if dims == 3 else (Hk * N * d, N * d, d))
    p64, ps = 0, (0, 0)
    if not isinstance(positions, int):
        if positions.get_device() != q.get_device() or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError(f"positions: need int32 or int64 on {q.device}, got {positions.dtype} on {positions.device}")
        if positions.shape == (N,):
            ps = (0, positions.stride(0))
        elif dims == 4 and positions.shape == (B, N):
            ps = positions.stride()
        else:
            raise ValueError(f"positions: {tuple(positions.shape)} does not go with q {tuple(q.shape)}")
        p64 = int(positions.dtype == torch.int64)
    lay = _Layout()
    lay.head = _ROT_HEAD.pack(dt, d, 2 * inv_freq.shape[0], int(interleaved), int(inverse), p64, Hq, Hk, B, N)
    lay.strides = _Q12.pack(*_heads(q), *dense[0], *((0,) * 6 if k is None else (*_heads(k), *dense[1])))
    lay.tail = ps
    return lay
