"""A paged cache on plain tensors (include/kvevict_paged.h): new tokens into
their sequences' pages, attention over the pages, whole sequences out of them.
Argument checks and marshalling only, every step runs in the library's kernels;
streams, errors and capture are as in ops.py.

Pages are [pages][Hkv][page_size][d] in the keys' type (any strides of page,
head and token that are multiples of 16 bytes), or hold 4 bits a channel: uint8
[pages][Hkv][page_size][5 d / 8], a head's block in a page contiguous, with a
base and a step for every 32 channels of a token (paged_pool makes either).
block_table, int32 [B][W] on the device: token i of sequence b is row
i % page_size of page block_table[b][i // page_size]; entries that no token of
a call needs may hold anything. kv_lens, int32 [B] on the device: the tokens of
each sequence, the new ones of the call included. New tokens are [T][heads][d]:
T / B of every sequence, or, with starts (int32 [B + 1] on the device), those
of sequence b from row starts[b] to starts[b + 1]; they are the last of their
sequence.
"""
from __future__ import annotations

import struct

import torch

from . import ops
from ._lib import Q4
from .ops import _call, _error_word, _forward_only, _ints, _Layout, _like, _outputs, _remember, _scale, _strides, _workspace, _workspace_need

_INT_MAX = 2**31 - 1

# The argument structs of include/kvevict_paged.h, and their pieces.
_CACHE = "8i2P6qPq2P"
_APPEND, _GATHER, _ATTENTION = (struct.Struct("@" + _CACHE + f) for f in ("2P5q3Pq3if", "2P7qP", "5ifq3P4q2PN"))
_SHAPE, _PAGES, _TABLE = (struct.Struct("@" + f) for f in ("8i2P", "6q", "Pq2P"))
_APPEND_TAIL, _GATHER_TAIL, _ATTENTION_HEAD, _ATTENTION_TAIL = (struct.Struct("@" + f) for f in ("2P5q3Pq3if", "2P7qP", "5ifq", "3P4q2PN"))


def paged_pool(n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, *, dtype: torch.dtype = torch.bfloat16,
               four_bit: bool = False, device=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Empty pages for keys and values, [n_pages][n_kv_heads][page_size][head_dim] in dtype (zeros), or with 4 bits a
    channel: uint8 [n_pages][n_kv_heads][page_size][5 * head_dim // 8]."""
    if head_dim not in (64, 128) or page_size not in (16, 32, 64, 128, 256) or n_kv_heads < 1 or n_pages < 0:
        raise ValueError("paged_pool: need a head_dim of 64 or 128, a page_size of 16, 32, 64, 128 or 256, and heads")
    if dtype not in ops._DT:
        raise ValueError(f"paged_pool: need float32 or bfloat16, got {dtype}")
    shape, t = ((n_pages, n_kv_heads, page_size, 5 * head_dim // 8), torch.uint8) if four_bit else \
        ((n_pages, n_kv_heads, page_size, head_dim), dtype)
    k, v = (torch.zeros(shape, dtype=t, device=device if device is not None else "cuda") for _ in range(2))
    return k, v


def _pages_key(k_pages, v_pages, block_table, kv_lens):
    return (k_pages.dtype, v_pages.dtype, k_pages.get_device(), v_pages.get_device(), k_pages.shape, v_pages.shape, k_pages.stride(),
            v_pages.stride(), block_table.dtype, block_table.get_device(), block_table.shape, block_table.stride(), kv_lens.shape)


def _cache_layout(lay: _Layout, dtype: torch.dtype, device, d: int, Hkv: int | None, k_pages, v_pages, block_table) -> tuple:
    """Checks the pages and the table for heads of d elements of dtype; fills lay.head (shapes) and lay.strides, and
    returns the shapes. lay.tail: what follows the addresses of the table."""
    four = k_pages.dtype is torch.uint8
    row = 5 * d // 8 if four else d
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.dtype not in (dtype, torch.uint8) or t.dtype is not k_pages.dtype or t.device != device or t.dim() != 4 or t.shape != k_pages.shape \
                or t.shape[-1] != row or (Hkv is not None and t.shape[1] != Hkv):
            raise ValueError(f"{name}: need [pages][{'Hkv' if Hkv is None else Hkv}][page_size][{d}] of {dtype}, or [{5 * d // 8}] bytes at 4 bits, "
                             f"on {device}, k and v alike; got {t.dtype} {tuple(t.shape)} on {t.device}")
        if t.shape[2] not in (16, 32, 64, 128, 256) or d not in (64, 128):
            raise ValueError(f"{name}: need pages of 16, 32, 64, 128 or 256 tokens and heads of 64 or 128, got {tuple(t.shape)}")
        if four and t.numel() > 0 and (t.stride(3) != 1 or t.stride(2) != row):
            raise ValueError(f"{name}: a head's block in a page of 4 bits must be contiguous")
        if not four and t.stride(3) != 1 and t.numel() > 0:
            raise ValueError(f"{name}: the last axis must be contiguous")
        _strides(t[:, :, :1] if four else t, name)
    if block_table.dtype is not torch.int32 or block_table.device != device or block_table.dim() != 2 or \
            (block_table.shape[1] > 1 and block_table.stride(1) != 1) or (block_table.shape[0] > 1 and block_table.stride(0) < 0):
        raise ValueError(f"block_table: need int32 [B][W] on {device} with a contiguous last axis, got {block_table.dtype} "
                         f"{tuple(block_table.shape)} on {block_table.device}")
    P, H, S = k_pages.shape[:3]
    B, W = block_table.shape
    if W * S >= 2**30:
        raise ValueError(f"block_table: {W} pages of {S} tokens: need room for fewer than 2^30 tokens a sequence")
    dt = ops._DT[dtype]
    lay.batch = B
    lay.strides = _PAGES.pack(*k_pages.stride()[:3], *v_pages.stride()[:3])
    lay.out_strides = block_table.stride(0)
    return (dt, Q4 if four else dt, d, H, S, B, W, P)


def _cache_args(lay: _Layout, k_pages, v_pages, block_table, kv_lens, error_word) -> bytes:
    return b"".join((lay.head, struct.pack("@2P", k_pages.data_ptr(), v_pages.data_ptr()), lay.strides,
                     _TABLE.pack(block_table.data_ptr(), lay.out_strides, _ints(kv_lens, lay.batch, k_pages, "kv_lens"),
                                 _error_word(error_word, k_pages))))


def _per_sequence(tokens: int, starts, batch: int, name: str) -> None:
    if starts is None and (tokens % batch if batch else tokens):
        raise ValueError(f"{name}: {tokens} tokens for {batch} sequences: give starts, or the same number of every sequence")


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                 kv_lens: torch.Tensor, *, starts: torch.Tensor | None = None, inv_freq: torch.Tensor | None = None,
                 positions: torch.Tensor | None = None, interleaved: bool = False, scale: float = 1.0,
                 error_word: torch.Tensor | None = None) -> None:
    """New keys and values, k and v [T][Hkv][d], into the pages of their
    sequences; with inv_freq (fp64 on the device, see rotary_frequencies) the keys
    turned on the way as by rotary(), at `positions` (int32 or int64 [T] on the
    device; None: their places in their sequences). Rounded once, to the pages'
    type or to 4 bits. Tokens that the table has no page for are dropped and set
    DEV_BAD_PAGE or DEV_BAD_LENGTH in error_word (int32 on the device; None: see
    operator_errors). Pages that two sequences share must not be written."""
    if k.requires_grad or v.requires_grad or k_pages.requires_grad or v_pages.requires_grad:
        _forward_only("paged_append", k, v, k_pages, v_pages)
    key = ("append", k.dtype, v.dtype, k.get_device(), v.get_device(), k.shape, v.shape, k.stride(), v.stride(),
           *_pages_key(k_pages, v_pages, block_table, kv_lens), None if inv_freq is None else inv_freq.shape, interleaved,
           None if positions is None else (positions.dtype, positions.get_device(), positions.shape, positions.stride()), starts is None)
    lay = ops._layouts.get(key) or _remember(key, _append_layout(k, v, k_pages, v_pages, block_table, inv_freq, positions, interleaved, starts))
    if inv_freq is not None and (inv_freq.dtype is not torch.float64 or inv_freq.get_device() != k.get_device() or inv_freq.dim() != 1 or
                                 not inv_freq.is_contiguous()):
        raise ValueError(f"inv_freq: need a contiguous float64 vector on {k.device}")
    _call("kvevict_paged_append", k.get_device(), b"".join((
        _cache_args(lay, k_pages, v_pages, block_table, kv_lens, error_word),
        _APPEND_TAIL.pack(k.data_ptr(), v.data_ptr(), *lay.need, _ints(starts, lay.batch + 1, k, "starts"),
                          0 if inv_freq is None else inv_freq.data_ptr(), 0 if positions is None else positions.data_ptr(), *lay.tail, scale))))


def _append_layout(k, v, k_pages, v_pages, block_table, inv_freq, positions, interleaved, starts) -> _Layout:
    ops._dtype(k, "k")
    _like(k, k, 3, "k")
    _like(v, k, 3, "v", k.shape)
    T, H, d = k.shape
    for t, name in ((k, "k"), (v, "v")):
        _strides(t, name, 0)
    lay = _Layout()
    lay.head = struct.pack("@8i", *_cache_layout(lay, k.dtype, k.device, d, H, k_pages, v_pages, block_table))
    _per_sequence(T, starts, lay.batch, "k")
    p64, ps = 0, 0
    if positions is not None:
        if positions.device != k.device or positions.dtype not in (torch.int32, torch.int64) or positions.shape != (T,):
            raise ValueError(f"positions: need int32 or int64 [{T}] on {k.device}, got {positions.dtype} {tuple(positions.shape)} on {positions.device}")
        p64, ps = int(positions.dtype is torch.int64), positions.stride(0)
    R = 0 if inv_freq is None else 2 * inv_freq.shape[0]
    if R > d:
        raise ValueError(f"inv_freq: {R // 2} frequencies for heads of {d}")
    lay.need = (k.stride(1), k.stride(0), v.stride(1), v.stride(0), T)
    lay.tail = (ps, p64, R, int(interleaved))
    return lay


def paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, *,
                 max_k: int | None = None, k_starts: torch.Tensor | None = None, rows: int | None = None,
                 dtype: torch.dtype = torch.bfloat16, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                 error_word: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Whole sequences out of their pages, as window_attention() takes them (a
    prompt's next chunk attends to them that way): padded, [B][Hkv][max_k][d], or
    with k_starts (int32 [B + 1] on the device) packed, [rows][Hkv][d]. k_out and
    v_out: where to (their shapes then stand for max_k or rows). Pages of 4 bits give
    `dtype`, or k_out's type. Rows behind a sequence's kv_lens are not written (in
    outputs made here they hold anything); longer sequences than there are rows are
    cut and set DEV_BAD_LENGTH in error_word. Returns (k_out, v_out)."""
    if k_pages.requires_grad or v_pages.requires_grad or k_out is not None or v_out is not None:
        _forward_only("paged_gather", k_pages, v_pages, k_out, v_out)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out, v_out: give both or neither")
    if k_out is None:
        most = max_k if k_starts is None else rows
        if most is None or most < 0 or most >= 2**30:
            raise ValueError("paged_gather: give k_out and v_out, or max_k (with k_starts: rows), 0 to 2^30 - 1")
        t = dtype if k_pages.dtype is torch.uint8 else k_pages.dtype
        if t not in ops._DT or k_pages.dim() != 4:
            raise ValueError(f"paged_gather: need pages of 4 axes and float32 or bfloat16, got {tuple(k_pages.shape)} and {t}")
        d = k_pages.shape[-1] * 8 // 5 if k_pages.dtype is torch.uint8 else k_pages.shape[-1]
        shape = (block_table.shape[0], k_pages.shape[1], most, d) if k_starts is None else (most, k_pages.shape[1], d)
        k_out, v_out = k_pages.new_empty(shape, dtype=t), k_pages.new_empty(shape, dtype=t)
    key = ("gather", k_out.dtype, v_out.dtype, k_out.get_device(), v_out.get_device(), k_out.shape, v_out.shape, k_out.stride(), v_out.stride(),
           *_pages_key(k_pages, v_pages, block_table, kv_lens), k_starts is None)
    lay = ops._layouts.get(key) or _remember(key, _gather_layout(k_pages, v_pages, block_table, k_starts, k_out, v_out))
    _call("kvevict_paged_gather", k_out.get_device(), b"".join((
        _cache_args(lay, k_pages, v_pages, block_table, kv_lens, error_word),
        _GATHER_TAIL.pack(k_out.data_ptr(), v_out.data_ptr(), *lay.need, _ints(k_starts, lay.batch + 1, k_out, "k_starts")))))
    return k_out, v_out


def _gather_layout(k_pages, v_pages, block_table, k_starts, k_out, v_out) -> _Layout:
    ops._dtype(k_out, "k_out")
    packed = k_starts is not None
    dims = 3 if packed else 4
    _like(k_out, k_out, dims, "k_out")
    _like(v_out, k_out, dims, "v_out", k_out.shape)
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _strides(t, name)
    lay = _Layout()
    H, rows, d = k_out.shape[1], k_out.shape[0 if packed else 2], k_out.shape[-1]
    lay.head = struct.pack("@8i", *_cache_layout(lay, k_out.dtype, k_out.device, d, H, k_pages, v_pages, block_table))
    if not packed and k_out.shape[0] != lay.batch:
        raise ValueError(f"k_out: {k_out.shape[0]} sequences, block_table has {lay.batch}")
    strides = [(0, t.stride(1), t.stride(0)) if packed else t.stride()[:3] for t in (k_out, v_out)]
    lay.need = (*strides[0], *strides[1], rows)
    return lay


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, kv_lens: torch.Tensor, *,
                    q_starts: torch.Tensor | None = None, max_q: int | None = None, max_k: int | None = None, n_sink: int = 0,
                    window: int | None = None, scale: float | None = None, out: torch.Tensor | None = None,
                    lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None,
                    error_word: torch.Tensor | None = None):
    """Attention of the new tokens, q [T][Hq][d], over their sequences' pages: a
    query at position p sees the keys up to p that are among the first n_sink or the
    newest `window` (None: all), as in window_attention(). T / B tokens of every
    sequence (one: a decode step; a few: drafted ones), or with q_starts (and max_q,
    the longest; 0 counts as 1) any number: of a sequence with more than max_q the
    first ones are taken, and DEV_BAD_LENGTH is set in error_word. max_k, the most
    keys of a sequence, only steers the launch (None: as many as the table holds,
    which a table much wider than its sequences makes a slower plan of).
    Returns out (as q), or (out, lse [T][Hq]) with return_lse or an lse tensor; a row
    that sees nothing gives 0 and -inf. bf16 queries round the probabilities to bf16
    for the product with V, and over 4 bits want V's steps above 2^-50, its bases
    below 2^60 and queries below 2^118; fp32 ones are computed in fp32. For the many
    tokens of a prompt's chunk paged_gather() and window_attention() are faster."""
    if q.requires_grad or k_pages.requires_grad or v_pages.requires_grad or (out is not None and out.requires_grad):
        _forward_only("paged_attention", q, k_pages, v_pages, out)
    key = ("attention", q.dtype, q.get_device(), q.shape, q.stride(), *_pages_key(k_pages, v_pages, block_table, kv_lens), n_sink, window,
           scale, max_q, max_k, q_starts is None)
    lay = ops._layouts.get(key) or _remember(key, _attention_layout(q, k_pages, v_pages, block_table, q_starts, max_q, max_k, n_sink, window, scale))
    given = out is not None
    out, lse = _outputs(q, out, lse, return_lse, lay.lse_shape)
    os = (out.stride(1), out.stride(0)) if given else lay.out_shape
    workspace, wp, wn = _workspace(workspace, lay.need, q)
    _call("kvevict_paged_attention", q.get_device(), b"".join((
        _cache_args(lay, k_pages, v_pages, block_table, kv_lens, error_word), lay.tail,
        _ATTENTION_TAIL.pack(q.data_ptr(), out.data_ptr(), 0 if lse is None else lse.data_ptr(), q.stride(1), q.stride(0), *os,
                             _ints(q_starts, lay.batch + 1, q, "q_starts"), wp, wn))))
    return out if lse is None else (out, lse)


def _attention_layout(q, k_pages, v_pages, block_table, q_starts, max_q, max_k, n_sink, window, scale) -> _Layout:
    ops._dtype(q, "q")
    _like(q, q, 3, "q")
    _strides(q, "q")
    T, Hq, d = q.shape
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window: need at least 1, or None for no window")
    if n_sink < 0:
        raise ValueError("n_sink: need 0 or more")
    if q_starts is not None and max_q is None:
        raise ValueError("q_starts: give max_q, the most new tokens of a sequence")
    if (max_q is not None and max_q < 0) or (max_k is not None and max_k < 0):
        raise ValueError("max_q, max_k: need 0 or more")
    lay = _Layout()
    shape = _cache_layout(lay, q.dtype, q.device, d, None, k_pages, v_pages, block_table)
    if Hq % shape[3]:
        raise ValueError(f"q: {Hq} heads, the pages have {shape[3]}")
    _per_sequence(T, q_starts, lay.batch, "q")
    lay.head = struct.pack("@8i", *shape)
    # (a call that launches nothing would not report sequences with new tokens that max_q = 0 denies)
    lay.tail = _ATTENTION_HEAD.pack(Hq, min(n_sink, _INT_MAX), min(window, _INT_MAX), min(max(max_q or 0, 1), _INT_MAX), min(max_k or 0, _INT_MAX),
                                    _scale(scale), T)
    lay.lse_shape = q.shape[:2]
    lay.out_shape = (d, Hq * d)  # a dense output's strides
    # (of the starts only their presence counts for the size)
    lay.need = _workspace_need("kvevict_paged_attention", b"".join((
        lay.head, bytes(16), lay.strides, _TABLE.pack(0, 0, 0, 0), lay.tail,
        _ATTENTION_TAIL.pack(0, 0, 0, 0, 0, 0, 0, 0 if q_starts is None else 16, 0, 0))))
    return lay
