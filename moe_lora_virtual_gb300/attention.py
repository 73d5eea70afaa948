"""Binding of the attention half of a decoder layer (``include/mol_attn.h``).

Rotary positions, appending to a paged cache of keys and values, attention of the new
tokens over it. As in the package itself the functions keep the C names, marshal
arguments and raise ``MolError`` on a status; operands are on the current device.
Outputs and scratch that are not passed in are allocated on the stream that the call is
enqueued on. Nothing records gradients: operands that require them give outputs that do
not. A cache is a pair of bf16 tensors [pages, page_size, heads, head_dim] of one shape and
the same strides, the heads' values next to each other; a buffer laid out [pages, heads,
page_size, head_dim] is passed as its ``transpose(1, 2)``.
"""

from __future__ import annotations

import ctypes
import math
import operator
from typing import NamedTuple, Optional

import torch

from . import block as _block
from .block import _bf16, _call, _empty, _entry, _f32, _flat, _here, _i32, _stream

import moe_lora_virtual_gb300 as _mol

ATTN_EXPORTS = ("mol_rope", "mol_cache_append", "mol_paged_attention",
                "mol_paged_attention_workspace_bytes")
MOL_ROPE_MAX_HEAD_DIM = 512
MOL_ATTN_MAX_GROUP = 64

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_SZ = ctypes.c_size_t


class _RopeTable(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("rotary_dim", _I32), ("interleaved", _I32), ("magnitude", _F32)]


class _PagedCache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("page_stride", _I64), ("token_stride", _I64),
                ("head_stride", _I64), ("num_pages", _I64), ("page_size", _I32),
                ("num_heads", _I32), ("head_dim", _I32)]


_ROPE, _CACHE = ctypes.POINTER(_RopeTable), ctypes.POINTER(_PagedCache)
ATTN_SIGS = {
    "mol_rope": (_I32, [_P, _I64, _I64, _P, _ROPE, _I64, _I32, _I32, _P, _I64, _I64, _P]),
    "mol_cache_append": (_I32, [_P, _I64, _I64, _P, _I64, _I64, _P, _P, _ROPE, _I64, _CACHE, _P,
                                _I64, _I64, _I32, _P, _I64, _I64, _P]),
    "mol_paged_attention": (_I32, [_P, _I64, _I64, _CACHE, _P, _I64, _I32, _P, _P, _I64, _I64, _I32,
                                   _F32, _I32, _P, _I64, _I64, _P, _SZ, _P]),
    "mol_paged_attention_workspace_bytes": (_SZ, [_I64, _I64, _I32, _I32, _I32]),
}


class Rope(NamedTuple):
    """Rotary positions: pair i of a head's first 2 * len(inv_freq) values is turned by
    position * inv_freq[i] and multiplied by magnitude."""
    inv_freq: torch.Tensor      # fp32 [rotary_dim / 2]
    interleaved: bool = False   # pairs (2i, 2i + 1); else (i, i + rotary_dim / 2)
    magnitude: float = 1.0


def rope_frequencies(rotary_dim: int, base: float = 10000.0, *, interleaved: bool = False,
                     scaling: Optional[str] = None, factor: float = 1.0, trained: int = 0,
                     slow_turns: float = 1.0, fast_turns: float = 32.0,
                     magnitude: Optional[float] = None, device=None) -> Rope:
    """The frequencies base^(-2i / rotary_dim), for contexts `factor` times the trained ones scaled by

    "linear"  division by factor (positions interpolated);
    "base"    a larger base, base * factor^(rotary_dim / (rotary_dim - 2)): the fastest pair keeps its
              frequency, the slowest is divided by factor;
    "parts"   pairs that turn fast_turns times or more over the `trained` tokens kept, those that turn
              slow_turns times or fewer divided by factor, a ramp between them over the pair's index;
              magnitude 0.1 * ln(factor) + 1 unless given."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError(f"rotary_dim: expected an even number, got {rotary_dim}")
    if scaling not in (None, "linear", "base", "parts"):
        raise ValueError(f"scaling: expected None, 'linear', 'base' or 'parts', got {scaling!r}")
    if not factor >= 1.0 or not base > 1.0:
        raise ValueError("factor: expected 1 or more, base: more than 1")
    n = rotary_dim // 2
    i = torch.arange(n, dtype=torch.float64)
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-i / n)
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if trained < 1 or not 0 < slow_turns < fast_turns:
            raise ValueError("scaling 'parts': expected trained tokens and 0 < slow_turns < fast_turns")
        # the pair (a real number) that turns so many times over the trained tokens
        at = [n * math.log(trained / (2 * math.pi * turns)) / math.log(base)
              for turns in (fast_turns, slow_turns)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary_dim - 1)
        divided = ((i - low) / max(high - low, 0.001)).clamp(0.0, 1.0)
        f = f * (1 - divided) + f / factor * divided
        if magnitude is None:
            magnitude = 0.1 * math.log(factor) + 1.0
    return Rope(f.to(device=device, dtype=torch.float32), interleaved,
                1.0 if magnitude is None else magnitude)


def _number(x) -> int:
    """x as an int32 argument takes it: one past its ends becomes the nearer end (ctypes would keep its
    low 32 bits, which may be any number)."""
    return min(max(operator.index(x), -(1 << 31)), (1 << 31) - 1)


def _heads(t: torch.Tensor, name: str):
    """(token stride, head stride) of a CUDA operand [tokens, heads, head_dim]."""
    if t.dtype != _bf16 or not t.is_cuda:
        _mol._need(t, _bf16, name)
    _here(t, name)
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] > 1):
        raise ValueError(f"{name}: expected [tokens, heads, head_dim] with the head's values next to "
                         "each other")
    # a single token or head has no stride that matters
    head = stride[1] if shape[1] > 1 else 8 * -(-shape[2] // 8)
    return stride[0] if shape[0] > 1 else max(8, 8 * -(-shape[1] * head // 8)), head


def _same(t: torch.Tensor, shape, name: str) -> None:
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _rope_table(rope: Rope) -> _RopeTable:
    f = rope.inv_freq
    if f.dim() != 1:
        raise ValueError("inv_freq: expected one dimension")
    return _RopeTable(_flat(f, _f32, "inv_freq", f.shape), _number(2 * f.shape[0]),
                      _number(int(rope.interleaved)), rope.magnitude)


def _paged(k: torch.Tensor, v: torch.Tensor) -> _PagedCache:
    for t, name in ((k, "k_cache"), (v, "v_cache")):
        if t.dtype != _bf16 or not t.is_cuda:
            _mol._need(t, _bf16, name)
        _here(t, name)
        if t.dim() != 4 or (t.stride(3) != 1 and t.shape[3] > 1):
            raise ValueError(f"{name}: expected [pages, page_size, heads, head_dim] with the head's "
                             "values next to each other")
    _same(v, k.shape, "v_cache")
    if v.stride() != k.stride():
        raise ValueError("k_cache, v_cache: expected the same strides")
    s, n = k.stride(), k.shape
    # a single page, token or head has no stride that matters
    return _PagedCache(k.data_ptr(), v.data_ptr(), s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0,
                       s[2] if n[2] > 1 else 0, n[0], *(_number(x) for x in n[1:]))


def _like(out: Optional[torch.Tensor], x: torch.Tensor, stream, name: str) -> torch.Tensor:
    if out is None:
        return _empty(x.shape, _bf16, x, stream)
    _same(out, x.shape, name)
    return out


def mol_rope(x: torch.Tensor, positions: torch.Tensor, rope: Rope,
             out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """x bf16 [T, heads, head_dim] with positions int32 [T] turned into it; out may be `x`."""
    if _block._native is not None and out is None and stream is None:
        done = _block._native.rope(_entry("mol_rope"), x, positions, rope[0], int(rope[1]), rope[2])
        if done is not None:
            return done
    xt, xh = _heads(x, "x")
    T, H, D = x.shape
    table = _rope_table(rope)
    pp = _flat(positions, _i32, "positions", (T,))
    out = _like(out, x, stream, "out")
    ot, oh = _heads(out, "out")
    _call("mol_rope", x.data_ptr(), xt, xh, pp, table, T, H, D, out.data_ptr(), ot, oh,
          _stream(stream, x))
    return out


def mol_cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor,
                     v_cache: torch.Tensor, slots: torch.Tensor,
                     positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                     q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                     stream=None) -> Optional[torch.Tensor]:
    """Writes k (turned by positions with `rope`) and v, bf16 [T, kv_heads, head_dim], into slots
    int32 [T] of the cache (page * page_size + offset; outside the cache, as -1: not written), and
    returns q bf16 [T, heads, head_dim] turned likewise (None without q). q_out may be `q`; tokens
    name different slots."""
    if _block._native is not None and q_out is None and stream is None:
        f, interleaved, magnitude = (None, 0, 1.0) if rope is None else rope
        done = _block._native.cache_append(_entry("mol_cache_append"), k, v, k_cache, v_cache, slots,
                                           positions, f, int(interleaved), magnitude, q)
        if done is not None:
            return None if done is True else done
    kt, kh = _heads(k, "k")
    vt, vh = _heads(v, "v")
    T, H, D = k.shape
    _same(v, k.shape, "v")
    cache = _paged(k_cache, v_cache)
    if (H, D) != tuple(k_cache.shape[2:]):
        raise ValueError(f"k: expected {k_cache.shape[2]} heads of {k_cache.shape[3]}, got {H} of {D}")
    sp = _flat(slots, _i32, "slots", (T,))
    table = pp = None
    if rope is not None:
        if positions is None:
            raise ValueError("positions: needed with rope")
        table, pp = _rope_table(rope), _flat(positions, _i32, "positions", (T,))
    qp, qt, qh, Hq, op, ot, oh = None, 0, 0, 0, None, 0, 0
    if q is not None:
        if rope is None:
            raise ValueError("q: needs rope")
        qt, qh = _heads(q, "q")
        Hq = q.shape[1]
        _same(q, (T, Hq, D), "q")
        q_out = _like(q_out, q, stream, "q_out")
        ot, oh = _heads(q_out, "q_out")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out: needs q")
    _call("mol_cache_append", k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, sp, pp, table, T, cache, qp,
          qt, qh, Hq, op, ot, oh, _stream(stream, k))
    return q_out


def mol_paged_attention_workspace_bytes(num_seqs: int, num_tokens: int, num_q_heads: int,
                                        num_kv_heads: int, head_dim: int) -> int:
    """Bytes of workspace that serve every mol_paged_attention of at most num_seqs sequences and
    num_tokens tokens of these heads (of a long-lived buffer: of the largest sizes)."""
    return (_mol._lib or _mol.library()).mol_paged_attention_workspace_bytes(
        num_seqs, num_tokens, _number(num_q_heads), _number(num_kv_heads), _number(head_dim))


def mol_paged_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                        page_table: torch.Tensor, kv_lens: torch.Tensor,
                        q_starts: Optional[torch.Tensor] = None, *, scale: Optional[float] = None,
                        window: int = 0, out: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out [T, heads, head_dim]: attention of q's rows, each sequence's last tokens, over its cache.

    page_table int32 [B, pages] (entries outside the cache, as -1: tokens that no row sees); kv_lens
    int32 [B]: cached tokens, the new ones among them; q_starts int32 [B + 1]: where each sequence's
    rows begin (None: a row each), not decreasing (else no row is written); window > 0: the last
    tokens that a row sees, its own among them (2^31 - 1 and more: all of them); scale:
    head_dim^-0.5 unless given. Rows that see nothing, or whose every score is -infinity, are 0; rows
    of no sequence keep what out held. workspace: mol_paged_attention_workspace_bytes of scratch, of
    these sizes or larger ones. out may be `q`."""
    if _block._native is not None and out is None and workspace is None and stream is None:
        done = _block._native.paged_attention(
            _entry("mol_paged_attention"), _entry("mol_paged_attention_workspace_bytes"), q, k_cache,
            v_cache, page_table, kv_lens, q_starts, q.shape[-1] ** -0.5 if scale is None else scale,
            window)
        if done is not None:
            return done
    qt, qh = _heads(q, "q")
    T, H, D = q.shape
    cache = _paged(k_cache, v_cache)
    kv_heads = k_cache.shape[2]
    if D != k_cache.shape[3]:
        raise ValueError(f"q: expected heads of {k_cache.shape[3]}, got {D}")
    if page_table.dtype != _i32 or not page_table.is_cuda:
        _mol._need(page_table, _i32, "page_table")
    _here(page_table, "page_table")
    if page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table: expected [sequences, pages] with unit column stride")
    B, pages = page_table.shape
    lens = _flat(kv_lens, _i32, "kv_lens", (B,))
    starts = None if q_starts is None else _flat(q_starts, _i32, "q_starts", (B + 1,))
    if starts is None and T != B:
        raise ValueError(f"q: expected a row for each of {B} sequences, got {T} (q_starts gives others)")
    out = _like(out, q, stream, "out")
    ot, oh = _heads(out, "out")
    need = mol_paged_attention_workspace_bytes(B, T, H, kv_heads, D)
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, q, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace: expected a contiguous CUDA tensor")
    else:
        _here(workspace, "workspace")
    _call("mol_paged_attention", q.data_ptr(), qt, qh, cache, page_table.data_ptr(),
          page_table.stride(0) if B > 1 else pages, pages, lens, starts, B, T, H,
          D ** -0.5 if scale is None else scale, _number(window), out.data_ptr(), ot, oh,
          workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream, q))
    return out
