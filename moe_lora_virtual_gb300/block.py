"""Binding of the MoE block around the LoRA path (``include/mol_block.h``).

Norms between blocks, the router's choice, the experts for a few tokens and the
4-bit linear. As in the package itself the functions keep the C names, marshal
arguments and raise ``MolError`` on a status; operands are on the current device.
Outputs that are not passed in are allocated, like scratch, on the stream that the
call is enqueued on: with ``stream`` they are that stream's tensors. ``w4_pack``,
``w4_quantize`` and ``w4_unpack`` lay 4-bit weights out once, with torch operations on
the tensors' own device.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional, Union

import torch

import moe_lora_virtual_gb300 as _mol
from .build import native_current

_native = None  # the common case of each call in one native step; None from it: the Python path below
if native_current():  # (one that was built for another PyTorch might load, and fail later)
    try:
        from . import _block_native as _native
    except ImportError:
        pass

BLOCK_EXPORTS = ("mol_block_norm", "mol_moe_route", "mol_moe_gate_up", "mol_moe_down",
                 "mol_moe_forward", "mol_moe_workspace_bytes", "mol_moe_down_split",
                 "mol_moe_forward_split", "mol_w4_linear")
MOL_NORM_MAX_H = 16384
MOL_ROUTE_MAX_EXPERTS = 1024
MOL_ROUTE_MAX_TOPK = 32
MOL_MOE_MAX_TOKENS = 128
MOL_MOE_MAX_PAIRS = 1024
MOL_MOE_MAX_EXPERTS = 1024
MOL_MOE_MAX_WIDTH = 65536
MOL_W4_MAX_TOKENS = 64
MOL_F32, MOL_BF16 = 0, 1

_P, _I32, _I64, _F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
_SZ = ctypes.c_size_t
BLOCK_SIGS = {
    "mol_block_norm": (_I32, [_P, _I64, _P, _I64, _P, _P, _I64, _F32, _P, _F32, _I64, _I32, _P,
                              _I64, _P, _I64, _P]),
    "mol_moe_route": (_I32, [_P, _I32, _I64, _I64, _I32, _I32, _I32, _F32, _P, _P, _P]),
    "mol_moe_gate_up": (_I32, [_P, _I64, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _I32, _P, _I64,
                               _P, _P]),
    "mol_moe_down": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _I32, _P, _I64, _P,
                            _I64, _P]),
    "mol_moe_forward": (_I32, [_P, _I64, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _I32,
                               _P, _P, _I64, _P]),
    "mol_moe_workspace_bytes": (_SZ, [_I64, _I32, _I32, _I32, _I32, _I32]),
    "mol_moe_down_split": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _I32, _P, _I64,
                                  _P, _SZ, _P, _I64, _P]),
    "mol_moe_forward_split": (_I32, [_P, _I64, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                     _I32, _P, _P, _SZ, _P, _I64, _P]),
    "mol_w4_linear": (_I32, [_P, _I64, _I64, _I32, _I32, _P, _P, _I32, _P, _I64, _P]),
}


class W4(NamedTuple):
    """4-bit weight rows: value[..., k] = scales[..., k // group] * (q - 8).

    The byte layout is that of ``include/mol_block.h``; ``w4_pack`` makes it."""
    qweight: torch.Tensor   # uint8 [..., N, Kp // 2], Kp = in_features rounded up to 256
    scales: torch.Tensor    # bf16 [..., N, Kp // group]
    in_features: int
    group: int


Weights = Union[torch.Tensor, W4]
GROUPS = (32, 64, 128)
# Input j of a word's eight sits at bit _SHIFTS[j].
_SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)


def _padded(k: int) -> int:
    return (k + 255) // 256 * 256


def w4_pack(q: torch.Tensor, scales: torch.Tensor, group: int) -> W4:
    """Packs q (integers 0..15, [..., N, K]) and scales ([..., N, ceil(K / group)])."""
    if group not in GROUPS:
        raise ValueError(f"group: expected one of {GROUPS}, got {group}")
    K = q.shape[-1]
    groups = -(-K // group)
    if scales.shape != q.shape[:-1] + (groups,):
        raise ValueError(f"scales: expected {tuple(q.shape[:-1]) + (groups,)}, "
                         f"got {tuple(scales.shape)}")
    if q.dtype.is_floating_point or q.dtype.is_complex:
        raise TypeError(f"q: expected integers, got {q.dtype}")
    if q.numel() and (int(q.min()) < 0 or int(q.max()) > 15):
        raise ValueError("q: expected integers 0..15")
    Kp, lead = _padded(K), q.shape[:-1]
    padded = torch.full((*lead, Kp), 8, dtype=torch.uint8, device=q.device)
    padded[..., :K] = q
    # inputs [block, i, t, j] -> words [block, t, i], byte b = inputs at bits 8b and 8b + 4
    v = padded.view(*lead, Kp // 128, 4, 4, 8).transpose(-3, -2)
    order = sorted(range(8), key=lambda j: _SHIFTS[j])
    v = v[..., order]
    qweight = (v[..., 0::2] | (v[..., 1::2] << 4)).reshape(*lead, Kp // 2).contiguous()
    s = torch.zeros(*lead, Kp // group, dtype=torch.bfloat16, device=q.device)
    s[..., :groups] = scales.to(torch.bfloat16)
    return W4(qweight, s, K, group)


def w4_quantize(w: torch.Tensor, group: int = 128) -> W4:
    """Rounds weight rows [..., N, K] to 4 bits, to the nearest step: a group's step, its scale, is the
    least that keeps its values within -8 and 7 steps, then rounded to bf16 (values that this leaves
    outside are clipped to them)."""
    if group not in GROUPS:
        raise ValueError(f"group: expected one of {GROUPS}, got {group}")
    K = w.shape[-1]
    groups = -(-K // group)
    f = torch.zeros(*w.shape[:-1], groups * group, dtype=torch.float32, device=w.device)
    f[..., :K] = w
    f = f.view(*w.shape[:-1], groups, group)
    s = torch.maximum(f.amax(-1) / 7, -f.amin(-1) / 8).to(torch.bfloat16)
    step = torch.where(s > 0, s, torch.ones_like(s)).to(torch.float32).unsqueeze(-1)
    q = torch.clamp(torch.round(f / step), -8, 7).add_(8).to(torch.uint8)
    return w4_pack(q.view(*w.shape[:-1], groups * group)[..., :K], s, group)


def w4_unpack(w: W4) -> torch.Tensor:
    """fp32 weight rows [..., N, K] of packed ones."""
    lead = w.qweight.shape[:-1]
    v = torch.stack([w.qweight & 15, w.qweight >> 4], -1).view(*lead, -1, 4, 4, 8)
    order = sorted(range(8), key=lambda j: _SHIFTS[j])
    back = [order.index(j) for j in range(8)]
    v = v[..., back].transpose(-3, -2).reshape(*lead, -1, w.group).to(torch.float32) - 8
    v = v * w.scales.to(torch.float32).unsqueeze(-1)
    return v.reshape(*lead, -1)[..., :w.in_features]


# The checks below read each property of a tensor once and allocate like their input: what a call
# costs on the host is what the smallest calls take.
_bf16, _f32, _i32 = torch.bfloat16, torch.float32, torch.int32


def _here(t: torch.Tensor, name: str) -> None:
    """A call launches on the current device, so all of its operands have to be there."""
    at = torch.cuda.current_device()
    if t.get_device() != at:
        raise ValueError(f"{name}: expected a tensor on the current device, cuda:{at}, got one on "
                         f"cuda:{t.get_device()}")


def _rows(t: torch.Tensor, dtype, name: str) -> int:
    """Row stride of a 2-D CUDA operand with unit column stride."""
    if t.dtype != dtype or not t.is_cuda:
        _mol._need(t, dtype, name)
    _here(t, name)
    stride, shape = t.stride(), t.shape
    if len(stride) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{name}: expected a 2-D tensor with unit column stride")
    # a single row (or none) has no stride that matters
    return stride[0] if shape[0] > 1 else max(shape[1], 8 * -(-shape[1] // 8))


def _flat(t: torch.Tensor, dtype, name: str, shape) -> int:
    if t.dtype != dtype or not t.is_cuda:
        _mol._need(t, dtype, name)
    _here(t, name)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor of shape {tuple(shape)}, got "
                         f"{tuple(t.shape)}")
    return t.data_ptr()


def _vector(t: Optional[torch.Tensor], name: str, n: int):
    return None if t is None else _flat(t, _bf16, name, (n,))


def _weights(w: Weights, name: str, lead, K: int):
    """(data, scales, group) of bf16 rows or packed 4-bit rows [*lead, K]."""
    if isinstance(w, W4):
        if w.in_features != K:
            raise ValueError(f"{name}: expected {K} inputs, got {w.in_features}")
        if w.group not in GROUPS:
            raise ValueError(f"{name}: group is one of {GROUPS}, got {w.group}")
        Kp = _padded(K)
        return (_flat(w.qweight, torch.uint8, name, (*lead, Kp // 2)),
                _flat(w.scales, _bf16, name + " scales", (*lead, Kp // w.group)), w.group)
    return _flat(w, _bf16, name, (*lead, K)), None, 0


def _native_weights(w: Weights):
    return w if isinstance(w, W4) else (w, None, w.shape[-1], 0)


def _lead(w: Weights) -> torch.Size:
    return (w.qweight if isinstance(w, W4) else w).shape[:-1]


def _delta(delta: Optional[torch.Tensor], pairs: int, width: int):
    if delta is None:
        return None, 0
    stride = _rows(delta, _bf16, "delta")
    if delta.shape != (pairs, width):
        raise ValueError(f"delta: expected shape {(pairs, width)}, got {tuple(delta.shape)}")
    return delta.data_ptr(), stride


def _empty(shape, dtype, like: torch.Tensor, stream) -> torch.Tensor:
    """A new tensor of the call, allocated on the stream that the call is enqueued on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with _mol._on(stream, like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _out(out: Optional[torch.Tensor], shape, like: torch.Tensor, stream, name: str = "out"):
    if out is None:
        return _empty(shape, _bf16, like, stream), shape[1]
    stride = _rows(out, _bf16, name)
    if out.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(out.shape)}")
    return out, stride


def _call(name: str, *args) -> None:
    status = getattr(_mol._lib or _mol.library(), name)(*args)
    if status != 0:
        raise _mol.MolError(name, status)


def _entry(name: str) -> int:
    """Address of a C entry point of the library in use."""
    lib = _mol._lib or _mol.library()
    addresses = lib.__dict__.setdefault("_block_entries", {})
    if name not in addresses:
        addresses[name] = ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
    return addresses[name]


def _stream(stream, t: torch.Tensor) -> int:
    """The stream given, or the current one of the tensor's device."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def mol_block_norm(y: torch.Tensor, residual: torch.Tensor, pre_weight: Optional[torch.Tensor], *,
                   post_weight: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None,
                   residual_scale: float = 1.0, eps: float = 1e-6,
                   residual_out: Optional[torch.Tensor] = None,
                   normed: Optional[torch.Tensor] = None, stream=None):
    """residual + residual_scale * gate * rms(y; post_weight), and its rms(.; pre_weight).

    y, residual bf16 [T, H]; post_weight, pre_weight bf16 [H] or None; gate bf16 [H], [T, H] or
    None. Returns (residual_out, normed); normed is None without pre_weight. residual_out may be
    `residual`, normed may be `y`."""
    if _native is not None and residual_out is None and normed is None and stream is None:
        done = _native.block_norm(_entry("mol_block_norm"), y, residual, pre_weight, post_weight,
                                  gate, residual_scale, eps)
        if done is not None:
            return done
    shape = T, H = y.shape
    ys = _rows(y, _bf16, "y")
    rs = _rows(residual, _bf16, "residual")
    if residual.shape != shape:
        raise ValueError(f"residual: expected shape {tuple(y.shape)}, got {tuple(residual.shape)}")
    gp, gs = None, 0
    if gate is not None:
        if gate.dim() == 1:
            gp = _flat(gate, _bf16, "gate", (H,))
        else:
            gp, gs = gate.data_ptr(), _rows(gate, _bf16, "gate")
            if gate.shape != y.shape:
                raise ValueError(f"gate: expected shape {(H,)} or {tuple(y.shape)}, got "
                                 f"{tuple(gate.shape)}")
    post, pre = _vector(post_weight, "post_weight", H), _vector(pre_weight, "pre_weight", H)
    residual_out, ros = _out(residual_out, shape, y, stream, "residual_out")
    ns = 0
    if pre is not None:
        normed, ns = _out(normed, shape, y, stream, "normed")
    elif normed is not None:
        raise ValueError("normed: needs pre_weight")
    _call("mol_block_norm", y.data_ptr(), ys, residual.data_ptr(), rs, post, gp, gs, residual_scale,
          pre, eps, T, H, residual_out.data_ptr(), ros,
          None if normed is None else normed.data_ptr(), ns, _stream(stream, y))
    return residual_out, normed


def mol_moe_route(logits: torch.Tensor, topk: int, renormalize: bool = True, scale: float = 1.0,
                  topk_ids: Optional[torch.Tensor] = None,
                  topk_weights: Optional[torch.Tensor] = None, stream=None):
    """(topk_ids int32, topk_weights fp32), [T, topk] each, of router logits fp32 or bf16 [T, E]."""
    if _native is not None and topk_ids is None and topk_weights is None and stream is None:
        done = _native.moe_route(_entry("mol_moe_route"), logits, topk, int(renormalize), scale)
        if done is not None:
            return done
    bf16 = logits.dtype == _bf16
    stride = _rows(logits, _bf16 if bf16 else _f32, "logits")
    T, E = logits.shape
    if topk_ids is None:
        topk_ids = _empty((T, topk), _i32, logits, stream)
    if topk_weights is None:
        topk_weights = _empty((T, topk), _f32, logits, stream)
    _call("mol_moe_route", logits.data_ptr(), MOL_BF16 if bf16 else MOL_F32, stride, T, E, topk,
          int(renormalize), scale, _flat(topk_ids, _i32, "topk_ids", (T, topk)),
          _flat(topk_weights, _f32, "topk_weights", (T, topk)), _stream(stream, logits))
    return topk_ids, topk_weights


def mol_moe_gate_up(x: torch.Tensor, topk_ids: torch.Tensor, w_gate_up: Weights,
                    act: Optional[torch.Tensor] = None, delta: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """act [T * topk, I] = silu(gate) * up of each pair's expert; rows without one are not written.

    x bf16 [T, H]; topk_ids int32 [T, topk]; w_gate_up bf16 [E, 2I, H] or W4; delta bf16
    [T * topk, 2I]: rows a LoRA gate_up stage added into zeros."""
    if _native is not None and act is None and stream is None:
        done = _native.moe_gate_up(_entry("mol_moe_gate_up"), x, topk_ids, *_native_weights(w_gate_up),
                                   delta)
        if done is not None:
            return done
    (T, H), k = x.shape, topk_ids.shape[1]
    E, I2 = _lead(w_gate_up)
    if I2 % 2:
        raise ValueError(f"w_gate_up: expected as many up rows as gate rows, got {I2} in all")
    wp, sp, group = _weights(w_gate_up, "w_gate_up", (E, I2), H)
    dp, ds = _delta(delta, T * k, I2)
    if act is None:
        act = _empty((T * k, I2 // 2), _bf16, x, stream)
    _call("mol_moe_gate_up", x.data_ptr(), _rows(x, _bf16, "x"),
          _flat(topk_ids, _i32, "topk_ids", (T, k)), T, k, E, H, I2 // 2, wp, sp, group, dp,
          ds, _flat(act, _bf16, "act", (T * k, I2 // 2)), _stream(stream, x))
    return act


def mol_moe_workspace_bytes(num_tokens: int, topk: int, num_experts: int, hidden: int, inter: int,
                            group: int = 0) -> int:
    """Bytes of workspace mol_moe_down and mol_moe_forward use for these sizes (often 0)."""
    return (_mol._lib or _mol.library()).mol_moe_workspace_bytes(num_tokens, topk, num_experts,
                                                                 hidden, inter, group)


def _workspace(workspace: Optional[torch.Tensor], like: torch.Tensor, stream, *shape):
    """(pointer, bytes, tensor) of the workspace for these sizes: the one given, or a new one."""
    need = mol_moe_workspace_bytes(*shape)
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty(need, torch.uint8, like, stream)
    if not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace: expected a contiguous CUDA tensor")
    _here(workspace, "workspace")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def mol_moe_down(act: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                 w_down: Weights, out: Optional[torch.Tensor] = None,
                 delta: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """out [T, H] = sum over a token's pairs of topk_weights * (w_down[e] . act + delta).

    act bf16 [T * topk, I]; w_down bf16 [E, H, I] or W4; delta bf16 [T * topk, H]: rows a LoRA down
    stage added into zeros; workspace: mol_moe_workspace_bytes of scratch."""
    if _native is not None and out is None and workspace is None and stream is None:
        done = _native.moe_down(_entry("mol_moe_down_split"), _entry("mol_moe_workspace_bytes"), act,
                                topk_ids, topk_weights, *_native_weights(w_down), delta)
        if done is not None:
            return done
    T, k = topk_ids.shape
    E, H = _lead(w_down)
    I = act.shape[1]
    wp, sp, group = _weights(w_down, "w_down", (E, H), I)
    dp, ds = _delta(delta, T * k, H)
    out, os = _out(out, (T, H), act, stream)
    ws, wsb, workspace = _workspace(workspace, act, stream, T, k, E, H, I, group)
    _call("mol_moe_down_split", _flat(act, _bf16, "act", (T * k, I)),
          _flat(topk_ids, _i32, "topk_ids", (T, k)),
          _flat(topk_weights, _f32, "topk_weights", (T, k)), T, k, E, H, I, wp, sp, group,
          dp, ds, ws, wsb, out.data_ptr(), os, _stream(stream, act))
    return out


def mol_moe_forward(x: torch.Tensor, topk_ids: torch.Tensor, topk_weights: torch.Tensor,
                    w_gate_up: Weights, w_down: Weights, out: Optional[torch.Tensor] = None,
                    act: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """The experts of a MoE layer for a few tokens: mol_moe_gate_up, then mol_moe_down.

    x bf16 [T, H]; topk_ids int32 and topk_weights fp32 [T, topk]; weights bf16 [E, 2I, H] and
    [E, H, I], or both W4 of one group; scratch: act bf16 [T * topk, I], workspace of
    mol_moe_workspace_bytes."""
    if (_native is not None and out is None and act is None and workspace is None
            and stream is None):
        done = _native.moe_forward(_entry("mol_moe_forward_split"),
                                   _entry("mol_moe_workspace_bytes"), x, topk_ids, topk_weights,
                                   *_native_weights(w_gate_up), *_native_weights(w_down))
        if done is not None:
            return done
    (T, H), k = x.shape, topk_ids.shape[1]
    E, I2 = _lead(w_gate_up)
    I = I2 // 2
    gp, gsp, group = _weights(w_gate_up, "w_gate_up", (E, 2 * I), H)
    wp, wsp, group_down = _weights(w_down, "w_down", (E, H), I)
    if group != group_down:
        raise ValueError("w_gate_up, w_down: expected the same type and group")
    if act is None:
        act = _empty((T * k, I), _bf16, x, stream)
    out, os = _out(out, (T, H), x, stream)
    ws, wsb, workspace = _workspace(workspace, x, stream, T, k, E, H, I, group)
    _call("mol_moe_forward_split", x.data_ptr(), _rows(x, _bf16, "x"),
          _flat(topk_ids, _i32, "topk_ids", (T, k)),
          _flat(topk_weights, _f32, "topk_weights", (T, k)), T, k, E, H, I, gp, gsp, wp,
          wsp, group, _flat(act, _bf16, "act", (T * k, I)), ws, wsb, out.data_ptr(), os,
          _stream(stream, x))
    return out


def mol_w4_linear(x: torch.Tensor, w: W4, out: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """out [T, N] = x [T, K] . w^T with 4-bit weight rows [N, K]."""
    if not isinstance(w, W4):
        raise TypeError("w: expected W4")
    if _native is not None and out is None and stream is None:
        done = _native.w4_linear(_entry("mol_w4_linear"), x, *w)
        if done is not None:
            return done
    T, K = x.shape
    (N,) = _lead(w)
    wp, sp, group = _weights(w, "w", (N,), K)
    out, os = _out(out, (T, N), x, stream)
    _call("mol_w4_linear", x.data_ptr(), _rows(x, _bf16, "x"), T, K, N, wp, sp, group,
          out.data_ptr(), os, _stream(stream, x))
    return out
