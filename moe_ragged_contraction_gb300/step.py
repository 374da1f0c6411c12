"""Operators of a training step around the expert products (argument
marshalling only; see include/mxfp8_step.h): tokens sorted by expert and back,
with the router's weights and the gradients of both directions, and the global
norm and clipping of gradients.

``stream``: as in moe_layer and muon_update. The gradients are operators of
their own (token_dispatch_grad, token_combine_grad): tensors that require a
gradient are refused while gradients are being recorded, and tensors with a
forward-mode tangent."""
from __future__ import annotations

from array import array
from operator import attrgetter, index, methodcaller
from typing import NamedTuple

from . import _lib
from . import experts as _experts
from .experts import _int32, _sizes


class TokenPlan(NamedTuple):
    """A routing's rows: offs int32 [local] (inclusive group ends), slot int32 [T, top_k] (the row of each pair, or -1)
    and src int32 [rows] (the pair t * top_k + j of each row, or -1), all on one CUDA device."""
    offs: "object"
    slot: "object"
    src: "object"


def _check(t, dtype, shape, name, device):
    """Raises unless t is a contiguous tensor of that dtype and shape on that CUDA device."""
    if isinstance(t, _experts._torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    _lib._expect(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the first argument on cuda:{device}")


def _new(stream, shape, dtype, like):
    if stream is None:
        return _experts._torch.empty(shape, dtype=dtype, device=like.device)
    return _lib._empty(stream, shape, dtype, like.device)


def _begin(t, name, stream):
    torch = _experts._torch or _experts._torch_module()
    device, st = _experts._device_and_stream(t, name, stream)
    return torch, _lib._lib or _lib.load(), device, st


def _plan(torch, plan, device):
    """(slot, src, T, top_k, rows) of a plan."""
    _, slot, src = plan
    if not (isinstance(slot, torch.Tensor) and isinstance(src, torch.Tensor)):
        raise ValueError("plan must be a TokenPlan: offs [local], slot [T, top_k] and src [rows]")
    shape, rows = slot.shape, src.shape
    if len(shape) != 2 or len(rows) != 1:
        raise ValueError("plan must be a TokenPlan: offs [local], slot [T, top_k] and src [rows]")
    _check(slot, torch.int32, shape, "plan.slot", device)
    _check(src, torch.int32, rows, "plan.src", device)
    if shape[1] >> 31:
        raise ValueError(f"top_k={shape[1]} is out of range")
    return slot, src, shape[0], shape[1], rows[0]


def _columns(t):
    """H of a tensor [.., H]."""
    H = t.shape[-1] if t.dim() else 0
    if H >> 31:
        raise ValueError(f"H={H} is out of range")
    return H


def token_plan_rows(T: int, top_k: int, local: int, align: int = 32) -> int:
    """Rows of the sorted buffers that hold every routing of T tokens (see include/mxfp8_step.h)."""
    T, v = index(T), _sizes(top_k, local, align)
    rows = int((_lib._lib or _lib.load()).mxfp8_token_plan_rows(T, *v)) if v and 0 <= T < 2 ** 31 else -1
    if rows < 0:
        raise ValueError(f"unsupported sizes T={T}, top_k={top_k}, local={local}, align={align}")
    return rows


def token_plan(ids, local, *, first_expert=0, align=32, rows=None, out=None, stream=None):
    """The plan of a routing (see include/mxfp8_step.h).

    ids: int32 or int64 [T, top_k], the experts each token chose; those from
    first_expert on, ``local`` of them, are here, all other entries (-1 for padding
    tokens) are absent. Groups end on multiples of ``align``: 32 for
    wgrad_grouped, any for grouped_gemm. rows: the rows of the sorted buffers, a
    multiple of align (default: enough for every routing, token_plan_rows); pairs
    beyond them are dropped, with a bit of device_status(). Returns (or fills)
    ``out``: TokenPlan(offs, slot, src).
    """
    torch, lib, device, st = _begin(ids, "ids", stream)
    if ids.dtype is not torch.int32 and ids.dtype is not torch.int64:
        raise TypeError(f"ids must be torch.int32 or torch.int64, got {ids.dtype}")
    if ids.dim() != 2:
        raise ValueError(f"ids must be [T, top_k], got {list(ids.shape)}")
    _check(ids, ids.dtype, ids.shape, "ids", device)
    T, k = ids.shape
    k, local, first_expert, align = _int32(k, "top_k"), _int32(local, "local"), _int32(first_expert, "first_expert"), _int32(align, "align")
    i32 = torch.int32
    if rows is None:
        rows = token_plan_rows(T, k, local, align) if out is None else out[2].shape[0]
    else:
        rows = _int32(rows, "rows")
    if out is None:
        if rows < 0 or local < 0:
            raise ValueError(f"rows={rows} and local={local} must not be negative")
        out = TokenPlan(_new(stream, (local,), i32, ids), _new(stream, (T, k), i32, ids), _new(stream, (rows,), i32, ids))
    else:
        out = TokenPlan(*out)
        for t, shape, name in zip(out, ((local,), (T, k), (rows,)), ("out.offs", "out.slot", "out.src")):
            _check(t, i32, shape, name, device)
    offs, slot, src = out
    rc = lib.mxfp8_token_plan(ids.data_ptr(), 0 if ids.dtype is i32 else 1, T, k, first_expert, local, align, rows, offs.data_ptr(),
                              slot.data_ptr(), src.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return out


def token_dispatch(x, plan, *, out=None, stream=None):
    """Rows sorted by expert (see include/mxfp8_step.h): x bf16 [T, H] -> out bf16 [rows, H], zeros on padding rows."""
    torch, lib, device, st = _begin(x, "x", stream)
    slot, src, T, k, rows = _plan(torch, plan, device)
    H = _columns(x)
    _check(x, torch.bfloat16, (T, H), "x", device)
    if out is None:
        out = _new(stream, (rows, H), torch.bfloat16, x)
    else:
        _check(out, torch.bfloat16, (rows, H), "out", device)
    if (x.requires_grad or out.requires_grad) and torch.is_grad_enabled():
        _experts._refuse_gradients(x=x, out=out)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((("x", x), ("out", out)))
    rc = lib.mxfp8_token_dispatch(x.data_ptr(), T, H, k, slot.data_ptr(), src.data_ptr(), rows, out.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return out


def token_dispatch_mxfp8(x, plan, *, q=None, s=None, stream=None):
    """The rows of token_dispatch quantised along H, grouped_gemm's X (see include/mxfp8_step.h):
    x bf16 [T, H] -> (q uint8 [rows, H] E4M3, s uint8 [rows, H/32] E8M0)."""
    torch, lib, device, st = _begin(x, "x", stream)
    slot, src, T, k, rows = _plan(torch, plan, device)
    H = _columns(x)
    _check(x, torch.bfloat16, (T, H), "x", device)
    u8 = torch.uint8
    if q is None:
        q = _new(stream, (rows, H), u8, x)
    else:
        _check(q, u8, (rows, H), "q", device)
    if s is None:
        s = _new(stream, (rows, H // 32), u8, x)
    else:
        _check(s, u8, (rows, H // 32), "s", device)
    if x.requires_grad and torch.is_grad_enabled():
        _experts._refuse_gradients(x=x)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((("x", x),))
    rc = lib.mxfp8_token_dispatch_mxfp8(x.data_ptr(), T, H, k, slot.data_ptr(), src.data_ptr(), rows, q.data_ptr(), s.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return q, s


def token_dispatch_grad(dxs, plan, *, out=None, stream=None):
    """The gradient of token_dispatch (see include/mxfp8_step.h): dxs bf16 [rows, H] -> out bf16 [T, H],
    the sum of each token's rows."""
    torch, lib, device, st = _begin(dxs, "dxs", stream)
    slot, src, T, k, rows = _plan(torch, plan, device)
    H = _columns(dxs)
    _check(dxs, torch.bfloat16, (rows, H), "dxs", device)
    if out is None:
        out = _new(stream, (T, H), torch.bfloat16, dxs)
    else:
        _check(out, torch.bfloat16, (T, H), "out", device)
    if (dxs.requires_grad or out.requires_grad) and torch.is_grad_enabled():
        _experts._refuse_gradients(dxs=dxs, out=out)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((("dxs", dxs), ("out", out)))
    rc = lib.mxfp8_token_dispatch_grad(dxs.data_ptr(), rows, T, H, k, slot.data_ptr(), out.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return out


def token_combine(y, weights, plan, *, out=None, stream=None):
    """Back to token order with the router's weights (see include/mxfp8_step.h): y bf16 [rows, H], weights fp32
    [T, top_k] -> out bf16 [T, H], the weighted sum of each token's rows."""
    torch, lib, device, st = _begin(y, "y", stream)
    slot, src, T, k, rows = _plan(torch, plan, device)
    H = _columns(y)
    _check(y, torch.bfloat16, (rows, H), "y", device)
    _check(weights, torch.float32, (T, k), "weights", device)
    if out is None:
        out = _new(stream, (T, H), torch.bfloat16, y)
    else:
        _check(out, torch.bfloat16, (T, H), "out", device)
    if (y.requires_grad or weights.requires_grad or out.requires_grad) and torch.is_grad_enabled():
        _experts._refuse_gradients(y=y, weights=weights, out=out)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((("y", y), ("weights", weights), ("out", out)))
    rc = lib.mxfp8_token_combine(y.data_ptr(), rows, weights.data_ptr(), T, H, k, slot.data_ptr(), out.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return out


def token_combine_grad(dout, y, weights, plan, *, dy=None, dweights=None, stream=None):
    """The gradients of token_combine (see include/mxfp8_step.h): dout bf16 [T, H], y bf16 [rows, H], weights fp32
    [T, top_k] -> (dy bf16 [rows, H], zeros on padding rows; dweights fp32 [T, top_k], 0 for absent pairs).
    dy may be y."""
    torch, lib, device, st = _begin(dout, "dout", stream)
    slot, src, T, k, rows = _plan(torch, plan, device)
    H = _columns(dout)
    bf16, f32 = torch.bfloat16, torch.float32
    _check(dout, bf16, (T, H), "dout", device)
    _check(y, bf16, (rows, H), "y", device)
    _check(weights, f32, (T, k), "weights", device)
    if dy is None:
        dy = torch.empty_like(y) if stream is None else _new(stream, (rows, H), bf16, dout)
    else:
        _check(dy, bf16, (rows, H), "dy", device)
    if dweights is None:
        dweights = torch.empty_like(weights) if stream is None else _new(stream, (T, k), f32, dout)
    else:
        _check(dweights, f32, (T, k), "dweights", device)
    if (dout.requires_grad or y.requires_grad or weights.requires_grad or dy.requires_grad or dweights.requires_grad) and torch.is_grad_enabled():
        _experts._refuse_gradients(dout=dout, y=y, weights=weights, dy=dy, dweights=dweights)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((("dout", dout), ("y", y), ("weights", weights), ("dy", dy), ("dweights", dweights)))
    rc = lib.mxfp8_token_combine_grad(dout.data_ptr(), y.data_ptr(), weights.data_ptr(), T, H, k, slot.data_ptr(), src.data_ptr(), rows,
                                      dy.data_ptr(), dweights.data_ptr(), st)
    if rc:
        _lib.check(rc)
    return dy, dweights


# ------------------------------------------------------------------ gradients

_PLAIN = None  # the tensor types whose attributes are the base class's


def _table(torch, tensors, device, name):
    """(pointers, sizes, types) of a list of tensors, as arrays."""
    kinds = set(map(type, tensors))
    T = torch.Tensor
    if kinds <= _PLAIN:  # the list may be long: by map over the base class's own attributes
        contiguous, where, address, numel, dtype = T.is_contiguous, T.get_device, T.data_ptr, T.numel, T.dtype.__get__
    else:
        for k in kinds:
            if not issubclass(k, T):
                raise TypeError(f"{name} must be torch.Tensors, got {k.__name__}")
        contiguous, where, address, numel = (methodcaller(m) for m in ("is_contiguous", "get_device", "data_ptr", "numel"))
        dtype = attrgetter("dtype")
    if not all(map(contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    if tensors and set(map(where, tensors)) != {device}:
        raise ValueError(f"{name} must all be on cuda:{device}")
    types = list(map(_TYPES.get, map(dtype, tensors)))
    if None in types:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {tensors[types.index(None)].dtype}")
    return array("Q", map(address, tensors)), array("q", map(numel, tensors)), array("i", types)


_TYPES = {}
_requires_grad = attrgetter("requires_grad")


def _grads(grads, stream, norm=None):
    torch = _experts._torch or _experts._torch_module()
    global _PLAIN
    if _PLAIN is None:
        _TYPES.update({torch.bfloat16: 0, torch.float32: 1})
        _PLAIN = {torch.Tensor, torch.nn.Parameter}
    if isinstance(grads, torch.Tensor):
        raise TypeError("grads must be a list of tensors")
    grads = list(grads)
    first = grads[0] if grads else norm
    if first is None:
        raise ValueError("grads is empty: there is no device to work on")
    device, st = _experts._device_and_stream(first, "grads", stream)
    return torch, _lib._lib or _lib.load(), grads, device, st


def _address(a):
    return a.buffer_info()[0]


def _workspace(torch, workspace, device, st):
    """Arguments from the workspace on, and the entry point's ending."""
    if workspace is None:
        return "", (st,)
    _check(workspace, torch.uint8, (workspace.numel(),), "workspace", device)
    return "_ws", (workspace.data_ptr(), workspace.numel(), st)


def grad_norm(grads, *, out=None, workspace=None, stream=None):
    """Global 2-norm of a list of gradients (see include/mxfp8_step.h): bf16 or fp32 tensors of any shapes.
    Returns (or fills) ``out``: fp32 [] on their device."""
    torch, lib, grads, device, st = _grads(grads, stream, out)
    ptrs, sizes, types = _table(torch, grads, device, "grads")
    if out is None:
        out = _new(stream, (), torch.float32, grads[0])
    else:
        _check(out, torch.float32, (), "out", device)
    if torch.is_grad_enabled() and any(map(_requires_grad, (*grads, out))):
        _experts._refuse_gradients(grads=next((t for t in grads if t.requires_grad), None), out=out)
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((*(("grads", t) for t in grads), ("out", out)))
    end, rest = _workspace(torch, workspace, device, st)
    rc = getattr(lib, "mxfp8_grad_norm" + end)(_address(ptrs), _address(sizes), _address(types), len(grads), out.data_ptr(), *rest)
    if rc:
        _lib.check(rc)
    return out


def clip_grads(grads, max_norm, *, norm=None, eps=1e-6, out=None, workspace=None, stream=None):
    """Gradients scaled so that their global norm is at most max_norm (see include/mxfp8_step.h): each becomes
    min(1, max_norm / (norm + eps)) times itself, in place or in the tensors of ``out`` (same shapes and dtypes).
    norm: fp32 [] on their device where the norm is known (over several ranks, say), else it is computed.
    Returns the norm before clipping.
    """
    torch, lib, grads, device, st = _grads(grads, stream, norm)
    ptrs, sizes, types = _table(torch, grads, device, "grads")
    outs = None
    if out is not None:
        out = list(out)
        if len(out) != len(grads):
            raise ValueError(f"out must hold {len(grads)} tensors, got {len(out)}")
        outs, _, out_types = _table(torch, out, device, "out")
        if out_types != types or any(o.shape != g.shape for o, g in zip(out, grads)):
            raise ValueError("out must have the shapes and dtypes of grads")
    if torch.is_grad_enabled() and any(map(_requires_grad, (*grads, *(out or ())))):
        _experts._refuse_gradients(grads=next((t for t in grads if t.requires_grad), None),
                                   out=next((t for t in out or () if t.requires_grad), None))
    if torch.autograd.forward_ad._current_level >= 0:
        _experts._refuse_tangents((*(("grads", t) for t in grads), *(("out", t) for t in out or ()), ("norm", norm)))
    known = None
    if norm is None:
        norm = _new(stream, (), torch.float32, grads[0])
    else:
        _check(norm, torch.float32, (), "norm", device)
        known = norm.data_ptr()
    end, rest = _workspace(torch, workspace, device, st)
    rc = getattr(lib, "mxfp8_clip_grads" + end)(_address(ptrs), _address(sizes), _address(types), len(grads), float(max_norm), float(eps), known,
                                                norm.data_ptr(), _address(outs) if outs is not None else None, *rest)
    if rc:
        _lib.check(rc)
    return norm


def grad_workspace_bytes(n: int) -> int:
    """Scratch of one grad_norm or clip_grads call on n tensors (0 if n is invalid)."""
    v = _sizes(n)
    return int(_lib.load().mxfp8_grad_workspace_bytes(*v)) if v else 0
