"""Operators on the expert weights (argument marshalling only; see
include/mxfp8_experts.h): the orthogonalised update of a stack of gradients
and the whole expert layer for a few tokens.

``stream``: the stream that runs the call (default: the current one). The inputs
have to be ready there, and an output that the call allocates belongs to it:
order its use on other streams as with any tensor of another stream. Neither
operator has a backward pass: tensors that require a gradient are refused while
gradients are being recorded."""
from __future__ import annotations

from operator import index

from . import _lib

_SCORES = {"softmax": 0, "sigmoid": 1}

_torch = None
_raw_stream = None  # device index -> handle of the current stream


def _torch_module():
    global _torch, _raw_stream
    if _torch is None:
        import torch

        # the public call builds a Stream object, several microseconds on a slow host
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _torch = torch
    return _torch


def _check(t, dtype, shape, name, device):
    """Raises unless t is a contiguous tensor of that dtype and shape on that CUDA device."""
    if not (isinstance(t, _torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous()):
        _lib._expect(t, dtype, name)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, x or grad on cuda:{device}")


def _refuse_gradients(**tensors):
    names = [name for name, t in tensors.items() if t is not None and t.requires_grad]
    raise ValueError(f"{', '.join(names)} requires a gradient, which this operator does not have: detach it or call under torch.no_grad()")


def _int32(v, name):
    """v as an int that the library's 32-bit arguments hold (ctypes would take it modulo 2^32)."""
    v = index(v)
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name}={v} is out of range")
    return v


def _sizes(*v):
    """Sizes as 32-bit integers; None where one does not fit."""
    v = [index(i) for i in v]
    return v if all(-0x80000000 <= i <= 0x7fffffff for i in v) else None


def _device_and_stream(t, name, stream):
    torch = _torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    device = t.get_device()
    if torch.cuda.current_device() != device or (stream is not None and stream.device_index != device):
        raise ValueError(f"{name} is on cuda:{device}: make it the current device, with a stream of that device")
    return device, _raw_stream(device) if stream is None else stream.cuda_stream


def moe_layer(x, router, w13, s13, w2, s2, top_k, *, bias=None, first_expert=0, score="softmax", renormalize=True,
              scale=1.0, out=None, topk_ids=None, topk_weights=None, workspace=None, stream=None):
    """A whole expert layer for a few tokens (see include/mxfp8_experts.h).

    x: bf16 [T, H], T <= 128; router: bf16 [experts, H]; w13: uint8 [local, 2 I, H]
    (E4M3, gate rows then up rows), s13: uint8 [local, 2 I, H/32] (E8M0); w2: uint8
    [local, H, I], s2: uint8 [local, H, I/32]; bias: fp32 [experts] or None, added to
    the score for the choice only. The experts held here are first_expert ..
    first_expert + local. score: "softmax" or "sigmoid". Returns (or fills) ``out``:
    bf16 [T, H]; topk_ids (int32 [T, top_k]) and topk_weights (fp32 [T, top_k]) are
    filled when given.
    """
    torch = _torch or _torch_module()
    device, st = _device_and_stream(x, "x", stream)
    if not (type(top_k) is int and type(first_expert) is int and 0 <= top_k < 1024 > first_expert >= 0):  # (the checks' cost counts at one token)
        top_k, first_expert = _int32(top_k, "top_k"), _int32(first_expert, "first_expert")
    if x.dim() != 2 or w13.dim() != 3 or router.dim() != 2:
        raise ValueError("x must be [T, H], router [experts, H] and w13 [local, 2 I, H]")
    T, H = x.shape
    experts = router.shape[0]
    local, I2 = w13.shape[:2]
    I = I2 // 2
    u8, bf16, f32 = torch.uint8, torch.bfloat16, torch.float32
    _check(x, bf16, (T, H), "x", device)
    _check(router, bf16, (experts, H), "router", device)
    _check(w13, u8, (local, 2 * I, H), "w13", device)
    _check(s13, u8, (local, 2 * I, H // 32), "s13", device)
    _check(w2, u8, (local, H, I), "w2", device)
    _check(s2, u8, (local, H, I // 32), "s2", device)
    bias_p = ids_p = weights_p = None
    if bias is not None:
        _check(bias, f32, (experts,), "bias", device)
        bias_p = bias.data_ptr()
    if score not in _SCORES:
        raise ValueError(f"score must be one of {sorted(_SCORES)}, got {score!r}")
    if out is None:
        out = torch.empty_like(x) if stream is None else _lib._empty(stream, x.shape, bf16, x.device)
    else:
        _check(out, bf16, (T, H), "out", device)
    if topk_ids is not None:
        _check(topk_ids, torch.int32, (T, top_k), "topk_ids", device)
        ids_p = topk_ids.data_ptr()
    if topk_weights is not None:
        _check(topk_weights, f32, (T, top_k), "topk_weights", device)
        weights_p = topk_weights.data_ptr()
    if (x.requires_grad or router.requires_grad or out.requires_grad or (bias is not None and bias.requires_grad)
            or (topk_weights is not None and topk_weights.requires_grad)) and torch.is_grad_enabled():
        _refuse_gradients(x=x, router=router, bias=bias, out=out, topk_weights=topk_weights)
    lib = _lib._lib or _lib.load()
    args = (x.data_ptr(), T, router.data_ptr(), bias_p, w13.data_ptr(), s13.data_ptr(), w2.data_ptr(), s2.data_ptr(),
            experts, first_expert, local, H, I, top_k, _SCORES[score], 1 if renormalize else 0, scale, out.data_ptr(),
            ids_p, weights_p)
    if workspace is None:
        rc = lib.mxfp8_moe_layer(*args, st)
    else:
        _check(workspace, u8, (workspace.numel(),), "workspace", device)
        rc = lib.mxfp8_moe_layer_ws(*args, workspace.data_ptr(), workspace.numel(), st)
    if rc:
        _lib.check(rc)
    return out


def moe_layer_workspace_bytes(T: int, experts: int, local: int, H: int, I: int, top_k: int) -> int:
    """Scratch of one moe_layer call (0 if the sizes are invalid)."""
    v = _sizes(T, experts, local, H, I, top_k)
    return int(_lib.load().mxfp8_moe_layer_workspace_bytes(*v)) if v else 0


def muon_update(grad, momentum=None, *, mu=0.95, nesterov=True, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7,
                out=None, workspace=None, stream=None):
    """Orthogonalised update of a stack of gradients (see include/mxfp8_experts.h).

    grad: bf16 or fp32 [E, N, K] (or one matrix [N, K]), e.g. what wgrad_grouped
    returns; momentum: fp32 of the same shape, updated in place, or None. coeffs:
    (a, b, c) of one step X <- a X + (b A + c A A) X, A = X X^T; refused where the
    iteration can leave the range of the products' operands. Returns (or fills)
    ``out``: bf16, the shape of grad.
    """
    torch = _torch or _torch_module()
    device, st = _device_and_stream(grad, "grad", stream)
    if type(steps) is not int or not 0 <= steps < 1024:
        steps = _int32(steps, "steps")
    shape = grad.shape
    if len(shape) == 3:
        E, N, K = shape
    elif len(shape) == 2:
        E, (N, K) = 1, shape
    else:
        raise ValueError(f"grad must be [E, N, K] or [N, K], got {list(shape)}")
    dtype = grad.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise TypeError(f"grad must be torch.bfloat16 or torch.float32, got {dtype}")
    _check(grad, dtype, shape, "grad", device)
    momentum_p = None
    if momentum is not None:
        _check(momentum, torch.float32, shape, "momentum", device)
        momentum_p = momentum.data_ptr()
    if out is None:
        out = torch.empty_like(grad, dtype=torch.bfloat16) if stream is None else _lib._empty(stream, shape, torch.bfloat16, grad.device)
    else:
        _check(out, torch.bfloat16, shape, "out", device)
    if (grad.requires_grad or out.requires_grad or (momentum is not None and momentum.requires_grad)) and torch.is_grad_enabled():
        _refuse_gradients(grad=grad, momentum=momentum, out=out)
    a, b, c = coeffs
    lib = _lib._lib or _lib.load()
    args = (grad.data_ptr(), 0 if dtype is torch.bfloat16 else 1, momentum_p, E, N, K, mu, 1 if nesterov else 0, steps,
            a, b, c, eps, out.data_ptr())
    if workspace is None:
        rc = lib.mxfp8_muon_update(*args, st)
    else:
        _check(workspace, torch.uint8, (workspace.numel(),), "workspace", device)
        rc = lib.mxfp8_muon_update_ws(*args, workspace.data_ptr(), workspace.numel(), st)
    if rc:
        _lib.check(rc)
    return out


def muon_update_workspace_bytes(E: int, N: int, K: int) -> int:
    """Scratch of one muon_update call (0 if the sizes are invalid)."""
    v = _sizes(E, N, K)
    return int(_lib.load().mxfp8_muon_update_workspace_bytes(*v)) if v else 0
