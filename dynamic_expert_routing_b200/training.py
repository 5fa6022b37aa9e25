"""The training operators that belong to no layer handle: the load-balance loss and its gradient,
8-bit activation checkpoints, the routing's slot gradients from a checkpoint, and the router's
linear backward.  Every step runs in the library's kernels; the native module _training
(csrc/binding.cpp) checks the tensors, allocates the outputs and calls the library.

Each call runs on the current stream of its tensors' device, or on `stream` of that device, for which its
outputs and scratch are then allocated; the tensors of a returned dict share one allocation (a loss over
packed sequences has its own).
Tensors that a call cannot take raise ValueError (TypeError where a tensor is expected and
something else given), a refusal by the library BeamError.
"""
from __future__ import annotations

import os

import torch

from . import _lib

CKPT_BLOCK = 32   # columns that share a scale
BINDING_PATH = os.path.join(_lib.HERE, "_training.so")

_ops = None


def _native():
    """The native module, bound to the loaded library; there is no fallback."""
    global _ops
    lib = _lib.load()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"{BINDING_PATH} is missing: build it with "
                           "`python -m dynamic_expert_routing_b200.build`")
    from . import _training
    _training.bind(lib._name, _lib.check)
    _ops = _training
    return _ops


def on_stream(stream, tensor):
    """The context in which a call on `tensor` runs on `stream`, a stream of the tensor's device."""
    if isinstance(tensor, torch.Tensor) and tensor.device != stream.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {tensor.device}")
    return torch.cuda.stream(stream)


def _run(name: str, stream, *args):
    first = args[0]
    with on_stream(stream, first.get("q") if isinstance(first, dict) else first):
        return getattr(_ops or _native(), name)(*args)


def balance_loss(logits: torch.Tensor, topk_id: torch.Tensor, valid: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None, stream=None) -> dict:
    """The load-balance loss of router logits [T][E] (float32 or bfloat16; rows may be strided)
    and their Top-K assignments topk_id [T][K] int32, over the whole batch or per packed sequence
    (cu_seqlens [n_seq + 1] int32), leaving out the tokens with valid [T] (uint8 or bool) = 0.  Returns
    loss (a float32 scalar tensor), counts [G][E] int32 (slots per expert), prob [G][E] float32
    (mean router probabilities) and tokens [G] int32.  See beam_balance_forward."""
    if stream is not None:
        return _run("balance_loss", stream, logits, topk_id, valid, cu_seqlens)
    return (_ops or _native()).balance_loss(logits, topk_id, valid, cu_seqlens)


def balance_loss_backward(logits: torch.Tensor, topk_id: torch.Tensor, balance: dict,
                          scale: float = 1.0, valid: torch.Tensor | None = None,
                          cu_seqlens: torch.Tensor | None = None,
                          d_gate_logit: torch.Tensor | None = None,
                          d_mask_logit: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """scale * dL_bal/dlogits [T][E] float32 for balance_loss's inputs and its result `balance`
    (counts and tokens are read).  With the routing's slot gradients d_gate_logit and
    d_mask_logit [T][K] float32 the result is the whole gradient of x [W_r | W_m], [T][2E]: the
    gate gradients added at topk_id, the mask gradients in the last E columns.  See
    beam_balance_backward."""
    args = (logits, topk_id, balance, scale, valid, cu_seqlens, d_gate_logit, d_mask_logit)
    if stream is not None:
        return _run("balance_loss_backward", stream, *args)
    return (_ops or _native()).balance_loss_backward(*args)


def checkpoint_save(x: torch.Tensor, stream=None) -> dict:
    """x [rows][d] (float32, bfloat16 or float16; rows may be strided) in 8 bits per value: a
    dict of q [rows][d rounded up to 32] int8, scale [rows][ceil(d / 32)] uint8 and d.  A block of
    32 columns shares a power-of-two scale: values are kept to within 1/127 of the block's largest.
    Rows may be taken out of q and scale by indexing both alike.  See beam_checkpoint_save."""
    if stream is not None:
        return _run("checkpoint_save", stream, x)
    return (_ops or _native()).checkpoint_save(x)


def checkpoint_load(ckpt: dict, dtype: torch.dtype = torch.float32, stream=None) -> torch.Tensor:
    """The values of a checkpoint, [rows][d] float32, bfloat16 (both exact) or float16."""
    if not isinstance(dtype, torch.dtype):
        raise TypeError(f"dtype must be a torch.dtype, got {dtype!r}")
    if stream is not None:
        return _run("checkpoint_load", stream, ckpt, dtype)
    return (_ops or _native()).checkpoint_load(ckpt, dtype)


def checkpoint_route_grad(ckpt: dict, gate: torch.Tensor, mask_logit: torch.Tensor, dy: torch.Tensor,
                          reg_scale: float = 0.0, segment_len: int = 0, stream=None) -> dict:
    """The routing's slot gradients from a checkpoint of the expert outputs (row t K + k = token
    t's slot k): dghat, d_gate_logit and d_mask_logit [T][K] float32 for gate and mask_logit
    [T][K] float32, the upstream gradient dy [T][d] (float32 or bfloat16; rows may be strided),
    reg_scale = dL/dL_reg and the layer's segment_len.  See beam_checkpoint_route_grad."""
    args = (ckpt, gate, mask_logit, dy, reg_scale, segment_len)
    if stream is not None:
        return _run("checkpoint_route_grad", stream, *args)
    return (_ops or _native()).checkpoint_route_grad(*args)


def router_weight_grad(ckpt: dict, dlogits: torch.Tensor, parts: int = 1, stream=None) -> torch.Tensor:
    """dW [d][C] float32 = x^T dlogits of a router logits = x W, with x [T][d] from a checkpoint
    and dlogits [T][C] float32 or bfloat16 (rows may be strided).  parts > 1 gives
    [parts][d][C / parts] (2: W_r and W_m; L: a mask generator's layers)."""
    if stream is not None:
        return _run("router_weight_grad", stream, ckpt, dlogits, parts)
    return (_ops or _native()).router_weight_grad(ckpt, dlogits, parts)


def router_input_grad(dlogits: torch.Tensor, w: torch.Tensor, stream=None) -> torch.Tensor:
    """dx [T][d] float32 = dlogits W^T of a router logits = x W, for dlogits [T][C] and w [d][C]
    (each float32 or bfloat16; rows may be strided)."""
    if stream is not None:
        return _run("router_input_grad", stream, dlogits, w)
    return (_ops or _native()).router_input_grad(dlogits, w)
