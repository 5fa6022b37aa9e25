"""The training operators that belong to no layer handle: the load-balance loss and its gradient,
8-bit activation checkpoints, the routing's slot gradients from a checkpoint, and the router's
linear backward.  As in layer.py, every step runs in the library's kernels; this module checks
the tensors, allocates the outputs and passes pointers.

Each call runs on the current stream of its tensors' device, or on the keyword `stream`.
"""
from __future__ import annotations

import functools

import torch

from . import _lib
from ._lib import BEAM_DTYPE_BF16, BEAM_DTYPE_F16, BEAM_DTYPE_F32, check

_DTYPES = {torch.float32: BEAM_DTYPE_F32, torch.bfloat16: BEAM_DTYPE_BF16}
_CKPT_DTYPES = {**_DTYPES, torch.float16: BEAM_DTYPE_F16}
CKPT_BLOCK = 32   # columns that share a scale
# (torch.empty is called with the sizes as separate arguments throughout: a tuple of them costs a
# microsecond more, and a small call launches in five.)


_raw_stream = torch._C._cuda_getCurrentRawStream


@functools.lru_cache(maxsize=1024)
def _balance_workspace(T: int, E: int, n_seq: int) -> int:
    return _lib.load().beam_balance_workspace(T, E, n_seq)


@functools.lru_cache(maxsize=1024)
def _weight_grad_workspace(T: int, d: int, C: int, device: int) -> int:
    return _lib.load().beam_router_weight_grad_workspace(T, d, C)


def _on_stream(fn):
    """Runs fn(first, ..., stream=None) with `stream` (or the current stream of the first
    argument's device) as the current stream: the outputs and the scratch are then allocated for
    the stream that uses them."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is not None:
            with torch.cuda.stream(stream):
                return fn(*args, **kw)
        first = args[0] if args else next(iter(kw.values()))
        index = (first["q"] if isinstance(first, dict) else first).get_device()   # -1 on the host
        if index >= 0 and index != torch._C._cuda_getDevice():
            with torch.cuda.device(index):
                return fn(*args, **kw)
        return fn(*args, **kw)
    return call


def _stream(device: torch.device) -> int:
    """The handle of the device's current stream (the raw query: torch.cuda.current_stream()
    builds a Stream object, 3 us of a call that launches in 5)."""
    return _raw_stream(device.index)


def _matrix(name: str, t: torch.Tensor, dtypes: dict, device=None):
    """(type, rows, cols, row stride) of a 2-dimensional CUDA tensor with contiguous rows."""
    dt = dtypes.get(t.dtype)
    if dt is None or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-dimensional CUDA tensor of dtype "
                         f"{' or '.join(str(d) for d in dtypes)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    rows, cols = t.shape
    ld, inner = t.stride()
    if rows <= 1:
        ld = cols
    if (inner != 1 and cols > 1) or ld < cols:
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    return dt, rows, cols, ld


def _array(name: str, t: torch.Tensor, dtype, shape, device) -> int:
    """A contiguous CUDA tensor of the given type, shape and device; returns its address."""
    if t.dtype != dtype or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return t.data_ptr()


def _groups(T, dev, topk_id, valid, cu_seqlens):
    if topk_id.dim() != 2 or topk_id.shape[0] != T:
        raise ValueError("topk_id must have the shape [T][K]")
    K = topk_id.shape[1]
    ids = _array("topk_id", topk_id, torch.int32, (T, K), dev)
    v = None if valid is None else _array("valid", valid, torch.uint8, (T,), dev)
    if cu_seqlens is None:
        return K, ids, v, None, 0
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 2:
        raise ValueError("cu_seqlens must hold the sequences' bounds: n_seq + 1 values")
    n = cu_seqlens.shape[0] - 1
    return K, ids, v, _array("cu_seqlens", cu_seqlens, torch.int32, (n + 1,), dev), n


@_on_stream
def balance_loss(logits: torch.Tensor, topk_id: torch.Tensor, valid: torch.Tensor | None = None,
                 cu_seqlens: torch.Tensor | None = None) -> dict:
    """The load-balance loss of router logits [T][E] (float32 or bfloat16; rows may be strided)
    and their Top-K assignments topk_id [T][K] int32, over the whole batch or per packed sequence
    (cu_seqlens [n_seq + 1] int32), leaving out the tokens with valid [T] uint8 = 0.  Returns
    loss (a float32 scalar tensor), counts [G][E] int32 (slots per expert), prob [G][E] float32
    (mean router probabilities) and tokens [G] int32.  See beam_balance_forward."""
    dt, T, E, ld = _matrix("logits", logits, _DTYPES)
    dev = logits.device
    K, ids, v, cu, n = _groups(T, dev, topk_id, valid, cu_seqlens)
    lib = _lib.load()
    G = max(1, n)
    size = _balance_workspace(T, E, n)
    loss = torch.empty((), dtype=torch.float32, device=dev)
    prob = torch.empty(G, E, dtype=torch.float32, device=dev)
    counts = torch.empty(G, E, dtype=torch.int32, device=dev)
    tokens = torch.empty(G, dtype=torch.int32, device=dev)
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    check(lib.beam_balance_forward(logits.data_ptr(), dt, T, E, ld, ids, K, v, cu, n,
                                   loss.data_ptr(), prob.data_ptr(), counts.data_ptr(),
                                   tokens.data_ptr(), None if ws is None else ws.data_ptr(), size,
                                   _stream(dev)))
    return dict(loss=loss, counts=counts, prob=prob, tokens=tokens)


@_on_stream
def balance_loss_backward(logits: torch.Tensor, topk_id: torch.Tensor, balance: dict,
                          scale: float = 1.0, valid: torch.Tensor | None = None,
                          cu_seqlens: torch.Tensor | None = None,
                          d_gate_logit: torch.Tensor | None = None,
                          d_mask_logit: torch.Tensor | None = None) -> torch.Tensor:
    """scale * dL_bal/dlogits [T][E] float32 for balance_loss's inputs and its result `balance`
    (counts and tokens are read).  With the routing's slot gradients d_gate_logit and
    d_mask_logit [T][K] float32 the result is the whole gradient of x [W_r | W_m], [T][2E]: the
    gate gradients added at topk_id, the mask gradients in the last E columns.  See
    beam_balance_backward."""
    dt, T, E, ld = _matrix("logits", logits, _DTYPES)
    dev = logits.device
    K, ids, v, cu, n = _groups(T, dev, topk_id, valid, cu_seqlens)
    G = max(1, n)
    counts = _array("balance['counts']", balance["counts"], torch.int32, (G, E), dev)
    tokens = _array("balance['tokens']", balance["tokens"], torch.int32, (G,), dev)
    if (d_gate_logit is None) != (d_mask_logit is None):
        raise ValueError("d_gate_logit and d_mask_logit come together")
    gr = gl = None
    if d_gate_logit is not None:
        gr = _array("d_gate_logit", d_gate_logit, torch.float32, (T, K), dev)
        gl = _array("d_mask_logit", d_mask_logit, torch.float32, (T, K), dev)
    out = torch.empty(T, E if gr is None else 2 * E, dtype=torch.float32, device=dev)
    check(_lib.load().beam_balance_backward(logits.data_ptr(), dt, T, E, ld, ids, K, v, cu,
                                            n, counts, tokens, scale, gr, gl, out.data_ptr(), _stream(dev)))
    return out


@_on_stream
def checkpoint_save(x: torch.Tensor) -> dict:
    """x [rows][d] (float32, bfloat16 or float16; rows may be strided) in 8 bits per value: a
    dict of q [rows][d rounded up to 32] int8, scale [rows][ceil(d / 32)] uint8 and d.  A block of
    32 columns shares a power-of-two scale: values are kept to within 1/127 of the block's largest.
    Rows may be taken out of q and scale by indexing both alike.  See beam_checkpoint_save."""
    dt, n, d, ld = _matrix("x", x, _CKPT_DTYPES)
    dev, nb = x.device, -(-d // CKPT_BLOCK)
    q = torch.empty(n, nb * CKPT_BLOCK, dtype=torch.int8, device=dev)
    scale = torch.empty(n, nb, dtype=torch.uint8, device=dev)
    check(_lib.load().beam_checkpoint_save(x.data_ptr(), dt, n, d, ld, q.data_ptr(),
                                           scale.data_ptr(), _stream(dev)))
    return dict(q=q, scale=scale, d=d)


def _checkpoint(ckpt: dict):
    """(q, scale, rows, d) of a checkpoint, checked."""
    q, scale, d = ckpt["q"], ckpt["scale"], int(ckpt["d"])
    n, nb = q.shape[0], -(-d // CKPT_BLOCK)
    if not q.is_cuda or d < 1:
        raise ValueError("a checkpoint holds CUDA tensors q and scale and a width d >= 1")
    return (_array("checkpoint q", q, torch.int8, (n, nb * CKPT_BLOCK), q.device),
            _array("checkpoint scale", scale, torch.uint8, (n, nb), q.device), n, d)


@_on_stream
def checkpoint_load(ckpt: dict, dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """The values of a checkpoint, [rows][d] float32, bfloat16 (both exact) or float16."""
    dt = _CKPT_DTYPES.get(dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {dtype}")
    q, scale, n, d = _checkpoint(ckpt)
    dev = ckpt["q"].device
    y = torch.empty(n, d, dtype=dtype, device=dev)
    check(_lib.load().beam_checkpoint_load(q, scale, n, d, y.data_ptr(), dt, _stream(dev)))
    return y


@_on_stream
def checkpoint_route_grad(ckpt: dict, gate: torch.Tensor, mask_logit: torch.Tensor, dy: torch.Tensor,
                          reg_scale: float = 0.0, segment_len: int = 0) -> dict:
    """The routing's slot gradients from a checkpoint of the expert outputs (row t K + k = token
    t's slot k): dghat, d_gate_logit and d_mask_logit [T][K] float32 for gate and mask_logit
    [T][K] float32, the upstream gradient dy [T][d] (float32 or bfloat16; rows may be strided),
    reg_scale = dL/dL_reg and the layer's segment_len.  See beam_checkpoint_route_grad."""
    q, scale, n, d = _checkpoint(ckpt)
    dev = ckpt["q"].device
    if gate.dim() != 2:
        raise ValueError("gate must have the shape [T][K]")
    T, K = gate.shape
    g = _array("gate", gate, torch.float32, (T, K), dev)
    l = _array("mask_logit", mask_logit, torch.float32, (T, K), dev)
    dt, rows, cols, ld = _matrix("dy", dy, _DTYPES, dev)
    if rows != T or cols != d or n != T * K:
        raise ValueError(f"dy must be [T][d] and the checkpoint hold T*K rows: got dy {tuple(dy.shape)}, "
                         f"{n} rows of {d} values, gate {(T, K)}")
    out = [torch.empty(T, K, dtype=torch.float32, device=dev) for _ in range(3)]
    check(_lib.load().beam_checkpoint_route_grad(q, scale, T, K, d, g, l, dy.data_ptr(), dt, ld,
                                                 segment_len, reg_scale, out[0].data_ptr(),
                                                 out[1].data_ptr(), out[2].data_ptr(), _stream(dev)))
    return dict(dghat=out[0], d_gate_logit=out[1], d_mask_logit=out[2])


@_on_stream
def router_weight_grad(ckpt: dict, dlogits: torch.Tensor, parts: int = 1) -> torch.Tensor:
    """dW [d][C] float32 = x^T dlogits of a router logits = x W, with x [T][d] from a checkpoint
    and dlogits [T][C] float32 or bfloat16 (rows may be strided).  parts > 1 gives
    [parts][d][C / parts] (2: W_r and W_m; L: a mask generator's layers)."""
    q, scale, n, d = _checkpoint(ckpt)
    dev = ckpt["q"].device
    dt, T, C, ld = _matrix("dlogits", dlogits, _DTYPES, dev)
    if T != n:
        raise ValueError(f"dlogits has {T} rows, the checkpoint {n}")
    if parts < 1 or C % parts:
        raise ValueError(f"parts={parts} must divide the {C} columns of dlogits")
    f32 = dict(dtype=torch.float32, device=dev)
    dw = torch.empty(d, C, **f32) if parts == 1 else torch.empty(parts, d, C // parts, **f32)
    lib = _lib.load()
    size = _weight_grad_workspace(T, d, C, dev.index)   # the split depends on the device's SMs
    ws = torch.empty(size, dtype=torch.uint8, device=dev) if size > 0 else None
    check(lib.beam_router_weight_grad(q, scale, T, d, dlogits.data_ptr(), dt, ld, C, parts, dw.data_ptr(),
                                      None if ws is None else ws.data_ptr(), size, _stream(dev)))
    return dw


@_on_stream
def router_input_grad(dlogits: torch.Tensor, w: torch.Tensor) -> torch.Tensor:
    """dx [T][d] float32 = dlogits W^T of a router logits = x W, for dlogits [T][C] and w [d][C]
    (each float32 or bfloat16; rows may be strided)."""
    dt, T, C, ld = _matrix("dlogits", dlogits, _DTYPES)
    dev = dlogits.device
    wt, d, cols, lw = _matrix("w", w, _DTYPES, dev)
    if cols != C:
        raise ValueError(f"w must have dlogits' {C} columns")
    dx = torch.empty(T, d, dtype=torch.float32, device=dev)
    check(_lib.load().beam_router_input_grad(dlogits.data_ptr(), dt, ld, T, C, w.data_ptr(),
                                             wt, lw, d, dx.data_ptr(), d, _stream(dev)))
    return dx
