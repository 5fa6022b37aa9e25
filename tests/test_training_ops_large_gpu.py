"""The training operators at sizes where their kernels' loops turn: more tiles than CTA pairs (a second unit of
the persistent linear backward, a second resident operand, several drains of an accumulator per tile) and
several passes of a CTA over its run of tokens (balance loss and gradient), with ragged ends.

The 64-bit results are formed here with torch in float64 on the GPU.  u = 2^-24.  A sum of n products is within
(n + 64) u of the sum of the magnitudes (a float32 sum in any order; the tensor cores' additions truncate, 2 u
each, but over at most 256 terms before a rounded sum, and small terms have an accumulator of their own).
"""
import ctypes

import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def beam():
    import dynamic_expert_routing_b200 as b
    return b


def rnd(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), dtype=torch.float32, device="cuda")


def wide(t, dtype, ld):
    """The values in `dtype` as rows cut out of a tensor that is ld columns wider."""
    return torch.nn.functional.pad(t.to(DT[dtype]), (0, ld))[:, :t.shape[1]]


def close(got, a, b, n):
    """got = a b (float64 factors) within the rounding of a sum of n products."""
    want = a @ b
    assert bool(((got.double() - want).abs() <= (n + 64) * U * (a.abs() @ b.abs()) + 1e-35).all())


# 74 pairs of CTAs on the device; tiles are 256 x 128
INPUT = [
    # one k step, 5 tiles of n walked with A resident, 79 > 74 units: some pairs convert a second A
    (20000, 640, 64, "f32", "f32", 0), (20000, 640, 64, "f32", "bf16", 0), (20000, 640, 64, "bf16", "bf16", 0),
    # the same with odd rows and two k steps, the second ragged
    (20001, 700, 67, "f32", "f32", 3), (19901, 389, 67, "bf16", "f32", 1), (20001, 650, 120, "f32", "bf16", 8),
    # three (f32 x bf16) and seven (bf16) resident steps
    (19009, 400, 190, "f32", "bf16", 2), (21000, 1000, 424, "bf16", "bf16", 0),
    # too long to be resident: the ring carries both, several drains per tile, several tiles per pair
    (6000, 1536, 424, "f32", "bf16", 0), (6001, 1537, 425, "f32", "f32", 0), (5003, 2000, 700, "bf16", "bf16", 4),
]


@pytest.mark.parametrize("T,D,C,dtype,wdtype,ld", INPUT)
def test_input_grad_over_many_units(T, D, C, dtype, wdtype, ld):
    b = beam()
    g, w = wide(rnd(1, T, C), dtype, ld), wide(rnd(2, D, C), wdtype, ld)
    dx = b.router_input_grad(g, w)
    close(dx, g.double(), w.double().t(), C)
    assert torch.equal(b.router_input_grad(g, w), dx)


@pytest.mark.parametrize("storage", ["fp32", "bf16"])
def test_layer_input_grad_over_many_units(storage):
    """W in a layer's own order (its rows the logits), A resident and walked over 4 tiles of n."""
    spec = synth.LayerSpec("small", 512, 30, 4, 256, storage=storage)
    w = {k: v.cuda().contiguous() for k, v in synth.make_layer(spec, seed=0).items() if isinstance(v, torch.Tensor)}
    layer = beam().BeamMoE(w, spec.top_k, max_tokens=64)
    T, C, D = 20003, 60, 512
    g, dx = rnd(1, T, C), torch.empty((T, D), device="cuda")
    assert beam().load().beam_moe_router_input_grad(layer._h, ctypes.c_void_p(g.data_ptr()), C, T, ctypes.c_void_p(dx.data_ptr()),
                                                    D, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    wm = torch.cat([w["w_router"], w["w_mask"]], 1).double()
    close(dx, g.double(), wm.t(), C)


WEIGHT = [
    # 96 tiles on 74 pairs, 11 k steps: a second tile, three drains each
    (700, 4096, 700, 0), (701, 4001, 701, 3),
    # 24 tiles, k in 3 slices of up to 43 steps
    (8192, 1536, 424, 0), (4500, 1530, 421, 1),
    # tiles of 64 columns: 16 tiles in 4 slices; 79 tiles, unsliced
    (8192, 4096, 16, 0), (700, 20000, 50, 2),
    # one tile in 65 slices, the last step ragged
    (16390, 100, 100, 8),
]


@pytest.mark.parametrize("T,D,C,ld", WEIGHT)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weight_grad_over_many_units(T, D, C, ld, dtype):
    b = beam()
    c = b.checkpoint_save(rnd(1, T, D))
    x, g = b.checkpoint_load(c).double(), wide(rnd(2, T, C), dtype, ld)
    dw = b.router_weight_grad(c, g)
    close(dw, x.t(), g.double(), T)
    assert torch.equal(b.router_weight_grad(c, g), dw)


# ------------------------------------------------------------------------------ balance loss
def members(T, cu, valid):
    """[G][T] float64: 1 where the token counts in the group."""
    cu = [0, T] if cu is None else cu.tolist()
    m = torch.zeros((len(cu) - 1, T), dtype=torch.float64, device="cuda")
    for i in range(len(cu) - 1):
        m[i, cu[i]:cu[i + 1]] = 1
    return m if valid is None else m * (valid != 0)


BALANCE = [
    # rows of 32 lanes: 3 passes of the loss, 2 of the gradient, a ragged end
    (6001, 256, 8, "f32", 0, None), (6001, 256, 32, "bf16", 9, 0.7), (9007, 212, 16, "f32", 5, 0.9),
    # 8 lanes: 5 and 3 passes; sequences that start and end inside a run, some empty
    (40001, 60, 4, "f32", 0, 0.5), (40001, 60, 4, "bf16", 37, 0.8), (40001, 60, 4, "f32", 300, None),
    # a lane per row: 2 passes and 1; 2 and 16 lanes
    (100003, 8, 2, "f32", 6, 0.9), (200001, 8, 2, "bf16", 0, None), (70001, 16, 6, "f32", 11, 0.6), (30011, 120, 5, "bf16", 20, 0.8),
]


@pytest.mark.parametrize("T,E,K,dtype,seqs,keep", BALANCE)
def test_balance_over_many_passes(T, E, K, dtype, seqs, keep):
    b = beam()
    logits = wide(2 * rnd(1, T, E), dtype, 0 if E % 8 else 4)
    ids = torch.topk(logits.float(), K, dim=1).indices.int()
    valid = None if keep is None else (torch.rand(T, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda") < keep).to(torch.uint8)
    cu = None
    if seqs:
        cu = torch.sort(torch.randint(3, T - 5, (seqs + 1,), generator=torch.Generator(device="cuda").manual_seed(3),
                                      device="cuda")).values.int()
        cu[1] = cu[0]                                       # an empty one
    out = b.balance_loss(logits, ids, valid=valid, cu_seqlens=cu)
    inside = members(T, cu, valid)
    n = inside.sum(1)
    x = logits.double()
    p = torch.softmax(x, 1)
    chosen = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_add_(1, ids.long(), torch.ones_like(ids, dtype=torch.float64))
    counts = inside @ chosen
    per = torch.where(n > 0, 1 / n.clamp(min=1), 0.0)[:, None]
    prob, f, act = (inside @ p) * per, counts * per * (E / K), int((n > 0).sum())
    assert torch.equal(out["counts"].double(), counts) and torch.equal(out["tokens"].double(), n)
    R = float((x.amax(1) - x.amin(1)).max())
    tol = (R + 20 + T / 64 + 64) * U                        # a softmax's roundings and the additions in a row
    assert bool(((out["prob"].double() - prob).abs() <= tol * prob + 1e-30).all())
    loss = float((f * prob).sum() / act)
    assert abs(float(out["loss"]) - loss) <= (tol + (E + 64) * U) * loss
    # the gradient: p (f - sum f p), the bracket of the size of the group's largest |f - 1|
    scale, gr, gl = 0.7, rnd(5, T, K), rnd(6, T, K)
    ft, w = inside.t() @ f, (inside * per * (scale / act)).sum(0)[:, None]
    d = w * p * (ft - (ft * p).sum(1, keepdim=True))
    size = inside.t() @ ((f - 1).abs().amax(1, keepdim=True) + 1e-6)
    bound = w * p * size * 2 * (R + 20 + 16) * U
    got = b.balance_loss_backward(logits, ids, out, scale=scale, valid=valid, cu_seqlens=cu)
    assert bool(((got.double() - d).abs() <= bound + 1e-37).all())
    full = torch.cat([d, torch.zeros_like(d)], 1)
    full.scatter_add_(1, ids.long(), gr.double()).scatter_add_(1, ids.long() + E, gl.double())
    got = b.balance_loss_backward(logits, ids, out, scale=scale, valid=valid, cu_seqlens=cu, d_gate_logit=gr, d_mask_logit=gl)
    bound = torch.nn.functional.pad(bound, (0, E)) + 2 * U * full.abs()
    assert bool(((got.double() - full).abs() <= bound + 1e-37).all())


# ------------------------------------------------------------------------------ checkpoints and slots
@pytest.mark.parametrize("N,D,dtype", [(9001, 4100, "f32"), (30001, 333, "bf16"), (200003, 40, "f32")])
def test_checkpoint_over_many_blocks(N, D, dtype):
    """Many CTAs, odd widths: each value within half a step of its block of 32, steps the smallest that fit."""
    b = beam()
    x = wide(rnd(1, N, D), dtype, 5)
    c = b.checkpoint_save(x)
    y = b.checkpoint_load(c).double()
    nb = c["scale"].shape[1]
    a = torch.nn.functional.pad(x.double(), (0, nb * 32 - D)).view(N, nb, 32).abs().amax(2)
    step = torch.exp2(c["scale"].double() - 127)
    assert bool((a <= 127 * step).all()) and bool((a > 127 * step / 2).all())
    assert bool(((y - x.double()).abs() <= step.repeat_interleave(32, 1)[:, :D] / 2).all())
    assert not c["q"][:, D:].any()


@pytest.mark.parametrize("T,K,D,seg,dtype", [(20001, 4, 1030, 0, "f32"), (30000, 2, 513, 0, "bf16"), (9000, 20, 300, 7, "bf16")])
def test_route_grad_over_many_tokens(T, K, D, seg, dtype):
    b = beam()
    S = max(1, seg)
    lead = torch.arange(T, device="cuda") // S * S
    gate, l = torch.softmax(rnd(2, T, K), 1)[lead].contiguous(), (6 * rnd(3, T, K))[lead].contiguous()
    dy = wide(rnd(4, T, D), dtype, 1)
    c = b.checkpoint_save(rnd(1, T * K, D))
    out = b.checkpoint_route_grad(c, gate, l, dy, reg_scale=0.5, segment_len=seg)
    y, dyd = b.checkpoint_load(c).double().view(T, K, D), dy.double()
    s = torch.einsum("tkd,td->tk", y, dyd)
    mag = torch.einsum("tkd,td->tk", y.abs(), dyd.abs())
    eps = (D + 64) * U
    assert bool(((out["dghat"].double() - s).abs() <= eps * mag).all())
    G = -(-T // S)
    of = torch.arange(T, device="cuda") // S
    run = torch.zeros((G, K), dtype=torch.float64, device="cuda").index_add_(0, of, s)
    rmag = torch.zeros((G, K), dtype=torch.float64, device="cuda").index_add_(0, of, mag)
    size = torch.bincount(of).double()[:, None]
    g, ls = gate[::S].double(), l[::S].double()
    slope = torch.sigmoid(ls) * torch.sigmoid(-ls)
    dm = (run * g + size * (0.5 / (T * K))) * slope
    dg = run * (ls >= 0)
    dr = g * (dg - (g * dg).sum(1, keepdim=True))
    err = (eps + (S + 16) * U) * rmag
    assert bool(((out["d_mask_logit"][::S].double() - dm).abs() <= err * slope + 16 * U * dm.abs() + 1e-30).all())
    assert bool(((out["d_gate_logit"][::S].double() - dr).abs() <= err + (err * g).sum(1, keepdim=True) +
                 (K + 16) * U * (rmag + rmag.sum(1, keepdim=True))).all())
    off = torch.arange(T, device="cuda") % S != 0
    assert not out["d_mask_logit"][off].any() and not out["d_gate_logit"][off].any()
