"""The training operators on the GPU against the float64 oracle (oracle/training.py).

Tolerances count roundings, u = 2^-24 being half a float32 step relative to the value:
  * the checkpoint format is exact (power-of-two scales): equal bytes;
  * a softmax probability: x - m is rounded (u |x - m| in the exponent), exp is within 2 steps
    (4 u), the sum of E positive terms has at most log2(32) + E/32 <= 13 rounded additions, and
    the reciprocal and the product round once each: (R + 20) u relative for a logit range R;
  * sums of positive terms over T tokens: at most T/64 + 64 additions in a row, one u each;
  * dot products and matrix products of n terms: (n + 64) u times the sum of the magnitudes
    (the float32 sum in any order; the tensor cores' additions truncate, 2 u each, but run over
    at most 128 terms before a rounded sum).
"""
import numpy as np
import pytest
import torch

from oracle import training as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def beam():
    import dynamic_expert_routing_b200 as b
    return b


def rnd(seed, *shape, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32) * scale


def np64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------------------ balance loss
def bal_case(T, E, K, dtype, seqs, valid, ld=0, seed=0, spread=1.0):
    logits = rnd(seed, T, E + ld, scale=spread).to(DT[dtype])
    topk = torch.topk(logits[:, :E].float(), K, dim=1).indices.to(torch.int32)
    cu = None
    if seqs is not None:
        cu = torch.tensor(seqs, dtype=torch.int32)
    v = None
    if valid is not None:
        v = (torch.rand(T, generator=torch.Generator().manual_seed(seed + 1)) < valid).to(torch.uint8)
    return logits, topk, cu, v


def dev(t):
    return None if t is None else t.cuda()


BAL = [
    (1, 8, 2, "f32", None, None), (1, 1, 1, "f32", None, None), (64, 8, 2, "bf16", None, None),
    (63, 2, 1, "f32", None, 0.5), (65, 33, 5, "bf16", [0, 1, 1, 64, 65], None),
    (323, 64, 6, "f32", [0, 5, 5, 70, 130, 300], 0.7), (1000, 212, 16, "bf16", None, 0.9),
    (777, 256, 32, "f32", [0, 777], None), (5000, 60, 4, "bf16", [0, 64, 128, 4097, 4990], 0.3),
    (40, 20, 3, "f32", [0, 0, 0, 0], None), (200, 96, 8, "f32", None, 0.0),
    (130, 255, 7, "f32", [7, 20, 90], None),
]


@pytest.mark.parametrize("T,E,K,dtype,seqs,valid", BAL)
@pytest.mark.parametrize("ld", [0, 5])
def test_balance_loss_and_gradient(T, E, K, dtype, seqs, valid, ld):
    b = beam()
    logits, topk, cu, v = bal_case(T, E, K, dtype, seqs, valid, ld)
    dl = logits.cuda()[:, :E]
    x = np64(logits)[:, :E]
    out = b.balance_loss(dl, topk.cuda(), valid=dev(v), cu_seqlens=dev(cu))
    r = ref.balance(x, topk.numpy(), E, K, seqs, None if v is None else v.numpy())
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), r["counts"])
    np.testing.assert_array_equal(out["tokens"].cpu().numpy(), r["tokens"])
    R = float(np.ptp(x, axis=1).max())
    tol = (R + 20 + T / 64 + 64) * U
    np.testing.assert_allclose(np64(out["prob"]), r["prob"], rtol=tol, atol=1e-30)
    assert abs(float(out["loss"]) - r["loss"]) <= (tol + (E + 64) * U) * r["loss"] + 1e-30
    # gradient: p (f - sum f p); the bracket's terms are of the size of max |f - 1| + 1
    scale = 0.37
    d = b.balance_loss_backward(dl, topk.cuda(), out, scale=scale, valid=dev(v), cu_seqlens=dev(cu))
    dr = ref.balance_grad(x, topk.numpy(), E, K, scale, seqs, None if v is None else v.numpy())
    gs = ref.groups(T, seqs, None if v is None else v.numpy())
    act = sum(1 for g in gs if g)
    bound = np.zeros((T, E))
    for i, g in enumerate(gs):
        if g:
            f = np.abs(r["counts"][i] * E / (K * len(g)) - 1).max() + 1e-6
            bound[g] = scale / (act * len(g)) * ref.softmax(x[g]) * f * 2 * (R + 20 + 16) * U
    assert (np.abs(np64(d) - dr) <= bound + 1e-37).all()
    # joined with slot gradients
    gr, gl = rnd(5, T, K), rnd(6, T, K)
    full = b.balance_loss_backward(dl, topk.cuda(), out, scale=scale, valid=dev(v), cu_seqlens=dev(cu),
                                   d_gate_logit=gr.cuda(), d_mask_logit=gl.cuda())
    want = np.zeros((T, 2 * E))
    want[:, :E] = dr
    for t in range(T):
        for k in range(K):
            want[t, topk[t, k]] += float(gr[t, k])
            want[t, E + topk[t, k]] += float(gl[t, k])
    assert full.shape == (T, 2 * E)
    assert (np.abs(np64(full) - want) <= np.pad(bound, ((0, 0), (0, E))) + 2 * U * np.abs(want) + 1e-37).all()


def test_balance_many_sequences():
    """More sequences than the reduction has threads, most of a single token, some empty."""
    b = beam()
    T, E, K = 3000, 24, 3
    logits, topk, _, _ = bal_case(T, E, K, "f32", None, None, seed=9)
    cu = sorted(int(i) for i in np.random.RandomState(0).randint(0, T + 1, 1400))
    out = b.balance_loss(logits.cuda(), topk.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    r = ref.balance(np64(logits), topk.numpy(), E, K, cu)
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), r["counts"])
    np.testing.assert_allclose(np64(out["prob"]), r["prob"], rtol=150 * U, atol=1e-30)
    assert abs(float(out["loss"]) - r["loss"]) <= 250 * U * r["loss"]


def test_balance_hostile_values():
    """Closed experts (-inf), rows with none open, NaN and infinities in rows that are left out,
    the lowest float as a mask value, ids outside the range, an id twice in a row."""
    b = beam()
    T, E, K = 70, 40, 4
    logits, topk, _, _ = bal_case(T, E, K, "f32", None, None, seed=3)
    logits[:, 7] = -np.inf
    logits[:, 8] = torch.finfo(torch.float32).min
    logits[11] = -np.inf
    valid = torch.ones(T, dtype=torch.uint8)
    logits[20], logits[21] = np.nan, np.inf
    valid[20] = valid[21] = 0
    logits[60:] = np.nan                                # behind the last sequence
    topk[60:] = 1 << 30
    topk[3] = torch.tensor([-1, 5, 5, 40])
    cu = [0, 10, 60]
    args = (logits.cuda(), topk.cuda())
    kw = dict(valid=valid.cuda(), cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    out = b.balance_loss(*args, **kw)
    r = ref.balance(np64(logits), topk.numpy(), E, K, cu, valid.numpy())
    np.testing.assert_array_equal(out["counts"].cpu().numpy(), r["counts"])
    np.testing.assert_allclose(np64(out["prob"]), r["prob"], rtol=150 * U, atol=1e-30)
    gr, gl = rnd(1, T, K), rnd(2, T, K)
    d = np64(b.balance_loss_backward(*args, out, scale=2.0, d_gate_logit=gr.cuda(), d_mask_logit=gl.cuda(), **kw))
    want = np.zeros((T, 2 * E))
    want[:, :E] = ref.balance_grad(np64(logits), topk.numpy(), E, K, 2.0, cu, valid.numpy())
    for t in range(T):
        for k in range(K):
            e = int(topk[t, k])
            if 0 <= e < E:
                want[t, e] += float(gr[t, k])
                want[t, E + e] += float(gl[t, k])
    np.testing.assert_allclose(d, want, rtol=1e-5, atol=1e-6)
    # a NaN in a row that counts is not hidden
    logits[0, 0] = np.nan
    assert torch.isnan(b.balance_loss(logits.cuda(), topk.cuda(), **kw)["loss"])


def test_balance_gradient_against_differences():
    """Central differences of the oracle's loss with the counts fixed."""
    b = beam()
    T, E, K = 12, 9, 2
    logits, topk, _, v = bal_case(T, E, K, "f32", None, 0.7, seed=4)
    out = b.balance_loss(logits.cuda(), topk.cuda(), valid=v.cuda())
    d = np64(b.balance_loss_backward(logits.cuda(), topk.cuda(), out, valid=v.cuda()))
    x, h = np64(logits), 1e-5
    for t, j in ((0, 0), (3, 8), (7, 4), (11, 2)):
        up, dn = x.copy(), x.copy()
        up[t, j] += h
        dn[t, j] -= h
        num = (ref.balance(up, topk.numpy(), E, K, None, v.numpy())["loss"] -
               ref.balance(dn, topk.numpy(), E, K, None, v.numpy())["loss"]) / (2 * h)
        assert abs(num - d[t, j]) <= 1e-6 * np.abs(d).max() + 1e-9


def test_empty_batches():
    b = beam()
    ids = torch.zeros((0, 2), dtype=torch.int32, device="cuda")
    z = torch.zeros((0, 8), device="cuda")
    out = b.balance_loss(z, ids)
    assert float(out["loss"]) == 0 and int(out["counts"].sum()) == 0 and int(out["tokens"][0]) == 0
    assert b.balance_loss_backward(z, ids, out).shape == (0, 8)
    c = b.checkpoint_save(z)
    assert b.checkpoint_load(c).shape == (0, 8)
    w = b.router_weight_grad(c, torch.zeros((0, 5), device="cuda"))
    assert w.shape == (8, 5) and not w.any()
    assert b.router_input_grad(torch.zeros((0, 5), device="cuda"), torch.zeros((7, 5), device="cuda")).shape == (0, 7)
    e = torch.zeros((0, 3), device="cuda")
    assert b.checkpoint_route_grad(c, e, e, z)["dghat"].shape == (0, 3)
    slots = torch.zeros((0, 2), device="cuda")
    g = b.balance_loss_backward(z, ids, out, d_gate_logit=slots, d_mask_logit=slots)
    assert g.shape == (0, 16)
    assert b.router_weight_grad(c, g, parts=2).shape == (2, 8, 8)


# ------------------------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("N,D,pad", [(1, 1, 0), (3, 31, 0), (5, 32, 0), (7, 33, 3), (64, 256, 0), (33, 1413, 27),
                                     (130, 1536, 8), (2, 8192, 0), (300, 40, 1)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_checkpoint_round_trip(N, D, pad, dtype):
    b = beam()
    x = (rnd(N + D, N, D + pad) * torch.exp(rnd(1, N, 1))).to(DT[dtype])[:, :D]
    c = b.checkpoint_save(x.cuda() if pad == 0 else torch.nn.functional.pad(x.cuda(), (0, pad))[:, :D])
    q, byte = ref.encode(np64(x))
    np.testing.assert_array_equal(c["q"].cpu().numpy(), q)
    np.testing.assert_array_equal(c["scale"].cpu().numpy(), byte)
    y = ref.decode(q, byte, D)
    assert np.abs(y - np64(x)).max() <= np.abs(np64(x)).max() / 127
    for t in DT.values():
        np.testing.assert_array_equal(np64(b.checkpoint_load(c, t)), np64(torch.from_numpy(y).to(t)))


def test_checkpoint_extreme_values():
    """Zeros, subnormals, the largest floats, powers of two, values on the scale's border, ties,
    infinities and NaN; each block keeps its own."""
    b = beam()
    fmax, tiny = float(np.finfo(np.float32).max), 2.0 ** -149
    rows = [[0.0], [tiny], [-tiny, 2.0 ** -126], [fmax], [-fmax, 1.0], [127.0], [np.nextafter(np.float32(127), np.float32(200))],
            [-127.0 * 2 ** 10, 0.5 * 2 ** 10, 1.5 * 2 ** 10, 2.5 * 2 ** 10], [2.0 ** -120 * 127, 2.0 ** -121],
            [np.inf, 1.0], [-np.inf], [np.nan, 3.0], [65504.0, -65504.0, 60000.0], [2.0 ** 127]]
    x = torch.zeros((len(rows), 70))
    for i, r in enumerate(rows):
        x[i, 33:33 + len(r)] = torch.tensor(r, dtype=torch.float64).float()
        x[i, 0] = 1.0
    c = b.checkpoint_save(x.cuda())
    q, byte = ref.encode(np64(x))
    np.testing.assert_array_equal(c["scale"].cpu().numpy(), byte)
    np.testing.assert_array_equal(c["q"].cpu().numpy(), q)
    want = ref.decode(q, byte, 70)
    assert np.nanmax(np.abs(want)) <= fmax and (byte == 255).sum() == 3
    np.testing.assert_array_equal(np64(b.checkpoint_load(c)), want)
    np.testing.assert_array_equal(np64(b.checkpoint_load(c, torch.bfloat16)), want)
    half = np64(b.checkpoint_load(c, torch.float16))
    np.testing.assert_array_equal(half[12], np.clip(want[12], -65504, 65504))


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("order", ["neighbours", "mixed"])
def test_checkpoint_every_16_bit_value(dtype, order):
    """All 65536 patterns, in blocks of neighbouring values and in mixed ones (most of those hold a NaN for
    float16, so the values alone are mixed); every decoded value in each type, float16's rounding included."""
    b = beam()
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    if order == "mixed":
        v = v[torch.isfinite(v)]
        v = v[torch.from_numpy(np.random.default_rng(5).permutation(v.numel()))]
    v = v[:v.numel() // 256 * 256].reshape(-1, 256)
    c = b.checkpoint_save(v.cuda())
    q, byte = ref.encode(np64(v))
    np.testing.assert_array_equal(c["scale"].cpu().numpy(), byte)
    np.testing.assert_array_equal(c["q"].cpu().numpy(), q)
    want = ref.decode(q, byte, 256)
    for out in (torch.float32, torch.bfloat16):
        np.testing.assert_array_equal(np64(b.checkpoint_load(c, out)), want)
    half = np.clip(want, -65504, 65504).astype(np.float16).astype(np.float64)
    np.testing.assert_array_equal(np64(b.checkpoint_load(c, torch.float16)), half)


def test_checkpoint_past_32_bit_offsets():
    b = beam()
    N, D = (1 << 20) + 3, 4128
    x = torch.zeros((N, D), dtype=torch.bfloat16, device="cuda")
    tail = rnd(0, 5, D).bfloat16()
    x[-5:] = tail.cuda()
    x[7] = tail[0].cuda()
    c = b.checkpoint_save(x)
    q, byte = ref.encode(np64(tail))
    np.testing.assert_array_equal(c["q"][-5:].cpu().numpy(), q)
    np.testing.assert_array_equal(c["q"][7].cpu().numpy(), q[0])
    del x
    y = b.checkpoint_load(c, torch.bfloat16)
    np.testing.assert_array_equal(np64(y[-5:]), ref.decode(q, byte, D))
    assert not y[8:-5].any()


# ------------------------------------------------------------------------------ slot gradients
@pytest.mark.parametrize("T,K,D,seg", [(1, 1, 32, 0), (1, 2, 4096, 0), (33, 2, 4096, 0), (7, 32, 100, 0), (50, 6, 2048, 16),
                                       (37, 16, 1536, 16), (5, 3, 1, 0), (300, 5, 257, 7), (9, 4, 8191, 65536),
                                       (700, 8, 64, 256), (2000, 16, 96, 0), (2500, 2, 1500, 0),
                                       (2500, 1, 1025, 0), (2400, 2, 2560, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_grad_from_checkpoint(T, K, D, seg, dtype):
    b = beam()
    S = max(1, seg)
    y = rnd(1, T * K, D)
    lead = torch.arange(T) // S * S
    gate = torch.softmax(rnd(2, T, K), 1)[lead].contiguous()
    ml = rnd(3, T, K)[lead].contiguous()
    ml[0, 0] = 0.0                       # the mask's border: kept
    dy = rnd(4, T, D + 3).to(DT[dtype])[:, :D]
    c = b.checkpoint_save(y.cuda())
    out = b.checkpoint_route_grad(c, gate.cuda(), ml.cuda(), torch.nn.functional.pad(dy.cuda(), (0, 3))[:, :D],
                                  reg_scale=0.5, segment_len=seg)
    q, byte = ref.encode(np64(y))
    yv = ref.decode(q, byte, D).reshape(T, K, D)
    s, dr, dl = ref.route_grad(yv, np64(gate), np64(ml), np64(dy), 0.5, S)
    mag = np.einsum("tkd,td->tk", np.abs(yv), np.abs(np64(dy)))
    eps = (D + 64) * U
    assert (np.abs(np64(out["dghat"]) - s) <= eps * mag).all()
    # the decision's sums: the dots' errors and S additions, then a few roundings on values of
    # at most the segment's magnitude (gates and sigmoid' are at most 1)
    seg_mag = np.zeros((T, K))
    for t in range(0, T, S):
        seg_mag[t] = mag[t:t + S].sum(0)
    err = (eps + (min(S, T) + 16) * U) * seg_mag
    assert (np.abs(np64(out["d_mask_logit"]) - dl) <= err + 16 * U * np.abs(dl) + 1e-30).all()
    assert (np.abs(np64(out["d_gate_logit"]) - dr) <= err + (err * np64(gate)).sum(1, keepdims=True) +
            (K + 16) * U * (seg_mag + seg_mag.sum(1, keepdims=True)) + 1e-30).all()
    off = np.arange(T) % S != 0
    assert not np64(out["d_gate_logit"])[off].any() and not np64(out["d_mask_logit"])[off].any()


@pytest.mark.parametrize("T,K,D", [(3, 20, 1537), (2400, 2, 1100), (2, 2, 4096), (3, 8, 2048)])
def test_route_grad_lost_blocks_stay_in_their_slot(T, K, D):
    """A non-finite value loses its block: its own slot's gradients are NaN, the token's other slots and
    the other tokens' get the numbers that they get without it."""
    b = beam()
    y = rnd(1, T * K, D)
    gate, ml, dy = torch.softmax(rnd(2, T, K), 1), rnd(3, T, K).abs(), rnd(4, T, D)
    def run(v):
        out = b.checkpoint_route_grad(b.checkpoint_save(v.cuda()), gate.cuda(), ml.cuda(), dy.cuda())
        return np64(out["dghat"])
    clean = run(y)
    for t, k, c in [(0, 0, 0), (T - 1, K - 1, D - 1), (T // 2, K // 2, D // 2), (1, K - 1, 512)]:
        v = y.clone()
        v[t * K + k, c] = float("inf")
        got = run(v)
        assert np.isnan(got[t, k])
        got[t, k] = clean[t, k]
        np.testing.assert_array_equal(got, clean)


# ------------------------------------------------------------------------------ linear backward
LIN = [(1, 32, 1), (1, 2048, 128), (5, 1, 3), (63, 256, 16), (64, 64, 64), (65, 129, 65), (128, 128, 128),
       (1003, 200, 120), (257, 1536, 424), (130, 100, 513), (4100, 64, 16), (2, 33, 1000)]


@pytest.mark.parametrize("T,D,C", LIN)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ld", [0, 3, 8])
def test_router_weight_grad(T, D, C, dtype, ld):
    b = beam()
    x = rnd(1, T, D)
    g = rnd(2, T, C + ld).to(DT[dtype])[:, :C]
    c = b.checkpoint_save(x.cuda())
    dg = torch.nn.functional.pad(g.cuda(), (0, ld))[:, :C]
    dw = np64(b.router_weight_grad(c, dg))
    xv, gv = ref.decode(*ref.encode(np64(x)), D), np64(g)
    assert (np.abs(dw - xv.T @ gv) <= (T + 64) * U * (np.abs(xv).T @ np.abs(gv)) + 1e-35).all()
    parts = next(p for p in (4, 2, 3, 5, 1) if C % p == 0)
    if parts > 1:
        split = b.router_weight_grad(c, dg, parts=parts)
        assert split.shape == (parts, D, C // parts)
        np.testing.assert_array_equal(np64(split).transpose(1, 0, 2).reshape(D, C), dw)


@pytest.mark.parametrize("T,D,C", LIN)
@pytest.mark.parametrize("dtype,wdtype,ld", [("f32", "f32", 0), ("f32", "bf16", 3), ("bf16", "f32", 0), ("bf16", "bf16", 8),
                                             ("f32", "bf16", 8), ("bf16", "bf16", 0)])
def test_router_input_grad(T, D, C, dtype, wdtype, ld):
    b = beam()
    g, w = rnd(1, T, C + ld).to(DT[dtype])[:, :C], rnd(2, D, C + ld).to(DT[wdtype])[:, :C]
    pad = lambda t: torch.nn.functional.pad(t.cuda(), (0, ld))[:, :C]  # noqa: E731
    dx = np64(b.router_input_grad(pad(g), pad(w)))
    gv, wv = np64(g), np64(w)
    assert (np.abs(dx - gv @ wv.T) <= (C + 64) * U * (np.abs(gv) @ np.abs(wv).T) + 1e-35).all()


def test_linear_backward_small_and_large_magnitudes():
    """Gradients far from 1 keep float32's precision: no narrower type limits their range."""
    b = beam()
    x, g, w = rnd(1, 200, 96), rnd(2, 200, 24), rnd(3, 96, 24)
    c = b.checkpoint_save(x.cuda())
    xv = ref.decode(*ref.encode(np64(x)), 96)
    for s in (1e-25, 1e-6, 1e25):
        gs = (g * s).cuda()
        want = xv.T @ np64(gs)
        assert np.abs(np64(b.router_weight_grad(c, gs)) - want).max() <= 264 * U * (np.abs(xv).T @ np.abs(np64(gs))).max()
        want = np64(gs) @ np64(w).T
        assert np.abs(np64(b.router_input_grad(gs, w.cuda())) - want).max() <= 88 * U * (np.abs(np64(gs)) @ np.abs(np64(w)).T).max()


# ------------------------------------------------------------------------------ how they are called
def _all_ops(b, s):
    bal = b.balance_loss(s["logits"], s["ids"], valid=s["valid"], cu_seqlens=s["cu"])
    yc, xc = b.checkpoint_save(s["y"]), b.checkpoint_save(s["x"])
    slots = b.checkpoint_route_grad(yc, s["gate"], s["ml"], s["dy"], reg_scale=0.1)
    g = b.balance_loss_backward(s["logits"], s["ids"], bal, scale=0.01, valid=s["valid"], cu_seqlens=s["cu"],
                                d_gate_logit=slots["d_gate_logit"], d_mask_logit=slots["d_mask_logit"])
    return dict(loss=bal["loss"], counts=bal["counts"], dw=b.router_weight_grad(xc, g, parts=2),
                dx=b.router_input_grad(g, s["w"]), x=b.checkpoint_load(xc), **slots)


def _op_state(seed=0, T=300, D=256, E=24, K=4):
    logits = rnd(seed, T, E)
    return dict(logits=logits.cuda(), ids=torch.topk(logits, K, dim=1).indices.int().cuda(),
                valid=(rnd(seed + 1, T) > -1).to(torch.uint8).cuda(),
                cu=torch.tensor([0, 17, 200, T - 9], dtype=torch.int32).cuda(), y=rnd(seed + 2, T * K, D).half().cuda(),
                x=rnd(seed + 3, T, D).bfloat16().cuda(), gate=torch.softmax(rnd(seed + 4, T, K), 1).cuda(),
                ml=rnd(seed + 5, T, K).cuda(), dy=rnd(seed + 6, T, D).cuda(), w=rnd(seed + 7, D, 2 * E).bfloat16().cuda())


def test_training_step_repeats_bit_for_bit_on_other_streams_and_in_graphs():
    b = beam()
    s, s2 = _op_state(0), _op_state(50)
    first, second = _all_ops(b, s), _all_ops(b, s2)
    for k, v in _all_ops(b, s).items():
        assert torch.equal(v, first[k]), k
    # two streams at once
    st = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i, state in enumerate((s, s2, s, s2)):
        with torch.cuda.stream(st[i % 2]):
            got.append(_all_ops(b, state))
    torch.cuda.synchronize()
    for r, want in zip(got, (first, second, first, second)):
        for k, v in r.items():
            assert torch.equal(v, want[k]), k
    # two captured graphs, replayed in turn and with new inputs
    graphs = []
    for state in (s, s2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = _all_ops(b, state)
        graphs.append((g, out))
    for g, _ in graphs + graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for (_, out), want in zip(graphs, (first, second)):
        for k, v in out.items():
            assert torch.equal(v, want[k]), k
    for k in s:
        s[k].copy_(s2[k])
    graphs[0][0].replay()
    torch.cuda.synchronize()
    for k, v in graphs[0][1].items():
        assert torch.equal(v, second[k]), k


def test_stream_argument():
    b = beam()
    x = rnd(0, 400, 512).cuda()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    c = b.checkpoint_save(x, stream=st)
    y = b.checkpoint_load(c, stream=st)
    st.synchronize()
    assert torch.equal(y, b.checkpoint_load(b.checkpoint_save(x)))


def test_training_ops_argument_checks():
    b = beam()
    f, i = torch.zeros((4, 8), device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    bad = pytest.raises((ValueError, TypeError, b.BeamError))
    with bad: b.balance_loss(f.double(), i)
    with bad: b.balance_loss(f.half(), i)
    with bad: b.balance_loss(f.t(), i)
    with bad: b.balance_loss(f[:1].expand(4, 8), i)
    with bad: b.balance_loss(f, i.long())
    with bad: b.balance_loss(f, i[:3])
    with bad: b.balance_loss(f, torch.zeros((4, 33), dtype=torch.int32, device="cuda"))
    with bad: b.balance_loss(torch.zeros((4, 257), device="cuda"), i)
    with bad: b.balance_loss(f, i, valid=torch.ones(3, dtype=torch.uint8, device="cuda"))
    with bad: b.balance_loss(f, i, cu_seqlens=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with bad: b.balance_loss(f, i.cpu())
    ok = b.balance_loss(f, i)
    with bad: b.balance_loss_backward(f, i, ok, scale=float("nan"))
    with bad: b.balance_loss_backward(f, i, ok, d_gate_logit=torch.zeros((4, 2), device="cuda"))
    with bad: b.balance_loss_backward(f, i, dict(counts=ok["counts"][:, :7], tokens=ok["tokens"]))
    with bad: b.checkpoint_save(f.int())
    with bad: b.checkpoint_save(f[0])
    with bad: b.checkpoint_save(torch.zeros((1, 65537), device="cuda"))
    c = b.checkpoint_save(f)
    with bad: b.checkpoint_load(c, torch.int8)
    with bad: b.checkpoint_load(dict(q=c["q"][:, :16], scale=c["scale"], d=8))
    with bad: b.checkpoint_load(dict(q=c["q"], scale=c["scale"], d=33))
    g = torch.zeros((2, 2), device="cuda")
    with bad: b.checkpoint_route_grad(c, g, g, torch.zeros((2, 7), device="cuda"))
    with bad: b.checkpoint_route_grad(c, g[:1], g[:1], torch.zeros((1, 8), device="cuda"))
    with bad: b.checkpoint_route_grad(c, g, g, torch.zeros((2, 8), device="cuda"), segment_len=-1)
    with bad: b.checkpoint_route_grad(c, g, g, torch.zeros((2, 8), device="cuda"), reg_scale=float("inf"))
    with bad: b.router_weight_grad(c, torch.zeros((3, 5), device="cuda"))
    with bad: b.router_weight_grad(c, torch.zeros((4, 5), device="cuda"), parts=2)
    with bad: b.router_input_grad(f, torch.zeros((3, 7), device="cuda"))
    with bad: b.router_input_grad(f.half(), f)
    torch.cuda.synchronize()
