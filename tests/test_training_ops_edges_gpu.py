"""The training operators where a value, a size or an order of calls leaves the ordinary: results
against 64-bit formulas written here or in oracle/training.py.

u = 2^-24 is half a float32 step relative to the value; each tolerance counts roundings of it.
"""
import ctypes

import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def beam():
    import dynamic_expert_routing_b200 as b
    return b


def rnd(seed, *shape, scale=1.0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float32) * scale


def np64(t):
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------------------ linear backward
def full_limbs(n, seed):
    """float32 values whose lower 16 bits are all ones: the second and third 8 bits of the significand are
    as large as they get beside the first."""
    r = np.random.default_rng(seed)
    bits = (r.integers(124, 131, n) << 23) | (r.integers(0, 128, n) << 16) | 0xffff | (r.integers(0, 2, n) << 31)
    bits[0] = 0x3f80ffff
    return torch.from_numpy(bits.astype(np.uint32).view(np.float32).copy())


# One product of two float32 numbers.  The leading limbs' product has 16 bits: exact.  The other seven are below
# 2^-6 of the whole together, and their accumulator truncates each addition, 2^-23 of its content:
# 7 * 2^-29 < 0.25 u; the pair left out is below 2^-30; the float32 sum of both accumulators rounds once, u.
PRODUCT = 1.5 * U


def test_input_grad_product_of_two_float32_numbers():
    g, w = full_limbs(200, 1)[:, None], full_limbs(300, 2)[:, None]
    want = np64(g) @ np64(w).T
    dx = np64(beam().router_input_grad(g.cuda(), w.cuda()))
    assert (np.abs(dx - want) / np.abs(want)).max() <= PRODUCT


def test_layer_input_grad_product_of_two_float32_numbers():
    """The same with a float32 layer's own router matrix, which is kept with its other order of W."""
    spec = synth.LayerSpec("odd_e", 320, 13, 3, 128, storage="fp32")
    w = {k: v.cuda().contiguous() for k, v in synth.make_layer(spec, seed=0).items() if isinstance(v, torch.Tensor)}
    T, E, D = 70, spec.n_experts, spec.d_model
    w["w_router"] = full_limbs(D * E, 3).view(D, E).cuda()
    layer = beam().BeamMoE(w, spec.top_k, max_tokens=T)
    col = 5
    g = torch.zeros((T, 2 * E))
    g[:, col] = full_limbs(T, 4)
    want = np64(g)[:, col:col + 1] @ np64(w["w_router"])[:, col:col + 1].T
    g, dx = g.cuda(), torch.empty((T, D), device="cuda")
    lib = beam().load()
    assert lib.beam_moe_router_input_grad(layer._h, ctypes.c_void_p(g.data_ptr()), 2 * E, T,
                                          ctypes.c_void_p(dx.data_ptr()), D,
                                          ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    assert (np.abs(np64(dx) - want) / np.abs(want)).max() <= PRODUCT


# ------------------------------------------------------------------------------ slot gradients
@pytest.mark.parametrize("seg", [0, 4])
@pytest.mark.parametrize("K", [2, 11, 32])
def test_mask_gradient_of_confident_masks(K, seg):
    """sigmoid'(l) far from 0: the dots are exact (small integers), so d_mask_logit has the roundings of the gate's
    product (u), of sigma(l) and sigma(-l) (an exponential of 2 steps, 4 u, an addition and a division: 6 u
    at most, 2 u where the exponential is small) and of two more products: 11 u, 16 u allowed."""
    T, D, S = 24, 32, max(1, seg)
    r = np.random.default_rng(K)
    lead = np.arange(T) // S * S
    l = np.resize(np.float32([-80, -20, -10, -1, 0, 1, 10, 14, 17, 20, 25, 40, 80]), (T, K))[lead]
    gate = r.integers(1, 256, (T, K)).astype(np.float32)[lead] / 256
    y, dy = r.integers(-8, 9, (T * K, D)).astype(np.float32), r.integers(1, 5, (T, D)).astype(np.float32)
    y[:, 0] = 8                                             # exact in steps of 2^-3, and no dot is 0
    y[:, 1:] = np.abs(y[:, 1:])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    out = beam().checkpoint_route_grad(beam().checkpoint_save(t(y)), t(gate), t(l), t(dy), segment_len=seg)
    s = np.einsum("tkd,td->tk", y.reshape(T, K, D).astype(np.float64), dy.astype(np.float64))
    np.testing.assert_array_equal(np64(out["dghat"]), s)
    l64, want = l.astype(np.float64), np.zeros((T, K))
    e = np.exp(-np.abs(l64))
    for i in range(0, T, S):
        want[i] = s[i:i + S].sum(0) * gate[i] * (e / (1 + e) ** 2)[i]
    np.testing.assert_allclose(np64(out["d_mask_logit"]), want, rtol=16 * U, atol=0)


# ------------------------------------------------------------------------------ a layer's calls
def small_layer(T, **kw):
    spec = synth.LayerSpec("small", 512, 16, 4, 256, **kw)
    w = {k: v.cuda().contiguous() for k, v in synth.make_layer(spec, seed=0).items() if isinstance(v, torch.Tensor)}
    return beam().BeamMoE(w, spec.top_k, max_tokens=T, segment_len=spec.segment_len), synth.make_tokens(spec, T, seed=0).cuda()


def test_the_handle_waits_for_its_input_gradient():
    """beam_moe_router_input_grad reads the handle's router matrices: it belongs to the pending work that
    beam_moe_destroy (and beam_moe_host_wait, which waits for the same event) waits for."""
    layer, _ = small_layer(8)
    g, dx = torch.ones((8, 32), device="cuda"), torch.empty((8, 512), device="cuda")
    st, before = torch.cuda.Stream(), torch.cuda.Event()
    lib = beam().load()

    def call():
        assert lib.beam_moe_router_input_grad(layer._h, ctypes.c_void_p(g.data_ptr()), 32, 8, ctypes.c_void_p(dx.data_ptr()),
                                              512, ctypes.c_void_p(st.cuda_stream)) == 0

    torch.cuda.synchronize()
    call()                                      # the first call loads the kernel
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(400_000_000)          # about 0.2 s
        before.record()
    call()
    assert not before.query()                   # the stream is still asleep
    layer.host_wait()
    assert before.query()
    torch.cuda.synchronize()


def test_layer_calls_captured_into_a_graph():
    """checkpoint and backward_checkpoint captured and replayed give the eager results, and the handle still answers."""
    T = 96
    layer, x = small_layer(T)
    dy = rnd(1, T, 512).cuda()
    layer.forward(x, train=True)

    def both():
        c = layer.checkpoint(x)
        return dict(layer.backward_checkpoint(c, dy, reg_scale=0.2), q=c["y"]["q"], logits=c["logits"])
    want = both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    assert layer.stats()["tokens"] == T
    np.testing.assert_array_equal(layer.routing(T)["topk_id"].shape, (T, layer.top_k))
    layer.host_wait()


def test_launch_count_includes_the_checkpoint_calls():
    layer, x = small_layer(32)
    layer.forward(x, train=True)
    n = layer.launch_count()
    c = layer.checkpoint(x)                     # expert outputs, logits
    assert layer.launch_count() == n + 2
    layer.backward_checkpoint(c, torch.ones((32, 512), device="cuda"))
    assert layer.launch_count() == n + 3        # dx; the other operators belong to no handle


def test_balance_backward_reads_topk_only_with_slot_gradients():
    b = beam()
    T, E, K = 37, 12, 3
    logits = rnd(0, T, E).cuda()
    ids = torch.topk(logits, K, dim=1).indices.int()
    bal = b.balance_loss(logits, ids)
    want = b.balance_loss_backward(logits, ids, bal, scale=0.5)
    got = torch.empty_like(want)
    lib, p = b.load(), lambda t: ctypes.c_void_p(t.data_ptr())
    slots = torch.zeros((T, K), device="cuda")

    def call(gr, gl, out):
        return lib.beam_balance_backward(p(logits), 0, T, E, E, None, K, None, None, 0, p(bal["counts"]), p(bal["tokens"]),
                                         ctypes.c_float(0.5), gr, gl, p(out),
                                         ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert call(None, None, got) == 0
    assert torch.equal(got, want)
    assert call(p(slots), p(slots), torch.empty((T, 2 * E), device="cuda")) == 1        # BEAM_ERR_INVALID_ARG
    torch.cuda.synchronize()


def test_balance_takes_bool_masks():
    b = beam()
    T, E, K = 300, 24, 4
    logits = rnd(0, T, E).cuda()
    ids = torch.topk(logits, K, dim=1).indices.int()
    mask = rnd(1, T).cuda() > -0.5
    byte = mask.to(torch.uint8)
    want, got = b.balance_loss(logits, ids, valid=byte), b.balance_loss(logits, ids, valid=mask)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(b.balance_loss_backward(logits, ids, got, valid=mask),
                       b.balance_loss_backward(logits, ids, want, valid=byte))
    with pytest.raises(ValueError):
        b.balance_loss(logits, ids, valid=mask.float())


def test_a_balance_dict_without_one_of_its_parts():
    b = beam()
    logits, ids = rnd(0, 6, 8).cuda(), torch.zeros((6, 2), dtype=torch.int32, device="cuda")
    bal = b.balance_loss(logits, ids)
    for key in ("counts", "tokens"):
        with pytest.raises(ValueError, match=key):
            b.balance_loss_backward(logits, ids, {k: v for k, v in bal.items() if k != key})
        with pytest.raises(TypeError, match=key):
            b.balance_loss_backward(logits, ids, dict(bal, **{key: 3}))


def test_layer_calls_on_a_given_stream():
    T = 64
    layer, x = small_layer(T)
    dy = rnd(2, T, 512).cuda()
    layer.forward(x, train=True)
    want = layer.backward_checkpoint(layer.checkpoint(x), dy, reg_scale=0.1)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)               # the current stream is busy: nothing may wait for it or run on it
    layer.forward(x, train=True, stream=st)
    got = layer.backward_checkpoint(layer.checkpoint(x, stream=st), dy, reg_scale=0.1, stream=st)
    st.synchronize()
    for k, v in want.items():
        assert torch.equal(got[k], v), k
    torch.cuda.synchronize()


def test_a_kept_loss_keeps_little_else():
    b = beam()
    logits, ids = rnd(0, 400, 60).cuda(), torch.zeros((400, 4), dtype=torch.int32, device="cuda")
    cu = torch.arange(0, 401, 5, dtype=torch.int32, device="cuda")
    out = b.balance_loss(logits, ids, cu_seqlens=cu)
    assert out["prob"].shape == (80, 60)
    assert out["loss"].untyped_storage().nbytes() <= 4096
    assert b.balance_loss(logits, ids)["loss"].untyped_storage().nbytes() <= 4096


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_backward_of_values_that_are_not_finite(dtype, bad):
    """They reach their own row or column of the result, where nothing finite is left (NaN from a float32
    operand, an infinity or NaN from a bfloat16 one); every other number is the one without them."""
    b = beam()
    T, D, C = 300, 200, 70
    x, g, w = rnd(1, T, D).cuda(), rnd(2, T, C).to(dtype).cuda(), rnd(3, D, C).to(dtype).cuda()
    x[x == 0] = 1
    c = b.checkpoint_save(x)
    dw, dx = b.router_weight_grad(c, g), b.router_input_grad(g, w)
    gb, wb = g.clone(), w.clone()
    gb[130, 65], wb[7, 3] = bad, bad

    def check(got, want, reached):
        assert not torch.isfinite(got[reached]).any()
        if dtype == torch.float32 or bad != bad:
            assert torch.isnan(got[reached]).all()
        assert torch.equal(got[~reached], want[~reached])
    at = torch.zeros((D, C), dtype=torch.bool, device="cuda")
    at[:, 65] = b.checkpoint_load(c)[130] != 0
    skip = ~at[:, 65]
    got = b.router_weight_grad(c, gb)
    got[skip, 65] = dw[skip, 65]                # 0 times an infinity: NaN or not, by the operand's type
    check(got, dw, at)
    at = torch.zeros((T, D), dtype=torch.bool, device="cuda")
    at[130] = True
    check(b.router_input_grad(gb, w), dx, at)
    at = torch.zeros((T, D), dtype=torch.bool, device="cuda")
    at[:, 7] = True
    check(b.router_input_grad(g, wb), dx, at)
