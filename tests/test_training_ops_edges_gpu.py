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
