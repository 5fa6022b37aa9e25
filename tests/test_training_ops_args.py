"""Refusals of the training operators on a machine without a GPU: the C ABI rejects bad sizes and
pointers before it touches CUDA, the binding rejects tensors that are not on a device; and the
checkpoint format's oracle on values worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import training as ref


@pytest.fixture(scope="module")
def lib():
    from dynamic_expert_routing_b200 import build, _lib
    build.build()
    return _lib.load()


P = 4096          # an aligned address that no refused call reads
F32, BF16, F16 = 0, 1, 2
BAD = 1           # BEAM_ERR_INVALID_ARG


def _balance(lib, x=P, dt=F32, T=4, E=8, ld=8, ids=P, K=2, valid=None, cu=None, n=0, loss=P, ws=P, size=1 << 20):
    return lib.beam_balance_forward(x, dt, T, E, ld, ids, K, valid, cu, n, loss, P, P, P, ws, size, None)


def test_balance_refusals(lib):
    for kw in (dict(T=-1), dict(E=0), dict(E=257), dict(K=0), dict(K=33), dict(dt=F16), dict(dt=9), dict(ld=7),
               dict(x=None), dict(x=P + 2), dict(ids=None), dict(ids=P + 1), dict(n=3), dict(cu=P, n=0),
               dict(cu=P, n=65537), dict(cu=P + 2, n=2), dict(loss=None), dict(loss=P + 1), dict(cu=P, n=2, ws=None),
               dict(cu=P, n=2, ws=P + 8), dict(T=10000, size=16)):
        assert _balance(lib, **kw) == BAD, kw
        assert lib.beam_moe_last_error()
    assert lib.beam_balance_workspace(-1, 8, 0) == -1
    assert lib.beam_balance_workspace(4, 0, 0) == -1
    assert lib.beam_balance_workspace(4, 8, 70000) == -1
    assert 0 == lib.beam_balance_workspace(4, 8, 0) < lib.beam_balance_workspace(4, 8, 1) < lib.beam_balance_workspace(70000, 256, 64)
    back = lambda scale=1.0, gr=None, gl=None, out=P, counts=P: lib.beam_balance_backward(  # noqa: E731
        P, F32, 4, 8, 8, P, 2, None, None, 0, counts, P, scale, gr, gl, out, None)
    assert back(scale=float("nan")) == BAD and back(gr=P) == BAD and back(out=None) == BAD
    assert back(counts=None) == BAD and back(gr=P + 1, gl=P) == BAD


def test_checkpoint_refusals(lib):
    save = lambda x=P, dt=F32, n=4, d=8, ld=8, q=P, s=P: lib.beam_checkpoint_save(x, dt, n, d, ld, q, s, None)  # noqa: E731
    for kw in (dict(n=-1), dict(d=0), dict(d=65537), dict(ld=7), dict(dt=3), dict(x=None), dict(x=P + 2), dict(q=None),
               dict(q=P + 8), dict(s=None), dict(n=1 << 31)):
        assert save(**kw) == BAD, kw
    assert lib.beam_checkpoint_load(P, P, 4, 8, None, F32, None) == BAD
    assert lib.beam_checkpoint_load(P, P, 4, 8, P, 7, None) == BAD
    assert lib.beam_checkpoint_load(P + 1, P, 4, 8, P, F32, None) == BAD
    assert lib.beam_checkpoint_load(P, P, 4, 8, P + 4, F32, None) == BAD
    # nothing to do: no CUDA call
    assert save(n=0, x=None, q=None, s=None) == 0 and lib.beam_checkpoint_load(None, None, 0, 8, None, F32, None) == 0


def test_gradient_refusals(lib):
    rg = lambda T=4, K=2, d=8, gate=P, dy=P, dt=F32, ld=8, seg=0, reg=0.0, out=P: lib.beam_checkpoint_route_grad(  # noqa: E731
        P, P, T, K, d, gate, P, dy, dt, ld, seg, reg, out, P, P, None)
    for kw in (dict(T=-1), dict(K=0), dict(K=33), dict(d=0), dict(gate=None), dict(gate=P + 2), dict(dy=None), dict(dt=F16),
               dict(ld=4), dict(seg=-1), dict(seg=65537), dict(reg=float("inf")), dict(out=None), dict(out=P + 2),
               dict(T=1 << 30, K=32)):
        assert rg(**kw) == BAD, kw
    ig = lambda T=4, C=5, d=8, g=P, dt=F32, ld=5, w=P, wt=F32, lw=5, dx=P, lx=8: lib.beam_router_input_grad(  # noqa: E731
        g, dt, ld, T, C, w, wt, lw, d, dx, lx, None)
    for kw in (dict(T=-1), dict(C=0), dict(C=(1 << 20) + 1, ld=1 << 21, lw=1 << 21), dict(d=0), dict(g=None), dict(g=P + 2), dict(dt=F16),
               dict(ld=4), dict(w=None), dict(wt=F16), dict(lw=4), dict(dx=None), dict(dx=P + 1), dict(lx=7),
               dict(lx=1 << 31)):
        assert ig(**kw) == BAD, kw
    wg = lambda q=P, T=4, d=8, g=P, dt=F32, ld=6, C=6, parts=1, dw=P: lib.beam_router_weight_grad(  # noqa: E731
        q, P, T, d, g, dt, ld, C, parts, dw, None, 0, None)
    for kw in (dict(q=None), dict(q=P + 8), dict(T=-1), dict(d=0), dict(g=None), dict(g=P + 1), dict(dt=F16), dict(ld=5),
               dict(C=0), dict(parts=0), dict(parts=4), dict(dw=None), dict(dw=P + 2)):
        assert wg(**kw) == BAD, kw
    assert lib.beam_router_weight_grad_workspace(-1, 8, 6) == -1
    assert lib.beam_router_weight_grad_workspace(4, 8, 0) == -1
    assert lib.beam_router_weight_grad_workspace(0, 8, 6) == 0


def test_layer_checkpoint_null_handle(lib):
    assert lib.beam_moe_checkpoint(None, 1, P, P, P, P, P, None, None) == BAD
    assert lib.beam_moe_router_input_grad(None, P, 8, 1, P, 8, None) == BAD


def test_binding_refuses_host_tensors():
    import dynamic_expert_routing_b200 as beam
    f, i = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32)
    c = dict(q=torch.zeros((4, 32), dtype=torch.int8), scale=torch.zeros((4, 1), dtype=torch.uint8), d=8)
    for call in (lambda: beam.balance_loss(f, i), lambda: beam.balance_loss_backward(f, i, {}),
                 lambda: beam.checkpoint_save(f), lambda: beam.checkpoint_load(c),
                 lambda: beam.checkpoint_route_grad(c, f, f, f), lambda: beam.router_weight_grad(c, f),
                 lambda: beam.router_input_grad(f, f)):
        with pytest.raises(ValueError):
            call()


def test_oracle_format_by_hand():
    # 127 fits exponent 0; the next float needs 1; 1.0 alone: 64 * 2^-6
    q, byte = ref.encode(np.array([[127.0, 0.5, 1.5], [128.0, 1.0, 3.0], [1.0, 0, 0], [0, 0, 0]]))
    assert byte[:, 0].tolist() == [127, 128, 121, 7]
    assert q[0, :3].tolist() == [127, 0, 2] and q[1, :3].tolist() == [64, 0, 2] and q[2, 0] == 64
    assert ref.decode(q, byte, 3).tolist() == [[127, 0, 2], [128, 0, 4], [1, 0, 0], [0, 0, 0]]


def test_oracle_balance_by_hand():
    # uniform probabilities: P = 1/E, so the loss is 1 whatever the assignment
    b = ref.balance(np.zeros((6, 4)), np.array([[0, 1]] * 6), 4, 2)
    assert abs(b["loss"] - 1) < 1e-15 and b["counts"].tolist() == [[6, 6, 0, 0]]
    # everything on one expert with probability 1: E
    x = np.full((5, 4), -np.inf)
    x[:, 2] = 0
    assert ref.balance(x, np.full((5, 1), 2), 4, 1)["loss"] == 4
    # the loss does not move along a row's constant direction
    g = ref.balance_grad(np.random.RandomState(0).randn(7, 5), np.random.RandomState(1).randint(0, 5, (7, 2)), 5, 2, 1.0)
    assert np.abs(g.sum(1)).max() < 1e-15
