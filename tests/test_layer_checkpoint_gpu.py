"""BeamMoE.checkpoint / backward_checkpoint: the routing's backward from an 8-bit checkpoint of a training
forward, with the balance loss, as one training step uses them together.

What is compared: the checkpoint's routing and logits with the handle's own; the slot gradients with
backward_router's up to the rounding of the expert outputs (each value is off by at most half its
block's step, so a dot product by at most half the sum of |dy| times the steps); dW and dx with the
float64 products of the checkpoint's x and the step's own dense logit gradient (the float32 sum of n
terms: (n + 64) 2^-24 of the sum of the magnitudes).
"""
import numpy as np
import pytest
import torch

import synth
from oracle import training as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def beam():
    import dynamic_expert_routing_b200 as b
    return b


def np64(t):
    return t.detach().cpu().double().numpy()


def make(spec, T, seed=0, max_tokens=None, keep_rate=0.5):
    w = synth.make_layer(spec, seed=seed, keep_rate=keep_rate)
    wd = {k: v.cuda().contiguous() for k, v in w.items() if isinstance(v, torch.Tensor)}
    layer = beam().BeamMoE(wd, spec.top_k, max_tokens=max_tokens or T, segment_len=spec.segment_len)
    return layer, wd, synth.make_tokens(spec, T, seed=seed).cuda()


SPECS = [
    (synth.SPECS["tiny"], 64), (synth.SPECS["tiny"], 1),
    (synth.LayerSpec("small", 512, 16, 4, 256, n_shared=1, d_ff_shared=128), 20),
    (synth.LayerSpec("small", 512, 16, 4, 256, n_shared=1, d_ff_shared=128), 300),
    (synth.LayerSpec("e60", 1024, 60, 4, 256), 100),
    (synth.LayerSpec("fine", 768, 212, 16, 128), 150),
    (synth.LayerSpec("seg", 512, 60, 4, 256, segment_len=16), 16 * 9 + 5),
    (synth.LayerSpec("odd_e", 320, 13, 3, 128, storage="fp32"), 70),
    (synth.LayerSpec("k1", 256, 8, 1, 128), 33),
]


@pytest.mark.parametrize("spec,T", SPECS, ids=[f"{s.name}_{t}" for s, t in SPECS])
def test_backward_from_a_checkpoint(spec, T):
    b = beam()
    layer, wd, x = make(spec, T)
    E, K, D, S = spec.n_experts, spec.top_k, spec.d_model, max(1, spec.segment_len)
    dy = torch.randn((T, D), generator=torch.Generator().manual_seed(3)).cuda()
    layer.forward(x, train=True)
    now = layer.backward_router(x, dy, reg_scale=0.3, slots=True)
    r = layer.routing(T)
    c = layer.checkpoint(x)
    np.testing.assert_array_equal(c["topk_id"].cpu().numpy(), r["topk_id"])
    np.testing.assert_array_equal(c["gate"].cpu().numpy(), r["gate"])
    np.testing.assert_array_equal(c["mask_logit"].cpu().numpy(), r["mask_logit"])
    rows = -(-T // S)
    assert c["logits"].shape == (rows, 2 * E) and c["x"]["q"].shape[0] == rows
    # the logits are those that the routing saw: the mask logits of the chosen experts are its own
    lead = c["topk_id"][::S].long()
    assert torch.equal(torch.gather(c["logits"][:, E:], 1, lead), c["mask_logit"][::S])
    top = torch.topk(c["logits"][:, :E], K, dim=1).values
    assert torch.equal(torch.gather(c["logits"][:, :E], 1, lead), top)
    # another forward overwrites the handle's state, not the checkpoint
    layer.forward(x.flip(0).contiguous(), train=True)
    ids = c["topk_id"][::S].contiguous()
    valid = torch.ones(rows, dtype=torch.uint8, device="cuda")
    valid[rows // 2] = 0
    bal = b.balance_loss(c["logits"][:, :E], ids, valid=valid)
    g = layer.backward_checkpoint(c, dy, reg_scale=0.3, balance=bal, balance_scale=0.7, valid=valid)
    # slots: within the expert outputs' rounding of the gradient from the handle
    step = np64(torch.where(c["y"]["scale"] > 0, 2.0 ** (c["y"]["scale"].double() - 127), 0.0).cpu())
    half = 0.5 * np.repeat(step, 32, 1)[:, :D].reshape(T, K, D)
    y8 = ref.decode(c["y"]["q"].cpu().numpy(), c["y"]["scale"].cpu().numpy(), D).reshape(T, K, D)
    mag = np.einsum("tkd,td->tk", np.abs(y8) + half, np.abs(np64(dy)))
    bound = np.einsum("tkd,td->tk", half, np.abs(np64(dy))) + 2 * (D + 64) * U * mag
    assert (np.abs(np64(g["dghat"]) - np64(now["dghat"])) <= bound).all()
    # and exactly the formulas' from what the checkpoint holds
    s, dr, dl = ref.route_grad(y8, np64(c["gate"]), np64(c["mask_logit"]), np64(dy), 0.3, S)
    scale = np.abs(mag).max() + 1
    assert np.abs(np64(g["dghat"]) - s).max() <= (D + 64) * U * scale
    assert np.abs(np64(g["d_gate_logit"]) - dr).max() <= (D + S + 64) * U * scale * S * K
    assert np.abs(np64(g["d_mask_logit"]) - dl).max() <= (D + S + 64) * U * scale * S
    # the dense logit gradient, and the products with x and W
    dense = np.zeros((rows, 2 * E))
    dense[:, :E] = ref.balance_grad(np64(c["logits"][:, :E]), ids.cpu().numpy(), E, K, 0.7, None, valid.cpu().numpy())
    for i in range(rows):
        for k in range(K):
            dense[i, ids[i, k]] += float(g["d_gate_logit"][i * S, k])
            dense[i, E + ids[i, k]] += float(g["d_mask_logit"][i * S, k])
    xv = ref.decode(c["x"]["q"].cpu().numpy(), c["x"]["scale"].cpu().numpy(), D)
    wm = np.concatenate([np64(wd["w_router"]), np64(wd["w_mask"])], 1)
    small = 64 * U * np.abs(dense).max()             # what the dense gradient's own rounding leaves
    dw = np.concatenate([np64(g["dw_router"]), np64(g["dw_mask"])], 1)
    assert (np.abs(dw - xv.T @ dense) <= (rows + 64) * U * (np.abs(xv).T @ np.abs(dense)) + small * np.abs(xv).sum(0)[:, None] + 1e-30).all()
    dx = np64(g["dx"])
    assert (np.abs(dx[::S] - dense @ wm.T) <= (2 * E + 64) * U * (np.abs(dense) @ np.abs(wm).T) + small * np.abs(wm).sum(1) + 1e-30).all()
    off = np.arange(T) % S != 0
    assert not dx[off].any()
    # 8-bit activations against the full-precision gradient: the rounding is random, a few in a thousand
    if T > 32:
        base = layer.backward_checkpoint(c, dy, reg_scale=0.3)
        for k in ("dw_router", "dw_mask", "dx"):
            rel = float((base[k] - now[k]).norm() / now[k].norm().clamp(min=1e-30))
            # a block's step is at most 2/127 of its largest value: an error of 2/127/sqrt(12) = 0.0046 of
            # that, 4 times the root mean square at most here; x and y each add theirs
            assert rel <= 2 * 4 * 0.0046 or float(now[k].norm()) == 0, (k, rel)


def test_micro_batches_keep_their_own_state():
    """Two forwards, then two backwards: each equals the one taken right after its forward."""
    spec = synth.LayerSpec("small", 512, 16, 4, 256)
    layer, _, x = make(spec, 256, max_tokens=256)
    xs = [x[:200].contiguous(), x[56:].flip(0).contiguous()]
    dys = [torch.randn((200, 512), generator=torch.Generator().manual_seed(i)).cuda() for i in (1, 2)]
    alone = []
    for xi, dy in zip(xs, dys):
        layer.forward(xi, train=True)
        alone.append(layer.backward_checkpoint(layer.checkpoint(xi), dy, reg_scale=0.1))
    cs = []
    for xi in xs:
        layer.forward(xi, train=True)
        cs.append(layer.checkpoint(xi))
    for i in (1, 0):
        g = layer.backward_checkpoint(cs[i], dys[i], reg_scale=0.1)
        for k in g:
            assert torch.equal(g[k], alone[i][k]), k


def test_checkpoint_after_a_replayed_forward_on_a_stream():
    """The forward replays a captured graph on its second call; the checkpoint is the same."""
    spec = synth.LayerSpec("e60", 1024, 60, 4, 256)
    layer, _, x = make(spec, 128)
    y = torch.empty((128, 1024), device="cuda")
    st = torch.cuda.Stream()
    got = []
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(3):
            layer.forward(x, train=True, out=y)
            got.append(layer.checkpoint(x))
    torch.cuda.synchronize()
    for c in got[1:]:
        for k in ("topk_id", "gate", "mask_logit", "logits"):
            assert torch.equal(c[k], got[0][k]), k
        assert torch.equal(c["y"]["q"], got[0]["y"]["q"]) and torch.equal(c["x"]["q"], got[0]["x"]["q"])


def test_checkpoint_order_errors():
    b = beam()
    spec = synth.LayerSpec("small", 512, 16, 4, 256)
    layer, _, x = make(spec, 64)
    with pytest.raises(b.BeamError):
        layer.checkpoint(x)                     # no forward yet
    layer.forward(x)
    with pytest.raises(b.BeamError):
        layer.checkpoint(x)                     # not a training forward
    layer.forward(x, train=True)
    with pytest.raises(b.BeamError):
        layer.checkpoint(x[:32])                # another token count
    with pytest.raises(ValueError):
        layer.checkpoint(x.float())
    c = layer.checkpoint(x)
    with pytest.raises(ValueError):
        layer.backward_checkpoint(c, torch.zeros((32, 512), device="cuda"))
    with pytest.raises(ValueError):
        layer.backward_checkpoint(c, torch.zeros((64, 512), device="cuda"), balance_scale=1.0)
