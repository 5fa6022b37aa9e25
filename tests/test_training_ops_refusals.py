"""How the training operators refuse a call, on a machine without a GPU: what is raised for a dict that is no
checkpoint, for a stream of another device, for sizes out of range, and when the native module is built again."""
import pytest
import torch


@pytest.fixture(scope="module")
def beam():
    from dynamic_expert_routing_b200 import build
    build.build()
    import dynamic_expert_routing_b200
    return dynamic_expert_routing_b200


def ckpt(**kw):
    c = dict(q=torch.zeros((4, 32), dtype=torch.int8), scale=torch.zeros((4, 1), dtype=torch.uint8), d=8)
    c.update(kw)
    return {k: v for k, v in c.items() if v is not ...}


@pytest.mark.parametrize("key", ["q", "scale", "d"])
def test_a_checkpoint_without_one_of_its_parts(beam, key):
    """ValueError for a missing part, TypeError for one of another type; never another exception."""
    f = torch.zeros((4, 8))
    for call in (beam.checkpoint_load, lambda c: beam.router_weight_grad(c, f), lambda c: beam.checkpoint_route_grad(c, f, f, f)):
        with pytest.raises(ValueError, match=key):
            call(ckpt(**{key: ...}))
        with pytest.raises(TypeError, match=key):
            call(ckpt(**{key: "8"}))
        with pytest.raises(TypeError, match=key):
            call(ckpt(**{key: None}))


class OtherStream:
    """A stream of a device that no tensor here is on."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_a_stream_of_another_device(beam):
    """A call runs on its tensors' device; a stream of another one is refused, not passed over."""
    f, i, st = torch.zeros((4, 8)), torch.zeros((4, 2), dtype=torch.int32), OtherStream()
    layer = object.__new__(beam.BeamMoE)
    layer._h = None
    for call in (lambda: beam.balance_loss(f, i, stream=st), lambda: beam.balance_loss_backward(f, i, {}, stream=st),
                 lambda: beam.checkpoint_save(f, stream=st), lambda: beam.checkpoint_load(ckpt(), stream=st),
                 lambda: beam.checkpoint_route_grad(ckpt(), f, f, f, stream=st),
                 lambda: beam.router_weight_grad(ckpt(), f, stream=st), lambda: beam.router_input_grad(f, f, stream=st),
                 lambda: layer.checkpoint(f, stream=st), lambda: layer.backward_checkpoint({}, f, stream=st)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_balance_and_its_scale_come_together(beam):
    """A balance result without balance_scale would leave its term out, a scale without a result has no term."""
    layer = object.__new__(beam.BeamMoE)
    layer._h, dy = None, torch.zeros((4, 8))
    with pytest.raises(ValueError, match="balance_scale"):
        layer.backward_checkpoint({}, dy, balance={})
    with pytest.raises(ValueError, match="balance_scale"):
        layer.backward_checkpoint({}, dy, balance_scale=0.5)


def test_the_native_module_belongs_to_one_torch(monkeypatch):
    """_training.so holds the installed torch's C++ ABI: under another torch or Python it is stale."""
    import importlib.metadata
    import sysconfig

    from dynamic_expert_routing_b200 import build
    build.build()
    assert not build.stale()
    version = importlib.metadata.version
    with monkeypatch.context() as m:
        m.setattr(importlib.metadata, "version", lambda name: "1.0" if name == "torch" else version(name))
        assert build.stale()
    with monkeypatch.context() as m:
        m.setattr(sysconfig, "get_config_var", lambda name: ".cpython-30.so")
        assert build.stale()
    assert not build.stale()


def test_workspace_sizes_out_of_range(beam):
    """-1 for every size that the call itself refuses."""
    lib = beam.load()
    assert lib.beam_router_weight_grad_workspace((1 << 30) + 1, 8, 6) == -1
    assert lib.beam_router_weight_grad_workspace(1 << 30, 65536, 6) == -1     # too many tiles
    assert lib.beam_router_weight_grad_workspace(4, 65537, 6) == -1
    assert lib.beam_router_weight_grad_workspace(4, 8, (1 << 20) + 1) == -1
    assert lib.beam_router_weight_grad_workspace(1 << 30, 32, 6) >= 0
