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
