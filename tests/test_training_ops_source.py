"""Properties of the training operators' sources that no run can show, on a machine without a GPU."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dynamic_expert_routing_b200", "csrc")
HEADERS = ("balance.cuh", "checkpoint.cuh", "ckpt_handle.cuh", "ckpt_route_grad.cuh", "router_linear.cuh")


def code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


def functions(text):
    """The text cut at every definition: names are looked up within one kernel."""
    return re.split(r"(?=__global__ void|__device__ __forceinline__)", text)


def test_shared_arrays_read_as_vectors_are_aligned():
    """The language aligns a __shared__ array of 4-byte values to 4 bytes only.  One that a kernel reads or
    writes as a 16-byte vector, by its name or by a pointer into it, says so itself."""
    found = 0
    for name in HEADERS:
        for body in functions(code(name)):
            for align, array in re.findall(r"(?<!extern )__shared__\s+(__align__\(16\)\s+)?(?:float|int|uint32_t)\s+(\w+)\[", body):
                names = {array} | set(re.findall(r"\*\s*(\w+)\s*=\s*&?" + array + r"\b", body))
                wide = any(re.search(r"reinterpret_cast<(?:const )?(?:float4|uint4|int4)\*>\(&?" + n + r"\b", body) for n in names)
                if wide:
                    found += 1
                    assert align, f"{name}: {array} is accessed as a 16-byte vector and only 4-byte aligned"
    assert found
