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


def test_arrivals_in_another_cta_have_cluster_scope():
    """An mbarrier arrival or wait without a scope has the CTA's, which orders nothing between two CTAs: an
    arrival at a barrier of another CTA says .cluster, the shared memory that it announces is released and acquired
    at cluster scope, and the MMA issuer's waits for another CTA's phases are the cluster ones."""
    ptx = code("tc_ptx.cuh")
    remote = re.findall(r"mbarrier\.arrive[\w.]*shared::cluster", ptx)
    assert remote and all(re.match(r"mbarrier\.arrive\.(release|relaxed)\.cluster\.", r) for r in remote), remote
    lin = code("router_linear.cuh")
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive_cluster\(", lin)]
    assert arrivals and all("fence_release_shared();" in lin[max(0, at - 120):at] for at in arrivals)
    issuer = lin[lin.index("kMmaWarp && rank == 0"):lin.index("tc_mma_f16_pair")]
    waits = re.findall(r"mbar_wait(<true>)?\((?:full|tempty)_bar", issuer)
    assert len(waits) == 2 and all(waits) and "fence_acquire_shared();" in issuer


def test_launch_sizes_ask_the_device():
    """The number of SMs is the device's (num_sms), not written out."""
    assert not re.search(r"\b148\b", code("train_ops.cu"))
