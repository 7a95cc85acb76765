"""The instances of the kernels around the routed experts that the library
holds are the ones that its calls can launch, no more."""
import re

import pytest

import mixture_experts_forward_moe_amd as moe


def instances(kernel):
    """Template arguments of the instances of a kernel in the library (the
    names by which the host code registers them)."""
    data = open(moe.LIB_PATH, "rb").read()
    found = re.findall(rb"_ZN3moe12_GLOBAL__N_1\d+" + kernel + rb"I((?:L[ib]\d+E)+)E", data)
    return {tuple(int(v) for v in re.findall(rb"L[ib](\d+)E", args)) for args in found}


def test_router_instances():
    """Experts of a lane; choice, with a bias, statistics.  Choice and
    statistics of more than 512 experts are two launches."""
    want = {(v, s, b, t) for v in (4, 8, 16, 32, 64)
            for s, b, t in ((0, 0, 1), (1, 0, 0), (1, 1, 0), (1, 0, 1), (1, 1, 1)) if not (v == 64 and s and t)}
    assert instances(rb"router_kernel") == want


def test_norm_instances():
    """Threads, vectors a thread, past the caches: rows of up to 8192 values
    go to 1024 threads only while they are fewer than 1024."""
    shapes = [(64, 1), (128, 1), (256, 1), (256, 2), (256, 3), (256, 4), (1024, 1), (1024, 2)]
    assert instances(rb"rmsnorm_kernel") == {(t, v, p) for t, v in shapes for p in (0, 1)} - {(1024, 1, 1)}


@pytest.mark.parametrize("kernel,count", [(b"rmsnorm_backward_kernel", 14), (b"router_backward_kernel", 5),
                                          (b"balance_small_kernel", 3), (b"linear_stream_kernel", 2),
                                          (b"linear_big_kernel", 2)])
def test_other_instances(kernel, count):
    assert len(instances(kernel)) == count
