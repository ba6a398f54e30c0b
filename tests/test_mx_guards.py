"""What the microscaled and routing calls guard against besides wrong arguments: order of
a wave's LDS accesses, operands that are no whole tuples, plans and sizes at their limits,
a machine without the extension module."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mq():
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


@pytest.mark.parametrize("source", ["mx_gemm.hip", "mx_quant.hip", "route.hip"])
def test_lanes_hand_lds_over_through_fences(source):
    """A wave barrier alone orders no memory accesses for the compiler: lanes that read
    what others of their wave stored do so behind mx_wave_sync, which fences both sides."""
    csrc = os.path.join(ROOT, "dense_sparse_bit_amd", "csrc")
    assert "__builtin_amdgcn_wave_barrier" not in open(os.path.join(csrc, source)).read()
    helper = re.search(r"void mx_wave_sync\(\) \{(.*?)\}", open(os.path.join(csrc, "mx_device.h")).read(), re.S).group(1)
    calls = re.findall(r"__builtin_amdgcn_(\w+)\(([^)]*)\)", helper)
    assert calls == [("fence", '__ATOMIC_RELEASE, "wavefront", "local"'), ("wave_barrier", ""),
                     ("fence", '__ATOMIC_ACQUIRE, "wavefront", "local"')]
