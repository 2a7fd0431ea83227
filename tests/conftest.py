import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU")
    config.addinivalue_line("markers", "slow: takes more than a few seconds on the CPU")


def gemm_tol(k: int, ref_absmax: float) -> float:
    """Acceptance bound for bf16-in / fp32-accumulate GEMM outputs:
    max |gpu - ref| <= 2e-2 * sqrt(K / 4096) * max |ref|."""
    return 2e-2 * (k / 4096.0) ** 0.5 * ref_absmax


@pytest.fixture(scope="session")
def tol():
    return gemm_tol


# Tests that hold a wrong value, each with the test that holds the right one.
WRONG_VALUES = {
    "tests/test_gpu_linear.py::test_grad_derivatives_far_out_are_zero_or_one":
        "SiLU's derivative at -40 is exp(-40) (1 - 40) = -1.66e-16, a bf16 number, not 0: "
        "tests/test_gpu_feedforward_bits.py::test_own_derivative_far_out",
}


def pytest_collection_modifyitems(items):
    for item in items:
        reason = WRONG_VALUES.get(item.nodeid)
        if reason:
            item.add_marker(pytest.mark.xfail(reason=reason, strict=True))
