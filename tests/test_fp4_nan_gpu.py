"""The tests of 4-bit products, experts and layers once more under a comparison
that a NaN in a bf16 result cannot pass (fp4_checks.check)."""
import pytest

import fp4_checks
import test_fp4_gemm_gpu as tests
from test_fp4_gemm_gpu import (clean, fp4, ops, test_experts_module, test_experts_product,  # noqa: F401
                               test_experts_product_in_rounds_of_tiles, test_forward_call_by_expert,
                               test_forward_call_equals_cast_and_product, test_layer_step, test_product,
                               test_product_in_rounds_of_tiles, test_strided_output_keeps_its_surroundings)

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def strict(monkeypatch):
    monkeypatch.setattr(tests, "check", fp4_checks.check)
