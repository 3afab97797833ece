"""Both stacks refuse a q6_K form that is none before they touch a weight (on the CPU)."""
import pytest

from quantized_prefill_gemm_amd.stack import ExpertStack, Stack


@pytest.mark.parametrize("q6", ["", "Raw", "expand", None])
def test_q6_form(q6):
    with pytest.raises(ValueError, match="q6 form"):
        Stack([None], 4, q6=q6)
    with pytest.raises(ValueError, match="q6 form"):
        ExpertStack([None], [None], 4, 2, 1, q6=q6)
