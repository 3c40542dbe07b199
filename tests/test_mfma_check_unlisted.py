"""CPU tests of the check of matrix results where the instruction that writes over a result's registers is one whose
length the check does not know: it may be a short one that ends first, and is reported."""
import pytest

from test_mfma_check import MFMA, findings
from test_mfma_check_rewrites import OVER


@pytest.mark.parametrize("op", ["v_mfma_f32_4x4x4_16b_bf16", "v_mfma_scale_f32_16x16x128_f8f6f4", "v_mfma_f64_16x16x4_f64"])
def test_an_unknown_length_is_reported(op):
    assert len(findings(MFMA, OVER.replace("v_mfma_f32_16x16x32_bf16", op), "s_endpgm")) == 1


def test_an_unknown_length_is_the_longest_where_it_is_written_over():
    long = "v_mfma_f32_4x4x4_16b_bf16 a[60:63], v[88:89], v[96:97], a[60:63]"
    assert len(findings(long, OVER, "s_endpgm")) == 1
