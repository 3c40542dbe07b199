"""CPU tests of the check of matrix results where another matrix instruction writes over a result's registers without
reading them: one that takes as long ends later, and what it leaves of the result is still followed."""
import pytest

from test_mfma_check import MFMA, findings

OVER = "v_mfma_f32_16x16x32_bf16 a[62:65], v[8:11], v[4:7], v[0:3]"


def test_an_instruction_as_long_may_write_over_it():
    assert findings(MFMA, OVER, "s_endpgm") == []
    assert findings(MFMA, "v_mfma_f32_16x16x128_f8f6f4 a[62:65], v[8:15], v[16:23], v[0:3]", "s_endpgm") == []


def test_a_shorter_one_may_not():
    long = "v_mfma_f32_16x16x128_f8f6f4 a[60:63], v[88:95], v[96:103], a[60:63]"
    assert len(findings(long, OVER, "s_endpgm")) == 1


@pytest.mark.parametrize("use", ["v_mfma_f32_16x16x32_bf16 a[62:65], v[8:11], v[4:7], a[62:65]",
                                 "v_mfma_f32_16x16x32_bf16 a[62:65], a[60:63], v[4:7], v[0:3]"])
def test_one_that_reads_of_it_may_not(use):
    assert len(findings(MFMA, use, "s_endpgm")) == 1


@pytest.mark.parametrize("register,found", [("a60", 1), ("a61", 1), ("a66", 0)])
def test_the_rest_of_the_result_is_followed(register, found):
    assert len([f for f in findings(MFMA, OVER, f"v_accvgpr_read_b32 v40, {register}", "s_endpgm") if f[1] == MFMA]) == found


def test_the_new_result_is_followed():
    assert len(findings(MFMA, OVER, "v_accvgpr_read_b32 v40, a64", "s_endpgm")) == 1
