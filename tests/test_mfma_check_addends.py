"""CPU tests of the check of matrix results where a result is the next instruction's addend: that one may write anywhere,
and what it leaves of the result is still followed."""
import pytest

from test_mfma_check import MFMA, findings

ELSEWHERE = "v_mfma_f32_16x16x32_bf16 a[58:61], v[8:11], v[4:7], a[60:63]"


def test_the_sum_may_go_to_overlapping_registers():
    assert findings(MFMA, ELSEWHERE, "s_endpgm") == []
    # the overlapping ones are its result then
    assert findings(MFMA, ELSEWHERE, "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[4:7], a[58:61]", "s_endpgm") == []


def test_an_operand_is_no_addend():
    assert len(findings(MFMA, "v_mfma_f32_16x16x32_bf16 a[58:61], a[60:63], v[4:7], a[60:63]", "s_endpgm")) == 1


@pytest.mark.parametrize("register,found", [("a62", 1), ("a63", 1), ("a57", 0)])
def test_the_rest_of_the_result_is_followed(register, found):
    assert len(findings(MFMA, ELSEWHERE, f"v_accvgpr_read_b32 v40, {register}", "s_endpgm")) == found
