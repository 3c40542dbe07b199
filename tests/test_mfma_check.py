"""CPU tests of the matrix-result hazard checker that the build runs on its assembly."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("mfma_check_under_test",
                                              os.path.join(ROOT, "selective_state_space_mssm_amd", "mfma_check.py"))
chk = importlib.util.module_from_spec(spec)
spec.loader.exec_module(chk)

MFMA = "v_mfma_f32_16x16x32_bf16 a[60:63], v[88:91], v[96:99], a[60:63]"


def findings(*body):
    return chk.check_asm("kernel:\n" + "".join(f"\t{l}\n" if not l.endswith(":") else l + "\n" for l in body) + ".Lfunc_end0:\n")


@pytest.mark.parametrize("use", ["v_accvgpr_read_b32 v40, a63", "v_accvgpr_write_b32 a60, v1", "ds_write_b128 v1, a[60:63]",
                                 "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], a[60:63], v[0:3]",
                                 "v_mfma_f32_16x16x32_bf16 a[62:65], v[8:11], v[4:7], a[62:65]"])
def test_early_use_is_found(use):
    assert len(findings(MFMA, use, "s_endpgm")) == 1
    assert len(findings(MFMA, "s_nop 5", use, "s_endpgm")) == 1     # 6 of 7
    assert findings(MFMA, "s_nop 6", use, "s_endpgm") == []


def test_longer_instructions_wait_longer():
    f8 = "v_mfma_f32_16x16x128_f8f6f4 v[0:3], v[8:15], v[16:23], v[0:3]"
    assert findings(f8, "s_nop 7", "s_nop 1", "v_mov_b32 v9, v3", "s_endpgm")      # 10 of 11
    assert not findings(f8, "s_nop 7", "s_nop 2", "v_mov_b32 v9, v3", "s_endpgm")


def test_accumulating_on_the_same_registers_is_fine():
    assert findings(MFMA, MFMA, MFMA, "s_endpgm") == []
    assert findings(MFMA, "v_mfma_f32_16x16x32_bf16 v[0:3], v[8:11], v[4:7], a[60:63]", "s_endpgm") == []


def test_every_path_is_followed():
    # the exit branch leaves two instructions before the read; the fall-through path has enough
    body = [MFMA, "s_cbranch_vccnz .LBB0_1"] + ["s_nop 7"] + [".LBB0_2:", "v_accvgpr_read_b32 v40, a63", "s_endpgm",
                                                          ".LBB0_1:", "s_branch .LBB0_2"]
    got = findings(*body)
    assert len(got) == 1 and got[0][3] == 2


def test_other_registers_and_loops_end():
    assert findings(".LBB0_0:", MFMA, "v_mov_b32 v40, a59", "s_cbranch_scc1 .LBB0_0", "s_endpgm") == []
