"""CPU test: sizes of mssm_lora whose launches would have 2^32 threads or more are refused on the host.  Tiles have 16 or
more rows, and 256 columns and threads; float32 of a rank above 64 goes by 16 rows however many there are."""
import ctypes

import pytest

from test_lora_abi import SHAPE, lora, mssm

lib = mssm.lib


def accepted(rows, n, rank, dtype, out):
    return lib.mssm_lora_workspace_bytes(ctypes.byref(mssm.LoraProblem(rows, 64, n, rank, 4, dtype, out))) > 0


@pytest.mark.parametrize("rank,tile", [(128, 16), (65, 16), (64, 32)])
def test_float32(rank, tile):
    for n in (1, 256, 257, 2560):
        most = ((1 << 24) - 1) // -(-n // 256) * tile  # rows
        most = min(most, (1 << 28) - 1)
        assert accepted(most, n, rank, 0, 0)
        assert not accepted(most + 1, n, rank, 0, 0) and lora(rows=most + 1, n=n, rank=rank, dtype=0, out=0) == SHAPE


@pytest.mark.parametrize("dtype,out", [(1, 1), (1, 0), (2, 1)])
def test_narrow_types(dtype, out):
    assert accepted((1 << 28) - 1, 256, 128, dtype, out)
    assert not accepted((1 << 28) - 1, 600, 128, dtype, out)
    assert lora(rows=(1 << 28) - 1, n=600, rank=128, dtype=dtype, out=out, x_scale=0x10000 if dtype == 2 else None) == SHAPE
