"""CPU tests of mssm_lora's refusals, with the documented status codes, before any HIP call."""
import ctypes

import pytest

mssm = pytest.importorskip("selective_state_space_mssm_amd")
lib = mssm.lib
FAKE, MIS = 0x10000, 0x10004
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4, -5, -6


def v(x):
    return None if x is None else ctypes.c_void_p(x)


def lora(rows=64, k=64, n=64, rank=8, adapters=4, dtype=1, out=1, null=False, ws=FAKE, wsb=1 << 60, **kw):
    p = mssm.LoraProblem(rows, k, n, rank, adapters, dtype, out)
    d = {"x": FAKE, "x_scale": FAKE if dtype == 2 else None, "a": FAKE, "b": FAKE, "scale": None, "index": FAKE, "y": FAKE, **kw}
    return lib.mssm_lora(None if null else ctypes.byref(p), *[v(x) for x in d.values()], v(ws), wsb, None)


def test_refusals():
    assert lora(null=True) == NULL
    for kw in ({"dtype": 3}, {"dtype": -1}, {"out": 2}, {"dtype": 0, "out": 1}):
        assert lora(**kw) == DTYPE, kw
    for kw in ({"rows": 0}, {"k": 0}, {"n": 0}, {"rank": 0}, {"adapters": 0}, {"rows": 1 << 28}, {"k": 1 << 20}, {"n": 1 << 23},
               {"adapters": 1 << 31}, {"rows": 1 << 27, "n": 1 << 20}):
        assert lora(**kw) == SHAPE, kw
    assert lora(rank=129) == UNSUPPORTED
    for n in ("x", "a", "b", "index", "y"):
        assert lora(**{n: None}) == NULL, n
    for n in ("x", "a", "b", "index", "y", "scale", "ws"):
        assert lora(**{n: MIS}) == ALIGN, n
    assert lora(dtype=2, x_scale=None) == NULL and lora(x_scale=FAKE) == NULL and lora(dtype=2, x_scale=MIS) == ALIGN
    for rows in (1, 64, 65, 4000):
        need = lib.mssm_lora_workspace_bytes(ctypes.byref(mssm.LoraProblem(rows, 2560, 64, 16, 4, 1, 1)))
        assert need >= rows * 16 * 4 and lora(rows=rows, k=2560, rank=16, wsb=need - 1) == WORKSPACE
    assert lora(ws=None) == WORKSPACE
    assert lib.mssm_lora_workspace_bytes(None) == 0
    assert lib.mssm_lora_workspace_bytes(ctypes.byref(mssm.LoraProblem(4, 4, 4, 129, 1, 1, 1))) == 0


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    x, a, b, i, y = z(4, 8), z(2, 3, 8), z(2, 6, 3), z(4, dtype=torch.int32), z(4, 6)
    with pytest.raises(ValueError, match="GPU"):
        mssm.lora(x, a, b, i, y)
    with pytest.raises(ValueError, match="must be"):
        mssm.lora(x, a[0], b, i, y)
    with pytest.raises(TypeError):
        mssm.lora(x.half(), a, b, i, y)
