"""CPU tests of the C ABI in include/mssm_block.h: what it declares is exported
and bound, and invalid arguments are refused on the host with the documented
status codes, before any HIP call (no valid call is made here)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mssm_block.h")

mssm = pytest.importorskip("selective_state_space_mssm_amd")
lib = mssm.lib
FAKE, MIS = 0x10000, 0x10004  # aligned stand-in, misaligned
OK_NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4, -5, -6


def v(x):
    return None if x is None else ctypes.c_void_p(x)


def test_exports_every_declared_function():
    src = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:mssm_status|size_t)\s+(mssm_\w+)\s*\(", src, re.M)))
    assert names == sorted(mssm.BLOCK_EXPORTS)
    for n in names:
        assert hasattr(lib, n)
        assert n.removeprefix("mssm_") in mssm.__all__ or n.endswith("_bytes")
    for name, value in (("MSSM_MAX_BEAMS", mssm.MAX_BEAMS), ("MSSM_MAX_BEAM_STATES", mssm.MAX_BEAM_STATES), ("MSSM_F8", mssm.MSSM_F8)):
        assert re.search(rf"#define {name} {value}\b", src)


def norm(q8=False, rows=4, dim=64, dtype=1, rdtype=0, eps=1e-5, null=False, **kw):
    p = mssm.NormProblem(rows, dim, dtype, rdtype, eps)
    names = ["x", "residual", "weight", "y"] + (["scale"] if q8 else []) + ["residual_out"]
    args = [v(kw.get(n, FAKE)) for n in names]
    fn = lib.mssm_add_rmsnorm_q8 if q8 else lib.mssm_add_rmsnorm
    return fn(None if null else ctypes.byref(p), *args, None)


@pytest.mark.parametrize("q8", [False, True])
def test_norm_refusals(q8):
    assert norm(q8, null=True) == OK_NULL
    for kw in ({"dtype": 2}, {"dtype": -1}, {"rdtype": 2}):
        assert norm(q8, **kw) == DTYPE
    for kw in ({"rows": 0}, {"dim": 0}, {"rows": -1}, {"rows": 1 << 31}, {"dim": 1 << 24}, {"eps": -1.0}, {"eps": float("nan")}):
        assert norm(q8, **kw) == SHAPE, kw
    for n in ["x", "weight", "y"] + (["scale"] if q8 else []):
        assert norm(q8, **{n: None}) == OK_NULL, n
    for n in ["x", "residual", "weight", "y", "residual_out"] + (["scale"] if q8 else []):
        assert norm(q8, **{n: MIS}) == ALIGN, n


def linear(rows=64, k=64, n=64, dtype=1, out=1, act=0, null=False, ws=FAKE, wsb=1 << 40, **kw):
    p = mssm.LinearProblem(rows, k, n, dtype, out, act)
    eight = FAKE if dtype == 2 else None
    d = {"x": FAKE, "x_scale": eight, "w": FAKE, "w_scale": eight, "bias": None, "residual": None, "y": FAKE, **kw}
    return lib.mssm_linear(None if null else ctypes.byref(p), *[v(a) for a in d.values()], v(ws), wsb, None)


def test_linear_refusals():
    assert linear(null=True) == OK_NULL
    for kw in ({"dtype": 3}, {"dtype": -1}, {"out": 2}, {"dtype": 0, "out": 1}):
        assert linear(**kw) == DTYPE, kw
    for kw in ({"rows": 0}, {"k": 0}, {"n": 0}, {"rows": 1 << 31}, {"n": 1 << 31}, {"k": 1 << 20}):
        assert linear(**kw) == SHAPE, kw
    assert linear(act=4) == UNSUPPORTED and linear(act=-1) == UNSUPPORTED
    for n in ("x", "w", "y"):
        assert linear(**{n: None}) == OK_NULL, n
    assert linear(dtype=2, x_scale=None) == OK_NULL and linear(dtype=2, w_scale=None) == OK_NULL
    assert linear(x_scale=FAKE) == OK_NULL and linear(w_scale=FAKE) == OK_NULL  # scales of operands that take none
    for n in ("x", "w", "bias", "residual", "y", "ws"):
        assert linear(**{n: MIS}) == ALIGN, n
    assert linear(dtype=2, x_scale=MIS) == ALIGN


def beam(batch=2, beams=4, vocab=100, dtype=0, end=-1, null=False, ws=FAKE, wsb=1 << 40, **kw):
    p = mssm.BeamProblem(batch, beams, vocab, dtype, end)
    d = {"logits": FAKE, "scores": FAKE, "finished": None, "scores_out": FAKE, "parent": FAKE, "token": FAKE,
         "finished_out": None, **kw}
    return lib.mssm_beam_select(None if null else ctypes.byref(p), *[v(a) for a in d.values()], v(ws), wsb, None)


def test_beam_select_refusals():
    assert beam(null=True) == OK_NULL
    assert beam(dtype=2) == DTYPE
    for kw in ({"batch": 0}, {"beams": 0}, {"vocab": 0}, {"vocab": 1 << 27}, {"batch": 1 << 30}, {"end": 100}, {"end": -2}):
        assert beam(**kw) == SHAPE, kw
    assert beam(beams=17) == UNSUPPORTED
    for n in ("logits", "scores", "scores_out", "parent", "token"):
        assert beam(**{n: None}) == OK_NULL, n
        assert beam(**{n: MIS}) == ALIGN, n
    assert beam(finished=FAKE) == SHAPE  # finished beams need an end_token
    assert beam(ws=None) == WORKSPACE
    p = mssm.BeamProblem(2, 4, 100, 0, -1)
    need = lib.mssm_beam_select_workspace_bytes(ctypes.byref(p))
    assert need > 0 and beam(wsb=need - 1) == WORKSPACE
    assert lib.mssm_beam_select_workspace_bytes(ctypes.byref(mssm.BeamProblem(2, 17, 100, 0, -1))) == 0


def reorder(batch=2, beams=4, parent=FAKE, count=1, layers=3, nbytes=64, data=FAKE, null=False):
    st = (mssm.BeamState * max(1, count))(*[mssm.BeamState(data, layers, nbytes) for _ in range(max(1, count))])
    return lib.mssm_beam_reorder(batch, beams, v(parent), count, None if null else st, None)


def test_beam_reorder_refusals():
    for kw in ({"batch": 0}, {"beams": 0}, {"count": 0}, {"layers": 0}, {"nbytes": 0}, {"nbytes": 1 << 31}, {"batch": 1 << 29},
               {"layers": 1 << 30}):
        assert reorder(**kw) == SHAPE, kw
    assert reorder(beams=17) == UNSUPPORTED and reorder(count=17) == UNSUPPORTED
    assert reorder(parent=None) == OK_NULL and reorder(null=True) == OK_NULL and reorder(data=None) == OK_NULL
    assert reorder(parent=MIS) == ALIGN and reorder(data=MIS) == ALIGN


def test_workspace_queries_refuse_invalid_problems():
    assert lib.mssm_linear_workspace_bytes(ctypes.byref(mssm.LinearProblem(0, 64, 64, 1, 1, 0))) == 0
    assert lib.mssm_linear_workspace_bytes(None) == 0 and lib.mssm_beam_select_workspace_bytes(None) == 0


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    x, w = torch.zeros(2, 8), torch.zeros(8)
    with pytest.raises(ValueError, match="GPU"):
        mssm.add_rmsnorm(x, w)
    with pytest.raises(ValueError, match="GPU"):
        mssm.add_rmsnorm_q8(x, w, x)
    with pytest.raises(ValueError, match="GPU"):
        mssm.linear(x, torch.zeros(4, 8))
    with pytest.raises(ValueError, match="activation"):
        mssm.linear(x, torch.zeros(4, 8), activation="tanh")
    with pytest.raises(TypeError):
        mssm.linear(x.half(), torch.zeros(4, 8).half())
    with pytest.raises(ValueError):
        mssm.linear(x, w)
    with pytest.raises(ValueError, match="GPU"):
        mssm.beam_select(torch.zeros(1, 2, 5), torch.zeros(1, 2))
    with pytest.raises(ValueError):
        mssm.beam_select(torch.zeros(2, 5), torch.zeros(1, 2))
    with pytest.raises(ValueError, match="GPU"):
        mssm.beam_reorder(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, 2, 4))
