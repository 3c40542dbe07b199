"""CPU tests of the C ABI in include/mssm_gdr.h: what it declares is exported and
bound, and invalid arguments are refused on the host with the documented status
codes, before any HIP call (no valid call is made here)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "mssm_gdr.h")

mssm = pytest.importorskip("selective_state_space_mssm_amd")
lib = mssm.lib
FAKE, MIS = 0x10000, 0x10004  # aligned stand-in, misaligned
NULL, SHAPE, DTYPE, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4, -5, -6
BIG = 1 << 60


def v(x):
    return None if x is None else ctypes.c_void_p(x)


def problem(tokens=128, seqs=2, groups=2, heads=4, k=64, vd=64, dtype=1, norm=1, scale=1.0):
    return mssm.GdrProblem(tokens, seqs, groups, heads, k, vd, dtype, norm, scale)


INPUTS = ["q", "k", "v", "g", "beta"]
FORWARD = INPUTS + ["h0", "offsets", "y", "h_final"]
SAVED = INPUTS + ["offsets", "ctx", "ctx_bytes", "dy", "dh_final", "dq", "dk", "dv", "dg", "dbeta", "dh0"]
BACKWARD = INPUTS + ["h0", "offsets", "dy", "dh_final", "dq", "dk", "dv", "dg", "dbeta", "dh0"]
STEP = INPUTS + ["slots", "state", "y"]
OPTIONAL = {"h0", "offsets", "h_final", "dh_final", "dh0", "slots"}


def call(name, p, ws=FAKE, wsb=BIG, **kw):
    names = {"fwd": FORWARD, "fwd_train": FORWARD, "bwd_saved": SAVED, "bwd": BACKWARD, "step": STEP}[name]
    args = [kw.get(n, BIG) if n == "ctx_bytes" else v(kw.get(n, None if n in OPTIONAL else FAKE)) for n in names]
    memory = [] if name == "step" else [v(ws), wsb]
    return getattr(lib, "mssm_gdr_" + name)(None if p is None else ctypes.byref(p), *args, *memory, None)


CALLS = ["fwd", "fwd_train", "bwd_saved", "bwd", "step"]


def required(name):
    names = {"fwd": FORWARD, "fwd_train": FORWARD, "bwd_saved": SAVED, "bwd": BACKWARD, "step": STEP}[name]
    return [n for n in names if n not in OPTIONAL and n != "ctx_bytes"]


def test_exports_every_declared_function():
    src = open(HEADER).read()
    names = sorted(set(re.findall(r"^\s*(?:mssm_status|size_t)\s+(mssm_\w+)\s*\(", src, re.M)))
    assert names == sorted(mssm.GDR_EXPORTS)
    for n in names:
        assert hasattr(lib, n)
        assert n.removeprefix("mssm_") in mssm.__all__ or n.endswith("_bytes")
    for name, value in (("MSSM_GDR_MAX_KEY_DIM", mssm.GDR_MAX_KEY_DIM), ("MSSM_GDR_MAX_VALUE_DIM", mssm.GDR_MAX_VALUE_DIM)):
        assert re.search(rf"#define {name} {value}\b", src)


@pytest.mark.parametrize("name", CALLS)
def test_problems_are_refused(name):
    assert call(name, None) == NULL
    for kw in ({"dtype": 2}, {"dtype": -1}):
        assert call(name, problem(**kw)) == DTYPE, kw
    sizes = [{n: x} for n in ("tokens", "seqs", "groups", "heads", "k", "vd") for x in (0, -1)]
    for kw in sizes + [{"heads": 3}, {"scale": float("nan")}, {"scale": float("inf")}, {"tokens": 1 << 31}]:
        assert call(name, problem(**kw)) == SHAPE, kw
    for kw in ({"k": 8}, {"k": 40}, {"k": 144}, {"vd": 24}, {"vd": 528}):
        assert call(name, problem(**kw)) == UNSUPPORTED, kw


@pytest.mark.parametrize("name", CALLS)
def test_pointers_are_refused(name):
    p = problem(tokens=2) if name == "step" else problem()
    for n in required(name):
        assert call(name, p, **{n: None}) == NULL, n
        assert call(name, p, **{n: MIS}) == ALIGN, n
    for n in OPTIONAL & set({"fwd": FORWARD, "fwd_train": FORWARD, "bwd_saved": SAVED, "bwd": BACKWARD, "step": STEP}[name]):
        assert call(name, p, **{n: MIS}) == ALIGN, n


@pytest.mark.parametrize("name", CALLS[:-1])
def test_workspaces_are_refused(name):
    p = problem()
    assert call(name, p, ws=None) == WORKSPACE
    assert call(name, p, ws=MIS) == ALIGN
    size = {"fwd": "fwd_workspace", "fwd_train": "ctx", "bwd_saved": "bwd_saved_workspace", "bwd": "bwd_workspace"}[name]
    need = getattr(lib, f"mssm_gdr_{size}_bytes")(ctypes.byref(p))
    assert need > 0 and call(name, p, wsb=need - 1) == WORKSPACE
    if name == "bwd_saved":
        ctx = lib.mssm_gdr_ctx_bytes(ctypes.byref(p))
        assert call(name, p, ctx_bytes=ctx - 1) == WORKSPACE
    # sequences of one length, and launches that hold every chunk
    assert call(name, problem(tokens=127)) == SHAPE
    assert call(name, problem(tokens=127), offsets=FAKE, ws=None) == WORKSPACE
    assert call(name, problem(tokens=1 << 30, heads=1 << 10, seqs=1, groups=1)) == SHAPE
    assert call(name, problem(heads=1 << 17, groups=1)) == SHAPE      # a chunk's rows beyond 2^31 bytes
    assert call(name, problem(groups=1 << 17, heads=1 << 17, k=64, vd=16)) == SHAPE


def test_steps_are_refused():
    assert call("step", problem(tokens=3)) == SHAPE                    # three rows of two states, without slots
    assert call("step", problem(tokens=1 << 30, seqs=1 << 30)) == SHAPE
    assert call("step", problem(tokens=1, groups=1, heads=(1 << 20) + 1)) == SHAPE


def test_queries_refuse_invalid_problems():
    for name in mssm.GDR_EXPORTS:
        if name.endswith("_bytes"):
            assert getattr(lib, name)(None) == 0
            assert getattr(lib, name)(ctypes.byref(problem(k=40))) == 0


def test_the_workspace_holds_every_chunk_of_packed_sequences():
    # chunks of any lengths have slots of their own below tokens / 64 + seqs
    import random
    r = random.Random(0)
    for _ in range(200):
        n, total = r.randint(1, 20), r.randint(1, 3000)
        ends = [0] + sorted(r.randint(0, total) for _ in range(n - 1)) + [total]
        used = [a // 64 + i + c for i, (a, b) in enumerate(zip(ends, ends[1:])) for c in range(-(-(b - a) // 64))]
        assert len(set(used)) == len(used) and (not used or max(used) < total // 64 + n)


def test_offsets_that_are_none_name_no_slot_outside():
    # clamped as on the device: start to 0 .. tokens, end to start .. tokens
    import random
    r = random.Random(1)
    for _ in range(500):
        n, total = r.randint(1, 9), r.randint(1, 700)
        wild = lambda: r.choice([r.randint(-100, 800), r.randint(0, total), -2 ** 31, 2 ** 31 - 1])  # noqa: E731
        offsets = [wild() for _ in range(n + 1)]
        for i, (a, b) in enumerate(zip(offsets, offsets[1:])):
            a = min(max(a, 0), total)
            b = a if b < a else min(b, total)
            assert a // 64 + i < total // 64 + n
            assert all(a // 64 + i + c < total // 64 + n for c in range(-(-(b - a) // 64)))


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    q, val, g = z(1, 8, 2, 16), z(1, 8, 4, 16), z(1, 8, 4)
    for fn in (lambda *a, **k: mssm.gdr_fwd(*a, **k), mssm.gdr_fwd_train):
        with pytest.raises(ValueError, match="GPU"):
            fn(q, q, val, g, g)
        with pytest.raises(ValueError, match="v must be"):
            fn(q, q, z(8, 4, 16), g, g)
    with pytest.raises(ValueError, match="GPU"):
        mssm.gdr_bwd(q, q, val, g, g, val)
    with pytest.raises(ValueError, match="GPU"):
        mssm.gdr_bwd_saved(q, q, val, g, g, val, z(1))
    with pytest.raises(ValueError, match="GPU"):
        mssm.gdr_step(q[0], q[0], val[0], g[0], g[0], z(8, 4, 16, 16))
    with pytest.raises(ValueError, match="v_t must be"):
        mssm.gdr_step(q, q, val, g, g, z(8, 4, 16, 16))


@pytest.mark.parametrize("name", ["gdr_step", "lora"])
def test_forward_only_is_said(name):
    assert "Forward only: no gradient is recorded." in " ".join(getattr(mssm, name).__doc__.split())
