"""Check of compiled gfx950 assembly for matrix-instruction result hazards.

The result of a ``v_mfma`` instruction may be touched by another instruction
only some wait states after its issue (its passes of 4 cycles, plus 3 for the
matrix-core types and 2 for float32; an instruction is one wait state, ``s_nop
N`` is N + 1).  The compiler inserts them, but the accumulator reads behind a
loop exit have been seen to get none, on the path of the exit alone (an 8-bit
product wrong in the last two values of its last accumulator).  ``check_asm``
follows every path from every matrix instruction and reports each instruction
that reads or writes part of its result too early.  Matrix instructions that take
it whole as their accumulator are interlocked and are not reported, nor are those
that only write to its registers and are known (``PASSES``) to take as long or
longer: matrix instructions of one length end in the order in which they begin.

``__graft_entry__.build`` runs it on the assembly of the library it builds and
fails the build on any finding.
"""
from __future__ import annotations

import re
import sys

PASSES = {"v_mfma_f32_16x16x32_bf16": 4, "v_mfma_f32_16x16x4_f32": 8, "v_mfma_f32_32x32x2_f32": 16,
          "v_mfma_f32_16x16x128_f8f6f4": 8}
_LABEL = re.compile(r"^([.\w$]+):")
_REG = re.compile(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])")
_ENDS = ("s_branch", "s_endpgm", "s_setpc_b64", "s_trap")


def _regs(text):
    out = set()
    for kind, one, lo, hi in _REG.findall(text):
        out.update((kind, i) for i in (range(int(lo), int(hi) + 1) if lo else (int(one),)))
    return out


def needed(op: str) -> int:
    """Wait states between a matrix instruction and the first use of its result."""
    passes = PASSES.get(op, 16)
    return passes + (2 if op.endswith("_f32") else 3)


def _adds_to(dst, op, args):
    """A matrix instruction with the whole result as its addend, which it does not read as an operand: it writes after
    the result is there, wherever to."""
    if not op.startswith("v_mfma"):
        return False
    parts = [_regs(p) for p in re.split(r",\s*(?![^\[]*\])", args)[:4]]
    return parts[3:] == [dst] and not any(dst & p for p in parts[1:3])


def _overwrites(dst, first, op, args):
    """A matrix instruction that reads nothing of the result and takes at least as long: they end in order, so what it
    writes of the result's registers is its own."""
    if not op.startswith("v_mfma") or op not in PASSES or PASSES[op] < PASSES.get(first, 16):  # unlisted: maybe a short one
        return False
    return not any(dst & _regs(p) for p in re.split(r",\s*(?![^\[]*\])", args)[1:4])


def _interlocked(dst, op, args):
    """A matrix instruction that takes the result as its whole accumulator, and touches it nowhere else in part."""
    if not op.startswith("v_mfma"):
        return False
    parts = [_regs(p) for p in re.split(r",\s*(?![^\[]*\])", args)[:4]]
    return _adds_to(dst, op, args) or all(not (dst & p) or (dst == p and i == 0) for i, p in enumerate(parts))


def _functions(text):
    name, body = None, []
    for line in text.splitlines():
        line = line.split(";")[0].rstrip()
        m = _LABEL.match(line)
        if m and not m.group(1).startswith((".L", "L")):
            if name:
                yield name, body
            name, body = m.group(1), []
        elif name and line.startswith(".Lfunc_end"):
            yield name, body
            name, body = None, []
        elif name and line.strip():
            body.append(line.strip())
    if name:
        yield name, body


def check_function(body):
    """[(matrix instruction, offending instruction, wait states)]"""
    ins, at = [], {}
    for line in body:
        m = _LABEL.match(line)
        if m:
            at[m.group(1)] = len(ins)
        elif not line.startswith("."):
            op, _, args = line.partition(" ")
            ins.append((op.split("\t")[0], (op + " " + args).split(None, 1)[1] if args or "\t" in op else ""))
    found = []
    for i, (op, args) in enumerate(ins):
        if not op.startswith("v_mfma"):
            continue
        dst = frozenset(_regs(args.split(",")[0]))
        limit, seen, todo = needed(op), {}, [(i + 1, 0, dst)]
        while todo:
            k, waited, dst = todo.pop()
            while k < len(ins) and waited < limit:
                if seen.get((k, dst), limit) <= waited:
                    break
                seen[k, dst] = waited
                o, a = ins[k]
                after = _overwrites(dst, op, o, a)
                if dst & _regs(a) and not after and not _interlocked(dst, o, a):
                    found.append((f"{op} {args}", f"{o} {a}", waited))
                    break
                if after or _adds_to(dst, o, a):
                    dst -= _regs(a.split(",")[0])  # those are its own result from here on
                    if not dst:
                        break
                if o.startswith(("s_cbranch", "s_branch")) and a.split()[-1] in at:
                    todo.append((at[a.split()[-1]], waited + 1, dst))
                if o in _ENDS:
                    break
                waited += int(a, 0) + 1 if o == "s_nop" else 1
                k += 1
    return found


def check_asm(text: str):
    """[(function, matrix instruction, offending instruction, wait states)]"""
    return [(name, *f) for name, body in _functions(text) for f in check_function(body)]


if __name__ == "__main__":
    bad = [(p, f) for p in sys.argv[1:] for f in check_asm(open(p).read())]
    for p, f in bad:
        print(f"{p}: {f[0]}: {f[1]} -> {f[2]} after {f[3]} wait states, {needed(f[1].split()[0])} needed")
    sys.exit(1 if bad else 0)
