"""Path-sensitive check of gfx950 assembly for matrix steps chained too closely.

A matrix step that takes the result of one with another opcode as its
accumulator may start in the pipeline before that result is whole: the compiler
puts no wait between the two, and a 16x16x32 step three instructions behind a
16x16x16 one has read the accumulator's old contents.  The 4-bit kernels start a
sum on the bf16 step and go on with the step of the input's type, and keep at
least 32 cycles between the two; this check reads that distance off the compiled
code.

Model: every matrix step leaves (destination registers, opcode, cycles behind it); an
instruction's cycles are a lower bound: a 16x16x32 matrix step 16, another vector
instruction 4, s_nop n n + 1, anything else none.  Entries older than ``NEED``
cycles are dropped.  From the kernel entry, both successors of every conditional
branch are followed to a fixpoint of (instruction, entries).  A matrix step whose
accumulator input overlaps an entry of another opcode is a hazard.
"""
import re

from tests.lds_read_check import _LABEL, _regs

NEED = 32


def chain_hazards(lines) -> tuple:
    """({instruction: cycles between its accumulator's step and it}, matrix steps,
    their opcodes) of one function's assembly lines."""
    f = [l.split(";")[0].strip() for l in lines]
    f = [l for l in f if l and (not l.startswith(".") or _LABEL.match(l))]
    labels = {l[:-1]: k for k, l in enumerate(f) if _LABEL.match(l)}
    found, seen = {}, set()
    work = [(0, frozenset())]
    while work:
        pc, pend = work.pop()
        while pc < len(f):
            if (pc, pend) in seen:
                break
            seen.add((pc, pend))
            line = f[pc]
            op = line.split()[0]
            if op == "s_endpgm":
                break
            if op == "s_branch":
                pc = labels[line.split()[1]]
                continue
            if op.startswith("s_cbranch"):
                work.append((labels[line.split()[1]], pend))
            cost = 0
            if op.startswith("v_mfma"):
                dst, _, _, acc = [a.strip() for a in line.split(None, 1)[1].split(",")][:4]
                reads = _regs(acc)
                for regs, other, since in pend:
                    if other != op and reads & regs:
                        found[f"{line} after {other}"] = min(since, found.get(line, since))
                out = frozenset(_regs(dst))
                pend = frozenset((r, o, s) for r, o, s in pend if not r & out) | {(out, op, -16)}
                cost = 16
            elif op == "s_nop":
                cost = int(line.split()[1], 0) + 1
            elif op.startswith("v_"):
                cost = 4
            if cost:
                pend = frozenset((r, o, s + cost) for r, o, s in pend if s + cost < NEED)
            pc += 1
    steps = [l for l in f if l.startswith("v_mfma")]
    return found, len(steps), len({l.split()[0] for l in steps})


def file_chain_hazards(text: str, kernel: str) -> tuple:
    """Hazards of every function whose name contains ``kernel``: ({name: hazards},
    functions, functions with matrix steps of several opcodes)."""
    found, n, mixed = {}, 0, 0
    for m in re.finditer(rf"^(_Z\w*{kernel}\w*):.*?^\.Lfunc_end", text, re.M | re.S):
        n += 1
        bad, steps, opcodes = chain_hazards(m.group(0).split("\n")[1:])
        mixed += opcodes > 1
        if bad:
            found[m.group(1)] = bad
    return found, n, mixed
