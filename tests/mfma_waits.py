"""Reads of a matrix instruction's sums that come too early, found in the assembly of this package's kernels.

The sums of an MFMA of n passes are in their registers n + 4 wait states after it (n + 2 for fp32 operands); every
instruction is at least one state and s_nop k is k + 1.  Nothing in the machine holds back an instruction of
another kind that reads or writes those registers before.  The states are counted along every path: an instruction's
registers carry the largest number still to wait for over the ways that lead to it.
"""
import re

PASSES = {"f32_32x32x64_f8f6f4": 16, "f32_16x16x128_f8f6f4": 8, "f32_32x32x16_bf16": 8, "f32_16x16x32_bf16": 4,
          "i32_32x32x32_i8": 8, "i32_16x16x64_i8": 4, "f32_16x16x4_f32": 8}
MATRIX = re.compile(r"v_mfma_(?:scale_)?(\w+)$")
REGISTERS = re.compile(r"^[-|]*([va])(?:(\d+)|\[(\d+):(\d+)\])\|?$")


def registers(operand):
    m = REGISTERS.match(operand)
    if not m:
        return []
    lo, hi = (m.group(2), m.group(2)) if m.group(2) else m.group(3, 4)
    return [(m.group(1), i) for i in range(int(lo), int(hi) + 1)]


def states_after(kind):
    return PASSES[kind] + (2 if kind.endswith("_f32") else 4)


def kernels(assembly):
    """(name, lines) of every function."""
    name, body = None, []
    for line in assembly.splitlines():
        m = re.match(r"^(_Z\w+):", line)
        if m:
            name, body = m.group(1), []
        elif name and re.match(r"^\s*\.section|^\.Lfunc_end", line):
            yield name, body
            name = None
        elif name:
            body.append(line)


def early_reads(lines):
    """([(instruction, matrix instruction, states short)], how many matrix instructions) of one function."""
    code, labels = [], {}
    for line in lines:
        line = re.split(r";|//", line)[0].strip()
        m = re.match(r"^(\.?[\w.$]+):$", line)
        if m:
            labels[m.group(1)] = len(code)
        elif line and not line.startswith("."):
            op, _, rest = line.partition(" ")
            operands = [o.split()[0] for o in re.split(r",(?![^\[]*\])", rest) if o.strip()]
            code.append((op.strip(), operands, line))
    pending, todo, found = [None] * len(code), [], {}
    if code:
        pending[0] = {}
        todo.append(0)
    while todo:
        at = todo.pop()
        op, operands, line = code[at]
        matrix = MATRIX.match(op)
        touched = []
        if matrix:                         # sums that another one adds to wait for themselves; row and column operands do not
            touched = [r for o in operands[1:3] + operands[4:] for r in registers(o)]
        elif re.match(r"(v|ds|global|buffer|flat)_", op):
            touched = [r for o in operands for r in registers(o)]
        for r in touched:
            if r in pending[at]:
                found[(at, r)] = pending[at][r]
        states = int(operands[0], 0) + 1 if op == "s_nop" else 1
        after = {r: (n - states, source) for r, (n, source) in pending[at].items() if n > states}
        if matrix:
            after.update((r, (states_after(matrix.group(1)), at)) for r in registers(operands[0]))
        if op == "s_branch":
            ways = [labels[operands[0]]]
        elif op.startswith("s_cbranch"):
            ways = [at + 1, labels[operands[0]]]
        elif op == "s_endpgm":
            ways = []
        else:
            ways = [at + 1]
        for way in ways:
            if way >= len(code):
                continue
            if pending[way] is None:
                pending[way] = dict(after)
                todo.append(way)
            else:
                more = {r: v for r, v in after.items() if pending[way].get(r, (0,))[0] < v[0]}
                if more:
                    pending[way].update(more)
                    todo.append(way)
    count = sum(bool(MATRIX.match(op)) for op, _, _ in code)
    return sorted({(code[at][2], code[source][2], n) for (at, _), (n, source) in found.items()}), count
