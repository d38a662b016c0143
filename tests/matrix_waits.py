"""Wait states between a matrix instruction and the first use of its result,
along every path of a disassembled gfx950 kernel.

The matrix core writes its result some cycles after issue, and a vector or
memory instruction that reads (or overwrites) those registers earlier gets the
old value: the hardware does not wait, the compiler has to put other
instructions or s_nop between.  An instruction takes one wait state, s_nop N
takes N + 1; a result of P passes (4 cycles each) needs P + 4.  Another matrix
instruction may take the result as its whole accumulator input without waiting;
as an operand, or a part of it as accumulator, it needs the same P + 4."""
import re

# 2048 multiply-adds a pass of 16-bit values, 4096 of 8-bit ones
PASSES = {"v_mfma_f32_16x16x32_f16": 4, "v_mfma_f32_32x32x16_f16": 8,
          "v_mfma_f32_16x16x128_f8f6f4": 8, "v_mfma_scale_f32_16x16x128_f8f6f4": 8}
_LINE = re.compile(r"^\s+(\S.*?)\s*// ([0-9A-F]+):(.*)$")
_HEAD = re.compile(r"^([0-9a-f]+) <(.+)>:$")
_REG = re.compile(r"-?\|?([av])(?:\[(\d+):(\d+)\]|(\d+))")
_VECTOR = ("v_", "ds_", "global_", "buffer_", "flat_", "scratch_")


def _regs(op):
    m = _REG.match(op)
    if not m:
        return frozenset()
    lo = int(m.group(2) or m.group(4))
    return frozenset((m.group(1), i) for i in range(lo, int(m.group(3) or lo) + 1))


def functions(text):
    """(name, [(mnemonic, operands, branch target or None)]) of a listing of
    llvm-objdump -d --no-show-raw-insn."""
    name, base, rows = None, 0, []

    def done():
        at = {a: i for i, (a, _, _, _) in enumerate(rows)}
        return name, [(n, o, at.get(t)) for _, n, o, t in rows]
    for line in text.splitlines():
        m = _HEAD.match(line)
        if m:
            if name and rows:
                yield done()
            name, base, rows = m.group(2), int(m.group(1), 16), []
            continue
        m = _LINE.match(line)
        if not m or name is None:
            continue
        n, _, rest = m.group(1).partition(" ")
        target = None
        if n.startswith(("s_branch", "s_cbranch")):
            t = re.search(r"<[^>]*?(?:\+0x([0-9a-f]+))?>", m.group(3))
            target = base + int(t.group(1) or "0", 16)
        rows.append((int(m.group(2), 16), n, [x.strip() for x in rest.split(",")], target))
    if name and rows:
        yield done()


def _next(code, i):
    n, _, target = code[i]
    if n.startswith("s_endpgm"):
        return []
    out = [] if target is None else [target]
    if not n.startswith("s_branch") and i + 1 < len(code):
        out.append(i + 1)
    return out


def _touches(code, j, d):
    """Whether instruction j needs the results d of an earlier matrix
    instruction to have arrived, and what of d is left behind it."""
    n, ops, _ = code[j]
    if not n.startswith(_VECTOR):
        return False, d
    regs = [_regs(o) for o in ops]
    if n.startswith("v_mfma"):   # (matrix instructions write in order of issue)
        part = bool(regs[3] & d) and not regs[3] >= d
        return part or any(r & d for r in regs[1:3]), d - regs[0]
    return any(r & d for r in regs), d


def shortages(code):
    """(index of the matrix instruction, index of the use, wait states between,
    wait states needed) wherever a path is too short; KeyError for a matrix
    instruction whose passes are not listed."""
    found = []
    for i, (n, ops, _) in enumerate(code):
        if not n.startswith(("v_mfma", "v_smfmac")):
            continue
        need = PASSES[n] + 4
        todo, seen = [(j, 0, _regs(ops[0])) for j in _next(code, i)], set()
        while todo:
            j, waits, d = todo.pop()
            if waits >= need or not d or (j, waits, d) in seen:
                continue
            seen.add((j, waits, d))
            short, d = _touches(code, j, d)
            if short:
                found.append((i, j, waits, need))
                continue
            m, o, _ = code[j]
            step = int(o[0], 0) + 1 if m == "s_nop" else 1
            todo += [(k, waits + step, d) for k in _next(code, j)]
    return found
