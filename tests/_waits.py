"""The waits that a matrix instruction's registers need, looked for in compiled kernels.

The hardware does not hold back a vector, LDS or memory instruction that touches the
result of a matrix instruction still on its way (for p passes of four cycles: p + 4
instructions or wait states after it; 18 for the 64-bit one), nor a vector instruction
that overwrites the sums it still reads (p - 1): the compiler has to put others
between.  A later matrix instruction that takes the sums over waits by itself.  Test
infrastructure."""
import re

OTHERS = ("v_", "ds_", "buffer_", "global_", "flat_", "scratch_")


def passes(op):
    m, n, k = map(int, re.search(r"_(\d+)x(\d+)x(\d+)", op).groups())
    if "f64" in op:
        return None
    rate = 4 if "f8f6f4" in op else 2 if "fp8" in op or "bf8" in op else 1
    return max(4, m * n * k * 2 // 4096 // rate)  # at the fastest type's rate: the fewest


def registers(operands):
    found = set()
    for kind, one, first, last in re.findall(r"\b([va])(?:(\d+)\b|\[(\d+):(\d+)\])",
                                             " ".join(operands)):
        found |= {(kind, i) for i in range(int(one or first), int(one or last) + 1)}
    return frozenset(found)


def functions(assembly):
    """{name: [(label or operation, operands)]}; a label's operands are None."""
    out, code = {}, None
    for line in assembly.splitlines():
        line = line.split(";")[0].strip()
        name = re.match(r"(_Z\w+|[a-z]\w*):$", line)
        label = re.match(r"(\.LBB\w+):$", line)
        if name:
            code = out.setdefault(name[1], [])
        elif code is None or not line:
            continue
        elif label:
            code.append((label[1], None))
        elif line.startswith("."):
            if line.startswith(".section"):
                code = None
        else:
            op, _, rest = line.partition(" ")
            code.append((op, [x.strip() for x in re.split(r",(?![^\[]*\])", rest)] if rest else []))
    return out


def too_early(code):
    """(matrix instruction, the one after it, wait states between, wait states needed)."""
    labels = {op: i for i, (op, args) in enumerate(code) if args is None}
    found = set()
    for at, (op, args) in enumerate(code):
        if args is None or not op.startswith(("v_mfma", "v_smfma")):
            continue
        p, result = passes(op), registers(args[:1])
        found |= follow(code, labels, at, result, 18 if p is None else p + 4, True)
        found |= follow(code, labels, at, registers(args[3:4]) - result, (p or 16) - 1, False)
    return found


def follow(code, labels, at, held, need, result):
    found, best, ways = set(), {}, [(at + 1, 0, held)]
    while ways:
        i, waits, held = ways.pop()
        while i < len(code) and waits < need and held:
            op, args = code[i]
            i += 1
            if args is None:
                if best.get((i, held), need) <= waits:
                    break
                best[i, held] = waits
                continue
            if op == "s_endpgm":
                break
            if op.startswith("s_cbranch"):
                ways.append((labels[args[-1]], waits + 1, held))
            elif op == "s_branch":
                i = labels[args[0]]
            elif op == "s_nop":
                waits += int(args[0], 0)
            elif op.startswith(("v_mfma", "v_smfma")):
                if result and registers(args[1:3]) & held:
                    found.add((code[at][0], op, waits, need))
                held -= registers(args[:1]) | (registers(args[3:4]) if result else frozenset())
            elif op.startswith(OTHERS):
                # what overwrites sums that are still read is a vector instruction
                touched = registers(args if result else args[:1] if op.startswith("v_") else [])
                if touched & held:
                    found.add((code[at][0], op, waits, need))
                held -= touched
            waits += 1
    return found
