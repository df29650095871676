"""The built kernels' code, on the CPU, along every way that the program can
take, loops among them, where the matrix instructions are inline assembly: their
results are read 18 states after them at the earliest, and between a vector
instruction and the matrix instruction that reads what it wrote are two states
at the least (the compiler counts neither for inline assembly)."""

import functools
import re

from test_lib_matrix_waits import KERNELS, NEEDED
from test_lib_matrix_waits import registers as _registers
from test_lib_wait_states import listings  # noqa: F401  (a fixture)

registers = functools.lru_cache(None)(_registers)
BEFORE = 3           # counted as NEEDED, from the one instruction to the other


def kernels(listing):
    """{function: [(address, operation, operands, the branch's target or None)]}."""
    found, function = {}, None
    for line in listing.splitlines():
        m = re.match(r"([0-9a-f]+) <(.*)>:", line)
        if m:
            function = m.group(2) if KERNELS in m.group(2) else None
            start = int(m.group(1), 16)
            continue
        text, _, comment = line.partition("//")
        if function is None or not line.startswith("\t") or not comment:
            continue
        op, _, rest = text.strip().partition(" ")
        operands = [v.strip() for v in re.split(r",|\s", rest) if v.strip()]
        m = re.search(r"<.*?(?:\+0x([0-9a-f]+))?>", comment)
        target = start + int(m.group(1) or "0", 16) if m and op.startswith(("s_branch", "s_cbranch")) else None
        found.setdefault(function, []).append((int(comment.split(":")[0], 16), op, operands, target))
    return found


def ways(code, places, at, states):
    """(instruction, states since) of what can follow instruction `at` within so many states."""
    seen, todo = {}, [(at, 0)]
    while todo:
        k, since = todo.pop()
        _, op, operands, target = code[k]
        if k != at or since:
            if seen.get(k, states) <= since:
                continue
            seen[k] = since
        since += int(operands[0], 0) + 1 if op == "s_nop" else 1
        if since >= states:
            continue
        if target is not None:
            todo.append((places[target], since))
        if op not in ("s_branch", "s_endpgm", "s_setpc_b64") and k + 1 < len(code):
            todo.append((k + 1, since))
    return [(code[k], since) for k, since in seen.items()]


def too_soon(listing):
    """(number of matrix instructions, [(function, instruction, states from the one to the other)])."""
    count, found = 0, []
    for function, code in kernels(listing).items():
        places = {address: k for k, (address, _, _, _) in enumerate(code)}
        for k, (_, op, operands, _) in enumerate(code):
            if not op.startswith("v_") or not operands:
                continue
            matrix = op.startswith("v_mfma")
            count += matrix
            out = registers(operands[0])
            for (_, other, reads, _), since in ways(code, places, k, NEEDED if matrix else BEFORE):
                if other.startswith("v_mfma"):
                    near = not matrix and any(out & registers(v) for v in reads[1:])
                else:
                    near = matrix and any(out & registers(v) for v in reads)
                if near and since < (NEEDED if matrix else BEFORE):
                    found.append((function, other + " " + " ".join(reads), since))
    return count, found


def _listing(*lines):
    return "\n".join(["0000000000000100 <wide_kernel>:"] + ["\t%s // %012X: 00000000 %s" % (text, 0x100 + 4 * k, comment)
                                                            for k, (text, comment) in enumerate(lines)])


def test_following_branches():
    product = ("v_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]", "")
    read = ("v_accvgpr_read_b32 v9, a3", "")
    wait = ("s_nop 7", "")
    # the read stands before the product, and follows it by the loop's branch
    loop = [read, wait, product, ("s_cbranch_scc1 65532", "<wide_kernel>")]
    assert [f[2] for f in too_soon(_listing(*loop))[1]] == [2]
    assert too_soon(_listing(*(loop[:3] + [wait, wait, ("s_nop 0", "")] + loop[3:]))) == (1, [])
    # a branch over the wait
    over = [product, ("s_cbranch_scc1 2", "<wide_kernel+0x10>"), wait, wait, read]
    assert [f[2] for f in too_soon(_listing(*over))[1]] == [2]
    # factors
    factor = ("v_mov_b32_e32 v5, v9", "")
    assert [f[2] for f in too_soon(_listing(factor, ("s_nop 0", ""), product))[1]] == [2]
    assert too_soon(_listing(factor, ("s_nop 1", ""), product)) == (1, [])
    assert too_soon(_listing(product, product))[1] == []


def test_no_way_is_too_short(listings):  # noqa: F811
    seen = [too_soon(x) for x in listings]
    assert sum(n for n, _ in seen) > 0
    found = [f for _, part in seen for f in part]
    assert not found, "%d of them, first %s" % (len(found), found[:3])
