"""The built kernels' code, on the CPU: where the matrix instructions are
inline assembly the compiler does not wait for their results.  A 32 x 32 x 16
product's are read 18 states after it at the earliest."""

import re

from test_lib_wait_states import listings  # noqa: F401  (a fixture)

NEEDED = 18
KERNELS = "wide_kernel"


def registers(operand):
    m = re.fullmatch(r"([av])(\d+)", operand)
    if m:
        return {(m.group(1), int(m.group(2)))}
    m = re.fullmatch(r"([av])\[(\d+):(\d+)\]", operand)
    return {(m.group(1), i) for i in range(int(m.group(2)), int(m.group(3)) + 1)} if m else set()


def early_reads(listing):
    """(number of matrix instructions, [(function, instruction, states)]) of the kernels."""
    count, found, function, written, at = 0, [], "", {}, 0
    for line in listing.splitlines():
        m = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if m:
            function, written = m.group(1), {}
            continue
        text = line.split("//")[0].strip()
        if KERNELS not in function or not line.startswith("\t") or not text:
            continue
        op, _, rest = text.partition(" ")
        operands = [v.strip() for v in re.split(r",|\s", rest) if v.strip()]
        if op.startswith("v_mfma"):
            count += 1
            written.update((r, at) for r in registers(operands[0]))
        else:
            for r in (r for v in operands for r in registers(v)):
                if r in written and at - written[r] < NEEDED:
                    found.append((function, text, at - written[r]))
        at += int(operands[0], 0) + 1 if op == "s_nop" else 1
    return count, found


def test_counting():
    near = "0 <wide_kernel>:\n\tv_mfma_f32_32x32x16_bf16 a[0:15], v[0:3], v[4:7], a[0:15]\n\ts_nop %d\n\tv_accvgpr_read_b32 v9, a3\n"
    assert early_reads(near % 15)[1] == [("wide_kernel", "v_accvgpr_read_b32 v9, a3", 17)]
    assert early_reads((near % 15).replace("\ts_nop", "\ts_nop 0\n\ts_nop")) == (1, [])
    assert early_reads((near % 0).replace("a3", "a16")) == (1, [])


def test_results_are_waited_for(listings):  # noqa: F811
    seen = [early_reads(x) for x in listings]
    assert sum(n for n, _ in seen) > 0
    found = [f for _, part in seen for f in part]
    assert not found, "%d of them, first %s" % (len(found), found[:3])
