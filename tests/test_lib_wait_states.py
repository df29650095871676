"""The built kernels' code, on the CPU: a vector instruction that writes a
scalar register needs five wait states before a memory instruction reads that
register (the compiler sees to it for its own instructions, not for those in
inline assembly)."""

import os
import re
import shutil
import subprocess

import pytest

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
NEEDED = 5


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    import lossless_entropy_coding_amd as ec
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    if not os.path.exists(ec.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    d = tmp_path_factory.mktemp("code")
    lib = shutil.copy(ec.LIB_PATH, d / "lib.so")
    subprocess.run([OBJDUMP, "--offloading", lib], cwd=d, check=True, capture_output=True)
    objects = sorted(p for p in d.iterdir() if p.name.endswith("gfx950"))
    assert objects
    return [subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", str(p)], check=True, capture_output=True,
                           text=True).stdout for p in objects]


def scalars(operand):
    """The scalar registers that an operand names."""
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return [int(m.group(1))]
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    return list(range(int(m.group(1)), int(m.group(2)) + 1)) if m else []


def short_waits(listing):
    """(function, instruction, wait states) of every memory instruction that follows too soon."""
    found, function, written, at = [], "", {}, 0
    for line in listing.splitlines():
        m = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if m:
            function, written = m.group(1), {}
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        op, _, rest = text.partition(" ")
        operands = [v.strip() for v in re.split(r",|\s", rest) if v.strip()]
        if op.startswith(("buffer_", "global_", "flat_", "scratch_")):
            for r in {r for v in operands for r in scalars(v)}:
                if r in written and at - written[r] < NEEDED:
                    found.append((function, text, at - written[r]))
        wait = int(operands[0], 0) + 1 if op == "s_nop" else 1
        at += wait
        if op.startswith("v_") and operands:
            outs = operands[:1] + (operands[1:2] if "_co_" in op or "div_scale" in op else [])
            for r in (r for v in outs for r in scalars(v)):
                written[r] = at
        elif op.startswith("s_") and operands:
            for r in scalars(operands[0]):      # written again, by the scalar unit
                written.pop(r, None)
        if op in ("s_branch", "s_endpgm", "s_setpc_b64"):
            written = {}
    return found


def test_counting():
    near = "0 <f>:\n\tv_readfirstlane_b32 s6, v1\n\ts_mov_b32 m0, s9\n\ts_nop %d\n\tbuffer_load_dwordx4 v8, s[4:7], 0 offen lds\n"
    assert short_waits(near % 2) == [("f", "buffer_load_dwordx4 v8, s[4:7], 0 offen lds", 4)]
    assert short_waits(near % 3) == []
    assert short_waits((near % 0).replace("s_mov_b32 m0, s9", "s_mov_b32 s6, 0")) == []


def test_memory_instructions_wait_for_their_scalars(listings):
    assert sum(x.count("buffer_load") for x in listings) > 0
    found = [f for x in listings for f in short_waits(x)]
    assert not found, "%d of them, first %s" % (len(found), found[:3])
