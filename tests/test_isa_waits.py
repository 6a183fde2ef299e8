"""Wait states that the hardware leaves to the program, in the built library's own code.

The compiler adds them between its instructions, but not inside an asm string:
  - a load into LDS takes its place from M0, one wait state or more after a scalar
    instruction wrote it;
  - a vector memory instruction reads a scalar register five wait states or more
    after a vector instruction wrote it.
An instruction is one wait state, s_nop n is n + 1."""
import os
import re
import shutil
import subprocess

import pytest

from indexer_topk_long_amd import build as B

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
_SGPR = re.compile(r"\bs\[(\d+):(\d+)\]|\bs(\d+)\b|\b(vcc)\b")
_WRITES_SGPR = ("v_readfirstlane", "v_readlane", "v_cmp")                       # their first operand
_CARRY_OUT = ("v_add_co", "v_sub_co", "v_subrev_co", "v_addc_co", "v_subb_co", "v_subbrev_co", "v_mad_u64", "v_mad_i64",
              "v_div_scale")                                                    # their second one


def _sgprs(text):
    regs = set()
    for a, b, one, vcc in _SGPR.findall(text):
        regs |= set(range(int(a), int(b) + 1)) if a else {int(one)} if one else {vcc}
    return regs


def missing_waits(lines):
    """(copies into LDS, [(kernel, instruction, what)]) of a listing."""
    copies, found, kernel = 0, [], "?"
    since_m0, since = 99, {}
    for line in lines:
        line = line.split("//")[0].strip()
        label = re.match(r"^(?:[0-9a-f]+ )?<(.+)>:", line)
        if label:
            kernel, since_m0, since = label.group(1), 99, {}
            continue
        op, _, rest = line.partition(" ")
        if not re.match(r"^[a-z]+_", op):
            continue
        args = [x.strip() for x in rest.split(",")]
        if op.startswith(("global_", "buffer_", "flat_", "scratch_")):
            if "load_lds" in op or rest.endswith(" lds"):
                copies += 1
                if since_m0 < 1:
                    found.append((kernel, line, "M0"))
            if any(since.get(r, 99) < 5 for r in _sgprs(rest)):
                found.append((kernel, line, "scalar register"))
        states = int(args[0], 0) + 1 if op == "s_nop" else 1
        since_m0 += states
        since = {r: n + states for r, n in since.items() if n + states < 5}
        if op.startswith("s_") and args[0] == "m0":
            since_m0 = 0
        if op.startswith(_WRITES_SGPR):
            since.update(dict.fromkeys(_sgprs(args[0]), 0))
        elif op.startswith(_CARRY_OUT) and len(args) > 1:
            since.update(dict.fromkeys(_sgprs(args[1]), 0))
    return copies, found


@pytest.mark.parametrize("text,bad", [
    ("s_mov_b32 m0, s4|global_load_lds_dwordx4 v1, s[2:3]", 1),
    ("s_mov_b32 m0, s4|s_nop 0|global_load_lds_dwordx4 v1, s[2:3]", 0),
    ("s_add_u32 m0, s4, s5|buffer_load_dword v1, s[4:7], 0 offen lds", 1),
    ("s_mov_b32 m0, s4|v_add_u32_e32 v1, v2, v3|global_load_lds_dword v[1:2], off", 0),
    ("v_readfirstlane_b32 s3, v9|s_nop 3|global_load_dword v1, v2, s[2:3]", 1),
    ("v_readfirstlane_b32 s3, v9|s_nop 4|global_load_dword v1, v2, s[2:3]", 0),
    ("v_readfirstlane_b32 s4, v9|global_load_dword v1, v2, s[2:3]", 0),
])
def test_the_reading_of_listings(text, bad):
    assert len(missing_waits(text.split("|"))[1]) == bad


def test_no_wait_is_missing(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    if not os.path.exists(B.lib_path()):
        B.build()
    lib = shutil.copy(B.lib_path(), tmp_path)        # (its code objects are written beside it)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True)
    objects = [os.path.join(tmp_path, f) for f in sorted(os.listdir(tmp_path)) if f.endswith("gfx950")]
    assert objects
    copies, found = 0, []
    for path in objects:
        listing = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", path], check=True, capture_output=True, text=True)
        n, bad = missing_waits(listing.stdout.splitlines())
        copies, found = copies + n, found + bad
    assert copies > 0
    assert not found, f"{len(found)} places, the first {found[0]}; {copies} copies into LDS"
