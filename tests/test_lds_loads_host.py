"""Direct global->LDS loads in the built library keep the wait states that the hardware leaves to the program: one
between a scalar write of m0 and such a load, five between a vector instruction's write of a scalar register and a
load whose address (or m0) it is.  The loads are inline assembly, into which the compiler's own check does not look,
so the code as built is read: without the states a load may take an old m0 (its bytes land elsewhere in LDS) or half
of an old address."""
import os
import re
import struct
import subprocess

import pytest

import moe_w4a16_grouped_amd as moe

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
M0_STATES, BASE_STATES = 1, 5


def code_objects(path):
    """The gfx950 code objects of the library's offload bundles."""
    data, at = open(path, "rb").read(), 0
    while (at := data.find(b"__CLANG_OFFLOAD_BUNDLE__", at)) >= 0:
        count, p = struct.unpack_from("<Q", data, at + 24)[0], at + 32
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            if b"gfx950" in data[p + 24:p + 24 + length] and size:
                yield data[at + offset:at + offset + size]
            p += 24 + length
        at += 24


def scalars(operand):
    m = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if m:
        return {f"s{i}" for i in range(int(m[1]), int(m[2]) + 1)}
    return {operand} if re.match(r"(s\d+|m0)$", operand) else set()


def violations(lines):
    """(loads, faults) of one listing.  Wait states are the instructions between, s_nop n counting n + 1."""
    loads, faults, recent, kernel = 0, [], [], ""
    for line in lines:
        if line.endswith(">:\n"):
            kernel, recent = line.split("<")[1][:-3], []
            continue
        text = line.split("//")[0].strip()
        if not line.startswith("\t") or not text:
            continue
        op, _, rest = text.partition(" ")
        args = [a.strip() for a in rest.split(",")]
        if "load_lds" in op or ("_load_" in op and rest.endswith(" lds")):
            loads += 1
            reads = {"m0"}
            for a in args:
                reads |= scalars(a.split()[0])
            states = 0
            for o, a in reversed(recent):
                if states >= BASE_STATES:
                    break
                if o == "s_nop":
                    states += int(a[0], 0) + 1
                    continue
                wrote = scalars(a[0]) & reads if a[0] else set()
                if wrote and o.startswith("v_"):
                    faults.append((kernel, text, o, states))
                elif "m0" in wrote and states < M0_STATES:
                    faults.append((kernel, text, o, states))
                reads -= wrote
                states += 1
        recent = recent[-8:] + [(op, args)]
    return loads, faults


@pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")
def test_loads_to_lds_keep_their_wait_states(tmp_path):
    loads = 0
    for i, code in enumerate(code_objects(moe.LIB_PATH)):
        path = tmp_path / f"{i}.co"
        path.write_bytes(code)
        with subprocess.Popen([OBJDUMP, "-d", "--no-show-raw-insn", str(path)], stdout=subprocess.PIPE, text=True) as run:
            n, faults = violations(run.stdout)
        assert run.returncode == 0
        assert not faults, (len(faults), faults[:3])
        loads += n
    assert loads > 1000


def test_the_check_itself():
    """Both kinds of fault are found, and the states that mend them are counted."""
    head = ["0000 <kernel>:\n"]

    def faults(*text):
        return len(violations(head + [f"\t{t} // 000\n" for t in text])[1])

    load = "global_load_lds_dwordx4 v1, s[4:5]"
    assert faults("s_mov_b32 m0, s9", load) == 1
    assert faults("s_mov_b32 m0, s9", "s_nop 0", load) == 0
    assert faults("v_readfirstlane_b32 m0, v9", "s_nop 2", load) == 1
    assert faults("v_readfirstlane_b32 s5, v2", "s_nop 3", load) == 1
    assert faults("v_readfirstlane_b32 s5, v2", "s_nop 4", load) == 0
    assert faults("v_readlane_b32 s4, v2, 3", "s_mov_b32 m0, s9", "s_mov_b64 s[4:5], s[6:7]", load) == 0
    assert faults("v_readfirstlane_b32 s7, v2", "s_mov_b64 s[4:5], s[6:7]", load) == 0
    assert faults("v_add_u32 v1, v2, v3", "s_mov_b32 m0, s9", "v_mov_b32 v1, v2", "global_load_lds_dword v[2:3], off") == 0
