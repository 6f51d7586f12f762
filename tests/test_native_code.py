"""The library's own machine code, read without a GPU: what the compiler does not
look after, since the instructions are written by hand."""
import os
import re
import struct
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "combine_moe_dispatch_amd", "lib", "libmoe_ep.so")
LLVM = os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "llvm", "bin")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

# A vector memory instruction may read a scalar register five wait states after a
# vector instruction wrote it (v_readfirstlane and the like), and one after the
# scalar unit wrote m0; the hardware does not hold it back.
AFTER_VECTOR, AFTER_M0 = 5, 1


def device_objects(path, where):
    """Files of the gfx950 code objects of a shared library."""
    section = os.path.join(where, "fatbin")
    subprocess.run([os.path.join(LLVM, "llvm-objcopy"), "--dump-section", f".hip_fatbin={section}", path,
                    os.path.join(where, "copy")], check=True)
    with open(section, "rb") as f:
        data = f.read()
    found = []
    for m in re.finditer(MAGIC, data):
        at = m.start() + len(MAGIC)
        count = struct.unpack_from("<Q", data, at)[0]
        at += 8
        for _ in range(count):
            offset, size, length = struct.unpack_from("<QQQ", data, at)
            at += 24
            triple = data[at:at + length].decode()
            at += length
            if triple.endswith("gfx950") and size:
                name = os.path.join(where, f"{len(found)}.co")
                with open(name, "wb") as f:
                    f.write(data[m.start() + offset:m.start() + offset + size])
                found.append(name)
    return found


def instructions(path):
    """(kernel, its instructions in order) of a code object."""
    text = subprocess.run([os.path.join(LLVM, "llvm-objdump"), "-d", "--no-show-raw-insn", path], check=True,
                          capture_output=True, text=True).stdout
    name, code = None, []
    for line in text.splitlines():
        head = re.match(r"[0-9a-f]+ <(.*)>:", line)
        if head:
            if name:
                yield name, code
            name, code = head[1], []
        elif name and line.strip():
            code.append(line.split("//")[0].strip())
    if name:
        yield name, code


def scalars(operand):
    """Scalar registers that an operand names."""
    operand = operand.strip()
    wide = re.match(r"s\[(\d+):(\d+)\]$", operand)
    if wide:
        return {f"s{i}" for i in range(int(wide[1]), int(wide[2]) + 1)}
    if operand == "vcc":
        return {"vcc_lo", "vcc_hi"}
    return {operand} if re.match(r"s\d+$|vcc_(lo|hi)$|m0$", operand) else set()


def operands(line):
    return re.split(r",\s*|\s+", line.split(None, 1)[1]) if " " in line else []


def states_short(code, at):
    """The register that the memory instruction code[at] reads too early, or None."""
    reads = set().union(*(scalars(o) for o in operands(code[at]))) | {"m0"}
    states = 0
    for line in reversed(code[:at]):
        if states >= AFTER_VECTOR:
            return None
        if line.startswith("v_"):
            first = operands(line)[:2 if "_co_" in line or "div_scale" in line else 1]
            written = set().union(*(scalars(o) for o in first))
            if written & reads:
                return f"{states} wait states behind {line}"
        elif line.startswith("s_") and states < AFTER_M0 and re.match(r"s_\w+ m0,", line):
            return f"{states} wait states behind {line}"
        nop = re.match(r"s_nop (\w+)", line)
        states += int(nop[1], 0) + 1 if nop else 1
    return None if states >= AFTER_VECTOR else f"{states} wait states known"


def test_states_short():
    load = "buffer_load_dwordx4 v1, s[8:11], s4 offen lds"
    assert states_short(["v_readfirstlane_b32 s9, v3", "s_nop 3", load], 2)
    assert states_short(["v_readfirstlane_b32 s4, v3", "s_mov_b32 m0, s2", "s_nop 2", load], 3)
    assert states_short(["v_cmp_lt_i32_e64 s[10:11], v1, v2", "s_nop 3", load], 2)
    assert states_short(["s_nop 4", "s_mov_b32 m0, s2", load], 2)
    assert not states_short(["v_readfirstlane_b32 s9, v3", "s_nop 4", load], 2)
    assert not states_short(["v_readfirstlane_b32 s9, v3", "s_mov_b32 m0, s2", "s_nop 3", load], 3)
    assert not states_short(["s_nop 4", "v_readfirstlane_b32 s12, v9", "s_nop 0", load], 3)


@pytest.mark.skipif(not os.path.exists(os.path.join(LLVM, "llvm-objdump")), reason="no disassembler")
def test_loads_to_lds_wait_for_their_scalars(tmp_path):
    loads, early = 0, []
    for path in device_objects(LIB, str(tmp_path)):
        for name, code in instructions(path):
            for at, line in enumerate(code):
                if re.match(r"buffer_load\S* .*\blds\b", line):
                    loads += 1
                    short = states_short(code, at)
                    if short:
                        early.append(f"{name[:60]}: {line}: {short}")
    assert loads > 0
    assert not early, f"{len(early)} of {loads} loads, e.g. {early[:3]}"
