"""Wait states in the built gfx950 code around direct loads to LDS.

The CDNA ISA documents leave two distances to software: one wait state between
a scalar instruction that writes M0 and a load to LDS (which takes its LDS
address from M0), and five between a vector instruction that writes a scalar
register and a memory instruction that reads it.  The compiler keeps them for
its own instructions; these loads are written in asm, where it does not look.
The test reads liblh.so's own code objects back; no GPU is needed."""
import os
import re
import struct
import subprocess
import tempfile

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "nvfp4_scale_calibration_amd", "liblh.so")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

pytestmark = pytest.mark.skipif(not os.path.exists(OBJDUMP), reason="no llvm-objdump")


def code_objects(path):
    """The gfx950 code objects of a library: every offload bundle's entries."""
    data = open(path, "rb").read()
    found = []
    for m in re.finditer(re.escape(MAGIC), data):
        entries, at = struct.unpack_from("<Q", data, m.start() + 24)[0], m.start() + 32
        if not 1 <= entries <= 8:
            continue  # the magic as a string, not a bundle
        for _ in range(entries):
            off, size, n = struct.unpack_from("<QQQ", data, at)
            if b"gfx950" in data[at + 24:at + 24 + n] and size:
                found.append(data[m.start() + off:m.start() + off + size])
            at += 24 + n
    return found


def instructions(blob):
    """Instructions in order, None where a function starts."""
    with tempfile.NamedTemporaryFile(suffix=".co") as f:
        f.write(blob)
        f.flush()
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", f.name], check=True, capture_output=True,
                              text=True).stdout
    for line in text.split("\n"):
        if line.startswith("\t"):
            yield line.split("//")[0].strip()
        elif line.endswith(">:"):
            yield None


def scalars(operand):
    """The numbers of the scalar registers that an operand names."""
    m = re.fullmatch(r"s(\d+)", operand)
    if m:
        return {int(m.group(1))}
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    return {"vcc"} if operand == "vcc" else set()


def operands(ins):
    return [o.strip().split(" ")[0] for o in ins.split(" ", 1)[1].split(",")] if " " in ins else []


def writes_m0(ins):
    return ins.startswith("s_") and operands(ins)[:1] == ["m0"]


def vector_writes(ins):
    """Scalar registers written by a vector instruction (its first two operands can be results)."""
    if not ins.startswith("v_"):
        return set()
    ops = operands(ins)
    first = scalars(ops[0]) if ops else set()
    second = scalars(ops[1]) if len(ops) > 1 and re.match(r"v_(add_co|sub_co|subrev_co|addc_co|subb_co|subbrev_co|mad_u64|mad_i64|div_scale)", ins) else set()
    return first | second


def wait_states(ins):
    return int(operands(ins)[0], 0) + 1 if ins.startswith("s_nop") else 1


def faults(stream):
    """(number of direct loads, those that come too early)."""
    loads, early, recent = 0, [], []
    for ins in stream:
        if ins is None:
            recent = []
            continue
        if "_load_lds_" in ins:
            loads += 1
            if recent and writes_m0(recent[-1]):
                early.append((recent[-1], ins))
            reads = set().union(*(scalars(o) for o in operands(ins)))
            distance = 0
            for before in reversed(recent):
                if distance >= 5:
                    break
                if vector_writes(before) & reads:
                    early.append((before, ins))
                distance += wait_states(before)
        recent = (recent + [ins])[-8:]
    return loads, early


def test_the_reading_itself():
    good = ["s_mov_b32 m0, s4", "s_nop 0", "global_load_lds_dwordx4 v1, s[2:3]", "s_add_i32 m0, s5, 0x400",
            "v_add_u32_e32 v3, v4, v5", "global_load_lds_dword v[6:7], off", "v_readfirstlane_b32 s8, v1", "s_nop 4",
            "global_load_lds_ubyte v1, s[8:9] offset:16"]
    assert faults(iter(good)) == (3, [])
    assert len(faults(iter(["s_mov_b32 m0, s4", "global_load_lds_dwordx4 v1, s[2:3]"]))[1]) == 1
    assert len(faults(iter(["v_readfirstlane_b32 s3, v1", "s_nop 3", "global_load_lds_dwordx4 v1, s[2:3]"]))[1]) == 1
    assert len(faults(iter(["v_mad_u64_u32 v[2:3], s[2:3], v4, s8, 0", "global_load_lds_dwordx4 v1, s[2:3]"]))[1]) == 1
    assert faults(iter(["s_mov_b32 m0, s4", None, "global_load_lds_dwordx4 v1, s[2:3]"])) == (1, [])


def test_direct_loads_keep_their_distance():
    if not os.path.exists(LIB):
        import nvfp4_scale_calibration_amd._build as b
        b.build()
    total, early = 0, []
    for blob in code_objects(LIB):
        loads, bad = faults(instructions(blob))
        total, early = total + loads, early + bad
    assert total > 0, "no direct loads found: the code was not read"
    assert not early, "%d of %d direct loads come too early: %s" % (len(early), total, early[:4])
