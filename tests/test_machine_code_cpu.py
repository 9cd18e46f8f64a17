"""The library's own machine code, disassembled: a scalar register that a vector instruction
writes (a spilled value fetched by v_readlane, say) is read by a vector memory instruction
five wait states later at the earliest. The compiler sees to that among its own
instructions, but not for those inside assembly statements. And in the sources, no assembly
statement changes m0 behind the compiler's back."""
import glob
import os
import re
import shutil
import subprocess

import pytest

from mxfp4_microscaling_quantization_amd import mxq

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
STATES = 5


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{symbol: [instruction, ...]} of every kernel for gfx950."""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    tmp = str(tmp_path_factory.mktemp("code"))
    lib = shutil.copy(mxq.LIB_PATH, tmp)
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp)
    out = {}
    for obj in glob.glob(os.path.join(tmp, "*gfx950")):
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", obj], check=True, capture_output=True, text=True).stdout
        body = None
        for line in text.splitlines():
            head = re.match(r"[0-9a-f]+ <(\S+)>:", line)
            if head:
                body = out.setdefault(head.group(1), [])
            elif body is not None and line.startswith("\t"):
                body.append(line.split("//")[0].strip())
    return out


def registers(operand):
    """Scalar registers of one operand."""
    operand = operand.strip()
    m = re.match(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.match(r"s(\d+)\b", operand)
    if m:
        return {int(m.group(1))}
    m = re.match(r"(m0|vcc)", operand)
    return {m.group(1)} if m else set()


def written(instruction):
    """Scalar registers that a vector instruction writes."""
    op, _, rest = instruction.partition(" ")
    if not op.startswith("v_"):
        return set()
    operands = rest.split(",")
    regs = registers(operands[0])
    if len(operands) > 1 and re.search(r"_co_|div_scale|mad_[iu]64", op):
        regs |= registers(operands[1])
    return regs


def read(instruction):
    """Scalar registers that a vector memory instruction reads; None for other instructions."""
    op, _, rest = instruction.partition(" ")
    if not re.match(r"(buffer|global|scratch|flat)_", op):
        return None
    regs = set().union(*(registers(x) for x in rest.split(",")))
    return regs | {"m0"} if re.search(r"\blds\b", instruction) else regs


def hazards(body):
    found = []
    for i, ins in enumerate(body):
        regs = read(ins)
        if not regs:
            continue
        states, j = 0, i - 1
        while j >= 0 and states < STATES:
            before = body[j]
            if re.match(r"s_(branch|endpgm|setpc)", before):
                break
            if written(before) & regs:
                found.append((states, before, ins))
                break
            nop = re.match(r"s_nop (\d+)", before)
            states += int(nop.group(1)) + 1 if nop else 1
            j -= 1
    return found


def test_the_check_itself():
    load = "buffer_load_dword v4, s[4:7], s1 offen lds"
    assert hazards(["v_readlane_b32 s7, v253, 29", "s_mov_b32 m0, s0", "s_nop 0", load])
    assert hazards(["v_readfirstlane_b32 s1, v0", load]) and hazards(["v_readfirstlane_b32 m0, v0", load])
    assert not hazards(["v_readlane_b32 s7, v253, 29", "s_mov_b32 m0, s0", "s_nop 3", load])
    assert not hazards(["v_readlane_b32 s8, v253, 29", "s_mov_b32 s7, s0", load])
    assert hazards(["v_cmp_lt_i32_e64 s[6:7], v0, v1", "s_nop 3", load])


def test_scalar_registers_of_vector_memory_instructions(kernels):
    assert sum("mm_tile_kernel" in k for k in kernels) >= 36
    assert any(" lds" in ins for body in kernels.values() for ins in body)
    bad = {k: hazards(body) for k, body in kernels.items()}
    bad = {k: v for k, v in bad.items() if v}
    assert not bad, "\n".join(f"{k}: {len(v)}, first after {v[0][0]} wait states: {v[0][1]} | {v[0][2]}"
                              for k, v in bad.items())


def test_assembly_statements_leave_m0_to_the_compiler():
    """m0 is reserved, so a statement cannot name it as clobbered: it may only be an operand."""
    statements = []
    for path in glob.glob(os.path.join(os.path.dirname(mxq.LIB_PATH), "csrc*", "*")):
        statements += re.findall(r"\basm\b[^;]*;", open(path).read())
    loads = [s for s in statements if "buffer_load" in s]
    assert loads and all('"{m0}"' in s for s in loads)
    assert not [s for s in statements if re.search(r"\bm0\b", s.replace('"{m0}"', ""))]
