"""Scalar registers of loads into LDS that are written as instructions.

A vector instruction that writes a scalar register (v_readlane of a spilled
one, v_readfirstlane, a comparison) needs five wait states before a buffer load
reads it. The compiler keeps them for its own loads; it does not look into
inline assembly, whose text has to hold them itself, whatever the compiler puts
in front of it. Checked twice: in the sources, where every such load must stand
behind five wait states of its own block, and in the built library, where
nothing within five wait states of any load into LDS may write a scalar
register that it reads.
"""

import glob
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "combine_route_topk_amd")
OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WAITS = 5


def wait_states(instruction):
    """An instruction is one wait state; s_nop n stands for n + 1."""
    m = re.match(r"s_nop\s+(\w+)", instruction)
    return int(m.group(1), 0) + 1 if m else 1


def asm_blocks():
    """(file, instructions) of the inline assembly that holds a buffer load."""
    for path in sorted(glob.glob(os.path.join(PKG, "csrc", "*.h*"))):
        for block in re.findall(r'\basm\s+volatile\s*\(((?:\s*"(?:[^"\\]|\\.)*")+)', open(path).read()):
            text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', block))
            lines = [l.strip() for l in re.split(r"\\n|\\t|;", text) if l.strip()]
            if any(l.startswith("buffer_load") for l in lines):
                yield os.path.basename(path), lines


def test_hand_written_loads_hold_their_own_wait_states():
    blocks = list(asm_blocks())
    assert len(blocks) >= 2  # load_to_lds and Operand8::load
    for name, lines in blocks:
        first = next(i for i, l in enumerate(lines) if l.startswith("buffer_load"))
        assert all(l.startswith("s_") for l in lines[:first]), (name, lines)
        assert sum(wait_states(l) for l in lines[:first]) >= WAITS, (name, lines)


def scalar_registers(text):
    """Numbers of the scalar registers named in an operand list; vcc as 106 and 107."""
    found = {106, 107} if "vcc" in text else set()
    for a, b in re.findall(r"\bs\[(\d+):(\d+)\]", text):
        found |= set(range(int(a), int(b) + 1))
    return found | {int(n) for n in re.findall(r"\bs(\d+)\b", text)}


def written_by_vector(op, operands):
    """Scalar registers that a vector instruction writes."""
    if not op.startswith("v_"):
        return set()
    first, _, rest = operands.partition(",")
    if op.startswith(("v_readlane", "v_readfirstlane", "v_cmp")):
        return scalar_registers(first) or {106, 107}
    # carries out and division scales: the second operand
    if re.match(r"v_(add_co|sub_co|subrev_co|addc_co|subb_co|subbrev_co|div_scale|mad_u64|mad_i64)", op):
        return scalar_registers(rest.partition(",")[0])
    return set()


def written_by_scalar(op, operands):
    """Scalar registers that a scalar instruction writes, for which the hardware itself waits."""
    if not op.startswith("s_") or op.startswith(("s_cmp", "s_bitcmp")):
        return set()
    return scalar_registers(operands.partition(",")[0])


def test_the_reader_of_listings():
    assert wait_states("s_nop 0") == 1 and wait_states("s_nop 4") == 5 and wait_states("s_add_u32 m0, s1, s2") == 1
    assert scalar_registers("v8, s[24:27], s5 offen lds") == {24, 25, 26, 27, 5}
    assert written_by_vector("v_readlane_b32", "s4, v200, 12") == {4}
    assert written_by_vector("v_cmp_gt_i32_e32", "vcc, 64, v1") == {106, 107}
    assert written_by_vector("v_mad_u64_u32", "v[4:5], s[4:5], v1, s54, v[130:131]") == {4, 5}
    assert written_by_vector("v_lshl_or_b32", "v1, s1, 3, v138") == set()
    assert written_by_vector("s_add_u32", "s4, s5, s6") == set()
    assert written_by_scalar("s_add_u32", "s4, s5, s6") == {4} and written_by_scalar("s_mov_b64", "s[4:5], s[6:7]") == {4, 5}
    assert written_by_scalar("s_cmp_gt_u32", "s0, 0x7f") == set() and written_by_scalar("v_mov_b32_e32", "v0, s1") == set()


def test_no_vector_write_right_before_a_load_into_lds(tmp_path):
    lib = os.path.join(PKG, "libmoe_ep.so")
    if not os.path.exists(lib) or not os.path.exists(OBJDUMP):
        pytest.skip("no built library, or no disassembler")
    copy = str(tmp_path / "lib.so")  # the code objects are unpacked beside it
    shutil.copy(lib, copy)
    subprocess.run([OBJDUMP, "--offloading", copy], cwd=tmp_path, capture_output=True)
    images = glob.glob(copy + ".*gfx950*")
    if not images:
        pytest.skip("the disassembler does not unpack the library's code objects")
    loads = 0
    for image in images:
        dump = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", image], capture_output=True,
                              text=True, check=True).stdout
        recent = []  # of the instructions before, the latest last: (written by vector, by scalar, wait states)
        for line in dump.splitlines():
            parts = line.split("//")[0].strip().split(None, 1)
            if not parts or parts[0].endswith(":"):
                continue
            op, operands = parts[0], parts[1] if len(parts) > 1 else ""
            if op.startswith("buffer_load") and re.search(r"\blds\b", operands):
                loads += 1
                reads, distance = scalar_registers(operands), 0
                for vector, scalar, states in reversed(recent):
                    if distance >= WAITS:
                        break
                    assert not vector & reads, f"{line.strip()}: a scalar register written {distance} wait states before"
                    reads -= scalar  # what was written before that is not what the load reads
                    distance += states
            recent = recent[-8:] + [(written_by_vector(op, operands), written_by_scalar(op, operands),
                                     wait_states(op + " " + operands))]
    assert loads > 1000  # the products' kernels were among them
