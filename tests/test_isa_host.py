"""Wait states in the library's device code (built here; no GPU needed).

The transfers that go straight from memory to LDS are inline asm, which the compiler's hazard pass does not look into, so
what the hardware leaves to software is checked on the code that was built: between an instruction that writes M0 and a
load to LDS there is at least one other wait state (an `s_nop N` counts N + 1, any other instruction 1), and between a
vector instruction that writes a scalar register and a buffer access that reads it at least five.
"""
import os
import re
import shutil
import struct
import subprocess

import pytest

from post_weight_quantization_05_amd import _lib

LLVM = "/opt/rocm/llvm/bin"
OBJCOPY, OBJDUMP = os.path.join(LLVM, "llvm-objcopy"), os.path.join(LLVM, "llvm-objdump")
MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"

pytestmark = pytest.mark.skipif(
    not (os.path.exists(_lib.LIB_PATH) and os.path.exists(OBJDUMP) and os.path.exists(OBJCOPY)),
    reason="library or disassembler missing")


def _code_objects(blob):
    """The gfx950 code objects of a library's device section: each source's is a bundle of its own."""
    at = blob.find(MAGIC)
    while at >= 0:
        count, = struct.unpack_from("<Q", blob, at + len(MAGIC))
        p = at + len(MAGIC) + 8
        for _ in range(count):
            offset, size, idlen = struct.unpack_from("<QQQ", blob, p)
            name = blob[p + 24: p + 24 + idlen].decode()
            p += 24 + idlen
            if "gfx950" in name and size:
                yield blob[at + offset: at + offset + size]
        at = blob.find(MAGIC, at + len(MAGIC))


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("isa")
    fat = tmp / "fat.bin"
    copy = tmp / "lib.so"
    shutil.copy(_lib.LIB_PATH, copy)
    subprocess.run([OBJCOPY, f"--dump-section=.hip_fatbin={fat}", str(copy), os.devnull], check=True)
    out = []
    for i, code in enumerate(_code_objects(fat.read_bytes())):
        path = tmp / f"{i}.co"
        path.write_bytes(code)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(path)], check=True,
                              capture_output=True, text=True).stdout
        out.append([ln.split("//")[0].strip() for ln in text.splitlines()])
    assert out
    return out


def _states(ins):
    m = re.match(r"s_nop (\d+|0x[0-9a-f]+)", ins)
    return int(m.group(1), 0) + 1 if m else 1


def _scalars(operand):
    """Numbers of the scalar registers of one operand."""
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m.group(1)), int(m.group(2)) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m.group(1))} if m else set()


def _operands(ins):
    return [o.strip() for o in ins.split(None, 1)[1].split(",")] if " " in ins else []


def _before(lines, i, need):
    """The instructions that begin less than `need` wait states before instruction i."""
    states = 0
    while i > 0 and states < need:
        i -= 1
        ins = lines[i]
        if not ins or ins.endswith(":"):
            continue
        yield ins
        states += _states(ins)


def check_m0(lines):
    bad = []
    for i, ins in enumerate(lines):
        if re.match(r"(buffer|global|scratch)_load\w* .*\blds\b", ins) or re.match(r"(buffer|global)_load_lds", ins):
            bad += [(w, ins) for w in _before(lines, i, 1) if re.match(r"s_\w+ m0\b", w)]
    return bad


def check_scalars(lines):
    bad = []
    for i, ins in enumerate(lines):
        if re.match(r"buffer_(load|store|atomic)", ins):
            reads = set().union(*(_scalars(o.split()[0]) for o in _operands(ins) if o))
            for w in _before(lines, i, 5):
                # carries and the like go to a second result
                results = _operands(w)[:2 if re.match(r"v_\w*(_co_|div_scale|_mad_[iu]64)", w) else 1]
                if w.startswith("v_") and any(_scalars(r) & reads for r in results):
                    bad.append((w, ins))
    return bad


def test_the_checks_see_a_missing_wait():
    load = "buffer_load_dwordx4 v1, s[4:7], 0 offen lds"
    assert check_m0(["s_mov_b32 m0, s3", load])
    assert not check_m0(["s_mov_b32 m0, s3", "s_nop 0", load])
    assert check_scalars(["v_readlane_b32 s6, v9, 3", "s_mov_b32 m0, s3", "s_nop 2", load])
    assert not check_scalars(["v_readlane_b32 s6, v9, 3", "s_mov_b32 m0, s3", "s_nop 4", load])
    assert not check_scalars(["v_readlane_b32 s8, v9, 3", load])
    assert check_scalars(["v_add_co_u32_e64 v0, s[4:5], v1, v2", load])


def test_lds_loads_wait_for_m0(listings):
    loads = sum(bool(re.match(r"buffer_load.* lds\b", ins)) for lines in listings for ins in lines)
    assert loads > 100, loads
    for lines in listings:
        bad = check_m0(lines)
        assert not bad, (len(bad), bad[:3])


def test_buffer_accesses_wait_for_their_scalars(listings):
    for lines in listings:
        bad = check_scalars(lines)
        assert not bad, (len(bad), bad[:3])
