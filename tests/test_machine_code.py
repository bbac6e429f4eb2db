"""The built library's machine code against the wait states that the
hardware does not provide by itself.

The LDS DMAs are written in inline assembly, whose inside the compiler's
hazard pass does not see.  Two rules of the instruction set concern them:

  * a scalar write of M0 needs one wait state before a load whose
    destination is LDS (the load takes its LDS address from M0);
  * a scalar register that a vector instruction has written (a read lane, a
    comparison's mask) needs five before a memory instruction reads it.

Every instruction between two others is one wait state, `s_nop n` is n + 1.
"""
import os
import re
import shutil
import struct
import subprocess

import pytest

import mixture_experts_routed_grouped_amd as R

MAGIC = b"__CLANG_OFFLOAD_BUNDLE__"


def _objdump():
    for path in ("/opt/rocm/llvm/bin/llvm-objdump", shutil.which("llvm-objdump")):
        if path and os.path.exists(path):
            return path
    pytest.skip("llvm-objdump not available")


def _code_objects(path):
    """The gfx950 code objects of a library: every offload bundle's entries
    (offset, size, length of the target's name, name)."""
    with open(path, "rb") as f:
        data = f.read()
    out, at = [], data.find(MAGIC)
    while at >= 0:
        (n,), p = struct.unpack_from("<Q", data, at + 24), at + 32
        for _ in range(n if n < 16 else 0):
            offset, size, length = struct.unpack_from("<QQQ", data, p)
            name = data[p + 24:p + 24 + length]
            p += 24 + length
            if b"gfx950" in name and size:
                out.append(data[at + offset:at + offset + size])
        at = data.find(MAGIC, at + 24)
    return out


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """(function, [(mnemonic, operands), ..]) of every function."""
    if not os.path.exists(R.LIB_PATH):
        pytest.skip("librmoe.so is not built")
    tool, tmp, out = _objdump(), tmp_path_factory.mktemp("code"), []
    for i, obj in enumerate(_code_objects(R.LIB_PATH)):
        path = tmp / f"{i}.co"
        path.write_bytes(obj)
        text = subprocess.run([tool, "-d", "--no-show-raw-insn", str(path)], capture_output=True, text=True, check=True).stdout
        for line in text.splitlines():
            if line.endswith(">:"):
                out.append((line.split("<")[1][:-2], []))
            elif line.startswith("\t") and out:
                name, _, operands = line.split("//")[0].strip().partition(" ")
                out[-1][1].append((name, [o.strip() for o in operands.split(",")]))
    return out


def _states(name, operands):
    return int(operands[0]) + 1 if name == "s_nop" else 1


def _to_lds(name):
    return "_load_lds_" in name or (name.startswith("buffer_load") and name.endswith("_lds"))


def test_the_library_holds_lds_dmas(kernels):
    assert sum(_to_lds(n) for _, code in kernels for n, _ in code) > 1000


def test_m0_settles_before_an_lds_dma(kernels):
    bad = []
    for fn, code in kernels:
        for (name, operands), (after, _) in zip(code, code[1:]):
            if operands[0] == "m0" and _to_lds(after):
                bad.append((fn, name, after))
    assert not bad, f"{len(bad)} loads right behind the write of M0, the first in {bad[0]}"


def _scalars(operand):
    """Numbers of the scalar registers that an operand names (vcc as -1)."""
    if operand.startswith("vcc"):
        return {-1}
    m = re.match(r"s\[(\d+):(\d+)\]|s(\d+)\b", operand)
    if not m:
        return set()
    return {int(m[3])} if m[3] else set(range(int(m[1]), int(m[2]) + 1))


def _vector_writes(name, operands):
    """Scalar registers that a vector instruction writes."""
    if name.startswith(("v_readlane", "v_readfirstlane", "v_cmp_")):
        return _scalars(operands[0])
    if "_co_" in name or name.startswith("v_div_scale"):
        return _scalars(operands[1])
    return set()


def test_scalar_registers_settle_before_memory_instructions_read_them(kernels):
    bad = []
    for fn, code in kernels:
        recent = []                                    # (written registers, states passed since), newest last
        for name, operands in code:
            if name.startswith(("global_", "buffer_", "flat_", "scratch_")):
                read = set().union(*map(_scalars, operands))
                bad += [(fn, name, operands, n) for written, n in recent if n < 5 and written & read]
            passed = _states(name, operands)
            recent = [(w, n + passed) for w, n in recent if n + passed < 5]
            if name.startswith("s_"):                  # a scalar instruction's own result is ready at once
                recent = [(w - _scalars(operands[0]), n) for w, n in recent]
            written = _vector_writes(name, operands)
            if written:
                recent.append((written, 0))
            if name in ("s_branch", "s_endpgm"):
                recent = []
    assert not bad, f"{len(bad)} reads too early, the first {bad[0]}"
