"""The built library's machine code against the wait states that the
hardware does not provide by itself.

The LDS DMAs are written in inline assembly, whose inside the compiler's
hazard pass does not see.  This rule of the instruction set concerns them:

  * a scalar write of M0 needs one wait state before a load whose
    destination is LDS (the load takes its LDS address from M0).

Every instruction between two others is one wait state, `s_nop n` is n + 1.
"""
import os
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
