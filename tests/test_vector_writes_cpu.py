"""The built library's device code writes memory through vector instructions
alone: every instruction that stores, adds to memory or empties a cache is of
a family that does. (CPU only: the library's own code objects are
disassembled, nothing runs.)"""
import os
import re
import shutil
import subprocess

import pytest

import sample_gradient_clipping_layer_amd as dpc

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"
WRITES = re.compile(r"store|atomic|cache|scratch|wb")
VECTOR = re.compile(r"(global|flat|buffer|ds|scratch)_")


def _others(mnemonics):
    """Those that write, by their names, and are of no vector family."""
    return sorted({m for m in mnemonics if WRITES.search(m) and not VECTOR.match(m)})


def _mnemonics(listing):
    return set(re.findall(r"^[ \t]+([a-z]\w+)", listing, flags=re.M))


def test_the_built_library_writes_by_vector_instructions(tmp_path):
    if not os.path.exists(OBJDUMP):
        pytest.skip("llvm-objdump not available")
    if not os.path.exists(dpc.LIB_PATH):
        pytest.fail("libdpclip.so is not built (run __graft_entry__.build())")
    lib = shutil.copy(dpc.LIB_PATH, tmp_path / "lib.so")  # the code objects are written beside it
    subprocess.run([OBJDUMP, "--offloading", str(lib)], check=True, capture_output=True, timeout=120)
    objects = sorted(tmp_path.glob("lib.so.*gfx950"))
    csrc = os.path.join(os.path.dirname(dpc.LIB_PATH), "csrc")
    kernels = [n for n in os.listdir(csrc) if n.endswith(".hip") and "__global__" in open(os.path.join(csrc, n)).read()]
    assert len(objects) >= len(kernels) > 0  # one of every source with a kernel
    met = set()
    for o in objects:
        run = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--no-leading-addr", str(o)], check=True,
                             capture_output=True, text=True, timeout=120)
        met |= _mnemonics(run.stdout)
    assert not _others(met)
    assert {"global_load_dwordx4", "global_store_dwordx4", "s_endpgm", "v_mfma_f32_32x32x16_bf16"} <= met


def test_another_family_is_found():
    listing = "0000 <k>:\n\tglobal_store_dword v0, v1, s[0:1]\n\tx_store_dword x0, x1\n  s_nop 0\n\tx_cache_wb\n\tds_write_b32 v0, v1\n"
    assert _mnemonics(listing) == {"global_store_dword", "x_store_dword", "s_nop", "x_cache_wb", "ds_write_b32"}
    assert _others(_mnemonics(listing)) == ["x_cache_wb", "x_store_dword"]
