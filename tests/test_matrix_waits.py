"""The built library keeps the wait states behind its matrix instructions on
every path.  The compiler (ROCm 7.2) has left them out where a branch over
predicated loads lies between: the path of the taken branch then reads results
that have not arrived, silently.  No GPU is touched."""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from int4_weight_only_router_amd import build
from tests import matrix_waits as W

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"

# what the compiler made of a fragment's loads under "if (row < rows)"
BRANCH = """
0000000000001000 <kernel>:
\tv_mfma_f32_16x16x32_f16 a[4:7], v[110:113], v[206:209], a[4:7] // 000000001000:
\ts_and_saveexec_b64 s[24:25], s[6:7]                        // 000000001008:
\ts_cbranch_execz 6                                          // 00000000100C: <kernel+0x28>
\tglobal_load_dwordx4 v[134:137], v[138:139], off            // 000000001010:
\tglobal_load_dwordx4 v[122:125], v[138:139], off offset:64  // 000000001018:
\ts_nop 7                                                    // 000000001020:
\ts_nop 0                                                    // 000000001024:
\ts_or_b64 exec, exec, s[24:25]                              // 000000001028:
%s\tv_accvgpr_read_b32 v141, a7                                // 00000000102C:
\ts_endpgm                                                   // 000000001034:
"""


def _short(text):
    (_, code), = W.functions(text)
    return W.shortages(code)


def test_walk_takes_the_branch():
    assert _short(BRANCH % "") == [(0, 8, 3, 8)]
    # enough behind the join, or no branch
    assert _short(BRANCH.replace("102C", "1030") % "\ts_nop 4 // 00000000102C:\n") == []
    straight = "\n".join(l for l in (BRANCH % "").splitlines() if "cbranch" not in l)
    assert _short(straight) == []
    assert _short(straight.replace("s_nop 7", "s_nop 0")) == [(0, 7, 6, 8)]


def test_walk_of_matrix_chains():
    """The accumulator passes on at once; an operand, part of an accumulator, a
    store or an overwriting instruction has to wait."""
    chain = """
0000000000000000 <k>:
\tv_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], 0 // 000000000000:
\t%s // 000000000008:
\ts_endpgm // 000000000010:
"""
    for use, short in (("v_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], v[0:3]", False),
                       ("v_mfma_f32_16x16x32_f16 v[4:7], v[8:11], v[12:15], v[0:3]", False),
                       ("v_mfma_f32_16x16x32_f16 v[4:7], v[0:3], v[12:15], 0", True),
                       ("v_mfma_f32_16x16x32_f16 v[4:7], v[8:11], v[12:15], v[2:5]", True),
                       ("v_mfma_f32_16x16x32_f16 v[2:5], v[8:11], v[12:15], v[0:3]", False),
                       ("v_mov_b32_e32 v2, v20", True), ("v_mov_b32_e32 v20, v3", True),
                       ("global_store_dwordx4 v[30:31], v[0:3], off", True),
                       ("ds_write_b128 v9, v[0:3]", True), ("v_mov_b32_e32 v20, v4", False)):
        assert bool(_short(chain % use)) == short, use


def test_built_library(tmp_path):
    if not build.up_to_date():
        build.build()
    lib = shutil.copy(build.LIB, str(tmp_path / "lib.so"))
    subprocess.run([OBJDUMP, "--offloading", lib], check=True, capture_output=True, cwd=tmp_path)
    parts = sorted(str(p) for p in tmp_path.iterdir() if "gfx950" in p.name and p.stat().st_size)
    assert parts

    def listing(p):
        return subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", p], check=True,
                              capture_output=True, text=True).stdout
    with ThreadPoolExecutor(4) as ex:
        texts = list(ex.map(listing, parts))
    kernels = matrix = 0
    for text in texts:
        for name, code in W.functions(text):
            n = sum(c[0].startswith("v_mfma") for c in code)
            kernels, matrix = kernels + (n > 0), matrix + n
            for i, j, waits, need in W.shortages(code):
                pytest.fail("%s: %s %s, used by %s %s after %d of %d wait states" % (
                    (name,) + code[i][:2] + code[j][:2] + (waits, need)))
    assert kernels > 20 and matrix > 1000 and os.path.basename(lib) == "lib.so"
