"""load_to_lds names M0 as written: a load into LDS that the compiler makes behind it sets M0 again (from the assembly of a kernel
built here; no GPU needed)."""
import os
import re
import subprocess

from extreme_weight_quantization_amd import build

SOURCE = """
#include "aqlm_device.h"
__global__ void mixed(const char* p, uint32_t to) {
    extern __shared__ char lds[];
    __builtin_amdgcn_global_load_lds((const void*)(p + threadIdx.x * 16), aqlm::lds_ptr(lds), 16, 0, 0);
    aqlm::load_to_lds(to, p, threadIdx.x * 16);
    __builtin_amdgcn_global_load_lds((const void*)(p + 4096 + threadIdx.x * 16), aqlm::lds_ptr(lds), 16, 0, 0);
}
"""


def test_m0_is_set_for_every_load(tmp_path):
    src, out = tmp_path / "mixed.hip", tmp_path / "mixed.s"
    src.write_text(SOURCE)
    r = subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-I", build.CSRC, "-S", "--cuda-device-only", str(src), "-o", str(out)],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and os.path.exists(out), r.stderr
    assert "reserved" not in r.stderr
    seen = re.findall(r"s_mov_b32 m0|global_load_lds_dwordx4", out.read_text())
    assert seen == ["s_mov_b32 m0", "global_load_lds_dwordx4"] * 3
