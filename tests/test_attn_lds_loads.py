"""The loads into LDS that attn_device.hpp writes out set m0; the compiler has to know.  A kernel in
which its own loads into LDS stand around one of them is compiled (not run): after the written-out load
the base of the next is set again."""
import os
import re
import subprocess

import pytest

from gated_delta_rule_60_amd import build

SOURCE = """
#include <hip/hip_runtime.h>
#include "attn_device.hpp"
using namespace kda;
__device__ __forceinline__ void known(const char* p, char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)p, (KDA_LDS void*)lds, 4, 0, 0);
#endif
}
__global__ void probe(const char* p, float* out, int at) {
    __shared__ __attribute__((aligned(1024))) char lds[8192];
    const int lane = threadIdx.x;
    known(p + 4 * lane, lds + at);
    LOAD(buffer_rsrc(p, 4096), lds + 4096, 16 * lane, 0);
    known(p + 2048 + 4 * lane, lds + at);
    lds_ready();
    out[lane] = reinterpret_cast<float*>(lds)[lane];
}
"""


@pytest.mark.parametrize("load,written_out", [("load_lds16", "buffer_load_dwordx4"), ("load_lds4", "buffer_load_dword ")])
def test_m0_is_set_again_after_a_written_out_load(tmp_path, load, written_out):
    if not os.path.exists(build.hipcc()):
        pytest.skip("no compiler here")
    src, asm = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(SOURCE)
    subprocess.run([build.hipcc(), "-S", "--cuda-device-only", "-O3", "-std=c++17", f"--offload-arch={build.ARCH}",
                    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", f"-DLOAD={load}",
                    "-I", os.path.join(os.path.dirname(build.__file__), "csrc"), str(src), "-o", str(asm)],
                   check=True, capture_output=True)
    lines = [x.strip() for x in asm.read_text().splitlines()]
    mine = next(i for i, x in enumerate(lines) if x.startswith(written_out) and x.endswith("lds"))
    after = next(i for i in range(mine + 1, len(lines)) if lines[i].startswith("global_load_lds"))
    assert any(x.startswith("global_load_lds") for x in lines[:mine])
    assert any(re.match(r"s_\w+ m0,", x) for x in lines[mine + 1:after]), "\n".join(lines[mine - 8:after + 1])
