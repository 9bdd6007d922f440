"""The direct-to-LDS copies of f8_tile.h write M0 in inline assembly.  Compiled beside the compiler's own
instructions that read M0, each must make the compiler write it anew: otherwise a later copy of its own would go
to the last inline copy's address.  Shown on the assembly of a kernel that is built and not run (no GPU needed)."""

from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from block_quantized_weight_linear_amd import build

COPIES = {
    "f8_copy16": "q8k::f8_copy16(a, 16u * threadIdx.x, lds + 4096)",
    "f8_copy4": "q8k::f8_copy4(a, 4u * threadIdx.x, lds + 4096)",
    "f8_copy4_from": "q8k::f8_copy4_from(reinterpret_cast<const float*>(a) + threadIdx.x, lds + 4096)",
    "f8_copy16_or_zeros": "q8k::f8_copy16_or_zeros(a, 16u * threadIdx.x, threadIdx.x < 40, lds + 4096)",
}
SOURCE = """
#include "f8_tile.h"
extern "C" __global__ void copies(const uint8_t* a, float* out) {
    extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
    typedef __attribute__((address_space(3))) void* Lds;
    typedef __attribute__((address_space(1))) const void* Global;
    const uint32_t lds = q8k::f8_lds_address(smem);
    __builtin_amdgcn_global_load_lds((Global)(a + 16 * threadIdx.x), (Lds)lds, 16, 0, 0);
    %s;
    __builtin_amdgcn_global_load_lds((Global)(a + 8192 + 16 * threadIdx.x), (Lds)lds, 16, 2048, 0);
    q8k::wait_vmcnt_mem<0>();
    __syncthreads();
    out[threadIdx.x] = smem[threadIdx.x];
}
"""


@pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="no hipcc")
@pytest.mark.parametrize("copy", sorted(COPIES))
def test_m0_is_written_again(copy, tmp_path):
    source, out = tmp_path / "copies.hip", tmp_path / "copies.s"
    source.write_text(SOURCE % COPIES[copy])
    cmd = [build._hipcc(), *build.HIP_FLAGS, "-I", build.CSRC, "--offload-device-only", "-S", str(source), "-o", str(out)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    inline, theirs, own = False, False, 0  # inside inline assembly, M0 is an inline copy's, copies of the compiler's own
    for line in out.read_text().splitlines():
        if "#ASMSTART" in line or "#ASMEND" in line:
            inline = "#ASMSTART" in line
        elif re.search(r"\b\w+\s+m0,", line):
            theirs = inline
        elif "_load_lds_" in line and not inline:
            assert not theirs, f"{copy}: a copy of the compiler's own reads the M0 that the inline one wrote"
            own += 1
    assert own == 2
