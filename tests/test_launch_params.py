"""Parameters of launches whose parts are optional: one that its caller fills in
only in part asks for nothing else."""
import os
import shutil
import subprocess

import pytest

from lora_bypass_linear_amd import build

PROGRAM = r"""
#include <cstdio>
#include <cstring>
#include <new>
#include "kernels.h"

int main() {
    alignas(lyc::PrepParams) static unsigned char raw[sizeof(lyc::PrepParams)];
    std::memset(raw, 0x5A, sizeof raw);
    const lyc::PrepParams* p = new (raw) lyc::PrepParams;   // as `lyc::PrepParams p;` on a used stack
    const bool idle = p->r_pad == 0 && p->up_blocks == 0 && p->uc == nullptr && p->flagged == nullptr &&
                      p->down == nullptr && p->up == nullptr && p->dc == nullptr && p->dh == nullptr &&
                      p->dl == nullptr && p->dnorm == nullptr && p->N == 0 && p->K == 0 && p->rank == 0 &&
                      p->vec == 0 && p->c_dt == 0 && p->down_dt == 0 && p->up_dt == 0 && p->cast_n[0] == 0 &&
                      p->cast_n[1] == 0;
    std::printf("%s\n", idle ? "idle" : "garbage");
    return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_a_fresh_preparation_does_nothing(tmp_path):
    src, exe = tmp_path / "fresh.cpp", tmp_path / "fresh"
    src.write_text(PROGRAM)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(build.hipcc())))
    # (no dead-store elimination over the object's start: what was in its memory is still there)
    cmd = ["g++", "-std=c++17", "-O0", "-fno-lifetime-dse", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
           "-I", "/opt/rocm/include", "-I", os.path.join(build.HERE, "csrc"), "-I", os.path.join(build.ROOT, "include"),
           str(src), "-o", str(exe)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    assert subprocess.run([str(exe)], capture_output=True, text=True).stdout.strip() == "idle"
