"""Every source a profiled kernel is built from is part of the hash its summary
records, and 8-bit MFMA flops are counted."""
import csv
import os
import re

import pytest

from lora_bypass_linear_amd import profsum


def _includes(rel):
    """csrc headers that a source includes, through other headers too."""
    seen, todo = set(), [rel]
    while todo:
        at = todo.pop()
        if at in seen:
            continue
        seen.add(at)
        with open(os.path.join(profsum.HERE, at)) as f:
            todo += ["csrc/" + h for h in re.findall(r'#include "([a-z_0-9]+\.h)"', f.read())]
    return seen


@pytest.mark.parametrize("kind", sorted(profsum.SOURCES))
def test_hash_covers_the_headers(kind):
    assert _includes(profsum.SOURCES[kind][0]) == set(profsum.SOURCES[kind])


def test_every_kernel_file_of_a_profile_has_a_kind():
    mains = {v[0] for v in profsum.SOURCES.values()}
    for name in ("gemm", "hpass", "merge", "fp8gemm", "quant", "ortho"):
        assert f"csrc/{name}.hip" in mains


def test_mfma_flops_of_8_bit_kernels(tmp_path):
    d = tmp_path / "m"
    d.mkdir()
    with open(d / "x_counter_collection.csv", "w", newline="") as f:
        w = csv.writer(f)
        w.writerow(["Dispatch_Id", "Kernel_Name", "Counter_Name", "Counter_Value"])
        for c, v in (("SQ_VALU_MFMA_BUSY_CYCLES", 256000.0), ("SQ_INSTS_VALU_MFMA_MOPS_F8", 4000.0),
                     ("SQ_INSTS_VALU_MFMA_MOPS_F16", 0.0), ("GRBM_GUI_ACTIVE", 8000.0)):
            w.writerow([1, "fp8_gemm_kernel<A>", c, v])
    out = tmp_path / "m.txt"
    profsum.main(["mfma", str(d), "--kernel", "fp8_gemm_kernel", "--cmd", "c", "--out", str(out)])
    kv = dict(line.split(": ", 1) for line in out.read_text().splitlines() if ": " in line)
    assert float(kv["mfma_busy_fraction"]) == 0.25 and float(kv["mfma_flops_per_launch"]) == 4000.0 * 512
