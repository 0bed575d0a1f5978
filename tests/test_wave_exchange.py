"""Lanes of a wave that hand values to each other through LDS: the compiler may not
answer a lane's read with that lane's own last write (CPU; compiles for gfx950)."""
import glob
import os
import re
import subprocess

import pytest

from routing_permute_grouped_moe_amd import build

KERNEL = """
#include "%s/common.hpp"
extern "C" __global__ void exchange(const int* to, float* out) {
  __shared__ float v[64];
  const int lane = threadIdx.x;
  v[lane] = 0.f;
  wave_lds_sync();
  if (to[lane] != lane) v[to[lane]] = 1.f;
  wave_lds_sync();
  out[lane] = v[lane];
}
extern "C" __global__ void own(const float* in, float* out) {
  __shared__ float v[64];
  v[threadIdx.x] = in[threadIdx.x];
  wave_lds_sync();
  out[threadIdx.x] = v[threadIdx.x];
}
"""


def test_every_exchange_is_ordered_for_the_compiler():
    """Whether the barrier of a wave orders memory for the compiler is the compiler's
    affair: it stands in the one helper, between fences, which do."""
    at = []
    for path in sorted(glob.glob(os.path.join(build.CSRC, "*"))):
        with open(path) as f:
            text = f.read()
        at += [(os.path.basename(path), m.start()) for m in re.finditer("builtin_amdgcn_wave_barrier", text)]
        if path.endswith("common.hpp"):
            body = re.search(r"void wave_lds_sync\(\) \{(.*?)\n\}", text, re.S).group(1)
            assert [s.strip() for s in body.strip().splitlines()] == [
                '__builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");',
                "__builtin_amdgcn_wave_barrier();",
                '__builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");']
    assert [name for name, _ in at] == ["common.hpp"], at


@pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no hipcc")
def test_reads_stay_behind_the_exchange(tmp_path):
    src = tmp_path / "exchange.hip"
    src.write_text(KERNEL % build.CSRC)
    out = tmp_path / "exchange.ll"
    subprocess.run([build.HIPCC, *build.FLAGS, "--cuda-device-only", "-emit-llvm", "-S", str(src), "-o",
                    str(out)], check=True, capture_output=True, timeout=110)
    text = out.read_text()
    for name, stores in (("exchange", 2), ("own", 1)):
        body = re.search(r"define [^\n]*@%s\(.*?\n\}" % name, text, re.S).group(0)
        lds = re.findall(r"(load|store) float[^\n]*addrspace\(3\)", body)
        assert lds == ["store"] * stores + ["load"], (name, lds)
