"""The loads that write LDS past the registers (tiles.h), as they are assembled: the register
that holds their address in LDS is written by a scalar instruction, after which such a load
needs one wait state, and the compiler has to know that it changed (no GPU)."""
import os
import re
import shutil
import subprocess

import pytest

from post_weight_quantization_layer_amd import build as LB

pytestmark = pytest.mark.skipif(
    shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"), reason="needs hipcc")

KERNELS = """
#include "tiles.h"
using namespace gptq;
__global__ void copies(const uint8_t *p, uint32_t off, uint32_t lds) {
  copy16_to_lds(p, off * threadIdx.x, lds);
  copy4_to_lds(p, off * threadIdx.x, lds + 1024);
  copy16_to_lds(p + off * threadIdx.x, lds + 2048);
}
__global__ void beside(const uint32_t *p, uint32_t *out) {
  __shared__ uint32_t own[128], other[256];
  auto *at = (__attribute__((address_space(3))) uint32_t *)own;
  __builtin_amdgcn_global_load_lds(p + threadIdx.x, at, 4, 0, 0);
  copy16_to_lds(p + 4 * threadIdx.x, uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) uint32_t *)other)));
  __builtin_amdgcn_global_load_lds(p + 64 + threadIdx.x, at, 4, 0, 0);
  copies_done<0>();
  __syncthreads();
  out[threadIdx.x] = own[threadIdx.x] + other[threadIdx.x];
}
"""


@pytest.fixture(scope="module")
def instructions(tmp_path_factory):
    """Of each kernel, without comments, labels and directives."""
    at = tmp_path_factory.mktemp("copies")
    src, out = at / "copies.hip", at / "copies.s"
    src.write_text(KERNELS)
    r = subprocess.run([LB.hipcc(), *LB.compile_flags(), "--cuda-device-only", "-S", str(src), "-o",
                        str(out)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    got, name = {}, None
    for line in out.read_text().splitlines():
        line = line.split(";")[0].strip()
        start = re.match(r"_Z\d+(copies|beside)\w*:", line)
        if start:
            name = start.group(1)
            got[name] = []
        elif line.startswith("s_endpgm"):
            name = None
        elif name and line and not line.startswith(".") and not line.endswith(":"):
            got[name].append(line)
    return got


def writes_m0(line):
    return re.match(r"s_\w+ m0,", line)


@pytest.mark.parametrize("name,loads", [("copies", 3), ("beside", 3)])
def test_a_wait_state_between_the_address_and_the_load(instructions, name, loads):
    lines = instructions[name]
    at = [i for i, line in enumerate(lines) if re.match(r"global_load_lds_", line)]
    assert len(at) == loads
    for i in at:
        assert not writes_m0(lines[i - 1]), lines[i - 1:i + 1]


def test_the_compiler_sets_its_own_address_again(instructions):
    """Between a copy and the compiler's next load of that kind, which writes elsewhere."""
    lines = instructions["beside"]
    at = [i for i, line in enumerate(lines) if re.match(r"global_load_lds_", line)]
    for before, load in zip([0] + at, at):
        assert any(writes_m0(line) for line in lines[before:load]), lines[before:load + 1]
