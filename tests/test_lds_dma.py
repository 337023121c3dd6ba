"""Wait states of the direct global->LDS loads, read from the compiled code (no GPU).

A load that takes its base from SGPRs has to stand five wait states behind a vector
instruction that wrote them (v_readfirstlane of a base that the compiler keeps in vector
registers); behind a scalar one it need not wait. The loads are in asm blocks, where the
compiler does not see them, so the blocks have to hold the waits themselves."""
import os
import re
import subprocess

import pytest

from layer_wise_obs_amd import build

# a base that only a vector register can hold: loaded per lane, the same in all of them
SOURCE = """
#include "lds_dma.h"
#include "x3_pipe.h"
using namespace th;
extern "C" __global__ void one(const uint64_t* at, float* out) {
  __shared__ __attribute__((aligned(1024))) unsigned char sm[1024];
  lds_dma1(threadIdx.x * 16, (const void*)at[threadIdx.x], lds_address(sm));
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  out[threadIdx.x] = ((float*)sm)[threadIdx.x];
}
extern "C" __global__ void ten(const uint64_t* at, float* out) {
  __shared__ __attribute__((aligned(1024))) unsigned char sm[40960];
  const unsigned vo[5] = {threadIdx.x, threadIdx.x, threadIdx.x, threadIdx.x, threadIdx.x};
  lds_dma10s(vo, (const void*)at[threadIdx.x], (const void*)at[threadIdx.x + 64], sm);
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  out[threadIdx.x] = ((float*)sm)[threadIdx.x];
}
extern "C" __global__ void twelve(const uint64_t* at, float* out) {
  __shared__ __attribute__((aligned(1024))) unsigned char sm[49152];
  unsigned vo[12];
  for (int i = 0; i < 12; ++i) vo[i] = threadIdx.x;
  x3d::dma12s(vo, (const void*)at[threadIdx.x], sm);
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  out[threadIdx.x] = ((float*)sm)[threadIdx.x];
}
"""


def _sgprs(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]|s(\d+)", operand)
    if not m:
        return set()
    return set(range(int(m[1]), int(m[2]) + 1)) if m[1] else {int(m[3])}


def _loads(asm):
    """[(kernel, wait states since a vector instruction wrote the base)] of every load; 99
    where a scalar one wrote it."""
    out, kernel, code = [], None, []
    for line in asm.splitlines():
        line = line.split(";")[0].strip()
        if re.fullmatch(r"\w+:", line) and line[:-1] in ("one", "ten", "twelve"):
            kernel, code = line[:-1], []
        elif line and line[0] != "." and not line.endswith(":") and kernel:
            op, _, rest = line.partition(" ")
            args = [a.strip() for a in rest.split(",")]
            if op == "global_load_lds_dwordx4":
                waits = 0
                for o, a in reversed(code):
                    if o[:2] in ("v_", "s_") and _sgprs(a[0]) & _sgprs(args[1]):
                        out.append((kernel, waits if o[0] == "v" else 99))
                        break
                    waits += int(a[0]) + 1 if o == "s_nop" else 1
            code.append((op, args))
    return out


def test_bases_written_by_vector_instructions_are_waited_for(tmp_path):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    src, asm = tmp_path / "loads.hip", tmp_path / "loads.s"
    src.write_text(SOURCE)
    subprocess.run([build.HIPCC, *build.FLAGS, "-I", build.CSRC, "--cuda-device-only", "-S", str(src),
                    "-o", str(asm)], check=True, capture_output=True)
    loads = _loads(asm.read_text())
    assert [k for k, _ in loads].count("one") == 1
    assert [k for k, _ in loads].count("ten") == 10 and [k for k, _ in loads].count("twelve") == 12
    assert min(w for _, w in loads) >= 5, loads
