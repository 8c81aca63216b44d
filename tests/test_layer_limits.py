"""Index arithmetic of the layer operators where positions pass 32 bits, compiled for the host."""
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_22_amd", "csrc")
ROCM = "/opt/rocm/include"

PROGRAM = r"""
#include <cstdio>
#include "layer_internal.h"
int main() {
  long long t0, t1, len;
  while (std::scanf("%lld %lld %lld", &t0, &t1, &len) == 3) std::printf("%d\n", s6::chunk_tokens(t0, t1, len));
}
"""


def test_the_tokens_of_a_chunk_behind_and_before_the_end_of_its_row(tmp_path):
    if not os.path.exists(os.path.join(ROCM, "hip", "hip_runtime.h")):
        pytest.skip("ROCm headers not found")
    src, exe = tmp_path / "chunk.cpp", tmp_path / "chunk"
    src.write_text(PROGRAM)
    r = subprocess.run(["g++", "-std=c++17", "-w", "-D__HIP_PLATFORM_AMD__", "-I", ROCM, "-I", CSRC, "-I",
                        os.path.join(ROOT, "include"), str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    ends = [0, 1, 5, 31, 32, 33, 2 ** 31 - 1, 2 ** 31, 2 ** 31 + 33, 2 ** 32, 2 ** 32 + 7, 2 ** 40]
    cases = [(t0, t0 + c, n) for e in ends for t0 in {max(0, e + d) // 4 * 4 for d in (-64, -32, -4, 0, 4, 32)}
             for c in (1, 8, 32) for n in ends]
    r = subprocess.run([str(exe)], input="\n".join("%d %d %d" % c for c in cases), capture_output=True, text=True)
    got = [int(v) for v in r.stdout.split()]
    assert len(got) == len(cases)
    for (t0, t1, n), v in zip(cases, got):
        assert v == max(0, min(t1, n) - t0), (t0, t1, n, v)
