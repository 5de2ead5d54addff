"""The turn of a rotary pair, position times frequency modulo one turn in 64
bits, as the kernels' header computes it: compiled for the host with checks of
signed overflow, against whole numbers of any size."""
import os
import random
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

SOURCE = r"""
#include <cstdio>
#include "kv4_row.cuh"
int main() {
    unsigned long long f;
    long long p;
    while (scanf("%llu %lld", &f, &p) == 2) printf("%llu\n", (unsigned long long)strata::turn_of(f, (int32_t)p));
}
"""


def test_turn_wraps_without_signed_overflow(tmp_path):
    src, exe = tmp_path / "turns.cu", tmp_path / "turns"
    src.write_text(SOURCE)
    checks = ["-Xcompiler", "-fsanitize=signed-integer-overflow", "-Xcompiler", "-fno-sanitize-recover=all"]
    r = subprocess.run([NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", *checks, "-I",
                        os.path.join(ROOT, "bit_quantized_moe_warp_b200", "csrc"), "-o", str(exe), str(src), "-lubsan"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    rng = random.Random(0)
    cases = [(f, p) for f in (1, (1 << 61) + 12345, int((1 << 64) / 6.283185307179586)) for p in
             (0, 1, -1, 6, 7, -8, 131071, 2**31 - 1, -(2**31))]
    cases += [(rng.getrandbits(62), rng.randint(-(2**31), 2**31 - 1)) for _ in range(500)]
    r = subprocess.run([str(exe)], input="\n".join(f"{f} {p}" for f, p in cases), capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert [int(v) for v in r.stdout.split()] == [f * p % (1 << 64) for f, p in cases]
