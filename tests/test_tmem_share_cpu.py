"""The bound on the tensor memory of CTAs that share an SM (tmem_within), against a search of all sets of them; the
kernels' own static assertions go by it."""

import os
import subprocess

from mxfp8_block_scaled_inv_gb300 import build

PROGRAM = """
#include <cstdio>
#include "mxq_internal.h"
int main() {
  printf("%d %d %d %d\\n", mxq::kCtaSharedReserve, mxq::kLeastShared64, mxq::kLeastShared256, mxq::kLeastShared512);
  for (int room = 0; room <= mxq::kSmSharedBytes; room += 512) printf("%d ", mxq::tmem_within(room));
  printf("\\n%d %d\\n", mxq::tmem_never_short(1, 140 * 1024, 256), mxq::tmem_never_short(2, 100 * 1024, 512));
  for (int s : {0, 43 * 1024 - 1, 43 * 1024, 100 * 1024 - 1, 100 * 1024, 140 * 1024, 227 * 1024})
    printf("%d ", mxq::tmem_allowed(s));
}
"""


def test_against_a_search(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", build.INCLUDE, "-I",
                    os.path.join(build.cuda_home(), "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    reserve, *least = map(int, lines[0].split())
    kinds = [(b + reserve, cols) for b, cols in zip(least, (64, 256, 512))]
    best = {}

    def most(room):
        if room not in best:
            best[room] = max([c + most(room - b) for b, c in kinds if b <= room], default=0)
        return best[room]

    got = list(map(int, lines[1].split()))
    assert got == [most(512 * i) for i in range(len(got))] and len(got) == 457
    assert lines[2] == "1 0"
    assert lines[3].split() == ["0", "0", "64", "64", "256", "512", "512"]
