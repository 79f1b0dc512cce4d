"""The division of the 8-bit product's blocks of K among CTA pairs, and the
scales that each pair asks for, swept on the host: every block belongs to one
pair, and no request leaves its row, those of pairs without a share among them."""

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_convolution_gb300", "csrc")

# Every pair asks for the scales of four blocks before its loop, and in the loop for those of its next four while it
# has them. Where rows hold a multiple of four, a request reads all four; otherwise the first and what the row has
# of the others.
SWEEP = r"""
#include <cstdio>
#include "cc_fp8_shares.h"
using namespace cc;
int main() {
  int empty = 0;
  for (int pairs = 2; pairs <= 4; pairs *= 2)
    for (int kblocks = 1; kblocks <= 4096; ++kblocks) {
      const int share = share_blocks(kblocks, pairs);
      int next = 0;
      for (int p = 0; p < pairs; ++p) {
        const int first = p * share, blocks = blocks_in_share(kblocks, share, first);
        if (blocks > 0 && (first != next || first % 4 != 0)) return std::printf("%d/%d: share %d\n", kblocks, pairs, p), 1;
        next += blocks;
        empty += blocks == 0;
        for (int g = 0; g == 0 || g < blocks; g += 4) {
          const int from = g == 0 ? first_request(blocks, first) : first + g;
          const int last = kblocks % 4 == 0 ? from + 3 : from;
          if (last >= kblocks) return std::printf("%d/%d: pair %d reads scale %d\n", kblocks, pairs, p, last), 1;
          if (blocks > 0 && from != first + g) return std::printf("%d/%d: pair %d asks at %d\n", kblocks, pairs, p, from), 1;
        }
      }
      if (next != kblocks) return std::printf("%d/%d: %d blocks given out\n", kblocks, pairs, next), 1;
    }
  std::printf("%d empty shares\n", empty);
  return 0;
}
"""


@pytest.fixture(scope="module")
def sweep(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("shares")
    (d / "sweep.cpp").write_text(SWEEP)
    subprocess.run([cxx, "-std=c++17", "-O1", "-I", CSRC, "-o", str(d / "sweep"), str(d / "sweep.cpp")], check=True)
    return str(d / "sweep")


def test_every_request_for_scales_stays_in_its_row(sweep):
    run = subprocess.run([sweep], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
    assert int(run.stdout.split()[0]) > 0  # 17 to 24 blocks on four pairs, for one


def test_the_kernel_asks_by_these_rules():
    # a source check: what a pair without a share reads is never used, so that no output shows it
    text = open(os.path.join(CSRC, "gemm_fp8.cu")).read()
    assert "load_ahead(SPLIT ? first_request(kbs, kb0) : 0);" in text
    requests = [line.strip() for line in text.splitlines() if "load_ahead(" in line]
    assert requests == ["load_ahead(SPLIT ? first_request(kbs, kb0) : 0);", "load_ahead(kb0 + kb + 4);", "load_ahead(0);"]
    assert "const int kbs = SPLIT ? blocks_in_share(args.kblocks, args.kb_split, kb0) : 0;" in text
    assert "const int blocks = share_blocks(args.kblocks, next);" in text
