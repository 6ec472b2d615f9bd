"""Which entries of a caller's column lists the tiered GEMV reads, on the host: csrc/list_share.h,
which the kernels go by, walked over every chunk, wave and lane.  A list may end with its last
entry, so each entry that counts is read once by one wave and nothing else is."""

import os
import subprocess

import pytest

from oracle import tiers as otiers
from tests.test_gpu_parity import GEMV_CASES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "activation_sparse_tiered_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "list_share.h"
// argv: tiles, chunks, the two lists' entries; 64 lanes, 8 waves
int main(int argc, char** argv) {
  const int chunks = atoi(argv[1]), n[2] = {atoi(argv[2]), atoi(argv[3])};
  std::vector<int> reads[2];
  for (int i = 0; i < 2; ++i) reads[i].assign(n[i], 0);
  for (int c = 0; c < chunks; ++c)
    for (int w = 0; w < 8; ++w) {
      const spax::gemv::ListShare share(c, chunks, w, 8);
      const int mine[2] = {share.count(n[0]), share.count(n[1])};
      for (int p0 = 0; p0 < mine[0] || p0 < mine[1]; p0 += 64)
        for (int lane = 0; lane < 64; ++lane)
          for (int i = 0; i < 2; ++i) {
            const int e = share.entry(p0 + lane, mine[i]);
            if (e >= n[i]) return printf("entry %d of %d\n", e, n[i]), 1;
            if (e >= 0) ++reads[i][e];
          }
    }
  for (int i = 0; i < 2; ++i)
    for (int e = 0; e < n[i]; ++e)
      if (reads[i][e] != 1) return printf("entry %d read %d times\n", e, reads[i][e]), 1;
  return 0;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("list_reads")
    src, exe = d / "walk.cpp", d / "walk"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", str(exe)], check=True)
    return lambda *a: subprocess.run([str(exe), *map(str, a)], capture_output=True, text=True)


def _chunks(d_in):
    return sorted({1, 2, 3, max(1, d_in // 16), min(64, max(1, d_in // 16))})


@pytest.mark.parametrize("case", GEMV_CASES, ids=[f"{i}" for i in range(len(GEMV_CASES))])
def test_only_entries_that_count_are_read(walk, case):
    d_in, _, _, _, pf, pa = case
    for chunks in _chunks(d_in):
        r = walk(chunks, *otiers.counts_from_fractions(d_in, pf, pa))
        assert r.returncode == 0, (chunks, r.stdout)


@pytest.mark.parametrize("n", [(0, 0), (0, 1), (1, 0), (7, 4096), (511, 513), (32768, 0)])
@pytest.mark.parametrize("chunks", [1, 5, 64, 1024])
def test_lists_of_any_length(walk, n, chunks):
    r = walk(chunks, *n)
    assert r.returncode == 0, r.stdout
