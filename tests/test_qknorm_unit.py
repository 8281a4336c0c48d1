"""Where the lanes of the query and key norm's kernels read and write, for every width (CPU: the header compiled for the host)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "chunkwise_weight_recurrence_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#define __device__
#define __forceinline__ inline
#include "ttt_qknorm_unit.h"

template <int V, bool HALF> void check(int d, int rot) {
  if (d % V || (HALF && V > 1 && (rot / 2 % V || rot % V))) return;  // these rows take an element a lane
  std::vector<int> of_column(d, 0), of_pair(d / 2 + 1, 0);
  const int nr = HALF ? rot / 2 / V : 0, units = nr + (d - 2 * nr * V + 2 * V - 1) / (2 * V);
  for (int u = 0; u < units + 64; ++u) {  // lanes behind the last unit too
    const ttt::Unit<V, HALF> x(u, d, rot);
    bool ok = x.a >= 0 && x.a <= d && x.b >= x.a && x.b <= d && x.pairs >= 0 && x.pairs <= V && (u < units || (x.a == d && x.pairs == 0));
    for (int v = 0; v < V; ++v) {
      if (x.a < d) ok = ok && x.a + v < d && ++of_column[x.a + v] == 1;
      if (x.b < d) ok = ok && x.b + v < d && ++of_column[x.b + v] == 1;
    }
    for (int p = 0; p < x.pairs; ++p) {
      // the columns that the kernel turns by entry t + p: of one piece each, or neighbours in piece 2 p / V
      int first = HALF ? x.a + p : x.a + 2 * p, second = HALF ? x.b + p : x.a + 2 * p + 1;
      const int j = x.t + p;
      ok = ok && j >= 0 && j < rot / 2 && second < d && ++of_pair[j] == 1;  // no column behind rot is turned
      ok = ok && first == (HALF ? j : 2 * j) && second == (HALF ? j + rot / 2 : 2 * j + 1);
    }
    if (!ok) { std::printf("V %d half %d d %d rot %d unit %d\n", V, HALF, d, rot, u); std::exit(1); }
  }
  for (int c = 0; c < d; ++c)
    if (of_column[c] != 1) { std::printf("V %d half %d d %d rot %d column %d\n", V, HALF, d, rot, c); std::exit(1); }
  for (int j = 0; j < rot / 2; ++j)
    if (of_pair[j] != 1) { std::printf("V %d half %d d %d rot %d pair %d\n", V, HALF, d, rot, j); std::exit(1); }
}

int main() {
  for (int d = 1; d <= 512; ++d)
    for (int rot = 0; rot <= d; rot += 2) {
      check<8, true>(d, rot); check<8, false>(d, rot);
      check<4, true>(d, rot); check<4, false>(d, rot);
      check<1, true>(d, rot); check<1, false>(d, rot);
    }
  std::puts("all");
}
"""


@pytest.mark.skipif(not shutil.which("g++"), reason="needs g++")
def test_every_column_once_and_no_entry_of_another_token(tmp_path):
    src = tmp_path / "unit.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(tmp_path / "unit")], check=True)
    p = subprocess.run([str(tmp_path / "unit")], capture_output=True, text=True)
    assert p.returncode == 0 and p.stdout == "all\n", p.stdout
