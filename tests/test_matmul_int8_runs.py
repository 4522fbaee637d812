"""The runs of rows that the experts' 8-bit products work through, as the kernels compute
them, compiled for the host (no GPU): every row of an expert once, in runs of at most a
tile, up to the largest number of rows that the call takes."""
import subprocess

from moe_routing_precision_gb300 import _build

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "block/matmul_int8.cuh"

// Items of one tile of each expert: their runs follow one another and end at its last row.
static int check(const std::vector<long long>& ends, int nt, int tiles) {
  const int E = (int)ends.size() - 1;
  std::vector<int> first(E + 1);
  std::vector<int2> rows(E);
  for (int e = 0; e < E; ++e) {
    rows[e] = make_int2((int)ends[e], (int)ends[e + 1]);
    first[e + 1] = first[e] + (int)((ends[e + 1] - ends[e] + nt - 1) / nt);
  }
  const moe::ItemList list = {first.data(), rows.data(), E};
  for (int e = 0; e < E; ++e) {
    const long long len = ends[e + 1] - ends[e];
    const int n = first[e + 1] - first[e], tile = tiles - 1;
    for (int i = 0; i < n; i = i < 3 || i + 4 > n ? i + 1 : i + 1 + (n - 4 - i) / 7) {
      const moe::Item m = list.at((long long)first[e] * tiles + (long long)tile * n + i, tiles);
      if (m.e != e || m.tile != tile || m.n < 1 || m.n > nt) return 1;
      if (i == 0 && m.r0 != ends[e]) return 2;
      if (i == n - 1 && m.r0 + m.n != ends[e + 1]) return 3;
      if (i + 1 < n) {
        const moe::Item o = list.at((long long)first[e] * tiles + (long long)tile * n + i + 1, tiles);
        if (o.r0 != m.r0 + m.n || m.n % 16 != 0) return 4;
      }
    }
    if (len == 0 && n != 0) return 5;
  }
  return 0;
}

int main() {
  const long long most = (1ll << 31) - 1;
  const std::vector<std::vector<long long>> lists = {
      {0, 1}, {0, 129, 129, 130, 386, 1026}, {0, 33, 65, 97, 130}, {0, most}, {0, most - 1},
      {0, most - 200, most}, {0, 100, most}, {0, 2130800000ll}, {0, 2139100000ll},
      {0, 0, (1ll << 30) + 5, most}};
  for (const auto& l : lists)
    for (int nt : {32, 128, 256})
      for (int tiles : {1, 3, 300}) {
        const int r = check(l, nt, tiles);
        if (r) {
          std::printf("%lld rows, runs of %d, %d tiles: %d\n", l.back(), nt, tiles, r);
          return 1;
        }
      }
  std::puts("OK");
}
"""


def test_runs_cover_every_row(tmp_path):
    src = tmp_path / "runs.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "runs"
    r = subprocess.run([_build.nvcc_path(), *_build.ARCH, "-std=c++17", "--expt-relaxed-constexpr",
                        f"-I{_build.INCLUDE}", f"-I{_build.CSRC}", str(src), "-o", str(exe)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "OK", r.stdout
