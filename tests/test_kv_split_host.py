"""How an attention call is split into launches (host arithmetic, no GPU): each (sequence, KV head, row block) in exactly one launch, and no
launch with 2^31 tiles or more, which the kernels count in 32 bits. Compiled with nvcc for the host; skipped without it."""
import os
import subprocess

import pytest

from test_fold_layout_host import CSRC, ROOT, _nvcc

PROBE = r'''
#include <cstdio>
#include <vector>

#include "kv_attend.cuh"
using namespace pace::kv;
int main() {
  // heads, row blocks, batch, columns of the table, tokens a page, tokens a tile
  const long cases[][6] = {{8, 1, 64, 64, 64, 32},   {2, 17, 3, 1 << 18, 4096, 64}, {1, 1 << 17, 2, 1 << 15, 32, 32}, {8, 65536, 1, 1 << 20, 64, 32},
                           {256, 1, 2, 1 << 25, 32, 32}, {256, 32, 1, 1 << 18, 4096, 64}, {1, 64, 5, 1 << 25, 32, 32}, {1, 63, 1, 1 << 25, 32, 32}};
  for (const auto &c : cases) {
    AttendArgs a{};
    a.c.Hkv = (int)c[0], a.row_blocks = (int)c[1], a.c.batch = (int)c[2], a.c.table_cols = (int)c[3], a.c.page = (int)c[4];
    a.c.n_tokens = 1;
    const long all = c[0] * c[1];
    std::vector<int> seen(all * c[2], 0);
    long longest = 0, launches = 0;
    bool apart = true;
    by_batches(a, (int)c[5], [&](const AttendArgs &p, long line) {
      ++launches;
      longest = std::max(longest, line);
      const long b0 = p.c.lens - a.c.lens;
      apart = apart && p.c.table - a.c.table == b0 * c[3] && (p.items == all || p.c.batch == 1);
      for (long b = b0; b < b0 + p.c.batch; ++b)
        for (long i = p.item0; i < (long)p.item0 + p.items; ++i) seen[b * all + i] += 1;
      return cudaSuccess;
    });
    bool once = true;
    for (int n : seen) once = once && n == 1;
    std::printf("%ld %ld %d %d\n", longest, launches, (int)once, (int)apart);
  }
  return 0;
}
'''


def test_launches_cover_each_item_once_and_stay_in_32_bits(tmp_path):
    nvcc = _nvcc()
    if nvcc is None:
        pytest.skip("nvcc not available")
    src, exe = tmp_path / "probe.cu", tmp_path / "probe"
    src.write_text(PROBE)
    r = subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-I", CSRC, "-I", os.path.join(ROOT, "include"),
                        str(src), "-o", str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    rows = [[int(x) for x in line.split()] for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines()]
    assert len(rows) == 8
    for longest, launches, once, apart in rows:
        assert 0 < longest < 2 ** 31 and once and apart
    assert rows[0][1] == 1 and rows[-1][1] == 1          # (ordinary calls, and the largest that fits, are one launch)
