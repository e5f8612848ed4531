"""How the grouped products cut up their work, checked on the host: every k
block of every unit is done once, every row of an expert is in one chunk, and
the shares of cut units are found where their pairs write them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "swiglu_mlp_projection_gb300", "csrc")

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <map>
#include <vector>
#include "grouped_plan.cuh"
using namespace swg;
#define CHECK(c) do { if (!(c)) { printf("failed: %s (case %d)\n", #c, n); return 1; } } while (0)
int main() {
  srand(1);
  for (int n = 0; n < 20000; ++n) {
    Work w{};
    const uint32_t pick[] = {1, 2, 5, 70, 76};
    const uint32_t pairs = pick[rand() % 5];
    w.n_kb = 1 + rand() % (n % 3 ? 224 : 12);
    w.ncg = 1 + rand() % 60;
    w.cut = rand() % 4 != 0;
    w.min_kb = 1 << (rand() % 6);
    const uint32_t chunks = (uint32_t)(rand() % (n % 2 ? 300 : 6));
    const Schedule s = make_schedule(w, chunks, pairs);
    CHECK(s.units == chunks * (uint32_t)w.ncg && s.whole <= s.units && s.units - s.whole < pairs);
    std::vector<int> next(s.units, 0);            // k blocks done, in k order, of cut units
    std::vector<std::vector<uint32_t>> who(s.units), slot(s.units);
    std::vector<char> used(pairs * 2, 0);
    for (uint32_t p = 0; p < pairs; ++p) {
      WorkIter it(s, p);
      uint32_t u;
      int kb0, kb1;
      while (it.next(w, s, pairs, u, kb0, kb1)) {
        CHECK(u < s.units && kb0 == next[u] && kb1 > kb0 && kb1 <= w.n_kb);
        next[u] = kb1;
        if (kb0 == 0 && kb1 == w.n_kb) continue;
        CHECK(u >= s.whole);
        const uint32_t rel = u - s.whole, sl = p * s.q / (uint32_t)w.n_kb == rel ? 0 : 1;
        CHECK(!used[p * 2 + sl]);                 // a pair's slot holds one share
        used[p * 2 + sl] = 1;
        who[u].push_back(p);
        slot[u].push_back(sl);
      }
    }
    std::map<uint32_t, int> firsts;
    for (uint32_t u = 0; u < s.units; ++u) {
      CHECK(next[u] == w.n_kb);
      if (u < s.whole || who[u].empty()) continue;
      const Shares sh = shares_of(w, s, u - s.whole);
      CHECK(sh.count == who[u].size());
      for (uint32_t i = 0; i < sh.count; ++i) {
        CHECK(who[u][i] == sh.first + i);
        CHECK(slot[u][i] == (i == 0 ? sh.slot : 0));
      }
      CHECK(++firsts[sh.first] == 1);             // ... so do the arrival counters
    }
    // rows over chunks
    const int n_max = 32 * (1 + rand() % 8), m = 1 + rand() % 3000, nc = (m + n_max - 1) / n_max;
    int at = 0, first, count, most = 0;
    for (int c = 0; c < nc; ++c) {
      chunk_rows(m, nc, c, &first, &count);
      CHECK(first == at && count >= 0 && count <= n_max);
      if (c == 0) most = count;
      CHECK(count <= most);
      at += count;
    }
    CHECK(at == m);
  }
  printf("ok\n");
  return 0;
}
"""


def test_work_is_covered_once(tmp_path):
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "plan.cu"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "plan")
    r = subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-gencode",
                        "arch=compute_103a,code=sm_103a", str(src), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
