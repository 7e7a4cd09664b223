"""The tree decode's split (csrc/fa_internal.h), compiled as host code (no GPU): over shapes
and SM counts, the launch fits the workspace sized for it, the merge has a group of blocks
for every pair that can be split and no more groups than a GPU has shares, whatever the
batch, and every split pair is named once by the shares that its parts begin.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "exact_io_aware_16_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "fa_internal.h"
using namespace fa;
static int fail(const char* what, const fa_cache& c, int Hq, int T, int sms) {
  std::printf("%s: B %d Hkv %d cap %d Hq %d T %d sms %d\n", what, c.B, c.Hkv, c.cap, Hq, T, sms);
  return 1;
}
int main() {
  const int sms[] = {1, 2, 100, 148, 152, 160};
  const int Bs[] = {1, 2, 7, 32, 151, 303, 304, 305, 1000, 65536}, Hs[] = {1, 3, 8};
  const int caps[] = {1, 128, 129, 700, 9000}, Gs[] = {1, 5, 16}, Ts[] = {1, 5, 64};
  unsigned seed = 1;
  long long checked = 0, cuts = 0;
  for (int B : Bs) for (int H : Hs) for (int cap : caps) for (int G : Gs) for (int T : Ts) for (int sm : sms) {
    fa_cache c{};
    c.B = B, c.Hkv = H, c.cap = cap, c.d = 64;
    const int Hq = G * H;
    const TreePlan p = tree_plan(c, Hq, T, sm);
    const long long pairs = (long long)B * H;
    const size_t used = (size_t)p.slots * p.prow * (c.d + 1) * 4 + (p.slots ? (size_t)p.shares * 16 : 0);
    if (used > tree_workspace_bytes(c, Hq, T)) return fail("workspace", c, Hq, T, sm);
    ++checked;
    if (!p.slots) continue;
    const int groups = tree_merge_groups(B, H, p.shares);
    if (groups < 1 || groups > pairs || groups > 2 * kTreeMaxSms - 1) return fail("groups", c, Hq, T, sm);
    if (pairs * (cap / 128 + 5) > 20000) continue;
    // the shares of a ragged batch, as the kernel cuts them
    std::vector<int> nt(B);
    int total = 0;
    for (int b = 0; b < B; ++b) {
      seed = seed * 1664525u + 1013904223u;
      nt[b] = 1 + (seed >> 8) % ((cap + 127) / 128);
      total += H * (nt[b] + kTreePairCost);
    }
    const int size = (total + p.shares - 1) / p.shares;
    std::vector<int> named(pairs, 0);
    std::vector<int> split(pairs, 0);
    int u0 = 0;
    for (long long bh = 0; bh < pairs; ++bh) {
      const int n = nt[bh / H], u = u0 + kTreePairCost;
      split[bh] = (u + n - 1) / size - u / size;
      for (int s = 1; s < p.shares; ++s) {  // share s begins behind the pair's first tile
        const int unit0 = s * size < total ? s * size : total;
        if (unit0 < total && unit0 > u && unit0 < u + n && u / size == s - 1) ++named[bh];
      }
      u0 += n + kTreePairCost;
    }
    int cut = 0;
    for (long long bh = 0; bh < pairs; ++bh) {
      if (named[bh] != (split[bh] > 0)) return fail("named", c, Hq, T, sm);
      cut += split[bh] > 0;
    }
    if (cut > groups) return fail("more pairs split than groups", c, Hq, T, sm);
    cuts += cut;
  }
  std::printf("ok %lld %lld\n", checked, cuts);
  return 0;
}
"""


def test_tree_split_fits_its_workspace_and_its_merge(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("nvcc not found")
    src = tmp_path / "split.cu"
    src.write_text(PROGRAM)
    exe = tmp_path / "split"
    subprocess.run([nvcc, "-std=c++17", "-O1", "-I", CSRC, "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True)
    assert out.returncode == 0 and out.stdout.startswith("ok"), out.stdout
