"""The block -> unit maps of the expert GEMM launches (xcd_remap and
xcd_remap_dealt in csrc/common.h), compiled for the host with hipcc and run
on the CPU: every unit is taken by exactly one block of the launch's grid,
and the dealt units come first in their XCD's order, at most ceil(n / 8) per
XCD."""
import os
import subprocess

import pytest

from tests import isa_check as ic

pytestmark = pytest.mark.skipif(not os.path.exists(ic.HIPCC), reason="hipcc not installed")

PROGRAM = r"""
#include "common.h"
#include <cstdio>
#include <vector>
// Prints one line per failed case; nothing when every case holds.
int main() {
  const int K = moe::kNumXcd;
  int bad = 0;
  for (int nvalid = 0; nvalid <= 700; ++nvalid) {
    const int lasts[] = {0, 1, 7, 8, 9, 10, 16, 17, nvalid / 2, nvalid};
    for (int nlast : lasts) {
      if (nlast > nvalid) continue;
      for (int extra = 0; extra <= 24; extra += 8) {  // grids built from a larger capacity
        const int cap = nvalid + extra;
        const int plain_grid = (cap + K - 1) / K * K;
        const int dealt_grid = ((cap + K - 1) / K + 1) * K;
        std::vector<int> seen(nvalid, 0), seen2(nvalid, 0);
        std::vector<int> dealt_per_xcd(K, 0);
        for (int b = 0; b < plain_grid; ++b) {
          const int u = moe::xcd_remap(b, nvalid);
          if (u >= nvalid || u < -1) { printf("plain %d %d: %d\n", nvalid, b, u); ++bad; }
          else if (u >= 0) ++seen[u];
        }
        for (int b = 0; b < dealt_grid; ++b) {
          const int u = moe::xcd_remap_dealt(b, nvalid, nlast);
          if (u >= nvalid || u < -1) { printf("dealt %d %d %d: %d\n", nvalid, nlast, b, u); ++bad; continue; }
          if (u < 0) continue;
          ++seen2[u];
          const int xcd = b % K, slot = b / K;
          if (u >= nvalid - nlast) {
            // a dealt unit: before every routed unit of its XCD
            if (slot != dealt_per_xcd[xcd]) { printf("order %d %d %d\n", nvalid, nlast, b); ++bad; }
            ++dealt_per_xcd[xcd];
          }
        }
        for (int u = 0; u < nvalid; ++u)
          if (seen[u] != 1 || seen2[u] != 1) {
            printf("count %d %d %d: %d %d\n", nvalid, nlast, u, seen[u], seen2[u]);
            ++bad;
          }
        for (int x = 0; x < K; ++x)
          if (dealt_per_xcd[x] > (nlast + K - 1) / K) { printf("per xcd %d %d\n", nvalid, nlast); ++bad; }
      }
    }
  }
  return bad ? 1 : 0;
}
"""


def test_block_unit_maps_are_bijections(tmp_path):
    src = tmp_path / "remap.hip"
    src.write_text(PROGRAM)
    exe = tmp_path / "remap"
    subprocess.run([ic.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-I", ic.CSRC,
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[:2000]


PRODUCTS = r"""
#include "product_blocks.h"
#include <cstdio>
#include <vector>
using namespace moe;
// Prints one line per failed case; nothing when every case holds.
static int bad = 0;

// Weight gradients of ragged groups: every (range, group, tile) once.
void dealt(int G, int F, int K, int splits) {
  ProductArgs p{};
  int32_t some = 0;
  float out = 0;
  p.offsets = &some;
  p.y = &out;
  p.P = 1000, p.G = G, p.K = K, p.F = F, p.splits = splits, p.slices = 1, p.cus = 256;
  const int tiles = G * ((F + 127) / 128) * ((K + 255) / 256);
  const int grid = static_cast<int>(grid_of<kWeightGrad, Half<kWeightGrad>>(&p));
  std::vector<int> seen(tiles * splits, 0);
  for (int b = 0; b < grid; ++b) {
    const int u = dealt_unit(b, run_of(F, 128), tiles * splits);
    if (u >= 0) ++seen.at(u);
  }
  for (size_t u = 0; u < seen.size(); ++u)
    if (seen[u] != 1) { printf("dealt %d %d %d %d: %zu %d\n", G, F, K, splits, u, seen[u]); ++bad; }
}

// Big tiles with the last round's cut: every whole tile once, every slice of a cut one.
void cut(int rows, int cols, int cus, int slices) {
  ProductArgs p{};
  p.P = rows * 256 - 5, p.G = 1, p.K = 64, p.F = cols * 256 - 8;
  p.splits = 1, p.slices = slices, p.cus = cus;
  const int units = rows * cols;
  const int grid = static_cast<int>(grid_of<kForward, Big<kForward>>(&p));
  const int first = kNumXcd * (p.whole / kNumXcd);
  if (p.whole % cus || first > p.whole || units - p.whole >= cus) { printf("whole\n"); ++bad; }
  std::vector<int> seen(units * slices, 0);
  for (int b = 0; b < grid; ++b) {
    int part = -1;
    const int u = cut_unit(b, first, units, slices, &part);
    if (u >= 0) ++seen.at(u * slices + part);
  }
  for (int u = 0; u < units; ++u)
    for (int i = 0; i < slices; ++i)
      if (seen[u * slices + i] != (u < first ? i == 0 : 1)) {
        printf("cut %d %d %d %d: %d %d\n", rows, cols, cus, slices, u, seen[u * slices + i]);
        ++bad;
      }
}

int main() {
  for (int G : {1, 2, 7, 48, 288})
    for (int tiles = 1; tiles <= 9; ++tiles)
      for (int K : {8, 256, 264, 1288})
        for (int splits : {1, 2, 4, 8, 32, 512}) dealt(G, 128 * tiles - 8, K, splits);
  for (int cus : {256, 304, 252, 100, 64, 7, 1})
    for (int rows = 1; rows <= 40; ++rows)
      for (int cols : {1, 2, 3, 5, 9, 17, 44})
        for (int slices : {2, 4}) cut(rows, cols, cus, slices);
  return bad ? 1 : 0;
}
"""


def test_product_unit_maps_are_bijections(tmp_path):
    """The linear and grouped products' maps (csrc/product_blocks.h), over the
    grids that their launches take (CUs that the XCDs do not divide included)."""
    src = tmp_path / "products.hip"
    src.write_text(PRODUCTS)
    exe = tmp_path / "products"
    subprocess.run([ic.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-I", ic.CSRC,
                    "-I", ic.INCLUDE, str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout[:2000]
