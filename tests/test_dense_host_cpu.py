"""Host-side rules of the dense kernels, compiled from their header: no GPU."""
import subprocess

import pytest

TURNS = r"""
#include <cstdio>
#include "dense_common.cuh"
using namespace msa;
// Items of up to 2^24 tiles until 2^34 tiles have gone by: the count that the kernels keep names
// the place and phase of the full count in every ring, and stays behind the first filling.
int main() {
  for (int ring : {1, 2, 3, 4, 5, 8}) {
    for (int most : {1 << 24, (1 << 24) - 7, 1999993}) {
      long long all = 0;
      int x = 0;
      uint32_t r = 1;
      while (all < (1ll << 34)) {
        r = r * 1664525u + 1013904223u;
        const int n = most - (int)(r >> 12);  // the last 2^20 lengths below `most`
        all += n;
        x = dense_turn(x + n);
        if (x < 0 || x > (1 << 30) || all % ring != x % ring || ((all / ring) & 1) != ((x / ring) & 1) ||
            ((all >> 1) & 1) != ((x >> 1) & 1) || (all >= 8 && x < 8))
          return std::printf("ring %d: %lld counted as %d\n", ring, all, x), 1;
      }
    }
  }
  return 0;
}
"""


TABLE = r"""
#include <cstdio>
#include "dense_common.cuh"
using namespace msa;
// A last bucket that begins where no distance lies: the same table by distance wherever that is.
int main() {
  for (int G = 1; G <= kDenseMaxGroup; ++G) {
    DenseArgs a{};
    a.G = G, a.tpt = 128 / G, a.nb = 3, a.starts[1] = 7, a.starts[2] = 1 << 20;
    dense_lut_shape(&a);
    for (int last : {INT_MAX - 257, INT_MAX - 256, INT_MAX - 255, INT_MAX}) {
      DenseArgs b = a;
      b.starts[2] = last;
      dense_lut_shape(&b);
      if (a.lut_w < 0 || b.lut_w != a.lut_w || b.lut_stride != a.lut_stride)
        return std::printf("G %d, last start %d: %d distances, %d expected\n", G, last, b.lut_w,
                           a.lut_w), 1;
      if (b.lut_w > 0 && 127 + b.tpt + b.lut_w > b.lut_stride)
        return std::printf("G %d: the row of the table is too short\n", G), 1;
    }
  }
  return 0;
}
"""


def run(tmp_path, source):
    """Compiles a host program against the kernels' header and runs it."""
    from block_sparse_attention_proxy_gb300 import build

    src, exe = tmp_path / "host.cu", tmp_path / "host"
    src.write_text(source)
    r = subprocess.run([build.nvcc(), *build.ARCH, *build.FLAGS, "-I", build.CSRC, str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout


@pytest.mark.parametrize("source", [TURNS, TABLE], ids=["counts past 32 bits", "last start"])
def test_host_rules(tmp_path, source):
    run(tmp_path, source)
