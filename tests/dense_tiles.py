"""Sizes that reach every kernel of the 8-bit products and the shared expert, and the
rule that says so (csrc/dense_rule.h, asked through a small host program)."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "routed_expert_prefill_amd", "csrc")

MODES = ("bf16", "f32", "swiglu", "swiglu codes", "short")
TILES = ("32x32", "32x64", "64x64", "64x128", "64x128 two", "64x256", "128x256", "256x256")

# rows and weight rows (neither fills its last tile), tile for tile
PRODUCTS = {"32x32": (40, 130), "32x64": (257, 1000), "64x64": (500, 1100), "64x128": (1030, 1000),
            "64x128 two": (1999, 2001), "128x256": (3300, 2040)}
SHORT = {**PRODUCTS, "256x256": (7000, 2300)}
# groups of waves over the columns: a group's stages pass 64 at 64 * 128 columns for each
GROUPS = {"32x32": 8, "32x64": 4, "64x64": 2, "64x128": 2}


def columns(tile):
    """One block, two, some that are no multiple of the groups, more than 64 stages."""
    return 128, 256, 1152, 128 * (64 * GROUPS.get(tile, 1) + 1)


# T, d, f of the shared expert, by what computes gate and up
SHARED = {"few": [(1, 128, 128), (16, 1152, 640)],
          "swiglu 32x64": [(40, 2048, 128), (33, 32896, 128)],
          "swiglu 64x64": [(256, 512, 1152), (241, 16512, 1152)],
          "swiglu 64x128": [(401, 640, 1280), (390, 16512, 1280)],
          "swiglu codes 64x256": [(33, 256, 256), (300, 128, 384), (1000, 8320, 1152)],
          "swiglu codes 128x256": [(2049, 256, 1152), (3000, 8320, 1152)]}

_MAIN = r"""
#include <cstdio>
#include "dense_rule.h"
using namespace moe;
int main() {
  for (int m = 0; m < kMmModes; ++m)
    for (int i = 0; i < kMmTiles; ++i)
      if (kMmCosts[i].round[m] != 0) std::printf("has %d %d\n", m, i);
  int mode, M, N, K;
  while (std::scanf("%d %d %d %d", &mode, &M, &N, &K) == 4) {
    double t;
    const bool gateup = mode == kMmSwiglu;
    const bool codes = gateup && gateup_quantises(M, N, K);
    const int tile = mm_best(codes ? int(kMmSwigluCodes) : mode, M, N, K, &t);
    const long long bm = kMmCosts[tile].bm, bn = kMmCosts[tile].bn / (gateup ? 2 : 1);
    std::printf("is %d %d %d %d %lld\n", product_is_matvec(M, N, K, gateup, true),
                product_is_matvec(M, N, K, gateup, false), codes, tile,
                ((M - 1) / bm + 1) * ((N - 1) / bn + 1));
  }
}
"""


class Rule:
    """ask([(mode, M, N, K)]) -> [(few rows' kernel of codes, of bf16 rows, codes of h,
    tile, workgroups)]; has: the (mode, tile) that a size may choose."""

    def __init__(self, folder):
        source, self.program = os.path.join(folder, "rule.cpp"), os.path.join(folder, "rule")
        with open(source, "w") as f:
            f.write(_MAIN)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I" + CSRC, source, "-o", self.program],
                       check=True)
        self.has = set()
        self.ask([])

    def ask(self, sizes):
        text = "".join("%d %d %d %d\n" % (MODES.index(m), M, N, K) for m, M, N, K in sizes)
        out = subprocess.run([self.program], input=text, stdout=subprocess.PIPE, check=True, text=True).stdout
        got = []
        for line in out.splitlines():
            kind, *v = line.split()
            v = [int(x) for x in v]
            if kind == "has":
                self.has.add((MODES[v[0]], TILES[v[1]]))
            else:
                got.append((bool(v[0]), bool(v[1]), bool(v[2]), TILES[v[3]], v[4]))
        return got
