"""Which tiles the expert feed-forward block's products take, from the rule
itself (csrc/cc_ffn_rule.h compiled for the host with g++): the cases of the
GPU test of the tiles reach every tile size in every form, with all products
and both types."""
import os
import shutil
import subprocess

import pytest

from model_tiles import CASES

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "ring_allreduce_reduction_02_amd", "csrc")

# reads N E cap W F es vec and N * E counts; prints the form and tile of the six products on 256 compute units
PROGRAM = r"""
#include "cc_ffn_rule.h"
#include <cstdio>
#include <vector>
using namespace cc;
typedef unsigned long long ull;
int main() {
  int N, E, es, vec;
  ull cap, W, F;
  if (std::scanf("%d %d %llu %llu %llu %d %d", &N, &E, &cap, &W, &F, &es, &vec) != 7) return 1;
  FfnShape s{N, E, cap, W, F, 0, 0, {0, 0, 0}, es == 2 ? 2 : 1, es, 0};
  std::vector<ull> kept(N * E);
  for (ull& k : kept) {
    if (std::scanf("%llu", &k) != 1) return 1;
    k = std::min(k, cap);
  }
  for (int e = 0; e < E; ++e) {
    uint64_t n = 0;
    for (int i = 0; i < N; ++i) n += kept[i * E + e];
    s.rows += n;
    s.most = std::max<uint64_t>(s.most, n);
    for (int k = 0; k < kFfnTiles; ++k) s.mtiles[k] += (n + kFfnTile[k] - 1) / kFfnTile[k];
  }
  const struct { int kind; uint64_t M, cols; int grad; } products[] = {
      {K_GATEUP, 0, F, 0}, {K_DOWN, 0, W, 0}, {K_DHID, 0, F, 1}, {K_DX, 0, W, 1}, {K_DW, W, F, 1}, {K_DW, 2 * F, W, 1}};
  for (const auto& p : products) {
    const bool copied = ffn_copied(s, p.grad), fast = ffn_tiled(s, copied, vec);
    std::printf("%c%d ", copied ? 'c' : fast ? 't' : 'r', kFfnTile[ffn_pick_tile(s, p.kind, p.M, p.cols, fast, 256)]);
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not installed")
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, "-o", str(d / "rule"), str(d / "rule.cpp")],
                   check=True, timeout=120)

    def products(case, es, vec):
        N, E, cap, W, F, counts = case
        text = " ".join(str(v) for v in [N, E, cap, W, F, es, int(vec)] + [c for row in counts for c in row])
        return subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True, check=True,
                              timeout=20).stdout.split()
    return products


@pytest.mark.parametrize("es", [4, 2], ids=["f32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_each_case_reaches_its_tile(rule, name, es):
    case, offset = CASES[name]
    vec = offset == 0 and case[3] * es % 16 == 0 and case[4] * es % 16 == 0
    assert rule(case, es, vec) == [name] * 6


def test_all_forms_and_tiles_have_a_case():
    assert set(CASES) == {f + str(t) for f in "tcr" for t in (256, 128, 64)} - {"r256"}
