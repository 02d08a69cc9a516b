"""The split of the 4-bit attention's work over warps (csrc/kv4_split.h), on
the CPU.

The kernel walks a warp's run with these functions and the joining kernel finds
a segment's partial results with them. Checked here on the header's own
functions, compiled by g++ into a host program, for many batches of lengths
(empty ones among them), rows and warps: every block of every segment is walked
exactly once; the walk block by block (as copies are issued) and piece by piece
(as they are worked on) agree; the warps that the joining kernel reads for a
segment are exactly those that walked blocks of it; and no two results share a
slot.
"""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "blockwise_attn_ffn_bpt_b200", "csrc")

HARNESS = r"""
#include <cstdio>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>
#include "kv4_split.h"
using namespace bpt;
typedef std::tuple<int, int, int> Block;  // sequence, row, block
static int fail(const char* what, int i) { std::printf("FAIL %s in case %d\n", what, i); return 1; }
int check(int c, const std::vector<int>& nbs, int rows, uint32_t max_warps) {
  const int b = (int)nbs.size();
  uint32_t total = 0;
  for (int nb : nbs) total += kva_units(nb) * rows;
  if (!total) return 0;
  const KvaSplit split(total, max_warps);
  if (split.warps > max_warps || split.first(0) != 0 || split.first(split.warps) != total) return fail("runs", c);
  auto blocks = [&](int beta) { return nbs[beta]; };
  std::map<Block, uint32_t> walked;
  std::map<uint32_t, int> slots;
  for (uint32_t w = 0; w < split.warps; ++w) {
    const uint32_t t = split.first(w);
    const int n = (int)(split.first(w + 1) - t);
    if (split.warp_of(t) != w || split.warp_of(t + n - 1) != w) return fail("warp_of", c);
    uint32_t base = 0;
    int beta = 0;
    while (base + kva_units(nbs[beta]) * rows <= t) base += kva_units(nbs[beta++]) * rows;
    KvaPlace at = KvaPlace::in_sequence(beta, nbs[beta], t - base, n), next = at;
    std::vector<Block> issued, worked;
    while (next.left > 0) {
      issued.push_back(Block(next.beta, next.row, next.blk));
      next.advance(blocks, b, rows, 1);
    }
    while (at.left > 0) {
      const int piece = at.nb - at.blk < at.left ? at.nb - at.blk : at.left;
      if (piece <= 0 || at.beta >= b || at.row >= rows || at.nb != nbs[at.beta]) return fail("place", c);
      if (!slots.emplace(at.beta * rows + at.row + w, 0).second) return fail("slot", c);
      for (int k = 0; k < piece; ++k) worked.push_back(Block(at.beta, at.row, at.blk + k));
      at.advance(blocks, b, rows, piece);
    }
    if (issued != worked) return fail("walks", c);
    for (const Block& x : worked)
      if (!walked.emplace(x, w).second) return fail("twice", c);
  }
  uint32_t before = 0;
  size_t all = 0;
  for (int beta = 0; beta < b; ++beta) {
    const int nb = nbs[beta];
    all += (size_t)nb * rows;
    for (int row = 0; nb && row < rows; ++row) {
      const uint32_t first = before + kva_first_block(row, nb);
      std::set<uint32_t> by;
      for (int k = 0; k < nb; ++k) {
        if (!walked.count(Block(beta, row, k))) return fail("missing", c);
        by.insert(walked[Block(beta, row, k)]);
      }
      std::set<uint32_t> read;
      for (uint32_t w = split.warp_of(first); w <= split.warp_of(first + nb - 1); ++w) read.insert(w);
      if (by != read) return fail("join", c);
    }
    before += kva_units(nb) * rows;
  }
  if (walked.size() != all) return fail("count", c);
  if (!slots.empty() && slots.rbegin()->first >= (uint32_t)b * rows + split.warps) return fail("slots", c);
  return 0;
}
int main() {
  std::mt19937 r(1);
  for (int c = 0; c < 20000; ++c) {
    std::vector<int> nbs(1 + r() % 9);
    for (int& nb : nbs) nb = r() % 4 ? (int)(r() % (1u << (r() % 8))) : 0;
    const uint32_t warps = r() % 2 ? 1 + r() % 8 : 1 + r() % 300;
    if (check(c, nbs, 1 + r() % 6, warps)) return 1;
  }
  if (check(-1, {2048, 0, 1, 2047, 2048}, 64, 148 * 12)) return 1;
  std::printf("OK\n");
  return 0;
}
"""


def run(tmp_path, header_dir):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "harness.cpp"
    src.write_text(HARNESS)
    exe = tmp_path / "harness"
    subprocess.run([gxx, "-O2", "-std=c++17", "-I", str(header_dir), "-o", str(exe), str(src)], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True)


def test_every_block_is_walked_once_and_joined(tmp_path):
    res = run(tmp_path, CSRC)
    assert res.returncode == 0 and res.stdout.strip() == "OK", res.stdout


@pytest.mark.parametrize("good,bad", [
    ("longer = (each + 1) * rest;", "longer = each * rest;"),
    ("do ++beta;\n      while (beta < b && (nb = blocks(beta)) == 0);", "if (++beta < b) nb = blocks(beta);"),
    ("    left -= KVA_SWITCH;\n", ""),
    ("return row * (nb + KVA_SWITCH) + KVA_SWITCH;", "return row * (nb + KVA_SWITCH);"),
])
def test_planted_mistakes_are_caught(tmp_path, good, bad):
    text = open(os.path.join(CSRC, "kv4_split.h")).read()
    assert good in text
    (tmp_path / "kv4_split.h").write_text(text.replace(good, bad))
    res = run(tmp_path, tmp_path)
    assert "FAIL" in res.stdout
