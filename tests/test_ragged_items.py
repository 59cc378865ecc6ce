"""Host builds of what the kernels share their work out by: the closed form by which a block finds its work item
among packed sequences, against counting the items one by one, and the cut of items into pieces."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include "ragged_pick.cuh"
using namespace attn;
int main() {
  long bad = 0;
  for (int it = 0; it < 20000; ++it) {
    const int g = rand() % 5 == 0 ? 1 : 1 << (rand() % 6), shift = rand() % 2 ? 8 : 7, R = 1 << shift;
    const int bn = rand() % 2 ? 128 : 64;
    const int nq = rand() % 700, nk = rand() % 3 ? nq + rand() % 900 : rand() % 900;
    const bool causal = rand() % 2;
    const int nb = (int)(((long long)nq * g + R - 1) / R), most = (nk + bn - 1) / bn;
    for (int c = 0; c <= most + 1; ++c) {
      int count = 0;
      for (int qb = 0; qb < nb; ++qb) {
        int last = (int)(((long long)(qb + 1) * R + g - 1) / g);
        last = last < nq ? last : nq;
        count += (vis_end(last - 1, nq, nk, causal) + bn - 1) / bn >= c;
      }
      bad += count != ragged_items_from(c, nq, nk, nb, bn, shift, g, causal);
    }
  }
  std::printf("%ld\n", bad);
}
"""


PIECES = r"""
#include <cstdio>
#include <cstdlib>
#include <map>
#include "ragged_pick.cuh"
using namespace attn;
int main() {
  long bad = 0;
  for (int it = 0; it < 5000; ++it) {
    const int runs = rand() % 2 ? 148 : 1 + rand() % 20, pairs = 1 + rand() % 400, floor_ = 1 + rand() % 8;
    const long long longest = 1 + rand() % (rand() % 2 ? 300 : 9);
    std::map<int, int> slots;
    std::map<long long, long long> load;
    long long total = 0, a = 0, pieces = 0;
    static long long c[400];
    for (int i = 0; i < pairs; ++i) total += c[i] = rand() % 5 ? rand() % longest + 1 : 0;
    long long share = (total + runs - 1) / runs;
    share = share < floor_ ? floor_ : share;
    for (int i = 0; i < pairs; a += c[i++]) {
      const PieceRuns<long long> r = piece_runs<long long>(a, c[i], share);
      long long next = 0;
      for (long long v = r.first; v <= r.last; ++v, ++pieces) {
        const Piece<long long> x = piece_of<long long>(a, c[i], share, r, v);
        bad += x.lo != next || x.hi < x.lo || (x.hi == x.lo && c[i] > 0) || x.hi - x.lo > share;
        next = x.hi;
        load[v] += x.hi - x.lo;
        if (r.first == r.last) bad += x.slot != -1;
        else bad += x.slot < 0 || x.slot >= 2 * runs || slots[x.slot]++ > 0;
      }
      bad += next != c[i];
    }
    bad += pieces > pairs + runs;
    for (auto& l : load) bad += l.second > share;
  }
  std::printf("%ld\n", bad);
}
"""


def run(tmp_path, program):
    src = tmp_path / "items.cpp"
    src.write_text(program)
    exe = tmp_path / "items"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "exact_attention_140_b200", "csrc"),
                           str(src), "-o", str(exe)])
    return subprocess.check_output([str(exe)], text=True).strip()


def test_items_from_a_cost_on(tmp_path):
    assert run(tmp_path, PROGRAM) == "0"


def test_pieces(tmp_path):
    """The pieces of a pair are its tiles once, in order; no run holds more than its share; the slots of partial rows
    are in range and used once; and there are no more pieces than the list has room for."""
    assert run(tmp_path, PIECES) == "0"
