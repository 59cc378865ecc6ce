"""The closed form by which a block finds its work item among packed sequences, compiled for the host and
compared with counting the items one by one."""
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


def test_items_from_a_cost_on(tmp_path):
    src = tmp_path / "items.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "items"
    subprocess.check_call(["g++", "-O2", "-std=c++17", "-I", os.path.join(ROOT, "exact_attention_140_b200", "csrc"),
                           str(src), "-o", str(exe)])
    assert subprocess.check_output([str(exe)], text=True).strip() == "0"
