"""The runs of the few-token layer's down product (csrc/decode_runs.h), walked on the host as its wavefronts walk them, under
UndefinedBehaviorSanitizer: every pair of every entry once, and every place, the ones past the last run too, a valid entry's.
Without a shared expert, and with fewer runs than wavefronts, a wavefront stands past the end from the start."""
import subprocess

from mixture_experts_layer_33_amd import build as libbuild

DRIVER = r"""
#include <cstdio>
#include <vector>
#define __host__
#define __device__
#include "decode_runs.h"
using namespace moe;
int main() {
  long walks = 0, bad = 0;
  for (int routed : {1, 2, 3, 7, 16, 64, 256})
    for (int shared : {0, 1, 2, 4})
      for (int per : {1, 2, 3, 4, 5, 8, 9})
        for (int pers : {1, 2, 4, 7, 256})
          for (int run : {1, 4}) {
            if (shared == 0 && pers != 1) continue;
            const int entries = routed + shared, NW = 8;
            const D4Runs r = d4_runs(routed, entries, per, shared ? pers : 0, run);
            std::vector<std::vector<int>> seen(entries);
            for (int e = 0; e < entries; ++e) seen[e].assign(e < routed ? per : pers, 0);
            for (int w = 0; w < NW; ++w) {
              D4Place at{w, 0, 0, 0, 0};
              d4_set(r, at);
              for (int past = 0; past < 4;) {            // and a few places past the last run
                ++walks;
                const bool live = at.n < r.all;
                if (at.entry < 0 || at.entry >= entries || at.length < 1 || at.i < 0 || at.i >= at.length || at.from < 0) ++bad;
                else if (live && at.from + at.length > (int)seen[at.entry].size()) ++bad;
                else if (live) ++seen[at.entry][at.from + at.i];
                if (!live) ++past;
                d4_advance(r, NW, at);
              }
            }
            for (auto& e : seen)
              for (int n : e) bad += n != 1;
          }
  std::printf("%ld places, %ld wrong\n", walks, bad);
  return bad != 0;
}
"""


def test_every_pair_once_and_no_place_outside(tmp_path):
    src, exe = tmp_path / "walk.cpp", str(tmp_path / "walk")
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", libbuild.CSRC, str(src),
                    "-o", exe], check=True, timeout=300, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and ", 0 wrong" in r.stdout, r.stdout + r.stderr
