// How the wavefronts of the few-token layer's down product share the columns of all entries (an entry: an expert, or the shared
// one, with up to four of its tokens): every entry's 256-column pairs are cut into runs of up to `run`, counted through all
// entries, the routed ones first, and wavefront w takes runs w, w + NW, ...  Plain integers, so that the host can walk it too.
#pragma once

namespace moe {

struct D4Runs {
  int routed, entries;        // entries of routed experts, all entries
  int per, pers, run;         // pairs of a routed entry, of a shared one (0: there is none), of a run
  int runs, runss, all;       // runs of a routed entry, of a shared one, of all
};
struct D4Place {
  int n, i, entry, from, length;   // pair `i` of run number `n`, `length` long from pair `from` on, of an entry
};

__host__ __device__ inline D4Runs d4_runs(int routed, int entries, int per, int pers, int run) {
  const int runs = (per + run - 1) / run, runss = (pers + run - 1) / run;
  return {routed, entries, per, pers, run, runs, runss, routed * runs + (entries - routed) * runss};
}
// Run at.n from its first pair on.  Past the last run (a wavefront's place ends there, or stands there from the start): one pair of
// the last entry, which nothing multiplies.  Without a shared expert there is no run length to divide by there.
__host__ __device__ inline void d4_set(const D4Runs& r, D4Place& at) {
  at.i = 0;
  if (at.n >= r.all) {
    at.entry = r.entries - 1;
    at.from = 0;
    at.length = 1;
    return;
  }
  const bool shared = at.n >= r.routed * r.runs;
  const int q = shared ? at.n - r.routed * r.runs : at.n, of = shared ? r.runss : r.runs;
  const int en = q / of, k = q - en * of, left = (shared ? r.pers : r.per) - k * r.run;
  at.entry = shared ? r.routed + en : en;
  at.from = k * r.run;
  at.length = left < r.run ? left : r.run;
}
// The next pair, `step` runs further on after a run's last; whether that is another run.
__host__ __device__ inline bool d4_advance(const D4Runs& r, int step, D4Place& at) {
  if (++at.i < at.length) return false;
  at.n += step;
  d4_set(r, at);
  return true;
}

}  // namespace moe
