// Host run of the few-token kernel's weight stream (csrc/few_stream.h) against ring barriers that watch its rules.
//
// One warp streams the items of both phases; the wait numbered `fail` runs out.  The steps are the kernel's: fill before
// the routing, fill after it, phase 1, fill, phase 2, drain.  A stage's barrier counts phases as an mbarrier with one
// arrival does: a wait for a parity succeeds when the phase of that parity has ended, and the load ends it when it lands.
// Prints "ok" and the number of runs, or what broke.
#include <cstdio>
#include <cstdlib>

#include "few_stream.h"

using namespace moe::few;

static int param[6];

static void broke(const char* msg) {
  std::printf("%s (slices %d %d, shared %d, experts %d, warps %d, wait %d runs out)\n", msg, param[0], param[1], param[2],
              param[3], param[4], param[5]);
  std::exit(1);
}

struct Env {
  Phase ph[2];
  int queued[QUEUE];
  unsigned counter = 0, n_warps = 1;
  unsigned phases[NST] = {};   // ended
  bool flying[NST] = {};       // a load that has not landed
  bool full[NST] = {};         // landed, not taken
  int loads = 0;
  bool stopped = false;
  bool ran_out() const { return stopped; }
  const Phase& phase(int i) const { return ph[i]; }
  void queue(int at, int item) { queued[at] = item; }
  int expert(int j) const { return j; }
  unsigned draw() { return counter++; }
  unsigned warps() const { return n_warps; }
  void load(const Stream& s) {
    if (flying[s.stage]) broke("a load into a stage whose copy is on its way");
    if (full[s.stage]) broke("a load into a stage that has not been taken");
    flying[s.stage] = true;
    ++loads;
  }
  void land(int st) {
    if (flying[st]) {
      flying[st] = false;
      full[st] = true;
      ++phases[st];
    }
  }
  bool ended(int st, unsigned parity) const { return (phases[st] & 1u) != parity; }
  // an unlimited wait: the copy in flight lands, unless the wait returned at once
  void wait(int st, unsigned parity) {
    if (ended(st, parity)) return;
    if (!flying[st]) broke("a wait that nothing ends");
    land(st);
  }
};

// Phase PH of the warp; `waits` counts them, number `fail` runs out with the copy in flight.
static bool run_items(int PH, Env& env, Stream& st, Taken& tk, int known, int& waits, int fail) {
  const int base = PH == 0 ? 0 : env.ph[0].items;
  for (;;) {
    if (st.pushed == tk.head) return true;
    const int ticket = env.queued[tk.head & (QUEUE - 1)];
    if (ticket == NO_ITEM) return true;
    ++tk.head;
    const Item it = item_at(env.ph[PH], ticket - base);
    for (int ch = it.lo; ch < it.hi; ++ch) {
      if (waits++ == fail) {
        env.stopped = true;
        return false;
      }
      if (env.ended(tk.stage, tk.phase) && !env.full[tk.stage]) broke("a wait that succeeds on an empty stage");
      env.wait(tk.stage, tk.phase);
      env.full[tk.stage] = false;
      take(tk);
      stream_issue(st, known, env);
    }
  }
}

int main() {
  int runs = 0;
  for (int s1 = 0; s1 <= 3; ++s1)
    for (int s2 = 0; s2 <= 2; ++s2)
      for (int shared = 0; shared <= 2; ++shared)
        for (int touched = 1; touched <= 4; touched += 3)
          for (int warps = 1; warps <= 5; warps += 2)
            for (int fail = -1;; ++fail) {
              const int p[6] = {s1, s2, shared, touched, warps, fail};
              for (int i = 0; i < 6; ++i) param[i] = p[i];
              Env env;
              env.n_warps = warps;
              env.ph[0] = Phase{0, 11, 3, s1, 16, 0, NO_ITEM};
              env.ph[1] = Phase{0, 5, 2, s2, 16, 0, 0};
              Stream st{};
              st.ticket = warps / 2;
              Taken tk{0, 0u, 0};
              int waits = 0, known = (shared * env.ph[0].units) << s1;
              stream_start(st, known, env);
              for (int i = 0; i < 2; ++i) env.ph[i].items = ((shared + touched) * env.ph[i].units) << env.ph[i].s_log;
              known = env.ph[0].items;
              stream_start(st, known, env);
              bool ok = run_items(0, env, st, tk, known, waits, fail);
              // the loads of phase 2, whether or not a wait of phase 1 ran out
              known = NO_ITEM;
              stream_next_phase(st, known, env);
              if (ok) ok = run_items(1, env, st, tk, known, waits, fail);
              if (fail >= 0 && waits <= fail) break;  // past the last wait
              if (ok && waits != st.issued) broke("a chunk that was not taken");
              if (st.issued != env.loads) broke("a miscounted load");
              stream_drain(st, env);
              for (int i = 0; i < NST; ++i)
                if (env.flying[i]) broke("the end with a copy on its way");
              ++runs;
            }
  std::printf("ok %d\n", runs);
  return 0;
}
