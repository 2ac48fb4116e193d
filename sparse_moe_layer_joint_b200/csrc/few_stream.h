// few_stream.h -- a warp's weight stream in the layer for a few tokens (few_tokens.cu): which chunk of which item its
// lane 0 loads next, into which stage of the warp's ring, and what it waits for before the CTA leaves.
//
// A stage has one barrier, whose phase ends when the one load begun on it has landed.  So a stage may be loaded again
// only when its last chunk has been taken (a wait for it succeeded, and the products have read it): a second load
// before that would arrive on a phase that has no arrivals left, write where a copy is still landing, and leave the
// barrier's phases out of step with the count that stream_drain goes by.
//
// The stream touches tickets, loads and barriers only through Env, so that a host program can run it as well.
#pragma once

#ifdef __CUDACC__
#define FEW_FN __device__ __forceinline__
#else
#define FEW_FN inline
#endif

namespace moe {
namespace few {

constexpr int NST = 2;                // ring stages (chunks) per warp
constexpr int QUEUE = 8;              // a warp's items between their first load and their products
constexpr int NO_ITEM = 0x7fffffff;

// One of the two phases: its matrices' items.  Item t (of the phase) is slice t % S of block b of the j-th
// expert, t / S = j * units + b.
struct Phase {
  int k_bytes;  // bytes of a row
  int nch;      // chunks of a row
  int units;    // blocks of 16 rows per expert
  int s_log;
  int row_mul;  // first row of block b: b * row_mul
  int up_row;   // gated: rows from a gate row to its up row, else 0
  int items;    // of all its experts
};

// An item: slice s (chunks lo .. hi - 1) of block b of the j-th expert.
struct Item {
  int j, b, s, lo, hi;
};

FEW_FN Item item_at(const Phase& ph, int t) {
  Item it;
  it.s = t & ((1 << ph.s_log) - 1);
  const int u = t >> ph.s_log;
  it.j = u / ph.units;
  it.b = u - it.j * ph.units;
  it.lo = (ph.nch * it.s) >> ph.s_log;
  it.hi = (ph.nch * (it.s + 1)) >> ph.s_log;
  return it;
}

// The warp's weight stream, kept by its lane 0: item by item, a chunk at a time.
struct Stream {
  int ticket;        // the item being loaded (or held)
  unsigned int next; // the draw for the item after it, as the counter returned it: nothing may use it before it is needed
  int phase;
  int ch, hi;        // next chunk of the item, its end
  int row, e;        // the item's first row, and expert
  int stage, issued, pushed;
  bool ready;        // the item's place is known
};

// The consuming side, the same in every lane: the next chunk's stage and its phase bit, the next item's place in
// the queue.
struct Taken {
  int stage;
  unsigned int phase;
  int head;
};

FEW_FN void take(Taken& tk) {
  if (++tk.stage == NST) {
    tk.stage = 0;
    tk.phase ^= 1u;
  }
}

// Begin the stream's ticket: phase 1's items come first, then phase 2's.  Before the routing only the first
// `known` items can be placed; the stream then stops with its ticket in hand.
template <class Env>
FEW_FN void stream_begin(Stream& s, int known, Env&& env) {
  s.ready = false;
  if (s.ticket >= known) return;
  s.phase = s.ticket < env.phase(0).items ? 0 : 1;
  const Phase& ph = env.phase(s.phase);
  const int t = s.ticket - (s.phase ? env.phase(0).items : 0);
  const bool any = t < ph.items;
  env.queue(s.pushed++ & (QUEUE - 1), any ? s.ticket : NO_ITEM);
  if (!any) return;
  const Item it = item_at(ph, t);
  s.ch = it.lo;
  s.hi = it.hi;
  s.row = it.b * ph.row_mul;
  s.e = env.expert(it.j);
  s.ready = true;
  s.next = env.draw();
}

// Load the next chunk, if there is one, into the next stage, which holds none.
template <class Env>
FEW_FN void stream_issue(Stream& s, int known, Env&& env) {
  if (!s.ready) return;
  env.load(s);
  ++s.issued;
  s.stage = s.stage + 1 == NST ? 0 : s.stage + 1;
  if (++s.ch >= s.hi) {
    s.ticket = (int)(s.next + env.warps());  // every warp's first item is its own number
    stream_begin(s, known, env);
  }
}

// At the start, and again when the routing is known: the first chunks, before any has been taken.
template <class Env>
FEW_FN void stream_start(Stream& s, int known, Env&& env) {
  if (!s.ready) stream_begin(s, known, env);
  while (s.issued < NST && s.ready) stream_issue(s, known, env);
}

// Behind phase 1, every chunk of which has been taken: the first chunks of phase 2.  When a wait of the CTA has run out
// the warp may have left an item half way, with chunks on their way: the call does not come to phase 2, and nothing more
// is loaded.
template <class Env>
FEW_FN void stream_next_phase(Stream& s, int known, Env&& env) {
  if (env.ran_out()) return;
  const int full = s.issued + NST;
  stream_begin(s, known, env);
  while (s.issued < full && s.ready) stream_issue(s, known, env);
}

// Before the CTA leaves: wait for the last load of every stage.
template <class Env>
FEW_FN void stream_drain(const Stream& s, Env&& env) {
  for (int i = s.issued > NST ? s.issued - NST : 0; i < s.issued; ++i) env.wait(i % NST, (unsigned int)(i / NST) & 1u);
}

}  // namespace few
}  // namespace moe
