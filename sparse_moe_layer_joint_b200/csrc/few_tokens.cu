// few_tokens.cu -- the whole MoE layer for a few tokens (T <= 64) in one
// cooperative launch, with bf16 or 8-bit experts ("Inkling, Dissected" §02,
// §02b: s = sigmoid(x W_r^T); top-k of s + b; joint gates; y_e = W2_e act(W1_e x);
// out = sum of g y over the kept and the shared experts).
//
// What bounds it: the weights of the experts the tokens touch are read from HBM
// once, (touched + n_shared) * mats * d * d_ff values; everything else is small.
// So the kernel is a weight stream with the layer's other steps hidden behind it:
//
//   items     The weights are cut into items: 16 rows of one expert matrix (8 gate
//             rows and the 8 matching up rows for SwiGLU) by one of S slices of K.
//             Every warp of the grid (16 in one CTA an SM) takes the next item by
//             ticket, so one token's 8 experts keep every SM busy where 128-row
//             GEMM tiles would fill a fraction of them, and SMs that get more of
//             HBM's bandwidth do more of the work (with items dealt out in advance
//             the first SM had read its share after 52 us and the last after 84).
//   stream    Each warp has a ring of its own in shared memory (NST chunks of 256
//             bytes of K by 16 rows, 128 KB an SM) that its lane 0 fills by TMA, so
//             the stream needs no barrier, and runs on across items, from W1 into
//             W2, and behind the grid barriers.  The loads are marked evict-first:
//             a weight is read once, and L2 keeps what other kernels left there.
//   products  mma.sync m16n8k16 bf16 (m16n8k32 s8): weight rows are M, the expert's
//             tokens N (up to 8 a tile, 8 tiles).  At one to a few tokens an expert
//             the tensor pipe is almost idle at any instruction's rate, and this form
//             takes its operands straight from registers: K may be permuted as long
//             as both operands agree, so lane (r, c) holds 16 contiguous bytes of
//             rows r and r + 8 and of token r.  Each item leaves fp32 (int32) partial
//             sums of its slice.
//   phases    0  router logits, W_r's rows in groups of 16 by KS slices of K over
//                the CTAs (8-bit: the tokens' codes too); grid barrier, then every
//                CTA selects for all T tokens itself (a warp a token; more than 8
//                tokens are shared among the CTAs, with a barrier more)
//             1  items of W1; grid barrier; the slices' sums (8-bit, few tokens: one
//                sum that the slices were added to), activation, and h in fp32
//                precision: as bf16 high and low parts (the product with both
//                costs no extra weight traffic), or for 8-bit experts coded per row;
//                grid barrier
//             2  items of W2; grid barrier; out = the sum over the contributors'
//                slices in a fixed order
//             While the CTAs meet, HBM goes on with the rings of the next phase.
//
// The grid barriers need every CTA resident: the launch is cooperative, and every
// wait is bounded (wait_timeout_ns, MOE_STATUS_TIMEOUT).
//
// Measured (256 + 2 experts, top-6, GELU, d 7168, d_ff 2048, CUDA graphs of 8 batches;
// the HBM floor at 6.53 TB/s in brackets): one token 92 us in bf16 (72) and 55 in 8
// bits (37), 8 tokens 425 and 225, 64 tokens 1830 to 1940 and 910 to 1010; in separate
// launches (router, dispatch, grouped GEMMs, combine) 206 and 173, 512 and 354, 2120
// and 1080.  The weights
// stream at 6.1 to 7 TB/s; what remains beside them, 18 us at one token, is the
// launch, the router and its barrier (9), the two barriers around the hidden rows
// (8) and the last sums (5), less what the rings load meanwhile.  A layer of d 256
// is those steps alone: 18.6 us, where every CTA forms the few hidden rows itself.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "few_stream.h"
#include "int8.cuh"
#include "moe.h"
#include "moe_internal.h"
#include "sm100.cuh"

namespace moe {
namespace few {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BOX = 128;      // bytes of K of one row a TMA box holds (one swizzle atom)
constexpr int CHUNK = 256;    // and a chunk: two boxes side by side
constexpr int STEPS = CHUNK / 64;  // 64-byte steps of K (two MMA instructions each)
constexpr int ROWS = 16;      // weight rows of an item
constexpr int STAGE_BYTES = ROWS * CHUNK;
constexpr int BOX_BYTES = ROWS * BOX;
constexpr int NT_MAX = MOE_FEW_MAX_T / 8;
constexpr int KS_MAX = 8;     // K slices of the router phase
constexpr int S_MAX = 8;      // K slices of the experts' matrices
constexpr int E_LD = 272;     // pitch of a token's partial logits
constexpr int RED_COL = 20;   // floats per token column of a warp's logits tile (16 rows, padded: conflict-free)
constexpr int RED_TILE = 8 * RED_COL;
constexpr int MAX_CONTRIB = MOE_MAX_TOP_K + MOE_MAX_SHARED;
constexpr int SELECT_ALL_T = 8;
constexpr int ONE_SUM_T = 8;  // most tokens whose 8-bit experts' slices are added to one place (NTM 1)
constexpr int OWN_SUMS = THREADS * 16;    // most sums of W1 x of which every CTA forms all hidden rows (bf16)
constexpr int OWN_CODES = THREADS * 4;    // and most hidden values of which it codes all rows (8-bit)
constexpr int OWN_ROWS = OWN_CODES / 64;

struct Params {
  const uint8_t* x;    // [T, d] bf16
  const uint8_t* w_r;  // [E, d] bf16
  const float* bias;
  const float* offset;
  const float* w1s;  // [E, f1] channel scales (int8)
  const float* w2s;  // [E, d]
  int plain_map[2];  // W1's / W2's rows are not whole boxes: the map has three dimensions
  int T, d, f, n_routed, n_shared, k;
  int swiglu;
  float gate_scale;
  int32_t* topk_idx;
  float* gates;
  int32_t* counts;
  __nv_bfloat16* out;
  // scratch
  unsigned int* bar;  // [0 .. 3], [5]: grid barriers, [4] the ticket counter; zero at launch
  float* logits;      // [KS][T][E_LD] partial logits
  uint8_t* xq;        // [T, d] token codes (int8)
  float* xs;          // [T]
  float* u;           // [places][R, f1] sums of W1 x (int32 for 8-bit experts)
  uint8_t* h;         // bf16: [2][R, f] high and low parts; int8: [R, f] codes
  float* hs;          // [R] (int8)
  float* y;           // [places][R, d] sums of W2 h, right behind u
  int ks;             // K slices of the router phase
  int s_log[2];       // log2 of the K slices S1, S2
  uint64_t timeout_ns;
  unsigned int* status;
};

struct Smem {
  uint8_t ring[WARPS][NST][STAGE_BYTES];  // 128-byte swizzle; 1024-byte aligned
  uint64_t ring_full[WARPS][NST];
  int queue[WARPS][QUEUE];
  Phase ph[2];
  unsigned long long mask[MOE_MAX_ROUTED];  // tokens that picked each expert
  float gate[MOE_FEW_MAX_T * MAX_CONTRIB];
  short cnt[MOE_MAX_ROUTED], pre[MOE_MAX_ROUTED];  // each expert's tokens and their first row
  short list[MOE_MAX_ROUTED];           // touched experts in index order
  short pick[MOE_FEW_MAX_T * MOE_MAX_TOP_K];
  short row_of[MOE_FEW_MAX_T * MOE_MAX_TOP_K];   // row of each (token, slot)
  short row_exp[MOE_FEW_MAX_T * MOE_MAX_TOP_K];  // each routed row's expert and token
  uint8_t row_tok[MOE_FEW_MAX_T * MOE_MAX_TOP_K];
  int warp_rows[8], warp_touched[8];
  int n_touched;
  float score[SELECT_ALL_T * E_LD];
  uint32_t key[SELECT_ALL_T * E_LD];
  int flag[WARPS];
  int abort_flag;
  alignas(16) uint8_t own_h[OWN_SUMS * 4];  // the CTA's own hidden rows (bf16: high and low parts)
  uint32_t own_max[OWN_ROWS];
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory per CTA");
static_assert(sizeof(float) * WARPS * NT_MAX * RED_TILE <= WARPS * NST * STAGE_BYTES, "the router's sums use the ring");

template <bool I8>
struct AccT {
  using type = float;
};
template <>
struct AccT<true> {
  using type = int;
};

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One 64-byte step of K: lo / hi are 16 bytes of rows r and r + 8, b the same bytes of token r.
template <class T>
__device__ __forceinline__ void mma_step(T (&c)[4], const uint4& lo, const uint4& hi, const uint4& b) {
  mma(c, lo.x, hi.x, lo.y, hi.y, b.x, b.y);
  mma(c, lo.z, hi.z, lo.w, hi.w, b.z, b.w);
}

// The places of a warp's accumulators in its tile of the router's sums.
__device__ __forceinline__ void red_store(float* red, const float (&c)[4], int lane) {
  const int r = lane >> 2, col = 2 * (lane & 3);
  red[col * RED_COL + r] = c[0];
  red[(col + 1) * RED_COL + r] = c[1];
  red[col * RED_COL + r + 8] = c[2];
  red[(col + 1) * RED_COL + r + 8] = c[3];
}

__device__ __forceinline__ unsigned int ld_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Grid-wide barrier in two halves: every CTA arrives (its stores before that are visible to CTAs that have
// waited); the CTA goes on when all have.  The wait returns false when it ran out of time.
__device__ __forceinline__ void grid_arrive(unsigned int* ctr) {
  __syncthreads();
  if (threadIdx.x == 0) asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(ctr) : "memory");
}

__device__ __forceinline__ bool grid_wait(unsigned int* ctr, const Params& p, Smem* sm) {
  if (threadIdx.x == 0) {
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1; ld_acquire(ctr) < gridDim.x; ++it) {
      // (the clock: after the first poll, so that the shortest limit is noticed, then every eighth)
      if ((it & 7u) == 1 && globaltimer() - t0 > p.timeout_ns) {
        set_status(p.status, MOE_STATUS_TIMEOUT);
        sm->abort_flag = 1;
        break;
      }
    }
  }
  __syncthreads();
  return sm->abort_flag == 0;
}

__device__ __forceinline__ bool grid_barrier(unsigned int* ctr, const Params& p, Smem* sm) {
  grid_arrive(ctr);
  return grid_wait(ctr, p, sm);
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ Phase make_phase(int rows, int K, int elem, bool gated, int f, int s_log) {
  Phase ph;
  ph.k_bytes = K * elem;
  ph.nch = (ph.k_bytes + CHUNK - 1) / CHUNK;
  ph.units = gated ? f / (ROWS / 2) : rows / ROWS;
  ph.s_log = s_log;
  ph.row_mul = gated ? ROWS / 2 : ROWS;
  ph.up_row = gated ? f : 0;
  ph.items = 0;
  return ph;
}

__device__ __forceinline__ int expert_at(const Params& p, const Smem* sm, int j) {
  return j < p.n_shared ? p.n_routed + j : sm->list[j - p.n_shared];
}

// What the stream (few_stream.h) reaches: the call's tickets, the warp's ring and queue, the matrices.
struct StreamEnv {
  const CUtensorMap* tm1;
  const CUtensorMap* tm2;
  uint64_t pol;
  const Params& p;
  Smem* sm;

  __device__ __forceinline__ const Phase& phase(int i) const { return sm->ph[i]; }
  __device__ __forceinline__ void queue(int at, int item) { sm->queue[threadIdx.x >> 5][at] = item; }
  __device__ __forceinline__ int expert(int j) const { return expert_at(p, sm, j); }
  __device__ __forceinline__ unsigned int draw() { return atomicAdd(p.bar + 4, 1u); }
  // (a ring wait's flag is seen by every lane 0: a block barrier lies between phase 1's items and phase 2's first loads)
  __device__ __forceinline__ bool ran_out() const { return sm->abort_flag != 0; }
  __device__ __forceinline__ unsigned int warps() const { return gridDim.x * WARPS; }

  // The matrices' maps have K as blocks of 128 bytes next to each other in a dimension of their own, and the gate and up
  // rows likewise, so that one load brings the whole chunk; rows that are not whole blocks (8-bit, K an odd multiple of
  // 64) take a plain map and a load a box.
  __device__ __forceinline__ void load(const Stream& s) {
    const CUtensorMap* map = s.phase == 0 ? tm1 : tm2;
    const int warp = threadIdx.x >> 5;
    uint8_t* dst = sm->ring[warp][s.stage];
    uint64_t* bar = &sm->ring_full[warp][s.stage];
    mbar_arrive_expect_tx(bar, STAGE_BYTES);  // what lies past the row's end arrives as zeros
    if (!p.plain_map[s.phase]) {
      tma_load_5d_hint(dst, map, bar, 0, s.row, 0, s.ch * (CHUNK / BOX), s.e, pol);
    } else {
      const int up_row = sm->ph[s.phase].up_row;
      for (int h = 0; h < CHUNK / BOX; ++h) {
        const int x = s.ch * CHUNK + h * BOX;
        tma_load_3d_hint(dst + h * BOX_BYTES, map, bar, x, s.row, s.e, pol);
        if (up_row != 0) tma_load_3d_hint(dst + h * BOX_BYTES + BOX_BYTES / 2, map, bar, x, s.row + up_row, s.e, pol);
      }
    }
  }

  __device__ __forceinline__ void wait(int stage, uint32_t parity) {
    int no_abort = 0;
    mbar_wait(&sm->ring_full[threadIdx.x >> 5][stage], parity, wind_down_ns(p.timeout_ns), &no_abort, p.status);
  }
};

// An item's products: its chunks of 16 weight rows against the expert's n_e token rows, NT tiles of 8.
// b_base + row_of_col(col) * k_bytes is a token row; PARTS > 1: further parts b_part bytes apart.  False when
// the call has run out of time.
template <class T, int NT, int PARTS, class RowFn, class NextFn>
__device__ __forceinline__ bool item_products(T (&acc)[NT][4], int k_bytes, const Item& it, int n_e,
                                              const uint8_t* b_base, size_t b_part, RowFn row_of_col, Taken& tk,
                                              const Params& p, Smem* sm, NextFn next) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c4 = lane & 3;
  // 16-byte piece q of row r lies at piece q ^ (r % 8) of the row's 128 bytes
  const uint8_t* ring = sm->ring[warp][0] + r * BOX;
  const int at0 = (c4 ^ r) << 4, at1 = ((c4 + 4) ^ r) << 4;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint8_t* bp[NT];  // the lane's token rows
  constexpr bool EARLY = NT * PARTS <= 2;  // few enough to hold: the token loads go out before the wait
  uint4 b[EARLY ? NT * PARTS : 1][STEPS];  // (columns without a token stay zero)
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = j * 8 + r;
    bp[j] = col < n_e ? b_base + (size_t)row_of_col(col) * k_bytes + it.lo * CHUNK + c4 * 16 : nullptr;
    acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0;
  }
  if (EARLY) {
#pragma unroll
    for (int x = 0; x < NT * PARTS; ++x)
#pragma unroll
      for (int i = 0; i < STEPS; ++i) b[x][i] = zero;
  }
  for (int ch = it.lo; ch < it.hi; ++ch) {
    const int left = k_bytes - ch * CHUNK;  // bytes of the row from here on
    if (EARLY) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (bp[j]) {
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {
            const uint8_t* src = bp[j] + q * b_part;
            if (left >= CHUNK) {
#pragma unroll
              for (int i = 0; i < STEPS; ++i) b[j * PARTS + q][i] = load16(src + i * 64);
            } else {
#pragma unroll
              for (int i = 0; i < STEPS; ++i) b[j * PARTS + q][i] = i * 64 < left ? load16(src + i * 64) : zero;
            }
          }
          bp[j] += CHUNK;
        }
    }
    if (!__all_sync(0xffffffffu, mbar_wait(&sm->ring_full[warp][tk.stage], tk.phase, p.timeout_ns, &sm->abort_flag,
                                           p.status)))
      return false;
    const uint8_t* slot = ring + tk.stage * STAGE_BYTES;
    uint4 lo[STEPS], hi[STEPS];
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
      const uint8_t* at = slot + ((i & 1) ? at1 : at0) + (i >> 1) * BOX_BYTES;
      lo[i] = load16(at);
      hi[i] = load16(at + 8 * BOX);
    }
    take(tk);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          if (EARLY)
            mma_step(acc[j], lo[i], hi[i], b[j * PARTS + q][i]);
          else
            mma_step(acc[j], lo[i], hi[i], bp[j] && i * 64 < left ? load16(bp[j] + q * b_part + i * 64) : zero);
        }
      }
      if (!EARLY && bp[j]) bp[j] += CHUNK;
    }
    // The stage may be filled again now, and not before: the products needed every lane's pieces in registers.  A warp
    // barrier right behind the loads would order no more than their issue, and the copy writes by another path.
    __syncwarp();
    if (lane == 0) next();
    __syncwarp();
  }
  return true;
}

// An item's sum goes to its slice's place, to be added up in order later.  8-bit experts, up to ONE_SUM_T tokens: int32
// sums are exact in any order, so the slices are added to one place, zero at first, and the steps that wait for the sums
// read one slice instead of four or eight (one token, SwiGLU, d 4096, d_ff 1024: 37.3 instead of 39.9 us; d 7168, d_ff
// 2048: 54.8 instead of 55.5; with 13 tokens of d 2048, d_ff 768 the additions cost more than the reads, 83.6 instead of
// 83.2).
template <bool ONE_SUM, class T>
__device__ __forceinline__ void leave(T* to, T v) {
  if constexpr (ONE_SUM)
    atomicAdd(to, v);
  else
    *to = v;
}

template <bool I8>
__host__ __device__ __forceinline__ int places(int T, int s_log) {
  return I8 && T <= ONE_SUM_T ? 1 : 1 << s_log;
}

// Take this warp's items of phase PH and leave their sums at dst[(slice * R + row) * ld + column] (ONE_SUM: dst[row * ld +
// column]), column b's 16 rows (gated: gate rows at b * 8, up rows ph.up_row on).
template <class T, int PH, int PARTS, int NTM, class NextFn, class PushedFn>
__device__ __forceinline__ void run_items(const Params& p, const uint8_t* b_base, size_t b_part, T* dst, int ld, int R,
                                          Taken& tk, Smem* sm, NextFn next, PushedFn pushed) {
  constexpr bool ONE_SUM = std::is_same<T, int>::value && NTM == 1;  // T <= ONE_SUM_T
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Phase& ph = sm->ph[PH];
  const int base = PH == 0 ? 0 : sm->ph[0].items;
  const int hi_col = ph.up_row != 0 ? ph.up_row : ROWS / 2;
  for (;;) {
    if (pushed() == tk.head) return;  // the stream holds a ticket of the next phase
    __syncwarp();                     // lane 0's entry is there for every lane
    const int ticket = sm->queue[warp][tk.head & (QUEUE - 1)];
    if (ticket == NO_ITEM) return;
    ++tk.head;
    const Item it = item_at(ph, ticket - base);
    const bool shared = it.j < p.n_shared;
    const int e = expert_at(p, sm, it.j);
    const int n_e = shared ? p.T : sm->cnt[e];
    const int row0 = shared ? p.T * p.k + it.j * p.T : sm->pre[e];
    auto row = [&](int col) { return PH == 0 ? (shared ? col : (int)sm->row_tok[row0 + col]) : row0 + col; };
    T* to = dst + ((ONE_SUM ? 0 : (size_t)it.s * R) + row0) * ld + it.b * ph.row_mul + (lane >> 2);
    auto go = [&](auto n_tiles) {
      constexpr int NT = decltype(n_tiles)::value;
      T acc[NT][4];
      if (!item_products<T, NT, PARTS>(acc, ph.k_bytes, it, n_e, b_base, b_part, row, tk, p, sm, next)) return false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const int col = j * 8 + 2 * (lane & 3) + q;
          if (col < n_e) {
            leave<ONE_SUM>(to + (size_t)col * ld, acc[j][q]);
            leave<ONE_SUM>(to + (size_t)col * ld + hi_col, acc[j][q + 2]);
          }
        }
      return true;
    };
    bool ok = false;
    if (n_e <= 8) {
      ok = go(std::integral_constant<int, 1>{});
    } else if constexpr (NTM > 1) {
      if (n_e <= 16) {
        ok = go(std::integral_constant<int, 2>{});
      } else if constexpr (NTM > 2) {
        if (n_e <= 32)
          ok = go(std::integral_constant<int, 4>{});
        else
          ok = go(std::integral_constant<int, NTM>{});
      }
    }
    if (!ok) return;
  }
}

// A hidden row's expert and token.
__device__ __forceinline__ void row_owner(const Params& p, const Smem* sm, int r, int& e, int& t) {
  if (r < p.T * p.k) {
    e = sm->row_exp[r];
    t = sm->row_tok[r];
  } else {
    const int q = r - p.T * p.k;
    e = p.n_routed + q / p.T;
    t = q % p.T;
  }
}

// Four neighbouring columns of W1 x for row r: the slices' sums in order, scaled for 8-bit experts.
template <bool I8>
__device__ __forceinline__ void u_at(const Params& p, int R, int f1, int r, int c, float xs, const float* ws,
                                     float (&v)[4]) {
  using T = typename AccT<I8>::type;
  const int S = places<I8>(p.T, p.s_log[0]);
  const uint4* at = reinterpret_cast<const uint4*>(p.u + (size_t)r * f1 + c);
  float4 w4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (I8) w4 = __ldg(reinterpret_cast<const float4*>(ws + c));  // from HBM: ahead of the sums, which are in L2
  T a[4] = {0, 0, 0, 0};
#pragma unroll 8
  for (int s = 0; s < S; ++s) {
    const uint4 w = __ldcg(at + (size_t)s * R * f1 / 4);
    if constexpr (I8) {
      a[0] += (int)w.x;
      a[1] += (int)w.y;
      a[2] += (int)w.z;
      a[3] += (int)w.w;
    } else {
      a[0] += __uint_as_float(w.x);
      a[1] += __uint_as_float(w.y);
      a[2] += __uint_as_float(w.z);
      a[3] += __uint_as_float(w.w);
    }
  }
  const float m[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = I8 ? (float)a[i] * (xs * m[i]) : (float)a[i];
}

template <bool I8>
__device__ __forceinline__ void h_at(const Params& p, int R, int r, int c, float xs, const float* ws, float (&h)[4]) {
  const int f1 = p.swiglu ? 2 * p.f : p.f;
  u_at<I8>(p, R, f1, r, c, xs, ws, h);
  if (p.swiglu) {
    float up[4];
    u_at<I8>(p, R, f1, r, p.f + c, xs, ws, up);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = silu_f32(h[i]) * up[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = gelu_tanh_exp_f32(h[i]);
  }
}

// h = act(W1 x) of four columns as bf16 high and low parts.
__device__ __forceinline__ void hidden_parts(const Params& p, int R, int r, int c, uint2& hi, uint2& lo) {
  float h[4];
  h_at<false>(p, R, r, c, 0.0f, nullptr, h);
  uint32_t a[2], b[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    a[q] = pack_bf16x2(h[2 * q], h[2 * q + 1]);
    const float x = h[2 * q] - __uint_as_float(a[q] << 16), y = h[2 * q + 1] - __uint_as_float(a[q] & 0xffff0000u);
    // an infinite or NaN high part has no low part
    b[q] = pack_bf16x2(x - x == 0.0f ? x : 0.0f, y - y == 0.0f ? y : 0.0f);
  }
  hi = make_uint2(a[0], a[1]);
  lo = make_uint2(b[0], b[1]);
}

// The hidden rows' parts, four columns a thread over the whole grid.
__device__ __forceinline__ void finish_hidden(const Params& p, int R) {
  const int nv = p.f / 4;
  for (int i = (int)(threadIdx.x * gridDim.x + blockIdx.x); i < R * nv; i += THREADS * (int)gridDim.x) {
    const int r = i / nv, c = (i - r * nv) * 4;
    uint2 hi, lo;
    hidden_parts(p, R, r, c, hi, lo);
    uint8_t* to = p.h + ((size_t)r * p.f + c) * 2;
    *reinterpret_cast<uint2*>(to) = hi;
    *reinterpret_cast<uint2*>(to + (size_t)R * p.f * 2) = lo;
  }
}

// The largest |v| as integers: NaN and infinity stay the largest.
__device__ __forceinline__ uint32_t top_bits(const float (&v)[4]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

// 8-bit experts: a CTA a row, whose values stay in registers between their maximum and their codes (rows past
// 4 * HV * THREADS values are computed a second time).
__device__ __forceinline__ void code_hidden(const Params& p, Smem* sm, int R) {
  constexpr int HV = 1;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nv = p.f / 4, f1 = p.swiglu ? 2 * p.f : p.f;
  for (int r = (int)blockIdx.x; r < R; r += (int)gridDim.x) {
    int e, t;
    row_owner(p, sm, r, e, t);
    const float xs = __ldcg(p.xs + t);
    const float* ws = p.w1s + (size_t)e * f1;
    uint32_t m = 0;
    float keep[HV][4];
#pragma unroll
    for (int i = 0; i < HV; ++i)
      if (tid + i * THREADS < nv) {
        h_at<true>(p, R, r, (tid + i * THREADS) * 4, xs, ws, keep[i]);
        m = max(m, top_bits(keep[i]));
      }
    for (int c = tid + HV * THREADS; c < nv; c += THREADS) {
      float v[4];
      h_at<true>(p, R, r, c * 4, xs, ws, v);
      m = max(m, top_bits(v));
    }
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) sm->flag[warp] = (int)m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = max(m, (uint32_t)sm->flag[w]);
    const q8::RowScale rs = q8::row_scale(__uint_as_float(m));
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.h + (size_t)r * p.f);
#pragma unroll
    for (int i = 0; i < HV; ++i)
      if (tid + i * THREADS < nv) dst[tid + i * THREADS] = q8::code4_f32(keep[i], rs);
    for (int c = tid + HV * THREADS; c < nv; c += THREADS) {
      float v[4];
      h_at<true>(p, R, r, c * 4, xs, ws, v);
      dst[c] = q8::code4_f32(v, rs);
    }
    if (tid == 0) p.hs[r] = rs.scale;
    __syncthreads();
  }
}

// Few hidden values: every CTA forms all of them for itself, in its shared memory, and no barrier follows (2 tokens, d
// 256, d_ff 128: 18.6 instead of 20.2 us in bf16, 18.7 instead of 19.8 in 8 bits).  More values a thread lose: with 32
// for 8-bit experts one token at d 7168, d_ff 2048 took 63 us instead of 55, all SMs reading the same lines at once.
template <bool I8>
__device__ __forceinline__ bool own_rows(const Params& p, int R) {
  if (I8) return (long long)R * p.f <= OWN_CODES;
  return ((long long)R * (p.swiglu ? 2 * p.f : p.f) << p.s_log[0]) <= OWN_SUMS;
}

template <bool I8>
__device__ __forceinline__ void own_hidden(const Params& p, Smem* sm, int R) {
  const int nv = p.f / 4, tid = threadIdx.x;
  if constexpr (I8) {  // four values a thread; f is a multiple of 64, so 16 neighbouring threads share a row
    const int r = tid / nv, c = tid - r * nv;
    float h[4];
    if (r < R) {
      int e, t;
      row_owner(p, sm, r, e, t);
      const int f1 = p.swiglu ? 2 * p.f : p.f;
      h_at<true>(p, R, r, c * 4, __ldcg(p.xs + t), p.w1s + (size_t)e * f1, h);
      uint32_t m = top_bits(h);
      const uint32_t group = 0xffffu << (tid & 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(group, m, o));
      if ((tid & 15) == 0) atomicMax(&sm->own_max[r], m);
    }
    __syncthreads();
    if (r < R) {
      const q8::RowScale rs = q8::row_scale(__uint_as_float(sm->own_max[r]));
      reinterpret_cast<uint32_t*>(sm->own_h)[tid] = q8::code4_f32(h, rs);
      if (blockIdx.x == 0 && c == 0) p.hs[r] = rs.scale;  // every CTA's last sums read it, a barrier later
    }
  } else {
    for (int i = tid; i < R * nv; i += THREADS) {
      const int r = i / nv, c = (i - r * nv) * 4;
      uint2 hi, lo;
      hidden_parts(p, R, r, c, hi, lo);
      reinterpret_cast<uint2*>(sm->own_h)[i] = hi;
      reinterpret_cast<uint2*>(sm->own_h)[R * nv + i] = lo;
    }
  }
  __syncthreads();
}

// out[t, col] = sum over the contributors of gate * (sum of the slices).  A thread takes one contributor's four
// neighbouring columns, GL threads (a power of two) one token's contributors, added up in a fixed tree.  (Short code: it
// runs once, and instructions that are fetched for one use cost more than the loads they issue.)
template <bool I8>
__device__ __forceinline__ void finish_out(const Params& p, const Smem* sm, int R) {
  const int G = p.k + p.n_shared, S = places<I8>(p.T, p.s_log[1]);
  const int gl = G > 8 ? 4 : G > 4 ? 3 : G > 2 ? 2 : G > 1 ? 1 : 0;  // log2 GL
  const int nv = p.d / 4, total = (p.T * nv) << gl;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint4* y = reinterpret_cast<const uint4*>(p.y);
  // whole warps: 32 / GL vectors each, neighbouring warps on neighbouring SMs
  for (int i0 = (warp * (int)gridDim.x + (int)blockIdx.x) * 32; i0 < total; i0 += THREADS * (int)gridDim.x) {
    const int i = i0 + lane;
    const int q = i & ((1 << gl) - 1), v = i >> gl;
    const int t = v / nv, c = v - t * nv;
    float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (q < G && i < total) {
      const int r = q < p.k ? (int)sm->row_of[t * MOE_MAX_TOP_K + q] : p.T * p.k + (q - p.k) * p.T + t;
      const float g = sm->gate[t * MAX_CONTRIB + q];
      if constexpr (I8) {
        const int e = q < p.k ? (int)sm->pick[t * MOE_MAX_TOP_K + q] : p.n_routed + q - p.k;
        const float4 w = __ldg(reinterpret_cast<const float4*>(p.w2s + (size_t)e * p.d) + c);
        const float hs = __ldcg(p.hs + r);
        int n[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
          const uint4 u = __ldcg(y + ((size_t)s * R + r) * nv + c);
          n[0] += (int)u.x;
          n[1] += (int)u.y;
          n[2] += (int)u.z;
          n[3] += (int)u.w;
        }
        a[0] = g * ((float)n[0] * (hs * w.x));
        a[1] = g * ((float)n[1] * (hs * w.y));
        a[2] = g * ((float)n[2] * (hs * w.z));
        a[3] = g * ((float)n[3] * (hs * w.w));
      } else {
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
          const uint4 u = __ldcg(y + ((size_t)s * R + r) * nv + c);
          a[0] += __uint_as_float(u.x);
          a[1] += __uint_as_float(u.y);
          a[2] += __uint_as_float(u.z);
          a[3] += __uint_as_float(u.w);
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) a[x] *= g;
      }
    }
    for (int o = (1 << gl) >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int x = 0; x < 4; ++x) a[x] += __shfl_xor_sync(0xffffffffu, a[x], o);
    if (q == 0 && i < total)
      *reinterpret_cast<uint2*>(p.out + (size_t)t * p.d + c * 4) =
          make_uint2(pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3]));
  }
}

// Phase 0: partial logits of 16 router rows over one slice of K, all tokens.
template <int NTM>
__device__ __forceinline__ void router_partial(const Params& p, Smem* sm) {
  const int E = p.n_routed + p.n_shared;
  const int rg_n = (E + ROWS - 1) / ROWS;
  const int k_bytes = p.d * 2;
  const int nch = (k_bytes + BOX - 1) / BOX;  // 128-byte pieces of K
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = (p.T + 7) / 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int un = blockIdx.x; un < rg_n * p.ks; un += gridDim.x) {
    const int rg = un % rg_n, ks = un / rg_n;
    const int c_lo = (int)((long long)nch * ks / p.ks), c_hi = (int)((long long)nch * (ks + 1) / p.ks);
    const int r0 = min(rg * ROWS + (lane >> 2), E - 1), r1 = min(rg * ROWS + (lane >> 2) + 8, E - 1);
    const uint8_t* a0 = p.w_r + (size_t)r0 * k_bytes + (lane & 3) * 16;
    const uint8_t* a1 = p.w_r + (size_t)r1 * k_bytes + (lane & 3) * 16;
    float acc[NTM][4];
#pragma unroll
    for (int j = 0; j < NTM; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    for (int c = c_lo + warp; c < c_hi; c += WARPS) {
      const int off = c * BOX;
      const bool second = off + 64 < k_bytes;
      const uint4 lo0 = load16(a0 + off), hi0 = load16(a1 + off);
      const uint4 lo1 = second ? load16(a0 + off + 64) : zero, hi1 = second ? load16(a1 + off + 64) : zero;
#pragma unroll
      for (int j = 0; j < NTM; ++j) {
        if (j < nt) {
          const int t = j * 8 + (lane >> 2);
          const uint8_t* b = p.x + (size_t)t * k_bytes + (lane & 3) * 16 + off;
          const uint4 b0 = t < p.T ? load16(b) : zero;
          const uint4 b1 = t < p.T && second ? load16(b + 64) : zero;
          mma_step(acc[j], lo0, hi0, b0);
          mma_step(acc[j], lo1, hi1, b1);
        }
      }
    }
    // the sum over the warps, through the ring's memory (the stream has not begun)
    float* red = reinterpret_cast<float*>(sm->ring);
#pragma unroll
    for (int j = 0; j < NTM; ++j)
      if (j < nt) red_store(red + (warp * NTM + j) * RED_TILE, acc[j], lane);
    __syncthreads();
    for (int i = tid; i < p.T * ROWS; i += THREADS) {
      const int col = i >> 4, r = i & 15;
      const int e = rg * ROWS + r;
      const float* at = red + (col >> 3) * RED_TILE + (col & 7) * RED_COL + r;
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += at[w * NTM * RED_TILE];
      if (e < E) p.logits[((size_t)ks * p.T + col) * E_LD + e] = v;
    }
    __syncthreads();
  }
}

// Phase 0, 8-bit experts: the tokens' codes, from the last CTAs backwards (the first have router slices).
__device__ __forceinline__ void code_tokens(const Params& p, Smem* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nv = p.d / 8;
  for (int t = (int)gridDim.x - 1 - (int)blockIdx.x; t < p.T; t += gridDim.x) {
    const uint4* row = reinterpret_cast<const uint4*>(p.x + (size_t)t * p.d * 2);
    uint32_t m = 0;
    for (int i = tid; i < nv; i += THREADS) m = max(m, q8::abs_max_bits(row[i]));
    m = __reduce_max_sync(0xffffffffu, m);
    if (lane == 0) sm->flag[warp] = (int)m;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) m = max(m, (uint32_t)sm->flag[w]);
    const q8::RowScale rs = q8::row_scale(__uint_as_float(m << 16));
    for (int i = tid; i < nv; i += THREADS)
      *reinterpret_cast<uint2*>(p.xq + (size_t)t * p.d + (size_t)i * 8) = q8::code8(row[i], rs);
    if (tid == 0) p.xs[t] = rs.scale;
    __syncthreads();
  }
}

__device__ __forceinline__ float sigmoid_f32(float z) { return __frcp_rn(1.0f + __expf(-z)); }

// Order-preserving key of a score; NaN below every number, 0 is kept for "taken".
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v);
  if (!(v == v)) return 1u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Scores of `n` tokens from t0 on, a thread an expert of a token at a time: the logits' slices in order, and the
// selection's order keys.
__device__ __forceinline__ void score_tokens(const Params& p, Smem* sm, int t0, int n) {
  const int E = p.n_routed + p.n_shared;
  for (int i = threadIdx.x; i < n * E; i += THREADS) {
    const int tl = i / E, e = i - tl * E;
    const float* z = p.logits + (size_t)(t0 + tl) * E_LD + e;
    float part[KS_MAX];
#pragma unroll
    for (int q = 0; q < KS_MAX; ++q) {
      part[q] = 0.0f;
      if (q < p.ks) part[q] = __ldcg(z + (size_t)q * p.T * E_LD);
    }
    const bool routed = e < p.n_routed;
    const float bias = routed ? __ldg(p.bias + e) : 0.0f;
    float off = 0.0f;
    if (routed && p.offset) off = __ldg(p.offset + e);
    float v = part[0];
#pragma unroll
    for (int q = 1; q < KS_MAX; ++q) v += part[q];
    const float s = sigmoid_f32(v + off);
    sm->score[tl * E_LD + e] = s;
    sm->key[tl * E_LD + e] = routed ? order_key(s + bias) : 0u;
  }
}

// Select for token t (scores at tl) with one warp: k rounds of a warp-wide maximum (the lower index on equal
// scores), joint gates with the denominator summed in ascending expert index.
__device__ __forceinline__ void select_token(const Params& p, Smem* sm, int tl, int t, bool write) {
  const int lane = threadIdx.x & 31;
  const int G = p.k + p.n_shared;
  constexpr int PER = MOE_MAX_ROUTED / 32;
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) key[i] = i * 32 + lane < p.n_routed ? sm->key[tl * E_LD + i * 32 + lane] : 0u;
  // lane q < k: the q-th pick; then the shared experts
  int id = lane < G ? p.n_routed + lane - p.k : 0x7fffffff;
#pragma unroll 1
  for (int q = 0; q < p.k; ++q) {
    uint32_t best = 0;
    int e = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > best) {  // strictly: the lane's lowest index among equals
        best = key[i];
        e = i * 32 + lane;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, best);
    const int win = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)e : 0x7fffffffu);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i * 32 + lane == win) key[i] = 0;
    if (lane == q) id = win;
  }
  const float sc = lane < G ? sm->score[tl * E_LD + id] : 0.0f;
  int rank = 0;
#pragma unroll 1
  for (int q = 0; q < G; ++q) rank += __shfl_sync(0xffffffffu, id, q) < id;
  float den = 0.0f;
#pragma unroll 1
  for (int r = 0; r < G; ++r) {
    const uint32_t who = __ballot_sync(0xffffffffu, lane < G && rank == r);
    den += __shfl_sync(0xffffffffu, sc, __ffs(who) - 1);
  }
  if (lane < G) {
    const float g = __fmul_rn(__fdiv_rn(sc, den), p.gate_scale);
    sm->gate[t * MAX_CONTRIB + lane] = g;
    if (write) p.gates[t * G + lane] = g;
    if (lane < p.k) {
      sm->pick[t * MOE_MAX_TOP_K + lane] = (short)id;
      if (write) p.topk_idx[t * p.k + lane] = id;
    }
  }
}

// The routing tables of all tokens, built by every CTA for itself.  Up to SELECT_ALL_T tokens every CTA also makes the
// whole selection; more are shared among the CTAs, which then meet again (another barrier costs less than the
// other tokens' selections).  False when that barrier ran out of time.
__device__ __forceinline__ bool route_all(const Params& p, Smem* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.k + p.n_shared;
  if (p.T <= SELECT_ALL_T) {
    score_tokens(p, sm, 0, p.T);
    __syncthreads();
    if (warp < p.T) select_token(p, sm, warp, warp, warp % (int)gridDim.x == (int)blockIdx.x);
    __syncthreads();
  } else {
    for (int t = (int)blockIdx.x; t < p.T; t += (int)gridDim.x) {
      score_tokens(p, sm, t, 1);
      __syncthreads();
      if (warp == 0) select_token(p, sm, 0, t, true);
      __syncthreads();
    }
    if (!grid_barrier(&p.bar[5], p, sm)) return false;
    for (int i = tid; i < p.T * p.k; i += THREADS)
      sm->pick[i / p.k * MOE_MAX_TOP_K + i % p.k] = (short)__ldcg(p.topk_idx + i);
    for (int i = tid; i < p.T * G; i += THREADS) sm->gate[i / G * MAX_CONTRIB + i % G] = __ldcg(p.gates + i);
    __syncthreads();
  }
  for (int i = tid; i < p.T * p.k; i += THREADS) {
    const int t = i / p.k;
    atomicOr(&sm->mask[sm->pick[t * MOE_MAX_TOP_K + i - t * p.k]], 1ull << t);
  }
  __syncthreads();
  int n = 0, rows = 0, touched = 0;
  if (tid < MOE_MAX_ROUTED) {
    n = __popcll(sm->mask[tid]);
    rows = n;
    touched = n > 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, rows, o), b = __shfl_up_sync(0xffffffffu, touched, o);
      if (lane >= o) {
        rows += a;
        touched += b;
      }
    }
    if (lane == 31) {
      sm->warp_rows[warp] = rows;
      sm->warp_touched[warp] = touched;
    }
  }
  __syncthreads();
  if (tid < MOE_MAX_ROUTED) {
    for (int w = 0; w < warp; ++w) {
      rows += sm->warp_rows[w];
      touched += sm->warp_touched[w];
    }
    sm->pre[tid] = (short)(rows - n);
    sm->cnt[tid] = (short)n;
    if (n > 0) sm->list[touched - 1] = (short)tid;
    if (tid == MOE_MAX_ROUTED - 1) sm->n_touched = touched;
    if (blockIdx.x == 0 && tid < p.n_routed) p.counts[tid] = n;
  }
  __syncthreads();
  for (int i = tid; i < p.T * p.k; i += THREADS) {
    const int t = i / p.k, q = i - t * p.k;
    const int e = sm->pick[t * MOE_MAX_TOP_K + q];
    const int row = sm->pre[e] + __popcll(sm->mask[e] & ((1ull << t) - 1ull));
    sm->row_of[t * MOE_MAX_TOP_K + q] = (short)row;
    sm->row_tok[row] = (uint8_t)t;
    sm->row_exp[row] = (short)e;
  }
  __syncthreads();
  return true;
}

// NTM: tiles of 8 tokens an expert can have, 1, 2 or 8 by the call's T.  (The code for more than two needs more registers
// than there are; with it one token at d 7168, d_ff 2048 took 94 us instead of 91.  It spills 344 bytes a thread in bf16
// and 384 in 8 bits, which narrow layers feel: d 1024, d_ff 512, 64 + 2 experts take 47 and 39 us with 16 tokens, 57 and 43
// with 17.)
template <bool I8, int NTM>
__global__ void __launch_bounds__(THREADS, 1)
    few_tokens_kernel(const __grid_constant__ CUtensorMap tm1, const __grid_constant__ CUtensorMap tm2,
                      const Params p) {
  using T = typename AccT<I8>::type;
  extern __shared__ uint8_t smem_raw[];
  Smem* sm = reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int ELEM = I8 ? 1 : 2;
  const int f1 = p.swiglu ? 2 * p.f : p.f;

  if (tid < MOE_MAX_ROUTED) sm->mask[tid] = 0;
  if (tid < OWN_ROWS) sm->own_max[tid] = 0;
  if (tid < WARPS) {
    for (int i = 0; i < NST; ++i) mbar_init(&sm->ring_full[tid][i], 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    sm->abort_flag = 0;
    sm->ph[0] = make_phase(f1, p.d, ELEM, p.swiglu != 0, p.f, p.s_log[0]);
    sm->ph[0].items = NO_ITEM;  // not known yet
  }
  if (tid == 32) {
    sm->ph[1] = make_phase(p.d, p.f, ELEM, false, p.f, p.s_log[1]);
    tma_prefetch_desc(&tm1);
    tma_prefetch_desc(&tm2);
  }

  // phase 0
  if (I8 && NTM == 1) {
    // the sums of both phases begin at zero (they lie next to each other)
    uint4* at = reinterpret_cast<uint4*>(p.u);
    const int n = p.T * (p.k + p.n_shared) * ((f1 + p.d) / 4);
    for (int i = (int)blockIdx.x * THREADS + tid; i < n; i += (int)gridDim.x * THREADS) at[i] = make_uint4(0, 0, 0, 0);
  }
  if (I8) code_tokens(p, sm);
  router_partial<NTM>(p, sm);
  fence_proxy_async_smem();  // the ring's memory was the router's: TMA writes come after
  grid_arrive(&p.bar[0]);
  // the shared experts' weights need no routing: their items fill the ring behind the barrier
  Stream st;
  st.ticket = warp * (int)gridDim.x + (int)blockIdx.x;
  st.next = 0;
  st.stage = st.issued = st.pushed = 0;
  st.ready = false;
  const uint64_t pol = l2_policy_evict_first();
  auto env = [&]() { return StreamEnv{&tm1, &tm2, pol, p, sm}; };  // (kept as one object it cost registers)
  int known = (p.n_shared * sm->ph[0].units) << p.s_log[0];
  if (lane == 0) stream_start(st, known, env());
  Taken tk{0, 0u, 0};
  bool ok = grid_wait(&p.bar[0], p, sm);
  if (ok) {
    ok = route_all(p, sm);
  }
  if (ok) {
    const int n_exp = p.n_shared + sm->n_touched;
    if (tid < 2) sm->ph[tid].items = (n_exp * sm->ph[tid].units) << p.s_log[tid];
    __syncthreads();
    // Phase 2's weights wait until the CTA has arrived at the end of phase 1: their loads would hold up the stores, the
    // tickets and the barrier of a memory system that is busy with the last items of phase 1.
    known = sm->ph[0].items;
    if (lane == 0) stream_start(st, known, env());
    if (I8) {
      // the channel scales of the experts in use, which a few CTAs need at once later, into L2 meanwhile
      for (int j = (int)blockIdx.x; j < n_exp; j += (int)gridDim.x) {
        const int e = expert_at(p, sm, j);
        for (int i = tid; i < (f1 + p.d) / 32; i += THREADS) {
          const float* a = i < f1 / 32 ? p.w1s + (size_t)e * f1 + i * 32 : p.w2s + (size_t)e * p.d + (i - f1 / 32) * 32;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(a));
        }
      }
    }
    auto pushed = [&]() { return __shfl_sync(0xffffffffu, st.pushed, 0); };
    auto next = [&]() { stream_issue(st, known, env()); };
    const int R = p.T * (p.k + p.n_shared);

    // phase 1
    run_items<T, 0, 1, NTM>(p, I8 ? p.xq : p.x, 0, reinterpret_cast<T*>(p.u), f1, R, tk, sm, next, pushed);
    grid_arrive(&p.bar[1]);
    known = NO_ITEM;
    if (lane == 0) stream_next_phase(st, known, env());
    ok = grid_wait(&p.bar[1], p, sm);
    const bool own = NTM == 1 && own_rows<I8>(p, R);  // (more tokens have more rows; 64: the choice alone cost 3%)
    if (ok) {
      if (own) {
        own_hidden<I8>(p, sm, R);
      } else {
        if (I8)
          code_hidden(p, sm, R);
        else
          finish_hidden(p, R);
        ok = grid_barrier(&p.bar[2], p, sm);
      }
    }
    // phase 2
    if (ok) {
      run_items<T, 1, I8 ? 1 : 2, NTM>(p, own ? sm->own_h : p.h, (size_t)R * p.f * 2, reinterpret_cast<T*>(p.y), p.d, R,
                                       tk, sm, next, pushed);
      ok = grid_barrier(&p.bar[3], p, sm);
    }
    if (ok) finish_out<I8>(p, sm, R);
  }
  // nothing may still be landing in shared memory (only a call that ran out of time can have chunks left)
  if (lane == 0) stream_drain(st, env());
}

// Scratch layout: byte offsets of each part.
struct Layout {
  size_t bar, logits, xq, xs, u, h, hs, y, bytes;
  int s_log[2];
};

// log2 of the K slices of a matrix of nch chunks, for `units` blocks of 16 rows.  A phase ends when the last warp's last
// item does, so an item should be short beside the phase: at least one and a half items for each warp, and as long as they
// are fewer than sixteen each, at most 8 chunks of K (about 12 us).  Every item costs a ticket, its places and its partial
// sums, so it keeps at least two chunks.  (32 tokens, SwiGLU, d 4096: items of 32 chunks left the first SM idle for 34 us.)
// The warps are those of 148 SMs whatever the device has: the scratch's size goes by the slices and is computed without a
// device, and on another SM count only the balance is off.
constexpr double NOMINAL_WARPS = 148.0 * WARPS;

inline int slices_log(double units, int nch) {
  int s = 0;
  while ((1 << (s + 1)) <= S_MAX && (nch >> (s + 1)) >= 2 &&
         (units * (1 << s) < 1.5 * NOMINAL_WARPS || ((nch >> s) > 8 && units * (1 << s) < 16.0 * NOMINAL_WARPS)))
    ++s;
  return s;
}

inline Layout layout_of(int T, int d, int f, int n_routed, int n_shared, int k, bool swiglu, int elem) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  // experts that T tokens touch when each picks k of n at random
  double miss = 1.0;
  for (int t = 0; t < T; ++t) miss *= 1.0 - (double)k / n_routed;
  const double experts = n_shared + n_routed * (1.0 - miss);
  l.s_log[0] = slices_log(experts * (f / (swiglu ? ROWS / 2 : ROWS)), (d * elem + CHUNK - 1) / CHUNK);
  l.s_log[1] = slices_log(experts * (d / ROWS), (f * elem + CHUNK - 1) / CHUNK);
  const size_t R = (size_t)T * (k + n_shared);
  l.bar = take(8 * sizeof(unsigned int));
  l.logits = take((size_t)KS_MAX * T * E_LD * sizeof(float));
  l.xq = take((size_t)T * d);
  l.xs = take((size_t)T * sizeof(float));
  auto n_places = [&](int s_log) { return (size_t)(elem == 1 ? places<true>(T, s_log) : places<false>(T, s_log)); };
  l.u = take(R * (swiglu ? 2 * f : f) * sizeof(float) * n_places(l.s_log[0]));
  l.y = take(R * d * sizeof(float) * n_places(l.s_log[1]));
  l.h = take(R * f * sizeof(float));
  l.hs = take(R * sizeof(float));
  l.bytes = at;
  return l;
}

// Tensor map of expert matrices [E, rows, K], whose loads bring a chunk of 16 rows (gated: 8 gate rows and the 8 matching
// up rows, `rows` being both halves) as STAGE_BYTES: boxes of 128 bytes side by side in K.
inline int weight_map(CUtensorMap* map, const void* w, bool int8, int K, int rows, int E, bool gated, int* plain) {
  const int elem = int8 ? 1 : 2, box = BOX / elem;
  const uint64_t row = (uint64_t)K * elem;
  *plain = row % BOX != 0;
  if (*plain) return encode_tmap_u8(map, w, 3, K, rows, E, BOX, gated ? ROWS / 2 : ROWS);  // 8-bit rows alone
  const uint64_t half = gated ? rows / 2 : rows;
  const uint64_t dims[5] = {(uint64_t)box, half, gated ? 2ull : 1ull, row / BOX, (uint64_t)E};
  const uint64_t strides[4] = {row, half * row, BOX, (uint64_t)rows * row};
  const uint32_t boxes[5] = {(uint32_t)box, (uint32_t)(gated ? ROWS / 2 : ROWS), gated ? 2u : 1u, CHUNK / BOX, 1};
  return encode_tmap_5d(map, w, elem, dims, strides, boxes);
}

template <bool I8>
int run(const moe_bf16* x, const moe_bf16* w_router, const float* bias, const float* logit_offset, const void* w1,
        const float* w1s, const void* w2, const float* w2s, int T, int d, int d_ff, int n_routed, int n_shared,
        int top_k, float route_scale, int activation, int32_t* topk_idx, float* gates, int32_t* counts, moe_bf16* out,
        void* scratch, size_t scratch_bytes, void* stream) {
  if (!w_router || !bias || !w1 || !w2 || !counts || !scratch) return MOE_ERR_INVALID_ARG;
  if (T != 0 && (!x || !topk_idx || !gates || !out)) return MOE_ERR_INVALID_ARG;  // without elements: perhaps no address
  if (I8 && (!w1s || !w2s)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w1) || !aligned16(w2) || !aligned16(out) ||
      !aligned16(scratch) || !aligned4(bias) || !aligned4(logit_offset) || !aligned4(topk_idx) || !aligned4(gates) ||
      !aligned4(counts) || !aligned16(w1s) || !aligned16(w2s))
    return MOE_ERR_INVALID_ARG;
  if (T < 0 || d <= 0 || d_ff <= 0 || n_routed < 1 || n_shared < 0 || top_k < 1) return MOE_ERR_INVALID_ARG;
  if (top_k > MOE_MAX_TOP_K || top_k > n_routed) return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_GELU_TANH && activation != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (!(route_scale > 0.0f) || route_scale > 3.0e38f) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FEW_MAX_T || n_routed > MOE_MAX_ROUTED || n_shared > MOE_MAX_SHARED) return MOE_ERR_UNSUPPORTED;
  if (d % 64 != 0 || d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if (d > MOE_FEW_MAX_WIDTH || d_ff > MOE_FEW_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
  const Layout l = layout_of(T, d, d_ff, n_routed, n_shared, top_k, activation == MOE_ACT_SWIGLU, I8 ? 1 : 2);
  if (scratch_bytes < l.bytes) return MOE_ERR_SCRATCH;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0)
    return cudaMemsetAsync(counts, 0, sizeof(int32_t) * n_routed, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  int dev, sms;
  int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  unsigned int* status = status_ptr();
  if (!status) return MOE_ERR_CUDA;
  auto kfn = T <= ONE_SUM_T ? few_tokens_kernel<I8, 1>
             : T <= 16      ? few_tokens_kernel<I8, 2>
                            : few_tokens_kernel<I8, NT_MAX>;
  const size_t smem = sizeof(Smem) + 1024;
  if ((rc = ensure_smem_attr((const void*)kfn, smem)) != MOE_OK) return rc;

  uint8_t* base = static_cast<uint8_t*>(scratch);
  Params p{};
  p.x = reinterpret_cast<const uint8_t*>(x);
  p.w_r = reinterpret_cast<const uint8_t*>(w_router);
  p.bias = bias;
  p.offset = logit_offset;
  p.w1s = w1s;
  p.w2s = w2s;
  p.T = T;
  p.d = d;
  p.f = d_ff;
  p.n_routed = n_routed;
  p.n_shared = n_shared;
  p.k = top_k;
  p.swiglu = activation == MOE_ACT_SWIGLU;
  p.gate_scale = route_scale;
  p.topk_idx = topk_idx;
  p.gates = gates;
  p.counts = counts;
  p.out = reinterpret_cast<__nv_bfloat16*>(out);
  p.bar = reinterpret_cast<unsigned int*>(base + l.bar);
  p.logits = reinterpret_cast<float*>(base + l.logits);
  p.xq = base + l.xq;
  p.xs = reinterpret_cast<float*>(base + l.xs);
  p.u = reinterpret_cast<float*>(base + l.u);
  p.h = base + l.h;
  p.hs = reinterpret_cast<float*>(base + l.hs);
  p.y = reinterpret_cast<float*>(base + l.y);
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  p.s_log[0] = l.s_log[0];
  p.s_log[1] = l.s_log[1];
  CUtensorMap tm1, tm2;
  const int f1 = p.swiglu ? 2 * d_ff : d_ff;
  if ((rc = weight_map(&tm1, w1, I8, d, f1, n_routed + n_shared, p.swiglu != 0, &p.plain_map[0])) != MOE_OK) return rc;
  if ((rc = weight_map(&tm2, w2, I8, d_ff, d, n_routed + n_shared, false, &p.plain_map[1])) != MOE_OK) return rc;
  const int rg_n = (n_routed + n_shared + ROWS - 1) / ROWS;
  const int nch_r = (d * 2 + BOX - 1) / BOX;
  // a chunk of K for every warp, in slices of as many CTAs as there are (every slice is read again by every
  // CTA's selection, so no more than that)
  p.ks = (nch_r + WARPS - 1) / WARPS;
  if (p.ks > KS_MAX) p.ks = KS_MAX;
  if (p.ks > sms / rg_n) p.ks = sms / rg_n > 1 ? sms / rg_n : 1;

  // the barriers and the ticket counter start at zero
  if (cudaMemsetAsync(base + l.bar, 0, l.logits - l.bar, s) != cudaSuccess) return MOE_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kfn, tm1, tm2, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace few
}  // namespace moe

using namespace moe;

extern "C" size_t moe_few_tokens_scratch_bytes(int T, int d, int d_ff, int n_routed, int n_shared, int top_k) {
  if (T <= 0 || T > MOE_FEW_MAX_T || d <= 0 || d > MOE_FEW_MAX_WIDTH || d_ff <= 0 || d_ff > MOE_FEW_MAX_WIDTH ||
      n_routed < 1 || n_shared < 0 || n_shared > MOE_MAX_SHARED || top_k < 1 || top_k > MOE_MAX_TOP_K)
    return 256;
  // what any form of the call with up to T tokens needs (fewer tokens may have more slices of K, and need more)
  size_t most = 0;
  for (int t = 1; t <= T; ++t)
    for (int form = 0; form < 4; ++form) {
      const size_t b = few::layout_of(t, d, d_ff, n_routed, n_shared, top_k, (form & 1) != 0, 1 + (form >> 1)).bytes;
      most = b > most ? b : most;
    }
  return most;
}

extern "C" int moe_few_tokens(const moe_bf16* x, const moe_bf16* w_router, const float* bias,
                              const float* logit_offset, const moe_bf16* w1, const moe_bf16* w2, int T, int d,
                              int d_ff, int n_routed, int n_shared, int top_k, float route_scale, int activation,
                              int32_t* topk_idx, float* gates, int32_t* counts, moe_bf16* out, void* scratch,
                              size_t scratch_bytes, void* stream) {
  return few::run<false>(x, w_router, bias, logit_offset, w1, nullptr, w2, nullptr, T, d, d_ff, n_routed, n_shared,
                         top_k, route_scale, activation, topk_idx, gates, counts, out, scratch, scratch_bytes, stream);
}

extern "C" int moe_few_tokens_int8(const moe_bf16* x, const moe_bf16* w_router, const float* bias,
                                   const float* logit_offset, const int8_t* w1, const float* w1_scale,
                                   const int8_t* w2, const float* w2_scale, int T, int d, int d_ff, int n_routed,
                                   int n_shared, int top_k, float route_scale, int activation, int32_t* topk_idx,
                                   float* gates, int32_t* counts, moe_bf16* out, void* scratch, size_t scratch_bytes,
                                   void* stream) {
  return few::run<true>(x, w_router, bias, logit_offset, w1, w1_scale, w2, w2_scale, T, d, d_ff, n_routed, n_shared,
                        top_k, route_scale, activation, topk_idx, gates, counts, out, scratch, scratch_bytes, stream);
}
