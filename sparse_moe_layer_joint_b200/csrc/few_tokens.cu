// few_tokens.cu -- the whole MoE layer for a few tokens (T <= 64) in one
// cooperative launch, with bf16 or 8-bit experts ("Inkling, Dissected" §02,
// §02b: s = sigmoid(x W_r^T); top-k of s + b; joint gates; y_e = W2_e act(W1_e x);
// out = sum of g y over the kept and the shared experts).
//
// What bounds it: the weights of the experts the tokens touch are read from HBM
// once, (touched + n_shared) * mats * d * d_ff values; everything else is small.
// So the kernel is a weight stream with the layer's other steps hidden behind it:
//
//   weights   A unit of work is 16 rows of one expert matrix (8 gate rows and the
//             8 matching up rows for SwiGLU), a row's K split over kw warps of a
//             CTA.  Units of all touched experts are dealt round-robin to the CTAs
//             (one an SM), so one token's 8 experts spread over every SM where
//             128-row GEMM tiles would occupy a fraction of them.  Each thread
//             copies the 16-byte pieces it will itself feed to the tensor core into
//             a private ring of shared memory (cp.async, NST chunks of 128 bytes of
//             K by 16 rows a warp: up to 128 KB in flight an SM), so the stream
//             needs no barrier, and runs on across units, from W1 into W2, and
//             behind the grid barriers.
//   products  mma.sync m16n8k16 bf16 (m16n8k32 s8): weight rows are M, the expert's
//             tokens N (up to 8 a tile, 8 tiles).  At one to a few tokens an expert
//             the tensor pipe is almost idle at any instruction's rate, and this form
//             takes its weights straight from registers: K may be permuted as long
//             as both operands agree, so lane (r, c) holds 16 contiguous bytes of
//             rows r and r + 8 and of token r, which is exactly what it loads.
//   phases    0  router logits, W_r's rows in groups of 16 by KS slices of K over
//                the CTAs (8-bit: the tokens' codes too); grid barrier
//                then every CTA selects for all T tokens itself (a warp a token)
//             1  h = act(W1 x) for every (touched or shared expert, token) row, kept
//                in fp32 precision: as bf16 high and low parts (the product with
//                both costs no extra weight traffic), or for 8-bit experts fp32, coded per
//                row once the row is complete; grid barrier (8-bit: two)
//             2  y = W2 h in fp32; the CTA that completes a block of 16 output
//                columns (a counter per block) sums it over the experts in the
//                contributors' order, so the result does not depend on timing
//
// The grid barriers need every CTA resident: the launch is cooperative, and every
// wait is bounded (wait_timeout_ns, MOE_STATUS_TIMEOUT).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8.cuh"
#include "moe.h"
#include "moe_internal.h"
#include "sm100.cuh"

namespace moe {
namespace few {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int NST = 5;        // ring stages (chunks) per thread
constexpr int AHEAD = NST - 1;
constexpr int CHUNK = 128;    // bytes of K of one row a chunk holds
constexpr int ROWS = 16;      // weight rows of a unit
constexpr int NT_MAX = MOE_FEW_MAX_T / 8;
constexpr int KS_MAX = 8;     // K slices of the router phase
constexpr int E_LD = 272;     // pitch of a token's partial logits
constexpr int RED_NT = 4;     // token tiles reduced at a time
constexpr int RED_COL = 20;   // floats per token column of a reduced tile (16 rows, padded: conflict-free)
constexpr int RED_TILE = 8 * RED_COL;
constexpr int MAX_CONTRIB = MOE_MAX_TOP_K + MOE_MAX_SHARED;

struct Params {
  const uint8_t* x;    // [T, d] bf16
  const uint8_t* w_r;  // [E, d] bf16
  const float* bias;
  const float* offset;
  const uint8_t* w1;  // [E, f1, d] bf16 or int8
  const uint8_t* w2;  // [E, d, f]
  const float* w1s;   // [E, f1] channel scales (int8)
  const float* w2s;   // [E, d]
  int T, d, f, n_routed, n_shared, k;
  int swiglu;
  float gate_scale;
  int32_t* topk_idx;
  float* gates;
  int32_t* counts;
  __nv_bfloat16* out;
  // scratch
  unsigned int* bar;       // [4] grid barriers, zero at launch
  unsigned int* blk_done;  // [d / 16] experts finished per output block, zero at launch
  float* logits;           // [KS][T][E_LD] partial logits
  uint8_t* xq;             // [T, d] token codes (int8)
  float* xs;               // [T]
  uint8_t* h;              // bf16: [2][R, f] high and low parts; int8: [R, f] fp32
  uint8_t* hq;             // [R, f] row codes (int8)
  float* hs;               // [R]
  float* y;                // [R, d] fp32
  int ks;                  // K slices of the router phase
  int kw1, kw2;            // warps a row's K is split over, in phases 1 and 2
  uint64_t timeout_ns;
  unsigned int* status;
};

struct Smem {
  uint4 ring[NST * 4 * THREADS];
  float red[WARPS * RED_NT * RED_TILE];  // int32 sums for 8-bit experts
  unsigned long long mask[MOE_MAX_ROUTED];  // tokens that picked each expert
  float gate[MOE_FEW_MAX_T * MAX_CONTRIB];
  int pre[MOE_MAX_ROUTED];              // first row of each expert's tokens
  short list[MOE_MAX_ROUTED];           // touched experts in index order
  short pick[MOE_FEW_MAX_T * MOE_MAX_TOP_K];
  short row_of[MOE_FEW_MAX_T * MOE_MAX_TOP_K];  // row of each (token, slot)
  uint8_t row_tok[MOE_FEW_MAX_T * MOE_MAX_TOP_K];
  int warp_rows[8], warp_touched[8];
  int n_touched;
  int flag[WARPS];
  float warp_max[WARPS];
  int abort_flag;
};
static_assert(sizeof(Smem) + 16 <= 232448, "shared memory per CTA");

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

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

__device__ __forceinline__ unsigned int ld_acquire(const unsigned int* p) {
  unsigned int v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Every CTA arrives; the CTA goes on when all have.  False when the wait ran out of time.
__device__ __forceinline__ bool grid_barrier(unsigned int* ctr, const Params& p, Smem* sm) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(ctr, 1u);
    const uint64_t t0 = globaltimer();
    for (uint32_t it = 1; ld_acquire(ctr) < gridDim.x; ++it) {
      if ((it & 63u) == 0 && globaltimer() - t0 > p.timeout_ns) {
        set_status(p.status, MOE_STATUS_TIMEOUT);
        sm->abort_flag = 1;
        break;
      }
    }
    __threadfence();
  }
  __syncthreads();
  return sm->abort_flag == 0;
}

// What a phase's units look like to a warp.
struct Phase {
  const uint8_t* w;   // expert matrices
  size_t e_bytes;     // bytes of one expert's matrix
  int k_bytes;        // bytes of a row
  int nch;            // chunks of a row
  int units;          // units per expert
  int row_mul;        // first row of unit b: b * row_mul
  size_t hi_off;      // bytes from row r to the lane's second row
  int kw, wk;         // warps a row is split over, this warp's place among them
  int w0, stride;     // first unit of this warp's worker, workers in the grid
};

__device__ __forceinline__ Phase make_phase(const uint8_t* w, int rows, int K, int elem, int kw, bool gated, int f) {
  Phase ph;
  const int warp = threadIdx.x >> 5;
  ph.w = w;
  ph.k_bytes = K * elem;
  ph.e_bytes = (size_t)rows * ph.k_bytes;
  ph.nch = (ph.k_bytes + CHUNK - 1) / CHUNK;
  ph.row_mul = gated ? ROWS / 2 : ROWS;
  ph.units = gated ? f / (ROWS / 2) : rows / ROWS;
  ph.hi_off = (size_t)(gated ? f : ROWS / 2) * ph.k_bytes;
  ph.kw = kw;
  ph.wk = warp % kw;
  ph.w0 = (warp / kw) * (int)gridDim.x + (int)blockIdx.x;
  ph.stride = (WARPS / kw) * (int)gridDim.x;
  return ph;
}

// The warp's weight stream: chunk by chunk through its phase-1 units, then its phase-2 units.
struct Stream {
  int phase, u, c, stage;
  bool ready;  // (phase, u) is known and r0 points at it
  const uint8_t* r0;
};

__device__ __forceinline__ int expert_at(const Params& p, const Smem* sm, int j) {
  return j < p.n_shared ? p.n_routed + j : sm->list[j - p.n_shared];
}

__device__ __forceinline__ void stream_point(Stream& s, const Phase& ph, const Params& p, const Smem* sm) {
  const int j = s.u / ph.units, b = s.u - j * ph.units;
  const int lane = threadIdx.x & 31;
  s.r0 = ph.w + (size_t)expert_at(p, sm, j) * ph.e_bytes + (size_t)(b * ph.row_mul + (lane >> 2)) * ph.k_bytes +
         (lane & 3) * 16;
  s.ready = true;
}

// Find the stream's next unit; n_exp experts are known (before the routing only the shared ones, and the
// stream then stays within phase 1).
__device__ __forceinline__ void stream_settle(Stream& s, const Phase& p1, const Phase& p2, int n_exp, bool routed,
                                              const Params& p, const Smem* sm) {
  s.ready = false;
  if (s.phase == 1) {
    if (s.u < n_exp * p1.units) {
      stream_point(s, p1, p, sm);
      return;
    }
    if (!routed) return;
    s.phase = 2;
    s.u = p2.w0;
    s.c = p2.wk;
  }
  if (s.phase == 2 && s.u < n_exp * p2.units) stream_point(s, p2, p, sm);
}

// Issue the next chunk's copies (none when the stream has ended) and close their group.
__device__ __forceinline__ void stream_issue(Stream& s, const Phase& p1, const Phase& p2, int n_exp, bool routed,
                                             const Params& p, Smem* sm) {
  if (s.ready) {
    const bool one = s.phase == 1;
    const int k_bytes = one ? p1.k_bytes : p2.k_bytes;
    const size_t hi_off = one ? p1.hi_off : p2.hi_off;
    const int off = s.c * CHUNK;
    const uint32_t dst = smem_u32(&sm->ring[(size_t)s.stage * 4 * THREADS + threadIdx.x]);
    constexpr uint32_t step = THREADS * 16;
    cp_async_16(dst, s.r0 + off);
    cp_async_16(dst + step, s.r0 + hi_off + off);
    // a row of an odd number of 64-byte halves ends in a half chunk: its second half is zeros
    const bool second = off + 64 < k_bytes;
    const uint8_t* src = s.r0 + off + (second ? 64 : 0);
    cp_async_16_zfill(dst + 2 * step, src, second ? 16 : 0);
    cp_async_16_zfill(dst + 3 * step, src + hi_off, second ? 16 : 0);
    s.c += one ? p1.kw : p2.kw;
    if (s.c >= (one ? p1.nch : p2.nch)) {
      s.c = one ? p1.wk : p2.wk;
      s.u += one ? p1.stride : p2.stride;
      stream_settle(s, p1, p2, n_exp, routed, p, sm);
    }
  }
  cp_async_commit();
  s.stage = s.stage + 1 == NST ? 0 : s.stage + 1;
}

__device__ __forceinline__ uint4 load16(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }

__device__ __forceinline__ void group_sync(int group, int kw) {
  if (kw == 1)
    __syncwarp();
  else
    named_bar_sync(1 + group, kw * 32);
}

// The places of a warp's accumulators in its part of the reduction buffer.
template <class T>
__device__ __forceinline__ void red_store(T* red, const T (&c)[4], int lane) {
  const int r = lane >> 2, col = 2 * (lane & 3);
  red[col * RED_COL + r] = c[0];
  red[(col + 1) * RED_COL + r] = c[1];
  red[col * RED_COL + r + 8] = c[2];
  red[(col + 1) * RED_COL + r + 8] = c[3];
}

template <class T>
__device__ __forceinline__ T red_sum(const T* red, int kw, int at) {
  T v = red[at];
  for (int w = 1; w < kw; ++w) v += red[w * RED_NT * RED_TILE + at];
  return v;
}

// One unit: this warp's chunks of 16 weight rows against the expert's n_e token rows, NT tiles of 8, then the
// sum over the group's warps, handed to epi(column, row, value, value of row + 8) for columns < n_e and
// rows 0..7.  b_base + row(col) * k_bytes is a token row; PARTS > 1: further parts b_part bytes apart.
template <class T, int NT, int PARTS, class RowFn, class EpiFn, class NextFn>
__device__ __forceinline__ void unit(const Phase& ph, int n_e, const uint8_t* b_base, size_t b_part, RowFn row_of_col,
                                     int& stage, Smem* sm, NextFn next, EpiFn epi) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint8_t* bp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int col = j * 8 + (lane >> 2);
    bp[j] = col < n_e ? b_base + (size_t)row_of_col(col) * ph.k_bytes + (lane & 3) * 16 : nullptr;
  }
  T acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0;
  constexpr bool EARLY = NT * PARTS <= 2;  // few enough to hold: the token loads go out before the wait
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int c = ph.wk; c < ph.nch; c += ph.kw) {
    const int off = c * CHUNK;
    const bool second = off + 64 < ph.k_bytes;
    uint4 b[EARLY ? NT * PARTS : 1][2];
    if (EARLY) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < PARTS; ++q) {
          b[j * PARTS + q][0] = bp[j] ? load16(bp[j] + q * b_part + off) : zero;
          b[j * PARTS + q][1] = bp[j] && second ? load16(bp[j] + q * b_part + off + 64) : zero;
        }
    }
    cp_async_wait<AHEAD - 1>();
    const uint4* slot = &sm->ring[(size_t)stage * 4 * THREADS + tid];
    const uint4 lo0 = slot[0], hi0 = slot[THREADS], lo1 = slot[2 * THREADS], hi1 = slot[3 * THREADS];
    stage = stage + 1 == NST ? 0 : stage + 1;
    next();
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        uint4 b0, b1;
        if (EARLY) {
          b0 = b[j * PARTS + q][0];
          b1 = b[j * PARTS + q][1];
        } else {
          b0 = bp[j] ? load16(bp[j] + q * b_part + off) : zero;
          b1 = bp[j] && second ? load16(bp[j] + q * b_part + off + 64) : zero;
        }
        mma_step(acc[j], lo0, hi0, b0);
        mma_step(acc[j], lo1, hi1, b1);
      }
    }
  }
  const int group = warp / ph.kw;
  T* red = reinterpret_cast<T*>(sm->red);
  T* mine = red + warp * RED_NT * RED_TILE;
  const T* base = red + group * ph.kw * RED_NT * RED_TILE;
  const int g_tid = ph.wk * 32 + lane;
#pragma unroll
  for (int j0 = 0; j0 < NT; j0 += RED_NT) {
    if (j0 * 8 >= n_e) break;
    if (j0 > 0) group_sync(group, ph.kw);
#pragma unroll
    for (int j = j0; j < NT && j < j0 + RED_NT; ++j) red_store(mine + (j - j0) * RED_TILE, acc[j], lane);
    group_sync(group, ph.kw);
    const int cols = min(n_e - j0 * 8, RED_NT * 8);
    for (int i = g_tid; i < cols * 8; i += ph.kw * 32) {
      const int col = i >> 3, r = i & 7;
      const int at = (col >> 3) * RED_TILE + (col & 7) * RED_COL + r;
      epi(j0 * 8 + col, r, red_sum(base, ph.kw, at), red_sum(base, ph.kw, at + 8));
    }
  }
  group_sync(group, ph.kw);
}

template <class T, int PARTS, class RowFn, class EpiFn, class NextFn>
__device__ __forceinline__ void unit_any(const Phase& ph, int n_e, const uint8_t* b_base, size_t b_part,
                                         RowFn row_of_col, int& stage, Smem* sm, NextFn next, EpiFn epi) {
  if (n_e <= 8)
    unit<T, 1, PARTS>(ph, n_e, b_base, b_part, row_of_col, stage, sm, next, epi);
  else if (n_e <= 16)
    unit<T, 2, PARTS>(ph, n_e, b_base, b_part, row_of_col, stage, sm, next, epi);
  else
    unit<T, NT_MAX, PARTS>(ph, n_e, b_base, b_part, row_of_col, stage, sm, next, epi);
}

// Phase 0: partial logits of 16 router rows over one slice of K, all tokens.
__device__ __forceinline__ void router_partial(const Params& p, Smem* sm) {
  const int E = p.n_routed + p.n_shared;
  const int rg_n = (E + ROWS - 1) / ROWS;
  const int k_bytes = p.d * 2;
  const int nch = (k_bytes + CHUNK - 1) / CHUNK;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = (p.T + 7) / 8;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (int un = blockIdx.x; un < rg_n * p.ks; un += gridDim.x) {
    const int rg = un % rg_n, ks = un / rg_n;
    const int c_lo = (int)((long long)nch * ks / p.ks), c_hi = (int)((long long)nch * (ks + 1) / p.ks);
    const int r0 = min(rg * ROWS + (lane >> 2), E - 1), r1 = min(rg * ROWS + (lane >> 2) + 8, E - 1);
    const uint8_t* a0 = p.w_r + (size_t)r0 * k_bytes + (lane & 3) * 16;
    const uint8_t* a1 = p.w_r + (size_t)r1 * k_bytes + (lane & 3) * 16;
    float acc[NT_MAX][4];
#pragma unroll
    for (int j = 0; j < NT_MAX; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;
    for (int c = c_lo + warp; c < c_hi; c += WARPS) {
      const int off = c * CHUNK;
      const bool second = off + 64 < k_bytes;
      const uint4 lo0 = load16(a0 + off), hi0 = load16(a1 + off);
      const uint4 lo1 = second ? load16(a0 + off + 64) : zero, hi1 = second ? load16(a1 + off + 64) : zero;
#pragma unroll
      for (int j = 0; j < NT_MAX; ++j) {
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
#pragma unroll
    for (int j0 = 0; j0 < NT_MAX; j0 += RED_NT) {
      if (j0 < nt) {
#pragma unroll
        for (int j = j0; j < j0 + RED_NT; ++j)
          red_store(sm->red + warp * RED_NT * RED_TILE + (j - j0) * RED_TILE, acc[j], lane);
        __syncthreads();
        const int cols = min(p.T - j0 * 8, RED_NT * 8);
        for (int i = tid; i < cols * ROWS; i += THREADS) {
          const int col = i >> 4, r = i & 15;
          const int e = rg * ROWS + r;
          const float v = red_sum(sm->red, WARPS, (col >> 3) * RED_TILE + (col & 7) * RED_COL + r);
          if (e < E) p.logits[((size_t)ks * p.T + j0 * 8 + col) * E_LD + e] = v;
        }
        __syncthreads();
      }
    }
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

// Select for token t with one warp: scores, k rounds of a warp-wide maximum (the lower index on equal
// scores), joint gates with the denominator summed in ascending expert index.
__device__ __forceinline__ void select_token(const Params& p, Smem* sm, int t, bool write) {
  const int lane = threadIdx.x & 31;
  const int E = p.n_routed + p.n_shared;
  constexpr int PER = (MOE_MAX_ROUTED + MOE_MAX_SHARED + 31) / 32;
  float s[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    s[i] = 0.0f;
    key[i] = 0;
    if (e < E) {
      float z = 0.0f;
      for (int q = 0; q < p.ks; ++q) z += __ldcg(p.logits + ((size_t)q * p.T + t) * E_LD + e);
      if (e < p.n_routed) {
        if (p.offset) z += __ldg(p.offset + e);
        s[i] = sigmoid_f32(z);
        key[i] = order_key(s[i] + __ldg(p.bias + e));
      } else {
        s[i] = sigmoid_f32(z);
      }
    }
  }
  float sc[MOE_MAX_TOP_K];
  int id[MOE_MAX_TOP_K];
#pragma unroll
  for (int q = 0; q < MOE_MAX_TOP_K; ++q) {
    id[q] = 0x7fffffff;
    sc[q] = 0.0f;
    if (q < p.k) {
      uint32_t best = 0;
      int e = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (key[i] > best) {  // strictly: the lane's lowest index among equals
          best = key[i];
          e = i * 32 + lane;
        }
      const uint32_t top = __reduce_max_sync(0xffffffffu, best);
      e = (int)__reduce_min_sync(0xffffffffu, best == top ? (uint32_t)e : 0x7fffffffu);
      float mine = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * 32 + lane == e) {
          mine = s[i];
          key[i] = 0;
        }
      id[q] = e;
      sc[q] = __shfl_sync(0xffffffffu, mine, e & 31);
    }
  }
  float den = 0.0f;
  int prev = -1;
#pragma unroll
  for (int q = 0; q < MOE_MAX_TOP_K; ++q) {
    if (q < p.k) {
      int next = 0x7fffffff;
      float ns = 0.0f;
#pragma unroll
      for (int r = 0; r < MOE_MAX_TOP_K; ++r)
        if (id[r] > prev && id[r] < next) {
          next = id[r];
          ns = sc[r];
        }
      den += ns;
      prev = next;
    }
  }
  float sh[MOE_MAX_SHARED];
#pragma unroll
  for (int q = 0; q < MOE_MAX_SHARED; ++q) {
    sh[q] = 0.0f;
    if (q < p.n_shared) {
      const int e = p.n_routed + q;
      float mine = 0.0f;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * 32 + lane == e) mine = s[i];
      sh[q] = __shfl_sync(0xffffffffu, mine, e & 31);
      den += sh[q];
    }
  }
  if (lane == 0) {
    const int G = p.k + p.n_shared;
#pragma unroll
    for (int q = 0; q < MOE_MAX_TOP_K; ++q)
      if (q < p.k) {
        const float g = __fmul_rn(__fdiv_rn(sc[q], den), p.gate_scale);
        sm->gate[t * MAX_CONTRIB + q] = g;
        sm->pick[t * MOE_MAX_TOP_K + q] = (short)id[q];
        atomicOr(&sm->mask[id[q]], 1ull << t);
        if (write) {
          p.topk_idx[t * p.k + q] = id[q];
          p.gates[t * G + q] = g;
        }
      }
#pragma unroll
    for (int q = 0; q < MOE_MAX_SHARED; ++q)
      if (q < p.n_shared) {
        const float g = __fmul_rn(__fdiv_rn(sh[q], den), p.gate_scale);
        sm->gate[t * MAX_CONTRIB + p.k + q] = g;
        if (write) p.gates[t * G + p.k + q] = g;
      }
  }
}

// The routing tables of all tokens, built by every CTA for itself.
__device__ __forceinline__ void route_all(const Params& p, Smem* sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int t = warp; t < p.T; t += WARPS) select_token(p, sm, t, t % (int)gridDim.x == (int)blockIdx.x);
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
    sm->pre[tid] = rows - n;
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
  }
  __syncthreads();
}

// 8-bit experts, between the phases: each warp codes whole rows of h.
__device__ __forceinline__ void code_hidden(const Params& p, int R) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int nv = p.f / 4;
  for (int r = warp * (int)gridDim.x + (int)blockIdx.x; r < R; r += WARPS * (int)gridDim.x) {
    const float4* row = reinterpret_cast<const float4*>(p.h) + (size_t)r * nv;
    float m = 0.0f;
    bool bad = false;
    for (int i = lane; i < nv; i += 32) {
      const float4 v = row[i];
      const float a = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
      bad |= !(v.x - v.x == 0.0f) || !(v.y - v.y == 0.0f) || !(v.z - v.z == 0.0f) || !(v.w - v.w == 0.0f);
      m = fmaxf(m, a);
    }
    m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
    if (__any_sync(0xffffffffu, bad)) m = INFINITY;
    const q8::RowScale rs = q8::row_scale(m);
    for (int i = lane; i < nv; i += 32) {
      const float4 v = row[i];
      const float a[4] = {v.x, v.y, v.z, v.w};
      reinterpret_cast<uint32_t*>(p.hq)[(size_t)r * nv + i] = q8::code4_f32(a, rs);
    }
    if (lane == 0) p.hs[r] = rs.scale;
  }
}

template <bool I8>
__global__ void __launch_bounds__(THREADS, 1) few_tokens_kernel(const Params p) {
  using T = typename AccT<I8>::type;
  extern __shared__ uint8_t smem_raw[];
  Smem* sm = reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 15) & ~uintptr_t(15));
  const int tid = threadIdx.x;
  constexpr int ELEM = I8 ? 1 : 2;
  const int f1 = p.swiglu ? 2 * p.f : p.f;
  const Phase p1 = make_phase(p.w1, f1, p.d, ELEM, p.kw1, p.swiglu != 0, p.f);
  const Phase p2 = make_phase(p.w2, p.d, p.f, ELEM, p.kw2, false, p.f);

  if (tid < MOE_MAX_ROUTED) sm->mask[tid] = 0;
  if (tid == 0) sm->abort_flag = 0;

  // the shared experts' first weights need no routing: their copies run behind phase 0
  Stream st;
  st.phase = 1;
  st.u = p1.w0;
  st.c = p1.wk;
  st.stage = 0;
  int issued = 0;
  stream_settle(st, p1, p2, p.n_shared, false, p, sm);
  for (; issued < AHEAD && st.ready; ++issued) stream_issue(st, p1, p2, p.n_shared, false, p, sm);

  if (I8) code_tokens(p, sm);
  router_partial(p, sm);
  bool ok = grid_barrier(&p.bar[0], p, sm);
  if (ok) {
    route_all(p, sm);
    const int n_exp = p.n_shared + sm->n_touched;
    if (!st.ready) stream_settle(st, p1, p2, n_exp, true, p, sm);
    for (; issued < AHEAD; ++issued) stream_issue(st, p1, p2, n_exp, true, p, sm);
    auto next = [&]() { stream_issue(st, p1, p2, n_exp, true, p, sm); };
    int stage = 0;
    const int R = p.T * (p.k + p.n_shared);

    // phase 1: hidden rows
    for (int u = p1.w0; u < n_exp * p1.units; u += p1.stride) {
      const int j = u / p1.units, b = u - j * p1.units;
      const int e = expert_at(p, sm, j);
      const bool shared = j < p.n_shared;
      const int n_e = shared ? p.T : __popcll(sm->mask[e]);
      const int row0 = shared ? p.T * p.k + j * p.T : sm->pre[e];
      auto tok = [&](int col) { return shared ? col : (int)sm->row_tok[row0 + col]; };
      auto put = [&](int col, int hc, float v) {
        const size_t at = (size_t)(row0 + col) * p.f + hc;
        if (I8) {
          reinterpret_cast<float*>(p.h)[at] = v;
        } else {
          const __nv_bfloat16 hi = __float2bfloat16_rn(v);
          __nv_bfloat16* hp = reinterpret_cast<__nv_bfloat16*>(p.h);
          hp[at] = hi;
          // an infinite or NaN high part has no low part
          const float lo = v - __bfloat162float(hi);
          hp[at + (size_t)R * p.f] = __float2bfloat16_rn(lo - lo == 0.0f ? lo : 0.0f);
        }
      };
      auto epi = [&](int col, int r, T a, T c) {
        float va = (float)a, vc = (float)c;
        const int ra = b * p1.row_mul + r;  // weight row of a; c's is 8 on, or the up row
        if (I8) {
          const float xs = __ldcg(p.xs + tok(col));
          const float* ws = p.w1s + (size_t)e * f1;
          va *= xs * __ldg(ws + ra);
          vc *= xs * __ldg(ws + (p.swiglu ? p.f + ra : ra + 8));
        }
        if (p.swiglu) {
          put(col, ra, silu_f32(va) * vc);
        } else {
          put(col, ra, gelu_tanh_exp_f32(va));
          put(col, ra + 8, gelu_tanh_exp_f32(vc));
        }
      };
      unit_any<T, 1>(p1, n_e, I8 ? p.xq : p.x, 0, tok, stage, sm, next, epi);
    }
    ok = grid_barrier(&p.bar[1], p, sm);
    if (I8 && ok) {
      code_hidden(p, R);
      ok = grid_barrier(&p.bar[2], p, sm);
    }

    // phase 2: expert outputs, and the sum over the experts of each completed block of columns
    for (int u = p2.w0; ok && u < n_exp * p2.units; u += p2.stride) {
      const int j = u / p2.units, b = u - j * p2.units;
      const int e = expert_at(p, sm, j);
      const bool shared = j < p.n_shared;
      const int n_e = shared ? p.T : __popcll(sm->mask[e]);
      const int row0 = shared ? p.T * p.k + j * p.T : sm->pre[e];
      auto row = [&](int col) { return row0 + col; };
      auto epi = [&](int col, int r, T a, T c) {
        float va = (float)a, vc = (float)c;
        const int ra = b * ROWS + r;
        if (I8) {
          const float hs = __ldcg(p.hs + row0 + col);
          va *= hs * __ldg(p.w2s + (size_t)e * p.d + ra);
          vc *= hs * __ldg(p.w2s + (size_t)e * p.d + ra + 8);
        }
        float* yr = p.y + (size_t)(row0 + col) * p.d + ra;
        yr[0] = va;
        yr[8] = vc;
      };
      unit_any<T, I8 ? 1 : 2>(p2, n_e, I8 ? p.hq : p.h, (size_t)R * p.f * 2, row, stage, sm, next, epi);
      // unit() ended with the group's barrier: its stores are issued; the last expert to arrive adds up
      const int group = (tid >> 5) / p2.kw, g_tid = p2.wk * 32 + (tid & 31);
      if (g_tid == 0) {
        __threadfence();
        sm->flag[group] = atomicAdd(&p.blk_done[b], 1u) == (unsigned)(n_exp - 1);
        __threadfence();
      }
      group_sync(group, p2.kw);
      if (sm->flag[group]) {
        for (int i = g_tid; i < p.T * ROWS; i += p2.kw * 32) {
          const int t = i / ROWS, col = b * ROWS + i % ROWS;
          float a = 0.0f;
          for (int q = 0; q < p.k; ++q)
            a = fmaf(sm->gate[t * MAX_CONTRIB + q],
                     __ldcg(p.y + (size_t)sm->row_of[t * MOE_MAX_TOP_K + q] * p.d + col), a);
          for (int q = 0; q < p.n_shared; ++q)
            a = fmaf(sm->gate[t * MAX_CONTRIB + p.k + q],
                     __ldcg(p.y + (size_t)(p.T * p.k + q * p.T + t) * p.d + col), a);
          p.out[(size_t)t * p.d + col] = __float2bfloat16_rn(a);
        }
      }
      group_sync(group, p2.kw);  // the flag is free again
    }
  }
  cp_async_wait<0>();
}

// Scratch layout: byte offsets of each part.
struct Layout {
  size_t bar, blk, logits, xq, xs, h, hq, hs, y, bytes;
};

inline Layout layout_of(int T, int d, int f, int n_shared, int k) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const size_t R = (size_t)T * (k + n_shared);
  l.bar = take(4 * sizeof(unsigned int));
  l.blk = take((size_t)(d / ROWS) * sizeof(unsigned int));
  l.logits = take((size_t)KS_MAX * T * E_LD * sizeof(float));
  l.xq = take((size_t)T * d);
  l.xs = take((size_t)T * sizeof(float));
  l.h = take(R * f * sizeof(float));
  l.hq = take(R * f);
  l.hs = take(R * sizeof(float));
  l.y = take(R * d * sizeof(float));
  l.bytes = at;
  return l;
}

// Warps a row is split over: a power of two that leaves each warp at least four chunks, so the sum over the
// warps at a unit's end stays small beside the unit.
inline int split_for(int nch) {
  int kw = 1;
  while (kw < WARPS && nch / (2 * kw) >= 4) kw *= 2;
  return kw;
}

template <bool I8>
int run(const moe_bf16* x, const moe_bf16* w_router, const float* bias, const float* logit_offset, const void* w1,
        const float* w1s, const void* w2, const float* w2s, int T, int d, int d_ff, int n_routed, int n_shared,
        int top_k, float route_scale, int activation, int32_t* topk_idx, float* gates, int32_t* counts, moe_bf16* out,
        void* scratch, size_t scratch_bytes, void* stream) {
  if (!x || !w_router || !bias || !w1 || !w2 || !topk_idx || !gates || !counts || !out || !scratch)
    return MOE_ERR_INVALID_ARG;
  if (I8 && (!w1s || !w2s)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w1) || !aligned16(w2) || !aligned16(out) ||
      !aligned16(scratch) || !aligned4(bias) || !aligned4(logit_offset) || !aligned4(topk_idx) || !aligned4(gates) ||
      !aligned4(counts) || !aligned4(w1s) || !aligned4(w2s))
    return MOE_ERR_INVALID_ARG;
  if (T < 0 || d <= 0 || d_ff <= 0 || n_routed < 1 || n_shared < 0 || top_k < 1) return MOE_ERR_INVALID_ARG;
  if (top_k > MOE_MAX_TOP_K || top_k > n_routed) return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_GELU_TANH && activation != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  if (!(route_scale > 0.0f) || route_scale > 3.0e38f) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FEW_MAX_T || n_routed > MOE_MAX_ROUTED || n_shared > MOE_MAX_SHARED) return MOE_ERR_UNSUPPORTED;
  if (d % 64 != 0 || d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if (d > MOE_FEW_MAX_WIDTH || d_ff > MOE_FEW_MAX_WIDTH) return MOE_ERR_UNSUPPORTED;
  const Layout l = layout_of(T, d, d_ff, n_shared, top_k);
  if (scratch_bytes < l.bytes) return MOE_ERR_SCRATCH;
  cudaStream_t s = (cudaStream_t)stream;
  if (T == 0)
    return cudaMemsetAsync(counts, 0, sizeof(int32_t) * n_routed, s) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  int dev, sms;
  int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  unsigned int* status = status_ptr();
  if (!status) return MOE_ERR_CUDA;
  auto kfn = few_tokens_kernel<I8>;
  const size_t smem = sizeof(Smem) + 16;
  if ((rc = ensure_smem_attr((const void*)kfn, smem)) != MOE_OK) return rc;

  uint8_t* base = static_cast<uint8_t*>(scratch);
  Params p{};
  p.x = reinterpret_cast<const uint8_t*>(x);
  p.w_r = reinterpret_cast<const uint8_t*>(w_router);
  p.bias = bias;
  p.offset = logit_offset;
  p.w1 = static_cast<const uint8_t*>(w1);
  p.w2 = static_cast<const uint8_t*>(w2);
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
  p.blk_done = reinterpret_cast<unsigned int*>(base + l.blk);
  p.logits = reinterpret_cast<float*>(base + l.logits);
  p.xq = base + l.xq;
  p.xs = reinterpret_cast<float*>(base + l.xs);
  p.h = base + l.h;
  p.hq = base + l.hq;
  p.hs = reinterpret_cast<float*>(base + l.hs);
  p.y = reinterpret_cast<float*>(base + l.y);
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  const int elem = I8 ? 1 : 2;
  p.kw1 = split_for((d * elem + CHUNK - 1) / CHUNK);
  p.kw2 = split_for((d_ff * elem + CHUNK - 1) / CHUNK);
  const int rg_n = (n_routed + n_shared + ROWS - 1) / ROWS;
  const int nch_r = (d * 2 + CHUNK - 1) / CHUNK;
  p.ks = sms / rg_n;
  p.ks = p.ks < 1 ? 1 : (p.ks > KS_MAX ? KS_MAX : p.ks);
  if (p.ks > nch_r) p.ks = nch_r;

  // the barriers and block counters (adjacent at the start of the scratch) start at zero
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
  if (cudaLaunchKernelEx(&cfg, kfn, p) != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace few
}  // namespace moe

using namespace moe;

extern "C" size_t moe_few_tokens_scratch_bytes(int T, int d, int d_ff, int n_routed, int n_shared, int top_k) {
  (void)n_routed;
  if (T <= 0 || d <= 0 || d_ff <= 0 || n_shared < 0 || top_k < 1) return 256;
  return few::layout_of(T, d, d_ff, n_shared, top_k).bytes;
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
