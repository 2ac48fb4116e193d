// int8.cu -- 8-bit codes of rows (int8.cuh), for weights (a row is an output
// channel) and activations (a row is a token), and the dispatch that codes each
// token once and writes it to its experts' rows.
//
// Bound: HBM, 2 bytes read and 1 (dispatch: top_k or top_k + 1) written a value.
// A row is held in registers between its maximum and its codes (VEC 16-byte
// vectors a thread, TPR threads a row), so it is read once; rows of more than
// 16384 values are read a second time, from L2.  A value costs one conversion, one
// fma and three quarters of a byte permute (int8.cuh): 24570 rows of 2048 take 25.8
// us in the kernel alone (5.9 TB/s; 28 a call when calls follow each other), the
// dispatch of 16384 tokens of 4096 to six experts 94 (6.4 TB/s; 98), one 2048 x 7168
// matrix 12 (7.9 when it lies in L2; its 1024 blocks are 1.4 waves of the 740 that 96
// registers a thread allow), the dispatch of 64 tokens of 7168 3.1 (8).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8.cuh"
#include "moe.h"
#include "moe_internal.h"

namespace moe {
namespace q8 {

struct Params {
  const uint4* x;
  long long rows;
  int nv;  // 16-byte vectors per row
  // dispatch: the row's copies
  const int32_t* token_row;  // null: q and scale alone
  int k;
  int n_rows;
  uint2* xq;
  float* xs;
  uint2* q;  // may be null
  float* scale;
};

constexpr int MIN_THREADS = 128;

// Maximum over the TPR threads that share a row (a power of two; whole warps above 32).
template <int TPR, int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part) {
  if (TPR >= 32) {
    m = __reduce_max_sync(0xffffffffu, m);
  } else {
#pragma unroll
    for (int o = TPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  }
  if (TPR <= 32) return m;
  constexpr int WPR = TPR > 32 ? TPR / 32 : 1;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) part[warp] = m;
  __syncthreads();
  const int first = warp / WPR * WPR;
#pragma unroll
  for (int i = 0; i < WPR; ++i) m = max(m, part[first + i]);
  return m;
}

// TPR threads a row, each holding VEC of its 16-byte vectors; LONG: rows with more than TPR * VEC of them.
template <int TPR, int VEC, bool LONG, int THREADS>
__global__ void __launch_bounds__(THREADS) code_rows_kernel(const Params p) {
  __shared__ uint32_t part[THREADS / 32];
  const int lane = threadIdx.x % TPR;
  const long long r = (long long)blockIdx.x * (THREADS / TPR) + threadIdx.x / TPR;
  const bool live = r < p.rows;  // a dead row's threads still take part in the block's maximum
  const uint4* row = p.x + r * p.nv;
  uint4 v[VEC];
  uint32_t m = 0;
  if (live) {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const int c = lane + i * TPR;
      v[i] = c < p.nv ? __ldg(row + c) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) m = max(m, abs_max_bits(v[i]));
    if (LONG)
      for (int c = lane + VEC * TPR; c < p.nv; c += TPR) m = max(m, abs_max_bits(__ldg(row + c)));
  }
  m = row_max<TPR, THREADS>(m, part);
  if (!live) return;
  const RowScale rs = row_scale(__uint_as_float(m << 16));
  // the row's copies: its place in token order, and the rows its experts take
  long long to[MOE_MAX_TOP_K];
#pragma unroll
  for (int j = 0; j < MOE_MAX_TOP_K; ++j) {
    to[j] = -1;
    if (p.token_row && j < p.k) {
      const int t = __ldg(p.token_row + r * p.k + j);
      if (t >= 0 && t < p.n_rows) to[j] = t;
    }
  }
  auto put = [&](int c, const uint4& src) {
    const uint2 code = code8(src, rs);
    if (p.q) p.q[r * p.nv + c] = code;
    if (p.token_row) {
#pragma unroll
      for (int j = 0; j < MOE_MAX_TOP_K; ++j)
        if (to[j] >= 0) p.xq[to[j] * p.nv + c] = code;
    }
  };
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const int c = lane + i * TPR;
    if (c < p.nv) put(c, v[i]);
  }
  if (LONG)
    for (int c = lane + VEC * TPR; c < p.nv; c += TPR) put(c, __ldg(row + c));
  if (lane == 0) {
    if (p.scale) p.scale[r] = rs.scale;
#pragma unroll
    for (int j = 0; j < MOE_MAX_TOP_K; ++j)
      if (to[j] >= 0) p.xs[to[j]] = rs.scale;
  }
}

template <int TPR, int VEC, bool LONG = false>
int launch(const Params& p, cudaStream_t s) {
  constexpr int THREADS = TPR > MIN_THREADS ? TPR : MIN_THREADS;
  const long long blocks = (p.rows + THREADS / TPR - 1) / (THREADS / TPR);
  if (blocks > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  code_rows_kernel<TPR, VEC, LONG, THREADS><<<(int)blocks, THREADS, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Threads a row.  Many rows: 16 vectors a thread, so that few threads hold a row's loads in flight and short blocks
// replace each other (30000 rows of 7168: 98 us at 64 threads, 111 at 128, 123 at 256).  Few rows, where latency counts,
// and the dispatch, whose stores outweigh its loads: 8 vectors (one token of 4096, top-6: 6.1 against 8.2 us; 16384 tokens:
// 94 against 97).
int run(const Params& p, cudaStream_t s) {
  if (p.nv > 2048) return launch<512, 8, true>(p, s);
  if (p.nv <= 32) return launch<8, 4>(p, s);
  if (p.rows <= 1024 || p.token_row) {
    if (p.nv <= 128) return launch<32, 4>(p, s);
    if (p.nv <= 256) return launch<32, 8>(p, s);
    if (p.nv <= 512) return launch<64, 8>(p, s);
    if (p.nv <= 1024) return launch<128, 8>(p, s);
    return launch<256, 8>(p, s);
  }
  if (p.nv <= 64) return launch<16, 4>(p, s);
  if (p.nv <= 128) return launch<16, 8>(p, s);
  if (p.nv <= 256) return launch<32, 8>(p, s);
  if (p.nv <= 512) return launch<32, 16>(p, s);
  if (p.nv <= 1024) return launch<64, 16>(p, s);
  return launch<128, 16>(p, s);
}

}  // namespace q8
}  // namespace moe

using namespace moe;

extern "C" int moe_int8_quantize_rows(const moe_bf16* x, long long rows, int K, int8_t* q, float* scale,
                                      void* stream) {
  if (rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return K % 8 != 0 ? MOE_ERR_UNSUPPORTED : MOE_OK;  // tensors without elements may have no address
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned4(scale)) return MOE_ERR_INVALID_ARG;
  if (K % 8 != 0) return MOE_ERR_UNSUPPORTED;
  q8::Params p{};
  p.x = reinterpret_cast<const uint4*>(x);
  p.rows = rows;
  p.nv = K / 8;
  p.q = reinterpret_cast<uint2*>(q);
  p.scale = scale;
  return q8::run(p, (cudaStream_t)stream);
}

extern "C" int moe_int8_dispatch(const moe_bf16* x, const int32_t* token_row, int T, int d, int top_k, int n_rows,
                                 int8_t* xq, float* xs, int8_t* xq_tok, float* xs_tok, void* stream) {
  if (T < 0 || d <= 0 || top_k < 1 || top_k > MOE_MAX_TOP_K || n_rows < 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return d % 8 != 0 ? MOE_ERR_UNSUPPORTED : MOE_OK;  // tensors without elements may have no address
  if (!x || !token_row || !xq || !xs || !aligned16(x) || !aligned4(token_row) || !aligned16(xq) || !aligned4(xs) ||
      !aligned16(xq_tok) || !aligned4(xs_tok) || (xq_tok == nullptr) != (xs_tok == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  q8::Params p{};
  p.x = reinterpret_cast<const uint4*>(x);
  p.rows = T;
  p.nv = d / 8;
  p.token_row = token_row;
  p.k = top_k;
  p.n_rows = n_rows;
  p.xq = reinterpret_cast<uint2*>(xq);
  p.xs = xs;
  p.q = reinterpret_cast<uint2*>(xq_tok);
  p.scale = xs_tok;
  return q8::run(p, (cudaStream_t)stream);
}
