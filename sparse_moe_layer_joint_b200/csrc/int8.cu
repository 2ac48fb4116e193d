// int8.cu -- 8-bit codes of rows (int8.cuh), for weights (a row is an output
// channel) and activations (a row is a token), and the dispatch that codes each
// token once and writes it to its experts' rows.
//
// Bound: HBM, 2 bytes read and 1 (dispatch: top_k or top_k + 1) written a value.
// A row is held in registers between its maximum and its codes (VEC 16-byte
// vectors a thread, TPR threads a row), so it is read once; rows too long for
// that are read a second time, from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "int8.cuh"
#include "moe.h"
#include "moe_internal.h"

namespace moe {
namespace q8 {

constexpr int THREADS = 256;
constexpr int VEC = 4;  // 16-byte vectors of a row a thread holds

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

// Maximum over the TPR threads that share a row (a power of two; whole warps above 32).
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* part) {
  constexpr int W = TPR < 32 ? TPR : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (TPR <= 32) return m;
  const int warp = threadIdx.x >> 5;
  constexpr int WPR = TPR > 32 ? TPR / 32 : 1;
  __syncthreads();  // the previous row's parts have been read
  if ((threadIdx.x & 31) == 0) part[warp] = m;
  __syncthreads();
  const int first = warp / WPR * WPR;
  for (int i = 0; i < WPR; ++i) m = max(m, part[first + i]);
  return m;
}

template <int TPR, bool LONG>
__global__ void __launch_bounds__(THREADS) code_rows_kernel(const Params p) {
  __shared__ uint32_t part[THREADS / 32];
  constexpr int RPB = THREADS / TPR;  // rows a block works on at once
  const int lane = threadIdx.x % TPR;
  // every thread runs every iteration (the row maximum is a block-wide step)
  for (long long r0 = (long long)blockIdx.x * RPB; r0 < p.rows; r0 += (long long)gridDim.x * RPB) {
    const long long r = r0 + threadIdx.x / TPR;
    const bool live = r < p.rows;
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
    m = row_max<TPR>(m, part);
    if (!live) continue;
    const RowScale rs = row_scale(__uint_as_float(m << 16));
    auto put = [&](int c, const uint4& src) {
      const uint2 code = code8(src, rs);
      if (p.q) p.q[r * p.nv + c] = code;
      if (p.token_row)
        for (int j = 0; j < p.k; ++j) {
          const int to = __ldg(p.token_row + r * p.k + j);
          if (to >= 0 && to < p.n_rows) p.xq[(long long)to * p.nv + c] = code;
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
      if (p.token_row)
        for (int j = 0; j < p.k; ++j) {
          const int to = __ldg(p.token_row + r * p.k + j);
          if (to >= 0 && to < p.n_rows) p.xs[to] = rs.scale;
        }
    }
  }
}

template <int TPR, bool LONG>
int launch(const Params& p, int sms, cudaStream_t s) {
  constexpr int RPB = THREADS / TPR;
  const long long want = (p.rows + RPB - 1) / RPB;
  const long long most = (long long)sms * 8;
  code_rows_kernel<TPR, LONG><<<(int)(want < most ? want : most), THREADS, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

// Threads a row: the fewest (of 8 to 256) whose VEC vectors hold the whole row.
int run(const Params& p, cudaStream_t s) {
  int dev, sms;
  const int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  if (p.nv <= 8 * VEC) return launch<8, false>(p, sms, s);
  if (p.nv <= 32 * VEC) return launch<32, false>(p, sms, s);
  if (p.nv <= 64 * VEC) return launch<64, false>(p, sms, s);
  if (p.nv <= 128 * VEC) return launch<128, false>(p, sms, s);
  if (p.nv <= 256 * VEC) return launch<256, false>(p, sms, s);
  return launch<256, true>(p, sms, s);
}

}  // namespace q8
}  // namespace moe

using namespace moe;

extern "C" int moe_int8_quantize_rows(const moe_bf16* x, long long rows, int K, int8_t* q, float* scale,
                                      void* stream) {
  if (rows < 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q) || !aligned4(scale)) return MOE_ERR_INVALID_ARG;
  if (K % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
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
  if (!x || !token_row || !xq || !xs || !aligned16(x) || !aligned4(token_row) || !aligned16(xq) || !aligned4(xs) ||
      !aligned16(xq_tok) || !aligned4(xs_tok) || (xq_tok == nullptr) != (xs_tok == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (d % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
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
