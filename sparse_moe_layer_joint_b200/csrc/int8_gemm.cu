// int8_gemm.cu -- the experts' products in 8-bit codes with a scale for each
// token (A row) and each output channel (weight row): the grouped GEMM of
// grouped_gemm.cuh on kind::i8 tensor cores.  The int32 sums are exact, so a
// result is one product of the two scales and the sum, whatever the tiling.
//
// Why single CTAs of 128 x 256, although a pair's 256 x 256 tile reads a third less into
// each SM: 128-row tiles leave less of a group's last tile empty, and where they do not
// the power limit, not the reads, sets the pace of calls that follow each other.  Even
// groups, calls back to back, pairs with four and with five stages against single CTAs:
// 144 to 256 rows a group (K 7168, N 2048, GELU) 6 to 9% slower with four, 1% faster to
// 4% slower with five (224 rows: 1112 and 1043 against 1051 us); 512 rows 4 and 1%
// slower; 1536 rows 11 and 9%; 64 to 128 and 320 to 384 rows, whose last 256-row tile is
// half empty, 33 to 70%; random or skewed sizes of 192 to 512 rows on average 5 to 41%.
// (The fastest of eight repetitions, before the limit sets in, was up to 8% faster on pairs.)
// Eight epilogue warps drain one accumulator while the other fills, and send their
// outputs through shared memory so that every store is whole sectors.
//
// What bounds it.  Many rows: 8-bit products take half the tensor time of bf16 at the
// same bytes a row of K, so a 128 x 256 tile asks L2 for 96 bytes a clock, more than
// the 64 or so that an SM gets, and under a sustained load the power limit lowers the
// clock.  256 groups of 192 rows, K 7168, N 2048, GELU: 219 us a quarter of it alone
// (1.65 POP/s; the weights and rows take 163 at 6.53 TB/s), 990 to 1120 us for all of
// it back to back (by GPU).  32 groups of 1536 rows: 585 to 640 us (2.25 to 2.47
// POP/s).  Few rows: the weights.  256 groups of 1.5 rows, K 4096, 2 x 1024 channels
// (SwiGLU): 279 to 300 us, 5.6 to 6.0 TB/s.
#include <cuda_runtime.h>
#include <stdint.h>

#include "grouped_gemm.cuh"
#include "moe.h"
#include "moe_internal.h"

using namespace moe;
using namespace moe::gffn;

extern "C" int moe_int8_grouped_gemm(const int8_t* aq, const float* a_scale, const int32_t* offsets, int n_groups,
                                     int n_rows, int expert_base, const int8_t* wq, const float* w_scale, int N,
                                     int K, int epilogue, moe_bf16* out, void* stream) {
  if (n_groups < 0 || n_rows < 0 || expert_base < 0 || N <= 0 || K <= 0) return MOE_ERR_INVALID_ARG;
  if (epilogue != MOE_INT8_EPI_BF16 && epilogue != MOE_INT8_EPI_GELU && epilogue != MOE_INT8_EPI_SWIGLU)
    return MOE_ERR_INVALID_ARG;
  const bool empty = n_rows == 0 || n_groups == 0;  // tensors without elements may have no address
  if (!empty && (!aq || !a_scale || !wq || !w_scale || !out)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(aq) || !aligned4(a_scale) || !aligned4(offsets) || !aligned16(wq) || !aligned16(w_scale) ||
      !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || K > 131072 || N % 32 != 0 || N > 0x3fffffff || n_groups > MOE_MAX_GROUPS)
    return MOE_ERR_UNSUPPORTED;
  if (empty) return MOE_OK;
  const bool identity = offsets == nullptr;
  const long long out_rows = identity ? (long long)n_groups * n_rows : n_rows;
  if (out_rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;

  cudaStream_t s = (cudaStream_t)stream;
  int dev, sms;
  int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  unsigned int* status = status_ptr();
  if (!status) return MOE_ERR_CUDA;

  const bool swiglu = epilogue == MOE_INT8_EPI_SWIGLU;
  const int w_rows = swiglu ? 2 * N : N;
  constexpr int TILE_M = Cfg<false, 4, false, true>::TILE_M;
  const long long tiles_upper = identity ? (long long)n_groups * ((n_rows + TILE_M - 1) / TILE_M)
                                         : (n_rows + TILE_M - 1) / TILE_M + n_groups;

  GemmSpec g{};
  g.a0 = aq;
  g.a0_rows = (uint64_t)n_rows;
  g.b = wq + (size_t)expert_base * w_rows * K;
  g.b_rows = (uint64_t)w_rows;
  Params& p = g.p;
  p.offsets = offsets;
  p.G_r = identity ? 0 : n_groups;
  p.G_s = identity ? n_groups : 0;
  p.routed_rows = n_rows;
  p.shared_rows = n_rows;
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  p.n_major_rows = n_major_rows_for(4);
  p.a_scale = a_scale;
  p.b_scale = w_scale + (size_t)expert_base * w_rows;
  p.b_scale_ld = w_rows;
  p.C0 = p.C1 = reinterpret_cast<__nv_bfloat16*>(out);
  p.c0_limit = p.c1_limit = (int)out_rows;
  p.c1_stride = n_rows;
  p.N = N;
  p.K = K;
  p.n_tiles_n = swiglu ? (N + SWIGLU_OUT - 1) / SWIGLU_OUT : (N + BN - 1) / BN;
  p.b_up_row = N;
  p.ldc = N;
  switch (epilogue) {
    case MOE_INT8_EPI_BF16: return run_gemm<EPI_NONE, true>(g, false, 4, sms, tiles_upper, s);
    case MOE_INT8_EPI_GELU: return run_gemm<EPI_GELU, true>(g, false, 4, sms, tiles_upper, s);
    default: return run_gemm<EPI_SWIGLU, true>(g, false, 4, sms, tiles_upper, s);
  }
}
