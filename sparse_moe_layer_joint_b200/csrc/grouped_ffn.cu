// grouped_ffn.cu -- the expert MLPs y = W2_e gelu(W1_e x) over groups of rows
// ("Inkling, Dissected" §02: an expert is two matmuls with a nonlinearity), as
// two launches of one persistent, warp-specialised tcgen05 grouped GEMM:
//
//   GEMM1:  H[rows of e] = gelu(X[rows of e] . W1_e^T)   (bf16 out, GELU fused)
//   GEMM2:  Y[rows of e] =      H[rows of e] . W2_e^T    (bf16 out)
//
// Groups.  A launch covers G_r "routed" groups, whose rows are given by device
// offsets (the dispatch layout), followed by G_s "shared" groups that each see
// the same `shared_rows` rows (every token).  Group g uses expert g of the
// weight tensors it is given, so one launch can run the 256 routed and the 2
// shared experts of the layer together.  The tile list, (group, row tile,
// column tile) with the column index fastest, is built on the device from the
// offsets, so the host never reads the per-expert counts.
//
// Per CTA (persistent, static round-robin over tiles):
//   warp 0      TMA producer into a shared-memory ring of A and B tiles
//               (128-byte swizzle, full/empty mbarriers); in gathering launches
//               the routed A rows come from the token rows through the row
//               indices, one tile::gather4 load (four rows) per lane and stage
//   warp 1      TMEM owner + MMA issuer (one thread): tcgen05.mma kind::f16,
//               bf16 in, fp32 accumulators in TMEM: two 256-column
//               accumulator buffers so the epilogue of tile i overlaps the
//               main loop of tile i+1 (one 512-column buffer for WIDE tiles)
//   warps 2-5   epilogue (2-9 for WIDE tiles): tcgen05.ld, activation, bf16,
//               16-byte stores of each row's 64-byte chunks
// Variants:
//   PAIR = false  one CTA per 128 x 256 tile (4-stage ring of 48 KB)
//   PAIR = true   a cluster of two CTAs per 256 x 256 tile with
//                 tcgen05.mma.cta_group::2 (M = 256): CTA rank r holds A rows
//                 r*128.. and B rows (output columns) r*128.. in its own
//                 shared memory and accumulator rows r*128.. in its own TMEM;
//                 both CTAs' loads signal the leader's full barrier, the
//                 leader's MMA thread issues for the pair and commits to both
//                 CTAs' barriers, both epilogues release the accumulator on
//                 the leader.  Per CTA this halves the B operand's shared-
//                 memory traffic (6-stage ring of 32 KB).
//   WIDE          pair tiles of 256 x 512 accumulator columns (see Cfg): 25% fewer
//                 L2 bytes per FLOP and one accumulator, which the epilogue hands
//                 back as soon as it holds its share as packed bf16 registers
//                 (the stores then overlap the next tile's MMAs); SwiGLU tiles
//                 hold 256 gate and the 256 matching up columns; the default for
//                 pair launches (MOE_GEMM_WIDE=0: 256 x 256).
//   half tiles    (pairs, GELU and plain epilogues, groups of at most 1024 rows
//                 on average) a group's last row tile with at most 128 rows runs
//                 as an M = 128 pair MMA: 64 rows a CTA, whose 64 x 256 result
//                 TMEM holds folded (lanes 0-63 the first 128 columns, lanes
//                 64-127 the other 128), at half the MMA work.
// Ragged groups: a tile's A rows may run past its group (into the next
// group's rows, or past the tensor where TMA fills zeros); the epilogue writes
// only the group's own rows.
#include <cuda_runtime.h>
#include <stdint.h>

#include "grouped_gemm.cuh"
#include "moe.h"
#include "moe_internal.h"

using namespace moe;
using namespace moe::gffn;

extern "C" int moe_grouped_ffn(const moe_bf16* rows, const int32_t* offsets, int n_groups, int n_rows,
                               int expert_base, const moe_bf16* w1, const moe_bf16* w2, int d, int d_ff,
                               int activation, moe_bf16* h_scratch, moe_bf16* y, void* stream) {
  if (n_groups < 0 || n_rows < 0 || expert_base < 0 || d <= 0 || d_ff <= 0) return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_GELU_TANH && activation != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool swiglu = activation == MOE_ACT_SWIGLU;
  const int w1_rows = swiglu ? 2 * d_ff : d_ff;  // SwiGLU: gate rows, then up rows
  if (!aligned16(rows) || !aligned16(w1) || !aligned16(w2) || !aligned16(h_scratch) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  if (!rows || !w1 || !w2 || !h_scratch || !y) return MOE_ERR_INVALID_ARG;
  if (d % 64 != 0 || d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if (n_groups > MOE_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
  if (n_rows == 0 || n_groups == 0) return MOE_OK;
  const bool identity = (offsets == nullptr);
  if (!identity && !aligned4(offsets)) return MOE_ERR_INVALID_ARG;
  const long long h_rows = identity ? (long long)n_groups * n_rows : n_rows;
  if (h_rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;

  cudaStream_t s = (cudaStream_t)stream;
  int dev, sms;
  int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  unsigned int* status = status_ptr();
  if (!status) return MOE_ERR_CUDA;

  const bool pair = choose_pair(h_rows, n_groups);
  const int tile_m = pair ? Cfg<true, 4>::TILE_M : Cfg<false, 4>::TILE_M;
  const long long tiles_upper = identity ? (long long)n_groups * ((n_rows + tile_m - 1) / tile_m)
                                         : (n_rows + tile_m - 1) / tile_m + n_groups;

  Params p{};
  p.offsets = offsets;
  p.G_r = identity ? 0 : n_groups;
  p.G_s = identity ? n_groups : 0;
  p.routed_rows = n_rows;
  p.shared_rows = n_rows;
  p.a_sh_map = 0;
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  p.hints = hints_for();
  p.n_major_rows = n_major_rows_for();
  p.prefetch_kb = prefetch_for();

  GemmSpec g1{};
  g1.a0 = rows;
  g1.a0_rows = (uint64_t)n_rows;
  g1.b = reinterpret_cast<const __nv_bfloat16*>(w1) + (size_t)expert_base * w1_rows * d;
  g1.b_rows = (uint64_t)w1_rows;
  g1.p = p;
  g1.p.a_sh_base = 0;
  g1.p.a_sh_stride = 0;  // every shared group reads rows 0..n_rows-1
  g1.p.C0 = g1.p.C1 = reinterpret_cast<__nv_bfloat16*>(h_scratch);
  g1.p.c0_limit = g1.p.c1_limit = (int)h_rows;
  g1.p.c1_base = 0;
  g1.p.c1_stride = n_rows;
  g1.p.N = d_ff;
  g1.p.K = d;
  g1.p.n_tiles_n = swiglu ? (d_ff + SWIGLU_OUT - 1) / SWIGLU_OUT : (d_ff + BN - 1) / BN;
  g1.p.b_up_row = d_ff;
  g1.p.ldc = d_ff;
  const double flop = 2.0 * (double)h_rows * d * d_ff;  // GEMM2; GEMM1 has w1_rows / d_ff times as many
  rc = swiglu ? run_split<EPI_SWIGLU>(g1, pair, stages_for(pair, wide_for(pair, EPI_SWIGLU), 1, 2.0 * flop), sms, tiles_upper, s)
              : run_split<EPI_GELU>(g1, pair, stages_for(pair, wide_for(pair, EPI_GELU), 1, flop), sms, tiles_upper, s);
  if (rc != MOE_OK) return rc;

  GemmSpec g2{};
  g2.a0 = h_scratch;
  g2.a0_rows = (uint64_t)h_rows;
  g2.b = reinterpret_cast<const __nv_bfloat16*>(w2) + (size_t)expert_base * d * d_ff;
  g2.p = p;
  g2.p.a_sh_base = 0;
  g2.p.a_sh_stride = n_rows;
  g2.p.C0 = g2.p.C1 = reinterpret_cast<__nv_bfloat16*>(y);
  g2.p.c0_limit = g2.p.c1_limit = (int)h_rows;
  g2.p.c1_base = 0;
  g2.p.c1_stride = n_rows;
  g2.p.N = d;
  g2.p.K = d_ff;
  g2.p.n_tiles_n = (d + BN - 1) / BN;
  g2.p.ldc = d;
  return run_split<EPI_NONE>(g2, pair, stages_for(pair, wide_for(pair, EPI_NONE), 2, flop), sms, tiles_upper, s);
}

extern "C" int moe_experts_ffn(const moe_bf16* x, const moe_bf16* x_perm, const int32_t* row_token,
                               const int32_t* offsets, int T, int n_routed, int n_shared, int top_k,
                               const moe_bf16* w1, const moe_bf16* w2, int d, int d_ff, int activation,
                               moe_bf16* h_scratch, moe_bf16* y_perm, moe_bf16* y_shared, void* stream) {
  if (T < 0 || n_routed < 0 || n_shared < 0 || top_k < 1 || d <= 0 || d_ff <= 0) return MOE_ERR_INVALID_ARG;
  if (activation != MOE_ACT_GELU_TANH && activation != MOE_ACT_SWIGLU) return MOE_ERR_INVALID_ARG;
  const bool swiglu = activation == MOE_ACT_SWIGLU;
  const int w1_rows = swiglu ? 2 * d_ff : d_ff;  // SwiGLU: gate rows, then up rows
  if (n_routed + n_shared > MOE_MAX_GROUPS) return MOE_ERR_UNSUPPORTED;
  if (d % 64 != 0 || d_ff % 64 != 0) return MOE_ERR_UNSUPPORTED;
  if (!w1 || !w2 || !h_scratch || !aligned16(w1) || !aligned16(w2) || !aligned16(h_scratch))
    return MOE_ERR_INVALID_ARG;
  const bool gather = (x_perm == nullptr);  // routed rows gathered from x through row_token
  if (n_routed > 0 && (!offsets || !y_perm || !aligned16(x_perm) || !aligned4(offsets) || !aligned16(y_perm)))
    return MOE_ERR_INVALID_ARG;
  if (n_routed > 0 && gather && (!x || !row_token || !aligned16(x) || !aligned4(row_token)))
    return MOE_ERR_INVALID_ARG;
  if (n_shared > 0 && (!x || !y_shared || !aligned16(x) || !aligned16(y_shared))) return MOE_ERR_INVALID_ARG;
  const long long R = (long long)T * top_k;
  const long long h_rows = R + (long long)n_shared * T;
  if (h_rows > 0x7fffffffLL) return MOE_ERR_UNSUPPORTED;
  if (T == 0 || n_routed + n_shared == 0) return MOE_OK;

  cudaStream_t s = (cudaStream_t)stream;
  int dev, sms;
  int rc = device_info(&dev, &sms);
  if (rc != MOE_OK) return rc;
  unsigned int* status = status_ptr();
  if (!status) return MOE_ERR_CUDA;

  const int G = n_routed + n_shared;
  const bool pair = choose_pair(h_rows, G);
  const int tile_m = pair ? Cfg<true, 4>::TILE_M : Cfg<false, 4>::TILE_M;
  const long long tiles_upper =
      (R + tile_m - 1) / tile_m + n_routed + (long long)n_shared * ((T + tile_m - 1) / tile_m);

  Params p{};
  p.offsets = offsets;
  p.G_r = n_routed;
  p.G_s = n_shared;
  p.routed_rows = (int)R;
  p.shared_rows = T;
  p.timeout_ns = wait_timeout_ns();
  p.status = status;
  p.hints = hints_for();
  p.n_major_rows = n_major_rows_for();
  p.prefetch_kb = prefetch_for();

  // GEMM1: routed rows from x_perm, or gathered from x through row_token (map 0), shared rows from x
  // (map 1); H = [routed rows | shared s rows]
  GemmSpec g1{};
  const bool routed_gather = n_routed > 0 && gather;
  g1.a0 = (n_routed > 0 && !gather) ? (const void*)x_perm : (const void*)x;
  g1.a0_rows = (n_routed > 0 && !gather) ? (uint64_t)R : (uint64_t)T;
  g1.a0_box_rows = routed_gather ? 1u : 128u;  // gather4 loads take a tensor map whose box is one row
  g1.a1 = n_shared > 0 ? (const void*)x : nullptr;
  g1.a1_rows = (uint64_t)T;
  g1.b = w1;
  g1.b_rows = (uint64_t)w1_rows;
  g1.p = p;
  g1.p.gather_rows = routed_gather ? row_token : nullptr;
  g1.p.gather_limit = T;
  g1.p.a_sh_map = (n_routed > 0 || n_shared == 0) ? 1 : 0;
  g1.p.a_sh_base = 0;
  g1.p.a_sh_stride = 0;
  g1.p.C0 = g1.p.C1 = reinterpret_cast<__nv_bfloat16*>(h_scratch);
  g1.p.c0_limit = (int)R;
  g1.p.c1_base = (int)R;
  g1.p.c1_stride = T;
  g1.p.c1_limit = (int)h_rows;
  g1.p.N = d_ff;
  g1.p.K = d;
  g1.p.n_tiles_n = swiglu ? (d_ff + SWIGLU_OUT - 1) / SWIGLU_OUT : (d_ff + BN - 1) / BN;
  g1.p.b_up_row = d_ff;
  g1.p.ldc = d_ff;
  const double flop = 2.0 * (double)h_rows * d * d_ff;  // GEMM2; GEMM1 has w1_rows / d_ff times as many
  rc = swiglu ? run_split<EPI_SWIGLU>(g1, pair, stages_for(pair, wide_for(pair, EPI_SWIGLU), 1, 2.0 * flop), sms, tiles_upper, s)
              : run_split<EPI_GELU>(g1, pair, stages_for(pair, wide_for(pair, EPI_GELU), 1, flop), sms, tiles_upper, s);
  if (rc != MOE_OK) return rc;

  // GEMM2: all A rows from H (map 0); routed outputs to y_perm, shared outputs to y_shared
  GemmSpec g2{};
  g2.a0 = h_scratch;
  g2.a0_rows = (uint64_t)h_rows;
  g2.b = w2;
  g2.p = p;
  g2.p.a_sh_map = 0;
  g2.p.a_sh_base = (int)R;
  g2.p.a_sh_stride = T;
  g2.p.C0 = reinterpret_cast<__nv_bfloat16*>(y_perm);
  g2.p.c0_limit = (int)R;
  g2.p.C1 = reinterpret_cast<__nv_bfloat16*>(y_shared);
  g2.p.c1_base = 0;
  g2.p.c1_stride = T;
  g2.p.c1_limit = n_shared * T;
  g2.p.N = d;
  g2.p.K = d_ff;
  g2.p.n_tiles_n = (d + BN - 1) / BN;
  g2.p.ldc = d;
  return run_split<EPI_NONE>(g2, pair, stages_for(pair, wide_for(pair, EPI_NONE), 2, flop), sms, tiles_upper, s);
}
