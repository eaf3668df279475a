// Launch functions of the 8-bit checkpoints, of the experts' forward and
// backward pass that use them, and of the layer for a few tokens.
#pragma once

#include "common.h"

namespace moe {

// rows of activations <-> E4M3 codes [T][C] and scales [T][ceil(C / 128)]
hipError_t launch_checkpoint_rows(const void* src, int dtype, long T, int C,
                                  long stride, uint8_t* codes, float* scales,
                                  hipStream_t s);
hipError_t launch_restore_rows(const uint8_t* codes, const float* scales,
                               long T, int C, int dtype, long stride,
                               void* dst, hipStream_t s);
// Rows of checkpointed x [T][C] and of d [T][C], bf16, C a multiple of 128:
// x_out[r] = x[row_token[r]] and d_out[r] = d[row_token[r]] for r < *n_rows (at
// most cap), and x_all[t] = x[t] unless null
hipError_t launch_gather_pair(const uint8_t* codes, const float* scales,
                              const bf16_t* d, const int32_t* row_token,
                              const int32_t* n_rows, int cap, int T, int C,
                              bf16_t* x_out, bf16_t* d_out, bf16_t* x_all,
                              hipStream_t s);

// Rows of the experts' intermediate arrays: routed ones [0, offsets[P]), the
// shared expert's [cap, cap + T).
struct ExpertRows {
  const int32_t* n_routed;    // device: offsets + P
  int cap, T, has_shared, I;
};
// gu [rows][2 I] float32 (gate, then up) -> h = silu(gate) * up in bf16, and
// the checkpoints of gu and of the layer's input x [T][H]
hipError_t launch_swiglu_save(const ExpertRows& r, const float* gu, bf16_t* h,
                              uint8_t* codes, float* scales, const bf16_t* x,
                              int H, uint8_t* x_codes, float* x_scales,
                              hipStream_t s);
// Backward of it from the checkpoint: dh [rows][I] float32 (of the unweighted
// output) -> dgu [rows][2 I] and the weighted h [rows][I] in bf16, and (unless
// null) d_topk_w [T][k]: sum_i dh h of a pair's row, 0 for one that is not
// local.
struct PairRows {
  const int32_t* row_token;   // [cap]
  const float* row_weight;    // [cap]
  const int32_t* pair_row;    // [T][k]
  int k;
};
hipError_t launch_swiglu_backward(const ExpertRows& r, const PairRows& p,
                                  const float* dh, const uint8_t* codes,
                                  const float* scales, bf16_t* dgu, bf16_t* hw,
                                  float* d_topk_w, hipStream_t s);

// Rows of the training GEMMs' tiles: 256, in small passes 64 (gemm_train.hip).
int train_tile_rows(const moe_problem* p);
// The tile list of the training GEMMs: balanced tiles of up to BM rows, the
// shared expert's spread evenly among the routed ones.
hipError_t launch_train_tiles(const int32_t* offsets, int P, int has_shared,
                              int T, int BM, int4* tiles, int32_t* count,
                              hipStream_t s);
// The training GEMMs over that list (see gemm_ring.h).
struct TrainGemm {
  int tile_rows;              // train_tile_rows
  const int4* tiles;
  const int32_t* tile_count;
  int P, cap, T, H, I, has_shared;
  const moe_weights* w;
};
// out [rows][2 I] float32: x Wg, then x Wu, x gathered through a_rows
hipError_t launch_gemm_gate_up(const TrainGemm& g, const bf16_t* x,
                               const int32_t* a_rows, float* out,
                               hipStream_t s);
// y_routed [cap][H], y_shared [T][H] float32: h Wd
hipError_t launch_gemm_down(const TrainGemm& g, const bf16_t* h,
                            float* y_routed, float* y_shared, hipStream_t s);
// out [rows][I] float32: d Wd^T, d [T][H] gathered through a_rows
hipError_t launch_gemm_down_back(const TrainGemm& g, const bf16_t* d,
                                 const int32_t* a_rows, float* out,
                                 hipStream_t s);
// dx_routed [cap][H], dx_shared [T][H] float32: dg Wg^T + du Wu^T
hipError_t launch_gemm_gate_up_back(const TrainGemm& g, const bf16_t* dgu,
                                    float* dx_routed, float* dx_shared,
                                    hipStream_t s);

// Weight gradients (gemm_wgrad.hip): for every group of rows and product, a^T b
// over the group's rows, written to [M][N0] arrays: columns [0, N0) of b to
// out[0], the others to out[1].
struct WeightProduct {
  int M, N, N0;               // columns of a and of b, of an output; multiples of 128
  const bf16_t* a;            // routed rows, in order
  const bf16_t* b;
  const bf16_t* a_shared;     // the shared group's
  const bf16_t* b_shared;
  long lda, ldb;
  void* out[2];               // [P][M][N0]
  void* out_shared[2];        // the shared group's
};
struct WeightGrad {
  int P, T, has_shared;
  const int32_t* offsets;     // [P + 1]
  int dtype;                  // of the outputs
  WeightProduct product[2];
};
hipError_t launch_weight_grad(const WeightGrad& g, hipStream_t s);

}  // namespace moe
