// Launch functions and shared helpers of the operators around the expert
// layer: scored routing, the residual norm, and the combine's gradients.
#pragma once

#include "common.h"

namespace moe {

hipError_t launch_count_ids(const int32_t* ids, int n, int E, int32_t* counts,
                            hipStream_t s);

// Scored routing.  `counts` (optional) needs route_scored_partials(...) int32
// of scratch when that is not 0; route_scored_scratch(...) serves every batch
// of up to T tokens.
size_t route_scored_partials(const moe_router* r);
size_t route_scored_scratch(const moe_router* r);
hipError_t launch_route_scored(const moe_router* r, const void* logits,
                               const float* bias, int32_t* ids, float* w,
                               int32_t* counts, int32_t* partials,
                               hipStream_t s);
hipError_t launch_route_scored_backward(const moe_router* r,
                                        const void* logits,
                                        const int32_t* ids, const float* d_w,
                                        void* d_logits, hipStream_t s);

// Residual norm; `comb` gives the combined expert rows in place of y.
struct CombineSource {
  const float* y_perm;
  const int32_t* pair_row;
  const float* w;
  const float* y_shared;   // or null
  int k, cap;
  void* block_out;         // or null
};
struct NormArgs {
  const void* y;           // or null
  const void* resid;
  const void* post_gain;   // or null
  const float* gate;       // or null
  const void* pre_gain;    // or null
  void* resid_out;         // or null
  void* x_out;             // or null
};
hipError_t launch_residual_norm(const moe_norm* n, const NormArgs& a,
                                const CombineSource* comb, hipStream_t s);

struct NormGradArgs {
  const void* y;           // or null
  const void* resid_out;   // or null
  const void* post_gain;   // or null
  const float* gate;       // or null
  const void* pre_gain;    // or null
  const void* d_x;         // or null
  const void* d_resid_out; // or null
  void* d_y;               // or null
  void* d_resid;           // or null
  float* d_post;           // or null
  float* d_gate;           // or null
  float* d_pre;            // or null
};
size_t norm_grad_partials(const moe_norm* n);   // floats of scratch
size_t norm_grad_scratch(const moe_norm* n);    // ... for up to T rows
hipError_t launch_residual_norm_backward(const moe_norm* n,
                                         const NormGradArgs& a,
                                         float* partials, hipStream_t s);

hipError_t launch_combine_backward(const void* d_out, int out_dtype,
                                   const float* y_perm,
                                   const int32_t* pair_row, const float* w,
                                   int T, int H, int k, int cap,
                                   float* d_y_perm, float* d_w,
                                   float* d_y_shared, hipStream_t s);

}  // namespace moe
