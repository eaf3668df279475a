// GEMMs of the experts' training passes on the ring of gemm_ring.h: the gate
// and up products kept apart for their checkpoint, down, and the backward of
// both from the forward's packed weights.  The backward's reduction runs over
// the weight's output channels, 16 of which are the rows of a packed block,
// so its operand comes out of LDS transposed (ds_read_b64_tr_b16) and no
// second copy of the weights is laid out.
#include "gemm_ring.h"
#include "train.h"

namespace moe {

namespace {

GArgs args(const TrainGemm& g, int K, int N) {
  GArgs a{};
  a.tiles = g.tiles;
  a.tile_count = g.tile_count;
  a.P = g.P;
  a.cap = g.cap;
  a.K = K;
  a.N = N;
  return a;
}

template <int MODE>
hipError_t launch(GArgs& a, int columns, int chunk, hipStream_t s) {
  a.nb_per_tile = (a.N + columns - 1) / columns;
  a.chunk_cols = chunk_cols(a.nb_per_tile, chunk);
  // persistent: one workgroup per CU (128 KiB of LDS)
  k_gemm_bf16<MODE, kGemmTM, kGemmTN, kGemmWM, kGemmWN>
      <<<256, 64 * kGemmWM * kGemmWN, 0, s>>>(a);
  return hipGetLastError();
}

constexpr int kColumns = 32 * kGemmTN * kGemmWN;       // of a tile's B

}  // namespace

hipError_t launch_gemm_gate_up(const TrainGemm& g, const bf16_t* x,
                               const int32_t* a_rows, float* out,
                               hipStream_t s) {
  GArgs a = args(g, g.H, g.I);
  a.a_routed = a.a_shared = x;
  a.a_rows = a_rows;
  a.w0_arr = g.w->w_gate;
  a.w1_arr = g.w->w_up;
  a.w0_sh = g.w->sh_gate;
  a.w1_sh = g.w->sh_up;
  a.y_routed = out;
  return launch<G_PAIR>(a, kColumns / 2, 8, s);
}

hipError_t launch_gemm_down(const TrainGemm& g, const bf16_t* h,
                            float* y_routed, float* y_shared, hipStream_t s) {
  GArgs a = args(g, g.I, g.H);
  a.a_routed = h;
  a.a_shared = h + (size_t)g.cap * g.I;
  a.w0_arr = g.w->w_down;
  a.w0_sh = g.w->sh_down;
  a.y_routed = y_routed;
  a.y_shared = y_shared;
  if (a.N % kColumns == 0) return launch<G_DOWN>(a, kColumns, 4, s);
  return launch<G_DOWN_ANY>(a, kColumns, 4, s);
}

hipError_t launch_gemm_down_back(const TrainGemm& g, const bf16_t* d,
                                 const int32_t* a_rows, float* out,
                                 hipStream_t s) {
  GArgs a = args(g, g.H, g.I);
  a.a_routed = a.a_shared = d;
  a.a_rows = a_rows;
  a.w0_arr = g.w->w_down;
  a.w0_sh = g.w->sh_down;
  a.y_routed = out;
  a.y_shared = out + (size_t)g.cap * g.I;
  return launch<G_BACK>(a, kColumns, 8, s);
}

hipError_t launch_gemm_gate_up_back(const TrainGemm& g, const bf16_t* dgu,
                                    float* dx_routed, float* dx_shared,
                                    hipStream_t s) {
  GArgs a = args(g, 2 * g.I, g.H);
  a.a_routed = dgu;
  a.a_shared = dgu + (size_t)g.cap * 2 * g.I;
  a.w0_arr = g.w->w_gate;
  a.w1_arr = g.w->w_up;
  a.w0_sh = g.w->sh_gate;
  a.w1_sh = g.w->sh_up;
  a.y_routed = dx_routed;
  a.y_shared = dx_shared;
  return launch<G_BACK>(a, kColumns, 4, s);
}

}  // namespace moe
