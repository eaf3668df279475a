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

// One workgroup, a thread a group.  Tiles of routed groups wait for their
// weights where an expert has some hundred rows, the shared expert's for the
// matrix cores: side by side they fill each other's gaps.  Routed tile r goes
// to place r + floor(r S / R), shared tile j to j + ceil((j + 1) R / S), of R
// and S of them.
__global__ __launch_bounds__(1024) void k_train_tiles(
    const int32_t* __restrict__ offsets, int P, int has_shared, int T, int BM,
    int4* __restrict__ tiles, int32_t* __restrict__ count) {
  __shared__ int32_t wave_sum[16];
  const int g = threadIdx.x, lane = g & 63, wv = g >> 6;
  const int start = g < P ? offsets[g] : 0;
  const int rows = g < P ? offsets[g + 1] - start : 0;
  int per = 1, sper = 1;
  const int n = tile_split(rows, BM, 1, &per);
  const int S = has_shared ? tile_split(T, BM, 1, &sper) : 0;
  int upto = n;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d, 64);
    if (lane >= d) upto += o;
  }
  if (lane == 63) wave_sum[wv] = upto;
  __syncthreads();
  int before = upto - n, R = 0;
  for (int v = 0; v < 16; ++v) {
    if (v < wv) before += wave_sum[v];
    R += wave_sum[v];
  }
  for (int i = 0; i < n; ++i) {
    const long r = before + i;
    tiles[r + (R > 0 ? r * S / R : 0)] = make_int4(g, start + i * per, min(per, rows - i * per), 0);
  }
  for (int j = g; j < S; j += 1024)
    tiles[j + ((long)(j + 1) * R + S - 1) / S] = make_int4(P, j * sper, min(sper, T - j * sper), 0);
  if (g == 0) count[0] = R + S;
}

}  // namespace

hipError_t launch_train_tiles(const int32_t* offsets, int P, int has_shared,
                              int T, int BM, int4* tiles, int32_t* count,
                              hipStream_t s) {
  k_train_tiles<<<1, 1024, 0, s>>>(offsets, P, has_shared, T, BM, tiles, count);
  return hipGetLastError();
}

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
