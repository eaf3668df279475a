// GEMMs of the experts' training passes on the ring of gemm_ring.h: the gate
// and up products kept apart for their checkpoint, down, and the backward of
// both from the forward's packed weights.  The backward's reduction runs over
// the weight's output channels, 16 of which are the rows of a packed block,
// so its operand comes out of LDS transposed (ds_read_b64_tr_b16) and no
// second copy of the weights is laid out.
//
// 4096 tokens of 7168 x 2048, 32 of 256 experts (128 rows each) and the shared
// one: gate/up 535-545 us, down 320-325, back through down 355-360, back through
// gate and up 630 (0.7 to 0.9 PFLOP/s).  Routed tiles are half full and
// wait for their weights (2.9 GB a pass); the shared expert's tiles between them
// fill the gaps, and an output in float32 (134 to 235 MB) is the price of an
// activation that is checkpointed from unrounded products.
#include <algorithm>
#include <cmath>

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

// Small passes, whose 256 x 256 tiles would not fill the GPU and whose time is
// the latency of their stages: 64 rows x 64 columns of B (G_PAIR: 32 of gate
// and 32 of up) from four wavefronts of 32 x 32, stages of 64 of the reduction
// (16 KiB), four in LDS and one in registers, two workgroups a CU.  509 tokens
// of 1024 x 512, 2 of 16 experts each: gate/up 13.2 us, down 9.6, back through
// down 10.1 and through gate and up 14.8 (12.5 in the mean); stages of 128, one
// workgroup a CU 18.8, 11.4 and 15 in the mean of the two; the ring on 256 x 256
// tiles 23.7, 14.5 and 23.9, on 64 x 128 tiles (stages of 32) 25.4, 15.4 and 29.
constexpr int kSmallRows = 64, kSmallColumns = 64;

template <int MODE>
__global__ __launch_bounds__(256, 2) void k_gemm_small(GArgs a) {
  // a stage: 64 rows of 128 bytes, their 8 chunks at chunk ^ (row % 8), then
  // the weight's 8 packed blocks
  __shared__ u32x4_t l0[1024], l1[1024], l2[1024], l3[1024];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  const int c16 = lane & 15, c32 = lane & 31, hi = (lane >> 4) & 1, ks = lane >> 5;
  const int K = a.K, N = a.N, KT = K / 64;
  const int total = a.tile_count[0] * a.nb_per_tile;
  for (int item = blockIdx.x; item < total; item += gridDim.x) {
    const int tile = item / a.nb_per_tile, nb = item - tile * a.nb_per_tile;
    const int4 td = a.tiles[tile];
    const int g = td.x, row0 = td.y, nrows = td.z;
    const bool sh = g == a.P;
    const char* W0 = (const char*)(sh ? a.w0_sh : a.w0_arr[g]);
    const char* W1 = a.w1_arr ? (const char*)(sh ? a.w1_sh : a.w1_arr[g]) : W0;
    // a transfer moves eight rows of A (lane: row lane / 8, chunk slot lane %
    // 8), or one block of the weight
    const char* arow[2];
    const char* block[2];
    const char* block1[2];               // G_BACK: of the reduction's second half
    const int half = MODE == G_BACK && a.w1_arr ? KT / 2 : KT;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int x = w + 4 * h, r = 8 * x + (lane >> 3);
      const int rr = row0 + (r < nrows ? r : 0);       // (padded rows: unused)
      const size_t src = sh ? rr : (a.a_rows ? a.a_rows[rr] : rr);
      arow[h] = (const char*)(sh ? a.a_shared : a.a_routed) + src * K * 2 + (((lane ^ r) & 7) * 16);
      block1[h] = nullptr;
      if (MODE == G_BACK) {              // block x: 16 of the reduction, 32 columns
        const size_t at = ((size_t)(x >> 1) * (N / 32) + nb * 2 + (x & 1)) * 1024 + lane * 16;
        block[h] = W0 + at;
        block1[h] = W1 + at - (size_t)half * N * 128;
      } else {                           // 16 columns, 32 of the reduction
        const int col = x >> 1;
        const char* W = MODE == G_PAIR && col >= 2 ? W1 : W0;
        const int n16 = MODE == G_PAIR ? nb * 2 + (col & 1) : nb * 4 + col;
        block[h] = W + ((size_t)n16 * (K / 32) + (x & 1)) * 1024 + lane * 16;
      }
    }
    auto issue = [&](int kt, u32x4_t* L) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds_dma16(arow[h] + (size_t)kt * 128, L + (w + 4 * h) * 64);
        const char* b = MODE != G_BACK ? block[h] + (size_t)kt * 2048
                        : (kt < half ? block[h] : block1[h]) + (size_t)kt * N * 128;
        lds_dma16(b, L + 512 + (w + 4 * h) * 64);
      }
    };
    f32x16_t acc = {};
    const int row = wm * 32 + c32;
    const int tr = ((8 * ks + (c16 >> 2)) + 16 * (2 * hi + ((c16 >> 1) & 1))) * 16 +
                   (c16 & 1) * 8 + 8192 + wn * 1024;
    auto load = [&](const u32x4_t* L, u32x4_t (&fa)[4], u32x4_t (&fb)[4]) {
      int t = tr;
      asm volatile("" : "+v"(t));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        fa[s] = L[row * 8 + ((2 * s + ks) ^ (row & 7))];
        if constexpr (MODE == G_BACK) {
          const u32x2g_t lo = lds_read_tr(L, t + s * 2048);
          const u32x2g_t up = lds_read_tr(L, t + s * 2048 + 64);
          fb[s] = u32x4_t{lo.x, lo.y, up.x, up.y};
        } else {
          fb[s] = L[512 + ((2 * wn + hi) * 2 + (s >> 1)) * 64 + c16 + 16 * (2 * (s & 1) + ks)];
        }
      }
    };
    lds_barrier();                       // the previous item is done with the ring
    const int last = KT - 1;
    issue(0, l0);
    issue(min(1, last), l1);
    issue(min(2, last), l2);
    issue(min(3, last), l3);
    u32x4_t fa0[4], fb0[4], fa1[4], fb1[4];
    WAIT_VMCNT(12);
    lds_barrier();
    load(l0, fa0, fb0);
    // step k: wait for this wavefront's part of stage k + 1 (8 younger
    // transfers), barrier (stage k + 1 complete, stage k read), fetch stage
    // k + 4 into stage k's slot, read stage k + 1, multiply stage k.  Past the
    // end the last stage is fetched and read again, and goes unused.
#define SMALL_STEP(S, L, NEXT, A, B, NA, NB)                                 \
    {                                                                        \
      WAIT_VMCNT(8);                                                         \
      lds_barrier();                                                         \
      issue(min(kt + S + 4, last), L);                                       \
      load(NEXT, NA, NB);                                                    \
      __builtin_amdgcn_sched_barrier(0);                                     \
      if (S < 2 || kt + S < KT)                                              \
        for (int s = 0; s < 4; ++s) acc = mfma32b(A[s], B[s], acc);          \
    }
    // (KT is even.  A way out of the loop in its middle would cost the
    // compiler the knowledge of which slot is read, and it would wait for all.)
    for (int kt = 0; kt < KT; kt += 4) {
      SMALL_STEP(0, l0, l1, fa0, fb0, fa1, fb1)
      SMALL_STEP(1, l1, l2, fa1, fb1, fa0, fb0)
      SMALL_STEP(2, l2, l3, fa0, fb0, fa1, fb1)
      SMALL_STEP(3, l3, l0, fa1, fb1, fa0, fb0)
    }
#undef SMALL_STEP
    WAIT_VMCNT(0);                       // the trailing re-reads have landed
    // lane: column c32, rows 8 (r / 4) + 4 ks + r % 4
    float* y;
    int ld = N;
    if (MODE == G_PAIR) {
      ld = 2 * N;
      y = a.y_routed + ((size_t)(sh ? a.cap : 0) + row0) * ld + wn * N + nb * 32 + c32;
    } else {
      y = (sh ? a.y_shared : a.y_routed) + (size_t)row0 * ld + nb * 64 + wn * 32 + c32;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int at = wm * 32 + 8 * (r >> 2) + 4 * ks + (r & 3);
      if (at < nrows) y[(size_t)at * ld] = acc[r];
    }
  }
}

// `share`: outputs a column block has, of the columns of its B (G_PAIR: half)
template <int MODE>
hipError_t launch(const TrainGemm& g, GArgs& a, int share, int chunk, hipStream_t s) {
  if (g.tile_rows == kSmallRows) {
    a.nb_per_tile = a.N * share / kSmallColumns;
    k_gemm_small<MODE><<<512, 256, 0, s>>>(a);
    return hipGetLastError();
  }
  const int columns = 32 * kGemmTN * kGemmWN / share;
  a.nb_per_tile = (a.N + columns - 1) / columns;
  a.chunk_cols = chunk_cols(a.nb_per_tile, chunk);
  // persistent: one workgroup per CU (128 KiB of LDS)
  k_gemm_bf16<MODE, kGemmTM, kGemmTN, kGemmWM, kGemmWN>
      <<<256, 64 * kGemmWM * kGemmWN, 0, s>>>(a);
  return hipGetLastError();
}

// One workgroup, a thread a group.  Tiles of routed groups wait for their
// weights where an expert has some hundred rows, the shared expert's for the
// matrix cores: side by side they fill each other's gaps.  Routed tile r goes
// to place r + floor(r S / R), shared tile j to j + ceil((j + 1) R / S), of R
// and S of them.  4096 tokens of 7168 x 2048, 32 of 256 experts: gate/up 536 us,
// down 321, back through down 358, back through gate and up 630 (1845 in all);
// the routed tiles first 546, 345, 360 and 643 (1894), the shared first 566, 344,
// 346 and 662 (1918).
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

// Small tiles where the gate and up products are up to 96 of their stages a CU
// (tiles of evenly loaded groups x columns x reduction).  Whole passes on small
// and on 256 x 256 tiles, forward and backward, us: 16 experts of 1024 x 512,
// 2 a token, 1021 tokens (32 stages) 56 and 75 against 74 and 99, 2039 tokens
// (64) 82 and 108 against 96 and 125, 4093 tokens (128) 125 and 177 against
// 110 and 163; of 2048 x 1024, 509 tokens (64) 81 and 136 against 98 and 158,
// 2039 tokens (256) 182 and 262 against 147 and 238.
int train_tile_rows(const moe_problem* p) {
  const double pairs = (double)p->T * p->k * p->num_local / p->E;
  const double groups = std::max(1.0, std::min((double)p->num_physical, pairs));
  const double tiles = groups * std::ceil(pairs / groups / kSmallRows) +
                       (p->has_shared ? std::ceil((double)p->T / kSmallRows) : 0.0);
  return tiles * (2.0 * p->I / kSmallColumns) * (p->H / 64) <= 96.0 * 256 ? kSmallRows : kGemmRows;
}

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
  return launch<G_PAIR>(g, a, 2, 8, s);
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
  return launch<G_DOWN_ANY>(g, a, 1, 4, s);
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
  return launch<G_BACK>(g, a, 1, 8, s);
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
  return launch<G_BACK>(g, a, 1, 4, s);
}

}  // namespace moe
