// Gradients of the combine (moe_combine_backward).
//
// A workgroup holds its token's d_out row in registers, walks the token's
// local slots, and for each reads the expert row once for the weight's
// gradient and writes the row's gradient.  Bound by HBM, per local row H * 4
// bytes in and out: 4096 x 7168, 32 of 256 experts here and a shared one, 80
// us = 5.1 TB/s (one piece of four columns at a time and sums through LDS: 98
// us).
#include <type_traits>

#include "block.h"
#include "rows.h"

namespace moe {

namespace {

// A thread takes two pieces of four columns a pass and a workgroup as many
// threads as the row needs, up to 1024 (4096 x 7168: 79 us; 256 threads with
// four pieces and two passes 85 us, 512 with four pieces 80 us).
constexpr int kPieces = 2;
constexpr int kMostThreads = 1024;

// Every wavefront holds the token's slots in its lanes, so the walk over the
// local ones needs no exchange.  A pass's pieces of d_out and of a slot's row
// are requested together; rows are read and written once, past the caches in
// a batch that does not fit them (STREAM).
template <typename T, bool STREAM>
__global__ __launch_bounds__(kMostThreads) void k_combine_backward(
    const T* __restrict__ d_out, const float* __restrict__ y_perm,
    const int32_t* __restrict__ pair_row, const float* __restrict__ w, int T_,
    int H, int k, int cap, float* __restrict__ d_y_perm,
    float* __restrict__ d_w, float* __restrict__ d_y_shared) {
  __shared__ float part[2][kMostThreads / 64][MOE_KMAX];   // by token parity
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int NT = blockDim.x, waves = NT >> 6;
  int par = 0;
  for (long t = blockIdx.x; t < T_; t += gridDim.x, par ^= 1) {
    int row = -1;
    float wt = 0.0f;
    if (lane < k) {
      row = pair_row[t * k + lane];
      wt = w[t * k + lane];
      if (row >= cap) row = -1;
    }
    float sums = 0.0f;                         // lane j: slot j, this wavefront's columns
    for (int c0 = 0; c0 < H; c0 += 4 * kPieces * NT) {
      Piece pc[kPieces];
      f32x4_t d[kPieces];
#pragma unroll
      for (int v = 0; v < kPieces; ++v) {
        pc[v] = piece_at<4, kAligned>(c0 + 4 * (threadIdx.x + v * NT), H);
        d[v] = widen<T, 4>(own_cols<T, 4, kAligned>(
            load_piece<T, 4, kAligned, STREAM>(d_out + t * H, pc[v], H), pc[v]));
      }
      uint64_t m = __ballot(row >= 0);
      while (m) {
        const int j = __ffsll((unsigned long long)m) - 1;
        m &= m - 1;
        const size_t at = (size_t)__builtin_amdgcn_readlane(row, j) * H;
        if (d_w) {
          f32x4_t y[kPieces];
#pragma unroll
          for (int v = 0; v < kPieces; ++v)
            y[v] = widen<float, 4>(own_cols<float, 4, kAligned>(
                load_piece<float, 4, kAligned, STREAM>(y_perm + at, pc[v], H), pc[v]));
          float s = 0.0f;
#pragma unroll
          for (int v = 0; v < kPieces; ++v) s += dot_cols<4>(d[v], y[v]);
          s = wave_sum(s);
          if (lane == j) sums += s;
        }
        if (d_y_perm) {
          const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wt), j));
#pragma unroll
          for (int v = 0; v < kPieces; ++v)
            store_piece<float, 4, kAligned, STREAM>(d_y_perm + at, pc[v], H, wj * d[v]);
        }
      }
      if (d_y_shared) {
#pragma unroll
        for (int v = 0; v < kPieces; ++v)
          store_piece<float, 4, kAligned, STREAM>(d_y_shared + t * H, pc[v], H, d[v]);
      }
    }
    if (d_w) {
      if (lane < k) part[par][wv][lane] = sums;
      lds_barrier();
      if (threadIdx.x < k) {
        float s = part[par][0][lane];
        for (int v = 1; v < waves; ++v) s += part[par][v][lane];
        d_w[t * k + lane] = s;
      }
    }
  }
}

}  // namespace

hipError_t launch_combine_backward(const void* d_out, int out_dtype,
                                   const float* y_perm,
                                   const int32_t* pair_row, const float* w,
                                   int T, int H, int k, int cap,
                                   float* d_y_perm, float* d_w,
                                   float* d_y_shared, hipStream_t s) {
  const dim3 grid(T < (1 << 20) ? T : (1 << 20));
  const int nt = (H + 4 * kPieces - 1) / (4 * kPieces);
  const dim3 block(nt < kMostThreads ? (nt + 63) / 64 * 64 : kMostThreads);
  const bool stream = (double)T * H * 8 >= 64.0 * 1048576.0;
  by_type(out_dtype, [&](auto type) {
    using D = decltype(type);
    by_flag(stream, [&](auto st) {
      k_combine_backward<D, st.value><<<grid, block, 0, s>>>(
          (const D*)d_out, y_perm, pair_row, w, T, H, k, cap, d_y_perm, d_w,
          d_y_shared);
    });
  });
  return hipGetLastError();
}

}  // namespace moe
