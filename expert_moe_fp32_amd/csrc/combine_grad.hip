// Gradients of the combine (moe_combine_backward).
//
// A workgroup holds its token's d_out row in registers, walks the token's
// local slots, and for each reads the expert row once for the weight's
// gradient and writes the row's gradient.  Bound by HBM: per local row H * 4
// bytes in and out.
#include <type_traits>

#include "block.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kCols = 4 * kThreads;       // columns of one pass

template <typename T>
__device__ __forceinline__ f32x4_t load4(const T* p) {
  if constexpr (sizeof(T) == 4) {
    return *(const f32x4_t*)p;
  } else {
    typedef __attribute__((ext_vector_type(2))) uint32_t u2;
    const u2 u = *(const u2*)p;
    return f32x4_t{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u),
                   __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u)};
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void k_combine_backward(
    const T* __restrict__ d_out, const float* __restrict__ y_perm,
    const int32_t* __restrict__ pair_row, const float* __restrict__ w, int T_,
    int H, int k, int cap, float* __restrict__ d_y_perm,
    float* __restrict__ d_w, float* __restrict__ d_y_shared) {
  __shared__ float part[4][MOE_KMAX];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  for (long t = blockIdx.x; t < T_; t += gridDim.x) {
    __syncthreads();
    if (threadIdx.x < 4 * MOE_KMAX) part[0][threadIdx.x] = 0.0f;
    __syncthreads();
    for (int c0 = 0; c0 < H; c0 += kCols) {
      const int col = c0 + 4 * threadIdx.x;
      f32x4_t d = {0.f, 0.f, 0.f, 0.f};
      if (col < H) {
        d = load4<T>(d_out + t * H + col);
        if (d_y_shared) *(f32x4_t*)(d_y_shared + t * H + col) = d;
      }
      for (int j = 0; j < k; ++j) {
        const int row = pair_row[t * k + j];
        if (row < 0 || row >= cap) continue;
        const float wj = w[t * k + j];
        float s = 0.0f;
        if (col < H) {
          if (d_w) {
            const f32x4_t y = *(const f32x4_t*)(y_perm + (size_t)row * H + col);
            s = d.x * y.x + d.y * y.y + d.z * y.z + d.w * y.w;
          }
          if (d_y_perm) *(f32x4_t*)(d_y_perm + (size_t)row * H + col) = wj * d;
        }
        if (d_w) {
#pragma unroll
          for (int m = 32; m >= 1; m >>= 1) s += __shfl_xor(s, m, 64);
          if (lane == 0) part[wv][j] += s;
        }
      }
    }
    __syncthreads();
    if (d_w && threadIdx.x < k) {
      const int j = threadIdx.x;
      d_w[t * k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
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
  if (out_dtype == MOE_BF16)
    k_combine_backward<bf16_t><<<grid, kThreads, 0, s>>>(
        (const bf16_t*)d_out, y_perm, pair_row, w, T, H, k, cap, d_y_perm, d_w,
        d_y_shared);
  else
    k_combine_backward<float><<<grid, kThreads, 0, s>>>(
        (const float*)d_out, y_perm, pair_row, w, T, H, k, cap, d_y_perm, d_w,
        d_y_shared);
  return hipGetLastError();
}

}  // namespace moe
