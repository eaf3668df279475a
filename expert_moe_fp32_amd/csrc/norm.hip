// Residual norm (moe_residual_norm), the combine fused into it
// (moe_combine_norm), and its gradients.
//
// One workgroup holds a token's row in registers, eight neighbouring columns
// a thread and pass (VPT passes), so every array is read and written once and
// the two mean squares cost one exchange of a partial sum per wavefront each.
// Bound by HBM: forward 2 rows in, 2 rows out; backward 4 in, 2 out.
#include <type_traits>

#include "block.h"

namespace moe {

namespace {

typedef __attribute__((ext_vector_type(8))) float f32x8_t;
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

// ------------------------------------------------ eight columns of a row
// AL: the eight columns are all there and 16-byte aligned.  Otherwise `n` of
// them are there, at the alignment of the element type.
template <typename T, bool AL>
__device__ __forceinline__ f32x8_t load8(const T* p, int n) {
  f32x8_t v;
  if constexpr (sizeof(T) == 2) {
    if (AL || n >= 8) {
      const u32x4_t u = AL ? *(const u32x4_t*)p : (u32x4_t)*(const u32x4_any_t*)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(u[i] << 16);
        v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_to_f32(p[i]) : 0.0f;
    }
  } else {
    if (AL || n >= 8) {
      f32x4_t a, b;
      if (AL) {
        a = *(const f32x4_t*)p;
        b = *(const f32x4_t*)(p + 4);
      } else {
        a = *(const f32x4_any_t*)p;
        b = *(const f32x4_any_t*)(p + 4);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
  }
  return v;
}

template <typename T, bool AL>
__device__ __forceinline__ void store8(T* p, f32x8_t v, int n) {
  if constexpr (sizeof(T) == 2) {
    typedef __attribute__((ext_vector_type(8))) __bf16 b8;
    const b8 b = __builtin_convertvector(v, b8);   // nearest even
    const u32x4_t u = __builtin_bit_cast(u32x4_t, b);
    if (AL) {
      *(u32x4_t*)p = u;
    } else if (n >= 8) {
      *(u32x4_any_t*)p = u;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (bf16_t)(u[i >> 1] >> (16 * (i & 1)));
    }
  } else {
    const f32x4_t a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
    if (AL) {
      *(f32x4_t*)p = a;
      *(f32x4_t*)(p + 4) = b;
    } else if (n >= 8) {
      *(f32x4_any_t*)p = a;
      *(f32x4_any_t*)(p + 4) = b;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
    }
  }
}

// a gain vector's eight values, whichever type it is stored in
template <bool AL>
__device__ __forceinline__ f32x8_t load_gain(const void* g, int bf16, int col,
                                             int n, float offset) {
  f32x8_t v = bf16 ? load8<bf16_t, AL>((const bf16_t*)g + col, n)
                   : load8<float, AL>((const float*)g + col, n);
  v += offset;
  return v;
}

__device__ __forceinline__ float dot8(f32x8_t a, f32x8_t b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a[i], b[i], s);
  return s;
}

// sums of N values over the workgroup, the same in every thread; `buf` holds
// 16 x N floats and is not used again before another barrier
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float* buf) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int waves = blockDim.x >> 6;
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], m, 64);
  }
  if (waves == 1) return;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[wv * N + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.0f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += buf[w * N + i];
  }
}

struct NormRun {
  moe_norm n;
  NormArgs a;
  CombineSource c;
};

// ------------------------------------------------------------- forward
template <typename YT, typename RT, typename XT, bool AL, int VPT, bool COMB>
__global__ __launch_bounds__(1024) void k_residual_norm(NormRun q) {
  __shared__ float red[2][2][16];      // [row parity][mean square][wavefront]
  __shared__ int32_t s_row[2][MOE_KMAX];
  __shared__ float s_w[2][MOE_KMAX];
  __shared__ int s_n[2];
  const moe_norm& n = q.n;
  const int H = n.H, NT = blockDim.x;
  const float inv_h = 1.0f / (float)H;
  int par = 0;
  for (long t = blockIdx.x; t < n.T; t += gridDim.x, par ^= 1) {
    const RT* rr = (const RT*)q.a.resid + t * n.resid_stride;
    f32x8_t y[VPT], r[VPT];
    if constexpr (COMB) {
      if (threadIdx.x < 64) {          // the token's local slots, in order
        const int j = threadIdx.x;
        int row = j < q.c.k ? q.c.pair_row[t * q.c.k + j] : -1;
        const float w = j < q.c.k ? q.c.w[t * q.c.k + j] : 0.0f;
        if (row >= q.c.cap) row = -1;
        const uint64_t m = __ballot(row >= 0);
        if (row >= 0) {
          const int pos = __popcll(m & ((1ull << j) - 1ull));
          s_row[par][pos] = row;
          s_w[par][pos] = w;
        }
        if (j == 0) s_n[par] = __popcll(m);
      }
    }
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (threadIdx.x + v * NT), left = H - col;
      y[v] = 0.0f;
      r[v] = 0.0f;
      if (left <= 0) continue;
      if constexpr (COMB) {
        if (q.c.y_shared)
          y[v] = load8<float, AL>(q.c.y_shared + t * H + col, left);
      } else if (q.a.y) {
        y[v] = load8<YT, AL>((const YT*)q.a.y + t * n.block_stride + col, left);
      }
      r[v] = load8<RT, AL>(rr + col, left);
    }
    if constexpr (COMB) {
      // slots in order, then the shared expert, as moe_combine adds them
      f32x8_t acc[VPT];
#pragma unroll
      for (int v = 0; v < VPT; ++v) acc[v] = 0.0f;
      __syncthreads();
      const int ns = s_n[par];
      for (int j = 0; j < ns; ++j) {
        const float* yr = q.c.y_perm + (size_t)s_row[par][j] * H;
        const float w = s_w[par][j];
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int col = 8 * (threadIdx.x + v * NT), left = H - col;
          if (left <= 0) continue;
          const f32x8_t e = load8<float, AL>(yr + col, left);
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[v][i] = __builtin_fmaf(w, e[i], acc[v][i]);
        }
      }
#pragma unroll
      for (int v = 0; v < VPT; ++v) y[v] = q.c.y_shared ? acc[v] + y[v] : acc[v];
      if (q.c.block_out) {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int col = 8 * (threadIdx.x + v * NT), left = H - col;
          if (left > 0)
            store8<YT, AL>((YT*)q.c.block_out + t * n.block_stride + col, y[v], left);
        }
      }
    }
    if (q.a.post_gain) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < VPT; ++v) s[0] += dot8(y[v], y[v]);
      block_sum(s, red[par][0]);
      const float rs = 1.0f / sqrtf(s[0] * inv_h + n.eps);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int col = 8 * (threadIdx.x + v * NT), left = H - col;
        if (left <= 0) continue;
        y[v] = y[v] * rs * load_gain<AL>(q.a.post_gain, n.gain_dtype == MOE_BF16, col, left, n.gain_offset);
      }
    }
    if (q.a.gate) {
      const float* g = q.a.gate + (n.gate_rows > 1 ? t * n.gate_cols : 0);
      if (n.gate_cols == 1) {
        const float f = g[0];
#pragma unroll
        for (int v = 0; v < VPT; ++v) y[v] *= f;
      } else {
#pragma unroll
        for (int v = 0; v < VPT; ++v) {
          const int col = 8 * (threadIdx.x + v * NT), left = H - col;
          if (left > 0) y[v] *= load8<float, false>(g + col, left);
        }
      }
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (threadIdx.x + v * NT), left = H - col;
      if (left <= 0) continue;
      r[v] += n.residual_scale * y[v];
      s[0] += dot8(r[v], r[v]);
      if (q.a.resid_out)
        store8<RT, AL>((RT*)q.a.resid_out + t * n.resid_out_stride + col, r[v], left);
    }
    if (q.a.x_out) {
      block_sum(s, red[par][1]);
      const float rs = 1.0f / sqrtf(s[0] * inv_h + n.eps);
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int col = 8 * (threadIdx.x + v * NT), left = H - col;
        if (left <= 0) continue;
        store8<XT, AL>((XT*)q.a.x_out + t * n.out_stride + col,
                       r[v] * rs * load_gain<AL>(q.a.pre_gain, n.gain_dtype == MOE_BF16, col, left, n.gain_offset),
                       left);
      }
    }
  }
}

// ------------------------------------------------------------ backward
struct NormGradRun {
  moe_norm n;
  NormGradArgs a;
  float* part;      // [arrays][gridDim.x][H], then [gridDim.x] for a scalar
  int col_gate;     // the gate's gradient is a column sum
  int one_gate;     // ... is one number
};

template <typename YT, typename RT, typename XT, bool AL, int VPT>
__global__ __launch_bounds__(1024) void k_residual_norm_backward(NormGradRun q) {
  __shared__ float red[2][2][32];
  const moe_norm& n = q.n;
  const NormGradArgs& a = q.a;
  const int H = n.H, NT = blockDim.x;
  const float inv_h = 1.0f / (float)H;
  const bool gain_bf16 = n.gain_dtype == MOE_BF16;
  f32x8_t d_pre[VPT], d_post[VPT], d_gc[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) d_pre[v] = d_post[v] = d_gc[v] = 0.0f;
  float d_one = 0.0f;
  int par = 0;
  for (long t = blockIdx.x; t < n.T; t += gridDim.x, par ^= 1) {
    f32x8_t g[VPT], r[VPT], x[VPT], y[VPT];
    float s[2] = {0.0f, 0.0f}, sy = 0.0f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (threadIdx.x + v * NT), left = H - col;
      g[v] = r[v] = x[v] = y[v] = 0.0f;
      if (left <= 0) continue;
      if (a.d_resid_out)
        g[v] = load8<RT, AL>((const RT*)a.d_resid_out + t * n.resid_out_stride + col, left);
      if (a.d_x) {
        r[v] = load8<RT, AL>((const RT*)a.resid_out + t * n.resid_out_stride + col, left);
        x[v] = load8<XT, AL>((const XT*)a.d_x + t * n.out_stride + col, left);
      }
      if (a.y) y[v] = load8<YT, AL>((const YT*)a.y + t * n.block_stride + col, left);
    }
    float rs = 0.0f, ys = 1.0f;
    f32x8_t gp[VPT];
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (threadIdx.x + v * NT), left = H - col;
      gp[v] = 0.0f;
      if (left <= 0) continue;
      if (a.d_x) {
        gp[v] = x[v] * load_gain<AL>(a.pre_gain, gain_bf16, col, left, n.gain_offset);
        s[0] += dot8(r[v], r[v]);
        s[1] += dot8(r[v], gp[v]);
      }
      sy += dot8(y[v], y[v]);
    }
    float s3[3] = {s[0], s[1], sy};
    __shared__ float red3[2][48];
    block_sum(s3, red3[par]);
    if (a.d_x) {
      rs = 1.0f / sqrtf(s3[0] * inv_h + n.eps);
      const float c = s3[1] * inv_h * rs * rs;     // mean(gp r') rs^2
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        g[v] += rs * (gp[v] - c * r[v]);
        d_pre[v] += x[v] * r[v] * rs;
      }
    }
    if (a.post_gain) ys = 1.0f / sqrtf(s3[2] * inv_h + n.eps);
    if (a.d_resid) {
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int col = 8 * (threadIdx.x + v * NT), left = H - col;
        if (left > 0) store8<RT, AL>((RT*)a.d_resid + t * n.resid_stride + col, g[v], left);
      }
    }
    if (!a.d_y && !a.d_post && !a.d_gate) continue;
    // g: the gradient of residual_scale * gate * v from here on
    float sums[2] = {0.0f, 0.0f};    // gate's row sum, mean of the post-norm
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int col = 8 * (threadIdx.x + v * NT), left = H - col;
      if (left <= 0) continue;
      f32x8_t pg;
      pg = 1.0f;
      if (a.post_gain) pg = load_gain<AL>(a.post_gain, gain_bf16, col, left, n.gain_offset);
      g[v] *= n.residual_scale;
      if (a.gate) {
        const float* gt = a.gate + (n.gate_rows > 1 ? t * n.gate_cols : 0);
        const f32x8_t e = g[v] * (y[v] * ys * pg);
        if (n.gate_cols == 1) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sums[0] += e[i];
          g[v] *= gt[0];
        } else {
          if (q.col_gate) d_gc[v] += e;
          else if (a.d_gate) store8<float, false>(a.d_gate + t * H + col, e, left);
          g[v] *= load8<float, false>(gt + col, left);
        }
      }
      if (a.post_gain) {
        d_post[v] += g[v] * y[v] * ys;
        g[v] *= pg;
        sums[1] += dot8(g[v], y[v]);
      }
    }
    if (a.post_gain || (a.d_gate && n.gate_cols == 1)) block_sum(sums, red[par][0]);
    if (a.d_gate && n.gate_cols == 1) {
      if (q.one_gate) d_one += sums[0];
      else if (threadIdx.x == 0) a.d_gate[t] = sums[0];
    }
    if (a.d_y) {
      const float c = sums[1] * inv_h * ys * ys;
#pragma unroll
      for (int v = 0; v < VPT; ++v) {
        const int col = 8 * (threadIdx.x + v * NT), left = H - col;
        if (left <= 0) continue;
        if (a.post_gain) g[v] = ys * (g[v] - c * y[v]);
        store8<YT, AL>((YT*)a.d_y + t * n.block_stride + col, g[v], left);
      }
    }
  }
  float* part = q.part + (size_t)blockIdx.x * H;
  const size_t step = (size_t)gridDim.x * H;
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    const int col = 8 * (threadIdx.x + v * NT), left = H - col;
    if (left <= 0) continue;
    float* p = part + col;
    if (a.d_pre) { store8<float, false>(p, d_pre[v], left); p += step; }
    if (a.d_post) { store8<float, false>(p, d_post[v], left); p += step; }
    if (q.col_gate) store8<float, false>(p, d_gc[v], left);
  }
  if (q.one_gate && threadIdx.x == 0) {
    const int arrays = (a.d_pre ? 1 : 0) + (a.d_post ? 1 : 0);
    q.part[arrays * step + blockIdx.x] = d_one;
  }
}

// out[c] = sum over the workgroups' partial sums, in a fixed order
struct ColumnSums {
  const float* part[3];
  float* out[3];
};

__global__ __launch_bounds__(256) void k_column_sums(ColumnSums q, int parts,
                                                     int H) {
  __shared__ float s[4][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + c;
  const float* part = q.part[blockIdx.y];
  double v = 0.0;
  if (col < H)
    for (int p = w; p < parts; p += 4) v += (double)part[(size_t)p * H + col];
  s[w][c] = (float)v;
  __syncthreads();
  if (w == 0 && col < H)
    q.out[blockIdx.y][col] = (s[0][c] + s[1][c]) + (s[2][c] + s[3][c]);
}

__global__ __launch_bounds__(64) void k_one_sum(const float* part, int parts,
                                                float* out) {
  double v = 0.0;
  for (int p = threadIdx.x; p < parts; p += 64) v += (double)part[p];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  if (threadIdx.x == 0) *out = (float)v;
}

__global__ __launch_bounds__(256) void k_clear(float* p, long n) {
  for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += 256l * gridDim.x) p[i] = 0.0f;
}

bool al16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// rows of `stride` elements can move as whole 16-byte pieces
bool rows_aligned(const void* p, int dtype, int64_t stride) {
  return !p || (al16(p) && stride % (dtype == MOE_BF16 ? 8 : 4) == 0);
}

// threads and passes for a row of H columns
int row_threads(int H, int* vpt) {
  const int v = (H + 7) / 8;
  *vpt = v <= 1024 ? 1 : 2;
  const int nt = (v + *vpt - 1) / *vpt;
  return (nt + 63) / 64 * 64;
}

template <class F>
void by_type(int dtype, F f) {
  if (dtype == MOE_BF16) f(bf16_t{});
  else f(float{});
}

template <class F>
void by_flag(bool b, F f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

int norm_grad_grid(int T) { return T < 512 ? T : 512; }

}  // namespace

hipError_t launch_residual_norm(const moe_norm* n, const NormArgs& a,
                                const CombineSource* comb, hipStream_t s) {
  NormRun q{};
  q.n = *n;
  q.a = a;
  if (comb) q.c = *comb;
  bool al = n->H % 8 == 0 && rows_aligned(a.y, n->block_dtype, n->block_stride) &&
            rows_aligned(a.resid, n->resid_dtype, n->resid_stride) &&
            rows_aligned(a.resid_out, n->resid_dtype, n->resid_out_stride) &&
            rows_aligned(a.x_out, n->out_dtype, n->out_stride) &&
            al16(a.post_gain) && al16(a.pre_gain);
  if (comb)
    al = al && al16(comb->y_perm) && al16(comb->y_shared) &&
         rows_aligned(comb->block_out, n->block_dtype, n->block_stride);
  int vpt;
  const dim3 block(row_threads(n->H, &vpt));
  const dim3 grid(n->T < (1 << 20) ? n->T : (1 << 20));
  by_type(n->block_dtype, [&](auto yt) {
    by_type(n->resid_dtype, [&](auto rt) {
      by_type(n->out_dtype, [&](auto xt) {
        by_flag(al, [&](auto alt) {
          by_flag(comb != nullptr, [&](auto cb) {
            using Y = decltype(yt);
            using R = decltype(rt);
            using X = decltype(xt);
            if (vpt == 1)
              k_residual_norm<Y, R, X, alt.value, 1, cb.value><<<grid, block, 0, s>>>(q);
            else
              k_residual_norm<Y, R, X, alt.value, 2, cb.value><<<grid, block, 0, s>>>(q);
          });
        });
      });
    });
  });
  return hipGetLastError();
}

size_t norm_grad_partials(const moe_norm* n) {
  return (size_t)norm_grad_grid(n->T) * (3 * (size_t)n->H + 1);
}

hipError_t launch_residual_norm_backward(const moe_norm* n,
                                         const NormGradArgs& a,
                                         float* partials, hipStream_t s) {
  const bool gate_row = a.gate && n->gate_rows == 1;
  NormGradRun q{};
  q.n = *n;
  q.a = a;
  q.part = partials;
  q.one_gate = a.d_gate && gate_row && n->gate_cols == 1;
  q.col_gate = a.d_gate && gate_row && n->gate_cols > 1;
  const size_t H = n->H;
  if (n->T == 0) {
    if (!a.d_pre && !a.d_post && !q.one_gate && !q.col_gate) return hipSuccess;
    if (a.d_pre) k_clear<<<64, 256, 0, s>>>(a.d_pre, H);
    if (a.d_post) k_clear<<<64, 256, 0, s>>>(a.d_post, H);
    if (q.one_gate || q.col_gate) k_clear<<<64, 256, 0, s>>>(a.d_gate, n->gate_cols);
    return hipGetLastError();
  }
  const bool al = n->H % 8 == 0 && rows_aligned(a.y, n->block_dtype, n->block_stride) &&
                  rows_aligned(a.d_y, n->block_dtype, n->block_stride) &&
                  rows_aligned(a.resid_out, n->resid_dtype, n->resid_out_stride) &&
                  rows_aligned(a.d_resid_out, n->resid_dtype, n->resid_out_stride) &&
                  rows_aligned(a.d_resid, n->resid_dtype, n->resid_stride) &&
                  rows_aligned(a.d_x, n->out_dtype, n->out_stride) &&
                  al16(a.post_gain) && al16(a.pre_gain);
  int vpt;
  const dim3 block(row_threads(n->H, &vpt)), grid(norm_grad_grid(n->T));
  by_type(n->block_dtype, [&](auto yt) {
    by_type(n->resid_dtype, [&](auto rt) {
      by_type(n->out_dtype, [&](auto xt) {
        by_flag(al, [&](auto alt) {
          using Y = decltype(yt);
          using R = decltype(rt);
          using X = decltype(xt);
          if (vpt == 1)
            k_residual_norm_backward<Y, R, X, alt.value, 1><<<grid, block, 0, s>>>(q);
          else
            k_residual_norm_backward<Y, R, X, alt.value, 2><<<grid, block, 0, s>>>(q);
        });
      });
    });
  });
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ColumnSums c{};
  int arrays = 0;
  const size_t step = (size_t)grid.x * H;
  for (float* out : {a.d_pre, a.d_post, q.col_gate ? a.d_gate : nullptr})
    if (out) {
      c.part[arrays] = partials + arrays * step;
      c.out[arrays++] = out;
    }
  if (arrays)
    k_column_sums<<<dim3((n->H + 63) / 64, arrays), 256, 0, s>>>(c, grid.x, n->H);
  if (q.one_gate) k_one_sum<<<1, 64, 0, s>>>(partials + arrays * step, grid.x, a.d_gate);
  return hipGetLastError();
}

}  // namespace moe
