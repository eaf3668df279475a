// 8-bit checkpoints of activation rows (checkpoint.h has the format): rows to
// codes and scales, and back; and the experts' activation around them, with
// its backward.
//
// All of it is bound by memory.  A lane takes one access of 16 bytes of its
// widest array, so 16 lanes (bf16) or 32 (float32) hold a group of 128
// columns, whose largest magnitude is four DPP steps and at most one exchange
// between rows.  8192 x 7168 bf16: 32 us to codes, 30 us back (5.6 and 5.9
// TB/s; a copy of 256 MiB 5.3); 1021 x 2501 float32, rows at any alignment: 4.6.
#include <algorithm>

#include "checkpoint.h"
#include "rows.h"
#include "train.h"

namespace moe {

namespace {

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  v = row16_max(v);
  if (LANES == 32) v = fmaxf(v, __shfl_xor(v, 16, 64));
  return v;
}

// a piece's columns as float32
template <typename T, int W>
__device__ __forceinline__ void piece_values(Raw<T, W> r, float* v) {
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (sizeof(T) == 2)
      v[i] = __uint_as_float(i & 1 ? r[i >> 1] & 0xFFFF0000u : r[i >> 1] << 16);
    else
      v[i] = __uint_as_float(r[i]);
  }
}

// W codes at any alignment
template <int W>
struct CodesOf;
template <>
struct CodesOf<4> {
  typedef uint32_t V;
  typedef uint32_t Any __attribute__((aligned(1)));
};
template <>
struct CodesOf<8> {
  typedef u32x2v_t V;
  typedef u32x2v_t Any __attribute__((aligned(1)));
};
__device__ __forceinline__ uint32_t code_word(uint32_t v, int) { return v; }
__device__ __forceinline__ uint32_t code_word(u32x2v_t v, int i) { return v[i]; }

constexpr int kRowThreads = 256;

// A workgroup takes U runs of kRowThreads pieces of W columns; the pieces of
// a row are padded to whole groups.  FIT: kAligned (C a multiple of W, rows
// and codes aligned to their pieces) or kAny.  `first`: the launch's first group.
template <typename T, Fit FIT, int U>
__global__ __launch_bounds__(kRowThreads) void k_checkpoint_rows(
    const T* __restrict__ src, long stride, uint32_t first, uint32_t groups,
    uint32_t per_row, int C, uint8_t* __restrict__ codes,
    float* __restrict__ scales) {
  constexpr int W = 16 / (int)sizeof(T), LANES = 128 / W;
  constexpr uint32_t kPer = kRowThreads / LANES;       // groups a run
  const int lane = threadIdx.x & (LANES - 1);
  uint32_t g[U];
  long t[U];
  Piece c[U];
  Raw<T, W> r[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    g[u] = first + (blockIdx.x * U + u) * kPer + threadIdx.x / LANES;
    const uint32_t gg = min(g[u], groups - 1);
    t[u] = gg / per_row;
    const int n = (int)(gg - (uint32_t)t[u] * per_row);
    c[u] = piece_at<W, FIT>(n * 128 + lane * W, C);
    r[u] = load_piece<T, W, FIT, true>(src + t[u] * stride, c[u], C);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[W];
    piece_values<T, W>(own_cols<T, W, FIT>(r[u], c[u]), v);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) top = fmaxf(top, finite_size(v[i]));
    const int e = checkpoint_exponent(group_max<LANES>(top));
    const float inv = power_of_two(-e), limit = checkpoint_limit(e);
    typename CodesOf<W>::V q;
    if constexpr (W == 4) {
      q = checkpoint_codes(v[0], v[1], v[2], v[3], inv, limit);
    } else {
      q[0] = checkpoint_codes(v[0], v[1], v[2], v[3], inv, limit);
      q[1] = checkpoint_codes(v[4], v[5], v[6], v[7], inv, limit);
    }
    if (g[u] >= groups) continue;
    if (lane == 0) scales[g[u]] = power_of_two(e);
    uint8_t* to = codes + t[u] * C + c[u].col;
    if (c[u].col + W <= C) {
      if constexpr (FIT == kAligned)
        __builtin_nontemporal_store(q, (typename CodesOf<W>::V*)to);
      else
        *(typename CodesOf<W>::Any*)to = q;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (c[u].col + i < C) to[i] = (uint8_t)(code_word(q, i >> 2) >> (8 * (i & 3)));
    }
  }
}

template <typename T, Fit FIT, int U>
__global__ __launch_bounds__(kRowThreads) void k_restore_rows(
    const uint8_t* __restrict__ codes, const float* __restrict__ scales,
    uint32_t first, uint32_t groups, uint32_t per_row, int C,
    T* __restrict__ dst, long stride) {
  constexpr int W = 16 / (int)sizeof(T), LANES = 128 / W;
  constexpr uint32_t kPer = kRowThreads / LANES;
  typedef typename CodesOf<W>::V Codes;
  const int lane = threadIdx.x & (LANES - 1);
  long t[U];
  int col[U];
  Codes q[U];
  float s[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t g = first + (blockIdx.x * U + u) * kPer + threadIdx.x / LANES;
    const uint32_t gg = min(g, groups - 1);
    t[u] = gg / per_row;
    const int n = (int)(gg - (uint32_t)t[u] * per_row);
    col[u] = g < groups ? n * 128 + lane * W : C;      // past the row: nothing
    s[u] = scales[gg];
    const uint8_t* from = codes + t[u] * C + col[u];
    if (col[u] + W <= C) {
      if constexpr (FIT == kAligned) q[u] = __builtin_nontemporal_load((const Codes*)from);
      else q[u] = *(const typename CodesOf<W>::Any*)from;
    } else {
      uint32_t w[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col[u] + i < C) w[i >> 2] |= (uint32_t)from[i] << (8 * (i & 3));
      if constexpr (W == 4) q[u] = w[0];
      else q[u] = Codes{w[0], w[1]};
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float v[W];
#pragma unroll
    for (int i = 0; i < W / 4; ++i) code_values(code_word(q[u], i), v + 4 * i);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= s[u];
    Raw<T, W> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
      else r[i] = __float_as_uint(v[i]);
    }
    T* to = dst + t[u] * stride + col[u];
    if (col[u] + W <= C) {
      if constexpr (FIT == kAligned)
        __builtin_nontemporal_store(r, (Raw<T, W>*)to);
      else
        *(typename RawOf<16>::Any*)to = r;
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (col[u] + i < C) {
          if constexpr (sizeof(T) == 2) to[i] = (T)(r[i >> 1] >> (16 * (i & 1)));
          else to[i] = __uint_as_float(r[i]);
        }
      }
    }
  }
}

// Batches of fewer runs than this take one run a workgroup, so that they
// spread over the CUs; larger ones four, whose loads are in flight together.
// One run and four, to codes and back, us: bf16, 2048 runs (1024 x 4096) 5.0 and
// 4.9 against 5.3 and 5.0; 4096 runs 7.2 and 6.0 against 7.1 and 5.6; 5116 runs
// (4093 x 2501, no alignment) 8.7 and 7.2 against 9.6 and 7.2; 8192 runs 11.9 and
// 9.9 against 11.5 and 10.3; 28672 runs (8192 x 7168) 36.8 and 30.1 against 32.2
// and 29.9.  float32, 2552 runs (1021 x 2501) 4.4 and 4.4 against 5.1 and 4.5;
// 57344 runs (8192 x 7168) 58 and 53 against 50 and 50.
constexpr uint32_t kManyRuns = 8192;

// A launch has less than 2^32 threads (a larger grid runs only in part), so
// more groups than this take several.
constexpr uint32_t kLaunchBlocks = 1u << 23;

// `run`(first group, workgroups) over all groups, `per` of them a workgroup
template <class F>
hipError_t launch_groups(uint32_t groups, uint32_t per, F run) {
  const uint32_t blocks = (groups + per - 1) / per;
  for (uint32_t b = 0; b < blocks; b += kLaunchBlocks) {
    run(b * per, std::min(blocks - b, kLaunchBlocks));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename T>
hipError_t checkpoint_rows(const T* src, long Tn, int C, long stride,
                           uint8_t* codes, float* scales, hipStream_t s) {
  constexpr int W = 16 / (int)sizeof(T);
  const uint32_t per_row = (uint32_t)((C + 127) / 128);
  const uint32_t groups = (uint32_t)Tn * per_row;
  const uint32_t per = kRowThreads * W / 128, runs = (groups + per - 1) / per;
  const bool fits = C % W == 0 && stride % W == 0 &&
                    ((uintptr_t)src & 15) == 0 && ((uintptr_t)codes & (W - 1)) == 0;
#define RUN(FIT, U)                                                           \
  return launch_groups(groups, per * U, [&](uint32_t first, uint32_t blocks) { \
    k_checkpoint_rows<T, FIT, U><<<blocks, kRowThreads, 0, s>>>(              \
        src, stride, first, groups, per_row, C, codes, scales);               \
  })
  if (runs >= kManyRuns) {
    if (fits) RUN(kAligned, 4);
    RUN(kAny, 4);
  }
  if (fits) RUN(kAligned, 1);
  RUN(kAny, 1);
#undef RUN
}

template <typename T>
hipError_t restore_rows(const uint8_t* codes, const float* scales, long Tn,
                        int C, long stride, T* dst, hipStream_t s) {
  constexpr int W = 16 / (int)sizeof(T);
  const uint32_t per_row = (uint32_t)((C + 127) / 128);
  const uint32_t groups = (uint32_t)Tn * per_row;
  const uint32_t per = kRowThreads * W / 128, runs = (groups + per - 1) / per;
  const bool fits = C % W == 0 && stride % W == 0 &&
                    ((uintptr_t)dst & 15) == 0 && ((uintptr_t)codes & (W - 1)) == 0;
#define RUN(FIT, U)                                                           \
  return launch_groups(groups, per * U, [&](uint32_t first, uint32_t blocks) { \
    k_restore_rows<T, FIT, U><<<blocks, kRowThreads, 0, s>>>(                 \
        codes, scales, first, groups, per_row, C, dst, stride);               \
  })
  if (runs >= kManyRuns) {
    if (fits) RUN(kAligned, 4);
    RUN(kAny, 4);
  }
  if (fits) RUN(kAligned, 1);
  RUN(kAny, 1);
#undef RUN
}

// ------------------------------------------- the experts' activation
// Row of an index over the routed rows and, behind them, the shared expert's;
// -1 past both.
__device__ __forceinline__ int intermediate_row(const ExpertRows& r, int i) {
  const int n = *r.n_routed;
  if (i < n) return i;
  i -= n;
  return r.has_shared && i < r.T ? r.cap + i : -1;
}

// A group's 128 columns on 16 lanes: this lane's codes, and the scale.
__device__ __forceinline__ u32x2v_t checkpoint_eight(const float* v, float* scale) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_size(v[j]));
  const int e = checkpoint_exponent(row16_max(top));
  const float inv = power_of_two(-e), limit = checkpoint_limit(e);
  *scale = power_of_two(e);
  return u32x2v_t{checkpoint_codes(v[0], v[1], v[2], v[3], inv, limit),
                  checkpoint_codes(v[4], v[5], v[6], v[7], inv, limit)};
}

// A wavefront's 64 lanes are 16 lanes for each of four groups of 128
// channels, eight a lane.  Behind the rows' groups come those of the layer's
// input (one launch of 52 us at 4096 tokens of 7168 x 2048, 32 of 256 experts
// and the shared one, 5.5 TB/s; two launches 62, and 7.5 against 4.1 at 509
// tokens of 1024 x 512).  h is rounded to bf16, the type that the matrix cores
// take for the down product at their full rate, as in the layer's BF16 recipe:
// an output's error grows by it from 1.7e-3 of the output (its own rounding to
// bf16) to 2.3e-3 in root mean square.  The codes come from the unrounded
// products.
__global__ __launch_bounds__(256) void k_swiglu_save(
    ExpertRows r, const float* __restrict__ gu, bf16_t* __restrict__ h,
    uint8_t* __restrict__ codes, float* __restrict__ scales,
    const bf16_t* __restrict__ x, int H, uint8_t* __restrict__ x_codes,
    float* __restrict__ x_scales) {
  const int I = r.I, blocks = I / 128;
  const long count = (long)(*r.n_routed + (r.has_shared ? r.T : 0)) * blocks;
  const long all = count + (long)r.T * (H / 128);
  const int lane = threadIdx.x & 15;
  for (long q = (long)blockIdx.x * 16 + (threadIdx.x >> 4); q < all;
       q += (long)gridDim.x * 16) {
    if (q >= count) {
      const long g = q - count, at = g * 128 + lane * 8;
      float v[8];
      piece_values<bf16_t, 8>(*(const u32x4_t*)(x + at), v);
      float s;
      *(u32x2v_t*)(x_codes + at) = checkpoint_eight(v, &s);
      if (lane == 0) x_scales[g] = s;
      continue;
    }
    const int i = (int)(q / blocks), n = (int)(q - (long)i * blocks);
    const long row = intermediate_row(r, i);
    const long at = row * 2 * I + n * 128 + lane * 8;
    float v[2][8];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const f32x4_t a = *(const f32x4_t*)(gu + at + p * I);
      const f32x4_t b = *(const f32x4_t*)(gu + at + p * I + 4);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[p][j] = a[j];
        v[p][j + 4] = b[j];
      }
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float s;
      *(u32x2v_t*)(codes + at + p * I) = checkpoint_eight(v[p], &s);
      if (lane == 0) scales[row * 2 * blocks + p * blocks + n] = s;
    }
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = silu_f32(v[0][2 * j]) * v[1][2 * j];
      const float b = silu_f32(v[0][2 * j + 1]) * v[1][2 * j + 1];
      o[j] = pack_bf16(a, b);
    }
    *(u32x4_t*)(h + row * I + n * 128 + lane * 8) = o;
  }
}

// One workgroup a row, of as many wavefronts as the row fills, at most four
// (8192 x 2048: 35 us, 5.7 TB/s; 16384 x 768: 34 us, of four wavefronts 53).
// With q = sigmoid(g):
//   h = g q u,  dg = dh u q (1 + g (1 - q)),  du = dh g q
// times the row's route weight w; the weight's own gradient sums dh h over
// the row, per thread in column order, then over the threads.  dg, du and w h
// are rounded to bf16 once, for the products that follow: float32 operands would
// run at a sixteenth of the matrix cores' bf16 rate (141 TFLOP/s against 1195 of
// a library product), and a rounding of about 2^-9 in the mean is small beside the
// about 2^-5 of the codes they are made from.
__global__ __launch_bounds__(256) void k_swiglu_backward(
    ExpertRows r, PairRows pr, const float* __restrict__ dh,
    const uint8_t* __restrict__ codes, const float* __restrict__ scales,
    bf16_t* __restrict__ dgu, bf16_t* __restrict__ hw,
    float* __restrict__ d_topk_w) {
  if (d_topk_w) {                                // pairs without a row
    const int pairs = r.T * pr.k;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < pairs; i += gridDim.x * blockDim.x)
      if (pr.pair_row[i] < 0) d_topk_w[i] = 0.0f;
  }
  __shared__ float part[2][4];
  if (threadIdx.x < 8) ((float*)part)[threadIdx.x] = 0.0f;
  __syncthreads();
  const int I = r.I, blocks = I / 128;
  const int n = *r.n_routed + (r.has_shared ? r.T : 0);
  int turn = 0;
  for (int i = blockIdx.x; i < n; i += gridDim.x, turn ^= 1) {
    const long row = intermediate_row(r, i);
    const bool routed = row < r.cap && i < *r.n_routed;
    const float w = routed ? pr.row_weight[row] : 1.0f;
    float sum = 0.0f;
    for (int c = threadIdx.x * 8; c < I; c += blockDim.x * 8) {
      const long at = row * 2 * I + c;
      const u32x2v_t gc = *(const u32x2v_t*)(codes + at);
      const u32x2v_t uc = *(const u32x2v_t*)(codes + at + I);
      const float gs = scales[row * 2 * blocks + (c >> 7)];
      const float us = scales[row * 2 * blocks + blocks + (c >> 7)];
      const f32x4_t d0 = *(const f32x4_t*)(dh + row * I + c);
      const f32x4_t d1 = *(const f32x4_t*)(dh + row * I + c + 4);
      float g[8], u[8], dg[8], du[8], hv[8];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        code_values(gc[p], g + 4 * p);
        code_values(uc[p], u + 4 * p);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float gg = g[j] * gs, uu = u[j] * us;
        const float d = j < 4 ? d0[j & 3] : d1[j & 3];
        const float q = 1.0f / (1.0f + __expf(-gg)), a = gg * q;
        const float h = a * uu;
        sum = __builtin_fmaf(d, h, sum);
        hv[j] = w * h;
        const float dw = w * d;
        dg[j] = dw * uu * (q * __builtin_fmaf(gg, 1.0f - q, 1.0f));
        du[j] = dw * a;
      }
      u32x4_t og, ou, oh;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        og[j] = pack_bf16(dg[2 * j], dg[2 * j + 1]);
        ou[j] = pack_bf16(du[2 * j], du[2 * j + 1]);
        oh[j] = pack_bf16(hv[2 * j], hv[2 * j + 1]);
      }
      *(u32x4_t*)(dgu + at) = og;
      *(u32x4_t*)(dgu + at + I) = ou;
      *(u32x4_t*)(hw + row * I + c) = oh;
    }
    if (!routed || !d_topk_w) continue;          // uniform for the workgroup
    // (the slot whose row this is)
    long pair = -1;
    if ((int)threadIdx.x < pr.k) {
      pair = (long)pr.row_token[row] * pr.k + threadIdx.x;
      if (pr.pair_row[pair] != row) pair = -1;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = sum;
    __syncthreads();                             // (two buffers: one barrier a row)
    if (pair >= 0)
      d_topk_w[pair] = (part[turn][0] + part[turn][1]) + (part[turn][2] + part[turn][3]);
  }
}

// Sixteen columns a thread: 16 bytes of codes, twice 16 bytes of d and of each
// output (4096 tokens of 7168, 4096 rows and the shared expert's: 52 us).
__global__ __launch_bounds__(256) void k_gather_pair(
    const uint8_t* __restrict__ codes, const float* __restrict__ scales,
    const bf16_t* __restrict__ d, const int32_t* __restrict__ row_token,
    const int32_t* __restrict__ n_rows, int T, int C,
    bf16_t* __restrict__ x_out, bf16_t* __restrict__ d_out,
    bf16_t* __restrict__ x_all) {
  const uint32_t per_row = (uint32_t)C / 16;
  const int n = *n_rows;
  const long count = ((long)n + (x_all ? T : 0)) * per_row;
  for (long q = (long)blockIdx.x * 256 + threadIdx.x; q < count;
       q += (long)gridDim.x * 256) {
    const uint32_t r = (uint32_t)(q / per_row), c = (uint32_t)(q - (long)r * per_row) * 16;
    const bool routed = r < (uint32_t)n;
    const long t = routed ? row_token[r] : (int)(r - n);
    const u32x4_t code = *(const u32x4_t*)(codes + t * C + c);
    const float s = scales[t * (C / 128) + (c >> 7)];
    u32x4_t d0, d1, o[2];
    if (routed) {
      d0 = *(const u32x4_t*)(d + t * C + c);
      d1 = *(const u32x4_t*)(d + t * C + c + 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[4];
      code_values(code[i], v);
      o[i >> 1][2 * (i & 1)] = pack_bf16(v[0] * s, v[1] * s);
      o[i >> 1][2 * (i & 1) + 1] = pack_bf16(v[2] * s, v[3] * s);
    }
    const size_t at = (size_t)r * C + c;
    bf16_t* x = routed ? x_out + at : x_all + t * C + c;
    *(u32x4_t*)x = o[0];
    *(u32x4_t*)(x + 8) = o[1];
    if (routed) {
      *(u32x4_t*)(d_out + at) = d0;
      *(u32x4_t*)(d_out + at + 8) = d1;
    }
  }
}

}  // namespace

hipError_t launch_checkpoint_rows(const void* src, int dtype, long T, int C,
                                  long stride, uint8_t* codes, float* scales,
                                  hipStream_t s) {
  if (dtype == MOE_BF16)
    return checkpoint_rows((const bf16_t*)src, T, C, stride, codes, scales, s);
  return checkpoint_rows((const float*)src, T, C, stride, codes, scales, s);
}

hipError_t launch_restore_rows(const uint8_t* codes, const float* scales,
                               long T, int C, int dtype, long stride,
                               void* dst, hipStream_t s) {
  if (dtype == MOE_BF16)
    return restore_rows(codes, scales, T, C, stride, (bf16_t*)dst, s);
  return restore_rows(codes, scales, T, C, stride, (float*)dst, s);
}

hipError_t launch_swiglu_save(const ExpertRows& r, const float* gu, bf16_t* h,
                              uint8_t* codes, float* scales, const bf16_t* x,
                              int H, uint8_t* x_codes, float* x_scales,
                              hipStream_t s) {
  const long most = ((long)r.cap + (r.has_shared ? r.T : 0)) * (r.I / 128) +
                    (long)r.T * (H / 128);
  const long grid = (most + 15) / 16;
  k_swiglu_save<<<(unsigned)(grid < 4096 ? grid : 4096), 256, 0, s>>>(
      r, gu, h, codes, scales, x, H, x_codes, x_scales);
  return hipGetLastError();
}

hipError_t launch_swiglu_backward(const ExpertRows& r, const PairRows& p,
                                  const float* dh, const uint8_t* codes,
                                  const float* scales, bf16_t* dgu, bf16_t* hw,
                                  float* d_topk_w, hipStream_t s) {
  const long most = (long)r.cap + (r.has_shared ? r.T : 0);
  const int threads = r.I >= 256 * 8 ? 256 : (r.I + 511) / 512 * 64;
  const long grid = 4096 * 256 / threads;
  k_swiglu_backward<<<(unsigned)(most < grid ? most : grid), threads, 0, s>>>(
      r, p, dh, codes, scales, dgu, hw, d_topk_w);
  return hipGetLastError();
}

hipError_t launch_gather_pair(const uint8_t* codes, const float* scales,
                              const bf16_t* d, const int32_t* row_token,
                              const int32_t* n_rows, int cap, int T, int C,
                              bf16_t* x_out, bf16_t* d_out, bf16_t* x_all,
                              hipStream_t s) {
  const long most = (((long)cap + (x_all ? T : 0)) * (C / 16) + 255) / 256;
  k_gather_pair<<<(unsigned)(most < 8192 ? most : 8192), 256, 0, s>>>(
      codes, scales, d, row_token, n_rows, T, C, x_out, d_out, x_all);
  return hipGetLastError();
}

}  // namespace moe
