// Scored routing (moe_route_scored) and its gradient.
//
// A token's experts lie on a segment of 16 lanes (E <= 64, four tokens a
// wavefront) or a whole wavefront, EPL neighbouring experts a lane, so the
// lowest lane among equal values holds the lowest id.  Scores, choices and
// group scores are doubles: the chosen ids must be those of the definition,
// and in float32 neighbouring choices of some hundred experts collide within
// an ulp too often.  On this card a double operation issues at the rate of an
// unpacked float one.
#include <float.h>
#include <type_traits>

#include "block.h"

namespace moe {

namespace {

// An expert's choice: live values, kMasked for masked experts, and kGone for
// experts that are taken, outside the groups that stay, or padding.
constexpr double kMasked = -DBL_MAX;
#define kGone (-__builtin_inf())

template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp(double old, double v) {
  const uint64_t o = __double_as_longlong(old), b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_update_dpp((int)(uint32_t)o, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp((int)(o >> 32), (int)(b >> 32), CTRL, ROWS, 0xF, false);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}

__device__ __forceinline__ double read_lane(double v, int lane) {
  const uint64_t b = __double_as_longlong(v);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(b >> 32), lane);
  return __longlong_as_double(((uint64_t)hi << 32) | lo);
}

// Max / sum over a segment, the same value in every lane of it.  Row
// rotations by 8, 4, 2, 1 leave a row's result in its 16 lanes; row
// broadcasts carry it on to lane 63.
template <int LANES>
__device__ __forceinline__ double seg_max(double v) {
  v = fmax(v, dpp<0x128, 0xF>(v, v));
  v = fmax(v, dpp<0x124, 0xF>(v, v));
  v = fmax(v, dpp<0x122, 0xF>(v, v));
  v = fmax(v, dpp<0x121, 0xF>(v, v));
  if (LANES == 64) {
    v = fmax(v, dpp<0x142, 0xA>(v, v));
    v = fmax(v, dpp<0x143, 0xC>(v, v));
    v = read_lane(v, 63);
  }
  return v;
}

template <int LANES>
__device__ __forceinline__ double seg_sum(double v) {
  v += dpp<0x128, 0xF>(0.0, v);
  v += dpp<0x124, 0xF>(0.0, v);
  v += dpp<0x122, 0xF>(0.0, v);
  v += dpp<0x121, 0xF>(0.0, v);
  if (LANES == 64) {
    v += dpp<0x142, 0xA>(0.0, v);
    v += dpp<0x143, 0xC>(0.0, v);
    v = read_lane(v, 63);
  }
  return v;
}

// first lane of the segment at `base` whose predicate holds (it does in one)
template <int LANES>
__device__ __forceinline__ int seg_first(bool p, int base) {
  const uint64_t m = __ballot(p);
  if (LANES == 64) return __ffsll((unsigned long long)m) - 1;
  return base + __ffs((int)((m >> base) & 0xFFFFu)) - 1;
}

template <typename LT>
__device__ __forceinline__ double to_f64(LT v);
template <>
__device__ __forceinline__ double to_f64<float>(float v) { return (double)v; }
template <>
__device__ __forceinline__ double to_f64<bf16_t>(bf16_t v) { return (double)bf16_to_f32(v); }

// a logit, with NaN read as -inf
template <typename LT>
__device__ __forceinline__ double logit_of(LT v) {
  const double l = to_f64<LT>(v);
  return l == l ? l : -__builtin_inf();
}

__device__ __forceinline__ double sigmoid_f64(double l) {
  const double e = exp(-fabs(l));
  return (l >= 0.0 ? 1.0 : e) / (1.0 + e);
}

// exp(l - m) with m the row's largest logit: 0 throughout a masked row, equal
// shares for logits of +inf
__device__ __forceinline__ double softmax_num(double l, double m) {
  if (l == -__builtin_inf()) return 0.0;
  return l == m ? 1.0 : exp(l - m);
}

struct RouteArgs {
  const void* logits;
  const float* bias;
  int T, E, k, sigmoid, groups, keep, group_top, renorm, per;
  uint32_t per_inv;       // e / per == (e * per_inv) >> 20 for e < 1024
  float scale;
  int64_t stride;
  int32_t* ids;
  float* w;
};

constexpr int kWaves = 4;   // wavefronts a workgroup

template <int LANES, int EPL, typename LT>
__global__ __launch_bounds__(64 * kWaves) void k_route_scored(RouteArgs a) {
  constexpr int SEGS = 64 / LANES;
  __shared__ double lds_c[kWaves][SEGS][LANES * EPL];
  __shared__ double lds_g[kWaves][SEGS][64];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & (LANES - 1), seg = lane / LANES, base = seg * LANES;
  const int E = a.E, k = a.k;
  const int per_block = kWaves * SEGS;
  for (long t0 = (long)blockIdx.x * per_block; t0 < a.T;
       t0 += (long)gridDim.x * per_block) {
    const long tt = t0 + wv * SEGS + seg;
    const bool valid = tt < a.T;
    const long t = valid ? tt : a.T - 1;
    const LT* row = (const LT*)a.logits + t * a.stride;
    double l[EPL], c[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = r * EPL + i;
      l[i] = e < E ? logit_of<LT>(row[e]) : -__builtin_inf();
    }
    double m = 0.0, sum = 0.0;
    if (!a.sigmoid) {
      m = l[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) m = fmax(m, l[i]);
      m = seg_max<LANES>(m);
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = softmax_num(l[i], m);
        sum += c[i];
      }
      sum = seg_sum<LANES>(sum);
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = r * EPL + i;
      double v = a.sigmoid ? sigmoid_f64(l[i]) : (sum > 0.0 ? c[i] / sum : 0.0);
      if (a.bias) v += (double)a.bias[e < E ? e : 0];
      // NaN compares false: a NaN bias masks too
      c[i] = (l[i] > -__builtin_inf() && v > -__builtin_inf()) ? v : kMasked;
      if (e >= E) c[i] = kGone;
    }
    if (a.groups > 1) {
      double* ch = lds_c[wv][seg];
      double* gs = lds_g[wv][seg];
#pragma unroll
      for (int i = 0; i < EPL; ++i) ch[r * EPL + i] = c[i];
      __syncthreads();
      for (int g = r; g < a.groups; g += LANES) {
        double b0 = kMasked, b1 = kMasked;     // the group's two best
        for (int i = 0; i < a.per; ++i) {
          const double v = ch[g * a.per + i];
          b1 = fmax(b1, fmin(b0, v));
          b0 = fmax(b0, v);
        }
        gs[g] = (a.group_top == 2 && b1 > kMasked) ? b0 + b1 : b0;
      }
      __syncthreads();
      uint64_t stays = 0;                      // groups that stay
      for (int g = r; g < a.groups; g += LANES) {
        const double v = gs[g];
        int better = 0;
        for (int h = 0; h < a.groups; ++h)
          better += (gs[h] > v || (gs[h] == v && h < g)) ? 1 : 0;
        if (better < a.keep) stays |= 1ull << g;
      }
#pragma unroll
      for (int s = 1; s < LANES; s <<= 1) {
        const uint32_t lo = __shfl_xor((uint32_t)stays, s, 64);
        const uint32_t hi = __shfl_xor((uint32_t)(stays >> 32), s, 64);
        stays |= ((uint64_t)hi << 32) | lo;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const uint32_t g = ((uint32_t)(r * EPL + i) * a.per_inv) >> 20;
        if (!((stays >> (g & 63)) & 1)) c[i] = kGone;
      }
      __syncthreads();                         // lds_c is written again
    }
    int my_id = 0;
    for (int j = 0; j < k; ++j) {
      double best = c[0];
      int bi = 0;
#pragma unroll
      for (int i = 1; i < EPL; ++i)
        if (c[i] > best) { best = c[i]; bi = i; }
      const double top = seg_max<LANES>(best);
      const int owner = seg_first<LANES>(best == top, base);
      const int e = __shfl(r * EPL + bi, owner, 64);
      if (r == j) my_id = e;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (r * EPL + i == e) c[i] = kGone;
    }
    // lane j < k: the score of slot j again, from its logit
    const bool slot = r < k;
    const double lj = slot ? logit_of<LT>(row[my_id]) : -__builtin_inf();
    double s = a.sigmoid ? sigmoid_f64(lj) : (sum > 0.0 ? softmax_num(lj, m) / sum : 0.0);
    if (a.renorm) {
      const double S = seg_sum<LANES>(slot ? s : 0.0);
      s = S > 0.0 ? s / S : 0.0;
    }
    if (valid && slot) {
      a.ids[t * k + r] = my_id;
      a.w[t * k + r] = (float)((double)a.scale * s);
    }
  }
}

template <int LANES, int EPL, typename LT>
__global__ __launch_bounds__(64 * kWaves) void k_route_scored_backward(
    RouteArgs a, const int32_t* __restrict__ ids,
    const float* __restrict__ d_w, LT* __restrict__ d_logits) {
  constexpr int SEGS = 64 / LANES;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & (LANES - 1), seg = lane / LANES, base = seg * LANES;
  const int E = a.E, k = a.k;
  const int per_block = kWaves * SEGS;
  // a softmax with renormalised weights is the softmax over the k chosen:
  // only their logits are read
  const bool dense = !a.sigmoid && !a.renorm;
  for (long t0 = (long)blockIdx.x * per_block; t0 < a.T;
       t0 += (long)gridDim.x * per_block) {
    const long tt = t0 + wv * SEGS + seg;
    const bool valid = tt < a.T;
    const long t = valid ? tt : a.T - 1;
    const LT* row = (const LT*)a.logits + t * a.stride;
    int id = -1;
    double lj = -__builtin_inf(), dw = 0.0;
    if (r < k) {
      id = ids[t * k + r];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        lj = logit_of<LT>(row[id]);
        dw = (double)a.scale * (double)d_w[t * k + r];
      }
    }
    double p[EPL], m = 0.0, sum = 1.0;
    if (dense) {
      m = -__builtin_inf();
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = r * EPL + i;
        p[i] = e < E ? logit_of<LT>(row[e]) : -__builtin_inf();
        m = fmax(m, p[i]);
      }
      m = seg_max<LANES>(m);
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        p[i] = softmax_num(p[i], m);
        sum += p[i];
      }
      sum = seg_sum<LANES>(sum);
    } else if (!a.sigmoid) {
      m = seg_max<LANES>(lj);
    }
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
    double s = a.sigmoid ? sigmoid_f64(lj) : softmax_num(lj, m) * inv;
    double ds = dw;
    if (a.renorm) {
      const double S = seg_sum<LANES>(s);
      const double q = seg_sum<LANES>(s > 0.0 ? dw * s : 0.0);
      ds = S > 0.0 ? (dw - q / S) / S : 0.0;
    }
    // slot j's own part, and for a dense softmax the part of every expert
    double part = 0.0, all = 0.0;
    if (s > 0.0) {
      if (a.sigmoid) {
        const double e = exp(-fabs(lj));
        part = ds * e / ((1.0 + e) * (1.0 + e));
      } else {
        part = ds * s;
      }
    }
    if (dense) all = seg_sum<LANES>(part) * inv;
    double d[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) d[i] = dense && p[i] > 0.0 ? -p[i] * all : 0.0;
    for (int j = 0; j < k; ++j) {
      const int e = __shfl(id, base + j, 64);
      const double v = __shfl(part, base + j, 64);
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e == r * EPL + i) d[i] += v;
    }
    if (valid) {
      LT* out = d_logits + t * a.stride;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = r * EPL + i;
        if (e < E) {
          if constexpr (sizeof(LT) == 4) out[e] = (float)d[i];
          else out[e] = f32_to_bf16((float)d[i]);
        }
      }
    }
  }
}

// Expert counts of a large batch: a workgroup counts its share of the ids in
// LDS and stores its histogram; a second launch sums the histograms.
constexpr int kCountIds = 4096;     // ids a workgroup counts

__global__ __launch_bounds__(256) void k_count_share(
    const int32_t* __restrict__ ids, long n, int E, int32_t* __restrict__ part) {
  __shared__ int32_t h[4][MOE_EMAX];
  const int tid = threadIdx.x;
  for (int i = tid; i < 4 * E; i += 256) h[i / E][i % E] = 0;
  __syncthreads();
  const long b = (long)blockIdx.x * kCountIds;
  const long end = b + kCountIds < n ? b + kCountIds : n;
  for (long i = b + tid; i < end; i += 256) {
    const int e = ids[i];
    if ((unsigned)e < (unsigned)E) atomicAdd(&h[tid >> 6][e], 1);
  }
  __syncthreads();
  for (int e = tid; e < E; e += 256)
    part[(size_t)blockIdx.x * E + e] = h[0][e] + h[1][e] + h[2][e] + h[3][e];
}

__global__ __launch_bounds__(256) void k_count_sum(
    const int32_t* __restrict__ part, int parts, int E,
    int32_t* __restrict__ counts) {
  __shared__ int32_t s[4][64];
  const int c = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + c;
  int v = 0;
  if (e < E)
    for (int p = q; p < parts; p += 4) v += part[(size_t)p * E + e];
  s[q][c] = v;
  __syncthreads();
  if (q == 0 && e < E) counts[e] = s[0][c] + s[1][c] + s[2][c] + s[3][c];
}

RouteArgs route_args(const moe_router* r, const void* logits) {
  RouteArgs a{};
  a.logits = logits;
  a.T = r->T;
  a.E = r->E;
  a.k = r->k;
  a.sigmoid = r->score == MOE_SCORE_SIGMOID;
  a.groups = r->topk_groups == r->groups ? 1 : r->groups;   // all stay: none
  a.keep = r->topk_groups;
  a.group_top = r->group_top;
  a.renorm = r->renormalize;
  a.per = r->E / r->groups;
  a.per_inv = ((1u << 20) + a.per - 1) / a.per;
  a.scale = r->scale;
  a.stride = r->logits_stride;
  return a;
}

int route_grid(int T, int E) {
  const int per_block = kWaves * (E <= 64 ? 4 : 1);
  const long n = ((long)T + per_block - 1) / per_block;
  return (int)(n < 65536 ? n : 65536);
}

// calls f(integral LANES, integral EPL)
template <class F>
void by_experts(int E, F f) {
  using std::integral_constant;
  if (E <= 16) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (E <= 32) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128) f(integral_constant<int, 64>{}, integral_constant<int, 2>{});
  else if (E <= 256) f(integral_constant<int, 64>{}, integral_constant<int, 4>{});
  else if (E <= 512) f(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}

}  // namespace

size_t route_scored_partials(const moe_router* r) {
  const long n = (long)r->T * r->k;
  if (n <= 2 * kCountIds) return 0;
  return (size_t)((n + kCountIds - 1) / kCountIds) * r->E;
}

hipError_t launch_route_scored(const moe_router* r, const void* logits,
                               const float* bias, int32_t* ids, float* w,
                               int32_t* counts, int32_t* partials,
                               hipStream_t s) {
  RouteArgs a = route_args(r, logits);
  a.bias = bias;
  a.ids = ids;
  a.w = w;
  const dim3 grid(route_grid(r->T, r->E)), block(64 * kWaves);
  by_experts(r->E, [&](auto lanes, auto epl) {
    if (r->logits_dtype == MOE_F32)
      k_route_scored<lanes.value, epl.value, float><<<grid, block, 0, s>>>(a);
    else
      k_route_scored<lanes.value, epl.value, bf16_t><<<grid, block, 0, s>>>(a);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !counts) return e;
  const long n = (long)r->T * r->k;
  if (n <= 2 * kCountIds) return launch_count_ids(ids, (int)n, r->E, counts, s);
  const int parts = (int)((n + kCountIds - 1) / kCountIds);
  k_count_share<<<parts, 256, 0, s>>>(ids, n, r->E, partials);
  k_count_sum<<<(r->E + 63) / 64, 256, 0, s>>>(partials, parts, r->E, counts);
  return hipGetLastError();
}

hipError_t launch_route_scored_backward(const moe_router* r,
                                        const void* logits,
                                        const int32_t* ids, const float* d_w,
                                        void* d_logits, hipStream_t s) {
  const RouteArgs a = route_args(r, logits);
  const dim3 grid(route_grid(r->T, r->E)), block(64 * kWaves);
  by_experts(r->E, [&](auto lanes, auto epl) {
    if (r->logits_dtype == MOE_F32)
      k_route_scored_backward<lanes.value, epl.value, float>
          <<<grid, block, 0, s>>>(a, ids, d_w, (float*)d_logits);
    else
      k_route_scored_backward<lanes.value, epl.value, bf16_t>
          <<<grid, block, 0, s>>>(a, ids, d_w, (bf16_t*)d_logits);
  });
  return hipGetLastError();
}

}  // namespace moe
