// Scored routing (moe_route_scored) and its gradient.
//
// A token's experts lie on a segment of 16 lanes (E <= 64, four tokens a
// wavefront) or a whole wavefront, EPL neighbouring experts a lane, so the
// lowest lane among equal values holds the lowest id.
//
// The chosen ids must be those of the definition in 64 bits, and in float32
// neighbouring choices of some hundred experts collide within an ulp too
// often.  So a token is chosen in float32, the scores of the k chosen (which
// the weights need) are evaluated in double, and these prove the choice:
//   - the doubles stand in slot order (equal ones by id), and
//   - the last of them exceeds the best choice left behind by more than a
//     bound on float32's error, and likewise the last group that stays
//     exceeds the best that does not.
// The few tokens without that proof are chosen again in double throughout.
//
// Each lane sorts its few choices as integer keys in the order of the
// choices; a slot is then one max over the lanes' first keys in DPP steps of
// one instruction, and the owner moves its list up.  Bound by instructions
// (8192 tokens of 256 experts in 8 groups: 698 a token, 15 us; in double
// throughout 21 us) and, for a single token, by their latency (4.6 us).
#include <float.h>
#include <algorithm>
#include <type_traits>

#include "block.h"

namespace moe {

namespace {

// Choice of a masked expert, below every live one.
constexpr double kMasked = -DBL_MAX;

// Keys order as choices do: the bits of a double mapped to an unsigned order.
// Masked experts are all equal and come last; kGone is what is taken, outside
// the groups that stay, or padding.
constexpr uint64_t kMaskedKey = 1ull << 32, kGone = 0;
__device__ __forceinline__ uint64_t key_of(double c) {
  const uint64_t b = __double_as_longlong(c);
  return c == kMasked ? kMaskedKey : (b >> 63 ? ~b : b | (1ull << 63));
}

// A DPP move within rows of 16 lanes, every lane written (a lane without a
// source gets 0): no old value, so the compiler folds it into the operation.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return __builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __double_as_longlong(v);
  return __longlong_as_double(((uint64_t)dpp<CTRL>((uint32_t)(b >> 32)) << 32) | dpp<CTRL>((uint32_t)b));
}
// The row broadcasts: lane 15 (CTRL 0x142) or 31 (0x143) of the rows before
// into the rows of the mask, 0 elsewhere.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t bcast(uint32_t v) {
  return __builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}

__device__ __forceinline__ float read_lane(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
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
__device__ __forceinline__ uint32_t seg_max(uint32_t v) {
  v = max(v, dpp<0x128>(v));
  v = max(v, dpp<0x124>(v));
  v = max(v, dpp<0x122>(v));
  v = max(v, dpp<0x121>(v));
  if (LANES == 64) {
    v = max(v, bcast<0x142, 0xA>(v));
    v = max(v, bcast<0x143, 0xC>(v));
    v = __builtin_amdgcn_readlane((int)v, 63);
  }
  return v;
}
// floats as unsigned integers of the same order
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t m) {
  return __uint_as_float(m >> 31 ? m & 0x7FFFFFFFu : ~m);
}
template <int LANES>
__device__ __forceinline__ float seg_max(float v) {
  return from_order(seg_max<LANES>(order_of(v)));
}

// sum over the 16 lanes of a row / over a segment, in every lane of it
__device__ __forceinline__ double row_sum(double v) {
  v += dpp<0x128>(v);
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  return v + dpp<0x121>(v);
}
template <int LANES>
__device__ __forceinline__ double seg_sum(double v) {
  v = row_sum(v);
  if (LANES == 64)
    v = (read_lane(v, 0) + read_lane(v, 16)) + (read_lane(v, 32) + read_lane(v, 48));
  return v;
}

// a logit, with NaN read as -inf
__device__ __forceinline__ float logit_of(float v) { return v == v ? v : -__builtin_inff(); }
__device__ __forceinline__ float logit_of(bf16_t v) { return logit_of(bf16_to_f32(v)); }

// N logits at `p`; VEC: N * sizeof(LT) bytes aligned to 16 or to their size
template <int N, bool VEC, typename LT>
__device__ __forceinline__ void load_logits(const LT* p, int n, float* l) {
  if (VEC && n >= N) {
    constexpr int B = N * (int)sizeof(LT) < 16 ? N * (int)sizeof(LT) : 16;
    struct alignas(B) Block { LT v[B / sizeof(LT)]; };
    constexpr int M = B / sizeof(LT);
#pragma unroll
    for (int j = 0; j < N / M; ++j) {
      const Block b = ((const Block*)p)[j];
#pragma unroll
      for (int i = 0; i < M; ++i) l[j * M + i] = logit_of(b.v[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] = i < n ? logit_of(p[i]) : -__builtin_inff();
  }
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
  int vec, bias_vec;      // logits / bias rows load as vectors
  int whole;              // groups are runs of whole lanes, 2^share of them
  int share;              // 2^share lanes find a group's best, share <= 4
  uint32_t per_inv;       // e / per == (e * per_inv) >> 20 for e < 1024
  float scale;
  int64_t stride;
  int32_t* ids;
  float* w;
  int32_t* counts;        // or null: [gridDim.x][E], each workgroup's pairs
};

constexpr int kWaves = 8;   // wavefronts a workgroup

__device__ __forceinline__ double max_of(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double min_of(double a, double b) { return fmin(a, b); }
__device__ __forceinline__ float max_of(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float min_of(float a, float b) { return fminf(a, b); }

// the best two of two pairs of best ones, the second in another lane
template <int CTRL, typename V>
__device__ __forceinline__ void merge_best(V& a0, V& a1) {
  const V b0 = dpp<CTRL>(a0), b1 = dpp<CTRL>(a1);
  a1 = max_of(min_of(a0, b0), max_of(a1, b1));
  a0 = max_of(a0, b0);
}

// whether group g of score v is among the `keep` best; score(h) is group h's
template <class F>
__device__ __forceinline__ bool group_stays(int g, double v, int groups, int keep, F score) {
  int better = 0;
  for (int h = 0; h < groups; ++h) {
    const double s = score(h);
    better += (s > v || (s == v && h < g)) ? 1 : 0;
  }
  return better < keep;
}
template <class F>
__device__ __forceinline__ bool group_stays(int g, float v, int groups, int keep, F score) {
  // of equal scores the lower group's is above: order(v) less 1
  const uint32_t o = order_of(v);
  int better = 0;
  for (int h = 0; h < groups; ++h)
    better += order_of(score(h)) > (h < g ? o - 1 : o) ? 1 : 0;
  return better < keep;
}

// orders the scratch accesses of one wavefront's lanes
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Clears the keys of the experts whose group does not stay; V: float or
// double.  A group's two best choices are found by a run of neighbouring
// lanes: those that hold its experts, where groups are whole lanes, else as
// many as the segment has for a group, through `scratch` (LANES * EPL values
// of one token).
// For float *gap is the distance of the last group that stays from the best
// that does not, and *big the largest choice's magnitude; gap = +inf where
// the border lies at groups without a live expert.
template <int LANES, int EPL, typename V, typename K>
__device__ __forceinline__ void stay_mask(const RouteArgs& a, const V* c, K* key,
                                          V masked, int r, int base,
                                          double* scratch, float* gap,
                                          float* big) {
  const int e0 = r * EPL;
  const int sh = a.share, g = r >> sh;
  V b0 = masked, b1 = masked;
  if (a.whole) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      b1 = max_of(b1, min_of(b0, c[i]));
      b0 = max_of(b0, c[i]);
    }
  } else {
    V* ch = (V*)scratch;
    wave_fence();
#pragma unroll
    for (int i = 0; i < EPL; ++i) ch[e0 + i] = c[i];
    wave_fence();
    if (g < a.groups) {
#pragma unroll 4
      for (int i = r - (g << sh); i < a.per; i += 1 << sh) {
        const V v = ch[g * a.per + i];
        b1 = max_of(b1, min_of(b0, v));
        b0 = max_of(b0, v);
      }
    }
  }
  if (sh >= 1) merge_best<0xB1>(b0, b1);     // lanes 1 0 3 2
  if (sh >= 2) merge_best<0x4E>(b0, b1);     // lanes 2 3 0 1
  if (sh >= 3) merge_best<0x141>(b0, b1);    // half row mirrored
  if (sh >= 4) merge_best<0x140>(b0, b1);   // row mirrored
  V score = (a.group_top == 2 && b1 > masked) ? b0 + b1 : b0;
  const bool stays = group_stays(g, score, a.groups, a.keep, [&](int h) {
    if (LANES == 64) return read_lane(score, h << sh);
    return (V)__shfl(score, base + (h << sh), 64);
  }) && g < a.groups;
  if (gap) {
    if (g >= a.groups) score = masked;
    const float s32 = score > masked ? (float)score : -__builtin_inff();
    const float low = seg_max<LANES>(stays && score > masked ? -s32 : -__builtin_inff());
    const float next = seg_max<LANES>(stays ? -__builtin_inff() : s32);
    *gap = next == -__builtin_inff() ? __builtin_inff() : -low - next;
    *big = seg_max<LANES>(fmaxf(b0 > masked ? fabsf((float)b0) : 0.0f,
                                b1 > masked ? fabsf((float)b1) : 0.0f));
  }
  if (a.whole) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = stays ? key[i] : K(0);
  } else {
    const uint64_t kept = __ballot(stays) >> base;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const uint32_t h = ((uint32_t)(e0 + i) * a.per_inv) >> 20;
      if (!((kept >> ((h << sh) & 63)) & 1)) key[i] = K(0);
    }
  }
}

// A lane's keys in descending order, equal ones by id: neighbours only swap
// where the right one is larger.
template <int EPL, typename K>
__device__ __forceinline__ void sort_keys(K* key, uint32_t* id) {
#pragma unroll
  for (int n = EPL - 1; n > 0; --n) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      // (values, not elements: a conditional between two elements of an array
      // is an element, and its index would be chosen at run time)
      const K a = key[i], b = key[i + 1];
      const uint32_t ia = id[i], ib = id[i + 1];
      const bool up = b > a;
      key[i] = up ? b : a;
      key[i + 1] = up ? a : b;
      id[i] = up ? ib : ia;
      id[i + 1] = up ? ia : ib;
    }
  }
}

// the lanes whose first key is the largest of their segment
template <int LANES>
__device__ __forceinline__ uint64_t lanes_of_max(uint32_t key) {
  return __ballot(key == seg_max<LANES>(key));
}
template <int LANES>
__device__ __forceinline__ uint64_t lanes_of_max(uint64_t key) {
  const uint32_t hi = (uint32_t)(key >> 32);
  const uint64_t m = __ballot(hi == seg_max<LANES>(hi));
  if (__popcll(m) <= 64 / LANES) return m;
  // upper halves tie somewhere: the lower ones decide
  const uint32_t lo = (m >> (threadIdx.x & 63)) & 1 ? (uint32_t)key : 0u;
  return m & __ballot(lo == seg_max<LANES>(lo));
}

// The k largest keys of a segment's experts (lane r's are r * EPL + i): lane
// j < k gets the id of slot j; *left becomes the largest key that stays.  Up
// to 8 keys of 32 bits or 4 of 64 a lane are sorted first; more are scanned in
// every round, which needs no second array (sorting 16 spilled registers).
template <int LANES, int EPL, typename K>
__device__ __forceinline__ int take_slots(K* key, int k, int r, int base, K* left) {
  constexpr bool kSort = EPL * sizeof(K) <= 32;
  uint32_t id[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) id[i] = r * EPL + i;
  if constexpr (kSort) sort_keys<EPL>(key, id);
  int my_id = 0;
  for (int j = 0;; ++j) {
    K head = key[0];
    uint32_t head_id = id[0];
    if constexpr (!kSort) {
#pragma unroll
      for (int i = 1; i < EPL; ++i) {
        const K a = key[i];
        const bool up = a > head;
        head = up ? a : head;
        head_id = up ? r * EPL + i : head_id;
      }
    }
    if (j == k) {
      *left = head;
      break;
    }
    const uint64_t first = lanes_of_max<LANES>(head);
    int owner, e;
    if (LANES == 64) {
      owner = __ffsll((unsigned long long)first) - 1;
      e = __builtin_amdgcn_readlane((int)head_id, owner);
    } else {
      owner = base + __ffs((int)((first >> base) & 0xFFFFu)) - 1;
      e = __shfl((int)head_id, owner, 64);
    }
    if (r == j) my_id = e;
    if constexpr (kSort) {
      const bool mine = (int)(threadIdx.x & 63) == owner;
#pragma unroll
      for (int i = 0; i + 1 < EPL; ++i) {
        const K a = key[i], b = key[i + 1];
        const uint32_t ia = id[i], ib = id[i + 1];
        key[i] = mine ? b : a;
        id[i] = mine ? ib : ia;
      }
      const K a = key[EPL - 1];
      key[EPL - 1] = mine ? K(0) : a;
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = r * EPL + i == e ? K(0) : key[i];
    }
  }
  return my_id;
}

template <int LANES, int EPL, typename LT>
__global__ __launch_bounds__(64 * kWaves) void k_route_scored(RouteArgs a) {
  constexpr int SEGS = 64 / LANES;
  const float kInf = __builtin_inff();
  extern __shared__ double lds_groups[];   // groups of any size: a token's
  __shared__ int32_t hist[MOE_EMAX];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & (LANES - 1), seg = lane / LANES, base = seg * LANES;
  const int E = a.E, k = a.k, e0 = r * EPL;
  const int waves = blockDim.x >> 6, per_block = waves * SEGS;
  double* scratch = lds_groups + (wv * SEGS + seg) * (LANES * EPL);
  if (a.counts) {
    for (int e = threadIdx.x; e < E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
  }
  float l[EPL], b[EPL], ahead[EPL];
  auto fetch = [&](long t) {            // a token's logits, before its turn
    const LT* row = (const LT*)a.logits + min(t, (long)a.T - 1) * a.stride;
    if (a.vec) load_logits<EPL, true, LT>(row + e0, E - e0, ahead);
    else load_logits<EPL, false, LT>(row + e0, E - e0, ahead);
  };
  const long turn = (long)gridDim.x * per_block;
  const long t_first = (long)blockIdx.x * per_block + wv * SEGS + seg;
  fetch(t_first);
  if (a.bias) {                           // (a NaN reads as -inf: masked)
    if (a.bias_vec) load_logits<EPL, true, float>(a.bias + e0, E - e0, b);
    else load_logits<EPL, false, float>(a.bias + e0, E - e0, b);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) b[i] = 0.0f;
  }
  // value i of the lane that holds expert e, for each lane's own e
  auto of_expert = [&](const float* x, int e) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float f = __shfl(x[i], base + e / EPL, 64);
      v = e % EPL == i ? f : v;
    }
    return v;
  };
  for (long t = t_first; __ballot(t < a.T); t += turn) {
    const bool valid = t < a.T;
#pragma unroll
    for (int i = 0; i < EPL; ++i) l[i] = ahead[i];
    if (__ballot(t + turn < a.T)) fetch(t + turn);
    // float32 choices and a bound on a score's error.  Sigmoid, in 2^-24: the
    // exponent's argument s (1 - s) |l| 1.5 <= 0.34, its power s (1 - s) 2 <=
    // 0.5, the sum 1, the reciprocal 2, together below 4 = 2^-22; twice that
    // is taken.  Softmax scores are rounded from double.
    float c[EPL];
    double m = 0.0, sum = 0.0;
    float err;
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(l[i] * -1.44269504088896340736f));
      err = 0x1p-21f;
    } else {
      float top = l[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
      m = (double)seg_max<LANES>(top);
      double p[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        p[i] = softmax_num((double)l[i], m);
        sum += p[i];
      }
      sum = seg_sum<LANES>(sum);
      const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = (float)(p[i] * inv);
      err = 0x1p-23f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = l[i] > -kInf ? c[i] + b[i] : -kInf;
    bool sure = true;
    uint32_t key[EPL], left;              // masked choices are -inf, the lowest
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = e0 + i < E ? order_of(c[i]) : 0u;
    if (a.groups > 1) {
      float gap, big;
      stay_mask<LANES, EPL, float>(a, c, key, -kInf, r, base, scratch, &gap, &big);
      // two sums of two choices each, with their own rounding
      // (past 1e37 a float32 sum may overflow)
      sure = gap > 4.0f * (err + big * 0x1p-22f) && big < 1e37f;
    }
    int my_id = take_slots<LANES, EPL>(key, k, r, base, &left);
    const float next = from_order(max(seg_max<LANES>(left), order_of(-kInf)));
    // lane j < k: the score and choice of slot j in double
    const bool slot = r < k;
    const double low = -__builtin_inf();
    auto score_of = [&](double lj) {
      return a.sigmoid ? sigmoid_f64(lj) : (sum > 0.0 ? softmax_num(lj, m) / sum : 0.0);
    };
    double lj = (double)of_expert(l, my_id);
    if (!slot) lj = low;
    double s = score_of(lj);
    double v = low;
    const float bj = a.bias ? of_expert(b, my_id) : 0.0f;
    if (lj > low) v = s + (double)bj;
    {
      const double v1 = dpp<0x101>(v);                   // the next lane's
      const int id1 = (int)dpp<0x101>((uint32_t)my_id);
      if (r < k - 1 && v1 > low) sure = sure && (v > v1 || (v == v1 && my_id < id1));
      if (r == k - 1 && next > -kInf)
        sure = sure && v > (double)next + (double)(err + fabsf(next) * 0x1p-22f);
    }
    if (__ballot(!sure)) {
      double c64[EPL];
      uint64_t key64[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c64[i] = score_of((double)l[i]) + (double)b[i];
        if (!(c[i] > -kInf)) c64[i] = kMasked;
        key64[i] = e0 + i < E ? key_of(c64[i]) : kGone;
      }
      if (a.groups > 1)
        stay_mask<LANES, EPL, double>(a, c64, key64, kMasked, r, base, scratch, nullptr, nullptr);
      uint64_t rest;
      my_id = take_slots<LANES, EPL>(key64, k, r, base, &rest);
      lj = (double)of_expert(l, my_id);
      s = score_of(slot ? lj : low);
    }
    if (a.renorm) {
      const double S = row_sum(slot ? s : 0.0);   // the slots' lanes are a row
      s = S > 0.0 ? s / S : 0.0;
    }
    if (valid && slot) {
      a.ids[t * k + r] = my_id;
      a.w[t * k + r] = (float)((double)a.scale * s);
      if (a.counts) atomicAdd(&hist[my_id], 1);
    }
  }
  if (a.counts) {
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x)
      a.counts[(size_t)blockIdx.x * E + e] = hist[e];
  }
}

constexpr int kGradWaves = 4;

// N gradients, of which the row has n; VEC as for load_logits.  bf16 rounds
// the rounded float: off by 2^-24 of a value besides its half step.
template <int N, typename LT>
__device__ __forceinline__ void store_grad(LT* p, const float* d, int n, int vec) {
  auto put = [](float f) -> LT {
    if constexpr (sizeof(LT) == 4) return f;
    else return f32_to_bf16(f);
  };
  if (vec && n >= N) {
    constexpr int B = N * (int)sizeof(LT) < 16 ? N * (int)sizeof(LT) : 16;
    struct alignas(B) Block { LT v[B / sizeof(LT)]; };
    constexpr int M = B / sizeof(LT);
#pragma unroll
    for (int j = 0; j < N / M; ++j) {
      Block b;
#pragma unroll
      for (int i = 0; i < M; ++i) b.v[i] = put(d[j * M + i]);
      ((Block*)p)[j] = b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) p[i] = put(d[i]);
  }
}

template <int LANES, int EPL, typename LT>
__global__ __launch_bounds__(64 * kGradWaves) void k_route_scored_backward(
    RouteArgs a, const int32_t* __restrict__ ids,
    const float* __restrict__ d_w, LT* __restrict__ d_logits) {
  constexpr int SEGS = 64 / LANES;
  // a token's row of slot parts; only its own wavefront touches it
  __shared__ double lds_row[kGradWaves][SEGS][LANES * EPL];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int r = lane & (LANES - 1), seg = lane / LANES;
  const int E = a.E, k = a.k;
  const int per_block = kGradWaves * SEGS;
  double* parts = lds_row[wv][seg];
  // A softmax with renormalised weights is the softmax over the k chosen,
  // unless their scores among all E vanish (a bias lifted experts far below
  // the row's largest logit): the row is read for that alone, its sum only
  // where it can be (8192 x 256: 7.6 us; the k logits alone 5.9).
  const bool dense = !a.sigmoid && !a.renorm;
  for (long t0 = (long)blockIdx.x * per_block; t0 < a.T;
       t0 += (long)gridDim.x * per_block) {
    const long tt = t0 + wv * SEGS + seg;
    const bool valid = tt < a.T;
    const long t = valid ? tt : a.T - 1;
    const LT* row = (const LT*)a.logits + t * a.stride;
    float l[EPL];                      // requested ahead of the slots' chain
    if (!a.sigmoid) {
      if (a.vec) load_logits<EPL, true, LT>(row + r * EPL, E - r * EPL, l);
      else load_logits<EPL, false, LT>(row + r * EPL, E - r * EPL, l);
    }
    int id = -1;
    double lj = -__builtin_inf(), dw = 0.0;
    if (r < k) {
      id = ids[t * k + r];
      if (id < 0 || id >= E) id = -1;
      if (id >= 0) {
        lj = (double)logit_of(row[id]);
        dw = (double)a.scale * (double)d_w[t * k + r];
      }
    }
    double p[EPL], m = 0.0, sum = 1.0;
    bool vanish = false;               // the chosen scores are all 0
    if (!a.sigmoid) {
      float top = l[0];
#pragma unroll
      for (int i = 1; i < EPL; ++i) top = fmaxf(top, l[i]);
      const float best = dense ? 0.0f : seg_max<LANES>((float)lj);
      // (exp(-700) / 1024 is a normal number: nothing vanishes before)
      if (dense || __ballot(top - best > 700.0f)) {
        m = (double)seg_max<LANES>(top);
        sum = 0.0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          p[i] = softmax_num((double)l[i], m);
          sum += p[i];
        }
        sum = seg_sum<LANES>(sum);
        if (!dense) vanish = !(softmax_num((double)best, m) / sum > 0.0);
      }
      if (!dense) {
        m = (double)best;
        sum = 1.0;
      }
    }
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
    const double s = a.sigmoid ? sigmoid_f64(lj) : softmax_num(lj, m) * inv;
    // what a slot's part is the product of: the gradient of its weight less
    // the weights' mean of them, and the weight.  (1 / S alone may pass the
    // range of 64 bits, s / S does not.)
    double ds = dw, u = s;
    if (a.renorm) {
      const double S = row_sum(s);     // (the slots' lanes are a row)
      u = S > 0.0 && !vanish ? s / S : 0.0;
      ds = dw - row_sum(u > 0.0 ? dw * u : 0.0);
    }
    // slot j's own part, and for a dense softmax the part of every expert
    double part = 0.0, all = 0.0;
    if (u > 0.0) {
      part = ds * u;
      if (a.sigmoid) {                 // times 1 - s
        const double e = exp(-fabs(lj));
        part *= (lj >= 0.0 ? e : 1.0) / (1.0 + e);
      }
    }
    if (dense) all = seg_sum<LANES>(part) * inv;
    // slots to experts through LDS (an id given twice adds up): 8192 x 256
    // 6.6 us, against 9.5 us when every lane asked for each slot in turn
    wave_fence();
#pragma unroll
    for (int i = 0; i < EPL; ++i) parts[r * EPL + i] = 0.0;
    wave_fence();
    if (id >= 0) __hip_atomic_fetch_add(parts + id, part, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    wave_fence();
    float d[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      double v = parts[r * EPL + i];
      if (dense && p[i] > 0.0) v -= p[i] * all;
      d[i] = (float)v;
    }
    if (valid) store_grad<EPL, LT>(d_logits + t * a.stride + r * EPL, d, E - r * EPL, a.vec);
  }
}

// counts[e] = sum of the workgroups' counts: 16 experts a workgroup, 64 slices
// of the parts, four of them a wavefront
__global__ __launch_bounds__(1024) void k_count_sum(
    const int32_t* __restrict__ part, int parts, int E,
    int32_t* __restrict__ counts) {
  __shared__ int32_t s[16][16];
  const int c = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int e = blockIdx.x * 16 + c;
  int v = 0;
  if (e < E) {
#pragma unroll 8
    for (int p = q; p < parts; p += 64) v += part[(size_t)p * E + e];
  }
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if ((threadIdx.x & 63) < 16) s[threadIdx.x >> 6][c] = v;
  __syncthreads();
  if (threadIdx.x < 16 && e < E) {
    v = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) v += s[k][c];
    counts[e] = v;
  }
}

// Lanes a token's experts take, and experts a lane.  (256 experts on 16 lanes,
// four tokens a wavefront, took the same time for 8192 tokens and 1.7 times as
// long for one.)
int lanes_of(const moe_router* r) {
  return r->E <= 64 && r->groups <= 16 ? 16 : 64;
}
int per_lane(int E, int lanes) {
  int n = 1;
  while (lanes * n < E) n *= 2;
  return n;
}

// calls f(integral LANES, integral EPL)
template <class F>
void by_experts(int E, int lanes, F f) {
  using std::integral_constant;
  const int n = per_lane(E, lanes);
  if (lanes == 16) {
    integral_constant<int, 16> l;
    if (n == 1) f(l, integral_constant<int, 1>{});
    else if (n == 2) f(l, integral_constant<int, 2>{});
    else f(l, integral_constant<int, 4>{});
  } else {
    integral_constant<int, 64> l;
    if (n == 1) f(l, integral_constant<int, 1>{});
    else if (n == 2) f(l, integral_constant<int, 2>{});
    else if (n == 4) f(l, integral_constant<int, 4>{});
    else if (n == 8) f(l, integral_constant<int, 8>{});
    else f(l, integral_constant<int, 16>{});
  }
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
  const int all = lanes_of(r), n = per_lane(r->E, all);
  if (a.groups > 1) {
    const int lanes = a.per / n;
    a.whole = a.per % n == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
    while (a.share < 4 && (a.whole ? (1 << a.share) < lanes
                                   : (2 << a.share) * a.groups <= all))
      ++a.share;
  }
  const int bytes = r->logits_dtype == MOE_BF16 ? 2 : 4;
  const int piece = n * bytes < 16 ? n * bytes : 16;
  a.vec = (uintptr_t)logits % piece == 0 && r->logits_stride * bytes % piece == 0;
  a.scale = r->scale;
  a.stride = r->logits_stride;
  return a;
}

// Workgroups and wavefronts: a token's segment a wavefront's turn.  A few
// tokens share one workgroup, which then counts the experts by itself; more
// spread over the CUs; the wavefronts that stay on the GPU at once walk larger
// batches (128 tokens of 256 experts with counts: 7.1 us, 8.1 with 8
// wavefronts a workgroup throughout).
constexpr int kCus = 256;
struct RouteShape {
  int waves, grid;
};
RouteShape route_shape(const moe_router* r) {
  const int segs = 64 / lanes_of(r);
  const long w = ((long)r->T + segs - 1) / segs;
  RouteShape s;
  s.waves = (int)(w <= kWaves ? w : std::min<long>((w + kCus - 1) / kCus, kWaves));
  s.grid = (int)std::min<long>((w + s.waves - 1) / s.waves, 2 * kCus);
  return s;
}

}  // namespace

// Expert counts: a single workgroup stores its own; some thousand ids are
// counted again by one workgroup; beyond, every workgroup leaves its counts in
// the scratch and a second launch sums them.
static bool sums_counts(const moe_router* r, const RouteShape& s) {
  return s.grid > 1 && (long)r->T * r->k > 8192;
}

size_t route_scored_partials(const moe_router* r) {
  if (r->T == 0) return 0;
  const RouteShape s = route_shape(r);
  return sums_counts(r, s) ? (size_t)s.grid * r->E : 0;
}

// The grid falls whenever the wavefronts a workgroup grow: below kCus
// workgroups until they are kWaves, then it grows with T to its end.
size_t route_scored_scratch(const moe_router* r) {
  if (!route_scored_partials(r)) return 0;
  return (size_t)std::max(kCus, route_shape(r).grid) * r->E;
}

hipError_t launch_route_scored(const moe_router* r, const void* logits,
                               const float* bias, int32_t* ids, float* w,
                               int32_t* counts, int32_t* partials,
                               hipStream_t s) {
  RouteArgs a = route_args(r, logits);
  a.bias = bias;
  a.bias_vec = (uintptr_t)bias % 16 == 0;
  a.ids = ids;
  a.w = w;
  const RouteShape sh = route_shape(r);
  const bool sum = counts && sums_counts(r, sh);
  a.counts = sum ? partials : sh.grid == 1 ? counts : nullptr;
  const dim3 grid(sh.grid), block(64 * sh.waves);
  by_experts(r->E, lanes_of(r), [&](auto lanes, auto epl) {
    constexpr int L = lanes.value, N = epl.value;
    const size_t lds = a.groups > 1 && !a.whole
                           ? sizeof(double) * sh.waves * 64 * N : 0;
    if (r->logits_dtype == MOE_F32)
      k_route_scored<L, N, float><<<grid, block, lds, s>>>(a);
    else
      k_route_scored<L, N, bf16_t><<<grid, block, lds, s>>>(a);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !counts || sh.grid == 1) return e;
  if (!sum) return launch_count_ids(ids, r->T * r->k, r->E, counts, s);
  k_count_sum<<<(r->E + 15) / 16, 1024, 0, s>>>(partials, sh.grid, r->E, counts);
  return hipGetLastError();
}

hipError_t launch_route_scored_backward(const moe_router* r,
                                        const void* logits,
                                        const int32_t* ids, const float* d_w,
                                        void* d_logits, hipStream_t s) {
  RouteArgs a = route_args(r, logits);
  a.vec = a.vec && route_args(r, d_logits).vec;
  const int per_block = kGradWaves * (64 / lanes_of(r));
  const dim3 grid((int)std::min<long>(((long)r->T + per_block - 1) / per_block, 65536));
  const dim3 block(64 * kGradWaves);
  by_experts(r->E, lanes_of(r), [&](auto lanes, auto epl) {
    constexpr int L = lanes.value, N = epl.value;
    if (r->logits_dtype == MOE_F32)
      k_route_scored_backward<L, N, float><<<grid, block, 0, s>>>(a, ids, d_w, (float*)d_logits);
    else
      k_route_scored_backward<L, N, bf16_t><<<grid, block, 0, s>>>(a, ids, d_w, (bf16_t*)d_logits);
  });
  return hipGetLastError();
}

}  // namespace moe
