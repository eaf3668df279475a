// The whole layer for a few tokens (up to 16) in two kernels: gate/up with
// the router and the list of experts in use, then down with the combine.
//
// Bound by the experts' weights, each read once, and below some tens of MB by
// latency, of which the general layer's five launches are the largest part.
// A token is a column of the matrix instruction: 16 output channels (one
// packed weight block, A) times 16 tokens (B), whichever of them chose the
// expert -- a column does not touch another, so rows of x are never gathered
// or permuted and the columns of other tokens are simply not stored.
//
//   k_few_gate_up  every workgroup routes the tokens itself (16 tokens are
//                  one pass of four wavefronts; a launch of its own costs
//                  more) and lists the experts in use; item = 16 channels of
//                  one of them, gate and up, the reduction cut over the
//                  workgroup's wavefronts and joined in LDS; h in bf16.
//                  Workgroup 0 leaves the list and the weights behind.
//   k_few_down     workgroup = 16 output channels of all experts in use:
//                  (expert, 128 of the reduction) units are dealt to the
//                  wavefronts, each adds weight * product, and the sums are
//                  joined in LDS in wavefront order and rounded once.
//
// 16 tokens of 6144 x 2048, 12 of 32 experts in use: gate/up 113 us (604 MB, 5.3
// TB/s; 15 experts 6.3), down 79 (3.8: 384 workgroups are one and a half a CU).
// 4 tokens of 7168 x 2048 in FP8, 6 experts: 36 and 20 us (4.9 and 4.3 TB/s).  1
// token of 256 x 128: 5.2 and 3.2 us.  Measured and not kept: down's reduction cut
// into four workgroups a channel block, the last to arrive adding them (74 and
// 22 us; with a release fence each, which writes the L2 back, 210); two of its
// units ahead (the same); four workgroups of 256 threads a CU (the same).
//
// FP8 weights are widened to bf16 (exactly) in registers and the product of
// each 128-block is scaled in float32; activations stay bf16, since nothing
// here is bound by the matrix cores.  h is rounded to bf16 between the kernels,
// for either weights: the matrix instruction's type, half the bytes that every
// workgroup of the second kernel reads, and what the general layer's BF16 recipe
// rounds too (an output's error grows by it from 1.7e-3 of the output, its own
// rounding to bf16, to 2.3e-3 in root mean square).
//
// Against the general layer's launches, whole calls, us (32 of 256 experts, 8 a
// token): 1, 2, 4, 8, 12 and 16 tokens of 6144 x 2048 29, 38, 60, 108-124, 154-185
// and 184-215 against 77, 97, 103, 121-140, 160-165 and 175-180; of 7168 x 2048 in
// FP8 with a shared expert 28, 35, 57, 89, 130 and 175 against 75, 78, 87, 97, 115
// and 137; of 2048 x 768 15, 17, 23, 28, 34 and 39 against 39, 47, 48, 49, 49 and
// 50; 1 token of 256 x 128, 2 of 8 experts, 9.4 against 21.  So the launches are
// saved where few experts are in use; where some ten large ones are, their
// weights bind and the general kernels read them faster.
#include <type_traits>

#include "few.h"
#include "route_row.h"

namespace moe {

namespace {

constexpr int kFewThreads = 512, kWaves = kFewThreads / 64;

struct FewArgs {
  int T, H, I, E, k, e0, L, P, max_rep, has_shared;
  const float* logits;        // routed here (with bias), or null:
  const float* bias;
  const int32_t* ids;         // the routes, [T][k]
  const float* w;
  const int32_t* l2p;
  const int32_t* rep;
  const bf16_t* x;
  moe_weights mw;
  int32_t* counts;            // [E] or null
  FewList* list;
  bf16_t* h;                  // [entries][kFewTokens][I]
  void* out;
  int out_bf16;
};

// Experts in use, in the order of their physical ids (the shared one, id P,
// last), with the tokens that use each.
struct Lds {
  int32_t ids[kFewTokens * MOE_KMAX];
  float w[kFewTokens * MOE_KMAX];
  uint32_t tokens[MOE_EMAX];        // of a local expert: bit t
  uint32_t phys[MOE_LMAX];          // of a physical expert
  int32_t entry[kFewEntries];
  uint32_t mask[kFewEntries];
  int32_t wave_sum[kWaves];
  int32_t n;
};

template <int KPL, bool BIAS>
__device__ __forceinline__ void few_list(const FewArgs& a, Lds& s) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int pairs = a.T * a.k;
  for (int e = tid; e < a.L; e += kFewThreads) s.tokens[e] = 0;
  for (int p = tid; p < a.P; p += kFewThreads) s.phys[p] = 0;
  if constexpr (KPL > 0) {
    if (tid < 256) route_rows_block<KPL, BIAS>(a.logits, a.bias, a.T, a.E, a.k, s.ids, s.w, 0);
  } else if (tid < pairs) {
    s.ids[tid] = a.ids[tid];
    s.w[tid] = a.w[tid];
  }
  __syncthreads();
  const int t = tid / a.k;
  const int id = tid < pairs ? s.ids[tid] : -1;
  int e = id - a.e0;
  if (tid >= pairs || id < 0 || id >= a.E || e < 0 || e >= a.L) e = -1;
  if (e >= 0) atomicOr(&s.tokens[e], 1u << t);
  __syncthreads();
  // the n-th pair of an expert goes to its replica n mod R
  int p = e;
  if (e >= 0 && a.l2p) {
    const int n = __popc(s.tokens[e] & ((1u << t) - 1u));
    p = a.l2p[e * a.max_rep + n % min(max(a.rep[e], 1), a.max_rep)];
    if (p >= a.P) p = -1;
  }
  if (p >= 0) atomicOr(&s.phys[p], 1u << t);
  __syncthreads();
  int base = 0;
  for (int p0 = 0; p0 < a.P; p0 += kFewThreads) {
    const int q = p0 + tid;
    const uint32_t m = q < a.P ? s.phys[q] : 0;
    const uint64_t used = __ballot(m != 0);
    if (lane == 0) s.wave_sum[wv] = __popcll(used);
    __syncthreads();
    int at = base + __popcll(used & ((1ull << lane) - 1ull));
    for (int v = 0; v < kWaves; ++v) {
      if (v < wv) at += s.wave_sum[v];
      base += s.wave_sum[v];
    }
    if (m) {
      s.entry[at] = q;
      s.mask[at] = m;
      s.phys[q] = at;               // (from here on: the entry)
    }
    __syncthreads();
  }
  if (tid == 0) {
    if (a.has_shared) {
      s.entry[base] = a.P;
      s.mask[base] = (1u << a.T) - 1u;
      ++base;
    }
    s.n = base;
  }
  __syncthreads();
  if (blockIdx.x != 0) return;
  // what the second kernel needs
  FewList* o = a.list;
  for (int i = tid; i < s.n; i += kFewThreads) {
    o->entry[i] = s.entry[i];
    o->mask[i] = s.mask[i];
    if (s.entry[i] == a.P)
      for (int j = 0; j < kFewTokens; ++j) o->w[i][j] = 1.0f;
  }
  if (p >= 0) o->w[s.phys[p]][t] = s.w[tid];
  if (tid == 0) o->n = s.n;
  if (a.counts) {
    __syncthreads();
    uint32_t* hist = s.tokens;
    for (int i = tid; i < a.E; i += kFewThreads) hist[i] = 0;
    __syncthreads();
    if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1u);
    __syncthreads();
    for (int i = tid; i < a.E; i += kFewThreads) a.counts[i] = (int)hist[i];
  }
}

__device__ __forceinline__ f32x4_t mfma(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

// Eight E4M3 codes (two words) as bf16
__device__ __forceinline__ u32x4_t widen(uint32_t lo, uint32_t hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  const b2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const b2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const b2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const b2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return u32x4_t{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b),
                 __builtin_bit_cast(uint32_t, c), __builtin_bit_cast(uint32_t, d)};
}

// 128 of the reduction of a 16-channel run: 4 KiB of bf16, or 2 KiB of codes
// and their block's scale
template <bool FP8>
struct Unit {
  u32x4_t v[FP8 ? 2 : 4];
  float scale;
};
// run: the run's first byte; unit: which 128; block: the 128 x 128 block
template <bool FP8>
__device__ __forceinline__ Unit<FP8> load_unit(const void* run, int unit, const float* scales,
                                               int block, int lane) {
  Unit<FP8> r;
  constexpr int N = FP8 ? 2 : 4;
  const u32x4_t* p = (const u32x4_t*)((const char*)run + (size_t)unit * N * 1024) + lane;
#pragma unroll
  for (int i = 0; i < N; ++i) r.v[i] = load_global_nt(p + i * 64);
  r.scale = FP8 ? scales[block] : 1.0f;
  return r;
}

// A token's activations for a unit: lane's token, the reduction values that
// its weights stand at
template <bool FP8>
struct Act {
  u32x4_t v[4];
};
template <bool FP8>
__device__ __forceinline__ Act<FP8> load_act(const bf16_t* row, int unit, int q) {
  Act<FP8> r;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    r.v[s] = *(const u32x4_t*)(row + unit * 128 + (FP8 ? q * 32 + s * 8 : s * 32 + q * 8));
  return r;
}
template <bool FP8>
__device__ __forceinline__ f32x4_t unit_mfma(const Unit<FP8>& w, const Act<FP8>& x, f32x4_t acc) {
  if constexpr (FP8) {
    f32x4_t part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      part = mfma(widen(w.v[s >> 1][2 * (s & 1)], w.v[s >> 1][2 * (s & 1) + 1]), x.v[s], part);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(w.scale, part[i], acc[i]);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) acc = mfma(w.v[s], x.v[s], acc);
  }
  return acc;
}

template <bool FP8, int KPL, bool BIAS>
__global__ __launch_bounds__(kFewThreads, 2) void k_few_gate_up(FewArgs a) {
  __shared__ Lds s;
  __shared__ f32x4_t part[2][kWaves][2][64];
  few_list<KPL, BIAS>(a, s);
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int groups = a.I / 16, units = a.H / 128;
  const int total = s.n * groups;
  const int u0 = wv * units / kWaves, u1 = (wv + 1) * units / kWaves;
  const bf16_t* row = a.x + (size_t)min(c16, a.T - 1) * a.H;
  const size_t run_bytes = (size_t)a.H * 16 * (FP8 ? 1 : 2);
  struct Ptrs {
    const void* g;
    const void* u;
    const float* sg;
    const float* su;
  };
  auto pointers = [&](int item) -> Ptrs {
    const int p = __builtin_amdgcn_readfirstlane(s.entry[item / groups]), n = item % groups;
    const bool sh = p == a.P;
    Ptrs r;
    r.g = (const char*)(sh ? a.mw.sh_gate : a.mw.w_gate[p]) + n * run_bytes;
    r.u = (const char*)(sh ? a.mw.sh_up : a.mw.w_up[p]) + n * run_bytes;
    r.sg = r.su = nullptr;
    if constexpr (FP8) {
      r.sg = (sh ? a.mw.sh_s_gate : a.mw.s_gate[p]) + (size_t)(n / 8) * units;
      r.su = (sh ? a.mw.sh_s_up : a.mw.s_up[p]) + (size_t)(n / 8) * units;
    }
    return r;
  };
  Unit<FP8> g, u;
  Act<FP8> x;
  auto load = [&](const Ptrs& r, int unit) {
    g = load_unit<FP8>(r.g, unit, r.sg, unit, lane);
    u = load_unit<FP8>(r.u, unit, r.su, unit, lane);
    x = load_act<FP8>(row, unit, q);
  };
  int turn = 0;
  if ((int)blockIdx.x < total && u0 < u1) load(pointers(blockIdx.x), u0);
  for (int item = blockIdx.x; item < total; item += gridDim.x, turn ^= 1) {
    f32x4_t ag = {0.f, 0.f, 0.f, 0.f}, au = ag;
    if (u0 < u1) {
      const Ptrs r = pointers(item);
      for (int unit = u0; unit < u1; ++unit) {
        const Unit<FP8> gc = g, uc = u;
        const Act<FP8> xc = x;
        // the next unit, or the next item's first, in flight meanwhile
        if (unit + 1 < u1) load(r, unit + 1);
        else if (item + (int)gridDim.x < total) load(pointers(item + gridDim.x), u0);
        ag = unit_mfma<FP8>(gc, xc, ag);
        au = unit_mfma<FP8>(uc, xc, au);
      }
    }
    part[turn][wv][0][lane] = ag;
    part[turn][wv][1][lane] = au;
    __syncthreads();                       // (two buffers: one barrier an item)
    if (wv == (item & (kWaves - 1))) {     // one wavefront joins and stores
      f32x4_t sg = part[turn][0][0][lane], su = part[turn][0][1][lane];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) {
        sg += part[turn][v][0][lane];
        su += part[turn][v][1][lane];
      }
      const int e = item / groups, n = item - e * groups;
      if ((s.mask[e] >> c16) & 1) {        // channels 4 q .. of token c16
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          o[i] = (uint32_t)f32_to_bf16(silu_f32(sg[2 * i]) * su[2 * i]) |
                 (uint32_t)f32_to_bf16(silu_f32(sg[2 * i + 1]) * su[2 * i + 1]) << 16;
        *(uint2*)(a.h + ((size_t)e * kFewTokens + c16) * a.I + n * 16 + 4 * q) =
            make_uint2(o[0], o[1]);
      }
    }
  }
}

template <bool FP8>
__global__ __launch_bounds__(kFewThreads, 2) void k_few_down(FewArgs a) {
  __shared__ f32x4_t part[kWaves][64];
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c16 = lane & 15, q = lane >> 4;
  const int n = blockIdx.x, per = a.I / 128;           // 16 channels; units an expert
  const FewList* list = a.list;
  const int units = list->n * per;
  const int u0 = (int)((long)wv * units / kWaves), u1 = (int)((long)(wv + 1) * units / kWaves);
  const size_t run = (size_t)n * a.I * 16 * (FP8 ? 1 : 2);
  f32x4_t sum = {0.f, 0.f, 0.f, 0.f};
  Unit<FP8> w;
  Act<FP8> h;
  float wt = 0.0f;
  bool mine = false;
  auto load = [&](int unit) {
    const int e = unit / per, kb = unit - e * per;
    const int p = __builtin_amdgcn_readfirstlane(list->entry[e]);
    const bool sh = p == a.P;
    const float* sc = nullptr;
    if constexpr (FP8) sc = (sh ? a.mw.sh_s_down : a.mw.s_down[p]) + (size_t)(n / 8) * per;
    w = load_unit<FP8>((const char*)(sh ? a.mw.sh_down : a.mw.w_down[p]) + run, kb, sc, kb, lane);
    h = load_act<FP8>(a.h + ((size_t)e * kFewTokens + min(c16, a.T - 1)) * a.I, kb, q);
    mine = (list->mask[e] >> c16) & 1;
    wt = list->w[e][c16];
  };
  if (u0 < u1) load(u0);
  for (int unit = u0; unit < u1; ++unit) {
    const Unit<FP8> wc = w;
    const Act<FP8> hc = h;
    const float wtc = wt;
    const bool minec = mine;
    if (unit + 1 < u1) load(unit + 1);
    const f32x4_t y = unit_mfma<FP8>(wc, hc, f32x4_t{0.f, 0.f, 0.f, 0.f});
    // (other tokens' columns hold what the workspace held)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] = minec ? __builtin_fmaf(wtc, y[i], sum[i]) : sum[i];
  }
  part[wv][lane] = sum;
  __syncthreads();
  if (wv != 0) return;
#pragma unroll
  for (int v = 1; v < kWaves; ++v) sum += part[v][lane];
  if (c16 >= a.T) return;
  const size_t at = (size_t)c16 * a.H + n * 16 + 4 * q;
  if (a.out_bf16) {
    *(uint2*)((bf16_t*)a.out + at) =
        make_uint2((uint32_t)f32_to_bf16(sum[0]) | (uint32_t)f32_to_bf16(sum[1]) << 16,
                   (uint32_t)f32_to_bf16(sum[2]) | (uint32_t)f32_to_bf16(sum[3]) << 16);
  } else {
    *(f32x4_t*)((float*)a.out + at) = sum;
  }
}

template <bool FP8>
hipError_t launch(const FewArgs& a, int entries, hipStream_t s) {
  const long items = (long)entries * (a.I / 16);
  const unsigned grid = (unsigned)(items < 512 ? items : 512);   // two a CU
#define GATE_UP(KPL, BIAS) k_few_gate_up<FP8, KPL, BIAS><<<grid, kFewThreads, 0, s>>>(a)
  if (!a.logits) GATE_UP(0, false);
  else if (a.E <= 64) { if (a.bias) GATE_UP(4, true); else GATE_UP(4, false); }
  else { if (a.bias) GATE_UP(16, true); else GATE_UP(16, false); }
#undef GATE_UP
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_few_down<FP8><<<a.H / 16, kFewThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int few_entries(const moe_problem* p) {
  const long pairs = (long)kFewTokens * p->k;
  return (int)(pairs < p->num_physical ? pairs : p->num_physical) + p->has_shared;
}

hipError_t launch_few(const moe_problem* p, const FewCall& c, hipStream_t s) {
  FewArgs a{};
  a.T = p->T;
  a.H = p->H;
  a.I = p->I;
  a.E = p->E;
  a.k = p->k;
  a.e0 = p->expert_begin;
  a.L = p->num_local;
  a.P = p->num_physical;
  a.max_rep = p->max_replicas;
  a.has_shared = p->has_shared;
  a.logits = c.logits;
  a.bias = c.bias;
  a.ids = c.ids;
  a.w = c.w;
  a.l2p = c.l2p;
  a.rep = c.rep;
  a.x = c.x;
  a.mw = *c.weights;
  a.counts = c.counts;
  a.list = c.list;
  a.h = c.h;
  a.out = c.out;
  a.out_bf16 = p->out_dtype == MOE_BF16;
  const long pairs = (long)p->T * p->k;
  const int entries = (int)(pairs < p->num_physical ? pairs : p->num_physical) + p->has_shared;
  return p->weight_dtype == MOE_FP8_E4M3 ? launch<true>(a, entries, s) : launch<false>(a, entries, s);
}

}  // namespace moe
