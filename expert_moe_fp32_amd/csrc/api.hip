// C ABI of the MoE layer: argument validation, workspace layout and the
// launch sequence of each step.  No allocation, no synchronisation.
#include <algorithm>
#include <cmath>
#include <numeric>
#include <vector>

#include "block.h"
#include "common.h"
#include "few.h"
#include "train.h"

using namespace moe;

namespace {

struct Carver {  // hands out 256-byte aligned pieces of a workspace
  char* base;
  size_t used = 0;
  explicit Carver(void* b) : base((char*)b) {}
  template <class T>
  T* take(size_t count) {
    T* p = base ? (T*)(base + used) : nullptr;
    used += moe_align256(count * sizeof(T));
    return p;
  }
};

inline size_t dtype_bytes(int d) {
  return d == MOE_F32 ? 4 : (d == MOE_BF16 ? 2 : 1);
}

inline long cap_rows(const moe_problem* p) {
  return (long)p->T * std::min(p->k, p->num_local);
}

inline hipStream_t S(void* s) { return (hipStream_t)s; }

inline moe_status hip_status(hipError_t e) {
  return e == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// scratch of the dispatch step (also used by the layer)
struct DispatchScratch {
  int32_t* block_counts;
  int32_t* block_base;
  int32_t* block_ecounts;  // [nblk][E] partial expert counts
  uint8_t* xq;     // fp8: [T][H] codes of every token
  float* xs;       // fp8: [T][H/128]
};

DispatchScratch carve_dispatch(Carver& c, const moe_problem* p) {
  DispatchScratch d{};
  const size_t nb = (size_t)dispatch_blocks(p->T) * p->num_local;
  d.block_counts = c.take<int32_t>(nb);
  d.block_base = c.take<int32_t>(nb);
  d.block_ecounts = c.take<int32_t>((size_t)dispatch_blocks(p->T) * p->E);
  if (p->weight_dtype == MOE_FP8_E4M3) {
    d.xq = c.take<uint8_t>((size_t)p->T * p->H);
    d.xs = c.take<float>((size_t)p->T * (p->H / 128));
  }
  return d;
}

// Expected rows per physical expert: the local pairs over the physical
// experts, where a rank with fewer physical than logical experts (a
// group-wide placement whose other replicas sit on other ranks) expects
// about one logical expert's pairs per physical expert.
int rows_hint(const moe_problem* p) {
  const double pairs = (double)p->T * p->k * p->num_local / p->E;
  return (int)(pairs / std::max(p->num_physical, p->num_local) + 0.5);
}

struct FfnScratch {
  void* h;
  float* h_scales;
  float* h32;
  int4* tiles;
  int4* tiles_down;
  int32_t* tile_count;
  int max_tiles;
};

FfnScratch carve_ffn(Carver& c, const moe_problem* p) {
  FfnScratch f{};
  const long cap = cap_rows(p);
  const size_t hrows = (size_t)cap + (p->has_shared ? p->T : 0);
  const size_t hb = p->act_dtype == MOE_F32 ? 4
                    : (p->weight_dtype == MOE_FP8_E4M3 ? 1 : 2);
  f.h = c.take<char>(hrows * p->I * hb);
  if (p->weight_dtype == MOE_FP8_E4M3) {
    f.h_scales = c.take<float>(hrows * (p->I / 128));
    // float32 h only for the kernels that leave quantisation to a pass of
    // its own (the 32-row register-streaming kernel quantises in place)
    int balanced;
    if (ffn_fp8_tile_rows(rows_hint(p), p->H, p->I, &balanced) != 32)
      f.h32 = c.take<float>(hrows * p->I);
  }
  // descriptors: at most one per 16 rows plus one per group, and the four
  // quarters of a tall tile (groups of more than 32 rows) at most one per 8
  // rows of their group
  f.max_tiles = (int)(p->num_physical + 2 + (hrows + 15) / 16 + (hrows + 7) / 8);
  f.tiles = c.take<int4>((size_t)f.max_tiles);
  // 128-row tiles (or the FP8 streaming down pass's tiles: one per group of
  // up to 32 rows, tall tiles of up to 128 beyond): at most one partial tile
  // per group
  f.tiles_down = c.take<int4>((size_t)p->num_physical + 2 + hrows / 128);
  f.tile_count = c.take<int32_t>(4);
  return f;
}

moe_status launch_ffn_common(const moe_problem* p, const void* x_perm,
                             const float* x_perm_scales,
                             const int32_t* offsets, const void* x_shared,
                             const float* x_shared_scales,
                             const moe_weights* w, float* y_perm,
                             float* y_shared, const FfnScratch& fs,
                             hipStream_t s, hipEvent_t* events = nullptr,
                             const int32_t* a_rows = nullptr,
                             bool tiles_ready = false) {
  FfnArgs a{};
  a.a_rows = a_rows;
  a.tiles_ready = tiles_ready;
  a.H = p->H;
  a.I = p->I;
  a.P = p->num_physical;
  a.T = p->T;
  a.cap = (int)cap_rows(p);
  a.has_shared = p->has_shared;
  a.rows_hint = rows_hint(p);
  a.act = p->act_dtype;
  a.wdt = p->weight_dtype;
  a.offsets = offsets;
  a.a_routed = x_perm;
  a.a_routed_scales = x_perm_scales;
  a.a_shared = x_shared;
  a.a_shared_scales = x_shared_scales;
  a.w = w;
  a.h = fs.h;
  a.h_scales = fs.h_scales;
  a.h32 = fs.h32;
  a.y_routed = y_perm;
  a.y_shared = y_shared;
  a.tiles = fs.tiles;
  a.tiles_down = fs.tiles_down;
  a.tile_count = fs.tile_count;
  a.max_tiles = fs.max_tiles;
  a.events = events;
  return hip_status(launch_ffn(a, s));
}

moe_status check_weights(const moe_problem* p, const moe_weights* w) {
  if (!w || !w->w_gate || !w->w_up || !w->w_down)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->weight_dtype == MOE_FP8_E4M3 && (!w->s_gate || !w->s_up || !w->s_down))
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->has_shared) {
    if (!w->sh_gate || !w->sh_up || !w->sh_down) return MOE_ERR_INVALID_ARGUMENT;
    if (p->weight_dtype == MOE_FP8_E4M3 &&
        (!w->sh_s_gate || !w->sh_s_up || !w->sh_s_down))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

moe_status dispatch_impl(const moe_problem* p, const void* x,
                         const int32_t* ids, const float* tw,
                         const int32_t* l2p, const int32_t* rep,
                         void* x_perm, float* x_perm_scales, int32_t* offsets,
                         int32_t* row_token, float* row_weight,
                         int32_t* pair_row, const DispatchScratch& d,
                         hipStream_t s, hipEvent_t ev_index = nullptr,
                         bool materialize = true,
                         const DispatchExtras* extras = nullptr,
                         bool x_quantised = false) {
  DispatchArgs a{};
  a.T = p->T;
  a.k = p->k;
  a.expert_begin = p->expert_begin;
  a.num_local = p->num_local;
  a.P = p->num_physical;
  a.max_rep = l2p ? p->max_replicas : 1;
  a.H = p->H;
  a.ids = ids;
  a.w = tw;
  a.l2p = l2p;
  a.rep = rep;
  a.block_counts = d.block_counts;
  a.block_base = d.block_base;
  a.block_ecounts = d.block_ecounts;
  a.offsets = offsets;
  a.row_token = row_token;
  a.row_weight = row_weight;
  a.pair_row = pair_row;
  hipError_t e;
  DispatchExtras xt{};
  xt.E = p->E;
  if (extras) xt = *extras;
  if (dispatch_small_ok(p->T, p->E, p->num_local, p->num_physical))
    e = launch_dispatch_small(a, xt, s);
  else
    e = launch_dispatch_index(a, xt, s);
  if (e != hipSuccess) return MOE_ERR_HIP;
  if (ev_index) hipEventRecord(ev_index, s);
  const int cap = (int)cap_rows(p);
  const int32_t* nrows = offsets + p->num_physical;
  if (p->weight_dtype == MOE_FP8_E4M3) {
    if (!x_quantised)     // else done with the router (launch_route_quant_fp8)
      e = launch_quant_rows_fp8((const bf16_t*)x, p->T, p->H, d.xq, d.xs, s);
    if (e != hipSuccess || !materialize) return hip_status(e);
    e = launch_gather_rows(d.xq, (size_t)p->H, row_token, nrows, cap, x_perm, s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    // scales: H/128 floats per row, gathered 4 bytes at a time
    e = launch_gather_rows_words(d.xs, p->H / 128, row_token, nrows, cap,
                                 x_perm_scales, s);
    return hip_status(e);
  }
  if (!materialize) return MOE_OK;
  e = launch_gather_rows(x, (size_t)p->H * dtype_bytes(p->act_dtype),
                         row_token, nrows, cap, x_perm, s);
  return hip_status(e);
}

}  // namespace

extern "C" {

const char* moe_status_string(moe_status s) {
  switch (s) {
    case MOE_OK: return "ok";
    case MOE_ERR_INVALID_ARGUMENT: return "invalid argument";
    case MOE_ERR_UNSUPPORTED: return "unsupported dtype or shape";
    case MOE_ERR_WORKSPACE: return "workspace too small";
    case MOE_ERR_HIP: return "HIP launch failed";
  }
  return "unknown status";
}

moe_status moe_check_problem(const moe_problem* p) {
  if (!p) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T < 0 || p->H <= 0 || p->I <= 0 || p->E <= 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->k < 1 || p->k > p->E) return MOE_ERR_INVALID_ARGUMENT;
  if (p->expert_begin < 0 || p->num_local < 1 ||
      (long)p->expert_begin + p->num_local > p->E)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->num_physical < 1 || p->max_replicas < 1)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->has_shared != 0 && p->has_shared != 1) return MOE_ERR_INVALID_ARGUMENT;
  const int a = p->act_dtype, w = p->weight_dtype, o = p->out_dtype;
  if (a < 0 || a > 2 || w < 0 || w > 2 || o < 0 || o > 2) return MOE_ERR_INVALID_ARGUMENT;
  if (p->k > MOE_KMAX || p->E > MOE_EMAX || p->num_physical > MOE_LMAX)
    return MOE_ERR_UNSUPPORTED;
  if (o == MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  if (a == MOE_F32 && w == MOE_F32) {
    if (p->H % 4) return MOE_ERR_UNSUPPORTED;
  } else if (a == MOE_BF16 && w == MOE_BF16) {
    if (p->H % 128 || p->I % 128) return MOE_ERR_UNSUPPORTED;
  } else if (a == MOE_BF16 && w == MOE_FP8_E4M3) {
    // reductions of at most 128 scale blocks (the kernels keep a tile's
    // weight-scale column in LDS)
    if (p->quant_block != 128 || p->H % 128 || p->I % 128 || p->H > 16384 ||
        p->I > 16384)
      return MOE_ERR_UNSUPPORTED;
  } else {
    return MOE_ERR_UNSUPPORTED;
  }
  // row indices are 32-bit
  if ((double)p->T * p->k >= 2147483647.0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status moe_dispatch_workspace_size(const moe_problem* p, size_t* bytes) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  Carver c(nullptr);
  carve_dispatch(c, p);
  *bytes = c.used;
  return MOE_OK;
}

moe_status moe_ffn_workspace_size(const moe_problem* p, size_t* bytes) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  Carver c(nullptr);
  carve_ffn(c, p);
  *bytes = c.used;
  return MOE_OK;
}

namespace {
struct LayerScratch {
  int32_t* ids;
  float* tw;
  int32_t* counts;
  int32_t* offsets;
  int32_t* row_token;
  float* row_weight;
  int32_t* pair_row;
  void* x_perm;
  float* x_perm_scales;
  float* y_perm;
  float* y_shared;
  DispatchScratch d;
  FfnScratch f;
};

LayerScratch carve_layer(Carver& c, const moe_problem* p) {
  LayerScratch L{};
  const size_t Tk = (size_t)p->T * p->k;
  const size_t cap = (size_t)cap_rows(p);
  L.ids = c.take<int32_t>(Tk);
  L.tw = c.take<float>(Tk);
  L.counts = c.take<int32_t>((size_t)p->E);
  L.offsets = c.take<int32_t>((size_t)p->num_physical + 1);
  L.row_token = c.take<int32_t>(cap);
  L.row_weight = c.take<float>(cap);
  L.pair_row = c.take<int32_t>(Tk);
  // no permuted activation copy: the expert kernels gather rows themselves
  L.y_perm = c.take<float>(cap * p->H);
  if (p->has_shared) L.y_shared = c.take<float>((size_t)p->T * p->H);
  L.d = carve_dispatch(c, p);
  L.f = carve_ffn(c, p);
  return L;
}
}  // namespace

moe_status moe_layer_workspace_size(const moe_problem* p, size_t* bytes) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  Carver c(nullptr);
  carve_layer(c, p);
  *bytes = c.used;
  return MOE_OK;
}

moe_status moe_workspace_size(const moe_problem* p, size_t* bytes) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  size_t d = 0, f = 0, l = 0;
  moe_dispatch_workspace_size(p, &d);
  moe_ffn_workspace_size(p, &f);
  moe_layer_workspace_size(p, &l);
  *bytes = std::max(d, std::max(f, l));
  return MOE_OK;
}

moe_status moe_ffn_intermediate(const moe_problem* p, void* workspace,
                                size_t ws_bytes, void** h, float** h_scales) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (!h || !h_scales) return MOE_ERR_INVALID_ARGUMENT;
  size_t need;
  moe_ffn_workspace_size(p, &need);
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  Carver c(workspace);
  FfnScratch fs = carve_ffn(c, p);
  *h = fs.h;
  *h_scales = p->weight_dtype == MOE_FP8_E4M3 ? fs.h_scales : nullptr;
  return MOE_OK;
}

moe_status moe_route_topk(const moe_problem* p, const float* logits,
                          const float* bias, int32_t* topk_ids, float* topk_w,
                          int32_t* expert_counts, void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) {
    if (expert_counts)
      return hip_status(launch_fill_i32(expert_counts, 0, (size_t)p->E, S(stream)));
    return MOE_OK;
  }
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_route_topk(logits, bias, p->T, p->E, p->k, topk_ids,
                                      topk_w, expert_counts, S(stream)));
}

// 16-byte vector loads and stores touch the row arrays
static inline bool al16(const void* q) { return ((uintptr_t)q & 15) == 0; }

static moe_status check_map(const moe_problem* p, const int32_t* l2p,
                            const int32_t* rep) {
  if (!l2p) {
    if (rep || p->num_physical != p->num_local) return MOE_ERR_INVALID_ARGUMENT;
  } else if (!rep) {
    return MOE_ERR_INVALID_ARGUMENT;
  }
  return MOE_OK;
}

moe_status moe_dispatch(const moe_problem* p, const void* x,
                        const int32_t* topk_ids, const float* topk_w,
                        const int32_t* l2p, const int32_t* replica_count,
                        void* x_perm, float* x_perm_scales, int32_t* offsets,
                        int32_t* row_token, float* row_weight,
                        int32_t* pair_row, void* workspace, size_t ws_bytes,
                        void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if ((st = check_map(p, l2p, replica_count)) != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!x || !topk_ids || !topk_w || !x_perm || !offsets || !row_token ||
      !row_weight || !pair_row)
    return MOE_ERR_INVALID_ARGUMENT;
  if (p->weight_dtype == MOE_FP8_E4M3 && !x_perm_scales) return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(x) || !al16(x_perm)) return MOE_ERR_INVALID_ARGUMENT;
  size_t need;
  moe_dispatch_workspace_size(p, &need);
  if (need && (!workspace || ws_bytes < need)) return MOE_ERR_WORKSPACE;
  Carver c(workspace);
  DispatchScratch d = carve_dispatch(c, p);
  return dispatch_impl(p, x, topk_ids, topk_w, l2p, replica_count, x_perm,
                       x_perm_scales, offsets, row_token, row_weight, pair_row,
                       d, S(stream));
}

moe_status moe_grouped_ffn(const moe_problem* p, const void* x_perm,
                           const float* x_perm_scales, const int32_t* offsets,
                           const void* x_shared, const float* x_shared_scales,
                           const moe_weights* w, float* y_perm,
                           float* y_shared, void* workspace, size_t ws_bytes,
                           void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if ((st = check_weights(p, w)) != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!x_perm || !offsets || !y_perm) return MOE_ERR_INVALID_ARGUMENT;
  const bool fp8 = p->weight_dtype == MOE_FP8_E4M3;
  if (fp8 && !x_perm_scales) return MOE_ERR_INVALID_ARGUMENT;
  if (p->has_shared && (!x_shared || !y_shared || (fp8 && !x_shared_scales)))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(x_perm) || !al16(x_shared) || !al16(y_perm) || !al16(y_shared))
    return MOE_ERR_INVALID_ARGUMENT;
  size_t need;
  moe_ffn_workspace_size(p, &need);
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  Carver c(workspace);
  FfnScratch fs = carve_ffn(c, p);
  return launch_ffn_common(p, x_perm, x_perm_scales, offsets, x_shared,
                           x_shared_scales, w, y_perm, y_shared, fs, S(stream));
}

moe_status moe_combine(const moe_problem* p, const float* y_perm,
                       const int32_t* pair_row, const float* topk_w,
                       const float* y_shared, void* out, void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!y_perm || !pair_row || !topk_w || !out) return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(y_perm) || !al16(y_shared) || !al16(out)) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_combine(y_perm, pair_row, topk_w, y_shared, p->T,
                                   p->H, p->k, p->out_dtype, out, S(stream)));
}

// What the scored layer has in place of the router and the combine.
struct ScoredLayer {
  const moe_router* r;
  const moe_norm* n;      // or null: the combine ends the layer
  NormArgs norm;
};

static moe_status layer_impl(const moe_problem* p, const void* logits,
                             const float* bias, const void* x,
                             const moe_weights* w, const int32_t* l2p,
                             const int32_t* replica_count, void* out,
                             int32_t* expert_counts, void* workspace,
                             size_t ws_bytes, void* stream, hipEvent_t* ev,
                             const ScoredLayer* scored = nullptr) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  const moe_norm* n = scored ? scored->n : nullptr;
  if ((st = check_map(p, l2p, replica_count)) != MOE_OK) return st;
  if ((st = check_weights(p, w)) != MOE_OK) return st;
  hipStream_t s = S(stream);
  if (p->T == 0) {
    if (expert_counts)
      return hip_status(launch_fill_i32(expert_counts, 0, (size_t)p->E, s));
    return MOE_OK;
  }
  if (!logits || !x || (!n && !out)) return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(x) || (!n && !al16(out))) return MOE_ERR_INVALID_ARGUMENT;
  size_t need;
  moe_layer_workspace_size(p, &need);
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  Carver c(workspace);
  LayerScratch L = carve_layer(c, p);
  if (ev) hipEventRecord(ev[0], s);
  int32_t* counts = expert_counts ? expert_counts : L.counts;
  // The dispatch's single-workgroup stage counts the experts and writes the
  // FFN tile list, so neither needs a launch of its own.
  DispatchExtras extras{};
  extras.E = p->E;
  extras.counts = counts;
  extras.tiles = L.f.tiles;
  extras.tile_count = L.f.tile_count;
  extras.BM = ffn_tile_rows(p->act_dtype, p->weight_dtype, rows_hint(p),
                            p->H, p->I, &extras.balanced);
  extras.tallBM = ffn_tall_rows(p->act_dtype, p->weight_dtype, extras.BM);
  extras.tallBM2 = ffn_down_tall_rows(p->weight_dtype, extras.BM);
  if (extras.tallBM2) {           // the down pass's own list
    extras.tiles2 = L.f.tiles_down;
    extras.count2 = L.f.tile_count + 1;
  }
  extras.has_shared = p->has_shared;
  // FP8 recipe: the router and the activation quantiser share one launch
  // (the quantiser reads only x), so the router's latency hides under the
  // quantiser's stream; the route stage then holds both.
  const bool fp8_q =
      !scored && p->weight_dtype == MOE_FP8_E4M3 && p->E <= 256;
  const float* lf = (const float*)logits;
  const hipError_t re =
      scored ? launch_route_scored(scored->r, logits, bias, L.ids, L.tw,
                                   nullptr, nullptr, s)
      : fp8_q ? launch_route_quant_fp8(lf, bias, p->T, p->E, p->k, L.ids,
                                       L.tw, (const bf16_t*)x, p->H, L.d.xq,
                                       L.d.xs, s)
              : launch_route_topk(lf, bias, p->T, p->E, p->k, L.ids, L.tw,
                                  nullptr, s);
  if (re != hipSuccess) return MOE_ERR_HIP;
  if (ev) hipEventRecord(ev[1], s);
  st = dispatch_impl(p, x, L.ids, L.tw, l2p, replica_count, L.x_perm,
                     L.x_perm_scales, L.offsets, L.row_token, L.row_weight,
                     L.pair_row, L.d, s, ev ? ev[2] : nullptr,
                     /*materialize=*/false, &extras, /*x_quantised=*/fp8_q);
  if (st != MOE_OK) return st;
  if (ev) hipEventRecord(ev[3], s);
  // The expert kernels read each routed row straight from the token rows
  // through row_token (the permuted copy is never written); the shared
  // expert reads the same token rows in order.
  const bool fp8 = p->weight_dtype == MOE_FP8_E4M3;
  const void* xs = fp8 ? (const void*)L.d.xq : x;
  st = launch_ffn_common(p, xs, fp8 ? L.d.xs : nullptr, L.offsets,
                         p->has_shared ? xs : nullptr,
                         p->has_shared && fp8 ? L.d.xs : nullptr, w, L.y_perm,
                         L.y_shared, L.f, s, ev ? ev + 4 : nullptr,
                         L.row_token, /*tiles_ready=*/true);
  if (st != MOE_OK) return st;
  const float* ysh = p->has_shared ? L.y_shared : nullptr;
  if (n) {
    const CombineSource c{L.y_perm, L.pair_row, L.tw, ysh, p->k,
                          (int)cap_rows(p), out};
    st = hip_status(launch_residual_norm(n, scored->norm, &c, s));
  } else {
    st = hip_status(launch_combine(L.y_perm, L.pair_row, L.tw, ysh, p->T,
                                   p->H, p->k, p->out_dtype, out, s));
  }
  if (ev) hipEventRecord(ev[7], s);
  return st;
}

moe_status moe_layer_forward(const moe_problem* p, const float* logits,
                             const float* bias, const void* x,
                             const moe_weights* w, const int32_t* l2p,
                             const int32_t* replica_count, void* out,
                             int32_t* expert_counts, void* workspace,
                             size_t ws_bytes, void* stream) {
  return layer_impl(p, logits, bias, x, w, l2p, replica_count, out,
                    expert_counts, workspace, ws_bytes, stream, nullptr);
}

moe_status moe_layer_forward_timed(const moe_problem* p, const float* logits,
                                   const float* bias, const void* x,
                                   const moe_weights* w, const int32_t* l2p,
                                   const int32_t* replica_count, void* out,
                                   int32_t* expert_counts, void* workspace,
                                   size_t ws_bytes, void* stream,
                                   void* const* events) {
  if (!events) return MOE_ERR_INVALID_ARGUMENT;
  hipEvent_t ev[MOE_STAGE_EVENTS];
  for (int i = 0; i < MOE_STAGE_EVENTS; ++i) {
    if (!events[i]) return MOE_ERR_INVALID_ARGUMENT;
    ev[i] = (hipEvent_t)events[i];
  }
  return layer_impl(p, logits, bias, x, w, l2p, replica_count, out,
                    expert_counts, workspace, ws_bytes, stream, ev);
}

// ------------------------------------------------------- scored routing
moe_status moe_check_router(const moe_router* r) {
  if (!r) return MOE_ERR_INVALID_ARGUMENT;
  if (r->T < 0 || r->E < 1 || r->k < 1 || r->k > r->E)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->groups < 1 || r->E % r->groups || r->topk_groups < 1 ||
      r->topk_groups > r->groups || (r->group_top != 1 && r->group_top != 2))
    return MOE_ERR_INVALID_ARGUMENT;
  if ((long)r->topk_groups * (r->E / r->groups) < r->k)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->renormalize != 0 && r->renormalize != 1) return MOE_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(r->scale) || r->logits_stride < r->E)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->logits_dtype < MOE_F32 || r->logits_dtype > MOE_FP8_E4M3)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->logits_dtype == MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  if (r->k > MOE_KMAX || r->E > MOE_EMAX || r->groups > 64)
    return MOE_ERR_UNSUPPORTED;
  if ((double)r->T * r->k >= 2147483647.0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status moe_route_scored_workspace_size(const moe_router* r, size_t* bytes) {
  const moe_status st = moe_check_router(r);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = route_scored_scratch(r) * sizeof(int32_t);
  return MOE_OK;
}

moe_status moe_route_scored(const moe_router* r, const void* logits,
                            const float* bias, int32_t* topk_ids,
                            float* topk_w, int32_t* expert_counts,
                            void* workspace, size_t ws_bytes, void* stream) {
  const moe_status st = moe_check_router(r);
  if (st != MOE_OK) return st;
  if (r->T == 0) {
    if (expert_counts)
      return hip_status(launch_fill_i32(expert_counts, 0, (size_t)r->E, S(stream)));
    return MOE_OK;
  }
  if (!logits || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = route_scored_partials(r) * sizeof(int32_t);
  if (expert_counts && need && (!workspace || ws_bytes < need))
    return MOE_ERR_WORKSPACE;
  return hip_status(launch_route_scored(r, logits, bias, topk_ids, topk_w,
                                        expert_counts, (int32_t*)workspace,
                                        S(stream)));
}

moe_status moe_route_scored_backward(const moe_router* r, const void* logits,
                                     const int32_t* topk_ids,
                                     const float* d_topk_w, void* d_logits,
                                     void* stream) {
  const moe_status st = moe_check_router(r);
  if (st != MOE_OK) return st;
  if (r->T == 0) return MOE_OK;
  if (!logits || !topk_ids || !d_topk_w || !d_logits || d_logits == logits)
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_route_scored_backward(r, logits, topk_ids, d_topk_w,
                                                 d_logits, S(stream)));
}

// -------------------------------------------------------- residual norm
moe_status moe_check_norm(const moe_norm* n) {
  if (!n) return MOE_ERR_INVALID_ARGUMENT;
  if (n->T < 0 || n->H < 1) return MOE_ERR_INVALID_ARGUMENT;
  for (int d : {n->block_dtype, n->resid_dtype, n->out_dtype, n->gain_dtype})
    if (d < MOE_F32 || d > MOE_FP8_E4M3) return MOE_ERR_INVALID_ARGUMENT;
  if (!std::isfinite(n->eps) || n->eps < 0.0f ||
      !std::isfinite(n->gain_offset) || !std::isfinite(n->residual_scale))
    return MOE_ERR_INVALID_ARGUMENT;
  for (int64_t s : {n->block_stride, n->resid_stride, n->resid_out_stride,
                    n->out_stride})
    if (s < n->H) return MOE_ERR_INVALID_ARGUMENT;
  for (int d : {n->block_dtype, n->resid_dtype, n->out_dtype, n->gain_dtype})
    if (d == MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  if (n->H > 16384) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

static bool gate_shape_ok(const moe_norm* n) {
  return (n->gate_rows == 1 || n->gate_rows == n->T) &&
         (n->gate_cols == 1 || n->gate_cols == n->H);
}

// the operands that a forward call needs besides its block
static moe_status check_norm_forward(const moe_norm* n, const NormArgs& a) {
  if (!a.resid || (!a.resid_out && !a.x_out)) return MOE_ERR_INVALID_ARGUMENT;
  if ((a.pre_gain != nullptr) != (a.x_out != nullptr))
    return MOE_ERR_INVALID_ARGUMENT;
  if (a.gate && !gate_shape_ok(n)) return MOE_ERR_INVALID_ARGUMENT;
  // in place: the same rows
  if (a.resid_out == a.resid && n->resid_out_stride != n->resid_stride)
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status moe_residual_norm(const moe_norm* n, const void* y,
                             const void* resid, const void* post_gain,
                             const float* gate, const void* pre_gain,
                             void* resid_out, void* x_out, void* stream) {
  moe_status st = moe_check_norm(n);
  if (st != MOE_OK) return st;
  if (n->T == 0) return MOE_OK;
  const NormArgs a{y, resid, post_gain, gate, pre_gain, resid_out, x_out};
  if (!y && (post_gain || gate)) return MOE_ERR_INVALID_ARGUMENT;
  if ((st = check_norm_forward(n, a)) != MOE_OK) return st;
  return hip_status(launch_residual_norm(n, a, nullptr, S(stream)));
}

moe_status moe_residual_norm_workspace_size(const moe_norm* n, size_t* bytes) {
  const moe_status st = moe_check_norm(n);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = norm_grad_scratch(n) * sizeof(float);
  return MOE_OK;
}

moe_status moe_residual_norm_backward(
    const moe_norm* n, const void* y, const void* resid_out,
    const void* post_gain, const float* gate, const void* pre_gain,
    const void* d_x, const void* d_resid_out, void* d_y, void* d_resid,
    float* d_post_gain, float* d_gate, float* d_pre_gain, void* workspace,
    size_t ws_bytes, void* stream) {
  const moe_status st = moe_check_norm(n);
  if (st != MOE_OK) return st;
  if ((d_post_gain && !post_gain) || (d_gate && !gate) ||
      (d_pre_gain && !pre_gain))
    return MOE_ERR_INVALID_ARGUMENT;
  // (a batch of no rows may come without its row arrays)
  if (n->T > 0) {
    if (!y && (post_gain || gate)) return MOE_ERR_INVALID_ARGUMENT;
    if ((pre_gain != nullptr) != (d_x != nullptr)) return MOE_ERR_INVALID_ARGUMENT;
    if (pre_gain ? !resid_out : !d_resid_out) return MOE_ERR_INVALID_ARGUMENT;
    if (d_resid && d_resid == d_resid_out &&
        n->resid_out_stride != n->resid_stride)
      return MOE_ERR_INVALID_ARGUMENT;
    if (!d_y && !d_resid && !d_post_gain && !d_gate && !d_pre_gain)
      return MOE_ERR_INVALID_ARGUMENT;
    const size_t need = norm_grad_partials(n) * sizeof(float);
    if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  }
  if (gate && !gate_shape_ok(n)) return MOE_ERR_INVALID_ARGUMENT;
  const NormGradArgs a{y, resid_out, post_gain, gate, pre_gain, d_x,
                       d_resid_out, d_y, d_resid, d_post_gain, d_gate,
                       d_pre_gain};
  return hip_status(launch_residual_norm_backward(n, a, (float*)workspace,
                                                  S(stream)));
}

// ------------------------------------ the combine's end and its gradients
static moe_status check_combine_norm(const moe_problem* p, const moe_norm* n,
                                     const NormArgs& a) {
  moe_status st = moe_check_norm(n);
  if (st != MOE_OK) return st;
  if (n->T != p->T || n->H != p->H) return MOE_ERR_INVALID_ARGUMENT;
  return p->T == 0 ? MOE_OK : check_norm_forward(n, a);
}

moe_status moe_combine_norm(const moe_problem* p, const moe_norm* n,
                            const float* y_perm, const int32_t* pair_row,
                            const float* topk_w, const float* y_shared,
                            const void* resid, const void* post_gain,
                            const float* gate, const void* pre_gain,
                            void* block_out, void* resid_out, void* x_out,
                            void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  const NormArgs a{nullptr, resid, post_gain, gate, pre_gain, resid_out, x_out};
  if ((st = check_combine_norm(p, n, a)) != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!y_perm || !pair_row || !topk_w) return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(y_perm) || !al16(y_shared)) return MOE_ERR_INVALID_ARGUMENT;
  const CombineSource c{y_perm, pair_row, topk_w, y_shared, p->k,
                        (int)cap_rows(p), block_out};
  return hip_status(launch_residual_norm(n, a, &c, S(stream)));
}

moe_status moe_combine_backward(const moe_problem* p, const void* d_out,
                                const float* y_perm, const int32_t* pair_row,
                                const float* topk_w, float* d_y_perm,
                                float* d_topk_w, float* d_y_shared,
                                void* stream) {
  const moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!d_out || !pair_row || !topk_w || (d_topk_w && !y_perm) ||
      (!d_y_perm && !d_topk_w && !d_y_shared))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!al16(d_out) || !al16(y_perm) || !al16(d_y_perm) || !al16(d_y_shared))
    return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_combine_backward(
      d_out, p->out_dtype, y_perm, pair_row, topk_w, p->T, p->H, p->k,
      (int)cap_rows(p), d_y_perm, d_topk_w, d_y_shared, S(stream)));
}

moe_status moe_layer_forward_scored(
    const moe_problem* p, const moe_router* r, const moe_norm* n,
    const void* logits, const float* bias, const void* x,
    const moe_weights* w, const int32_t* l2p, const int32_t* replica_count,
    const void* resid, const void* post_gain, const float* gate,
    const void* pre_gain, void* out, void* resid_out, void* x_out,
    int32_t* expert_counts, void* workspace, size_t ws_bytes, void* stream) {
  moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if ((st = moe_check_router(r)) != MOE_OK) return st;
  if (r->T != p->T || r->E != p->E || r->k != p->k)
    return MOE_ERR_INVALID_ARGUMENT;
  const ScoredLayer sl{r, n, {nullptr, resid, post_gain, gate, pre_gain,
                              resid_out, x_out}};
  if (n) {
    if ((st = check_combine_norm(p, n, sl.norm)) != MOE_OK) return st;
  } else if (resid || post_gain || gate || pre_gain || resid_out || x_out) {
    return MOE_ERR_INVALID_ARGUMENT;
  }
  return layer_impl(p, logits, bias, x, w, l2p, replica_count, out,
                    expert_counts, workspace, ws_bytes, stream, nullptr, &sl);
}

// ------------------------------------------------------- a few tokens
namespace {
struct FewScratch {
  int32_t* ids;
  float* w;
  FewList* list;
  bf16_t* h;
};
FewScratch carve_few(Carver& c, const moe_problem* p) {
  FewScratch f{};
  f.ids = c.take<int32_t>((size_t)MOE_FEW_TOKENS * p->k);
  f.w = c.take<float>((size_t)MOE_FEW_TOKENS * p->k);
  f.list = c.take<FewList>(1);
  f.h = c.take<bf16_t>((size_t)few_entries(p) * MOE_FEW_TOKENS * p->I);
  return f;
}
moe_status check_few(const moe_problem* p) {
  const moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (p->T > MOE_FEW_TOKENS || p->act_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  // a workgroup for 16 of H in one launch of less than 2^32 threads; 16 of I
  // of every expert in use counted in 32 bits
  if (p->H >= 1 << 27 || (double)few_entries(p) * (p->I / 16) >= 2147483647.0 - 512.0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
}  // namespace

moe_status moe_layer_few_workspace_size(const moe_problem* p, size_t* bytes) {
  const moe_status st = check_few(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  Carver c(nullptr);
  carve_few(c, p);
  *bytes = c.used;
  return MOE_OK;
}

moe_status moe_layer_forward_few(const moe_problem* p, const moe_router* r,
                                 const void* logits, const float* bias,
                                 const void* x, const moe_weights* w,
                                 const int32_t* l2p,
                                 const int32_t* replica_count, void* out,
                                 int32_t* expert_counts, void* workspace,
                                 size_t ws_bytes, void* stream) {
  moe_status st = check_few(p);
  if (st != MOE_OK) return st;
  if (r) {
    if ((st = moe_check_router(r)) != MOE_OK) return st;
    if (r->T != p->T || r->E != p->E || r->k != p->k) return MOE_ERR_INVALID_ARGUMENT;
  }
  if ((st = check_map(p, l2p, replica_count)) != MOE_OK) return st;
  if ((st = check_weights(p, w)) != MOE_OK) return st;
  hipStream_t s = S(stream);
  if (p->T == 0) {
    if (expert_counts)
      return hip_status(launch_fill_i32(expert_counts, 0, (size_t)p->E, s));
    return MOE_OK;
  }
  if (!logits || !x || !out || !al16(x) || !al16(out)) return MOE_ERR_INVALID_ARGUMENT;
  size_t need;
  moe_layer_few_workspace_size(p, &need);
  if (!workspace || ws_bytes < need) return MOE_ERR_WORKSPACE;
  Carver c(workspace);
  const FewScratch f = carve_few(c, p);
  FewCall call{};
  call.x = (const bf16_t*)x;
  call.weights = w;
  call.l2p = l2p;
  call.rep = replica_count;
  call.counts = expert_counts;
  call.list = f.list;
  call.h = f.h;
  call.out = out;
  // a router inside the first kernel holds at most 256 experts
  if (!r && p->E <= 256) {
    call.logits = (const float*)logits;
    call.bias = bias;
  } else {
    const hipError_t e =
        r ? launch_route_scored(r, logits, bias, f.ids, f.w, nullptr, nullptr, s)
          : launch_route_topk((const float*)logits, bias, p->T, p->E, p->k,
                              f.ids, f.w, nullptr, s);
    if (e != hipSuccess) return MOE_ERR_HIP;
    call.ids = f.ids;
    call.w = f.w;
  }
  return hip_status(launch_few(p, call, s));
}

// --------------------------------------------------- 8-bit checkpoints
moe_status moe_check_rows(const moe_rows* r) {
  if (!r || r->rows < 0 || r->cols < 1 || r->stride < r->cols)
    return MOE_ERR_INVALID_ARGUMENT;
  if (r->dtype < MOE_F32 || r->dtype > MOE_FP8_E4M3) return MOE_ERR_INVALID_ARGUMENT;
  if (r->dtype == MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
  // a row's columns up to the end of its last group, and the groups of all
  // rows, are counted in 32 bits
  if (r->cols > 2147483647 - 127) return MOE_ERR_UNSUPPORTED;
  if ((double)r->rows * (((double)r->cols + 127.0) / 128.0) >= 2147483647.0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status moe_checkpoint_rows(const moe_rows* r, const void* src,
                               uint8_t* codes, float* scales, void* stream) {
  const moe_status st = moe_check_rows(r);
  if (st != MOE_OK) return st;
  if (r->rows == 0) return MOE_OK;
  if (!src || !codes || !scales) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_checkpoint_rows(src, r->dtype, r->rows, r->cols,
                                           r->stride, codes, scales, S(stream)));
}

moe_status moe_restore_rows(const moe_rows* r, const uint8_t* codes,
                            const float* scales, void* dst, void* stream) {
  const moe_status st = moe_check_rows(r);
  if (st != MOE_OK) return st;
  if (r->rows == 0) return MOE_OK;
  if (!codes || !scales || !dst) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_restore_rows(codes, scales, r->rows, r->cols,
                                        r->dtype, r->stride, dst, S(stream)));
}

// ------------------------------------------------ training the experts
namespace {
moe_status check_experts(const moe_problem* p) {
  const moe_status st = moe_check_problem(p);
  if (st != MOE_OK) return st;
  if (p->act_dtype != MOE_BF16 || p->weight_dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  // places of a weight gradient's tiles are divided by multiplication, and
  // rows with the shared expert's are counted, in 32 bits
  if (p->H > 65536 || p->I > 65536 || (double)p->T * (p->k + 1) >= 2147483647.0)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

bool saved_ok(const moe_saved* v) {
  return v && v->offsets && v->row_token && v->row_weight && v->pair_row &&
         v->x_codes && v->x_scales && v->gu_codes && v->gu_scales &&
         al16(v->x_codes) && al16(v->gu_codes);
}

struct ExpertsScratch {
  int4* tiles;
  int32_t* tile_count;
  // forward
  DispatchScratch d;
  float* gu;           // [rows][2 I]
  bf16_t* h;           // [rows][I] (backward: the weighted h)
  float* y;            // [cap][H] (backward: the rows' d_x, then their x and
                       // d_out in bf16)
  float* y_shared;     // [T][H]   (backward: likewise)
  // backward
  float* dh;           // [rows][I]
  bf16_t* dgu;         // [rows][2 I]
};

ExpertsScratch carve_experts(Carver& c, const moe_problem* p, bool backward) {
  ExpertsScratch e{};
  const size_t cap = (size_t)cap_rows(p), T = (size_t)p->T;
  const size_t rows = cap + (p->has_shared ? T : 0);
  // at most one tile per 16 rows (balanced tiles) and one per group
  e.tiles = c.take<int4>((size_t)p->num_physical + 2 + (rows + 15) / 16);
  e.tile_count = c.take<int32_t>(4);
  e.h = c.take<bf16_t>(rows * p->I);
  e.y = c.take<float>(cap * p->H);
  if (p->has_shared) e.y_shared = c.take<float>(T * p->H);
  if (backward) {
    e.dh = c.take<float>(rows * p->I);
    e.dgu = c.take<bf16_t>(rows * 2 * p->I);
  } else {
    e.d = carve_dispatch(c, p);
    e.gu = c.take<float>(rows * 2 * p->I);
  }
  return e;
}

size_t experts_need(const moe_problem* p, bool backward) {
  Carver c(nullptr);
  carve_experts(c, p, backward);
  return c.used;
}

TrainGemm train_gemm(const moe_problem* p, const moe_weights* w,
                     const ExpertsScratch& e) {
  return {train_tile_rows(p), e.tiles, e.tile_count, p->num_physical, (int)cap_rows(p), p->T,
          p->H, p->I, p->has_shared, w};
}
}  // namespace

moe_status moe_experts_workspace_size(const moe_problem* p, size_t* bytes) {
  const moe_status st = check_experts(p);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARGUMENT;
  *bytes = std::max(experts_need(p, false), experts_need(p, true));
  return MOE_OK;
}

moe_status moe_experts_forward(const moe_problem* p, const void* x,
                               const int32_t* topk_ids, const float* topk_w,
                               const int32_t* l2p,
                               const int32_t* replica_count,
                               const moe_weights* w, const moe_saved* saved,
                               void* out, void* workspace, size_t ws_bytes,
                               void* stream) {
  moe_status st = check_experts(p);
  if (st != MOE_OK) return st;
  if ((st = check_map(p, l2p, replica_count)) != MOE_OK) return st;
  if ((st = check_weights(p, w)) != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!x || !topk_ids || !topk_w || !out || !saved_ok(saved) || !al16(x) || !al16(out))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!workspace || ws_bytes < experts_need(p, false)) return MOE_ERR_WORKSPACE;
  hipStream_t s = S(stream);
  Carver c(workspace);
  const ExpertsScratch e = carve_experts(c, p, false);
  const int cap = (int)cap_rows(p);
  DispatchExtras extras{};
  extras.E = p->E;
  // with a shared expert its tiles go among the others, by a kernel of its own
  if (!p->has_shared) {
    extras.tiles = e.tiles;
    extras.tile_count = e.tile_count;
    extras.BM = train_tile_rows(p);
    extras.balanced = 1;
  }
  st = dispatch_impl(p, x, topk_ids, topk_w, l2p, replica_count, nullptr,
                     nullptr, saved->offsets, saved->row_token,
                     saved->row_weight, saved->pair_row, e.d, s, nullptr,
                     /*materialize=*/false, &extras);
  if (st != MOE_OK) return st;
  hipError_t h = hipSuccess;
  if (p->has_shared)
    h = launch_train_tiles(saved->offsets, p->num_physical, 1, p->T,
                           train_tile_rows(p), e.tiles, e.tile_count, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  const TrainGemm g = train_gemm(p, w, e);
  h = launch_gemm_gate_up(g, (const bf16_t*)x, saved->row_token, e.gu, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  const ExpertRows rows{saved->offsets + p->num_physical, cap, p->T,
                        p->has_shared, p->I};
  h = launch_swiglu_save(rows, e.gu, e.h, saved->gu_codes, saved->gu_scales,
                         (const bf16_t*)x, p->H, saved->x_codes,
                         saved->x_scales, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  h = launch_gemm_down(g, e.h, e.y, e.y_shared, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  return hip_status(launch_combine(e.y, saved->pair_row, topk_w, e.y_shared,
                                   p->T, p->H, p->k, p->out_dtype, out, s));
}

moe_status moe_experts_backward(const moe_problem* p, const moe_saved* saved,
                                const void* d_out, const moe_weights* w,
                                void* d_x, float* d_topk_w,
                                const moe_weight_grads* grads, void* workspace,
                                size_t ws_bytes, void* stream) {
  moe_status st = check_experts(p);
  if (st != MOE_OK) return st;
  if ((st = check_weights(p, w)) != MOE_OK) return st;
  if (!d_x && !d_topk_w && !grads) return MOE_ERR_INVALID_ARGUMENT;
  if (grads) {
    if (grads->dtype < MOE_F32 || grads->dtype > MOE_FP8_E4M3) return MOE_ERR_INVALID_ARGUMENT;
    if (grads->dtype == MOE_FP8_E4M3) return MOE_ERR_UNSUPPORTED;
    const void* all[6] = {grads->d_gate, grads->d_up, grads->d_down,
                          grads->sh_d_gate, grads->sh_d_up, grads->sh_d_down};
    for (int i = 0; i < (p->has_shared ? 6 : 3); ++i)
      if (!all[i] || !al16(all[i])) return MOE_ERR_INVALID_ARGUMENT;
  }
  hipStream_t s = S(stream);
  const size_t HI = (size_t)p->H * p->I;
  if (p->T == 0) {
    if (!grads) return MOE_OK;
    const size_t words = HI * (grads->dtype == MOE_F32 ? 4 : 2) / 4;
    void* routed[3] = {grads->d_gate, grads->d_up, grads->d_down};
    void* shared[3] = {grads->sh_d_gate, grads->sh_d_up, grads->sh_d_down};
    for (int i = 0; i < 3; ++i) {
      if (launch_fill_i32((int32_t*)routed[i], 0, words * p->num_physical, s) != hipSuccess)
        return MOE_ERR_HIP;
      if (p->has_shared && launch_fill_i32((int32_t*)shared[i], 0, words, s) != hipSuccess)
        return MOE_ERR_HIP;
    }
    return MOE_OK;
  }
  if (!d_out || !saved_ok(saved) || !al16(d_out) || !al16(d_x)) return MOE_ERR_INVALID_ARGUMENT;
  if (!workspace || ws_bytes < experts_need(p, true)) return MOE_ERR_WORKSPACE;
  if (d_x == d_out) return MOE_ERR_INVALID_ARGUMENT;   // (read after d_x is written)
  Carver c(workspace);
  const ExpertsScratch e = carve_experts(c, p, true);
  const int cap = (int)cap_rows(p), P = p->num_physical;
  const bf16_t* d = (const bf16_t*)d_out;
  hipError_t h = launch_train_tiles(saved->offsets, P, p->has_shared, p->T,
                                    train_tile_rows(p), e.tiles, e.tile_count, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  const TrainGemm g = train_gemm(p, w, e);
  h = launch_gemm_down_back(g, d, saved->row_token, e.dh, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  const ExpertRows rows{saved->offsets + P, cap, p->T, p->has_shared, p->I};
  const PairRows pairs{saved->row_token, saved->row_weight, saved->pair_row, p->k};
  h = launch_swiglu_backward(rows, pairs, e.dh, saved->gu_codes,
                             saved->gu_scales, e.dgu, e.h, d_topk_w, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  if (d_x) {
    h = launch_gemm_gate_up_back(g, e.dgu, e.y, e.y_shared, s);
    if (h != hipSuccess) return MOE_ERR_HIP;
    h = launch_combine(e.y, saved->pair_row, nullptr, e.y_shared, p->T, p->H,
                       p->k, MOE_BF16, d_x, s);
    if (h != hipSuccess) return MOE_ERR_HIP;
  }
  if (!grads) return MOE_OK;
  // the rows of both products' operands side by side, in the place of the
  // rows' d_x, which nobody needs any more
  const int H = p->H, I = p->I;
  bf16_t* xr = (bf16_t*)e.y;
  bf16_t* dr = xr + (size_t)cap * H;
  bf16_t* xs = (bf16_t*)e.y_shared;      // (null without a shared expert)
  h = launch_gather_pair(saved->x_codes, saved->x_scales, d, saved->row_token,
                         rows.n_routed, cap, p->T, H, xr, dr, xs, s);
  if (h != hipSuccess) return MOE_ERR_HIP;
  WeightGrad q{};
  q.P = P;
  q.T = p->T;
  q.has_shared = p->has_shared;
  q.offsets = saved->offsets;
  q.dtype = grads->dtype;
  // d_W_gate and d_W_up: x^T (dg | du); d_W_down: (w h)^T d_out
  q.product[0] = {H, 2 * I, I, xr, e.dgu, xs, e.dgu + (size_t)cap * 2 * I, H, 2 * I,
                  {grads->d_gate, grads->d_up},
                  {grads->sh_d_gate, grads->sh_d_up}};
  q.product[1] = {I, H, H, e.h, dr, e.h + (size_t)cap * I, d, I, H,
                  {grads->d_down, nullptr}, {grads->sh_d_down, nullptr}};
  return hip_status(launch_weight_grad(q, s));
}

moe_status moe_prepack_weights(const void* src, int32_t K, int32_t N,
                               int32_t dtype, int32_t layout, void* dst,
                               void* stream) {
  if (dtype != MOE_F32 && dtype != MOE_BF16 && dtype != MOE_FP8_E4M3)
    return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_LAYOUT_KN && layout != MOE_LAYOUT_NK)
    return MOE_ERR_INVALID_ARGUMENT;
  if (K < 0 || N < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype == MOE_BF16 && (N % 16 || K % 32)) return MOE_ERR_INVALID_ARGUMENT;
  if (dtype == MOE_FP8_E4M3 && (N % 16 || K % 128))
    return MOE_ERR_INVALID_ARGUMENT;
  if (K == 0 || N == 0) return MOE_OK;
  if (!src || !dst || src == dst) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_prepack(src, K, N, dtype, layout, dst, S(stream)));
}

moe_status moe_quantize_fp8_blocks(const float* w, int32_t K, int32_t N,
                                   int32_t block, int32_t layout,
                                   uint8_t* codes, float* scales,
                                   void* stream) {
  if (block != 128) return MOE_ERR_UNSUPPORTED;
  if (layout != MOE_LAYOUT_KN && layout != MOE_LAYOUT_NK)
    return MOE_ERR_INVALID_ARGUMENT;
  if (K < 0 || N < 0 || K % block || N % block) return MOE_ERR_INVALID_ARGUMENT;
  if (K == 0 || N == 0) return MOE_OK;
  if (!w || !codes || !scales) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(
      launch_quant_blocks_fp8(w, K, N, layout, codes, scales, S(stream)));
}

}  // extern "C"
