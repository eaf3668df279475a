// Residual norm (moe_residual_norm) and the combine fused into it
// (moe_combine_norm).
//
// A workgroup holds a token's row in registers, so every array is read and
// written once, and the two mean squares cost one exchange of a partial sum
// per wavefront each.  The workgroups stay and walk the rows: gains are read
// once, and a row's loads are in flight while the row before it is worked on.
// Bound by HBM: 8192 x 7168 bf16, both norms, 85 us = 5.5 TB/s (a workgroup a
// row without the prefetch: 100 us; the first kernel, gains read anew by every
// row: 151 us); combined from the expert rows 147 us = 5.6 TB/s.  One row is
// its chain of load, two exchanges and store: 4.4 us.
#include <algorithm>
#include <type_traits>

#include "block.h"
#include "rows.h"

namespace moe {

namespace {

struct NormRun {
  moe_norm n;
  NormArgs a;
  CombineSource c;
};

// KEEP: gains stay in registers and the next row is requested early.  Rows
// too long for that (H > 8192) take 1024 threads, which have half the
// registers, and do without both; but for aligned bf16 rows they spill 1 to 20
// registers, with the combine 27 to 36 (4096 x 16384 bf16 111 us = 4.8 TB/s,
// combine + norm 180 us = 5.2 TB/s).
constexpr int row_limit(int ept, bool keep) { return ept == 8 || !keep ? 1024 : 512; }

// YT: the type of y (COMB: of the shared expert's row, float32), RT: of
// resid; W columns a piece, EPT a thread
template <typename YT, typename RT, int W, Fit FIT, int EPT, bool COMB,
          bool STREAM, bool KEEP>
__global__ __launch_bounds__(row_limit(EPT, KEEP)) void k_residual_norm(NormRun q) {
  constexpr int P = EPT / W;
  typedef Cols<W> V;
  __shared__ float red[2][2][16];      // [row parity][mean square][wavefront]
  const moe_norm& n = q.n;
  const int H = n.H, NT = blockDim.x, lane = threadIdx.x & 63;
  const int waves = NT >> 6;
  const long G = gridDim.x;
  const float inv_h = 1.0f / (float)H;
  V post[KEEP ? P : 1], pre[KEEP ? P : 1];
  Piece pc[P];
#pragma unroll
  for (int v = 0; v < P; ++v) pc[v] = piece_at<W, FIT>(W * (threadIdx.x + v * NT), H);
  // (only the last pieces of a row can lie past its end: with 16 columns a
  // thread, those of the last pass)
  auto own = [&](auto raw, auto type, int v) {
    using T = decltype(type);
    if (EPT == 16 && v < P - 1) return raw;
    return own_cols<T, W, FIT>(raw, pc[v]);
  };
  auto gain = [&](const void* p, const V* kept, int v) -> V {
    if constexpr (KEEP) return kept[v];
    else return load_gain<W>(p, n.gain_dtype, pc[v].col, H, n.gain_offset);
  };
  Raw<YT, W> yq[P];
  Raw<RT, W> rq[P];
  Raw<float, 4> eq[P];                 // COMB: the first local slot's row
  int row = -1, row1 = -1;             // COMB: lane j holds slot j's row and
  float w = 0.0f, w1 = 0.0f;           //   weight, of this token and the next
  auto slots = [&](long t, int* rv, float* wv) {
    *rv = -1;
    *wv = 0.0f;
    if (lane < q.c.k && t < n.T) {
      *rv = q.c.pair_row[t * q.c.k + lane];
      *wv = q.c.w[t * q.c.k + lane];
      if (*rv >= q.c.cap) *rv = -1;
    }
  };
  auto expert_row = [&](int r, Raw<float, 4>* e) {
    const float* yr = q.c.y_perm + (size_t)r * H;
#pragma unroll
    for (int v = 0; v < P; ++v) e[v] = load_piece<float, 4, FIT, STREAM>(yr, pc[v], H);
  };
  // requests the rows of token t; `row` holds its slots
  auto fetch = [&](long t) {
    if constexpr (COMB) {
      const uint64_t m = __ballot(row >= 0);
      if (m) expert_row(__builtin_amdgcn_readlane(row, __ffsll((unsigned long long)m) - 1), eq);
      if (q.c.y_shared) {
#pragma unroll
        for (int v = 0; v < P; ++v)
          yq[v] = load_piece<YT, W, FIT, STREAM>((const YT*)q.c.y_shared + t * H, pc[v], H);
      }
    } else if (q.a.y) {
#pragma unroll
      for (int v = 0; v < P; ++v)
        yq[v] = load_piece<YT, W, FIT, STREAM>((const YT*)q.a.y + t * n.block_stride, pc[v], H);
    }
#pragma unroll
    for (int v = 0; v < P; ++v)
      rq[v] = load_piece<RT, W, FIT, STREAM>((const RT*)q.a.resid + t * n.resid_stride, pc[v], H);
  };
#pragma unroll
  for (int v = 0; v < P; ++v) yq[v] = 0u;
  if constexpr (COMB) {
    slots(blockIdx.x, &row, &w);
    slots(blockIdx.x + G, &row1, &w1);
  }
  if constexpr (KEEP) {
    fetch(blockIdx.x);
#pragma unroll
    for (int v = 0; v < P; ++v) {
      post[v] = pre[v] = 0.0f;
      if (q.a.post_gain) post[v] = load_gain<W>(q.a.post_gain, n.gain_dtype, pc[v].col, H, n.gain_offset);
      if (q.a.pre_gain) pre[v] = load_gain<W>(q.a.pre_gain, n.gain_dtype, pc[v].col, H, n.gain_offset);
    }
  }
  int par = 0;
  for (long t = blockIdx.x; t < n.T; t += G, par ^= 1) {
    if constexpr (!KEEP) fetch(t);
    V y[P], r[P];
#pragma unroll
    for (int v = 0; v < P; ++v) {
      y[v] = widen<YT, W>(own(yq[v], YT{}, v));
      r[v] = widen<RT, W>(own(rq[v], RT{}, v));
    }
    if constexpr (COMB) {
      // slots in order, then the shared expert, as moe_combine adds them
      V acc[P];
#pragma unroll
      for (int v = 0; v < P; ++v) acc[v] = 0.0f;
      auto add = [&](int j, const Raw<float, 4>* e) {
        const float wj = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(w), j));
#pragma unroll
        for (int v = 0; v < P; ++v) {
          const f32x4_t ev = widen<float, 4>(own(e[v], float{}, v));
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[v][i] = __builtin_fmaf(wj, ev[i], acc[v][i]);
        }
      };
      uint64_t m = __ballot(row >= 0);
      if (m) {
        add(__ffsll((unsigned long long)m) - 1, eq);
        m &= m - 1;
      }
      while (m) {                      // two further rows in flight at a time
        const int j = __ffsll((unsigned long long)m) - 1;
        m &= m - 1;
        const int j2 = m ? __ffsll((unsigned long long)m) - 1 : -1;
        m &= m - 1;
        Raw<float, 4> e[P], e2[P];
        expert_row(__builtin_amdgcn_readlane(row, j), e);
        if (j2 >= 0) expert_row(__builtin_amdgcn_readlane(row, j2), e2);
        add(j, e);
        if (j2 >= 0) add(j2, e2);
      }
#pragma unroll
      for (int v = 0; v < P; ++v) y[v] = q.c.y_shared ? acc[v] + y[v] : acc[v];
      row = row1;
      w = w1;
    }
    if constexpr (KEEP) {
      if (t + G < n.T) fetch(t + G);
    }
    if constexpr (COMB) {
      slots(t + 2 * G, &row1, &w1);
      if (q.c.block_out) {
#pragma unroll
        for (int v = 0; v < P; ++v)
          store_piece_as<W, FIT, STREAM>(n.block_dtype, q.c.block_out, t * n.block_stride, pc[v], H, y[v]);
      }
    }
    if (q.a.post_gain) {
      float s[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < P; ++v) s[0] += dot_cols<W>(y[v], y[v]);
      row_sum(s, red[par][0], 0, waves);
      const float rs = 1.0f / sqrtf(s[0] * inv_h + n.eps);
#pragma unroll
      for (int v = 0; v < P; ++v) y[v] = y[v] * rs * gain(q.a.post_gain, post, v);
    }
    if (q.a.gate) {
      const float* g = q.a.gate + (n.gate_rows > 1 ? t * n.gate_cols : 0);
      if (n.gate_cols == 1) {
        const float f = g[0];
#pragma unroll
        for (int v = 0; v < P; ++v) y[v] *= f;
      } else {
#pragma unroll
        for (int v = 0; v < P; ++v) y[v] *= load_f32<W, kAny>(g, pc[v], H);
      }
    }
    float s[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < P; ++v) {
      r[v] += n.residual_scale * y[v];
      s[0] += dot_cols<W>(r[v], r[v]);
      if (q.a.resid_out)
        store_piece<RT, W, FIT, STREAM>((RT*)q.a.resid_out + t * n.resid_out_stride, pc[v], H, r[v]);
    }
    if (q.a.x_out) {
      row_sum(s, red[par][1], 0, waves);
      const float rs = 1.0f / sqrtf(s[0] * inv_h + n.eps);
#pragma unroll
      for (int v = 0; v < P; ++v)
        store_piece_as<W, FIT, STREAM>(n.out_dtype, q.a.x_out, t * n.out_stride, pc[v], H,
                                       r[v] * rs * gain(q.a.pre_gain, pre, v));
    }
  }
}

template <typename YT, typename RT, int W, bool COMB>
void launch(const NormRun& q, bool al, bool stream, hipStream_t s) {
  const moe_norm& n = q.n;
  // Columns a thread: 8 where a row then fits 512 threads (combine + norm,
  // which holds three rows: 1024; 8192 x 7168 146 us against 167 us at 16).
  // Not by T: a row's sums have the same order whatever the batch.  (They
  // follow H and, through W, the types, alignment and strides of the rows.)
  const int v = (n.H + 7) / 8;
  const int ept = v <= (COMB ? 1024 : 512) ? 8 : 16;
  const bool keep = ept == 8 || v <= 1024;
  const int nt = ((n.H + ept - 1) / ept + 63) / 64 * 64;
  // the workgroups that stay on the GPU at once, at 16 wavefronts a CU
  const int per_cu = std::max(1, 16 / (nt / 64));
  const dim3 grid(std::min(n.T, 256 * per_cu)), block(nt);
  auto go = [&](auto alt, auto st) {
    constexpr Fit A = alt.value ? kAligned : kAny;
    constexpr bool S = st.value;
    if (ept == 8) k_residual_norm<YT, RT, W, A, 8, COMB, S, true><<<grid, block, 0, s>>>(q);
    else if (keep) k_residual_norm<YT, RT, W, A, 16, COMB, S, true><<<grid, block, 0, s>>>(q);
    else k_residual_norm<YT, RT, W, A, 16, COMB, S, false><<<grid, block, 0, s>>>(q);
  };
  if constexpr (W == 8) {              // only rows that are aligned
    by_flag(stream, [&](auto st) { go(std::true_type{}, st); });
  } else {
    if (!al) go(std::false_type{}, std::false_type{});
    else by_flag(stream, [&](auto st) { go(std::true_type{}, st); });
  }
}

}  // namespace

hipError_t launch_residual_norm(const moe_norm* n, const NormArgs& a,
                                const CombineSource* comb, hipStream_t s) {
  NormRun q{};
  q.n = *n;
  q.a = a;
  if (comb) q.c = *comb;
  auto aligned = [&](int W) {
    return n->H % W == 0 && rows_aligned(a.y, n->block_dtype, n->block_stride, W) &&
           rows_aligned(a.resid, n->resid_dtype, n->resid_stride, W) &&
           rows_aligned(a.resid_out, n->resid_dtype, n->resid_out_stride, W) &&
           rows_aligned(a.x_out, n->out_dtype, n->out_stride, W) &&
           rows_aligned(q.c.block_out, n->block_dtype, n->block_stride, W);
  };
  // Rows that do not fit the caches pass them by: norm of 8192 x 7168 84 us
  // against 92 us, combine + norm 146 us against 159 us; a decode batch of
  // 128, whose rows the caches hold, 6.0 us against 8.2 us with the hint.
  const bool stream = (double)n->T * n->H * 8 >= 64.0 * 1048576.0;
  const bool al4 = aligned(4);
  if (comb) {
    by_type(n->resid_dtype, [&](auto rt) {
      launch<float, decltype(rt), 4, true>(q, al4, stream, s);
    });
  } else if (n->block_dtype == MOE_BF16 && n->resid_dtype == MOE_BF16 &&
             n->out_dtype == MOE_BF16 && aligned(8)) {
    launch<bf16_t, bf16_t, 8, false>(q, true, stream, s);
  } else {
    by_type(n->block_dtype, [&](auto yt) {
      by_type(n->resid_dtype, [&](auto rt) {
        launch<decltype(yt), decltype(rt), 4, false>(q, al4, stream, s);
      });
    });
  }
  return hipGetLastError();
}

}  // namespace moe
