// Gradients of the residual norm (moe_residual_norm_backward).
//
// As the forward, a row lies in registers and the workgroups walk the rows
// with the next row's loads in flight; short rows share a workgroup.  With
//   rs = 1 / sqrt(mean r'^2 + eps), gp = d_x (o + pre)
//   g  = d_r' + rs (gp - r' rs^2 mean(gp r'))
//   ys = 1 / sqrt(mean y^2 + eps),  q = rscale gate g (o + post)
//   d_y = ys (q - y ys^2 mean(q y))
// the first exchange over the row carries mean r'^2, mean(gp r') and
// mean y^2, the second mean(q y) and the gate's row sum.  Gradients of gains
// and of a gate along the columns add up in registers over a workgroup's
// rows; a second launch sums the workgroups' rows in a fixed order.  Bound by
// HBM, four rows in and two out, and by the one workgroup of a long row that a
// CU's registers hold: 4096 x 7168 bf16 with all operands 76 us = 4.7 TB/s,
// and 5 us for the column sums (16 slices a column; 4 took 40 us).
#include <algorithm>
#include <type_traits>

#include "block.h"
#include "rows.h"

namespace moe {

namespace {

struct NormGradRun {
  moe_norm n;
  NormGradArgs a;
  float* part;      // [arrays][gridDim.x][H], then [gridDim.x] for one number
  int col_gate;     // the gate's gradient is a sum over the rows
  int one_gate;     // ... is one number
  int nt;           // threads a row
};

constexpr int kShare = 256;            // threads that short rows share
constexpr int kAlone = 256;            // batches whose rows share none

// FIT kExact: besides, every operand but the gate is there, so the row's code
// has no branches (with a branch a piece and operand the 4096 x 7168 case ran
// 103 us instead of 79: 1100 instructions a wavefront and row).
// KEEP: the next row is requested early.  Rows too long for that (H > 8192)
// take 1024 threads, which have half the registers: they do without, hold the
// gains' sums in LDS, read the gains anew and spill 47 to 164 registers
// (2048 x 16384 bf16 164 us = 2.5 TB/s).
// GV: a gate along the columns; with 16 columns in pieces of four it spills 5
// to 39 registers (4096 x 7168 float32 171 us, 131 us without a gate).
template <typename YT, typename RT, int W, int EPT, Fit FIT, bool KEEP,
          bool GV>
__global__ __launch_bounds__(KEEP ? 512 : 1024) void k_residual_norm_backward(NormGradRun q) {
  constexpr int P = EPT / W;
  constexpr bool FULL = FIT == kExact;
  constexpr int kHold = EPT == 8 ? kShare * EPT : 1;
  typedef Cols<W> V;
  __shared__ float red3[2][48], red2[2][32];    // by row parity
  __shared__ float hold[kHold];
  // two vectors of the row, each thread's own pieces: the gains, or their sums
  extern __shared__ __attribute__((aligned(16))) float lds[];
  const moe_norm& n = q.n;
  const NormGradArgs& a = q.a;
  const int H = n.H, NT = q.nt;
  const int R = blockDim.x / NT, rg = threadIdx.x / NT, tid = threadIdx.x - rg * NT;
  const int waves = NT >> 6, first = rg * waves;
  const float inv_h = 1.0f / (float)H;
  const bool x_bf16 = W == 8 || n.out_dtype == MOE_BF16;
  const bool has_x = FULL || a.d_x, has_post = FULL || a.post_gain;
  const bool to_block = FULL || a.d_y || a.d_post || a.d_gate;
  Piece pc[P];
#pragma unroll
  for (int v = 0; v < P; ++v) pc[v] = piece_at<W, FIT>(W * (tid + v * NT), H);
  // (only the last pieces of a row can lie past its end: with 16 columns a
  // thread, those of the last pass)
  auto own = [&](auto raw, auto type, int v) {
    using T = decltype(type);
    if (EPT == 16 && v < P - 1) return raw;
    return own_cols<T, W, FIT>(raw, pc[v]);
  };
  V d_pre[P], d_post[P], d_gc[GV ? P : 1];
  V* lds_pre = (V*)lds;                // piece v of thread tid: [tid + v NT]
  V* lds_post = lds_pre + P * NT;
  auto pre_of = [&](int v) -> V {
    if constexpr (KEEP) return lds_pre[tid + v * NT];
    return a.pre_gain ? load_gain<W>(a.pre_gain, n.gain_dtype, pc[v].col, H, n.gain_offset) : V(0.0f);
  };
  auto post_of = [&](int v) -> V {
    if constexpr (KEEP) return lds_post[tid + v * NT];
    return a.post_gain ? load_gain<W>(a.post_gain, n.gain_dtype, pc[v].col, H, n.gain_offset) : V(1.0f);
  };
  Raw<RT, W> gq[P], rq[P];
  Raw<YT, W> yq[P];
  u32x4_t xq[P];
  // (a row past the end reads the last one again and takes part in the
  // exchanges alone: zero times an infinity would not add zero)
  const long last = n.T - 1;
  auto fetch = [&](long t) {
    t = min(t, last);
    if (has_x) {
#pragma unroll
      for (int v = 0; v < P; ++v) {
        rq[v] = load_piece<RT, W, FIT, true>((const RT*)a.resid_out + t * n.resid_out_stride, pc[v], H);
        if (x_bf16) {
          const Raw<bf16_t, W> x = load_piece<bf16_t, W, FIT, true>((const bf16_t*)a.d_x + t * n.out_stride, pc[v], H);
#pragma unroll
          for (int i = 0; i < W / 2; ++i) xq[v][i] = x[i];
        } else {
          xq[v] = load_piece<float, 4, FIT, true>((const float*)a.d_x + t * n.out_stride, pc[v], H);
        }
      }
    }
    if (FULL || a.y) {
#pragma unroll
      for (int v = 0; v < P; ++v)
        yq[v] = load_piece<YT, W, FIT, true>((const YT*)a.y + t * n.block_stride, pc[v], H);
    }
    if (FULL || a.d_resid_out) {
#pragma unroll
      for (int v = 0; v < P; ++v)
        gq[v] = load_piece<RT, W, FIT, true>((const RT*)a.d_resid_out + t * n.resid_out_stride, pc[v], H);
    }
  };
#pragma unroll
  for (int v = 0; v < P; ++v) {        // operands that are absent stay zero
    gq[v] = 0u;
    rq[v] = 0u;
    yq[v] = 0u;
    xq[v] = 0u;
  }
  auto wide_x = [&](u32x4_t b, int v) -> V {
    if (x_bf16) {
      Raw<bf16_t, W> h;
#pragma unroll
      for (int i = 0; i < W / 2; ++i) h[i] = b[i];
      return widen<bf16_t, W>(own(h, bf16_t{}, v));
    }
    if constexpr (W == 4) return widen<float, 4>(own(b, float{}, v));
    return V(0.0f);
  };
  float d_one = 0.0f;
  int par = 0;
  const long step = (long)gridDim.x * R;
  const bool row_gate = !GV && a.d_gate;
  if (KEEP) fetch((long)blockIdx.x * R + rg);
#pragma unroll
  for (int v = 0; v < P; ++v) {
    d_pre[v] = d_post[v] = 0.0f;
    if constexpr (GV) d_gc[v] = 0.0f;
    V gp = 0.0f, gq1 = KEEP ? 1.0f : 0.0f;
    if (KEEP && a.pre_gain) gp = load_gain<W>(a.pre_gain, n.gain_dtype, pc[v].col, H, n.gain_offset);
    if (KEEP && a.post_gain) gq1 = load_gain<W>(a.post_gain, n.gain_dtype, pc[v].col, H, n.gain_offset);
    // the rows of a workgroup write the same values; a thread reads only what
    // it wrote
    lds_pre[tid + v * NT] = gp;
    lds_post[tid + v * NT] = gq1;
  }
  // every row of a workgroup takes part in its barriers, past the end too
  for (long t0 = (long)blockIdx.x * R; t0 < n.T; t0 += step, par ^= 1) {
    const long t = t0 + rg;
    const bool valid = !KEEP || t < n.T;       // (long rows share no workgroup)
    if (!KEEP) fetch(t);
    V g[P];
    Raw<RT, W> r[P];
    Raw<YT, W> y[P];
    u32x4_t x[P];
    float s[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int v = 0; v < P; ++v) {
      g[v] = widen<RT, W>(own(gq[v], RT{}, v));
      r[v] = own(rq[v], RT{}, v);
      y[v] = own(yq[v], YT{}, v);
      x[v] = xq[v];
      const V rv = widen<RT, W>(r[v]), yv = widen<YT, W>(y[v]);
      s[0] += dot_cols<W>(rv, rv);
      s[1] += dot_cols<W>(rv, wide_x(x[v], v) * pre_of(v));
      s[2] += dot_cols<W>(yv, yv);
    }
    if (KEEP) fetch(t + step);
    row_sum(s, red3[par], first, waves);
    const float rs = has_x ? 1.0f / sqrtf(s[0] * inv_h + n.eps) : 0.0f;
    const float c = s[1] * inv_h * rs * rs;
    const float ys = has_post ? 1.0f / sqrtf(s[2] * inv_h + n.eps) : 1.0f;
    const float ysr = ys * n.residual_scale;
    float s2[2] = {0.0f, 0.0f};        // q y ys, the gate's row
    if (valid) {
      const float gate1 = !GV && a.gate ? a.gate[n.gate_rows > 1 ? t : 0] : 1.0f;
#pragma unroll
      for (int v = 0; v < P; ++v) {
        const V rv = widen<RT, W>(r[v]), xv = wide_x(x[v], v);
        const V yv = widen<YT, W>(y[v]) * ysr;     // unit(y) rscale
        const V po = post_of(v);
        if constexpr (KEEP) d_pre[v] += xv * (rv * rs);
        else lds_pre[tid + v * NT] += xv * (rv * rs);
        g[v] += rs * (xv * pre_of(v) - c * rv);
        if (FULL || a.d_resid)
          store_piece<RT, W, FIT, true>((RT*)a.d_resid + t * n.resid_stride, pc[v], H, g[v]);
        if (!to_block) continue;
        V h = g[v] * yv;                 // what the gate's gradient sums, less po
        if constexpr (GV) {
          const V f = load_f32<W, FIT>(a.gate + (n.gate_rows > 1 ? t * H : 0), pc[v], H);
          if (q.col_gate) {
            d_gc[v] += h * po;
          } else if (a.d_gate) {
            const V e = h * po;
#pragma unroll
            for (int i = 0; i < W; i += 4)
              store_piece<float, 4, FIT, true>(a.d_gate + t * H, piece_at<4, FIT>(pc[v].col + i, H), H,
                                               f32x4_t{e[i], e[i + 1], e[i + 2], e[i + 3]});
          }
          h *= f;
          g[v] *= f;
        } else {
          s2[1] += dot_cols<W>(h, po);
          h *= gate1;
          g[v] *= gate1;
        }
        if constexpr (KEEP) d_post[v] += h;
        else lds_post[tid + v * NT] += h;
        s2[0] += dot_cols<W>(h, po);
        g[v] *= po;
      }
    }
    if (!to_block) continue;
    if (has_post || row_gate) row_sum(s2, red2[par], first, waves);
    if (row_gate) {
      if (q.one_gate) d_one += s2[1];
      else if (tid == 0 && valid) a.d_gate[t] = s2[1];
    }
    if (valid && (FULL || a.d_y)) {
      // ys (rscale q - y ys^2 mean(q y)); h summed q y ys already
      const float cy = has_post ? s2[0] * inv_h * ys * ys : 0.0f;
#pragma unroll
      for (int v = 0; v < P; ++v)
        store_piece<YT, W, FIT, true>((YT*)a.d_y + t * n.block_stride, pc[v], H,
                                      ysr * g[v] - cy * widen<YT, W>(y[v]));
    }
  }
  // the workgroup's sums over its rows
  float* part = q.part + (size_t)blockIdx.x * H;
  const size_t arrays = (size_t)gridDim.x * H;
  auto put = [&](V* d) {
    if constexpr (EPT == 8) {
      if (R > 1) {                     // rows that share the workgroup
        lds_barrier();
#pragma unroll
        for (int v = 0; v < P; ++v) {
#pragma unroll
          for (int i = 0; i < W; ++i) hold[(v * W + i) * kShare + threadIdx.x] = d[v][i];
        }
        lds_barrier();
        if (rg == 0) {
#pragma unroll
          for (int v = 0; v < P; ++v) {
#pragma unroll
            for (int i = 0; i < W; ++i) {
              for (int k = 1; k < R; ++k) d[v][i] += hold[(v * W + i) * kShare + k * NT + tid];
            }
          }
        }
      }
    }
    if (rg == 0) {
#pragma unroll
      for (int v = 0; v < P; ++v) {
#pragma unroll
        for (int i = 0; i < W; i += 4)
          store_piece<float, 4, FIT == kExact ? kExact : kAny, false>(
              part, piece_at<4, FIT == kExact ? kExact : kAny>(pc[v].col + i, H), H,
              f32x4_t{d[v][i], d[v][i + 1], d[v][i + 2], d[v][i + 3]});
      }
    }
    part += arrays;
  };
  if constexpr (!KEEP) {
#pragma unroll
    for (int v = 0; v < P; ++v) {
      d_pre[v] = lds_pre[tid + v * NT];
      d_post[v] = lds_post[tid + v * NT];
    }
  }
  if (a.d_pre) put(d_pre);
  if (a.d_post) put(d_post);
  if constexpr (GV) {
    if (q.col_gate) put(d_gc);
  }
  if (q.one_gate) {
    lds_barrier();
    if (tid == 0) red2[0][rg] = d_one;
    lds_barrier();
    if (threadIdx.x == 0) {
      for (int k = 1; k < R; ++k) d_one += red2[0][k];
      part[0 - (size_t)blockIdx.x * H + blockIdx.x] = d_one;
    }
  }
}

// out[c] = sum over the workgroups' rows; 16 slices of the rows, each summed
// in double, then the slices in order
struct ColumnSums {
  const float* part[3];
  float* out[3];
};

__global__ __launch_bounds__(1024) void k_column_sums(ColumnSums q, int parts,
                                                      int H) {
  __shared__ double s[16][64];
  const int c = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + c;
  const float* part = q.part[blockIdx.y];
  double v = 0.0;
  if (col < H) {
#pragma unroll 8
    for (int p = w; p < parts; p += 16) v += (double)part[(size_t)p * H + col];
  }
  s[w][c] = v;
  __syncthreads();
  if (w == 0 && col < H) {
#pragma unroll
    for (int k = 1; k < 16; ++k) v += s[k][c];
    q.out[blockIdx.y][col] = (float)v;
  }
}

__global__ __launch_bounds__(64) void k_one_sum(const float* part, int parts,
                                                float* out) {
  double v = 0.0;
  for (int p = threadIdx.x; p < parts; p += 64) v += (double)part[p];
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  if (threadIdx.x == 0) *out = (float)v;
}

__global__ __launch_bounds__(256) void k_clear(float* p, int n) {
  for (int i = blockIdx.x * 256 + threadIdx.x; i < n; i += 256 * gridDim.x) p[i] = 0.0f;
}

struct Shape {
  int ept, nt, rows, grid;   // columns and threads a row, rows a workgroup
  bool keep;
};
// As many workgroups as stay on the GPU at once: the registers leave room for
// 3 wavefronts a SIMD with 8 columns a thread, 2 with 16, and each workgroup
// starts at the same SIMD (rows of 320 threads: 24 us with one workgroup a
// CU, 29 us with two that run one after the other).
Shape grad_shape(int T, int H) {
  Shape s;
  const int v = (H + 7) / 8;
  s.ept = v <= 512 ? 8 : 16;
  s.keep = v <= 1024;
  s.nt = ((H + s.ept - 1) / s.ept + 63) / 64 * 64;
  s.rows = s.nt <= kShare / 2 && T > kAlone ? kShare / s.nt : 1;
  const int per_cu = std::max(1, (s.ept == 8 ? 3 : 2) / ((s.nt * s.rows + 255) / 256));
  s.grid = (int)std::min<long>(((long)T + s.rows - 1) / s.rows, 256 * per_cu);
  return s;
}

// EXACT: kExact, else the general code of the width W
template <typename YT, typename RT, int W, bool EXACT>
void launch(const NormGradRun& q, const Shape& sh, hipStream_t s) {
  constexpr Fit G = W == 8 ? kAligned : kAny, F = EXACT ? kExact : G;
  const dim3 grid(sh.grid), block(sh.nt * sh.rows);
  const size_t lds = 2 * sizeof(float) * sh.nt * sh.ept;
  by_flag(q.a.gate && q.n.gate_cols > 1, [&](auto gv) {
    constexpr bool GV = gv.value;
    if (sh.ept == 8)
      k_residual_norm_backward<YT, RT, W, 8, F, true, GV><<<grid, block, lds, s>>>(q);
    else if (sh.keep)
      k_residual_norm_backward<YT, RT, W, 16, F, true, GV><<<grid, block, lds, s>>>(q);
    else
      k_residual_norm_backward<YT, RT, W, 16, G, false, GV><<<grid, block, lds, s>>>(q);
  });
}

}  // namespace

size_t norm_grad_partials(const moe_norm* n) {
  return (size_t)grad_shape(n->T, n->H).grid * (3 * (size_t)n->H + 1);
}

// Workgroups grow with T but for one step down, where short rows begin to
// share them.
size_t norm_grad_scratch(const moe_norm* n) {
  moe_norm few = *n;
  few.T = std::min(n->T, kAlone);
  return std::max(norm_grad_partials(n), norm_grad_partials(&few));
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
    if (a.d_pre) k_clear<<<64, 256, 0, s>>>(a.d_pre, n->H);
    if (a.d_post) k_clear<<<64, 256, 0, s>>>(a.d_post, n->H);
    if (q.one_gate || q.col_gate) k_clear<<<64, 256, 0, s>>>(a.d_gate, n->gate_cols);
    return hipGetLastError();
  }
  const Shape sh = grad_shape(n->T, n->H);
  q.nt = sh.nt;
  auto aligned = [&](int W) {
    return n->H % W == 0 && rows_aligned(a.y, n->block_dtype, n->block_stride, W) &&
           rows_aligned(a.d_y, n->block_dtype, n->block_stride, W) &&
           rows_aligned(a.resid_out, n->resid_dtype, n->resid_out_stride, W) &&
           rows_aligned(a.d_resid_out, n->resid_dtype, n->resid_out_stride, W) &&
           rows_aligned(a.d_resid, n->resid_dtype, n->resid_stride, W) &&
           rows_aligned(a.d_x, n->out_dtype, n->out_stride, W) &&
           aligned16(a.gate) && aligned16(a.d_gate);
  };
  const bool exact = sh.keep && n->H == sh.ept * sh.nt && a.y && a.resid_out &&
                     a.post_gain && a.pre_gain && a.d_x && a.d_resid_out &&
                     a.d_y && a.d_resid && aligned(4);
  if (n->block_dtype == MOE_BF16 && n->resid_dtype == MOE_BF16 &&
      n->out_dtype == MOE_BF16 && aligned(8)) {
    by_flag(exact, [&](auto ex) { launch<bf16_t, bf16_t, 8, ex.value>(q, sh, s); });
  } else {
    by_type(n->block_dtype, [&](auto yt) {
      by_type(n->resid_dtype, [&](auto rt) {
        by_flag(exact, [&](auto ex) {
          launch<decltype(yt), decltype(rt), 4, ex.value>(q, sh, s);
        });
      });
    });
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ColumnSums c{};
  int arrays = 0;
  const size_t step = (size_t)sh.grid * H;
  for (float* out : {a.d_pre, a.d_post, q.col_gate ? a.d_gate : nullptr})
    if (out) {
      c.part[arrays] = partials + arrays * step;
      c.out[arrays++] = out;
    }
  if (arrays)
    k_column_sums<<<dim3((n->H + 63) / 64, arrays), 1024, 0, s>>>(c, sh.grid, n->H);
  if (q.one_gate) k_one_sum<<<1, 64, 0, s>>>(partials + arrays * step, sh.grid, a.d_gate);
  return hipGetLastError();
}

}  // namespace moe
