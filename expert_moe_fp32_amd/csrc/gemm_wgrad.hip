// Weight gradients of the experts: for every group of rows (a physical
// expert's, or the shared expert's) out = a^T b, reduced over the group's
// rows.  a is a column slice of the layer's input or of the weighted h, b of
// the gradients of gate and up or of the layer's output.
//
// Work item = 128 x 128 outputs of one group; a workgroup of 4 wavefronts
// (2 x 2 of 64 x 64), two workgroups a CU, so that one writes its outputs
// while the other multiplies: at some hundred rows a group the outputs are
// most of the traffic.  Both operands lie row by row, reduction first, so
// the MFMA operands (eight reduction values of one column a lane) come out of
// LDS by transposing reads.  Stages of 32 rows x (128 + 128) columns, 16 KiB,
// in a ring of four filled by global_load_lds three stages ahead.  A row's 16
// chunks of 16 bytes are stored at chunk ^ 4 (row % 4): the eight rows that a
// transposing read touches lie on all banks twice instead of eight times on a
// quarter of them.
//
// Rows past the group's end are re-reads of its last row; the last stage
// clears both operands there.
#include "gemm_ring.h"
#include "train.h"

namespace moe {

namespace {

constexpr int kTile = 128, kStage = 32, kTable = 2048;

struct WArgs {
  WeightGrad g;
  int mt, nt;                  // tiles along M and N
  int per;                     // tiles of a group for each XCD
};

// Clears the values of reduction rows >= n of a fragment half (4 rows)
__device__ __forceinline__ u32x2g_t keep_rows(u32x2g_t v, int n) {
  v.x &= n >= 2 ? ~0u : (n == 1 ? 0xFFFFu : 0u);
  v.y &= n >= 4 ? ~0u : (n == 3 ? 0xFFFFu : 0u);
  return v;
}

template <bool GA, bool GB, int OUT_BF16>
__global__ __launch_bounds__(256, 2) void k_weight_grad(WArgs q) {
  // a stage: rows of a, then rows of b, 256 bytes each
  __shared__ u32x4_t l0[1024], l1[1024], l2[1024], l3[1024];
  __shared__ int32_t table[kTable];
  const WeightGrad& g = q.g;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  // workgroup b runs on XCD b % 8, which takes a run of a group's tiles; the
  // shared expert, with most rows, comes first
  const int xcd = blockIdx.x & 7, i = blockIdx.x >> 3;
  const int gi = i / q.per, tile = xcd * q.per + (i - gi * q.per);
  if (tile >= q.mt * q.nt) return;
  const bool sh = g.has_shared && gi == 0;
  const int p = gi - (g.has_shared ? 1 : 0);
  const int m0 = tile / q.nt * kTile, n0 = tile % q.nt * kTile;
  const int row0 = sh ? 0 : g.offsets[p];
  const int n = sh ? g.T : g.offsets[p + 1] - row0;
  const char* abase = (const char*)(g.a + m0);
  const char* bbase = (const char*)(g.b + n0);
  // first row of an operand that is not gathered
  const int first = sh ? g.cap : row0;
  const int r4 = lane >> 4;                         // row of a transfer
  const int chunk = ((lane & 15) ^ (r4 << 2)) * 16;
  f32x16_t acc[2][2];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int y = 0; y < 2; ++y) acc[x][y] = f32x16_t{};

  // what a lane reads of a 32-column block: row 8 (lane / 32) + 4 h + q / 4 of
  // a substep's 16, columns 16 ((lane / 16) % 2) + 4 (q % 4), q = lane % 16
  const int kr = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  auto offset = [&](int col32) {                     // (row % 4 is kr % 4)
    return kr * 256 + ((col32 * 4 + piece) ^ ((kr & 3) << 2)) * 16 + (lane & 1) * 8;
  };
  const int oa[2] = {offset(wm * 2), offset(wm * 2 + 1)};
  const int ob[2] = {8192 + offset(wn * 2), 8192 + offset(wn * 2 + 1)};
  for (int c0 = 0; c0 < n; c0 += kTable) {
    const int rows = min(n - c0, kTable), KT = (rows + kStage - 1) / kStage;
    const int32_t* from = (GA ? g.a_rows : g.b_rows) + row0 + c0;
    __syncthreads();                     // (the ring is free again)
    for (int j = threadIdx.x; j < rows; j += 256) table[j] = sh ? c0 + j : from[j];
    __syncthreads();
    auto issue = [&](int k, u32x4_t* L) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int x = w + 4 * h;                      // rows 4 x .. 4 x + 3
        const int r = min(k * kStage + 4 * x + r4, rows - 1);
        const long plain = (long)first + c0 + r;
        const long ra = GA ? table[r] : plain, rb = GB ? table[r] : plain;
        lds_dma16(abase + ra * g.lda * 2 + chunk, L + x * 64);
        lds_dma16(bbase + rb * g.ldb * 2 + chunk, L + 512 + x * 64);
      }
    };
    // left: rows from this stage on (LAST: fewer than a stage)
    auto multiply = [&](auto last_c, const u32x4_t* L, int left) {
      constexpr bool LAST = decltype(last_c)::value;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        u32x4_t fa[2], fb[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          u32x2g_t alo = lds_read_tr(L, oa[x] + s * 4096);
          u32x2g_t ahi = lds_read_tr(L, oa[x] + s * 4096 + 1024);
          u32x2g_t blo = lds_read_tr(L, ob[x] + s * 4096);
          u32x2g_t bhi = lds_read_tr(L, ob[x] + s * 4096 + 1024);
          if (LAST) {
            const int m = left - 16 * s - 8 * (lane >> 5);
            alo = keep_rows(alo, m);
            ahi = keep_rows(ahi, m - 4);
            blo = keep_rows(blo, m);
            bhi = keep_rows(bhi, m - 4);
          }
          fa[x] = u32x4_t{alo.x, alo.y, ahi.x, ahi.y};
          fb[x] = u32x4_t{blo.x, blo.y, bhi.x, bhi.y};
        }
        // (operands swapped: a lane then holds four neighbouring columns of
        // the output's row)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int y = 0; y < 2; ++y) acc[x][y] = mfma32b(fb[y], fa[x], acc[x][y]);
      }
    };
    issue(0, l0);
    issue(1, l1);
    issue(2, l2);
    // Step k: wait for this wavefront's part of stage k (8 younger transfers
    // in flight), barrier (stage k complete, stage k - 1's slot free), issue
    // stage k + 3; past the end the last rows are read again, unused.
#define WGRAD_STEP(S, L, NEXT)                                               \
    if (kt + S < KT) {                                                       \
      WAIT_VMCNT(8);                                                         \
      lds_barrier();                                                         \
      issue(kt + S + 3, NEXT);                                               \
      const int left = rows - (kt + S) * kStage;                             \
      if (left >= kStage) multiply(std::false_type{}, L, left);              \
      else multiply(std::true_type{}, L, left);                              \
    }
    for (int kt = 0; kt < KT; kt += 4) {
      WGRAD_STEP(0, l0, l3)
      WGRAD_STEP(1, l1, l0)
      WGRAD_STEP(2, l2, l1)
      WGRAD_STEP(3, l3, l2)
    }
#undef WGRAD_STEP
    WAIT_VMCNT(0);                       // the trailing re-reads have landed
  }
  __syncthreads();
  // Outputs through LDS, each wavefront's 64 x 64 in a stage's slot, so that
  // a store instruction writes whole cache lines.  acc[x][y] of a lane: row
  // 32 x + lane % 32, columns 32 y + 8 (r / 4) + 4 (lane / 32) + r % 4.
  constexpr int B = OUT_BF16 ? 2 : 4, kRow = 64 * B / 16;     // chunks a row
  u32x4_t* mine = w == 0 ? l0 : w == 1 ? l1 : w == 2 ? l2 : l3;
  const int second = n0 >= g.N0 ? 1 : 0;
  char* out = (char*)(sh ? g.out_shared[second]
                         : (char*)g.out[second] + (size_t)p * g.M * g.N0 * B);
  out += ((size_t)(m0 + wm * 64) * g.N0 + (n0 - second * g.N0) + wn * 64) * B;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int row = 32 * x + (lane & 31);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f32x16_t& v = acc[x][y];
        const int col = 32 * y + 8 * r + 4 * (lane >> 5);
        if constexpr (OUT_BF16) {
          const u32x2g_t o = {(uint32_t)f32_to_bf16(v[4 * r]) | (uint32_t)f32_to_bf16(v[4 * r + 1]) << 16,
                              (uint32_t)f32_to_bf16(v[4 * r + 2]) | (uint32_t)f32_to_bf16(v[4 * r + 3]) << 16};
          const int c = (col >> 3) ^ (row & (kRow - 1));
          ((u32x2g_t*)(mine + row * kRow + c))[(col >> 2) & 1] = o;
        } else {
          const int c = (col >> 2) ^ (row & (kRow - 1));
          ((f32x4_t*)mine)[row * kRow + c] = f32x4_t{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
        }
      }
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < kRow; ++j) {
    const int at = j * 64 + lane, row = at / kRow, c = at & (kRow - 1);
    const u32x4_t v = mine[row * kRow + (c ^ (row & (kRow - 1)))];
    __builtin_nontemporal_store(v, (u32x4_t*)(out + (size_t)row * g.N0 * B) + c);
  }
}

}  // namespace

hipError_t launch_weight_grad(const WeightGrad& g, hipStream_t s) {
  WArgs q{};
  q.g = g;
  q.mt = g.M / kTile;
  q.nt = g.N / kTile;
  q.per = (q.mt * q.nt + 7) / 8;
  const int groups = g.P + (g.has_shared ? 1 : 0);
  const unsigned grid = (unsigned)groups * (unsigned)q.per * 8u;
  const bool bf16 = g.dtype == MOE_BF16;
  if (g.a_rows) {
    if (bf16) k_weight_grad<true, false, 1><<<grid, 256, 0, s>>>(q);
    else k_weight_grad<true, false, 0><<<grid, 256, 0, s>>>(q);
  } else {
    if (bf16) k_weight_grad<false, true, 1><<<grid, 256, 0, s>>>(q);
    else k_weight_grad<false, true, 0><<<grid, 256, 0, s>>>(q);
  }
  return hipGetLastError();
}

}  // namespace moe
