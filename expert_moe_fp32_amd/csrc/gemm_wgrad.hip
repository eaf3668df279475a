// Weight gradients of the experts: for every group of rows (a physical
// expert's, or the shared expert's) out = a^T b, reduced over the group's
// rows, for two products at once: the layer's input with the gradients of gate
// and up, and the weighted h with the gradient of the layer's output.
//
// A tile is 256 x 256 outputs of one group and product; a workgroup of 8
// wavefronts (2 x 4 of 128 x 64) has a CU to itself and goes from tile to
// tile.  At some hundred rows a group the outputs are most of the traffic, so
// nothing may drain between tiles: the reduction of all of a workgroup's
// tiles is one stream of stages (32 rows x (256 + 256) columns, 32 KiB) through
// a ring of four LDS slots, filled by global_load_lds four stages ahead across
// the tiles' borders, and a tile's stores are in flight while the next one
// multiplies (the vector-memory counter is in order, so the waits of its first
// steps allow for the stores).
//
// Both operands lie row by row, the reduction first, so the MFMA operands
// (eight reduction values of one column a lane) come out of LDS by transposing
// reads.  A row's 32 chunks of 16 bytes are stored at chunk ^ 4 (row % 4): the
// eight rows that a transposing read touches then lie on all banks twice
// instead of eight times on a quarter of them.
//
// Rows past a group's end are read from an array of zeros; a group's stages
// are rounded up to four (the slots' names are fixed in the code).
//
// Each XCD takes a run of tiles of equal cost, its 32 workgroups 32
// neighbouring tiles (4 x 8) at a time, which share their operands in its L2.
// The cost is a group's stages and little for the outputs, whose traffic other
// XCDs' products hide (4096 x 7168 x 2048, 32 of 256 experts and the shared
// one: 1.16 ms; outputs counted as 14 stages 1.89 ms; an eighth of every group
// to each XCD 1.16, and 64 uneven groups of 2048 x 768 294 instead of 253 us).
#include "checkpoint.h"
#include "gemm_ring.h"
#include "train.h"

namespace moe {

namespace {

constexpr int kTile = 256, kStage = 32;
constexpr int kSlots = 32;       // workgroups of an XCD
constexpr int kStrip = 4;        // tiles along M that a column of tiles takes

struct WArgs {
  WeightGrad g;
  int mt[2], nt[2];              // tiles along M and N of a product
  uint32_t inv_strip[2];         // 2^32 / (kStrip nt), rounded up
  int per_group;                 // tiles of a group
  int groups;
  int store_cost;                // of a tile's outputs, in stages
};

typedef const __attribute__((address_space(4))) int32_t* ConstInt;

// A row of zeros, for the rows past a group's end.
__device__ const u32x4_t kZeroRow[32] = {};

__device__ __forceinline__ int stages_of(int rows) {
  return rows <= 4 * kStage ? 4 : (rows + 4 * kStage - 1) / (4 * kStage) * 4;
}

template <int OUT_BF16>
__global__ __launch_bounds__(512) void k_weight_grad(WArgs q) {
  // a stage: 32 rows of a, then of b, 512 bytes each
  __shared__ u32x4_t l0[2048], l1[2048], l2[2048], l3[2048];
  __shared__ u32x4_t stage[8 * 256];
  const WeightGrad& g = q.g;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 2, wn = w & 3;
  const ConstInt offsets = (ConstInt)g.offsets;
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  const int shared = g.has_shared ? 1 : 0;       // group 0, then the experts
  // ---- this XCD's run of tiles: the cost of all groups, cut in eight
  int first_tile, last_tile;
  {
    const int each = (q.groups + 63) / 64;
    const int g0 = min(lane * each, q.groups), g1 = min(g0 + each, q.groups);
    long mine = 0;
    for (int i = g0; i < g1; ++i) {
      const int n = i < shared ? g.T : g.offsets[i - shared + 1] - g.offsets[i - shared];
      mine += (long)(stages_of(n) + q.store_cost) * q.per_group;
    }
    long upto = mine;                            // inclusive over the lanes
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const long o = __shfl_up(upto, d, 64);
      if (lane >= d) upto += o;
    }
    const long total = __shfl(upto, 63, 64);
    auto cut = [&](int x) -> int {
      const long target = total * x / 8;
      if (x == 8) return q.groups * q.per_group;
      // the lane whose groups hold the target, then the group, then the tile
      int tile = 0;
      const int owner = __ffsll((unsigned long long)__ballot(upto > target)) - 1;
      if (lane == owner) {
        long at = upto - mine;
        for (int i = g0; i < g1; ++i) {
          const int n = i < shared ? g.T : g.offsets[i - shared + 1] - g.offsets[i - shared];
          const long c = stages_of(n) + q.store_cost;
          if (at + c * q.per_group > target) {
            tile = i * q.per_group + (int)((target - at + c / 2) / c);
            break;
          }
          at += c * q.per_group;
        }
      }
      return __builtin_amdgcn_readlane(tile, owner);
    };
    first_tile = cut(xcd);
    last_tile = cut(xcd + 1);
  }
  const int f0 = first_tile + slot;
  if (f0 >= last_tile) return;

  // ---- where a tile's operands are
  struct Tile {
    int group, i, product, m0, n0, n, row0, stages;   // i: of its group's
  };
  auto rows_at = [&](Tile& t) {
    const bool sh = t.group < shared;
    const int e = sh ? 0 : t.group - shared;
    const int begin = offsets[e], end = offsets[e + 1];
    t.row0 = sh ? 0 : begin;
    t.n = sh ? g.T : end - begin;
    t.stages = stages_of(t.n);
  };
  // strips of kStrip tiles along M, column by column
  auto place = [&](Tile& t) {
    const int first = q.mt[0] * q.nt[0];
    t.product = t.i >= first ? 1 : 0;
    const int i = t.product ? t.i - first : t.i;
    const int mt = t.product ? q.mt[1] : q.mt[0], nt = t.product ? q.nt[1] : q.nt[0];
    const int strip = (int)__umulhi((uint32_t)i, t.product ? q.inv_strip[1] : q.inv_strip[0]);
    const int j = i - strip * kStrip * nt, high = min(kStrip, mt - strip * kStrip);
    // j / high for high of 1 to 4, j below 2^15
    const uint32_t inv = high == 4 ? 16384u : high == 3 ? 21846u : high == 2 ? 32768u : 65536u;
    const int col = (int)((uint32_t)j * inv >> 16);
    t.n0 = col * kTile;
    t.m0 = (strip * kStrip + j - col * high) * kTile;
  };
  auto next_tile = [&](Tile& t) {
    t.i += kSlots;
    if (t.i >= q.per_group) {
      do {
        t.i -= q.per_group;
        ++t.group;
      } while (t.i >= q.per_group);
      rows_at(t);
    }
    place(t);
  };
  // ---- the stream of stages, as it is read
  const int half = lane >> 5, c32 = lane & 31;
  // a lane's 16 bytes of a row: where the row's other half lies past the
  // operand's columns, the first half's again
  const int chunk = c32 ^ (((w & 1) * 2 + half) << 2);
  Tile in;                               // the tile read
  in.group = f0 / q.per_group;
  in.i = f0 - in.group * q.per_group;
  rows_at(in);
  place(in);
  Tile t = in;                           // the tile multiplied
  int in_f = f0, in_k = 0;
  // A lane's bytes of row 2 w + half of the next stage, and that row's number
  // in the group (its second row is 16 further); the bytes of 16 rows.
  const char *a_row, *b_row;
  size_t a_16, b_16;
  int row;
  auto open = [&]() {
    const WeightProduct& p = g.product[in.product];
    const bool sh = in.group < shared;
    const int a_off = (in.m0 + kTile > p.M ? chunk & 15 : chunk) * 16;
    const int b_off = (in.n0 + kTile > p.N ? chunk & 15 : chunk) * 16;
    row = 2 * w + half;
    a_16 = (size_t)p.lda * 32;
    b_16 = (size_t)p.ldb * 32;
    a_row = (const char*)((sh ? p.a_shared : p.a) + (size_t)(in.row0 + row) * p.lda + in.m0) + a_off;
    b_row = (const char*)((sh ? p.b_shared : p.b) + (size_t)(in.row0 + row) * p.ldb + in.n0) + b_off;
  };
  const char* const zeros = (const char*)kZeroRow + c32 * 16;
  const char *a_at[2], *b_at[2];         // what the next transfers read
  auto aim = [&]() {
    a_at[0] = row < in.n ? a_row : zeros;
    b_at[0] = row < in.n ? b_row : zeros;
    a_at[1] = row + 16 < in.n ? a_row + a_16 : zeros;
    b_at[1] = row + 16 < in.n ? b_row + b_16 : zeros;
  };
  auto issue = [&](u32x4_t* L) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      lds_dma16(a_at[h], L + (w + 8 * h) * 64);
      lds_dma16(b_at[h], L + 1024 + (w + 8 * h) * 64);
    }
  };
  // to the next stage, of the next tile behind a tile's last; past the end of
  // all the last stage again
  auto advance = [&]() {
    if (++in_k == in.stages) {
      if (in_f + kSlots < last_tile) {
        in_f += kSlots;
        next_tile(in);
        in_k = 0;
        open();
      } else {
        --in_k;
      }
    } else {
      row += kStage;
      a_row += 2 * a_16;
      b_row += 2 * b_16;
    }
    aim();
  };

  // what a lane reads of a 32-column block: row 8 (lane / 32) + 4 h + q / 4 of
  // a substep's 16, columns 16 ((lane / 16) % 2) + 4 (q % 4), q = lane % 16
  const int kr = 8 * (lane >> 5) + ((lane & 15) >> 2);
  const int piece = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
  int oa[4], ob[2];
#pragma unroll
  for (int x = 0; x < 4; ++x)
    oa[x] = kr * 512 + (((wm * 4 + x) * 4 + piece) ^ ((kr & 3) << 2)) * 16 + (lane & 1) * 8;
#pragma unroll
  for (int y = 0; y < 2; ++y)
    ob[y] = 16384 + kr * 512 + (((wn * 2 + y) * 4 + piece) ^ ((kr & 3) << 2)) * 16 + (lane & 1) * 8;

  f32x16_t acc[4][2];
  u32x4_t fa0[2][4], fb0[2][2], fa1[2][4], fb1[2][2];
  auto load = [&](const u32x4_t* L, u32x4_t (&fa)[2][4], u32x4_t (&fb)[2][2]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const u32x2g_t lo = lds_read_tr(L, ob[y] + s * 8192);
        const u32x2g_t up = lds_read_tr(L, ob[y] + s * 8192 + 2048);
        fb[s][y] = u32x4_t{lo.x, lo.y, up.x, up.y};
      }
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const u32x2g_t lo = lds_read_tr(L, oa[x] + s * 8192);
        const u32x2g_t up = lds_read_tr(L, oa[x] + s * 8192 + 2048);
        fa[s][x] = u32x4_t{lo.x, lo.y, up.x, up.y};
      }
    }
  };
  // (operands swapped: a lane then holds four neighbouring columns of an
  // output row)
  auto mma = [&](auto first_c, const u32x4_t (&fa)[2][4], const u32x4_t (&fb)[2][2]) {
    constexpr bool FIRST = decltype(first_c)::value;   // of a tile
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y)
          acc[x][y] = mfma32b(fb[s][y], fa[s][x], FIRST && s == 0 ? f32x16_t{} : acc[x][y]);
  };
  open();
  aim();
  issue(l0);
  advance();
  issue(l1);
  advance();
  issue(l2);
  advance();
  issue(l3);
  advance();
  WAIT_VMCNT(0);                         // (all four: the first steps' waits
  lds_barrier();                         // allow for stores that are not there)
  load(l0, fa0, fb0);
  constexpr int B = OUT_BF16 ? 2 : 4;
  constexpr int kStores = OUT_BF16 ? 16 : 32;    // of a tile, per wavefront
  // Step of stage k, in the slot CUR, from registers: wait for stage k + 1 (two
  // younger stages in flight, and in a tile's first three steps the last
  // tile's stores between them), barrier (stage k + 1 complete, stage k's slot
  // free), read stage k + 4 into it, and multiply while stage k + 1 is read
  // into the other registers.
#define WGRAD_STEP(FIRST, YOUNGER, CUR, NEXT, FA, FB, GA, GB)                \
    {                                                                        \
      WAIT_VMCNT(YOUNGER);                                                   \
      lds_barrier();                                                         \
      __builtin_amdgcn_sched_barrier(0);                                     \
      issue(CUR);                                                            \
      load(NEXT, GA, GB);                                                    \
      mma(std::bool_constant<FIRST>{}, FA, FB);                              \
      interleave<4, 16, 24>();                                               \
      __builtin_amdgcn_sched_barrier(0);                                     \
      advance();                                                             \
    }
  // (offsets through opaque moves: shared between the copies of a slot's
  // reads, their addresses lose which slot is read, and the compiler waits for
  // every transfer)
  auto anew = [&]() {
#pragma unroll
    for (int x = 0; x < 4; ++x) asm volatile("" : "+v"(oa[x]));
#pragma unroll
    for (int y = 0; y < 2; ++y) asm volatile("" : "+v"(ob[y]));
  };
#define WGRAD_QUAD(FIRST, YOUNGER)                                           \
    anew();                                                                  \
    WGRAD_STEP(FIRST, YOUNGER, l0, l1, fa0, fb0, fa1, fb1)                   \
    WGRAD_STEP(false, YOUNGER, l1, l2, fa1, fb1, fa0, fb0)                   \
    WGRAD_STEP(false, YOUNGER, l2, l3, fa0, fb0, fa1, fb1)                   \
    WGRAD_STEP(false, 8, l3, l0, fa1, fb1, fa0, fb0)
  for (int f = f0;;) {
    WGRAD_QUAD(true, 8 + kStores)
    for (int k = 4; k < t.stages; k += 4) { WGRAD_QUAD(false, 8) }
    // Outputs through the wavefront's own LDS, so that a store instruction
    // writes whole cache lines.  acc[x][y] of a lane: row 32 x + lane % 32,
    // columns 32 y + 8 (r / 4) + 4 (lane / 32) + r % 4.
    const WeightProduct& p = g.product[t.product];
    // (past an operand's columns its first half was read again: those
    // wavefronts hold, and store, the same outputs as the first half's)
    const int m = t.m0 + (t.m0 + wm * 128 < p.M ? wm * 128 : 0);
    const int col = t.n0 + (t.n0 + wn * 64 < p.N ? wn * 64 : wn * 64 - 128);
    const int second = col >= p.N0 ? 1 : 0;
    char* out;                           // (uniform; lanes add 32 bits)
    if (t.group < shared) out = (char*)p.out_shared[second];
    else out = (char*)p.out[second] + (size_t)(t.group - shared) * p.M * p.N0 * B;
    out += ((size_t)m * p.N0 + (col - second * p.N0)) * B;
    u32x4_t* st = stage + w * 256;
    // (the lane through an opaque move, so that the addresses are formed here
    // and not held through the multiplications)
    int le;
    asm volatile("v_mov_b32 %0, %1" : "=v"(le) : "v"(lane));
    const int mine = le & 31, swz = mine & 7, hi = le >> 5;
    // reading back: lane's row of eight, and its chunk of the row
    const int back = (le >> 3) * 8 + ((le & 7) ^ (le >> 3));
    const uint32_t to = (uint32_t)(le >> 3) * (uint32_t)(p.N0 * B) + (le & 7) * 16;
    const size_t eight = (size_t)8 * p.N0 * B;       // bytes of eight rows
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if constexpr (OUT_BF16) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f32x16_t& v = acc[x][y];
            const u32x2g_t o = {pack_bf16(v[4 * r], v[4 * r + 1]), pack_bf16(v[4 * r + 2], v[4 * r + 3])};
            ((u32x2g_t*)(st + mine * 8 + ((4 * y + r) ^ swz)))[hi] = o;
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < 4; ++j)
          __builtin_nontemporal_store(st[back + j * 64],
                                      (u32x4_t*)(out + (4 * x + j) * eight + to));
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      } else {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const f32x16_t& v = acc[x][y];
            ((f32x4_t*)st)[mine * 8 + ((2 * r + hi) ^ swz)] =
                f32x4_t{v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int j = 0; j < 4; ++j)
            __builtin_nontemporal_store(
                st[back + j * 64],
                (u32x4_t*)(out + (4 * x + j) * eight + 32 * y * B + to));
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          __builtin_amdgcn_wave_barrier();
        }
      }
    }
    f += kSlots;
    if (f >= last_tile) break;
    next_tile(t);
  }
#undef WGRAD_QUAD
#undef WGRAD_STEP
  WAIT_VMCNT(0);                         // the trailing re-reads have landed
}

}  // namespace

hipError_t launch_weight_grad(const WeightGrad& g, hipStream_t s) {
  WArgs q{};
  q.g = g;
  q.groups = g.P + (g.has_shared ? 1 : 0);
  for (int i = 0; i < 2; ++i) {
    q.mt[i] = (g.product[i].M + kTile - 1) / kTile;
    q.nt[i] = (g.product[i].N + kTile - 1) / kTile;
  }
  for (int i = 0; i < 2; ++i)
    q.inv_strip[i] = (uint32_t)((0x100000000ull + kStrip * q.nt[i] - 1) / (kStrip * q.nt[i]));
  q.per_group = q.mt[0] * q.nt[0] + q.mt[1] * q.nt[1];
  q.store_cost = g.dtype == MOE_BF16 ? 1 : 2;
  if (g.dtype == MOE_BF16) k_weight_grad<1><<<8 * kSlots, 512, 0, s>>>(q);
  else k_weight_grad<0><<<8 * kSlots, 512, 0, s>>>(q);
  return hipGetLastError();
}

}  // namespace moe
