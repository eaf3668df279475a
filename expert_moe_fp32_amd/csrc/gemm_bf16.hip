// Prefill-shaped grouped bf16 GEMM for the expert FFN -- gate/up with the
// fused SiLU epilogue, and down -- on the packed operand layout of ffn.hip.
//
// Work item = (tile of <= 256 rows of one group, 128 gate + 128 up columns,
// or 256 down columns).
// A workgroup of 8 wavefronts (2 x 4) computes 256 x 256 B-columns:
// wavefront (wm, wn) owns 128 rows x 64 columns = 4 x 2 MFMA blocks of
// 32 x 32 (128 fp32 accumulators per lane, two wavefronts per SIMD).  The
// reduction runs in 32-wide stages through LDS filled by
// global_load_lds_dwordx4 (each lane's 16 bytes land at the transfer's base
// + 16 * lane, so no registers stage the copy): B in a ring of 4 stages of 16
// column blocks of 1 KiB, A in 2 slots of a stage pair, where one transfer
// moves 8 whole 128-byte row segments (64 K), each read by 8 consecutive
// lanes, so every group of 8 lanes touches one cache line (lanes spread over
// 8 lines per group ran gate/up 6 % slower, 16 rows x 64 bytes slower
// still).  Every fragment read is one conflict-free ds_read_b128.  One
// barrier per stage; the DMA runs two to three stages ahead, and the
// fragments one stage ahead in registers, so after its barrier a stage's
// MFMAs start at once while its transfers and the next stage's reads are
// issued between them (gate/up 6 %, down 7 % faster than reading each
// stage's fragments after its barrier).
//
// Placement: workgroups are dealt round-robin to the 8 XCDs (workgroup b on
// XCD b % 8), and a round of the persistent loop gives each XCD a chunk of
// 32 items that run together and share operands through that XCD's L2: TG
// consecutive tiles x CB column blocks (TG x CB = 32).  A tile's A rows and
// a column block's weights are about the same size at these shapes (256
// rows or 256 columns over the same K), so a squarer chunk misses less:
// gate/up 4 tiles x 8 blocks, down 8 tiles x 4 blocks (prefill down 524 ->
// 488 us and 24 % fewer L2 misses than one tile's 28 blocks a chunk; gate/up,
// 7 % fewer misses at the same time, is bound by its issue rate rather than
// by these misses).
#include "gemm_ring.h"

namespace moe {

int gemm_tile_rows() { return kGemmRows; }

hipError_t launch_gemm_bf16_gateup(const FfnArgs& f, hipStream_t s) {
  const moe_weights* w = f.w;
  GArgs a{};
  a.tiles = f.tiles;
  a.tile_count = f.tile_count;
  a.P = f.P;
  a.cap = f.cap;
  a.K = f.H;
  a.N = f.I;
  a.a_routed = (const bf16_t*)f.a_routed;
  a.a_rows = f.a_rows;
  a.a_shared = (const bf16_t*)f.a_shared;
  a.w0_arr = w->w_gate;
  a.w1_arr = w->w_up;
  a.w0_sh = w->sh_gate;
  a.w1_sh = w->sh_up;
  a.h_out = (bf16_t*)f.h;
  a.nb_per_tile = a.N / (16 * kGemmTN * kGemmWN);  // 32 TN WN B-columns
  a.chunk_cols = chunk_cols(a.nb_per_tile, 8);     // 4 tiles x 8 blocks
  // persistent: one workgroup per CU (128 KiB of LDS)
  k_gemm_bf16<G_GATEUP, kGemmTM, kGemmTN, kGemmWM, kGemmWN>
      <<<256, 64 * kGemmWM * kGemmWN, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_gemm_bf16_down(const FfnArgs& f, hipStream_t s) {
  const moe_weights* w = f.w;
  GArgs a{};
  a.tiles = f.tiles;
  a.tile_count = f.tile_count;
  a.P = f.P;
  a.cap = f.cap;
  a.K = f.I;
  a.N = f.H;
  a.a_routed = (const bf16_t*)f.h;
  a.a_rows = nullptr;
  a.a_shared = (const bf16_t*)f.h + (size_t)f.cap * f.I;
  a.w0_arr = w->w_down;
  a.w1_arr = nullptr;
  a.w0_sh = w->sh_down;
  a.w1_sh = nullptr;
  a.y_routed = f.y_routed;
  a.y_shared = f.y_shared;
  a.nb_per_tile = a.N / (32 * kGemmTN * kGemmWN);  // 32 TN WN outputs
  a.chunk_cols = chunk_cols(a.nb_per_tile, 4);     // 8 tiles x 4 blocks
  k_gemm_bf16<G_DOWN, kGemmTM, kGemmTN, kGemmWM, kGemmWN>
      <<<256, 64 * kGemmWM * kGemmWN, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace moe
