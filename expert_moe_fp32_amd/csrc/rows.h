// Rows of a token held in a workgroup's registers: loads and stores of W
// neighbouring columns a thread, and sums over a row.
//
// A thread's piece of a pass is one access of 8 or 16 bytes, and a
// wavefront's accesses are contiguous: W = 8 where every row array is bf16,
// else W = 4 (a float32 array read as two 16-byte halves of 8 columns touches
// each cache line from two instructions, which with non-temporal loads fetched
// lines twice: combine + norm of 8192 x 7168 176 us against 164 us without
// the hint).
#pragma once

#include "common.h"

namespace moe {

typedef __attribute__((ext_vector_type(8))) float f32x8_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2v_t;

template <int W>
struct ColsOf;
template <>
struct ColsOf<4> {
  typedef f32x4_t F;
  typedef __attribute__((ext_vector_type(4))) __bf16 B;
};
template <>
struct ColsOf<8> {
  typedef f32x8_t F;
  typedef __attribute__((ext_vector_type(8))) __bf16 B;
};
template <int W>
using Cols = typename ColsOf<W>::F;

// W columns as they are stored: 8 or 16 bytes
template <int BYTES>
struct RawOf;
template <>
struct RawOf<8> {
  typedef u32x2v_t V;
  typedef u32x2v_t Any __attribute__((aligned(2)));
};
template <>
struct RawOf<16> {
  typedef u32x4_t V;
  typedef u32x4_t Any __attribute__((aligned(2)));
};
template <typename T, int W>
using Raw = typename RawOf<W * (int)sizeof(T)>::V;

// How a row of H columns lies over the pieces of its threads.
//   kExact    every piece is whole and aligned to its size
//   kAligned  pieces are aligned, and those past the row's end read as zero
//   kAny      rows at the alignment of their element type; the last piece may
//             be cut
enum Fit { kAny, kAligned, kExact };

// Where a thread's piece is read: at `at`, the piece's column or, past the
// row's last whole piece, the columns that end the row, `past` further left.
// So every load is unconditional and in bounds (rows of fewer than W columns
// apart, which read their columns one by one).
struct Piece {
  int col, at, past;
};
template <int W, Fit FIT>
__device__ __forceinline__ Piece piece_at(int col, int H) {
  Piece p;
  p.col = col;
  p.at = FIT == kExact ? col : min(col, max(H - W, 0));
  p.past = FIT == kExact ? 0 : col - p.at;
  return p;
}

template <typename T, int W, Fit FIT, bool NT>
__device__ __forceinline__ Raw<T, W> load_piece(const T* row, Piece c, int H) {
  typedef RawOf<W * (int)sizeof(T)> R;
  const T* p = row + c.at;
  if constexpr (FIT != kAny) {
    if constexpr (NT) return __builtin_nontemporal_load((const typename R::V*)p);
    else return *(const typename R::V*)p;
  } else {
    if (H < W) {
      Raw<T, W> r = 0u;
#pragma unroll
      for (int i = 0; i < W; ++i) {
        if (i < H) {
          if constexpr (sizeof(T) == 2) r[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
          else r[i] = __float_as_uint(p[i]);
        }
      }
      return r;
    }
    return *(const typename R::Any*)p;
  }
}

// A loaded piece's own columns: shifted down by `past` of them, zeros behind.
template <typename T, int W, Fit FIT>
__device__ __forceinline__ Raw<T, W> own_cols(Raw<T, W> r, Piece c) {
  if constexpr (FIT == kExact) return r;
  if constexpr (FIT == kAligned) return c.past > 0 ? Raw<T, W>(0u) : r;
  if constexpr (FIT == kAny) {
    constexpr int D = W * (int)sizeof(T) / 4;       // words
    int words = c.past;                             // to shift by
    if constexpr (sizeof(T) == 2) {
      words = c.past >> 1;
      if (c.past & 1) {
#pragma unroll
        for (int i = 0; i < D; ++i) r[i] = (r[i] >> 16) | (i + 1 < D ? r[i + 1] << 16 : 0u);
      }
    }
#pragma unroll
    for (int s = 1; s < D; s <<= 1) {
      if (words & s) {
#pragma unroll
        for (int i = 0; i < D; ++i) r[i] = i + s < D ? r[i + s] : 0u;
      }
    }
    return words >= D ? Raw<T, W>(0u) : r;
  }
}

template <typename T, int W>
__device__ __forceinline__ Cols<W> widen(Raw<T, W> r) {
  Cols<W> v;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      v[2 * i] = __uint_as_float(r[i] << 16);
      v[2 * i + 1] = __uint_as_float(r[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __uint_as_float(r[i]);
  }
  return v;
}

// Stores a piece; of a cut one the columns that the row has.  bf16 rounds to
// nearest even, as the hardware converts.
template <typename T, int W, Fit FIT, bool NT>
__device__ __forceinline__ void store_piece(T* row, Piece c, int H, Cols<W> v) {
  typedef RawOf<W * (int)sizeof(T)> R;
  Raw<T, W> r;
  if constexpr (sizeof(T) == 2) {
    r = __builtin_bit_cast(typename R::V, __builtin_convertvector(v, typename ColsOf<W>::B));
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) r[i] = __float_as_uint(v[i]);
  }
  T* p = row + c.col;
  if (FIT == kExact || c.col + W <= H) {
    if constexpr (FIT == kAny) *(typename R::Any*)p = r;
    else if constexpr (NT) __builtin_nontemporal_store(r, (typename R::V*)p);
    else *(typename R::V*)p = r;
  } else if (FIT == kAny && c.col < H) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if (c.col + i < H) {
        if constexpr (sizeof(T) == 2) p[i] = (bf16_t)(r[i >> 1] >> (16 * (i & 1)));
        else p[i] = __uint_as_float(r[i]);
      }
    }
  }
}

// the same for an array whose type is known at run time
template <int W, Fit FIT, bool NT>
__device__ __forceinline__ void store_piece_as(int dtype, void* rows, size_t row,
                                               Piece c, int H, Cols<W> v) {
  if (dtype == MOE_BF16) store_piece<bf16_t, W, FIT, NT>((bf16_t*)rows + row, c, H, v);
  else if constexpr (W == 4) store_piece<float, W, FIT, NT>((float*)rows + row, c, H, v);
}

// W columns of a float32 vector, zeros past its end
template <int W, Fit FIT>
__device__ __forceinline__ Cols<W> load_f32(const float* row, Piece c, int H) {
  Cols<W> v;
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const Piece h = piece_at<4, FIT>(c.col + i, H);
    const f32x4_t f = widen<float, 4>(own_cols<float, 4, FIT>(load_piece<float, 4, FIT, false>(row, h, H), h));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[i + k] = f[k];
  }
  return v;
}

// a gain's W values plus its offset, at any alignment and of either type;
// past the row's end the offset
template <int W>
__device__ __forceinline__ Cols<W> load_gain(const void* g, int dtype, int col,
                                             int H, float offset) {
  const Piece c = piece_at<W, kAny>(col, H);
  if (dtype == MOE_BF16)
    return widen<bf16_t, W>(own_cols<bf16_t, W, kAny>(load_piece<bf16_t, W, kAny, false>((const bf16_t*)g, c, H), c)) + offset;
  return load_f32<W, kAny>((const float*)g, c, H) + offset;
}

template <int W>
__device__ __forceinline__ float dot_cols(Cols<W> a, Cols<W> b) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) s = __builtin_fmaf(a[i], b[i], s);
  return s;
}

template <int CTRL, int ROWS>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(
                 0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}

// sum over the 16 lanes of a DPP row, in each of them
__device__ __forceinline__ float sum16(float v) {
  v = add_dpp<0x128, 0xF>(v);          // row rotations by 8, 4, 2, 1
  v = add_dpp<0x124, 0xF>(v);
  v = add_dpp<0x122, 0xF>(v);
  return add_dpp<0x121, 0xF>(v);
}

// sum over a wavefront, the same in every lane: row broadcasts carry the rows'
// sums on to lane 63
__device__ __forceinline__ float wave_sum(float v) {
  v = sum16(v);
  v = add_dpp<0x142, 0xA>(v);
  v = add_dpp<0x143, 0xC>(v);
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Sums of N values over a row's `waves` <= 16 wavefronts, the first of which
// is `first`; the same value in every thread of the row.  `buf` holds 16 x N
// floats and is written again only after another barrier.  All in DPP steps:
// shuffles through LDS took a third of the gradient kernel's row.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* buf, int first,
                                        int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) buf[i * 16 + wv] = v[i];
  }
  lds_barrier();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float p = lane < waves ? buf[i * 16 + first + lane] : 0.0f;
    v[i] = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(sum16(p))));
  }
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// rows whose pieces are whole and aligned at W columns
inline bool rows_aligned(const void* p, int dtype, int64_t stride, int W) {
  const int bytes = W * (dtype == MOE_BF16 ? 2 : 4);
  return !p || ((uintptr_t)p % bytes == 0 && stride % W == 0);
}

template <class F>
void by_type(int dtype, F f) {
  if (dtype == MOE_BF16) f(bf16_t{});
  else f(float{});
}

template <class F>
void by_flag(bool b, F f) {
  if (b) f(std::true_type{});
  else f(std::false_type{});
}

}  // namespace moe
