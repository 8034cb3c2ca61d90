// Tiles staged through registers: operands of any alignment and length, fp32
// and bf16, with the MFMA operands read from them.
#pragma once
#include "expert_tiles.hpp"
#include "mfma_nt.hpp"

namespace muon {
namespace ex {

using nt::bf16x8_t;
using nt::f32x16_t;
using nt::s16x4_t;
using nt::u32x2_t;

// Tile geometry of one type.  An operand's tile has `B` rows of BK elements
// (k-contiguous) or BK rows of B elements (k-major), cut into 16-byte chunks.
template <class T>
struct Tile;
template <>
struct Tile<bf16_t> {
  static constexpr int B = 128, SH = 7, BK = 64, PER = 8;   // PER: elements a chunk
  // 128-byte rows of swizzled chunks, as nt::load_frags reads them
  static __device__ __forceinline__ int at(int r, int c) { return r * 128 + ((c ^ nt::swz<128>(r)) << 4); }
  // 256-byte rows, as nt::load_frags_qt reads them
  static __device__ __forceinline__ int at_t(int r, int c) { return r * 256 + ((c ^ nt::swzt(r)) << 4); }
  static constexpr int BYTES = 128 * 128, BYTES_T = 64 * 256;
};
template <>
struct Tile<float> {
  static constexpr int B = 64, SH = 6, BK = 32, PER = 4;
  // rows padded by 16 bytes: 16-byte reads down 8 rows hit 8 bank groups
  static __device__ __forceinline__ int at(int r, int c) { return r * 144 + (c << 4); }
  static __device__ __forceinline__ int at_t(int r, int c) { return r * 272 + (c << 4); }
  static constexpr int BYTES = 64 * 144, BYTES_T = 32 * 272;
};

// One operand's way from memory to its tile through registers: any alignment,
// any length, rows that do not exist read as zero.
template <class T, bool KM>
struct Stager {
  using G = Tile<T>;
  static constexpr int CPR = KM ? G::B / G::PER : G::BK / G::PER;   // chunks a row
  static constexpr int ROWS = KM ? G::BK : G::B;
  static constexpr int NC = ROWS * CPR / 256;                       // chunks a thread
  const T* base;
  const int32_t* gather;
  int64_t row0, rows, src_rows;   // first source row, rows from there on, rows that gather may name
  int64_t ld;
  int32_t col0, cols;             // k-major: first column, row length; else: row length
  int64_t idx[NC];                // k-contiguous: source row of each chunk (-1: none)
  u32x4 v[NC];

  __device__ __forceinline__ int64_t source(int64_t r) const {
    if (r >= rows) return -1;
    if (!gather) return row0 + r;
    const int32_t g = gather[row0 + r];
    return g >= 0 && g < src_rows ? g : -1;
  }
  __device__ __forceinline__ void init(const void* b, const int32_t* g, int64_t r0, int64_t n_rows, int64_t sr,
                                       int32_t c0, int32_t n_cols) {
    base = static_cast<const T*>(b);
    gather = g;
    row0 = r0;
    rows = n_rows;
    src_rows = sr;
    ld = n_cols;
    col0 = c0;
    cols = n_cols;
    if (!KM) {
#pragma unroll
      for (int u = 0; u < NC; ++u) idx[u] = source((u * 256 + (int)threadIdx.x) / CPR);
    }
  }
  __device__ __forceinline__ void fetch(int64_t k0) {
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int id = u * 256 + (int)threadIdx.x, r = id / CPR, c = id % CPR;
      const int64_t src = KM ? source(k0 + r) : idx[u];
      const int64_t col = (KM ? (int64_t)col0 : k0) + c * G::PER;
      const int64_t left = cols - col;
      v[u] = src < 0 || left <= 0 ? u32x4{0u, 0u, 0u, 0u}
                                  : load16(base + src * ld + col, left < G::PER ? (int)left : G::PER);
    }
  }
  __device__ __forceinline__ void commit(char* lds) const {
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int id = u * 256 + (int)threadIdx.x, r = id / CPR, c = id % CPR;
      *reinterpret_cast<u32x4*>(lds + (KM ? G::at_t(r, c) : G::at(r, c))) = v[u];
    }
  }
};

// MFMA operands of one k-group (16 k of bf16, 8 of fp32) for the NT 32-wide
// slabs from `first` on.  Both operands of a product take the k values of a
// group in the same order, so their order does not matter.
template <bool KM, int NT>
__device__ __forceinline__ void fragments(u32x4 (&f)[NT], const char* lds, int first, int kg, int lane, bf16_t) {
  if constexpr (!KM) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      f[j] = *reinterpret_cast<const u32x4*>(lds + Tile<bf16_t>::at(first + 32 * j + (lane & 31), kg * 2 + (lane >> 5)));
  } else {
    // nt::load_frags_qt describes the transposing read
    const int g = lane >> 4, sl = lane & 15;
    const int k = kg * 16 + 8 * (g >> 1) + (sl >> 2);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int byte = (first + 32 * j + (g & 1) * 16 + 4 * (sl & 3)) * 2;
      const int a = ((byte >> 4) ^ nt::swzt(k)) * 16 + (byte & 15);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS s16x4_t*)(lds + k * 256 + a));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS s16x4_t*)(lds + (k + 4) * 256 + a));
      const u32x2_t l2 = __builtin_bit_cast(u32x2_t, lo), h2 = __builtin_bit_cast(u32x2_t, hi);
      f[j] = u32x4{l2[0], l2[1], h2[0], h2[1]};
    }
  }
}
template <bool KM, int NT>
__device__ __forceinline__ void fragments(u32x4 (&f)[NT], const char* lds, int first, int kg, int lane, float) {
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int x = first + 32 * j + (lane & 31), k = kg * 8 + 4 * (lane >> 5);
    if constexpr (!KM) {
      f[j] = *reinterpret_cast<const u32x4*>(lds + Tile<float>::at(x, k / 4));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        f[j][i] = *reinterpret_cast<const uint32_t*>(lds + Tile<float>::at_t(k + i, x / 4) + (x & 3) * 4);
    }
  }
}

// (Q, P) operands: the accumulator is the transposed tile, so lane l holds
// row l % 32 of the output and registers 4 g + 0..3 its columns 8 g + 4 (l / 32) + 0..3.
__device__ __forceinline__ f32x16_t multiply(u32x4 q, u32x4 p, f32x16_t acc, bf16_t) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, q), __builtin_bit_cast(bf16x8_t, p), acc,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x16_t multiply(u32x4 q, u32x4 p, f32x16_t acc, float) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(q[i]), __uint_as_float(p[i]), acc, 0, 0, 0);
  return acc;
}

}  // namespace ex
}  // namespace muon
