// bf16 contraction core of the grouped products: acc(i, j) += sum_k P Q with
// each operand either k-contiguous (tile rows of BK = 64 k) or k-major (64
// tile rows of BM or BN elements), copied global -> LDS by buffer_load ... lds
// (16 bytes a lane, no registers in between), two stages.
//
// It differs from the square core (mfma_nt.hpp, whose LDS layouts, swizzles
// and transposing reads it shares) in what the copies take: rows picked by an
// index array, row counts and lengths that end inside a tile, and operands of
// any size.  The descriptor's base advances with k, so lane offsets stay
// constant and below 2^31; a chunk that does not exist gets the offset kNone,
// past every descriptor's range, and arrives as zeros without a memory access.
#pragma once
#include "experts.hpp"
#include "mfma_nt.hpp"

namespace muon {
namespace ex {

constexpr uint32_t kNone = 0x80000000u;       // lane offset of a chunk that does not exist
constexpr uint32_t kRange = 0x7fffffffu;      // descriptor range: every real offset is below it
constexpr int kBK = 64;

template <int BM_, int BN_, int WGM_, int WGN_, bool PT_, bool QT_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr bool PT = PT_, QT = QT_;
  static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MT = WM / 32, NT = WN / 32;
  static constexpr int PB = BM * 128, STAGE = (BM + BN) * 128, LDS = 2 * STAGE;
  static constexpr int PR = BM / 8 / NW, QR = BN / 8 / NW;   // 1 KiB copies a wave makes of each operand
  static constexpr int NDS = (PT ? 2 : 1) * MT + (QT ? 2 : 1) * NT;
  static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0 && MT >= 1 && NT >= 1 && LDS <= 160 * 1024, "tile");
  static_assert((!PT || BM >= 128) && (!QT || BN >= 128), "k-major tile rows of 256 bytes or more");
};

// What a block's copies need to know of one operand.
struct Operand {
  const char* base;        // row 0 (k-contiguous: of the tile; k-major: of k = 0), column 0
  const int32_t* gather;   // indices of the tile's rows, or null: rows follow each other
  int64_t src_rows;        // rows that gather may name
  int64_t rows;            // rows that exist (k-contiguous: of the tile; k-major: k)
  int32_t col0, cols;      // k-major: first column; row length in elements (k-contiguous: K)
};

// k-contiguous: copy u of wave w holds tile rows (w NR + u) 8 + lane / 8.
template <int NR>
struct RowCopies {
  static_assert(NR % 2 == 0, "the swizzle phase must follow the copy index");
  const char* base;
  uint32_t voff[NR];
  int32_t col[2];      // first k of the lane's chunk in tile 0, even and odd copies
  int32_t cols;

  __device__ __forceinline__ void init(const Operand& o, int lane, int w) {
    base = o.base;
    cols = o.cols;
    const uint32_t ld = (uint32_t)o.cols * 2u;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int r = (w * NR + u) * 8 + lane / 8;
      const int chunk = (lane & 7) ^ nt::swz<128>(r);
      if (u < 2) col[u] = chunk * 8;
      int64_t src = r;
      bool ok = r < o.rows;
      if (ok && o.gather) {
        src = o.gather[r];
        ok = src >= 0 && src < o.src_rows;
      }
      voff[u] = ok ? (uint32_t)src * ld + (uint32_t)chunk * 16u : kNone;
    }
  }
  __device__ __forceinline__ void ahead(int, int, int) {}
  template <int U>
  __device__ __forceinline__ void step(MUON_LDS char* dst, __amdgpu_buffer_rsrc_t rs, const bool (&in)[2], int w) const {
    if constexpr (U < NR) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst + (w * NR + U) * 1024, 16, in[U & 1] ? voff[U] : kNone, 0, 0, 0);
      step<U + 1>(dst, rs, in, w);
    }
  }
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int, int w) {
    const auto rs = nt::make_rsrc(base + (int64_t)kt * 128, kRange);
    const bool in[2] = {kt * kBK + col[0] < cols, kt * kBK + col[1] < cols};
    step<0>(dst, rs, in, w);
  }
};

// k-major, B elements a row: copy u of wave w holds tile rows w NR RPI + u RPI
// + lane / CPR.  Rows past the last lie past the descriptor's range, which
// ends with the operand's last row.  GATHER: the indices of a wave's rows come
// one tile ahead, one a lane, and reach the copies through scalar registers.
template <int B, int NR, bool GATHER>
struct KCopies {
  static constexpr int CPR = B / 8, RPI = 64 / CPR, RPW = NR * RPI;   // chunks a row; rows a copy, a wave
  static_assert(RPI == 2 || RPI == 4, "rows a copy");
  static_assert(RPW <= 64, "rows a wave");
  const char* base;
  const int32_t* gather;
  uint32_t voff[NR];       // with GATHER the column's part alone
  uint32_t ld;
  int64_t rows, src_rows;
  int32_t idx;             // GATHER: row index of row (lane % RPW) of the next tile, -1: none

  __device__ __forceinline__ void init(const Operand& o, int lane, int w) {
    base = o.base;
    gather = o.gather;
    rows = o.rows;
    src_rows = o.src_rows;
    ld = (uint32_t)o.cols * 2u;
#pragma unroll
    for (int u = 0; u < NR; ++u) {
      const int r = (w * NR + u) * RPI + lane / CPR;
      const int chunk = (lane % CPR) ^ nt::swzt(r);
      const int c = o.col0 + chunk * 8;
      voff[u] = c < o.cols ? (uint32_t)c * 2u + (GATHER ? 0u : (uint32_t)r * ld) : kNone;
    }
  }
  // the indices of tile kt
  __device__ __forceinline__ void ahead(int kt, int lane, int w) {
    if constexpr (GATHER) {
      const int64_t k = (int64_t)kt * kBK + w * RPW + lane % RPW;
      idx = k < rows ? gather[k] : -1;
    }
  }
  template <int U>
  __device__ __forceinline__ void step(MUON_LDS char* dst, __amdgpu_buffer_rsrc_t rs, int lane, int w) const {
    if constexpr (U < NR) {
      uint32_t v = voff[U];
      if constexpr (GATHER) {
        int32_t s = __builtin_amdgcn_readlane(idx, U * RPI);
#pragma unroll
        for (int i = 1; i < RPI; ++i) {
          const int32_t t = __builtin_amdgcn_readlane(idx, U * RPI + i);
          s = lane / CPR >= i ? t : s;
        }
        v = s >= 0 && s < src_rows && v != kNone ? v + (uint32_t)s * ld : kNone;
      }
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, dst + (w * NR + U) * 1024, 16, v, 0, 0, 0);
      step<U + 1>(dst, rs, lane, w);
    }
  }
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int lane, int w) {
    if constexpr (GATHER) {
      step<0>(dst, nt::make_rsrc(base, kRange), lane, w);
    } else {
      const int64_t left = (rows - (int64_t)kt * kBK) * (int64_t)ld;
      step<0>(dst, nt::make_rsrc(base + (int64_t)kt * kBK * ld, left <= 0 ? 0u : left < kRange ? (uint32_t)left : kRange),
              lane, w);
    }
  }
};

// Fragments of k-group kg of NT 32-wide slabs from tile column or row `first`.
template <bool KM, int B, int NT>
__device__ __forceinline__ void slab_frags(u32x4 (&f)[NT], const MUON_LDS char* st, int first, int kg, int lane) {
  if constexpr (!KM) {
    const int r = lane & 31;
    const MUON_LDS char* p = st + (first + r) * 128 + (((kg * 2 + (lane >> 5)) ^ nt::swz<128>(r)) << 4);
#pragma unroll
    for (int j = 0; j < NT; ++j) f[j] = *(const MUON_LDS u32x4*)(p + j * 32 * 128);
  } else {
    // the transposing read: see nt::load_frags_qt
    const int g = lane >> 4, sl = lane & 15;
    const int k = kg * 16 + 8 * (g >> 1) + (sl >> 2);
    const int sw = nt::swzt(k);
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int byte = (first + 32 * j + (g & 1) * 16 + 4 * (sl & 3)) * 2;
      const int a = k * (B * 2) + (((byte >> 4) ^ sw) << 4) + (byte & 15);
      const nt::s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS nt::s16x4_t*)(st + a));
      const nt::s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MUON_LDS nt::s16x4_t*)(st + a + 4 * (B * 2)));
      const nt::u32x2_t l2 = __builtin_bit_cast(nt::u32x2_t, lo), h2 = __builtin_bit_cast(nt::u32x2_t, hi);
      f[j] = u32x4{l2[0], l2[1], h2[0], h2[1]};
    }
  }
}

template <class S>
struct TileFrags {
  u32x4 a[S::MT], b[S::NT];
  __device__ __forceinline__ void load(const MUON_LDS char* st, int kg, int lane, int wy, int wx) {
    slab_frags<S::PT, S::BM, S::MT>(a, st, wy * S::WM, kg, lane);
    slab_frags<S::QT, S::BN, S::NT>(b, st + S::PB, wx * S::WN, kg, lane);
  }
};

template <class S>
__device__ __forceinline__ void tile_mfma(nt::f32x16_t (&acc)[S::MT][S::NT], const TileFrags<S>& f) {
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(nt::bf16x8_t, f.b[j]),
                                                         __builtin_bit_cast(nt::bf16x8_t, f.a[i]), acc[i][j], 0, 0, 0);
}

template <class S, int NVM, int NDS>
__device__ __forceinline__ void tile_hint() {
#pragma unroll
  for (int i = 0; i < S::MT * S::NT; ++i) {
    MUON_SCHED(0x008, 1);
    if (i < NVM) MUON_SCHED(0x020, 1);
    if (i < NDS) MUON_SCHED(0x100, 1);
  }
}

// The k loop over nk >= 1 tiles of 64.  Tile kt sits in stage kt % 2; the
// fragments of a k-group are read one group ahead.  When the reads of a tile's
// last group are done and the copies of the next tile have landed, one
// barrier, and the copies of tile kt + 2 go into the stage just read; past the
// end they name no chunk and bring zeros that nothing reads.
template <class S, class PC, class QC>
__device__ __forceinline__ void tile_loop(nt::f32x16_t (&acc)[S::MT][S::NT], MUON_LDS char* lds, PC& cp, QC& cq,
                                          int nk, int lane, int w) {
  const int wy = w / S::WGN, wx = w % S::WGN;
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    cp.ahead(t, lane, w);
    cq.ahead(t, lane, w);
    cp.issue(lds + t * S::STAGE, t, lane, w);
    cq.issue(lds + t * S::STAGE + S::PB, t, lane, w);
  }
  cp.ahead(2, lane, w);
  cq.ahead(2, lane, w);
  __builtin_amdgcn_s_waitcnt(nt::kWaitVmLgkm0);
  nt::block_barrier();
  TileFrags<S> f0, f1;
  f0.load(lds, 0, lane, wy, wx);
  int stage = 0;
  for (int kt = 0; kt < nk; ++kt) {
    MUON_LDS char* st = lds + stage * S::STAGE;
#pragma unroll
    for (int g = 0; g < 3; ++g) {
      if (g & 1) {
        f0.load(st, g + 1, lane, wy, wx);
        tile_mfma<S>(acc, f1);
      } else {
        f1.load(st, g + 1, lane, wy, wx);
        tile_mfma<S>(acc, f0);
      }
      tile_hint<S, 0, S::NDS>();
    }
    __builtin_amdgcn_s_waitcnt(nt::kWaitVmLgkm0);   // the next tile landed, own reads done
    nt::block_barrier();
    cp.issue(st, kt + 2, lane, w);
    cq.issue(st + S::PB, kt + 2, lane, w);
    cp.ahead(kt + 3, lane, w);
    cq.ahead(kt + 3, lane, w);
    stage ^= 1;
    f0.load(lds + stage * S::STAGE, 0, lane, wy, wx);
    tile_mfma<S>(acc, f1);
    tile_hint<S, S::PR + S::QR, S::NDS>();
  }
  __builtin_amdgcn_s_waitcnt(nt::kWaitVmLgkm0);   // no copy outlives the loop
}

}  // namespace ex
}  // namespace muon
