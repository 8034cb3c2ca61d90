// bf16 contraction core of the grouped products: acc(i, j) += sum_k P Q with
// each operand either k-contiguous (tile rows of BK = 64 k) or k-major (64
// tile rows of BM or BN elements), copied global -> LDS by buffer_load ... lds
// (16 bytes a lane, no registers in between), two stages.
// A block walks a list of output tiles: the copies of its next tile's first
// k-tiles are issued before the stores of the last one, whose way to memory is
// then hidden behind the next tile's products.
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
constexpr int kStage = 65536, kQAt = 32768;   // LDS of a k-tile: that of the largest tile for all, so that stages may
                                              // hold k-tiles of different tiles

template <int BM_, int BN_, int WGM_, int WGN_, bool PT_, bool QT_>
struct Shape {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr bool PT = PT_, QT = QT_;
  static constexpr int NW = WGM * WGN, THREADS = 64 * NW;
  static constexpr int WM = BM / WGM, WN = BN / WGN, MT = WM / 32, NT = WN / 32;
  static constexpr int PR = BM / 8 / NW, QR = BN / 8 / NW;   // 1 KiB copies a wave makes of each operand
  static constexpr int NDS = (PT ? 2 : 1) * MT + (QT ? 2 : 1) * NT;
  static_assert(BM % (16 * NW) == 0 && BN % (16 * NW) == 0 && MT % 2 == 0 && NT >= 1 && BM <= 256 && BN <= 256, "tile");
  static_assert((!PT || BM >= 128) && (!QT || BN >= 128), "k-major tile rows of 256 bytes or more");
};

// A copy of 16 bytes a lane from memory to LDS (1 KiB at dst).  Written out, and
// not through the builtin, because the compiler otherwise waits for every copy
// in flight before a transposing LDS read, whose address it cannot tell from
// the copies' targets; tile_loop makes the waits that are needed.  No register
// is written (the compiler holds nothing in M0).  The idle cycles are those
// that M0 (1) and a descriptor written by a vector instruction (5) take before
// such a load reads them.
typedef __attribute__((address_space(3))) char lds_char;
__device__ __forceinline__ void copy_to_lds(lds_char* dst, u32x4 rsrc, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"((uint32_t)(uintptr_t)dst), "v"(voff), "s"(rsrc));
}
__device__ __forceinline__ u32x4 copy_rsrc(const char* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xffffu, bytes, (uint32_t)nt::kRsrcWord3};
}

// What a block's copies need to know of one operand.
struct Operand {
  const char* base;        // row 0 (k-contiguous: of the tile; k-major: of k = 0), column 0
  const int32_t* gather;   // indices of the tile's rows, or null: rows follow each other
  int32_t src_rows;        // rows that gather may name
  int32_t rows;            // rows that exist (k-contiguous: of the tile; k-major: k)
  int32_t col0, cols;      // k-major: first column; row length in elements (k-contiguous: K)
};

// k-contiguous: copy u < NR of wave w holds tile rows (w NR + u) 8 + lane / 8.
// A block's tiles differ in height, so NR <= 4 is an argument of the calls.
struct RowCopies {
  const char* base;
  uint32_t voff[4];
  int32_t col[2];      // first k of the lane's chunk in tile 0, even and odd copies
  int32_t cols;
  int32_t src[4];      // gathered source rows of the next init, -1: none

  // the source rows of an operand's tile rows; these loads may be in flight until init
  __device__ __forceinline__ void look(const Operand& o, int nr, int lane, int w) {
    if (!o.gather) return;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (w * nr + u) * 8 + lane / 8;
      src[u] = r < o.rows && u < nr ? o.gather[r] : -1;
    }
  }
  // nr: 2 or 4
  __device__ __forceinline__ void init(const Operand& o, int nr, int lane, int w) {
    base = o.base;
    cols = o.cols;
    const uint32_t ld = (uint32_t)o.cols * 2u;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (w * nr + u) * 8 + lane / 8;
      const int chunk = (lane & 7) ^ nt::swz<128>(r);
      if (u < 2) col[u] = chunk * 8;   // nr is even: the swizzle's phase follows the copy's index
      const int from = o.gather ? src[u] : r;
      const bool ok = o.gather ? from >= 0 && from < o.src_rows : r < o.rows;
      voff[u] = ok ? (uint32_t)from * ld + (uint32_t)chunk * 16u : kNone;
    }
  }
  __device__ __forceinline__ void ahead(int, int, int) {}
  template <int NR, int U = 0>
  __device__ __forceinline__ void step(MUON_LDS char* dst, u32x4 rs, const bool (&in)[2], int w) const {
    if constexpr (U < NR) {
      copy_to_lds(dst + (w * NR + U) * 1024, rs, in[U & 1] ? voff[U] : kNone);
      step<NR, U + 1>(dst, rs, in, w);
    }
  }
  template <int NR>
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int, int w) {
    const u32x4 rs = copy_rsrc(base + (int64_t)kt * 128, kRange);
    const bool in[2] = {kt * kBK + col[0] < cols, kt * kBK + col[1] < cols};
    step<NR>(dst, rs, in, w);
  }
};

// k-major, 64 NR elements a row (NR = 2 or 4 copies a wave): copy u of wave w
// holds tile rows w NR RPI + u RPI + lane / CPR.  Rows past the last lie past
// the descriptor's range, which ends with the operand's last row.  GATHER: the
// indices of a wave's rows come one tile ahead, one a lane, and reach the
// copies through scalar registers.
template <bool GATHER>
struct KCopies {
  const char* base;
  const int32_t* gather;
  uint32_t voff[4];        // with GATHER the column's part alone
  uint32_t ld;
  int32_t rows, src_rows;
  int32_t idx;             // GATHER: row index of row (lane % 8) of the next tile, -1: none

  template <int NR>
  struct Rows {
    static constexpr int CPR = 8 * NR, RPI = 64 / CPR;   // chunks a row; rows a copy
    static_assert(NR * RPI == 8, "a wave copies 8 of the 64 rows");
  };
  __device__ __forceinline__ void look(const Operand&, int, int, int) {}
  // nr: 2 or 4 copies
  __device__ __forceinline__ void init(const Operand& o, int nr, int lane, int w) {
    base = o.base;
    gather = o.gather;
    rows = o.rows;
    src_rows = o.src_rows;
    ld = (uint32_t)o.cols * 2u;
    const int shift = nr == 4 ? 5 : 4;   // log2 of the chunks a row
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (((w * nr + u) << 6) >> shift) + (lane >> shift);
      const int chunk = (lane & ((1 << shift) - 1)) ^ nt::swzt(r);
      const int c = o.col0 + chunk * 8;
      voff[u] = c < o.cols ? (uint32_t)c * 2u + (GATHER ? 0u : (uint32_t)r * ld) : kNone;
    }
  }
  // the indices of tile kt
  __device__ __forceinline__ void ahead(int kt, int lane, int w) {
    if constexpr (GATHER) {
      const uint32_t k = (uint32_t)kt * kBK + w * 8 + lane % 8;   // unsigned: up to 256 past rows < 2^31
      idx = k < (uint32_t)rows ? gather[k] : -1;
    }
  }
  template <int NR, int U = 0>
  __device__ __forceinline__ void step(MUON_LDS char* dst, u32x4 rs, int lane, int w) const {
    if constexpr (U < NR) {
      constexpr int CPR = Rows<NR>::CPR, RPI = Rows<NR>::RPI;
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
      copy_to_lds(dst + (w * NR + U) * 1024, rs, v);
      step<NR, U + 1>(dst, rs, lane, w);
    }
  }
  template <int NR>
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int lane, int w) {
    if constexpr (GATHER) {
      asm volatile("" : "+v"(idx));   // not looked at before the wait and barrier ahead of this
      step<NR>(dst, copy_rsrc(base, kRange), lane, w);
    } else {
      const int64_t left = (rows - (int64_t)kt * kBK) * (int64_t)ld;
      step<NR>(dst,
               copy_rsrc(base + (int64_t)kt * kBK * ld, left <= 0 ? 0u : left < kRange ? (uint32_t)left : kRange),
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
    slab_frags<S::QT, S::BN, S::NT>(b, st + kQAt, wx * S::WN, kg, lane);
  }
};

// Accumulators of a wave: those of the widest shape; smaller ones use the first of them.
typedef nt::f32x16_t Acc[4][2];

// Rows [I0, I1) of the wave's MFMA tiles.
template <class S, int I0 = 0, int I1 = S::MT>
__device__ __forceinline__ void tile_mfma(Acc& acc, const TileFrags<S>& f) {
#pragma unroll
  for (int i = I0; i < I1; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(nt::bf16x8_t, f.b[j]),
                                                         __builtin_bit_cast(nt::bf16x8_t, f.a[i]), acc[i][j], 0, 0, 0);
}

// An LDS read behind each of the first NDS products.
template <class S, int NDS>
__device__ __forceinline__ void tile_hint() {
#pragma unroll
  for (int i = 0; i < S::MT * S::NT; ++i) {
    MUON_SCHED(0x008, 1);
    if (i < NDS) MUON_SCHED(0x100, 1);
  }
}

// Wait until at most N of the wave's memory operations and, behind them, its
// last `stored` stores are in flight (operations of a wave complete in order).
template <int N, bool LGKM>
__device__ __forceinline__ void wait_behind(int stored) {
  constexpr int kKeep = LGKM ? ~0xF00 : ~0;
  if (stored == 16) __builtin_amdgcn_s_waitcnt(nt::waitcnt_vm(N + 16) & kKeep);
  else if (stored == 8) __builtin_amdgcn_s_waitcnt(nt::waitcnt_vm(N + 8) & kKeep);
  else __builtin_amdgcn_s_waitcnt(nt::waitcnt_vm(N) & kKeep);
}

// Copies of k-tile kt of a tile whose copies a wave are nrp and nrq (2 or 4).
template <class PC, class QC>
__device__ __forceinline__ void tile_issue(MUON_LDS char* st, PC& cp, QC& cq, int nrp, int nrq, int kt, int lane,
                                           int w) {
  if (nrp == 4) cp.template issue<4>(st, kt, lane, w);
  else cp.template issue<2>(st, kt, lane, w);
  if (nrq == 4) cq.template issue<4>(st + kQAt, kt, lane, w);
  else cq.template issue<2>(st + kQAt, kt, lane, w);
  cp.ahead(kt + 1, lane, w);
  cq.ahead(kt + 1, lane, w);
}

// The k loop over nk >= 2 tiles of 64 (the last ones may be zeros), the first
// of which has landed in stage `stage` and the second is on its way to the
// other, followed by `stored` stores.  The fragments of a k-group are read one
// group ahead.  When the reads of a k-tile's last group are done and the copies
// of the next one have landed, one barrier, and the copies of the one after
// that go into the stage just read.  For the last two k-tiles these are the
// next tile's first two: turn() makes cp and cq that tile's and tells whether
// there is one, and then(st, t) issues its k-tile t.  On return its first
// k-tile has landed, in stage `stage`.
template <class S, class PC, class QC, class Turn, class Then>
__device__ __forceinline__ void tile_loop(Acc& acc, MUON_LDS char* lds, PC& cp, QC& cq, int nk, int stored, int& stage,
                                          int lane, int w, Turn turn, Then then) {
  const int wy = w / S::WGN, wx = w % S::WGN;
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  TileFrags<S> f0, f1;
  f0.load(lds + stage * kStage, 0, lane, wy, wx);
  auto first_groups = [&](const MUON_LDS char* st) {
#pragma unroll
    for (int g = 0; g < 3; ++g) {
      if (g & 1) {
        f0.load(st, g + 1, lane, wy, wx);
        tile_mfma<S>(acc, f1);
      } else {
        f1.load(st, g + 1, lane, wy, wx);
        tile_mfma<S>(acc, f0);
      }
      tile_hint<S, S::NDS>();
    }
    wait_behind<0, true>(stored);   // the next k-tile landed, own reads done
    stored = 0;
    nt::block_barrier();
  };
  for (int kt = 0; kt < nk - 2; ++kt) {
    MUON_LDS char* st = lds + stage * kStage;
    first_groups(st);
    // the copies in two runs with products between them, the fragment reads with the second: 728 -> 703 us for the
    // training batch against both runs first and the products after (input gradient 419 -> 414, weight gradient
    // 252 -> 248, from 8 bits 818 -> 783); the reads ahead of all, or the products' first half, are slower
    stage ^= 1;
    cq.template issue<S::QR>(st + kQAt, kt + 2, lane, w);
    __builtin_amdgcn_sched_barrier(0);
    tile_mfma<S, 0, S::MT / 2>(acc, f1);
    __builtin_amdgcn_sched_barrier(0);
    f0.load(lds + stage * kStage, 0, lane, wy, wx);
    cp.template issue<S::PR>(st, kt + 2, lane, w);
    cp.ahead(kt + 3, lane, w);
    cq.ahead(kt + 3, lane, w);
    __builtin_amdgcn_sched_barrier(0);
    tile_mfma<S, S::MT / 2>(acc, f1);
  }
  const bool more = turn();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    MUON_LDS char* st = lds + stage * kStage;
    first_groups(st);
    if (more) then(st, t);
    stage ^= 1;
    if (t == 0) f0.load(lds + stage * kStage, 0, lane, wy, wx);
    tile_mfma<S>(acc, f1);
  }
}

// A tile's rows out of the accumulators: 32 rows of a wave's 64 columns at a
// time through 4 KiB of LDS of its own, so that a store instruction writes
// whole 128-byte runs of 8 rows.  8-byte group 2 c + h of row r is kept in chunk c ^ swz(r).
// Stores that reach past the tile name no address, so that a
// tile always makes 4 mt of them: returned for tile_loop's waits.
__device__ __forceinline__ int tile_store(const Acc& acc, int mt, MUON_LDS char* buf, bf16_t* out, int row0, int m_left,
                                          int col0, int N, int lane) {
  const auto rs = nt::make_rsrc(out, kRange);
  const int r = lane & 31, h = lane >> 5;
  MUON_LDS char* put = buf + r * 128 + h * 8;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i >= mt) break;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *(MUON_LDS u32x2*)(put + (((4 * j + g) ^ nt::swz<128>(r)) << 4)) =
            u32x2{pack2(acc[i][j][4 * g], acc[i][j][4 * g + 1]), pack2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
    u32x4 v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = u * 8 + lane / 8;
      v[u] = *(const MUON_LDS u32x4*)(buf + q * 128 + (((lane & 7) ^ nt::swz<128>(q)) << 4));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int q = row0 + 32 * i + u * 8 + lane / 8, c = col0 + 8 * (lane & 7);
      const uint32_t at = q < m_left && c < N ? ((uint32_t)q * (uint32_t)N + (uint32_t)c) * 2u : kNone;
      __builtin_amdgcn_raw_buffer_store_b128(v[u], rs, at, 0, 0);
    }
  }
  return 4 * mt;
}

}  // namespace ex
}  // namespace muon
