// Large bf16 tiles of the classifier's products: the contraction core of the
// expert layer (expert_mfma.hpp) with operands of one matrix each, walked by one
// block of eight waves a CU, and epilogues that a caller gives.
#pragma once
#include "expert_mfma.hpp"
#include "vocab.hpp"

namespace muon {
namespace vo {

constexpr int kWalkers = 256;
constexpr int kStoreBytes = 4096;   // LDS of each wave behind the stages, for stores

// 256 x 256 tiles, and halves of them where no more is left: 8 waves of 128 x
// 64, or of 64 x 64.
template <bool PT, bool QT>
struct Shapes {
  typedef Shape<256, 256, 2, 4, PT, QT> Full;
  typedef Shape<128, 256, 2, 4, PT, QT> Flat;
  typedef Shape<256, 128, 4, 2, PT, QT> Thin;
  static constexpr int LDS = 2 * kStage + 8 * kStoreBytes;
};
enum Cut { kFull = 0, kFlat = 1, kThin = 2 };
__device__ __forceinline__ int cut_of(int64_t m_left, int64_t n_left) {
  return m_left <= 128 ? kFlat : n_left <= 128 ? kThin : kFull;
}

// An operand's part of a tile: from its first row or column and first k on.
struct Panel {
  const char* base;
  uint32_t ld;         // bytes from row to row
  int32_t extent;      // rows (k-contiguous) or columns (k-major) from there on; the latter a multiple of 8
  int32_t k;           // k from there on; a multiple of 8 where it is contiguous
};

// k-contiguous: copy u of wave w holds tile rows (w nr + u) 8 + lane / 8 (RowCopies).
struct RowPanel {
  const char* base;
  uint32_t voff[4];
  int32_t col[2], k;
  __device__ __forceinline__ void init(const Panel& o, int nr, int lane, int w) {
    base = o.base;
    k = o.k;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (w * nr + u) * 8 + lane / 8;
      const int chunk = (lane & 7) ^ nt::swz<128>(r);
      if (u < 2) col[u] = chunk * 8;
      voff[u] = r < o.extent ? (uint32_t)r * o.ld + (uint32_t)chunk * 16u : kNone;
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
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int, int w) const {
    const bool in[2] = {kt * kBK + col[0] < k, kt * kBK + col[1] < k};
    step<NR>(dst, copy_rsrc(base + (int64_t)kt * 128, kRange), in, w);
  }
};

// k-major, 64 NR elements a row (KCopies): rows past the last lie past the
// descriptor's range.
struct ColPanel {
  const char* base;
  uint32_t voff[4], ld;
  int32_t k;
  __device__ __forceinline__ void init(const Panel& o, int nr, int lane, int w) {
    base = o.base;
    ld = o.ld;
    k = o.k;
    const int shift = nr == 4 ? 5 : 4;   // log2 of the chunks a row
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = (((w * nr + u) << 6) >> shift) + (lane >> shift);
      const int c = ((lane & ((1 << shift) - 1)) ^ nt::swzt(r)) * 8;
      voff[u] = c < o.extent ? (uint32_t)c * 2u + (uint32_t)r * ld : kNone;
    }
  }
  __device__ __forceinline__ void ahead(int, int, int) {}
  template <int NR, int U = 0>
  __device__ __forceinline__ void step(MUON_LDS char* dst, u32x4 rs, int w) const {
    if constexpr (U < NR) {
      copy_to_lds(dst + (w * NR + U) * 1024, rs, voff[U]);
      step<NR, U + 1>(dst, rs, w);
    }
  }
  template <int NR>
  __device__ __forceinline__ void issue(MUON_LDS char* dst, int kt, int, int w) const {
    // the last row ends with its columns, not with ld: what lies behind it is another's memory
    const int64_t left = (k - (int64_t)kt * kBK) * (int64_t)ld;
    step<NR>(dst, copy_rsrc(base + (int64_t)kt * kBK * ld, left <= 0 ? 0u : left < kRange ? (uint32_t)left : kRange), w);
  }
};

// An output tile: rows from m0, columns from n0, k-tiles [k0, k0 + nk) of part `part`.
struct OutTile {
  int32_t m0, n0, k0, nk, part;
};

__device__ __forceinline__ void make_scalar(OutTile& t) {
  t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
  t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
  t.k0 = __builtin_amdgcn_readfirstlane(t.k0);
  t.nk = __builtin_amdgcn_readfirstlane(t.nk);
  t.part = __builtin_amdgcn_readfirstlane(t.part);
}

// The lane again, as a value the compiler cannot see through: what follows from
// it is worked out where it is used instead of being held over the whole walk.
__device__ __forceinline__ int fresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// The tiles of an M x N output in `parts` runs of k, as eight lists, one an XCD
// (consecutive blocks go to the XCDs in turn), of which block b takes every 32nd
// from b / 8 on.  Eight row tiles are walked before the next column tile, so that
// an XCD's blocks share both operands in its L2.
struct Walk {
  uint32_t i, end, tiles_m, tiles_n, per_part;   // per_part: k-tiles of a part
  uint32_t k_tiles;
  __device__ __forceinline__ void init(int64_t m, int64_t n, int64_t k, uint32_t parts) {
    tiles_m = (uint32_t)((m + 255) / 256);
    tiles_n = (uint32_t)((n + 255) / 256);
    k_tiles = (uint32_t)((k + kBK - 1) / kBK);
    per_part = (k_tiles + parts - 1) / parts;
    const uint32_t total = tiles_m * tiles_n * parts, per = (total + 7) / 8, first = (blockIdx.x & 7) * per;
    end = first + per < total ? first + per : total;
    i = first + (blockIdx.x >> 3);
  }
  __device__ __forceinline__ bool next(OutTile& t) {
    constexpr uint32_t kRowGroup = 8;
    if (i >= end) return false;
    const uint32_t all = tiles_m * tiles_n, part = i / all, in = i - part * all;
    const uint32_t group = in / (kRowGroup * tiles_n), off = in - group * (kRowGroup * tiles_n);
    const uint32_t wide = tiles_m - group * kRowGroup < kRowGroup ? tiles_m - group * kRowGroup : kRowGroup;
    t.n0 = (int32_t)(off / wide * 256);
    t.m0 = (int32_t)((group * kRowGroup + off % wide) * 256);
    t.part = (int32_t)part;
    t.k0 = (int32_t)(part * per_part);
    t.nk = t.k0 >= (int32_t)k_tiles ? 0 : (int32_t)(k_tiles - t.k0 < per_part ? k_tiles - t.k0 : per_part);
    make_scalar(t);
    i += kWalkers / 8;
    return true;
  }
};

// A block's walk over o's tiles.  o gives the tile that is next, its operands (p,
// q), what is left of the output from it (m_left, n_left), and stores it: the
// number of store instructions that were its last (8 or 16, else 0).
template <class O>
__device__ __forceinline__ void walk_tiles(char* lds_, int lane0, int w, O& o) {
  typedef typename O::Sh::Full Full;
  typedef typename O::Sh::Flat Flat;
  typedef typename O::Sh::Thin Thin;
  MUON_LDS char* lds = (MUON_LDS char*)lds_;
  typename O::PC cp;
  typename O::QC cq;
  Acc acc;
  OutTile cur, next;
  auto cut = [&](const OutTile& t) { return cut_of(o.m_left(t), o.n_left(t)); };
  auto nrp = [&](const OutTile& t) { return cut(t) == kFlat ? Flat::PR : Full::PR; };
  auto nrq = [&](const OutTile& t) { return cut(t) == kThin ? Thin::QR : Full::QR; };
  auto init = [&](const OutTile& t) {
    const int lane = fresh(lane0);
    cp.init(o.p(t), nrp(t), lane, w);
    cq.init(o.q(t), nrq(t), lane, w);
  };
  bool more = o.next(cur);
  int stage = 0, stored = 0;
  if (more) {
    init(cur);
    tile_issue(lds, cp, cq, nrp(cur), nrq(cur), 0, lane0, w);
    tile_issue(lds + kStage, cp, cq, nrp(cur), nrq(cur), 1, lane0, w);
    __builtin_amdgcn_s_waitcnt(nt::kWaitVmLgkm0);
    nt::block_barrier();
  }
  while (more) {
    const int c = cut(cur), lane = fresh(lane0);
    const int nk = cur.nk < 2 ? 2 : cur.nk;
    more = o.next(next);
    auto turn = [&]() {
      if (more) init(next);
      return more;
    };
    auto then = [&](MUON_LDS char* st, int t) { tile_issue(st, cp, cq, nrp(next), nrq(next), t, lane, w); };
    if (c == kFull) tile_loop<Full>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    else if (c == kFlat) tile_loop<Flat>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    else tile_loop<Thin>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    const int row0 = c == kFull ? w / Full::WGN * Full::WM : c == kFlat ? w / Flat::WGN * Flat::WM
                                                                        : w / Thin::WGN * Thin::WM;
    const int col0 = c == kThin ? w % Thin::WGN * Thin::WN : w % Full::WGN * Full::WN;
    asm volatile("" ::: "memory");   // the stores stay behind the copies
    stored = o.store(acc, cur, c == kFull ? 4 : 2, row0, col0, lds + 2 * kStage + w * kStoreBytes, fresh(lane0));
    asm volatile("" ::: "memory");
    cur = next;
  }
}

// 32 rows of a wave's columns into its LDS and out again, so that a store
// instruction writes whole 128-byte runs of 8 rows: lane l then has 16 bytes from
// byte 16 (l % 8) of row 8 u + l / 8.  Lane l brings row l % 32.
template <class F>
__device__ __forceinline__ void put_row(MUON_LDS char* buf, int lane, int piece, F v) {   // 8 bytes, or 16
  const int r = lane & 31, h = lane >> 5;
  if constexpr (sizeof(F) == 8) *(MUON_LDS F*)(buf + r * 128 + h * 8 + ((piece ^ nt::swz<128>(r)) << 4)) = v;
  else *(MUON_LDS F*)(buf + r * 128 + (((2 * piece + h) ^ nt::swz<128>(r)) << 4)) = v;
}
__device__ __forceinline__ u32x4 get_row(const MUON_LDS char* buf, int lane, int u) {
  const int q = u * 8 + lane / 8;
  return *(const MUON_LDS u32x4*)(buf + q * 128 + (((lane & 7) ^ nt::swz<128>(q)) << 4));
}

}  // namespace vo
}  // namespace muon
