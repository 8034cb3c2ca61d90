// Large bf16 tiles of the classifier's products: the stages and fragments of the
// expert layer's core (expert_mfma.hpp) with operands of one matrix each, walked by
// one block of eight waves a CU, a k loop of its own and epilogues that a caller gives.
#pragma once
#include <type_traits>

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
  struct At {
    u32x4 rs;
    bool in[2];
  };
  __device__ __forceinline__ At at(int kt) const {
    return At{copy_rsrc(base + (int64_t)kt * 128, kRange), {kt * kBK + col[0] < k, kt * kBK + col[1] < k}};
  }
  // copy u of a wave's nr of a k-tile
  __device__ __forceinline__ void copy(const At& t, MUON_LDS char* dst, int nr, int u, int w) const {
    copy_to_lds(dst + (w * nr + u) * 1024, t.rs, t.in[u & 1] ? voff[u] : kNone);
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
  typedef u32x4 At;
  __device__ __forceinline__ At at(int kt) const {
    // k that does not exist lies past the range; in the last row that does, columns past extent have no address (init)
    const int64_t left = (k - (int64_t)kt * kBK) * (int64_t)ld;
    return copy_rsrc(base + (int64_t)kt * kBK * ld, left <= 0 ? 0u : left < kRange ? (uint32_t)left : kRange);
  }
  __device__ __forceinline__ void copy(const At& t, MUON_LDS char* dst, int nr, int u, int w) const {
    copy_to_lds(dst + (w * nr + u) * 1024, t, voff[u]);
  }
};

// All copies of a k-tile of one operand.
template <class C>
__device__ __forceinline__ void copy_all(MUON_LDS char* dst, const C& c, int nr, int kt, int w) {
  const typename C::At t = c.at(kt);
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < nr) c.copy(t, dst, nr, u, w);
}

// Fragment reads of a k-group one by one: first b, then a.
template <class S, int FROM, int TO>
__device__ __forceinline__ void read_frags(TileFrags<S>& f, const MUON_LDS char* st, int kg, int lane, int wy, int wx) {
  if constexpr (FROM < TO) {
    u32x4 v[1];
    if constexpr (FROM < S::NT) {
      slab_frags<S::QT, S::BN, 1>(v, st + kQAt, wx * S::WN + 32 * FROM, kg, lane);
      f.b[FROM] = v[0];
    } else {
      slab_frags<S::PT, S::BM, 1>(v, st, wy * S::WM + 32 * (FROM - S::NT), kg, lane);
      f.a[FROM - S::NT] = v[0];
    }
    read_frags<S, FROM + 1, TO>(f, st, kg, lane, wy, wx);
  }
}

// The products of one k-group, in this order, the fragment reads of another group
// spread behind them, and behind product m what copy(m) does.
template <class S, bool READ, int M = 0, class Copy>
__device__ __forceinline__ void products(Acc& acc, const TileFrags<S>& f, TileFrags<S>& next, const MUON_LDS char* st,
                                         int kg, int lane, int wy, int wx, Copy copy) {
  constexpr int N = S::MT * S::NT, R = S::MT + S::NT;
  if constexpr (M < N) {
    constexpr int i = M / S::NT, j = M % S::NT;
    acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(nt::bf16x8_t, f.b[j]),
                                                       __builtin_bit_cast(nt::bf16x8_t, f.a[i]), acc[i][j], 0, 0, 0);
    if constexpr (READ) read_frags<S, M * R / N, (M + 1) * R / N>(next, st, kg, lane, wy, wx);
    copy(std::integral_constant<int, M>());
    __builtin_amdgcn_sched_barrier(0);
    products<S, READ, M + 1>(acc, f, next, st, kg, lane, wy, wx, copy);
  }
}

// The k loop over nk >= 2 tiles of 64, with tile_loop's stages and waits: the first
// has landed in stage `stage`, the second is on its way to the other, followed by
// `stored` stores.  The copies of the k-tile after next go out one at a time between
// products: Q's behind the barrier that frees their stage, in the k-tile's last
// group, P's in the first group of the next k-tile.  8192 x 32000 x 4096, us (logits
// with 16-bit results, dx, dw): both operands' copies in two runs 1729, 1696, 1748; one
// at a time in the last group 1781, 1646, 1796; so 1657, 1615, 1683.  The rest is
// power: with copies that always hit L2 the MFMA pipes are busy 0.81 of the time
// at 1.57 GHz instead of 0.74 at 1.71 (dx), in the same time.
// For the last two k-tiles the copies are the next tile's first two: turn() makes cp,
// cq, nrp and nrq that tile's and tells whether there is one.
template <class S, class PC, class QC, class Turn>
__device__ __forceinline__ void walk_loop(Acc& acc, MUON_LDS char* lds, PC& cp, QC& cq, const int& nrp, const int& nrq,
                                          int nk, int stored, int& stage, int lane, int w, Turn turn) {
  constexpr int N = S::MT * S::NT;
  static_assert(N % S::PR == 0 && N % S::QR == 0, "the copies are spread evenly");
  const int wy = w / S::WGN, wx = w % S::WGN;
#pragma unroll
  for (int i = 0; i < S::MT; ++i)
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  TileFrags<S> f0, f1;
  auto none = [](auto) {};
  f0.load(lds + stage * kStage, 0, lane, wy, wx);
  auto first_groups = [&](const MUON_LDS char* st, auto copies) {
    products<S, true>(acc, f0, f1, st, 1, lane, wy, wx, copies);
    products<S, true>(acc, f1, f0, st, 2, lane, wy, wx, none);
    products<S, true>(acc, f0, f1, st, 3, lane, wy, wx, none);
    wait_behind<0, true>(stored);   // the next k-tile landed, own reads done
    stored = 0;
    nt::block_barrier();
  };
  for (int kt = 0; kt < nk - 2; ++kt) {
    MUON_LDS char* st = lds + stage * kStage;
    MUON_LDS char* other = lds + (stage ^ 1) * kStage;
    const typename PC::At tp = cp.at(kt + 1);
    if (kt)
      first_groups(st, [&](auto m) {
        constexpr int at = decltype(m)::value;
        if constexpr (at % (N / S::PR) == 0) cp.copy(tp, other, S::PR, at / (N / S::PR), w);
      });
    else first_groups(st, none);
    stage ^= 1;
    const typename QC::At tq = cq.at(kt + 2);
    products<S, true>(acc, f1, f0, other, 0, lane, wy, wx, [&](auto m) {
      constexpr int at = decltype(m)::value;
      if constexpr (at % (N / S::QR) == 0) cq.copy(tq, st + kQAt, S::QR, at / (N / S::QR), w);
    });
  }
  if (nk > 2) copy_all(lds + (stage ^ 1) * kStage, cp, S::PR, nk - 1, w);
  const bool more = turn();
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    MUON_LDS char* st = lds + stage * kStage;
    first_groups(st, none);
    if (more) {
      copy_all(st, cp, nrp, t, w);
      copy_all(st + kQAt, cq, nrq, t, w);
    }
    stage ^= 1;
    if (t == 0) f0.load(lds + stage * kStage, 0, lane, wy, wx);
    tile_mfma<S>(acc, f1);
  }
}

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
  int nrp = 0, nrq = 0;   // copies a wave makes of the operands of the tile that cp and cq are at
  auto cut = [&](const OutTile& t) { return cut_of(o.m_left(t), o.n_left(t)); };
  auto init = [&](const OutTile& t) {
    const int lane = fresh(lane0), c = cut(t);
    nrp = c == kFlat ? Flat::PR : Full::PR;
    nrq = c == kThin ? Thin::QR : Full::QR;
    cp.init(o.p(t), nrp, lane, w);
    cq.init(o.q(t), nrq, lane, w);
  };
  bool more = o.next(cur);
  int stage = 0, stored = 0;
  if (more) {
    init(cur);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      copy_all(lds + t * kStage, cp, nrp, t, w);
      copy_all(lds + t * kStage + kQAt, cq, nrq, t, w);
    }
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
    if (c == kFull) walk_loop<Full>(acc, lds, cp, cq, nrp, nrq, nk, stored, stage, lane, w, turn);
    else if (c == kFlat) walk_loop<Flat>(acc, lds, cp, cq, nrp, nrq, nk, stored, stage, lane, w, turn);
    else walk_loop<Thin>(acc, lds, cp, cq, nrp, nrq, nk, stored, stage, lane, w, turn);
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
