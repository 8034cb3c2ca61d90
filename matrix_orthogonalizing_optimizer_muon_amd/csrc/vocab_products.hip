// The classifier's three matrix products.
//
//   logits  l[s][v]   = sum_i x[rows[s]][i] w[v][i]      both k-contiguous
//   dx      dx[rows[s]][i] = sum_v dl[s][v] w[v][i]      w k-major
//   dw      dw[v][i]  = sum_s dl[s][v] x[rows[s]][i]     both k-major
//
// Logits are not stored (but for those of few rows, vocab_few.hip): what leaves the
// first product is, for each slab of columns, a row's largest exponent of two, rounded
// up, and the sum of 2^ the rest (kStats), these and 2^ the rest in as many bits as x
// has (kStatsExp, which k_rescale makes gradients of once the row's sum is known), or
// the logits' gradient without the targets' part (kGradient, where the sum is known
// before).
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "expert_stage.hpp"
#include "vocab_loss.hpp"
#include "vocab_walk.hpp"

namespace muon {
namespace vo {
namespace {

using nt::f32x16_t;

enum Product { kLogits = 0, kDx = 1, kDw = 2 };

__device__ __forceinline__ void store_exps(bf16_t* p, int cnt, const float* v) {
  const uint32_t a = pack_exps(v[0], v[1]), b = pack_exps(v[2], v[3]);
  if (cnt >= 4) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{a, b};
  } else {
    if (cnt > 0) p[0].bits = (uint16_t)a;
    if (cnt > 1) p[1].bits = (uint16_t)(a >> 16);
    if (cnt > 2) p[2].bits = (uint16_t)b;
  }
}
__device__ __forceinline__ void store_exps(float* p, int cnt, const float* v) { store4(p, cnt, v); }

// The targets' logits that a wave has go to picked: lane l has those of row l % 32
// (slot s, or -1: none) in columns first + 32 (v / 16) + 8 (v % 16 / 4) + 4 (l / 32) + v % 4
// for v < N, of value(v).
__device__ __forceinline__ int32_t value_at(int32_t c) { return (c >> 5) * 16 + ((c >> 3) & 3) * 4 + (c & 3); }

// `id`: the only target of the lane's row.
template <int N, class Value>
__device__ __forceinline__ void pick_one(const LossArgs& a, int32_t first, int64_t s, int32_t id, int lane,
                                         Value value) {
  const int32_t c = id - first;
  const bool hit = id >= first && c < 2 * N && ((c >> 2) & 1) == lane >> 5;
  if (!__any(hit)) return;
  const int32_t at = value_at(c);
  float x = 0.f;
#pragma unroll
  for (int v = 0; v < N; ++v) x = at == v ? value(v) : x;
  if (hit) a.picked[s] = x;
}

// 32 places of a row, 16 in each of its lanes: places j0 + 8 n + 4 (l / 32) + 0..3.
struct Places {
  u32x4 id[4];
  __device__ __forceinline__ void load(const LossArgs& a, int64_t s, int32_t j0, int lane) {
    const int32_t* p = a.ids + (s < 0 ? 0 : s) * a.kp;
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int32_t j = j0 + 8 * n + 4 * (lane >> 5);
      id[n] = u32x4{~0u, ~0u, ~0u, ~0u};
      if (s >= 0 && j < a.kp) id[n] = *reinterpret_cast<const u32x4*>(p + j);
    }
  }
  // A hit goes to the lane that has its column.  A lane notes one of its hits, as is
  // mostly all there is: k / (vocab / 64) for a row.  Where a lane has more, the wave's
  // 32 rows go through LDS (buf, 4 KB), from where lanes take theirs (gradients of 4000
  // rows of 500 x 1024, k = 64: 164 us, one by one 789).
  template <int N, class Value>
  __device__ __forceinline__ void pick(const LossArgs& a, int32_t first, int64_t s, int32_t j0, int lane,
                                       MUON_LDS char* buf, Value value) const {
    uint32_t note = 0, count = 0;   // place of the lane's 16, column
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t c = id[e / 4][e % 4] - (uint32_t)first;   // -1: far above
      note = c < 2 * N ? c + 256 * e : note;
      count += c < 2 * N;
    }
    if (__any(count > 1)) {
      const int r = lane & 31;
#pragma unroll
      for (int j = 0; j < N / 16; ++j) {
#pragma unroll
        for (int g = 0; g < 4; ++g)
          put_row(buf, lane, g, u32x4{__float_as_uint(value(16 * j + 4 * g)), __float_as_uint(value(16 * j + 4 * g + 1)),
                                      __float_as_uint(value(16 * j + 4 * g + 2)), __float_as_uint(value(16 * j + 4 * g + 3))});
        asm volatile("" ::: "memory");   // reads of other lanes' writes, in the wave's order
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t c = id[e / 4][e % 4] - (uint32_t)(first + 32 * j);
          if (c < 32)
            a.picked[s * a.kp + j0 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)] =
                *(const MUON_LDS float*)(buf + r * 128 + (((c >> 2) ^ nt::swz<128>(r)) << 4) + (c & 3) * 4);
        }
        asm volatile("" ::: "memory");
      }
      return;
    }
    uint64_t hits = __ballot(count == 1);
    while (hits) {
      const int h = __ffsll((unsigned long long)hits) - 1;
      hits &= hits - 1;
      const uint32_t n = __builtin_amdgcn_readlane(note, h);
      give<N>(a, s, j0, h, n >> 8, n & 255, lane, value);
    }
  }
  template <int N, class Value>
  static __device__ __forceinline__ void give(const LossArgs& a, int64_t s, int32_t j0, int h, uint32_t e, uint32_t c,
                                              int lane, Value value) {
    const int32_t at = value_at((int32_t)c);
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < N; ++v) x = at == v ? value(v) : x;
    if (lane == (h & 31) + 32 * (int)((c >> 2) & 1)) a.picked[s * a.kp + j0 + 8 * (e >> 2) + 4 * (h >> 5) + (e & 3)] = x;
  }
};

// An fp32 operand's way from memory to its tile (Stager's layout) where 31 bits
// address a tile's rows: loads through a descriptor and without a branch, so that a
// wait for one k-tile's leaves the next one's in flight (389 x 4099 x 515, dw: 31 ->
// 26 us).  Rows that do not exist lie past the descriptor's range or get no address.
// Of columns that do not, those of a k-contiguous operand are set to zero; of a
// k-major one they reach only outputs that do not exist.
template <bool KM>
struct Stager32 {
  using G = Tile<float>;
  static constexpr int CPR = KM ? G::B / G::PER : G::BK / G::PER, ROWS = KM ? G::BK : G::B, NC = ROWS * CPR / 256;
  const float* base;
  int64_t ld;
  int32_t rows, k;      // rows from base on (k-major: of k); k of a k-contiguous operand
  int32_t cols;         // of a k-major operand, from base on
  uint32_t voff[NC];
  u32x4 v[NC];

  // base: row 0 of the tile (k-major: k = 0, its first column); extent: rows, or columns, from there on
  __device__ __forceinline__ void init(const float* b, int64_t ld_, int32_t extent, int32_t k_) {
    base = b;
    ld = ld_;
    rows = KM ? k_ : extent;
    k = k_;
    cols = extent;
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int id = u * 256 + (int)threadIdx.x, r = id / CPR, c = id % CPR;
      const bool ok = KM ? c * G::PER < extent : r < extent;
      voff[u] = ok ? ((uint32_t)r * (uint32_t)ld + c * G::PER) * 4u : kNone;
    }
  }
  __device__ __forceinline__ void fetch(int64_t k0) {
    // to the end of the last row's columns: nothing behind the operand is read
    const int64_t left = (KM ? (rows - k0 - 1) * ld + cols : rows * ld - k0) * 4;
    const auto rs = nt::make_rsrc(base + (KM ? k0 * ld : k0), left <= 0 ? 0u : left < kRange ? (uint32_t)left : kRange);
#pragma unroll
    for (int u = 0; u < NC; ++u) {
      const int c = (u * 256 + (int)threadIdx.x) % CPR;
      v[u] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, voff[u], 0, 0));
      if constexpr (!KM) {
        const int64_t at = k0 + c * G::PER;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = at + i < k ? v[u][i] : 0u;
      }
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

// One output tile per block of 4 waves (2 x 2) and two LDS stages, as
// k_product's of the expert layer.  fp32: a k-tile's sum (32 products) is added to
// the total by itself, so that no value is rounded K / 2 times in a row (errors of
// the gradients of 389 x 4099 x 515: 4.0e-6 -> 1.2e-6 of their norm).
template <class T, int PRODUCT, int EPI, bool SHORT>
__global__ __launch_bounds__(256) void k_tile(LossArgs a, int32_t tiles_m, int32_t tiles_n) {
  using G = Tile<T>;
  constexpr bool PT = PRODUCT == kDw, QT = PRODUCT != kLogits;
  constexpr int PB = PT ? G::BYTES_T : G::BYTES, QB = QT ? G::BYTES_T : G::BYTES;
  constexpr int W = G::B / 2, NT = W / 32;
  static_assert(W == Slab<T>::kCols, "a wave's columns are a slab");
  __shared__ __attribute__((aligned(16))) char lds[2 * (PB + QB)];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wy = w >> 1, wx = w & 1;
  // an XCD (blocks go to them in turn) has one piece of a list that goes down 8 rows of tiles at a time, and w
  // or dl from memory once (logits of 103 x 100414 x 2048: 594 -> 551 us; 1000 x 32000 x 1024: 650 -> 631)
  const int64_t all = (int64_t)tiles_m * tiles_n, b = block_index(), t = (b & 7) * ((all + 7) / 8) + (b >> 3);
  if (b >> 3 >= (all + 7) / 8 || t >= all) return;
  const int64_t group = t / (8 * (int64_t)tiles_n), off = t - group * 8 * tiles_n;
  const int64_t wide = tiles_m - group * 8 < 8 ? tiles_m - group * 8 : 8;
  const int32_t n0 = (int32_t)(off / wide) * G::B;
  const int64_t m0 = (group * 8 + off % wide) * G::B;
  // rows of dl: two a slot where it is kept twice (bf16)
  const bool twice = sizeof(T) == 2 && PRODUCT != kLogits && a.twice;
  const int32_t slots = live_slots(a.ch), live = twice ? 2 * whole_slots(slots) : slots;
  const int32_t* rows = a.ch.rows + a.ch.slot0;
  const T* xs = twice ? static_cast<const T*>(a.xd) : static_cast<const T*>(a.xs) + a.ch.slot0 * a.ld;
  int64_t m_left;
  int32_t K;
  typename std::conditional<SHORT, Stager32<PT>, Stager<T, PT>>::type sp;
  typename std::conditional<SHORT, Stager32<QT>, Stager<T, QT>>::type sq;
  typedef decltype(sp) PStager;
  typedef decltype(sq) QStager;
  const T* wmat = static_cast<const T*>(a.w);
  if constexpr (PRODUCT == kLogits) {
    m_left = live - m0;
    if (m_left <= 0) return;
    K = a.dim;
    if constexpr (SHORT) {
      sp.init(xs + m0 * a.ld, a.ld, (int32_t)m_left, K);
      sq.init(wmat + (int64_t)n0 * a.ld, a.ld, a.vocab - n0, K);
    } else {
      sp.init(xs, nullptr, m0, m_left, 0, 0, a.dim);
      sq.init(wmat, nullptr, n0, a.vocab - n0, 0, 0, a.dim);
      sp.ld = sq.ld = a.ld;
    }
  } else {
    m_left = (PRODUCT == kDx ? live : a.vocab) - m0;
    if (m_left <= 0) return;
    // this block's part of the sum, of whole k-tiles
    const int32_t all = PRODUCT == kDx ? a.vocab : live, parts = PRODUCT == kDx ? a.parts.dx : a.parts.dw;
    const int64_t part = ((int64_t)all + parts * G::BK - 1) / (parts * G::BK) * G::BK, k0 = part * blockIdx.z;
    K = (int32_t)(all - k0 < 0 ? 0 : all - k0 < part ? all - k0 : part);
    const T* dl = static_cast<const T*>(a.dl);
    if constexpr (SHORT) {
      if constexpr (PRODUCT == kDx) {
        sp.init(dl + m0 * a.dl_ld + k0, a.dl_ld, (int32_t)m_left, K);
        sq.init(wmat + k0 * a.ld + n0, a.ld, a.dim - n0, K);
      } else {
        sp.init(dl + k0 * a.dl_ld + m0, a.dl_ld, (int32_t)m_left, K);
        sq.init(xs + k0 * a.ld + n0, a.ld, a.dim - n0, K);
      }
    } else {
      if constexpr (PRODUCT == kDx) {
        sp.init(dl + k0, nullptr, m0, m_left, 0, 0, K);
        sq.init(wmat, nullptr, k0, K, 0, n0, a.dim);
      } else {
        sp.init(dl, nullptr, k0, K, 0, (int32_t)m0, a.vocab);
        sq.init(xs, nullptr, k0, K, 0, n0, a.dim);
      }
      sp.ld = a.dl_ld;
      sq.ld = a.ld;
    }
  }
  f32x16_t acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int nk = (int)(((uint32_t)K + G::BK - 1) / G::BK);
  // the k-tile after next comes into one pair of stagers while the next one waits in the other
  PStager sp1 = sp;
  QStager sq1 = sq;
  if (nk) {
    sp.fetch(0);
    sq.fetch(0);
    sp.commit(lds);
    sq.commit(lds + PB);
  }
  if (nk > 1) {
    sp1.fetch(G::BK);
    sq1.fetch(G::BK);
  }
  auto step = [&](int kt, PStager& p2, QStager& q2, const PStager& p1, const QStager& q1) {
    __syncthreads();
    const char* st = lds + (kt & 1) * (PB + QB);
    char* next = lds + (~kt & 1) * (PB + QB);
    if (kt + 2 < nk) {
      p2.fetch((int64_t)(kt + 2) * G::BK);
      q2.fetch((int64_t)(kt + 2) * G::BK);
    }
    f32x16_t total;
    if constexpr (sizeof(T) == 4) {
      static_assert(sizeof(T) == 2 || NT == 1, "one total");
      total = acc[0][0];
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.f;
    }
#pragma unroll
    for (int kg = 0; kg < 4; ++kg) {
      u32x4 fp[NT], fq[NT];
      fragments<PT, NT>(fp, st, wy * W, kg, lane, T());
      fragments<QT, NT>(fq, st + PB, wx * W, kg, lane, T());
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = multiply(fq[j], fp[i], acc[i][j], T());
    }
    if constexpr (sizeof(T) == 4) acc[0][0] += total;
    if (kt + 1 < nk) {
      p1.commit(next);
      q1.commit(next + PB);
    }
  };
  for (int kt = 0; kt < nk; kt += 2) {
    step(kt, sp, sq, sp1, sq1);
    if (kt + 1 < nk) step(kt + 1, sp1, sq1, sp, sq);
  }
  if constexpr (sizeof(T) == 2 && PRODUCT != kLogits) {
    if (a.unit) {
      const float u = a.unit[1];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] *= u;
    }
    if (PRODUCT == kDx && twice) {   // a slot's two rows are a lane's
      static_assert(NT == 2, "32 rows, and what rounding left of them");
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[0][j] += acc[1][j];
    }
  }
  static_assert(sizeof(lds) >= 4 * 4096, "the waves' rows");
  if (PRODUCT == kLogits && a.kp > 1) __syncthreads();   // other waves' reads of the last k-tile
  // lane l has row l % 32 of a 32 x 32 tile, registers 4 g + 0..3 columns 8 g + 4 (l / 32) + 0..3
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const bool pair = PRODUCT == kDx && twice;
    if (pair && i) break;
    const int64_t r = pair ? (m0 + wy * W) / 2 + (lane & 31) : m0 + wy * W + 32 * i + (lane & 31);
    const bool exists = r < (pair ? slots : m0 + m_left);
    const int32_t c0 = n0 + wx * W + 4 * (lane >> 5);
    if constexpr (PRODUCT == kLogits) {
      if (n0 + wx * W >= a.vocab) continue;   // uniform over the wave
      const int64_t slot = exists ? r : -1;
      auto value = [&](int v) { return acc[i][v / 16][v % 16]; };
      if (a.kp == 1) {
        pick_one<16 * NT>(a, n0 + wx * W, slot, exists ? a.ids[r] : -1, lane, value);
      } else {
        for (int32_t j0 = 0; j0 < a.kp; j0 += 32) {
          Places p;
          p.load(a, slot, j0, lane);
          p.template pick<16 * NT>(a, n0 + wx * W, slot, j0, lane, (MUON_LDS char*)(lds + w * 4096), value);
        }
      }
      float e[NT][16];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int v = 0; v < 16; ++v) e[j][v] = acc[i][j][v];
      if constexpr (EPI != kGradient) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (c0 + 32 * j + 8 * (v / 4) + v % 4 < a.vocab) top = fmaxf(top, e[j][v]);
        const float n = whole_exponent<T>(a, fmaxf(top, __shfl_xor(top, 32, 64)));
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            e[j][v] = __builtin_amdgcn_exp2f(exponent(a, e[j][v], n, T()));
            if (c0 + 32 * j + 8 * (v / 4) + v % 4 < a.vocab) sum += e[j][v];
          }
        sum += __shfl_xor(sum, 32, 64);
        if (exists && lane < 32) {
          float* st = a.stats + 2 * ((int64_t)((n0 + wx * W) / W) * a.ch.size + r);
          st[0] = n;
          st[1] = sum;
        }
      } else {
        const float base = exists ? a.base[r] : 0.f, by = exists ? a.scale[r] * a.g[r] : 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) e[j][v] = __builtin_amdgcn_exp2f(exponent(a, e[j][v], base, T())) * by;
      }
      if constexpr (EPI != kStats) {
        if (exists) {
          T* out = static_cast<T*>(a.dl) + r * a.dl_ld;
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int32_t c = c0 + 32 * j + 8 * q;
              if (EPI == kStatsExp) store_exps(out + c, a.vocab - c, &e[j][4 * q]);
              else store4(out + c, a.vocab - c, &e[j][4 * q]);
            }
        }
      }
    } else if (exists) {
      constexpr bool DX = PRODUCT == kDx;
      const bool whole = (DX ? a.parts.dx : a.parts.dw) == 1;
      const int64_t at = (DX && whole ? (int64_t)rows[r] : r) * a.dim, sum_at = r * a.ld;
      float* sums = whole ? a.sums : a.sums_of_parts + (int64_t)blockIdx.z * (DX ? a.ch.size : a.vocab) * a.ld;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int32_t c = c0 + 32 * j + 8 * q;
          float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (!DX && whole && !a.first) {
            const u32x4 before = load16(sums + sum_at + c, a.dim - c);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] += __uint_as_float(before[u]);
          }
          if (whole && (DX || a.last)) store4(static_cast<T*>(DX ? a.dx : a.dw) + at + c, a.dim - c, v);
          else store4(sums + sum_at + c, a.dim - c, v);
        }
    }
  }
}

// --------------------------------------------------------------- large tiles

// The value that lane l ^ 32 has.
__device__ __forceinline__ float other_half(float v) {
  typedef uint32_t u32x2_s __attribute__((ext_vector_type(2)));
  const uint32_t x = __float_as_uint(v);
  // both registers hold v; the instruction exchanges the upper lanes of one with the lower lanes of the other
  const u32x2_s r = __builtin_bit_cast(u32x2_s, __builtin_amdgcn_permlane32_swap(x, x, false, false));
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Logits, 256 x 256 a tile.  A wave's 64 columns are a slab, 32 of them in each
// half of a row's two lanes.
template <int EPI>
struct LogitsWalk {
  typedef Shapes<false, false> Sh;
  typedef RowPanel PC;
  typedef RowPanel QC;
  const LossArgs& a;
  Walk walk;
  int32_t live;
  __device__ __forceinline__ bool next(OutTile& t) { return walk.next(t); }
  __device__ __forceinline__ int64_t m_left(const OutTile& t) const { return live - t.m0; }
  __device__ __forceinline__ int64_t n_left(const OutTile& t) const { return a.vocab - t.n0; }
  __device__ __forceinline__ Panel p(const OutTile& t) const {
    return Panel{static_cast<const char*>(a.xs) + (a.ch.slot0 + t.m0) * a.ld * 2, (uint32_t)a.ld * 2u, live - t.m0, a.ld};
  }
  __device__ __forceinline__ Panel q(const OutTile& t) const {
    return Panel{static_cast<const char*>(a.w) + (int64_t)t.n0 * a.ld * 2, (uint32_t)a.ld * 2u, a.vocab - t.n0, a.ld};
  }
  __device__ __forceinline__ int store(Acc& acc, const OutTile& t, int mt, int row0, int col0, MUON_LDS char* buf,
                                       int lane) const {
    const int32_t first = t.n0 + col0;
    if (first >= a.vocab) return 0;
    const int32_t left = a.vocab - first;   // columns of the slab that exist, where less than 64
    const int c = 4 * (lane >> 5);
    const auto rs = nt::make_rsrc(static_cast<char*>(a.dl) + ((int64_t)t.m0 * a.dl_ld + first) * 2, kRange);
    auto slot = [&](int i) {
      const int32_t r = t.m0 + row0 + 32 * i + (lane & 31);
      return i < mt && r < live ? r : -1;
    };
    // targets first: behind the stores of results their ids would wait for these
    if (a.kp == 1) {
      int32_t ids[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) ids[i] = slot(i) >= 0 ? a.ids[slot(i)] : -1;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < mt) pick_one<32>(a, first, slot(i), ids[i], lane, [&](int v) { return acc[i][v / 16][v % 16]; });
    } else {
      Places now, then;   // the next places on their way while these are looked at
      now.load(a, slot(0), 0, lane);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= mt) break;
        for (int32_t j0 = 0; j0 < a.kp; j0 += 32) {
          if (j0 + 32 < a.kp) then.load(a, slot(i), j0 + 32, lane);
          else then.load(a, i < 3 ? slot(i + 1) : -1, 0, lane);
          now.template pick<32>(a, first, slot(i), j0, lane, buf, [&](int v) { return acc[i][v / 16][v % 16]; });
          now = then;
        }
      }
    }
    float bases[4], scales[4];
    if constexpr (EPI == kGradient) {   // all rows' at once
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t r = t.m0 + row0 + 32 * i + (lane & 31);
        const bool exists = i < mt && r < live;
        bases[i] = exists ? a.base[r] : 0.f;
        scales[i] = exists ? a.scale[r] * a.g[r] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= mt) break;
      const int32_t r = t.m0 + row0 + 32 * i + (lane & 31);
      const bool exists = r < live;
      if (left < 64) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v)
            if (c + 32 * j + 8 * (v / 4) + v % 4 >= left) acc[i][j][v] = -INFINITY;
      }
      float n, by = 1.f;
      if constexpr (EPI != kGradient) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) top = fmaxf(top, acc[i][j][v]);
        n = whole_exponent<bf16_t>(a, fmaxf(top, other_half(top)));
      } else {
        n = bases[i];
        by = scales[i];
      }
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float e[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            e[u] = __builtin_amdgcn_exp2f(exponent(a, acc[i][j][4 * g + u], n, bf16_t()));
            if (EPI == kGradient) e[u] *= by;   // a column that does not exist: 0, or NaN where the row's are
            else sum += e[u];
          }
          if constexpr (EPI == kStatsExp) put_row(buf, lane, 4 * j + g, u32x2{pack_exps(e[0], e[1]), pack_exps(e[2], e[3])});
          if constexpr (EPI == kGradient) put_row(buf, lane, 4 * j + g, u32x2{pack2(e[0], e[1]), pack2(e[2], e[3])});
        }
      if constexpr (EPI != kGradient) {
        sum += other_half(sum);
        if (exists && lane < 32) {
          typedef float f32x2 __attribute__((ext_vector_type(2)));
          *reinterpret_cast<f32x2*>(a.stats + 2 * ((int64_t)(first / 64) * a.ch.size + r)) = f32x2{n, sum};
        }
      }
      if constexpr (EPI != kStats) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const u32x4 v = get_row(buf, lane, u);
          const int q = row0 + 32 * i + u * 8 + lane / 8;
          const uint32_t at = t.m0 + q < live ? (uint32_t)q * (uint32_t)(a.dl_ld * 2) + 16u * (lane & 7) : kNone;
          __builtin_amdgcn_raw_buffer_store_b128(v, rs, at, 0, 0);
        }
      }
    }
    return 0;
  }
};

template <int EPI>
__global__ __launch_bounds__(512, 2) void k_logits(LossArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[Shapes<false, false>::LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  LogitsWalk<EPI> o{a, {}, __builtin_amdgcn_readfirstlane(live_slots(a.ch))};
  o.walk.init(o.live, a.vocab, a.dim, 1);
  walk_tiles(lds, lane, w, o);
}

// The gradients' products.  Outputs go through LDS in fp32, 32 columns at a time,
// or in bf16, 64 at a time.
template <int PRODUCT>
struct GradWalk {
  static constexpr bool kX = PRODUCT == kDx;
  typedef Shapes<!kX, true> Sh;
  typedef typename std::conditional<kX, RowPanel, ColPanel>::type PC;
  typedef ColPanel QC;
  const LossArgs& a;
  Walk walk;
  int32_t live, slots;   // rows of dl, and slots
  __device__ __forceinline__ bool next(OutTile& t) { return walk.next(t); }
  __device__ __forceinline__ int32_t rows() const { return kX ? live : a.vocab; }
  __device__ __forceinline__ int64_t m_left(const OutTile& t) const { return rows() - t.m0; }
  __device__ __forceinline__ int64_t n_left(const OutTile& t) const { return a.dim - t.n0; }
  // k of the tile's part: a part of one k-tile runs two, the second of which reads zeros and not the next part's first
  __device__ __forceinline__ int32_t part_k(const OutTile& t, int64_t left) const {
    const int64_t part = (int64_t)t.nk * kBK;
    return (int32_t)(left < part ? left : part);
  }
  __device__ __forceinline__ Panel p(const OutTile& t) const {
    const char* dl = static_cast<const char*>(a.dl);
    const int64_t k = (int64_t)t.k0 * kBK;
    if (kX)
      return Panel{dl + (t.m0 * a.dl_ld + k) * 2, (uint32_t)a.dl_ld * 2u, live - t.m0, part_k(t, a.dl_ld - k)};
    return Panel{dl + (k * a.dl_ld + t.m0) * 2, (uint32_t)a.dl_ld * 2u, (int32_t)a.dl_ld - t.m0, part_k(t, live - k)};
  }
  __device__ __forceinline__ Panel q(const OutTile& t) const {
    const int64_t k = (int64_t)t.k0 * kBK;
    const char* from = kX ? static_cast<const char*>(a.w) + k * a.ld * 2
                          : a.twice ? static_cast<const char*>(a.xd) + k * a.ld * 2
                                    : static_cast<const char*>(a.xs) + (a.ch.slot0 + k) * a.ld * 2;
    return Panel{from + t.n0 * 2ll, (uint32_t)a.ld * 2u, a.ld - t.n0, part_k(t, (kX ? a.vocab : live) - k)};
  }
  __device__ __forceinline__ int store(Acc& acc, const OutTile& t, int mt, int row0, int col0, MUON_LDS char* buf,
                                       int lane) const {
    if (a.unit) {
      const float u = a.unit[1];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= mt) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] *= u;
      }
    }
    int32_t m0 = t.m0;
    if (kX && a.twice) {   // a slot's two rows are a lane's
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = acc[2 * i][j] + acc[2 * i + 1][j];
      mt /= 2;
      row0 /= 2;
      m0 /= 2;
    }
    const int32_t c0 = t.n0 + col0, m = (kX ? slots : a.vocab) - m0;
    const bool parts = (kX ? a.parts.dx : a.parts.dw) > 1;
    if (parts || (!kX && a.sums)) {   // sums: of a part, or of the chunks so far
      float* out = parts ? a.sums_of_parts + ((int64_t)t.part * (kX ? a.ch.size : a.vocab) + m0) * a.ld
                         : a.sums + (int64_t)t.m0 * a.ld;
      bf16_t* dw = static_cast<bf16_t*>(a.dw) + (int64_t)t.m0 * a.dim;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= mt) break;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int g = 0; g < 4; ++g)
            put_row(buf, lane, g, u32x4{__float_as_uint(acc[i][j][4 * g]), __float_as_uint(acc[i][j][4 * g + 1]),
                                        __float_as_uint(acc[i][j][4 * g + 2]), __float_as_uint(acc[i][j][4 * g + 3])});
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            u32x4 v = get_row(buf, lane, u);
            const int q = row0 + 32 * i + u * 8 + lane / 8, c = c0 + 32 * j + 4 * (lane & 7);
            if (q >= m || c >= a.ld) continue;
            const int64_t at = (int64_t)q * a.ld + c;
            if (!kX && !parts && !a.first) {
              const u32x4 before = *reinterpret_cast<const u32x4*>(out + at);
#pragma unroll
              for (int x = 0; x < 4; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) + __uint_as_float(before[x]));
            }
            if (!kX && !parts && a.last) {
              const float o[4] = {__uint_as_float(v[0]), __uint_as_float(v[1]), __uint_as_float(v[2]), __uint_as_float(v[3])};
              store4(dw + (int64_t)q * a.dim + c, a.dim - c, o);
            } else
              *reinterpret_cast<u32x4*>(out + at) = v;
          }
        }
      }
      return 0;
    }
    if (!kX && a.chunked)
      return tile_store(acc, mt, buf, static_cast<bf16_t*>(a.dw) + (int64_t)t.m0 * a.dim, row0, m < 256 ? m : 256, c0,
                        a.dim, lane);
    // rows of dx lie where rows[slot] says
    const int32_t* rows = a.ch.rows + a.ch.slot0 + m0;
    bf16_t* to = static_cast<bf16_t*>(kX ? a.dx : a.dw);
    int64_t row[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int q = row0 + 32 * i + u * 8 + lane / 8;
        row[i][u] = i >= mt || q >= m ? -1 : kX ? rows[q] : t.m0 + q;
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i >= mt) break;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          put_row(buf, lane, 4 * j + g, u32x2{pack2(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                                              pack2(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])});
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const u32x4 v = get_row(buf, lane, u);
        const int c = c0 + 8 * (lane & 7);
        if (row[i][u] < 0 || c >= a.dim) continue;
        bf16_t* p = to + row[i][u] * a.dim + c;
        if (a.chunked) {
          *reinterpret_cast<u32x4*>(p) = v;
        } else if (a.dim - c >= 8) {
          *reinterpret_cast<u32x4_any*>(p) = v;
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (c + x < a.dim) p[x].bits = (uint16_t)(v[x / 2] >> (16 * (x % 2)));
        }
      }
    }
    return 0;
  }
};

template <int PRODUCT>
__global__ __launch_bounds__(512, 2) void k_grad(LossArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[GradWalk<PRODUCT>::Sh::LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t slots = __builtin_amdgcn_readfirstlane(live_slots(a.ch));
  GradWalk<PRODUCT> o{a, {}, a.twice ? 2 * whole_slots(slots) : slots, slots};
  if (PRODUCT == kDx) o.walk.init(o.live, a.dim, a.vocab, (uint32_t)a.parts.dx);
  else o.walk.init(a.vocab, a.dim, o.live, (uint32_t)a.parts.dw);
  walk_tiles(lds, lane, w, o);
}

// The parts' sums, in their order: 512 columns of a slot of dx, which go to its row,
// or of a row of dw, which go on from the chunks before, are a wave's, or, where there
// are kManyParts and more, a block's, whose waves have a quarter of the parts each (64
// parts of one row: 5 us, by one wave 9.6).
constexpr int kManyParts = 12;
template <class T, int PRODUCT, bool MANY>
__global__ __launch_bounds__(256) void k_add(LossArgs a, int32_t units) {
  constexpr bool DX = PRODUCT == kDx;
  __shared__ float quarters[MANY ? 4 : 1][64][9];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t unit = MANY ? block_index() : block_index() * 4 + w;
  const int64_t s = unit / units;
  if (s >= (DX ? live_slots(a.ch) : a.vocab)) return;   // MANY: the whole block
  const int64_t c = (unit - s * units) * 512 + lane * 8;
  const int cnt = a.dim - c < 0 ? 0 : a.dim - c < 8 ? (int)(a.dim - c) : 8, parts = DX ? a.parts.dx : a.parts.dw;
  const int64_t size = (int64_t)(DX ? a.ch.size : a.vocab) * a.ld, at = s * a.ld + c;
  float sum[8] = {};
  if (!DX && !a.first && (!MANY || w == 0)) load8(a.sums + at, cnt, sum);
  const int32_t per = MANY ? (parts + 3) / 4 : parts, from = MANY ? w * per : 0, to = from + per < parts ? from + per : parts;
#pragma unroll 8
  for (int32_t p = from; p < to; ++p) {
    float v[8];
    load8(a.sums_of_parts + p * size + at, cnt, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += v[i];
  }
  if constexpr (MANY) {
    if (w) {
#pragma unroll
      for (int i = 0; i < 8; ++i) quarters[w][lane][i] = sum[i];
    }
    __syncthreads();
    if (w) return;
#pragma unroll
    for (int q = 1; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] += quarters[q][lane][i];
  }
  if (DX) store8(static_cast<T*>(a.dx) + (int64_t)a.ch.rows[a.ch.slot0 + s] * a.dim + c, cnt, sum);
  else if (a.last) store8(static_cast<T*>(a.dw) + s * a.dim + c, cnt, sum);
  else store8(a.sums + at, cnt, sum);
}

template <int EPI>
int launch_logits_large(const LossArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((k_logits<EPI>), dim3(kWalkers), dim3(512), 0, s, a);
  return launch_status("classifier product launch");
}

template <class T, int PRODUCT, int EPI>
int launch_tile(const LossArgs& a, int64_t m, int64_t n, int parts, hipStream_t s) {
  const int64_t tiles_n = ceil_div(n, Tile<T>::B), tiles_m = ceil_div(m, Tile<T>::B);
  const int64_t blocks = ceil_div(tiles_m * tiles_n, 8) * 8;
  auto* kernel = &k_tile<T, PRODUCT, EPI, false>;
  if constexpr (sizeof(T) == 4)
    if (a.vocab < (1 << 21) && a.dim < (1 << 21)) kernel = &k_tile<T, PRODUCT, EPI, true>;
  hipLaunchKernelGGL(kernel, grid_of_blocks(blocks, 256, (uint32_t)parts), dim3(256), 0, s, a, (int32_t)tiles_m, (int32_t)tiles_n);
  return launch_status("classifier product launch");
}

template <class T>
int launch_logits(const LossArgs& a, Epilogue e, hipStream_t s) {
  if (e == kStats) return launch_tile<T, kLogits, kStats>(a, a.ch.size, a.vocab, 1, s);
  if (e == kStatsExp) return launch_tile<T, kLogits, kStatsExp>(a, a.ch.size, a.vocab, 1, s);
  return launch_tile<T, kLogits, kGradient>(a, a.ch.size, a.vocab, 1, s);
}

template <class T, int PRODUCT>
int launch_grad(const LossArgs& a, hipStream_t s) {
  const int64_t m = PRODUCT == kDx ? a.ch.size : a.vocab, units = ceil_div(a.dim, 512);
  const int parts = PRODUCT == kDx ? a.parts.dx : a.parts.dw;
  if (a.large) {
    hipLaunchKernelGGL((k_grad<PRODUCT>), dim3(kWalkers), dim3(512), 0, s, a);
  } else {
    const int64_t rows = PRODUCT == kDx && a.twice ? 2 * whole_slots(a.ch.size) : m;
    const int rc = launch_tile<T, PRODUCT, kStats>(a, rows, a.dim, parts, s);
    if (rc) return rc;
  }
  if (parts >= kManyParts)
    hipLaunchKernelGGL((k_add<T, PRODUCT, true>), grid_of_blocks(m * units, 256), dim3(256), 0, s, a, (int32_t)units);
  else if (parts > 1)
    hipLaunchKernelGGL((k_add<T, PRODUCT, false>), grid_of_blocks(ceil_div(m * units, 4), 256), dim3(256), 0, s, a,
                       (int32_t)units);
  return launch_status("classifier product launch");
}

// Parts of a sum over k for the outputs of m x n: `at_once` tiles of b run side by
// side, so a part more brings the last round's idle ones work and costs 8 bytes an
// output (written and read, 4 TB/s).  us: what a k-tile takes one of them.
int parts_of(int64_t m, int64_t n, int64_t k, int64_t b, int64_t k_tile, int at_once, double us) {
  const double tiles = (double)ceil_div(m, b) * ceil_div(n, b), k_tiles = (double)ceil_div(k, k_tile);
  int best = 1;
  double least = 0;
  for (int p = 1; p <= 64 && (p == 1 || k_tiles >= 8.0 * p); ++p) {
    const double cost = ceil(tiles * p / at_once) * ceil(k_tiles / p) * us +
                        (p > 1 ? 4 + p * (double)m * n * 8 / 4e6 : 0);
    if (p == 1 || cost < least) {
      least = cost;
      best = p;
    }
  }
  return best;
}

}  // namespace

ProductParts product_parts(int dtype, int64_t tokens, int64_t vocab, int64_t dim, bool large) {
  const bool bf16 = dtype == MUON_BF16;
  const int64_t b = large ? 256 : bf16 ? Tile<bf16_t>::B : Tile<float>::B, k = bf16 ? kBK : Tile<float>::BK;
  const int at_once = (large ? 1 : bf16 ? 2 : 4) * kWalkers;   // by LDS
  const double us = large ? 1.7 : 2;
  return ProductParts{parts_of(tokens, dim, vocab, b, k, at_once, us), parts_of(vocab, dim, tokens, b, k, at_once, us)};
}

int logits_product(const LossArgs& a, int dtype, Epilogue e, hipStream_t s) {
  if (a.large) {
    if (e == kStats) return launch_logits_large<kStats>(a, s);
    return e == kStatsExp ? launch_logits_large<kStatsExp>(a, s) : launch_logits_large<kGradient>(a, s);
  }
  return dtype == MUON_BF16 ? launch_logits<bf16_t>(a, e, s) : launch_logits<float>(a, e, s);
}

int dx_product(const LossArgs& a, int dtype, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_grad<bf16_t, kDx>(a, s) : launch_grad<float, kDx>(a, s);
}

int dw_product(const LossArgs& a, int dtype, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_grad<bf16_t, kDw>(a, s) : launch_grad<float, kDw>(a, s);
}

}  // namespace vo
}  // namespace muon
