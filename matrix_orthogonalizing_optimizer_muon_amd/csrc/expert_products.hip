// Matrix products grouped by expert: rows sorted by expert times that expert's
// matrix, and the two gradients.  Row counts live on the device (offsets), so
// a launch has a block for every tile that could exist and each block looks
// its expert up; nothing waits for the host.
//
//   matmul       y[r]  = sum_i x[rows[r]][i] W_e[o][i]    both k-contiguous
//   input grad   dx[r] = sum_o dy[r][o] W_e[o][i]         W k-major
//   weight grad  dW_e[o][i] = sum_r dy[r][o] x[rows[r]][i]   both k-major
#include <hip/hip_runtime.h>

#include <type_traits>

#include "expert_few.hpp"
#include "expert_mfma.hpp"
#include "expert_stage.hpp"
#include "expert_tiles.hpp"
#include "experts.hpp"
#include "mfma_nt.hpp"

namespace muon {
namespace ex {

int restore_rows(const void* q, const uint8_t* scale, int kind, int64_t rows, int64_t cols, int dtype, void* x,
                 hipStream_t s);

namespace {

using nt::f32x16_t;

// One output tile per block of 4 waves (2 x 2), two LDS stages: the next
// k-tile's loads are in flight while this one is multiplied.  Takes what the
// others do not: fp32, and bf16 rows that are not whole 16-byte chunks.  Bound
// by the way through registers: 64 x 1408 x 1024 fp32, 4096 rows: 221 us.
template <class T, int MODE>
__global__ __launch_bounds__(256) void k_product(ProdArgs a) {
  using G = Tile<T>;
  constexpr bool PT = MODE == kWeightGrad, QT = MODE != kMatmul;
  constexpr int PB = PT ? G::BYTES_T : G::BYTES, QB = QT ? G::BYTES_T : G::BYTES;
  constexpr int W = G::B / 2, NT = W / 32;
  __shared__ __attribute__((aligned(16))) char lds[2 * (PB + QB)];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wy = w >> 1, wx = w & 1;
  const int64_t t = block_index();
  const int tn = (int)(t % a.tiles_n);
  const int64_t tm = t / a.tiles_n;
  const int n0 = tn * G::B;
  T* out = static_cast<T*>(a.out);
  int64_t out_row;   // first output row of the tile
  int m_left, K;
  Stager<T, PT> sp;
  Stager<T, QT> sq;
  if constexpr (MODE == kWeightGrad) {
    if (tm >= (int64_t)a.experts * a.tiles_m) return;
    const int e = (int)(tm / a.tiles_m), m0 = (int)(tm % a.tiles_m) * G::B;
    int64_t b, end;
    expert_rows(a.offsets, e, (int)a.n, lane, b, end);
    if (a.parts > 1) {   // this block's part, of whole k-tiles
      const int64_t part = ((end - b + a.parts - 1) / a.parts + G::BK - 1) / G::BK * G::BK;
      b += part * blockIdx.z;
      end = b + part < end ? b + part : end;
      b = b < end ? b : end;
    }
    K = (int)(end - b);
    m_left = a.M - m0;
    out_row = (int64_t)e * a.M + m0;
    sp.init(a.p, nullptr, b, K, 0, m0, a.M);
    sq.init(a.q, a.rows, b, K, a.x_rows, n0, a.N);
  } else {
    RowTile rt;
    if (!find_tile<G::SH>(a.offsets, a.experts, (int)a.n, tm, lane, rt)) return;
    m_left = (int)(rt.end - rt.begin);
    out_row = rt.begin;
    K = rt.e < a.experts ? a.K : 0;
    sp.init(a.p, a.rows, rt.begin, K ? m_left : 0, a.x_rows, 0, a.K);
    const int64_t w0 = (int64_t)(K ? rt.e : 0) * a.N * a.K;
    if constexpr (QT) sq.init(static_cast<const T*>(a.q) + w0, nullptr, 0, K, 0, n0, a.N);
    else sq.init(static_cast<const T*>(a.q) + w0, nullptr, n0, a.N - n0, 0, 0, a.K);
  }
  f32x16_t acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
  const int nk = (int)(((uint32_t)K + G::BK - 1) / G::BK);
  if (nk) {
    sp.fetch(0);
    sq.fetch(0);
    sp.commit(lds);
    sq.commit(lds + PB);
  }
  for (int kt = 0; kt < nk; ++kt) {
    __syncthreads();
    const char* st = lds + (kt & 1) * (PB + QB);
    char* next = lds + (~kt & 1) * (PB + QB);
    if (kt + 1 < nk) {
      sp.fetch((int64_t)(kt + 1) * G::BK);
      sq.fetch((int64_t)(kt + 1) * G::BK);
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
    if (kt + 1 < nk) {
      sp.commit(next);
      sq.commit(next + PB);
    }
  }
  const int64_t ldo = a.N;
  const bool whole = MODE != kWeightGrad || a.parts == 1;
  float* sums = whole ? nullptr : a.partial + (int64_t)blockIdx.z * a.experts * a.M * ldo;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int r = wy * W + 32 * i + (lane & 31);
    if (r < m_left) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = n0 + wx * W + 32 * j + 8 * g + 4 * (lane >> 5);
          const float v[4] = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]};
          if (whole) store4(out + (out_row + r) * ldo + c, a.N - c, v);
          else store4(sums + (out_row + r) * ldo + c, a.N - c, v);
        }
    }
  }
}

// The parts' sums, added in their order: a thread has four elements.
template <class T>
__global__ __launch_bounds__(256) void k_add_parts(const float* __restrict__ partial, T* __restrict__ out, int64_t n,
                                                   int parts) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int cnt = n - i < 4 ? (int)(n - i) : 4;
  float sum[4] = {};
  for (int p = 0; p < parts; ++p) {
    const u32x4 v = load16(partial + p * n + i, cnt);
#pragma unroll
    for (int u = 0; u < 4; ++u) sum[u] += __uint_as_float(v[u]);
  }
  store4(out + i, cnt, sum);
}

// ------------------------------------------------------------- large tiles

// Products of many rows.  65536 rows (8192 tokens to 8 of 64 experts) through
// 2816 x 2048: 695 to 724 us, 1044 to 1088 TFLOP/s; the input gradient of half
// of them 402 to 422 us, the weight gradient 770 us.  A k-tile of 64 takes a block
// about 1.7 us in the first: 1.25 without the copies (the MFMAs at the clock that
// power leaves), the rest for the copies, half of that for those that miss L2.
//
// The large kernels run one block of 8 waves per CU, each walking a list of
// output tiles: consecutive blocks go to the eight XCDs in turn, so block b has
// every 32nd tile from b / 8 on of the list of XCD b % 8.
constexpr int kWalkers = 256;
constexpr int kStoreBytes = 4096;   // LDS of each wave behind the stages, for tile_store

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
__device__ __forceinline__ int cut_of(int m_left, int n_left) {
  return m_left <= 128 ? kFlat : n_left <= 128 ? kThin : kFull;
}

// The experts' rows held across a wave: lane l has those of experts l per to
// (l + 1) per - 1, rows [lo, hi), and the row tiles of 256 up to their end.
// Offsets are read as find_tile reads them.
__device__ __forceinline__ int row_tiles_of(int rows) { return (int)(((uint32_t)rows + 255) >> 8); }
struct Spread {
  int per, lo, hi, upto;
};
__device__ __forceinline__ int offset_at(const int32_t* offsets, int experts, int n, int e) {
  if (e >= experts) return 0;
  const int v = offsets[e + 1];
  return v > n ? n : v;
}
__device__ __forceinline__ Spread spread(const int32_t* __restrict__ offsets, int experts, int n, int lane) {
  Spread s;
  s.per = (experts + 63) / 64;
  int top = 0;
  for (int i = 0; i < s.per; ++i) {
    const int v = offset_at(offsets, experts, n, lane * s.per + i);
    top = v > top ? v : top;
  }
  s.hi = wave_scan_max(top, lane);
  s.lo = __shfl_up(s.hi, 1, 64);
  if (lane == 0) s.lo = 0;
  int run = s.lo, tiles = 0;
  for (int i = 0; i < s.per; ++i) {
    const int v = offset_at(offsets, experts, n, lane * s.per + i);
    const int to = v > run ? v : run;
    tiles += row_tiles_of(to - run);
    run = to;
  }
  s.upto = wave_scan_add(tiles, lane);
  return s;
}
// Scalar read of an offset: the experts of a lane are told apart without the
// vector loads' counter, behind which a tile's stores would be waited for.
__device__ __forceinline__ int scalar_offset(const int32_t* offsets, int n, int e) {
  typedef const int32_t __attribute__((address_space(4))) * scalar_ptr;
  const int v = ((scalar_ptr)(uintptr_t)offsets)[__builtin_amdgcn_readfirstlane(e) + 1];
  return v > n ? n : v;
}

// An output tile: rows (of the weight gradient: k) [begin, end) of expert e.
struct Tile256 {
  int e, begin, end;
  int m0, n0;      // first output row (rows products: 0) and column
};

// Into scalar registers: divisions of scalars are done by the vector unit, which
// would leave all that follows from them there.
__device__ __forceinline__ void make_scalar(Tile256& t) {
  t.e = __builtin_amdgcn_readfirstlane(t.e);
  t.begin = __builtin_amdgcn_readfirstlane(t.begin);
  t.end = __builtin_amdgcn_readfirstlane(t.end);
  t.m0 = __builtin_amdgcn_readfirstlane(t.m0);
  t.n0 = __builtin_amdgcn_readfirstlane(t.n0);
}

// Tile t of a rows product, t < tiles of all experts.  Within an expert eight
// row tiles are walked before the next column tile, so that the blocks of an
// XCD, which work on neighbours of its list, share rows and columns in its L2.
__device__ __forceinline__ Tile256 rows_tile(const Spread& s, const int32_t* offsets, int experts, int n,
                                             uint32_t tiles_n, uint32_t t) {
  constexpr int kRowGroup = 8;
  const int tm = (int)(t / tiles_n);
  const uint64_t hit = __ballot(tm < s.upto);
  const int at = __ffsll((unsigned long long)hit) - 1;
  int run = __builtin_amdgcn_readlane(s.lo, at), to = __builtin_amdgcn_readlane(s.hi, at);
  int first = at ? __builtin_amdgcn_readlane(s.upto, at - 1) : 0, e = at * s.per;
  int count = row_tiles_of(to - run);
  if (s.per > 1) {
    for (;; ++e) {
      const int v = scalar_offset(offsets, n, e);
      to = v > run ? v : run;
      count = row_tiles_of(to - run);
      if (tm < first + count) break;
      first += count;
      run = to;
    }
  }
  const int in = (int)(t - (uint32_t)first * tiles_n);   // tile of the expert
  const int group = in / (int)(kRowGroup * tiles_n), off = in - group * (int)(kRowGroup * tiles_n);
  const int wide = count - group * kRowGroup < kRowGroup ? count - group * kRowGroup : kRowGroup;
  Tile256 r;
  r.e = e;
  r.n0 = off / wide * 256;
  r.m0 = 0;
  r.begin = run + ((group * kRowGroup + off % wide) << 8);
  r.end = to - r.begin > 256 ? r.begin + 256 : to;
  make_scalar(r);
  return r;
}

// The lane again, as a value the compiler cannot see through: what follows from
// it is worked out where it is used instead of being held in registers over the
// whole walk.
__device__ __forceinline__ int fresh(int lane) {
  asm volatile("" : "+v"(lane));
  return lane;
}

// A block's walk over the tiles that o.next() names, one after the other.  o
// also gives a tile's operands (p, q), its k and, where its outputs go, its
// first row and the rows left from there.
template <class O>
__device__ __forceinline__ void walk(char* lds_, int N, int lane0, int w, O& o) {
  typedef typename O::Sh::Full Full;
  typedef typename O::Sh::Flat Flat;
  typedef typename O::Sh::Thin Thin;
  MUON_LDS char* lds = (MUON_LDS char*)lds_;
  typename O::PC cp;
  typename O::QC cq;
  Acc acc;
  Tile256 cur, next;
  auto nrp = [&](const Tile256& t) { return o.cut(t) == kFlat ? Flat::PR : Full::PR; };
  auto nrq = [&](const Tile256& t) { return o.cut(t) == kThin ? Thin::QR : Full::QR; };
  auto init = [&](const Tile256& t) {   // after look(t)
    const int lane = fresh(lane0);
    cp.init(o.p(t), nrp(t), lane, w);
    cq.init(o.q(t), nrq(t), lane, w);
    cp.ahead(0, lane, w);
    cq.ahead(0, lane, w);
  };
  auto store = [&](const Tile256& t) {
    const int cut = o.cut(t);
    const int row0 = cut == kFull ? w / Full::WGN * Full::WM : cut == kFlat ? w / Flat::WGN * Flat::WM
                                                                           : w / Thin::WGN * Thin::WM;
    const int col0 = cut == kThin ? w % Thin::WGN * Thin::WN : w % Full::WGN * Full::WN;
    return tile_store(acc, cut == kFull ? 4 : 2, lds + 2 * kStage + w * kStoreBytes, o.out(t), row0, o.m_left(t),
                      t.n0 + col0, N, fresh(lane0));
  };
  bool more = o.next(cur);
  int stage = 0, stored = 0;
  if (more) {
    cp.look(o.p(cur), nrp(cur), lane0, w);
    init(cur);
    tile_issue(lds, cp, cq, nrp(cur), nrq(cur), 0, lane0, w);
    tile_issue(lds + kStage, cp, cq, nrp(cur), nrq(cur), 1, lane0, w);
    __builtin_amdgcn_s_waitcnt(nt::kWaitVmLgkm0);
    nt::block_barrier();
  }
  while (more) {
    const int cut = o.cut(cur), lane = fresh(lane0);
    const uint32_t tiles = ((uint32_t)o.k(cur) + kBK - 1) / kBK;
    const int nk = tiles < 2 ? 2 : (int)tiles;
    more = o.next(next);
    if (more) cp.look(o.p(next), nrp(next), lane, w);
    auto turn = [&]() {
      if (more) init(next);
      return more;
    };
    auto then = [&](MUON_LDS char* st, int t) { tile_issue(st, cp, cq, nrp(next), nrq(next), t, lane, w); };
    if (cut == kFull) tile_loop<Full>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    else if (cut == kFlat) tile_loop<Flat>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    else tile_loop<Thin>(acc, lds, cp, cq, nk, stored, stage, lane, w, turn, then);
    asm volatile("" ::: "memory");   // the stores stay behind the copies
    stored = store(cur);
    asm volatile("" ::: "memory");
    cur = next;
  }
}

// Zero to rows x cols elements at out (rows of N): by the threads of one block.
__device__ __forceinline__ void zero_block(bf16_t* out, int64_t rows, int cols, int64_t N) {
  const int chunks = cols / 8;
  for (int64_t i = threadIdx.x; i < rows * chunks; i += 512)
    *reinterpret_cast<u32x4*>(out + i / chunks * N + 8 * (i % chunks)) = u32x4{0u, 0u, 0u, 0u};
}

template <int MODE>
struct RowsWalk {
  static constexpr bool QT = MODE == kInputGrad;
  typedef Shapes<false, QT> Sh;
  typedef RowCopies PC;
  typedef typename std::conditional<QT, KCopies<false>, RowCopies>::type QC;
  const ProdArgs& a;
  const Spread& s;
  uint32_t i, end;   // the next tile and the last but one
  __device__ __forceinline__ bool next(Tile256& t) {
    if (i >= end) return false;
    t = rows_tile(s, a.offsets, a.experts, (int)a.n, a.tiles_n, i);
    i += kWalkers / 8;
    return true;
  }
  __device__ __forceinline__ int m_left(const Tile256& t) const { return t.end - t.begin; }
  __device__ __forceinline__ int cut(const Tile256& t) const { return cut_of(t.end - t.begin, a.N - t.n0); }
  __device__ __forceinline__ int k(const Tile256&) const { return a.K; }
  __device__ __forceinline__ bf16_t* out(const Tile256& t) const {
    return static_cast<bf16_t*>(a.out) + (int64_t)t.begin * a.N;
  }
  __device__ __forceinline__ Operand p(const Tile256& t) const {
    const char* x = static_cast<const char*>(a.p);
    if (a.rows) return Operand{x, a.rows + t.begin, (int32_t)a.x_rows, m_left(t), 0, a.K};
    return Operand{x + (int64_t)t.begin * a.K * 2, nullptr, 0, m_left(t), 0, a.K};
  }
  __device__ __forceinline__ Operand q(const Tile256& t) const {
    const char* x = static_cast<const char*>(a.q) + (int64_t)t.e * a.N * a.K * 2;
    if (QT) return Operand{x, nullptr, 0, a.K, t.n0, a.N};
    return Operand{x + (int64_t)t.n0 * a.K * 2, nullptr, 0, a.N - t.n0, 0, a.K};
  }
};

template <int MODE>
__global__ __launch_bounds__(512, 2) void k_rows_product(ProdArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[RowsWalk<MODE>::Sh::LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Spread s = spread(a.offsets, a.experts, (int)a.n, lane);
  const uint32_t total = (uint32_t)__builtin_amdgcn_readlane(s.upto, 63) * (uint32_t)a.tiles_n, per = (total + 7) / 8;
  const uint32_t first = (blockIdx.x & 7) * per, end = first + per < total ? first + per : total;
  RowsWalk<MODE> o{a, s, first + (blockIdx.x >> 3), end};
  walk(lds, a.N, lane, w, o);
  // the rows past the last expert's, 64 at a time
  const int64_t last = __builtin_amdgcn_readlane(s.hi, 63);
  for (int64_t r = last + 64 * (int64_t)blockIdx.x; r < a.n; r += 64 * kWalkers)
    zero_block(static_cast<bf16_t*>(a.out) + r * a.N, a.n - r < 64 ? a.n - r : 64, a.N, a.N);
}

// Weight gradient.  The experts' tiles in order of their rows' number, longest
// first (where a lane has each expert), are dealt to the XCDs in sets of at
// most 32 neighbours of one expert, which an XCD's 32 CUs take at once, sharing
// rows in its L2.  Sets go to the XCDs, and an XCD's tiles to its CUs, in turn
// there and back, so that none has the longer one of every round (4096 tokens,
// 8 of 64 experts, uneven, 2048 x 1408: mean over longest 0.79 -> 0.83, 272 -> 260 us).
template <bool GATHER>
struct WeightWalk {
  typedef Shapes<true, true> Sh;
  typedef KCopies<false> PC;
  typedef KCopies<GATHER> QC;
  const ProdArgs& a;
  const Spread& s;
  int rank;                      // of the lane's expert
  uint32_t i, sets, size;        // the XCD's places so far; sets of an expert, tiles of a set
  __device__ __forceinline__ bool next(Tile256& r) {
    const uint32_t tiles = (uint32_t)a.tiles_m * (uint32_t)a.tiles_n;
    for (;;) {
      const uint32_t cu = blockIdx.x >> 3, xcd = blockIdx.x & 7;
      const uint32_t place = i + (i / 32 & 1 ? 31 - cu : cu);
      const uint32_t j = place / size, set = j * 8 + (j & 1 ? 7 - xcd : xcd);
      const uint32_t q = __builtin_amdgcn_readfirstlane(set / sets), t = (set - q * sets) * size + (place - j * size);
      if (q >= (uint32_t)a.experts) return false;
      i += kWalkers / 8;
      if (t >= tiles) continue;
      if (s.per == 1) {
        r.e = __ffsll((unsigned long long)__ballot(rank == (int)q)) - 1;
        r.begin = __builtin_amdgcn_readlane(s.lo, r.e);
        r.end = __builtin_amdgcn_readlane(s.hi, r.e);
      } else {
        const int at = (int)q / s.per;
        r.e = at * s.per;
        r.begin = r.end = __builtin_amdgcn_readlane(s.lo, at);
        for (;; ++r.e) {
          const int v = scalar_offset(a.offsets, (int)a.n, r.e);
          r.end = v > r.begin ? v : r.begin;
          if (r.e == (int)q) break;
          r.begin = r.end;
        }
      }
      const int tm = (int)(t / (uint32_t)a.tiles_n);
      r.m0 = tm * 256;
      r.n0 = (int)(t - (uint32_t)tm * a.tiles_n) * 256;
      make_scalar(r);
      if (r.end > r.begin) return true;
      // no rows: zeros, whose stores come before those of the tile at hand and so are waited for with it
      zero_block(out(r) + r.n0, m_left(r), a.N - r.n0 < 256 ? a.N - r.n0 : 256, a.N);
    }
  }
  __device__ __forceinline__ int m_left(const Tile256& t) const { return a.M - t.m0 < 256 ? a.M - t.m0 : 256; }
  __device__ __forceinline__ int cut(const Tile256& t) const { return cut_of(a.M - t.m0, a.N - t.n0); }
  __device__ __forceinline__ int k(const Tile256& t) const { return t.end - t.begin; }
  __device__ __forceinline__ bf16_t* out(const Tile256& t) const {
    return static_cast<bf16_t*>(a.out) + ((int64_t)t.e * a.M + t.m0) * a.N;
  }
  __device__ __forceinline__ Operand p(const Tile256& t) const {
    return Operand{static_cast<const char*>(a.p) + (int64_t)t.begin * a.M * 2, nullptr, 0, k(t), t.m0, a.M};
  }
  __device__ __forceinline__ Operand q(const Tile256& t) const {
    const char* x = static_cast<const char*>(a.q);
    if (GATHER) return Operand{x, a.rows + t.begin, (int32_t)a.x_rows, k(t), t.n0, a.N};
    return Operand{x + (int64_t)t.begin * a.N * 2, nullptr, 0, k(t), t.n0, a.N};
  }
};

template <bool GATHER>
__global__ __launch_bounds__(512, 2) void k_weight_product(ProdArgs a) {
  __shared__ __attribute__((aligned(16))) char lds[WeightWalk<GATHER>::Sh::LDS];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Spread s = spread(a.offsets, a.experts, (int)a.n, lane);
  int rank = lane;
  if (s.per == 1) {
    const int mine = s.hi - s.lo;
    rank = 0;
    for (int j = 0; j < 64; ++j) {
      const int other = __builtin_amdgcn_readlane(mine, j);
      rank += other > mine || (other == mine && j < lane);
    }
  }
  const uint32_t tiles = (uint32_t)a.tiles_m * (uint32_t)a.tiles_n, sets = (tiles + 31) / 32;
  WeightWalk<GATHER> o{a, s, rank, 0, sets, (tiles + sets - 1) / sets};
  walk(lds, a.N, lane, w, o);
}

// --------------------------------------------------------------------- host

constexpr int64_t kMaxSide = (int64_t(1) << 24) - 1;

int check_product(int dtype, int64_t n, int64_t x_rows, int experts, int64_t outer, int64_t inner) {
  if (!good_dtype(dtype)) return fail(MUON_EUNSUPPORTED, "unsupported dtype");
  if (n < 0 || x_rows < 0 || experts < 1 || outer < 1 || inner < 1)
    return fail(MUON_EINVAL, "rows must be >= 0; experts, outer and inner >= 1");
  if (experts > kMaxExperts) return fail(MUON_EUNSUPPORTED, "more than 1024 experts");
  if (n > kMaxCount || x_rows > kMaxCount) return fail(MUON_EUNSUPPORTED, "2^31 rows or more");
  if (outer > kMaxSide || inner > kMaxSide) return fail(MUON_EUNSUPPORTED, "a matrix side of 2^24 or more");
  return MUON_OK;
}

int64_t side(int dtype) { return dtype == MUON_BF16 ? Tile<bf16_t>::B : Tile<float>::B; }

// Row tiles that n rows of `experts` experts (and the rows past them) can make.
int64_t row_tiles(int64_t n, int experts, int64_t b) {
  const int64_t cut = n < experts + 1 ? n : experts + 1;
  return n / b + cut;
}

template <int MODE>
int launch_product(ProdArgs a, int dtype, int64_t tiles_m, hipStream_t s) {
  a.tiles_n = (int32_t)ceil_div(a.N, side(dtype));
  const int64_t blocks = tiles_m * a.tiles_n;
  if (blocks > kMaxCount) return fail(MUON_EUNSUPPORTED, "more than 2^31 output tiles");
  const dim3 grid = grid_of_blocks(blocks, 256, (uint32_t)a.parts);
  if (dtype == MUON_BF16) hipLaunchKernelGGL((k_product<bf16_t, MODE>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((k_product<float, MODE>), grid, dim3(256), 0, s, a);
  return launch_status("grouped product launch");
}

// Whether the kernels for few rows take a rows product (and their blocks): where
// an expert has so few rows that its matrix's way from memory is what counts, or
// where the tile kernels would leave most CUs idle for one tile's length.
// Measured against the faster tile kernel, us (even experts):
//   n / experts 4, bf16, 64 x 2816 x 2048: 145 against 159 (input gradient 135, 128); at 8: 152, 160 (140, 128)
//   16, fp32, 64 x 1408 x 1024: 93 against 122 (75, 113); at 32: 159, 124 (108, 116)
//   blocks 1280, 8 x 1024 x 1024, bf16 16 against 16, fp32 30 against 32; 2560: 27, 23 and 51, 48
//   blocks 513, fp32, 8 x 257 x 513: 11 against 19
template <int MODE>
bool few(const ProdArgs& a, int dtype, int64_t* blocks) {
  *blocks = row_tiles(a.n, a.experts, 16) * ceil_div(a.N, MODE == kMatmul ? 32 : 64);
  return *blocks <= 1280 || (a.n <= (dtype == MUON_BF16 ? 4 : 16) * (int64_t)a.experts && *blocks <= kMaxCount);
}

template <int MODE>
int launch_few(ProdArgs a, int dtype, int64_t blocks, hipStream_t s) {
  a.tiles_n = (int32_t)ceil_div(a.N, MODE == kMatmul ? 32 : 64);
  const dim3 grid = grid_of_blocks(blocks, MODE == kMatmul ? 256 : 512);
  if (MODE == kMatmul) {
    if (dtype == MUON_BF16) hipLaunchKernelGGL((k_few_matmul<bf16_t, 2>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((k_few_matmul<float, 2>), grid, dim3(256), 0, s, a);
  } else {
    if (dtype == MUON_BF16) hipLaunchKernelGGL((k_few_input_grad<bf16_t>), grid, dim3(512), 0, s, a);
    else hipLaunchKernelGGL((k_few_input_grad<float>), grid, dim3(512), 0, s, a);
  }
  return launch_status("grouped product launch");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// The large kernels copy 16-byte chunks that a row holds whole and address an
// operand (that of gathered rows whole, else one tile's rows) by 31 bits.
bool chunked_sides(int dtype, int64_t c0, int64_t c1) {
  return dtype == MUON_BF16 && c0 % 8 == 0 && c1 % 8 == 0 && c0 < (1 << 21) && c1 < (1 << 21);
}
bool gathered_whole(int64_t x_rows, int64_t cols) { return x_rows * cols < (int64_t(1) << 30); }
bool chunked(const ProdArgs& a, int dtype, int64_t c0, int64_t c1, int64_t gathered_cols) {
  return chunked_sides(dtype, c0, c1) && aligned16(a.p) && aligned16(a.q) && aligned16(a.out) &&
         (!a.rows || gathered_whole(a.x_rows, gathered_cols));
}

template <int MODE>
int launch_rows(ProdArgs a, hipStream_t s) {
  a.tiles_n = (int32_t)ceil_div(a.N, 256);
  if (row_tiles(a.n, a.experts, 256) * a.tiles_n > kMaxCount)
    return fail(MUON_EUNSUPPORTED, "more than 2^31 output tiles");
  hipLaunchKernelGGL((k_rows_product<MODE>), dim3(kWalkers), dim3(512), 0, s, a);
  return launch_status("grouped product launch");
}

int launch_weight(ProdArgs a, hipStream_t s) {
  a.tiles_m = (int32_t)ceil_div(a.M, 256);
  a.tiles_n = (int32_t)ceil_div(a.N, 256);
  if ((int64_t)a.experts * a.tiles_m * a.tiles_n > kMaxCount / 2)   // 32 sets of 17 tiles are counted as 32 x 32 at most
    return fail(MUON_EUNSUPPORTED, "more than 2^30 output tiles");
  if (a.rows) hipLaunchKernelGGL((k_weight_product<true>), dim3(kWalkers), dim3(512), 0, s, a);
  else hipLaunchKernelGGL((k_weight_product<false>), dim3(kWalkers), dim3(512), 0, s, a);
  return launch_status("grouped weight gradient launch");
}

// Whether the weight gradient takes the small tiles although its rows would let
// it take the large ones, and the parts into which these cut an expert's rows.
// Small: at most one large tile a CU and few rows (8 x 1024 x 1024, 8 to 256
// rows: 9 to 11 us against 12 to 13; 1024 rows: 18 against 17), or so few large
// tiles that most CUs would idle over long sums.  Parts: until there are two
// blocks a CU, two k-tiles in a part on average.  Without and with them, us (bf16):
//   9 x 192 x 208, 26960 rows:  99, 29    5 x 64 x 1280, 28945 rows: 89, 40
//   2 x 512 x 512, 16384 rows: 185, 40    6 x 2752 x 64, 8016 rows:  28, 29
// With 128 large tiles (8 x 1024 x 1024, 16384 rows) the small ones take 141 us, the large ones 95; 128 x 128 x 128,
// 100000 rows, 24 in parts, 16.  No parts, and so no workspace, where the large ones take the sizes; the few calls of
// these whose arrays are off 16 bytes: 128 x 128 x 128, 100000 rows 21 without parts, 24 with; 64 x 64 20, 16.
struct WeightCut {
  bool small;
  int parts;
};
WeightCut weight_cut(int dtype, int64_t n, int64_t x_rows, int experts, int64_t outer, int64_t inner) {
  const int64_t large = experts * ceil_div(outer, 256) * ceil_div(inner, 256);
  const int64_t tiles = experts * ceil_div(outer, side(dtype)) * ceil_div(inner, side(dtype));
  const int64_t k_tile = dtype == MUON_BF16 ? Tile<bf16_t>::BK : Tile<float>::BK;
  const int64_t most = n / (experts * 2 * k_tile);
  int64_t parts = 2 * kWalkers / tiles;
  if (parts > most) parts = most;
  if (parts > 64) parts = 64;
  const bool few = large <= kWalkers && n <= 64 * (int64_t)experts;
  const bool by_large = large > 96 && chunked_sides(dtype, outer, inner) && gathered_whole(x_rows, inner);
  if (few || by_large || parts < 1) parts = 1;
  return WeightCut{few || (large <= 96 && parts > 1), (int)parts};
}

uint64_t dense_bytes(int dtype, int64_t x_rows, int64_t inner) {
  return ((uint64_t)x_rows * inner * (dtype == MUON_BF16 ? 2 : 4) + 15) / 16 * 16;
}
// Workspace of the weight gradient: a checkpoint's rows as dense values (`kept`; where there are rows to sum), and
// the parts' sums.
uint64_t weight_grad_bytes(int dtype, int64_t n, int64_t x_rows, int experts, int64_t outer, int64_t inner, bool kept) {
  const int parts = weight_cut(dtype, n, x_rows, experts, outer, inner).parts;
  return (kept && n > 0 ? dense_bytes(dtype, x_rows, inner) : 0) +
         (parts > 1 ? (uint64_t)parts * experts * outer * inner * 4 : 0);
}

}  // namespace
}  // namespace ex
}  // namespace muon

using namespace muon::ex;

extern "C" {

int muon_grouped_matmul(const void* x, const void* w, const int32_t* offsets, const int32_t* rows, int dtype,
                        int64_t n, int64_t x_rows, int experts, int64_t outer, int64_t inner, void* y, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_product(dtype, n, x_rows, experts, outer, inner))) return rc;
  if (n > 0 && !rows && x_rows != n) return fail(MUON_EINVAL, "x_rows must be n where rows is NULL");
  if (n == 0) return MUON_OK;
  if ((!x && x_rows) || !w || !offsets || !y) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  ProdArgs a = {x, w, y, offsets, rows, n, x_rows, experts, 0, (int32_t)outer, (int32_t)inner, 0, 0, 1, nullptr};
  int64_t blocks;
  if (few<kMatmul>(a, dtype, &blocks)) return launch_few<kMatmul>(a, dtype, blocks, static_cast<hipStream_t>(stream));
  if (chunked(a, dtype, inner, outer, inner))
    return launch_rows<kMatmul>(a, static_cast<hipStream_t>(stream));
  return launch_product<kMatmul>(a, dtype, row_tiles(n, experts, side(dtype)), static_cast<hipStream_t>(stream));
}

int muon_grouped_input_grad(const void* dy, const void* w, const int32_t* offsets, int dtype, int64_t n, int experts,
                            int64_t outer, int64_t inner, void* dx, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_product(dtype, n, n, experts, outer, inner))) return rc;
  if (n == 0) return MUON_OK;
  if (!dy || !w || !offsets || !dx) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  ProdArgs a = {dy, w, dx, offsets, nullptr, n, n, experts, 0, (int32_t)inner, (int32_t)outer, 0, 0, 1, nullptr};
  int64_t blocks;
  if (few<kInputGrad>(a, dtype, &blocks)) return launch_few<kInputGrad>(a, dtype, blocks, static_cast<hipStream_t>(stream));
  if (chunked(a, dtype, inner, outer, inner))
    return launch_rows<kInputGrad>(a, static_cast<hipStream_t>(stream));
  return launch_product<kInputGrad>(a, dtype, row_tiles(n, experts, side(dtype)), static_cast<hipStream_t>(stream));
}

int muon_grouped_weight_grad_workspace(int dtype, int64_t n, int64_t x_rows, int experts, int64_t outer,
                                       int64_t inner, int checkpoint, uint64_t* bytes) {
  muon::report_error(MUON_OK, "");
  if (!bytes) return fail(MUON_EINVAL, "NULL bytes");
  const int rc = check_product(dtype, n, x_rows, experts, outer, inner);
  if (rc) return rc;
  *bytes = weight_grad_bytes(dtype, n, x_rows, experts, outer, inner, checkpoint != 0);
  return MUON_OK;
}

int muon_grouped_weight_grad(const void* dy, const void* x, const void* q, const uint8_t* scale, int kind,
                             const int32_t* offsets, const int32_t* rows, int dtype, int64_t n, int64_t x_rows,
                             int experts, int64_t outer, int64_t inner, void* dw, void* workspace,
                             uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  const bool kept = q || scale;
  if ((rc = check_product(dtype, n, x_rows, experts, outer, inner))) return rc;
  if (n > 0 && !rows && x_rows != n) return fail(MUON_EINVAL, "x_rows must be n where rows is NULL");
  if (kept && x) return fail(MUON_EINVAL, "either x or its checkpoint, not both");
  if (kept && kind != MUON_INT8 && kind != MUON_E4M3) return fail(MUON_EUNSUPPORTED, "kind must be MUON_INT8 or MUON_E4M3");
  if (kept && x_rows > 0 && (!q || !scale)) return fail(MUON_EINVAL, "q and scale come together");
  if (!offsets || !dw || (n > 0 && !dy) || (n > 0 && x_rows > 0 && !kept && !x)) return fail(MUON_EINVAL, "NULL pointer");
  const uint64_t need = weight_grad_bytes(dtype, n, x_rows, experts, outer, inner, kept);
  if (need && (!workspace || workspace_bytes < need))
    return fail(MUON_EINVAL, "workspace of " + std::to_string(need) + " bytes needed");
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 15)) return fail(MUON_EINVAL, "workspace must be 16-byte aligned");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool restored = kept && n > 0;
  if (restored) {
    if ((rc = restore_rows(q, scale, kind, x_rows, inner, dtype, workspace, s))) return rc;
    x = workspace;
  }
  ProdArgs a = {dy, x, dw, offsets, rows, n, x_rows, experts, (int32_t)outer, (int32_t)inner, 0, 0, 0, 1, nullptr};
  const WeightCut cut = weight_cut(dtype, n, x_rows, experts, outer, inner);
  if (!cut.small && chunked(a, dtype, inner, outer, inner)) return launch_weight(a, s);
  a.tiles_m = (int32_t)ceil_div(outer, side(dtype));
  a.parts = cut.parts;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(workspace) + (restored ? dense_bytes(dtype, x_rows, inner) : 0));
  if ((rc = launch_product<kWeightGrad>(a, dtype, (int64_t)experts * a.tiles_m, s)) || cut.parts == 1) return rc;
  const int64_t count = experts * outer * inner;
  const dim3 grid((uint32_t)ceil_div(count, 1024));
  if (dtype == MUON_BF16)
    hipLaunchKernelGGL((k_add_parts<bf16_t>), grid, dim3(256), 0, s, a.partial, static_cast<bf16_t*>(dw), count, cut.parts);
  else
    hipLaunchKernelGGL((k_add_parts<float>), grid, dim3(256), 0, s, a.partial, static_cast<float*>(dw), count, cut.parts);
  return launch_status("weight gradient parts launch");
}

}  // extern "C"
