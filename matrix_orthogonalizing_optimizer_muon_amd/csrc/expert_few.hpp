// Products grouped by expert for few rows: what counts is how fast the experts'
// matrices come from memory.  A block has 16 rows of one expert and a narrow
// strip of output columns, its waves split k, and each brings its part of the
// matrix straight into the MFMA operands, several loads ahead, with no LDS in
// between (nothing is used twice); the waves' sums are added through LDS in a
// fixed order.
//
// v_mfma 16x16x32 (bf16) or 16x16x4 (fp32): lane l gives k values of row l % 16
// of either operand, and gets rows 4 (l / 16) + 0..3, column l % 16 of the
// product; the matrix is the first operand, so a lane holds one row of the
// output and consecutive columns of it.
#pragma once
#include "expert_tiles.hpp"
#include "mfma_nt.hpp"

namespace muon {
namespace ex {

typedef nt::f32x4_t Acc16;

template <class T>
struct Few {};
template <>
struct Few<bf16_t> {
  static constexpr int PER = 8;   // k values of a 16-byte chunk
};
template <>
struct Few<float> {
  static constexpr int PER = 4;
};

// One chunk of k values of both operands, in the same order.
__device__ __forceinline__ Acc16 multiply16(u32x4 w, u32x4 x, Acc16 acc, bf16_t) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(nt::bf16x8_t, w),
                                                 __builtin_bit_cast(nt::bf16x8_t, x), acc, 0, 0, 0);
}
__device__ __forceinline__ Acc16 multiply16(u32x4 w, u32x4 x, Acc16 acc, float) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w[i]), __uint_as_float(x[i]), acc, 0, 0, 0);
  return acc;
}

// The row that lane % 16 of a block's rows reads, or null: it does not exist, or
// names no row of x and is read as zeros.
template <class T>
__device__ __forceinline__ const T* few_row(const ProdArgs& a, const RowTile& rt, int lane) {
  const int64_t r = rt.begin + (lane & 15);
  if (r >= rt.end) return nullptr;
  int64_t src = r;
  if (a.rows) {
    src = a.rows[r];
    if (src < 0 || src >= a.x_rows) return nullptr;
  }
  return static_cast<const T*>(a.p) + src * a.K;
}

// The waves' sums, added in order of the waves; thread t < 64 NQ gets group
// t / 64 of NQ, lane t % 64's values.
template <int NW, int NQ>
__device__ __forceinline__ bool few_sum(Acc16 (&acc)[NQ], Acc16* lds, Acc16& sum) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int c = 0; c < NQ; ++c) lds[(w * NQ + c) * 64 + lane] = acc[c];
  __syncthreads();
  if (w >= NQ) return false;
  sum = lds[w * 64 + lane];
#pragma unroll
  for (int v = 1; v < NW; ++v) {
    const Acc16 o = lds[(v * NQ + w) * 64 + lane];
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += o[i];
  }
  return true;
}

// y[r] = x[r] W_e^T: strips of 16 CT columns, k in steps of 64 bytes a row.
// Bound by the matrices' way from memory: 8 rows of 8 experts, 2816 x 2048 bf16,
// 92 MB: 20 us, 4.6 TB/s; 222 rows of 59 experts, 2048 x 1408, 341 MB: 65 us, 5.2 TB/s.
// A column that does not exist reads another's values instead, which reach only
// results that are not stored.  A row that x does not have is zeros (its product
// with an infinity is NaN, as in the tiles): in bf16 its lanes load nothing, in
// fp32 they load from the matrix and are masked, which leaves the loads among the
// products (389 tokens of 513 x 257: 9.9 us, 10.9 with the branch).
template <class T, int CT>
__global__ __launch_bounds__(256) void k_few_matmul(ProdArgs a) {
  constexpr int PER = Few<T>::PER, STEP = 4 * PER, NW = 4, U = 4;
  constexpr bool BRANCH = sizeof(T) == 2;
  __shared__ Acc16 lds[NW * CT * 64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = block_index(), tm = t / a.tiles_n;
  const int n0 = (int)(t - tm * a.tiles_n) * 16 * CT;
  RowTile rt;
  if (!find_tile<4>(a.offsets, a.experts, (int)a.n, tm, lane, rt)) return;
  const bool live = rt.e < a.experts;
  Acc16 acc[CT] = {};
  const T* xr = live ? few_row<T>(a, rt, lane) : nullptr;
  if (live) {
    const T* wp[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int n = n0 + 16 * c + (lane & 15);
      wp[c] = static_cast<const T*>(a.q) + ((int64_t)rt.e * a.N + (n < a.N ? n : a.N - 1)) * a.K;
    }
    const T* xp = xr ? xr : wp[0];
    uint32_t keep = xr ? ~0u : 0u;
    asm volatile("" : "+v"(keep));   // a mask: the compiler would make a condition a branch around loads
    const int steps = a.K / STEP, at = PER * (lane >> 4);
    int s = w;
    for (; s + NW * (U - 1) < steps; s += NW * U) {
      u32x4 fw[U][CT], fx[U] = {};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + NW * u) * STEP + at;
#pragma unroll
        for (int c = 0; c < CT; ++c) fw[u][c] = *reinterpret_cast<const u32x4_any*>(wp[c] + k);
        if constexpr (!BRANCH) fx[u] = *reinterpret_cast<const u32x4_any*>(xp + k);
      }
      if constexpr (BRANCH) {
        if (xr) {
#pragma unroll
          for (int u = 0; u < U; ++u) fx[u] = *reinterpret_cast<const u32x4_any*>(xr + (s + NW * u) * STEP + at);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = multiply16(fw[u][c], BRANCH ? fx[u] : fx[u] & keep, acc[c], T());
    }
    for (; s <= steps; s += NW) {   // the last one ends inside a chunk, or has nothing
      const int k = s * STEP + at, left = a.K - k;
      if (s == steps && a.K % STEP == 0) break;
      const u32x4 fx = (left > 0 ? load16(xp + k, left) : u32x4{0u, 0u, 0u, 0u}) & keep;
#pragma unroll
      for (int c = 0; c < CT; ++c)
        acc[c] = multiply16(left > 0 ? load16(wp[c] + k, left) : u32x4{0u, 0u, 0u, 0u}, fx, acc[c], T());
    }
  }
  Acc16 v;
  if (!few_sum<NW>(acc, lds, v)) return;
  const int64_t r = rt.begin + (lane & 15);
  const int col = n0 + 16 * w + 4 * (lane >> 4);
  if (r < rt.end && col < a.N) {
    const float o[4] = {v[0], v[1], v[2], v[3]};
    store4(static_cast<T*>(a.out) + r * a.N + col, a.N - col, o);
  }
}

// Four columns of one row of the matrix, in a strip of 64: columns 4 (lane % 16) on.
__device__ __forceinline__ u32x2 load_cols(const bf16_t* p, int cnt) {
  if (cnt >= 4) return *reinterpret_cast<const u32x2_any*>(p);
  u32x2 v = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < cnt) v[i / 2] |= (uint32_t)p[i].bits << (16 * (i % 2));
  return v;
}
__device__ __forceinline__ u32x4 load_cols(const float* p, int cnt) { return load16(p, cnt); }

// The k values of column c from the PER rows of a lane.
__device__ __forceinline__ u32x4 column(const u32x2 (&v)[8], int c) {
  u32x4 f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = __builtin_amdgcn_perm(v[2 * i + 1][c / 2], v[2 * i][c / 2], c % 2 ? 0x07060302u : 0x05040100u);
  return f;
}
__device__ __forceinline__ u32x4 column(const u32x4 (&v)[4], int c) { return u32x4{v[0][c], v[1][c], v[2][c], v[3][c]}; }

template <class T>
struct Cols {};
template <>
struct Cols<bf16_t> {
  typedef u32x2 type;
};
template <>
struct Cols<float> {
  typedef u32x4 type;
};

// dx[r] = dy[r] W_e: strips of 64 columns.  A lane has 4 of them of PER rows of
// the matrix, so the operand for column 4 (l % 16) + c is put together from
// registers, and the product of c is rows 4 (l / 16) + i: columns 16 (l / 16) + 4 i + c.
// 8 rows of 8 experts, 2816 x 2048 bf16: 19 us.
template <class T>
__global__ __launch_bounds__(512) void k_few_input_grad(ProdArgs a) {
  constexpr int PER = Few<T>::PER, STEP = 4 * PER, NW = 8, U = 2;
  typedef typename Cols<T>::type cols_t;
  __shared__ Acc16 lds[NW * 4 * 64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = block_index(), tm = t / a.tiles_n;
  const int n0 = (int)(t - tm * a.tiles_n) * 64;
  RowTile rt;
  if (!find_tile<4>(a.offsets, a.experts, (int)a.n, tm, lane, rt)) return;
  const bool live = rt.e < a.experts;
  Acc16 acc[4] = {};
  const T* xr = live ? few_row<T>(a, rt, lane) : nullptr;
  if (live) {
    const int col = n0 + 4 * (lane & 15), at = PER * (lane >> 4);
    const int cnt = a.N - col;   // columns from there
    const T* wp = static_cast<const T*>(a.q) + (int64_t)rt.e * a.N * a.K + (cnt > 0 ? col : 0);
    const int steps = a.K / STEP;
    int s = w;
    const bool whole = a.N - n0 >= 64;
    for (; whole && s + NW * (U - 1) < steps; s += NW * U) {
      cols_t v[U][PER];
      u32x4 fx[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (s + NW * u) * STEP + at;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[u][i] = load_cols(wp + (int64_t)(k + i) * a.N, 4);
        fx[u] = xr ? *reinterpret_cast<const u32x4_any*>(xr + k) : u32x4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[c] = multiply16(column(v[u], c), fx[u], acc[c], T());
    }
    for (; s <= steps; s += NW) {
      const int k = s * STEP + at, left = a.K - k;
      if (s == steps && a.K % STEP == 0) break;
      const u32x4 fx = xr && left > 0 ? load16(xr + k, left) : u32x4{0u, 0u, 0u, 0u};
      cols_t v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        v[i] = cols_t{};
        if (i < left && cnt > 0) v[i] = load_cols(wp + (int64_t)(k + i) * a.N, cnt);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] = multiply16(column(v, c), fx, acc[c], T());
    }
  }
  // value i of group c is column 16 (lane / 16) + 4 i + c: exchanged so that a thread has four neighbours
  Acc16 by[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) by[i] = Acc16{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
  Acc16 sum;
  if (!few_sum<NW>(by, lds, sum)) return;
  const int64_t r = rt.begin + (lane & 15);
  const int col = n0 + 16 * (lane >> 4) + 4 * w;
  if (r < rt.end && col < a.N) {
    const float o[4] = {sum[0], sum[1], sum[2], sum[3]};
    store4(static_cast<T*>(a.out) + r * a.N + col, a.N - col, o);
  }
}

}  // namespace ex
}  // namespace muon
