// What the kernels of the products grouped by expert share: their arguments,
// which rows a block has, and accesses to rows of any length and alignment.
#pragma once
#include "experts.hpp"

namespace muon {
namespace ex {

enum Mode { kMatmul = 0, kInputGrad = 1, kWeightGrad = 2 };

struct ProdArgs {
  const void* p;            // x, dy, dy
  const void* q;            // W, W, x
  void* out;
  const int32_t* offsets;
  const int32_t* rows;      // gather of x's rows, or null
  int64_t n, x_rows;
  int32_t experts;
  int32_t M, N, K;          // M: weight grad only; K: not in the weight grad
  int32_t tiles_m, tiles_n; // tiles_m: weight grad only
  int32_t parts;            // weight grad by small tiles: parts of an expert's rows, 1 or more
  float* partial;           // with more than one: their sums, [parts][experts][M][N]
};

// Tile t of the rows cut by expert into tiles of 2^SH: expert and rows
// [begin, end) of the tile, end at most begin + 2^SH.  The rows past the last
// expert's are cut the same way, as those of expert `experts`.  Offsets are
// taken as their running maximum in [0, n], so that no input leads out of
// bounds.  Every wave of a block calls this with the same t; false: no such
// tile.
struct RowTile {
  int e;
  int64_t begin, end;
};
template <int SH>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ offsets, int experts, int n, int64_t t, int lane,
                                          RowTile& out) {
  int last = 0;       // end of the experts before this round of 64
  int64_t seen = 0;   // their tiles
  for (int e0 = 0; e0 < experts; e0 += 64) {
    int hi = e0 + lane < experts ? offsets[e0 + lane + 1] : 0;
    hi = hi > n ? n : hi;
    hi = wave_scan_max(hi > last ? hi : last, lane);
    int lo = __shfl_up(hi, 1, 64);
    if (lane == 0) lo = last;
    const int tiles = (int)(((uint32_t)(hi - lo) + (1u << SH) - 1) >> SH);
    const int upto = wave_scan_add(tiles, lane);
    const uint64_t hit = __ballot(t < seen + upto);
    if (hit) {
      const int at = __ffsll((unsigned long long)hit) - 1;
      const int b = __builtin_amdgcn_readlane(lo, at), e = __builtin_amdgcn_readlane(hi, at);
      const int before = __builtin_amdgcn_readlane(upto - tiles, at);
      out.e = e0 + at;
      out.begin = b + ((t - seen - before) << SH);
      out.end = out.begin + (1 << SH) < e ? out.begin + (1 << SH) : e;
      return true;
    }
    last = __builtin_amdgcn_readlane(hi, 63);
    seen += __builtin_amdgcn_readlane(upto, 63);
  }
  out.e = experts;
  out.begin = last + ((t - seen) << SH);
  out.end = out.begin + (1 << SH) < n ? out.begin + (1 << SH) : n;
  return out.begin < n;
}

// Rows [begin, end) of expert e, by the same reading of offsets.
__device__ __forceinline__ void expert_rows(const int32_t* __restrict__ offsets, int e, int n, int lane, int64_t& begin,
                                            int64_t& end) {
  int b = 0, m = 0;   // maxima of offsets[1..e] and of offsets[1..e+1]
  for (int i = lane; i <= e; i += 64) {
    const int v = offsets[i + 1];
    m = v > m ? v : m;
    if (i < e) b = v > b ? v : b;
  }
  b = (int)wave_max((uint32_t)b);
  m = (int)wave_max((uint32_t)m);
  begin = b < n ? b : n;
  end = m < n ? m : n;
}

// 16 bytes from any address, of which the first cnt elements exist.
__device__ __forceinline__ u32x4 load16(const bf16_t* p, int cnt) {
  if (cnt >= 8) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) v[i / 2] |= (uint32_t)p[i].bits << (16 * (i % 2));
  return v;
}
__device__ __forceinline__ u32x4 load16(const float* p, int cnt) {
  if (cnt >= 4) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < cnt) v[i] = __float_as_uint(p[i]);
  return v;
}

__device__ __forceinline__ void store4(bf16_t* p, int cnt, const float* v) {
  if (cnt >= 4) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) store1(p + i, v[i]);
  }
}
__device__ __forceinline__ void store4(float* p, int cnt, const float* v) {
  if (cnt >= 4) {
    *reinterpret_cast<u32x4_any*>(p) =
        u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < cnt) p[i] = v[i];
  }
}

}  // namespace ex
}  // namespace muon
