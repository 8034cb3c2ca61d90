// What the expert-layer operators (expert_rows.hip, expert_products.hip)
// share: bounds of their arguments, the device check, and the device helpers
// that read and write rows of any length and alignment.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "errors.hpp"
#include "muon.h"

namespace muon {
namespace ex {

constexpr int kMaxExperts = 1024;    // route: 16 logits a lane; products: the offsets one wave scans
constexpr int kMaxTopK = 64;         // route: one lane of a wave holds each choice
constexpr int kBlock = 32;           // columns of one row that share a checkpoint scale
constexpr int64_t kMaxCount = (int64_t(1) << 31) - 1;   // rows are int32 indices

inline int fail(int code, const std::string& msg) { return report_error(code, msg); }

// MUON_OK when the current device is a gfx950; the answer is looked up once
// per device.
int check_device();

inline int launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return fail(MUON_EHIP, std::string(what) + ": " + hipGetErrorString(e));
  return MUON_OK;
}

inline bool good_dtype(int d) { return d == MUON_F32 || d == MUON_BF16; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A grid of `blocks` >= 1 blocks.  A launch takes less than 2^32 threads along x:
// more blocks are laid out in rows along y, the last of which can go past
// `blocks`.  block_index() is a block's number in it.
inline dim3 grid_of_blocks(int64_t blocks, uint32_t threads, uint32_t z = 1) {
  const int64_t y = ceil_div(blocks, ((int64_t(1) << 32) - 1) / threads);
  return dim3((uint32_t)ceil_div(blocks, y), (uint32_t)y, z);
}

// ------------------------------------------------------------------ device

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// 16 and 8 bytes at any address: gfx950 global accesses take unaligned
// addresses, so a row that starts anywhere is read with the same instruction.
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ int64_t block_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

struct bf16_t { uint16_t bits; };

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }
// two fp32 to bf16, round to nearest even, NaN kept
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(bf16_t* p, float v) { p->bits = (uint16_t)pack2(v, 0.f); }

// Eight consecutive elements from any address, of which the first cnt exist;
// the others are zero and not touched in memory.
__device__ __forceinline__ void load8(const bf16_t* p, int cnt, float (&v)[8]) {
  if (cnt >= 8) {
    const u32x4 t = *reinterpret_cast<const u32x4_any*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(t[i] << 16);
      v[2 * i + 1] = __uint_as_float(t[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cnt ? to_f32(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* p, int cnt, float (&v)[8]) {
  if (cnt >= 8) {
    const u32x4 a = *reinterpret_cast<const u32x4_any*>(p);
    const u32x4 b = *reinterpret_cast<const u32x4_any*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cnt ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void store8(bf16_t* p, int cnt, const float (&v)[8]) {
  if (cnt >= 8) {
    *reinterpret_cast<u32x4_any*>(p) =
        u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) store1(p + i, v[i]);
  }
}
__device__ __forceinline__ void store8(float* p, int cnt, const float (&v)[8]) {
  if (cnt >= 8) {
    *reinterpret_cast<u32x4_any*>(p) = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]),
                                             __float_as_uint(v[2]), __float_as_uint(v[3])};
    *reinterpret_cast<u32x4_any*>(p + 4) = u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]),
                                                 __float_as_uint(v[6]), __float_as_uint(v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = v[i];
  }
}

// 2^n exactly, n in [-126, 127]
__device__ __forceinline__ float pow2f(int n) { return __uint_as_float((uint32_t)(n + 127) << 23); }

// Maximum over the wave by DPP: within rows of 16, then across them; lane 63
// holds the result.  Lanes without a source keep their own value.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#define MUON_DPP_MAX(ctrl, rows)                                                                          \
  {                                                                                                       \
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, ctrl, rows, 0xf, false);     \
    v = o > v ? o : v;                                                                                    \
  }
  MUON_DPP_MAX(0x111, 0xf)   // row_shr:1
  MUON_DPP_MAX(0x112, 0xf)   // row_shr:2
  MUON_DPP_MAX(0x114, 0xf)   // row_shr:4
  MUON_DPP_MAX(0x118, 0xf)   // row_shr:8
  MUON_DPP_MAX(0x142, 0xa)   // row_bcast:15 into rows 1 and 3
  MUON_DPP_MAX(0x143, 0xc)   // row_bcast:31 into rows 2 and 3
#undef MUON_DPP_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Inclusive scans over the wave.
__device__ __forceinline__ int wave_scan_add(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(v, o, 64);
    if (lane >= o) v += t;
  }
  return v;
}
__device__ __forceinline__ int wave_scan_max(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(v, o, 64);
    if (lane >= o && t > v) v = t;
  }
  return v;
}

}  // namespace ex
}  // namespace muon
