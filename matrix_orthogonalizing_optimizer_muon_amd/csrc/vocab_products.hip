// The classifier's three matrix products.
//
//   logits  l[s][v]   = sum_i x[rows[s]][i] w[v][i]      both k-contiguous
//   dx      dx[rows[s]][i] = sum_v dl[s][v] w[v][i]      w k-major
//   dw      dw[v][i]  = sum_s dl[s][v] x[rows[s]][i]     both k-major
//
// Logits are never stored: what leaves the first product is, for each slab of
// columns, a row's largest logit and the sum over it (kStats), these and
// exp((logit - largest) / tau) in as many bits as x has (kStatsExp, which k_rescale makes
// gradients of once the row's sum is known), or the logits' gradient without
// the targets' part (kGradient, where the sum is known before).
#include <hip/hip_runtime.h>

#include "expert_stage.hpp"
#include "vocab_loss.hpp"

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

// One output tile per block of 4 waves (2 x 2) and two LDS stages, as
// k_product's of the expert layer.  fp32: a k-tile's sum (32 products) is added to
// the total by itself, so that no value is rounded K / 2 times in a row (errors of
// the gradients of 389 x 4099 x 515: 4.0e-6 -> 1.2e-6 of their norm).
template <class T, int PRODUCT, int EPI>
__global__ __launch_bounds__(256) void k_tile(LossArgs a, int32_t tiles_n) {
  using G = Tile<T>;
  constexpr bool PT = PRODUCT == kDw, QT = PRODUCT != kLogits;
  constexpr int PB = PT ? G::BYTES_T : G::BYTES, QB = QT ? G::BYTES_T : G::BYTES;
  constexpr int W = G::B / 2, NT = W / 32;
  static_assert(W == Slab<T>::kCols, "a wave's columns are a slab");
  __shared__ __attribute__((aligned(16))) char lds[2 * (PB + QB)];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, wy = w >> 1, wx = w & 1;
  const int64_t t = block_index();
  const int64_t tm = t / tiles_n;
  const int32_t n0 = (int32_t)(t - tm * tiles_n) * G::B;
  const int64_t m0 = tm * G::B;
  const int32_t live = live_slots(a.ch);
  const int32_t* rows = a.ch.rows + a.ch.slot0;
  int64_t m_left;
  int32_t K;
  Stager<T, PT> sp;
  Stager<T, QT> sq;
  if constexpr (PRODUCT == kLogits) {
    m_left = live - m0;
    if (m_left <= 0) return;
    K = a.dim;
    sp.init(a.x, rows, m0, m_left, a.tokens, 0, a.dim);
    sq.init(a.w, nullptr, n0, a.vocab - n0, 0, 0, a.dim);
  } else if constexpr (PRODUCT == kDx) {
    m_left = live - m0;
    if (m_left <= 0) return;
    K = a.vocab;
    sp.init(a.dl, nullptr, m0, m_left, 0, 0, a.vocab);
    sq.init(a.w, nullptr, 0, K, 0, n0, a.dim);
  } else {
    m_left = a.vocab - m0;
    if (m_left <= 0) return;
    K = live;
    sp.init(a.dl, nullptr, 0, K, 0, (int32_t)m0, a.vocab);
    sq.init(a.x, rows, 0, K, a.tokens, n0, a.dim);
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
      sp.commit(next);
      sq.commit(next + PB);
    }
  }
  // lane l has row l % 32 of a 32 x 32 tile, registers 4 g + 0..3 columns 8 g + 4 (l / 32) + 0..3
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t r = m0 + wy * W + 32 * i + (lane & 31);
    const bool exists = r < m0 + m_left;
    const int32_t c0 = n0 + wx * W + 4 * (lane >> 5);
    if constexpr (PRODUCT == kLogits) {
      if (n0 + wx * W >= a.vocab) continue;   // uniform over the wave
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
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            e[j][v] = __builtin_amdgcn_exp2f((e[j][v] - base) * a.to_log2);
            if (c0 + 32 * j + 8 * (v / 4) + v % 4 < a.vocab) sum += e[j][v];
          }
        sum += __shfl_xor(sum, 32, 64);
        if (exists && lane < 32) {
          float* st = a.stats + 2 * ((int64_t)((n0 + wx * W) / W) * a.ch.size + r);
          st[0] = top;
          st[1] = sum;
        }
      } else {
        const float base = exists ? a.base[r] : 0.f, g = exists ? a.g[r] : 0.f;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int v = 0; v < 16; ++v) e[j][v] = probability(a, e[j][v], base, g);
      }
      if constexpr (EPI != kStats) {
        if (exists) {
          T* out = static_cast<T*>(a.dl) + r * a.vocab;
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
      const int64_t at = (PRODUCT == kDx ? (int64_t)rows[r] : r) * a.dim;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int32_t c = c0 + 32 * j + 8 * q;
          float v[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
          if (PRODUCT == kDw && !a.first) {
            const u32x4 before = load16(a.sums + at + c, a.dim - c);
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] += __uint_as_float(before[u]);
          }
          if (PRODUCT == kDx) store4(static_cast<T*>(a.dx) + at + c, a.dim - c, v);
          else if (a.last) store4(static_cast<T*>(a.dw) + at + c, a.dim - c, v);
          else store4(a.sums + at + c, a.dim - c, v);
        }
    }
  }
}

template <class T, int PRODUCT, int EPI>
int launch_tile(const LossArgs& a, int64_t m, int64_t n, hipStream_t s) {
  const int64_t tiles_n = ceil_div(n, Tile<T>::B), blocks = ceil_div(m, Tile<T>::B) * tiles_n;
  hipLaunchKernelGGL((k_tile<T, PRODUCT, EPI>), grid_of_blocks(blocks, 256), dim3(256), 0, s, a, (int32_t)tiles_n);
  return launch_status("classifier product launch");
}

template <class T>
int launch_logits(const LossArgs& a, Epilogue e, hipStream_t s) {
  if (e == kStats) return launch_tile<T, kLogits, kStats>(a, a.ch.size, a.vocab, s);
  if (e == kStatsExp) return launch_tile<T, kLogits, kStatsExp>(a, a.ch.size, a.vocab, s);
  return launch_tile<T, kLogits, kGradient>(a, a.ch.size, a.vocab, s);
}

}  // namespace

int logits_product(const LossArgs& a, int dtype, Epilogue e, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_logits<bf16_t>(a, e, s) : launch_logits<float>(a, e, s);
}

int dx_product(const LossArgs& a, int dtype, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_tile<bf16_t, kDx, kStats>(a, a.ch.size, a.dim, s)
                            : launch_tile<float, kDx, kStats>(a, a.ch.size, a.dim, s);
}

int dw_product(const LossArgs& a, int dtype, hipStream_t s) {
  return dtype == MUON_BF16 ? launch_tile<bf16_t, kDw, kStats>(a, a.vocab, a.dim, s)
                            : launch_tile<float, kDw, kStats>(a, a.vocab, a.dim, s);
}

}  // namespace vo
}  // namespace muon
