// The row-wise operators of a mixture-of-experts layer: the router and its
// gradient, the weighted sum of expert outputs back to their tokens and its
// gradient, checkpoints of activations in 8 bits, and the gated activation
// with or without such a checkpoint.  All of them are bound by memory (or by
// latency, for a few tokens); each reads its inputs and writes its outputs
// once.  Statistics, sums and products are fp32.
#include <hip/hip_runtime.h>

#include <cstring>
#include <mutex>

#include "experts.hpp"

namespace muon {
namespace ex {

int check_device() {
  static std::mutex mu;
  static bool known[64] = {};
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return fail(MUON_EHIP, std::string("hipGetDevice: ") + hipGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(MUON_EUNSUPPORTED, "device index out of range");
  std::lock_guard<std::mutex> lk(mu);
  if (known[dev]) return MUON_OK;
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) return fail(MUON_EHIP, std::string("hipGetDeviceProperties: ") + hipGetErrorString(e));
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0)
    return fail(MUON_EUNSUPPORTED, std::string("device is ") + prop.gcnArchName + ", not gfx950");
  known[dev] = true;
  return MUON_OK;
}

namespace {

constexpr int kTokensPerBlock = 64;   // a block's tokens: one bit each of a 64-bit word per expert
constexpr int kRouteThreads = 1024;

// x / d for x < 2^31: (mulhi(x, m) + x) >> s with s = ceil(log2 d)
struct FastDiv {
  uint32_t d, m, s;
};
FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  return FastDiv{d, (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1), s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t x, FastDiv f) { return (__umulhi(x, f.m) + x) >> f.s; }

// ------------------------------------------------------------------- router

// Order-preserving code of a logit: NaN counts as -inf, +inf as the largest
// finite value, -0 as +0.  kGone marks what was already taken (or does not
// exist); every real code, that of -inf included, is above it.
constexpr uint32_t kGone = 0u;
constexpr uint32_t kMasked = 0x007fffffu;   // the code of -inf

__device__ __forceinline__ float clean_logit(float l) {
  l = l != l ? -INFINITY : l;
  return fminf(l, 3.402823466e38f) + 0.f;
}
__device__ __forceinline__ uint32_t order_code(float l) {
  const uint32_t b = __float_as_uint(l);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_code(uint32_t c) {
  return __uint_as_float(c & 0x80000000u ? c ^ 0x80000000u : ~c);
}

// The k largest logits of one token, by one wave; lane j holds choice j (its
// logit and expert, -inf and -1 where nothing is left).  Lane l holds experts
// l, 64 + l, ...; the lowest index among equals is the first word v whose
// ballot is not empty, at its lowest lane.
template <int V>
__device__ __forceinline__ void choose(const float (&l)[V], int experts, int k, int lane, float& top, int& id) {
  uint32_t c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = lane + 64 * v < experts ? order_code(l[v]) : kGone;
  top = -INFINITY;
  id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t best = c[0];
#pragma unroll
    for (int v = 1; v < V; ++v) best = c[v] > best ? c[v] : best;
    const uint32_t m = wave_max(best);
    if (m <= kMasked) break;
    bool found = false;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const uint64_t hit = __ballot(c[v] == m);
      if (!found && hit) {
        found = true;
        const int at = __ffsll((unsigned long long)hit) - 1;
        if (lane == at) c[v] = kGone;
        if (lane == j) {
          top = from_code(m);
          id = 64 * v + at;
        }
      }
    }
  }
}

// The same for up to 16 choices of up to 256 experts by 16 lanes, so that a
// wave takes four tokens at once and a round costs it a quarter: lane l of a
// row holds experts l V to (l + 1) V - 1.  top0: the first choice's logit, in every lane.
#define MUON_ROW_STEP(op, v, o, ctrl)                                                                \
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false);                       \
  v = op
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  uint32_t o;
  MUON_ROW_STEP(o > v ? o : v, v, o, 0x128);   // row_ror:8, 4, 2, 1
  MUON_ROW_STEP(o > v ? o : v, v, o, 0x124);
  MUON_ROW_STEP(o > v ? o : v, v, o, 0x122);
  MUON_ROW_STEP(o > v ? o : v, v, o, 0x121);
  return v;
}
__device__ __forceinline__ uint32_t row_min(uint32_t v) {
  uint32_t o;
  MUON_ROW_STEP(o < v ? o : v, v, o, 0x128);
  MUON_ROW_STEP(o < v ? o : v, v, o, 0x124);
  MUON_ROW_STEP(o < v ? o : v, v, o, 0x122);
  MUON_ROW_STEP(o < v ? o : v, v, o, 0x121);
  return v;
}
#undef MUON_ROW_STEP
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int V>
__device__ __forceinline__ void choose_row(const float (&l)[V], int experts, int k, int li, float& top, int& id,
                                           float& top0) {
  uint32_t c[V];
#pragma unroll
  for (int v = 0; v < V; ++v) c[v] = li * V + v < experts ? order_code(l[v]) : kGone;
  top = top0 = -INFINITY;
  id = -1;
  for (int j = 0; j < k; ++j) {
    uint32_t m = c[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = c[v] > m ? c[v] : m;
    m = row_max(m);
    uint32_t e = 0xffffffffu;
#pragma unroll
    for (int v = V - 1; v >= 0; --v) e = c[v] == m ? (uint32_t)(li * V + v) : e;
    e = row_min(e);
#pragma unroll
    for (int v = 0; v < V; ++v) c[v] = e == (uint32_t)(li * V + v) ? kGone : c[v];
    const bool some = m > kMasked;
    if (j == 0 && some) top0 = from_code(m);
    if (li == j && some) {
      top = from_code(m);
      id = (int)e;
    }
  }
}

struct RouteArgs {
  const void* logits;
  float* weights;
  int32_t* chosen;
  int32_t* slots;
  int32_t* rows;
  int32_t* offsets;
  uint64_t* mask;      // [blocks][experts]: which of the block's tokens chose the expert
  uint8_t* count;      // [experts][stride]: how many of them; a row is a multiple of 16 bytes
  uint32_t* ahead;     // with the scan, [experts][blocks]: how many in earlier blocks
  uint32_t* total;     // with the scan, [experts]
  int64_t tokens;
  int32_t experts, k, normalize, blocks, stride;
};

// Places of one block's choices: an expert's rows are in order of the tokens,
// and a token chooses an expert once, so a choice's rank in its block is the
// number of lower tokens in the expert's mask.  before[e]: rows ahead of this
// block's rows of expert e.  The places past the last row are marked -1.
__device__ __forceinline__ void place(const RouteArgs& a, const uint64_t* mask, const uint32_t* before,
                                      uint32_t live, int64_t t0, int tokens) {
  for (int p = threadIdx.x; p < tokens * a.k; p += kRouteThreads) {
    const int64_t at = t0 * a.k + p;
    const int tl = p / a.k;
    const int id = a.chosen[at];
    int slot = -1;
    if (id >= 0) {
      slot = (int)(before[id] + __popcll(mask[id] & ((1ull << tl) - 1)));
      a.rows[slot] = (int32_t)(t0 + tl);
    }
    a.slots[at] = slot;
    if (at >= live) a.rows[at] = -1;
  }
}

// Exclusive prefix of n <= 1024 values over the block (thread e gives v of
// entry e); returns it and the sum of all.
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* sums, uint32_t* all) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t inc = (uint32_t)wave_scan_add((int)v, lane);
  if (lane == 63) sums[w] = inc;
  __syncthreads();
  uint32_t base = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kRouteThreads / 64; ++i) {
    base += i < w ? sums[i] : 0;
    total += sums[i];
  }
  *all = total;
  return base + inc - v;
}

// What follows the choices of a block's 64 tokens: with ONE (at most 64 tokens
// in all) the block finishes the sort, else it leaves its masks and counts.
template <bool ONE>
__device__ __forceinline__ void after_choice(const RouteArgs& a, const uint64_t* mask, uint32_t* before,
                                             uint32_t* sums, int64_t block, int tokens) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (ONE) {
    const uint32_t c = tid < a.experts ? (uint32_t)__popcll(mask[tid]) : 0;
    uint32_t live;
    const uint32_t b = block_prefix(c, sums, &live);
    if (tid < a.experts) {
      before[tid] = b;
      a.offsets[tid] = (int32_t)b;
    }
    if (tid == 0) a.offsets[a.experts] = (int32_t)live;
    __syncthreads();
    place(a, mask, before, live, 0, tokens);
  } else if (tid < a.experts) {
    a.mask[block * a.experts + tid] = mask[tid];
    a.count[(int64_t)tid * a.stride + block] = (uint8_t)__popcll(mask[tid]);
  }
}

// A block has 64 tokens, a wave takes four of them one after the other.
template <class T, int V, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void k_route_choose(RouteArgs a) {
  __shared__ uint64_t mask[64 * V];
  __shared__ uint32_t before[64 * V];
  __shared__ uint32_t sums[kRouteThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t block = ONE ? 0 : block_index(), t0 = block * kTokensPerBlock;
  if (!ONE && block >= a.blocks) return;
  const int tokens = (int)(a.tokens - t0 < kTokensPerBlock ? a.tokens - t0 : kTokensPerBlock);
  if (tid < 64 * V) mask[tid] = 0;
  __syncthreads();
  for (int tl = w; tl < tokens; tl += kRouteThreads / 64) {
    const int64_t t = t0 + tl;
    const T* src = static_cast<const T*>(a.logits) + t * a.experts;
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = lane + 64 * v < a.experts ? clean_logit(to_f32(src[lane + 64 * v])) : -INFINITY;
    float top;
    int id;
    choose<V>(l, a.experts, a.k, lane, top, id);
    const float base = fmaxf(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(top))), -3.402823466e38f);
    const float ex = expf(top - base);
    float sum = ex;
    if (!a.normalize) {
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += expf(l[v] - base);
    }
    sum = wave_sum(sum);
    if (lane < a.k) {
      a.weights[t * a.k + lane] = sum > 0.f ? ex / sum : 0.f;
      a.chosen[t * a.k + lane] = id;
      if (id >= 0) atomicOr((unsigned long long*)&mask[id], 1ull << tl);
    }
  }
  after_choice<ONE>(a, mask, before, sums, block, tokens);
}

// The block's 64 tokens at once, 16 lanes each: up to 16 V experts and 16
// choices.  16384 tokens of 64 experts, 8 choices: 6.6 us, and 13.5 us by
// k_route_choose: what bounds it is the vector instructions of the rounds.
template <class T, int V, bool ONE>
__global__ __launch_bounds__(kRouteThreads) void k_route_choose_rows(RouteArgs a) {
  __shared__ uint64_t mask[16 * V];
  __shared__ uint32_t before[16 * V];
  __shared__ uint32_t sums[kRouteThreads / 64];
  const int tid = threadIdx.x, li = tid & 15, tl = tid >> 4;
  const int64_t block = ONE ? 0 : block_index(), t0 = block * kTokensPerBlock, t = t0 + tl;
  if (!ONE && block >= a.blocks) return;
  const int tokens = (int)(a.tokens - t0 < kTokensPerBlock ? a.tokens - t0 : kTokensPerBlock);
  if (tid < 16 * V) mask[tid] = 0;
  __syncthreads();
  if (tl < tokens) {   // whole rows of 16 lanes
    const T* src = static_cast<const T*>(a.logits) + t * a.experts;
    float l[V];
#pragma unroll
    for (int v = 0; v < V; ++v) l[v] = li * V + v < a.experts ? clean_logit(to_f32(src[li * V + v])) : -INFINITY;
    float top, top0;
    int id;
    choose_row<V>(l, a.experts, a.k, li, top, id, top0);
    const float base = fmaxf(top0, -3.402823466e38f);
    const float ex = expf(top - base);
    float sum = ex;
    if (!a.normalize) {
      sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) sum += expf(l[v] - base);
    }
    sum = row_sum(sum);
    if (li < a.k) {
      a.weights[t * a.k + li] = sum > 0.f ? ex / sum : 0.f;
      a.chosen[t * a.k + li] = id;
      if (id >= 0) atomicOr((unsigned long long*)&mask[id], 1ull << tl);
    }
  }
  after_choice<ONE>(a, mask, before, sums, block, tokens);
}

// One block per expert: how many of its rows are in earlier blocks, for more blocks than a placing
// block can count by itself.
__global__ __launch_bounds__(kRouteThreads) void k_route_scan(RouteArgs a) {
  __shared__ uint32_t sums[kRouteThreads / 64];
  const uint8_t* c = a.count + (int64_t)blockIdx.x * a.stride;
  uint32_t* ahead = a.ahead + (int64_t)blockIdx.x * a.blocks;
  uint32_t run = 0;
  for (int b0 = 0; b0 < a.blocks; b0 += kRouteThreads) {
    const int b = b0 + threadIdx.x;
    const uint32_t v = b < a.blocks ? c[b] : 0;
    uint32_t all;
    const uint32_t at = block_prefix(v, sums, &all);
    if (b < a.blocks) ahead[b] = run + at;
    run += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = run;
}

// Sum of the first n of 16 byte counts, n any number.
__device__ __forceinline__ uint32_t sum_counts(u32x4 v, int n) {
  uint32_t s = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    const uint32_t keep = left >= 4 ? 0xffffffffu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    s = __builtin_amdgcn_sad_u8(v[i] & keep, 0u, s);
  }
  return s;
}

// Places of a block's choices.  Where the counts are few (counted_by_blocks) every
// block adds up all of them (bytes: 16 KiB of L2 reads a block for 16384 tokens
// of 64 experts), which saves the scan's launch: 4.8 us against 3.9 + 3.9.
template <bool SCANNED>
__global__ __launch_bounds__(kRouteThreads) void k_route_place(RouteArgs a) {
  __shared__ uint64_t mask[kMaxExperts];
  __shared__ uint32_t before[kMaxExperts];
  __shared__ uint32_t total[SCANNED ? 1 : kMaxExperts];
  __shared__ uint32_t sums[kRouteThreads / 64];
  const int tid = threadIdx.x;
  const int64_t block = block_index(), t0 = block * kTokensPerBlock;
  if (block >= a.blocks) return;
  const int tokens = (int)(a.tokens - t0 < kTokensPerBlock ? a.tokens - t0 : kTokensPerBlock);
  if (!SCANNED) {   // 16 threads add up an expert's counts
    const int li = tid & 15, me = (int)block;
    for (int e0 = 0; e0 < a.experts; e0 += kRouteThreads / 16) {
      const int e = e0 + tid / 16;
      uint32_t earlier = 0, all = 0;
      if (e < a.experts) {
        const u32x4* c = reinterpret_cast<const u32x4*>(a.count + (int64_t)e * a.stride);
        for (int b = 16 * li; b < a.blocks; b += 256) {
          const u32x4 v = c[b / 16];
          earlier += sum_counts(v, me - b);
          all += sum_counts(v, a.blocks - b);
        }
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) {
        earlier += __shfl_xor(earlier, o, 64);
        all += __shfl_xor(all, o, 64);
      }
      if (li == 0 && e < a.experts) {
        before[e] = earlier;
        total[e] = all;
      }
    }
    __syncthreads();
  }
  const uint32_t c = tid < a.experts ? (SCANNED ? a.total[tid] : total[tid]) : 0;
  uint32_t live;
  const uint32_t b = block_prefix(c, sums, &live);
  if (tid < a.experts) {
    mask[tid] = a.mask[block * a.experts + tid];
    before[tid] = b + (SCANNED ? a.ahead[(int64_t)tid * a.blocks + block] : before[tid]);
    if (block == 0) a.offsets[tid] = (int32_t)b;
  }
  if (block == 0 && tid == 0) a.offsets[a.experts] = (int32_t)live;
  __syncthreads();
  place(a, mask, before, live, t0, tokens);
}

// d_e = sum_{j: id_j = e} w_j dw_j - p_e sum_j w_j dw_j, where p is the
// softmax the weights came from: over the chosen (p_e = w_j, nothing but the
// chosen gets a gradient) or over all experts.  A wave per token.
template <class T, int V>
__global__ __launch_bounds__(256) void k_route_backward(const float* __restrict__ dw, const T* __restrict__ logits,
                                                        const float* __restrict__ weights,
                                                        const int32_t* __restrict__ chosen, T* __restrict__ out,
                                                        int64_t tokens, int experts, int k, int normalize) {
  const int lane = threadIdx.x & 63;
  const int64_t t = block_index() * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  int id = -1;
  float wd = 0.f, w = 0.f;
  if (lane < k) {
    id = chosen[t * k + lane];
    w = weights[t * k + lane];
    wd = id >= 0 ? w * dw[t * k + lane] : 0.f;
    w = id >= 0 ? w : 0.f;
  }
  const float dot = wave_sum(wd);
  const float add = normalize ? wd - w * dot : wd;
  float d[V];
  if (normalize) {
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = 0.f;
  } else {
    const T* src = logits + t * experts;
    float l[V];
    uint32_t best = kGone;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = lane + 64 * v < experts ? clean_logit(to_f32(src[lane + 64 * v])) : -INFINITY;
      const uint32_t c = order_code(l[v]);
      best = c > best ? c : best;
    }
    const float base = fmaxf(from_code(wave_max(best)), -3.402823466e38f);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = expf(l[v] - base);
      sum += l[v];
    }
    sum = wave_sum(sum);
    const float f = sum > 0.f ? -dot / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = l[v] * f;
  }
  for (int j = 0; j < k; ++j) {
    const int e = __builtin_amdgcn_readlane(id, j);
    const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(add), j));
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (e == lane + 64 * v) d[v] += x;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (lane + 64 * v < experts) store1(out + t * experts + lane + 64 * v, d[v]);
}

// The same for up to 16 V experts and 16 choices: 16 lanes a token, lane l with
// experts l V on; the choices' parts reach their experts through LDS.  16384
// tokens of 64 experts, 8 choices: 4.4 us, and 6.5 us with a token a wave.
template <class T, int V>
__global__ __launch_bounds__(256) void k_route_backward_rows(const float* __restrict__ dw,
                                                             const T* __restrict__ logits,
                                                             const float* __restrict__ weights,
                                                             const int32_t* __restrict__ chosen, T* __restrict__ out,
                                                             int64_t tokens, int experts, int k, int normalize) {
  __shared__ float part[16][16 * V + 1];
  const int li = threadIdx.x & 15, row = threadIdx.x >> 4;
  const int64_t t = block_index() * 16 + row;
#pragma unroll
  for (int v = 0; v < V; ++v) part[row][li * V + v] = 0.f;
  if (t >= tokens) return;   // a row's lanes are of one wave and share nothing with others
  int id = -1;
  float wd = 0.f, w = 0.f;
  if (li < k) {
    id = chosen[t * k + li];
    w = weights[t * k + li];
    wd = id >= 0 ? w * dw[t * k + li] : 0.f;
    w = id >= 0 ? w : 0.f;
  }
  const float dot = row_sum(wd);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  if (id >= 0 && id < experts) part[row][id] = normalize ? wd - w * dot : wd;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float d[V];
#pragma unroll
  for (int v = 0; v < V; ++v) d[v] = part[row][li * V + v];
  if (!normalize) {
    const T* src = logits + t * experts;
    float l[V];
    uint32_t best = kGone;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = li * V + v < experts ? clean_logit(to_f32(src[li * V + v])) : -INFINITY;
      const uint32_t c = order_code(l[v]);
      best = c > best ? c : best;
    }
    const float base = fmaxf(from_code(row_max(best)), -3.402823466e38f);
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      l[v] = expf(l[v] - base);
      sum += l[v];
    }
    sum = row_sum(sum);
    const float f = sum > 0.f ? -dot / sum : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] += l[v] * f;
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (li * V + v < experts) store1(out + t * experts + li * V + v, d[v]);
}

// ------------------------------------------------------------------ combine

// Eight elements as they lie in memory, and their values.
__device__ __forceinline__ void raw8(const bf16_t* p, u32x4 (&r)[1]) { r[0] = *reinterpret_cast<const u32x4_any*>(p); }
__device__ __forceinline__ void raw8(const float* p, u32x4 (&r)[2]) {
  r[0] = *reinterpret_cast<const u32x4_any*>(p);
  r[1] = *reinterpret_cast<const u32x4_any*>(p + 4);
}
__device__ __forceinline__ void values8(const u32x4 (&r)[1], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r[0][i] << 16);
    v[2 * i + 1] = __uint_as_float(r[0][i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void values8(const u32x4 (&r)[2], float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i / 4][i % 4]);
}

// out[t] = sum_j w_j y[slot_j]: a thread holds eight columns of one token.  The
// rows of eight choices (four in fp32) are on their way at once.  Bound by the
// rows' way from memory: 8192 tokens of 2048 bf16 columns and 8 choices take 76
// us (302 MB, 4.0 TB/s of the copy probe's 6.2; 80 us one row after the other, 77 with a wave a token
// and scalar loads of slots and weights).
template <class T>
__global__ __launch_bounds__(256) void k_combine(const T* __restrict__ y, const int32_t* __restrict__ slots,
                                                 const float* __restrict__ weights, T* __restrict__ out,
                                                 uint32_t items, FastDiv groups, int k, int64_t n, int64_t cols) {
  constexpr int R = sizeof(T) == 2 ? 1 : 2, U = 8 / R;
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;
  const uint32_t t = div_by(idx, groups), g = idx - t * groups.d;
  const int cnt = (int)(cols - 8 * (int64_t)g < 8 ? cols - 8 * (int64_t)g : 8);
  const T* yc = y + 8 * (int64_t)g;
  const int32_t* st = slots + (int64_t)t * k;
  const float* wt = weights + (int64_t)t * k;
  float acc[8] = {};
  int j0 = 0;
  if (cnt == 8) {
    for (; j0 + U <= k; j0 += U) {
      int32_t s[U];
      float w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = st[j0 + u];
        w[u] = wt[j0 + u];
      }
      u32x4 r[U][R];
#pragma unroll
      for (int u = 0; u < U; ++u) {   // a choice without a row reads row 0 and is left out
        s[u] = s[u] >= 0 && s[u] < n ? s[u] : -1;
        raw8(yc + (s[u] < 0 ? 0 : s[u]) * cols, r[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[8];
        values8(r[u], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = s[u] < 0 ? acc[i] : acc[i] + w[u] * v[i];
      }
    }
  }
  for (; j0 < k; ++j0) {
    const int32_t s = st[j0];
    const float w = wt[j0];
    if (s >= 0 && s < n) {
      float v[8];
      load8(yc + s * cols, cnt, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] += w * v[i];
    }
  }
  store8(out + (int64_t)t * cols + 8 * (int64_t)g, cnt, acc);
}

// dy[slot_j] = w_j dout[t], dw_j = <y[slot_j], dout[t]>: a wave per choice;
// the waves of one token sit side by side, so dout comes from cache but once.
// The wave of place p also clears row p of dy where no expert has it; such a
// row is written by no other wave, whatever slot names it.  The sizes above: 108
// us, 570 MB, 5.3 TB/s.
template <class T>
__global__ __launch_bounds__(256) void k_combine_backward(
    const T* __restrict__ dout, const T* __restrict__ y, const int32_t* __restrict__ slots,
    const float* __restrict__ weights, const int32_t* __restrict__ offsets, T* __restrict__ dy,
    float* __restrict__ dw, int experts, FastDiv k, int64_t n, int64_t cols) {
  const int lane = threadIdx.x & 63;
  const uint32_t p = (uint32_t)block_index() * 4 + (threadIdx.x >> 6);
  if (p >= n) return;
  const uint32_t t = div_by(p, k);
  const int32_t s = slots[p], live = offsets[experts];
  float dot = 0.f;
  if (s >= 0 && s < n) {
    const float w = weights[p];
    for (int64_t c = 8 * lane; c < cols; c += 512) {
      const int cnt = (int)(cols - c < 8 ? cols - c : 8);
      float a[8], b[8];
      load8(y + s * cols + c, cnt, a);
      load8(dout + t * cols + c, cnt, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dot += a[i] * b[i];
        b[i] *= w;
      }
      if (s < live) store8(dy + s * cols + c, cnt, b);
    }
  }
  dot = wave_sum(dot);
  if (lane == 0) dw[p] = dot;
  if ((int64_t)p >= live) {
    const float z[8] = {};
    for (int64_t c = 8 * lane; c < cols; c += 512) store8(dy + p * cols + c, (int)(cols - c < 8 ? cols - c : 8), z);
  }
}

// -------------------------------------------------------------- checkpoints

// Scale code (exponent + 127) of a block from the bits of its largest
// magnitude: the smallest power of two for which the block's values round to
// at most 127 in int8 (a value that rounds to 128 is held as 127), or do not
// exceed 448 in e4m3 (448 = 1.75 * 2^8).  The exponent is at least -126.  255
// marks a block that holds an infinity or NaN: it restores to NaN as a whole.
template <int KIND>
__device__ __forceinline__ int scale_code(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255;
  const int e = (int)(amax >> 23);
  int code = KIND == MUON_INT8 ? e - 6 : ((amax & 0x7fffffu) <= 0x600000u ? e - 8 : e - 7);
  return code < 1 ? 1 : code;
}

__device__ __forceinline__ uint32_t amax8(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    m = a > m ? a : m;
  }
  return m;
}

__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, false);   // lanes 1 0 3 2
  m = o > m ? o : m;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, false);            // lanes 2 3 0 1
  return o > m ? o : m;
}

// Eight values in 8 bits: round to nearest even.
template <int KIND>
__device__ __forceinline__ u32x2 encode8(const float (&v)[8], int code) {
  const float inv = code == 255 ? 0.f : pow2f(127 - code);
  u32x2 q = {0u, 0u};
  if (code == 255) return q;
  if (KIND == MUON_INT8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = (int)fminf(fmaxf(rintf(v[i] * inv), -127.f), 127.f);
      q[i / 4] |= (uint32_t)(r & 255) << (8 * (i % 4));
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      int t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h] * inv, v[4 * h + 1] * inv, 0, false);
      t = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * h + 2] * inv, v[4 * h + 3] * inv, t, true);
      q[h] = (uint32_t)t;
    }
  }
  return q;
}

template <int KIND>
__device__ __forceinline__ void decode8(u32x2 q, float (&v)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (KIND == MUON_INT8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * h + i] = (float)(int8_t)(q[h] >> (8 * i));
    } else {
      v[4 * h] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 0);
      v[4 * h + 1] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 1);
      v[4 * h + 2] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 2);
      v[4 * h + 3] = __builtin_amdgcn_cvt_f32_fp8((int)q[h], 3);
    }
  }
}

__device__ __forceinline__ float scale_of(uint8_t code) {
  return code == 255 ? __uint_as_float(0x7fc00000u) : code == 0 ? 0.f : pow2f((int)code - 127);
}

__device__ __forceinline__ void store_q(uint8_t* p, int cnt, u32x2 q) {
  if (cnt >= 8) {
    *reinterpret_cast<u32x2_any*>(p) = q;
  } else {
    for (int i = 0; i < cnt; ++i) p[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
  }
}
__device__ __forceinline__ u32x2 load_q(const uint8_t* p, int cnt) {
  if (cnt >= 8) return *reinterpret_cast<const u32x2_any*>(p);
  u32x2 q = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) q[i / 4] |= (uint32_t)p[i] << (8 * (i % 4));
  return q;
}

// Eight kept values of a row from column c on; a group that starts off a
// multiple of eight can reach into the next block.
template <int KIND>
__device__ __forceinline__ void load_kept(const uint8_t* q, const uint8_t* scale, int64_t c, int cnt, float (&v)[8]) {
  decode8<KIND>(load_q(q + c, cnt), v);
  const int64_t b = c / kBlock;
  const int in = (int)((b + 1) * kBlock - c);   // of the first block
  const float s0 = scale_of(scale[b]);
  const float s1 = in < cnt ? scale_of(scale[b + 1]) : s0;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= i < in ? s0 : s1;
}

// A thread encodes eight columns; four threads hold a block.  4099 x 2056 bf16:
// 7.4 us for 25 MB, most of it the launch and the way to memory; restoring 5.9.
template <class T, int KIND>
__global__ __launch_bounds__(256) void k_checkpoint(const T* __restrict__ x, uint8_t* __restrict__ q,
                                                    uint8_t* __restrict__ scale, uint32_t items, FastDiv groups,
                                                    int64_t cols, int64_t blocks) {
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;   // items is a multiple of four: whole quads leave
  const uint32_t r = div_by(idx, groups), g = idx - r * groups.d;
  const int64_t c = 8 * (int64_t)g;
  const int cnt = (int)(cols - c < 8 ? cols - c : 8);
  float v[8];
  load8(x + r * cols + c, cnt, v);
  const int code = scale_code<KIND>(quad_max(amax8(v)));
  store_q(q + r * cols + c, cnt, encode8<KIND>(v, code));
  if ((g & 3) == 0) scale[r * blocks + g / 4] = (uint8_t)code;
}

template <class T, int KIND>
__global__ __launch_bounds__(256) void k_restore(const uint8_t* __restrict__ q, const uint8_t* __restrict__ scale,
                                                 T* __restrict__ x, uint32_t items, FastDiv groups, int64_t cols,
                                                 int64_t blocks) {
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;
  const uint32_t r = div_by(idx, groups), g = idx - r * groups.d;
  const int64_t c = 8 * (int64_t)g;
  const int cnt = (int)(cols - c < 8 ? cols - c : 8);
  float v[8];
  load_kept<KIND>(q + r * cols, scale + r * blocks, c, cnt, v);
  store8(x + r * cols + c, cnt, v);
}

// ---------------------------------------------------------- gated activation

// 1 / (1 + e^-g) as (1 or t) / (1 + t), t = e^-|g|: nothing overflows, and a
// closed gate keeps its value down to the subnormals.  For bf16 outputs the
// hardware's exponential and reciprocal (about 1e-7 relative each) are far
// inside the rounding of the result; they flush subnormal results, so t is
// formed 2^8 too large and scaled down after.
template <class T>
__device__ __forceinline__ float sigmoid(float g);
template <>
__device__ __forceinline__ float sigmoid<float>(float g) {
  const float t = expf(-fabsf(g));
  return (g < 0.f ? t : 1.f) / (1.f + t);
}
template <>
__device__ __forceinline__ float sigmoid<bf16_t>(float g) {
  const float t = __builtin_amdgcn_exp2f(fmaf(-1.44269504f, fabsf(g), 8.f)) * 0.00390625f;
  return (g < 0.f ? t : 1.f) * __builtin_amdgcn_rcpf(1.f + t);
}

// h = g sigma(g) u of [g | u], and with KIND its 8-bit checkpoint in the same
// pass (f a multiple of 32, so that no block holds both g and u).  Bound by
// memory: 32768 x 1408 bf16 with its int8 checkpoint, 372 MB, 69 us, 5.4 TB/s.
template <class T, int KIND>
__global__ __launch_bounds__(256) void k_gated(const T* __restrict__ gu, T* __restrict__ h, uint8_t* __restrict__ q,
                                               uint8_t* __restrict__ scale, uint32_t items, FastDiv groups,
                                               int64_t f) {
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;
  const uint32_t r = div_by(idx, groups), grp = idx - r * groups.d;
  const int64_t c = 8 * (int64_t)grp, at = 2 * r * f + c;
  const int cnt = (int)(f - c < 8 ? f - c : 8);
  float g[8], u[8], o[8];
  load8(gu + at, cnt, g);
  load8(gu + at + f, cnt, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = g[i] * sigmoid<T>(g[i]) * u[i];
  store8(h + r * f + c, cnt, o);
  if (KIND >= 0) {
    const int cg = scale_code<KIND>(quad_max(amax8(g))), cu = scale_code<KIND>(quad_max(amax8(u)));
    store_q(q + at, 8, encode8<KIND>(g, cg));
    store_q(q + at + f, 8, encode8<KIND>(u, cu));
    if ((grp & 3) == 0) {
      uint8_t* s = scale + (2 * r * f + c) / kBlock;
      s[0] = (uint8_t)cg;
      s[f / kBlock] = (uint8_t)cu;
    }
  }
}

// dg = dh u sigma(g) (1 + g (1 - sigma(g))), du = dh g sigma(g), and h again
// (what the down projection's weight gradient reads), from [g | u] or from
// its checkpoint.  The sizes above, from the checkpoint: 464 MB, 76 us, 6.1 TB/s.
template <class T, int KIND>
__global__ __launch_bounds__(256) void k_gated_backward(const T* __restrict__ dh, const T* __restrict__ gu,
                                                        const uint8_t* __restrict__ q,
                                                        const uint8_t* __restrict__ scale, T* __restrict__ dgu,
                                                        T* __restrict__ h, uint32_t items, FastDiv groups, int64_t f,
                                                        int64_t blocks) {
  const uint32_t idx = blockIdx.x * 256 + threadIdx.x;
  if (idx >= items) return;
  const uint32_t r = div_by(idx, groups), grp = idx - r * groups.d;
  const int64_t c = 8 * (int64_t)grp, at = 2 * r * f;
  const int cnt = (int)(f - c < 8 ? f - c : 8);
  float g[8], u[8], d[8];
  if constexpr (KIND >= 0) {
    load_kept<KIND>(q + at, scale + r * blocks, c, cnt, g);
    load_kept<KIND>(q + at, scale + r * blocks, f + c, cnt, u);
  } else {
    load8(gu + at + c, cnt, g);
    load8(gu + at + f + c, cnt, u);
  }
  load8(dh + r * f + c, cnt, d);
  float dg[8], du[8], o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid<T>(g[i]), gs = g[i] * s;
    o[i] = gs * u[i];
    du[i] = d[i] * gs;
    dg[i] = d[i] * u[i] * s * (1.f + g[i] * (1.f - s));
  }
  store8(h + r * f + c, cnt, o);
  store8(dgu + at + c, cnt, dg);
  store8(dgu + at + f + c, cnt, du);
}

// --------------------------------------------------------------------- host

// Work items of eight columns each over `rows` >= 1 rows of `groups` groups.
int items_of(int64_t rows, int64_t groups, uint32_t* items, FastDiv* div) {
  if (groups > kMaxCount / rows) return fail(MUON_EUNSUPPORTED, "more than 2^31 groups of 8 columns");
  *items = (uint32_t)(rows * groups);
  *div = fast_div((uint32_t)groups);
  return MUON_OK;
}

dim3 grid_of(uint32_t items) { return dim3((items + 255) / 256); }

int route_blocks(int64_t tokens) { return (int)ceil_div(tokens, kTokensPerBlock); }

// Whether the placing blocks add up the counts by themselves; the others take the
// scan.  Each reads experts x blocks bytes, 64 experts a round.  A whole route
// call, us, without / with the scan, by tokens:
//            1024         16384        32768         65536
//     8:   7.8 / 9.7    8.3 / 10.1   11.3 / 12.8    20.1 / 19.1
//    64:   9.5 / 11.1  10.7 / 12.2   16.3 / 16.2    31.3 / 26.2
//   128:  13.8 / 14.9  15.5 / 16.5   26.7 / 24.7    53.5 / 40.9
//   256:  21.2 / 21.9  24.5 / 24.5   45.0 / 39.1   115 / 85
//  1024:  52.5 / 45.1  67.9 / 61.1   106 / 78      277 / 155
bool counted_by_blocks(int64_t blocks, int experts) {
  return experts <= 128 && blocks <= 512 && experts * blocks <= 32768;
}
int route_stride(int64_t tokens) { return (int)(ceil_div(route_blocks(tokens), 16) * 16); }

uint64_t route_bytes(int64_t tokens, int experts) {
  if (tokens <= kTokensPerBlock) return 0;
  const uint64_t blocks = (uint64_t)route_blocks(tokens);
  const uint64_t fixed = (blocks * 8 + (uint64_t)route_stride(tokens)) * experts;
  return (fixed + 15) / 16 * 16 + (counted_by_blocks((int64_t)blocks, experts) ? 0 : (blocks + 1) * experts * 4);
}

int check_route(int dtype, int64_t tokens, int experts, int k) {
  if (!good_dtype(dtype)) return fail(MUON_EUNSUPPORTED, "unsupported dtype");
  if (tokens < 0) return fail(MUON_EINVAL, "negative token count");
  if (experts < 1 || k < 1 || k > experts) return fail(MUON_EINVAL, "k must be in [1, experts]");
  if (experts > kMaxExperts || k > kMaxTopK)
    return fail(MUON_EUNSUPPORTED, "more than 1024 experts or 64 choices");
  if (tokens > kMaxCount / k) return fail(MUON_EUNSUPPORTED, "tokens * k must stay below 2^31");
  return MUON_OK;
}

template <class T, int V>
void launch_choose(const RouteArgs& a, hipStream_t s) {
  if (a.tokens <= kTokensPerBlock)
    hipLaunchKernelGGL((k_route_choose<T, V, true>), dim3(1), dim3(kRouteThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_route_choose<T, V, false>), grid_of_blocks(a.blocks, kRouteThreads), dim3(kRouteThreads), 0, s, a);
}
template <class T, int V>
void launch_choose_rows(const RouteArgs& a, hipStream_t s) {
  if (a.tokens <= kTokensPerBlock)
    hipLaunchKernelGGL((k_route_choose_rows<T, V, true>), dim3(1), dim3(kRouteThreads), 0, s, a);
  else
    hipLaunchKernelGGL((k_route_choose_rows<T, V, false>), grid_of_blocks(a.blocks, kRouteThreads), dim3(kRouteThreads), 0, s, a);
}

// Whether 16 lanes take a token, and the logits each of them has to hold then.
bool by_rows(int experts, int k) { return experts <= 256 && k <= 16; }
template <class F>
void by_row_width(int experts, F f) {
  if (experts <= 16) f(std::integral_constant<int, 1>());
  else if (experts <= 64) f(std::integral_constant<int, 4>());
  else if (experts <= 128) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

// f(std::integral_constant<int, V>) for the logits a lane has to hold
template <class F>
void by_width(int experts, F f) {
  if (experts <= 64) f(std::integral_constant<int, 1>());
  else if (experts <= 128) f(std::integral_constant<int, 2>());
  else if (experts <= 256) f(std::integral_constant<int, 4>());
  else if (experts <= 512) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 16>());
}

int check_rows(int dtype, int64_t rows, int64_t cols) {
  if (!good_dtype(dtype)) return fail(MUON_EUNSUPPORTED, "unsupported dtype");
  if (rows < 0 || cols < 1) return fail(MUON_EINVAL, "rows must be >= 0 and columns >= 1");
  if (rows > 0 && cols > 8 * kMaxCount) return fail(MUON_EUNSUPPORTED, "2^34 columns or more");
  return MUON_OK;
}

int check_kind(int kind) {
  if (kind != MUON_INT8 && kind != MUON_E4M3) return fail(MUON_EUNSUPPORTED, "kind must be MUON_INT8 or MUON_E4M3");
  return MUON_OK;
}

template <class T>
void launch_checkpoint(const void* x, int64_t cols, int kind, void* q, uint8_t* scale, uint32_t items, FastDiv div,
                       hipStream_t s) {
  const int64_t blocks = ceil_div(cols, kBlock);
  if (kind == MUON_INT8)
    hipLaunchKernelGGL((k_checkpoint<T, MUON_INT8>), grid_of(items), dim3(256), 0, s, (const T*)x, (uint8_t*)q, scale,
                       items, div, cols, blocks);
  else
    hipLaunchKernelGGL((k_checkpoint<T, MUON_E4M3>), grid_of(items), dim3(256), 0, s, (const T*)x, (uint8_t*)q, scale,
                       items, div, cols, blocks);
}

template <class T>
void launch_restore(const void* q, const uint8_t* scale, int64_t cols, int kind, void* x, uint32_t items,
                    FastDiv div, hipStream_t s) {
  const int64_t blocks = ceil_div(cols, kBlock);
  if (kind == MUON_INT8)
    hipLaunchKernelGGL((k_restore<T, MUON_INT8>), grid_of(items), dim3(256), 0, s, (const uint8_t*)q, scale, (T*)x,
                       items, div, cols, blocks);
  else
    hipLaunchKernelGGL((k_restore<T, MUON_E4M3>), grid_of(items), dim3(256), 0, s, (const uint8_t*)q, scale, (T*)x,
                       items, div, cols, blocks);
}

template <class T, int KIND>
void launch_gated(const void* gu, int64_t f, void* h, void* q, uint8_t* scale, uint32_t items, FastDiv div,
                  hipStream_t s) {
  hipLaunchKernelGGL((k_gated<T, KIND>), grid_of(items), dim3(256), 0, s, (const T*)gu, (T*)h, (uint8_t*)q, scale,
                     items, div, f);
}

template <class T>
void launch_gated_backward(const void* dh, const void* gu, const void* q, const uint8_t* scale, int kind, int64_t f,
                           void* dgu, void* h, uint32_t items, FastDiv div, hipStream_t s) {
  const int64_t blocks = ceil_div(2 * f, kBlock);
#define MUON_GATED_BACKWARD(K)                                                                                   \
  hipLaunchKernelGGL((k_gated_backward<T, K>), grid_of(items), dim3(256), 0, s, (const T*)dh, (const T*)gu,      \
                     (const uint8_t*)q, scale, (T*)dgu, (T*)h, items, div, f, blocks)
  if (!q) MUON_GATED_BACKWARD(-1);
  else if (kind == MUON_INT8) MUON_GATED_BACKWARD(MUON_INT8);
  else MUON_GATED_BACKWARD(MUON_E4M3);
#undef MUON_GATED_BACKWARD
}

}  // namespace

// Rows of a checkpoint as dense values (used by the products' weight gradient).
int restore_rows(const void* q, const uint8_t* scale, int kind, int64_t rows, int64_t cols, int dtype, void* x,
                 hipStream_t s) {
  if (rows == 0) return MUON_OK;
  uint32_t items;
  FastDiv div;
  int rc;
  if ((rc = items_of(rows, ceil_div(cols, 8), &items, &div))) return rc;
  if (dtype == MUON_BF16) launch_restore<bf16_t>(q, scale, cols, kind, x, items, div, s);
  else launch_restore<float>(q, scale, cols, kind, x, items, div, s);
  return launch_status("restore launch");
}

}  // namespace ex
}  // namespace muon

using namespace muon::ex;

extern "C" {

int muon_route_workspace(int64_t tokens, int experts, uint64_t* bytes) {
  muon::report_error(MUON_OK, "");
  if (!bytes) return fail(MUON_EINVAL, "NULL bytes");
  const int rc = check_route(MUON_F32, tokens, experts, 1);
  if (rc) return rc;
  *bytes = route_bytes(tokens, experts);
  return MUON_OK;
}

int muon_route(const void* logits, int dtype, int64_t tokens, int experts, int k, int normalize, float* weights,
               int32_t* chosen, int32_t* slots, int32_t* rows, int32_t* offsets, void* workspace,
               uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_route(dtype, tokens, experts, k))) return rc;
  if (!offsets || (tokens > 0 && (!logits || !weights || !chosen || !slots || !rows)))
    return fail(MUON_EINVAL, "NULL pointer");
  const uint64_t need = route_bytes(tokens, experts);
  if (need && (!workspace || workspace_bytes < need))
    return fail(MUON_EINVAL, "workspace of " + std::to_string(need) + " bytes needed");
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 15)) return fail(MUON_EINVAL, "workspace must be 16-byte aligned");
  if ((rc = check_device())) return rc;
  RouteArgs a;
  a.logits = logits;
  a.weights = weights;
  a.chosen = chosen;
  a.slots = slots;
  a.rows = rows;
  a.offsets = offsets;
  a.tokens = tokens;
  a.experts = experts;
  a.k = k;
  a.normalize = normalize ? 1 : 0;
  a.blocks = route_blocks(tokens);
  a.count = nullptr;
  a.mask = nullptr;
  a.ahead = a.total = nullptr;
  a.stride = route_stride(tokens);
  if (need) {
    uint8_t* at = static_cast<uint8_t*>(workspace);
    a.count = at;
    at += (int64_t)a.stride * experts;
    a.mask = reinterpret_cast<uint64_t*>(at);
    at += (int64_t)a.blocks * experts * 8;
    a.ahead = reinterpret_cast<uint32_t*>(at);
    a.total = a.ahead + (int64_t)a.blocks * experts;
  }
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (by_rows(experts, k)) {
    by_row_width(experts, [&](auto v) {
      if (dtype == MUON_BF16) launch_choose_rows<bf16_t, decltype(v)::value>(a, s);
      else launch_choose_rows<float, decltype(v)::value>(a, s);
    });
  } else {
    by_width(experts, [&](auto v) {
      if (dtype == MUON_BF16) launch_choose<bf16_t, decltype(v)::value>(a, s);
      else launch_choose<float, decltype(v)::value>(a, s);
    });
  }
  if ((rc = launch_status("route launch"))) return rc;
  if (!need) return MUON_OK;
  if (!counted_by_blocks(a.blocks, experts)) {
    hipLaunchKernelGGL(k_route_scan, dim3(experts), dim3(kRouteThreads), 0, s, a);
    if ((rc = launch_status("route scan launch"))) return rc;
    hipLaunchKernelGGL((k_route_place<true>), grid_of_blocks(a.blocks, kRouteThreads), dim3(kRouteThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_route_place<false>), grid_of_blocks(a.blocks, kRouteThreads), dim3(kRouteThreads), 0, s, a);
  }
  return launch_status("route place launch");
}

int muon_route_backward(const float* dweights, const void* logits, const float* weights, const int32_t* chosen,
                        int dtype, int64_t tokens, int experts, int k, int normalize, void* dlogits, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_route(dtype, tokens, experts, k))) return rc;
  if (tokens == 0) return MUON_OK;
  if (!dweights || !logits || !weights || !chosen || !dlogits) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (by_rows(experts, k)) {
    const dim3 grid = grid_of_blocks(ceil_div(tokens, 16), 256);
    by_row_width(experts, [&](auto v) {
      constexpr int V = decltype(v)::value;
      if (dtype == MUON_BF16)
        hipLaunchKernelGGL((k_route_backward_rows<bf16_t, V>), grid, dim3(256), 0, s, dweights, (const bf16_t*)logits,
                           weights, chosen, (bf16_t*)dlogits, tokens, experts, k, normalize);
      else
        hipLaunchKernelGGL((k_route_backward_rows<float, V>), grid, dim3(256), 0, s, dweights, (const float*)logits,
                           weights, chosen, (float*)dlogits, tokens, experts, k, normalize);
    });
    return launch_status("route backward launch");
  }
  const dim3 grid = grid_of_blocks(ceil_div(tokens, 4), 256);
  by_width(experts, [&](auto v) {
    constexpr int V = decltype(v)::value;
    if (dtype == MUON_BF16)
      hipLaunchKernelGGL((k_route_backward<bf16_t, V>), grid, dim3(256), 0, s, dweights, (const bf16_t*)logits,
                         weights, chosen, (bf16_t*)dlogits, tokens, experts, k, normalize);
    else
      hipLaunchKernelGGL((k_route_backward<float, V>), grid, dim3(256), 0, s, dweights, (const float*)logits, weights,
                         chosen, (float*)dlogits, tokens, experts, k, normalize);
  });
  return launch_status("route backward launch");
}

int muon_combine(const void* y, const int32_t* slots, const float* weights, int dtype, int64_t tokens, int k,
                 int64_t cols, void* out, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_rows(dtype, tokens, cols))) return rc;
  if (k < 1) return fail(MUON_EINVAL, "k must be positive");
  if (tokens > kMaxCount / k) return fail(MUON_EUNSUPPORTED, "tokens * k must stay below 2^31");
  if (tokens == 0) return MUON_OK;
  uint32_t items;
  FastDiv div;
  if ((rc = items_of(tokens, ceil_div(cols, 8), &items, &div))) return rc;
  if (!y || !slots || !weights || !out) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MUON_BF16)
    hipLaunchKernelGGL((k_combine<bf16_t>), grid_of(items), dim3(256), 0, s, (const bf16_t*)y, slots, weights,
                       (bf16_t*)out, items, div, k, tokens * k, cols);
  else
    hipLaunchKernelGGL((k_combine<float>), grid_of(items), dim3(256), 0, s, (const float*)y, slots, weights,
                       (float*)out, items, div, k, tokens * k, cols);
  return launch_status("combine launch");
}

int muon_combine_backward(const void* dout, const void* y, const int32_t* slots, const float* weights,
                          const int32_t* offsets, int dtype, int64_t tokens, int k, int experts, int64_t cols,
                          void* dy, float* dweights, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_rows(dtype, tokens, cols))) return rc;
  if (k < 1 || experts < 1) return fail(MUON_EINVAL, "k and experts must be positive");
  if (tokens > kMaxCount / k) return fail(MUON_EUNSUPPORTED, "tokens * k must stay below 2^31");
  if (tokens == 0) return MUON_OK;
  if (!dout || !y || !slots || !weights || !offsets || !dy || !dweights) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t n = tokens * k;
  const dim3 grid = grid_of_blocks(ceil_div(n, 4), 256);
  const FastDiv div = fast_div((uint32_t)k);
  if (dtype == MUON_BF16)
    hipLaunchKernelGGL((k_combine_backward<bf16_t>), grid, dim3(256), 0, s, (const bf16_t*)dout, (const bf16_t*)y,
                       slots, weights, offsets, (bf16_t*)dy, dweights, experts, div, n, cols);
  else
    hipLaunchKernelGGL((k_combine_backward<float>), grid, dim3(256), 0, s, (const float*)dout, (const float*)y, slots,
                       weights, offsets, (float*)dy, dweights, experts, div, n, cols);
  return launch_status("combine backward launch");
}

int muon_checkpoint(const void* x, int dtype, int64_t rows, int64_t cols, int kind, void* q, uint8_t* scale,
                    void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_rows(dtype, rows, cols)) || (rc = check_kind(kind))) return rc;
  if (rows == 0) return MUON_OK;
  uint32_t items;
  FastDiv div;
  if ((rc = items_of(rows, 4 * ceil_div(cols, kBlock), &items, &div))) return rc;
  if (!x || !q || !scale) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MUON_BF16) launch_checkpoint<bf16_t>(x, cols, kind, q, scale, items, div, s);
  else launch_checkpoint<float>(x, cols, kind, q, scale, items, div, s);
  return launch_status("checkpoint launch");
}

int muon_restore(const void* q, const uint8_t* scale, int kind, int64_t rows, int64_t cols, int dtype, void* x,
                 void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_rows(dtype, rows, cols)) || (rc = check_kind(kind))) return rc;
  if (rows == 0) return MUON_OK;
  if (!x || !q || !scale) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  return restore_rows(q, scale, kind, rows, cols, dtype, x, static_cast<hipStream_t>(stream));
}

int muon_gated(const void* gu, int dtype, int64_t rows, int64_t cols, int kind, void* h, void* q, uint8_t* scale,
               void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  const bool keep = q || scale;
  if ((rc = check_rows(dtype, rows, cols)) || (keep && (rc = check_kind(kind)))) return rc;
  if (rows == 0) return MUON_OK;
  // blocks that hold both g and u cannot be encoded by the fused kernel
  const bool fused = keep && cols % kBlock == 0;
  uint32_t items, kitems = 0;
  FastDiv div, kdiv = {};
  if ((rc = items_of(rows, ceil_div(cols, 8), &items, &div)) ||
      (keep && !fused && (rc = items_of(rows, 4 * ceil_div(2 * cols, kBlock), &kitems, &kdiv))))
    return rc;
  if (!gu || !h || (keep && (!q || !scale))) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool bf = dtype == MUON_BF16;
  if (!fused) {
    if (bf) launch_gated<bf16_t, -1>(gu, cols, h, nullptr, nullptr, items, div, s);
    else launch_gated<float, -1>(gu, cols, h, nullptr, nullptr, items, div, s);
    if ((rc = launch_status("gated launch")) || !keep) return rc;
    if (bf) launch_checkpoint<bf16_t>(gu, 2 * cols, kind, q, scale, kitems, kdiv, s);
    else launch_checkpoint<float>(gu, 2 * cols, kind, q, scale, kitems, kdiv, s);
    return launch_status("checkpoint launch");
  }
  if (bf) {
    if (kind == MUON_INT8) launch_gated<bf16_t, MUON_INT8>(gu, cols, h, q, scale, items, div, s);
    else launch_gated<bf16_t, MUON_E4M3>(gu, cols, h, q, scale, items, div, s);
  } else {
    if (kind == MUON_INT8) launch_gated<float, MUON_INT8>(gu, cols, h, q, scale, items, div, s);
    else launch_gated<float, MUON_E4M3>(gu, cols, h, q, scale, items, div, s);
  }
  return launch_status("gated launch");
}

int muon_gated_backward(const void* dh, const void* gu, const void* q, const uint8_t* scale, int kind, int dtype,
                        int64_t rows, int64_t cols, void* dgu, void* h, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  const bool kept = q || scale;
  if ((rc = check_rows(dtype, rows, cols)) || (kept && (rc = check_kind(kind)))) return rc;
  if (kept && gu) return fail(MUON_EINVAL, "either gu or its checkpoint, not both");
  if (rows == 0) return MUON_OK;
  uint32_t items;
  FastDiv div;
  if ((rc = items_of(rows, ceil_div(cols, 8), &items, &div))) return rc;
  if (!dh || !dgu || !h || (kept ? (!q || !scale) : !gu)) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MUON_BF16) launch_gated_backward<bf16_t>(dh, gu, q, scale, kind, cols, dgu, h, items, div, s);
  else launch_gated_backward<float>(dh, gu, q, scale, kind, cols, dgu, h, items, div, s);
  return launch_status("gated backward launch");
}

}  // extern "C"
