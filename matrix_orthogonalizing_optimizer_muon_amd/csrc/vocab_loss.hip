// The classifier's losses over a vocabulary without the logits in memory: cross
// entropy against one target a row, and distillation from a teacher's k largest
// logits, with the gradients of x and w.
//
//   l = x w^T;  lse = log sum_v exp(l_v / tau);  q: a row's target distribution
//   loss = tau^2 (sum_j q_j log q_j + sum_j q_j (lse - l_{id_j} / tau))
//   dl_v = g tau (exp(l_v / tau - lse) - sum_{j: id_j = v} q_j)
//   dx = dl w;  dw = dl^T x
//
// Cross entropy is k = 1, q = 1, tau = 1.  Around the products
// (vocab_products.hip) the kernels here find the rows that count and their
// targets, join the slabs' sums, and put the targets' part into dl: its entries
// there are written from the fp32 logits that the first product picked out, so
// that exp(..) - q loses nothing to the rounding of dl before the difference.
//
// dl is the products' operand and so in the type of x: bf16 rounds an entry by
// 2^-8 of what it is at the most, as it would a logits gradient in memory (in the
// loss's own pass it is rounded before, too, to 16 bits of its own: pack_exps).
#include <hip/hip_runtime.h>

#include <math.h>

#include "vocab_loss.hpp"

namespace muon {
namespace vo {
namespace {

// ---------------------------------------------------------------------- rows

template <class TT, class I>
__global__ __launch_bounds__(256) void k_teacher(const TT* __restrict__ teacher, const I* __restrict__ ids,
                                                 int64_t tokens, int32_t k, int32_t vocab, float inv_tau,
                                                 int32_t* __restrict__ id, float* __restrict__ q,
                                                 float* __restrict__ term) {
  const int lane = threadIdx.x & 63;
  const int64_t t = block_index() * 4 + (threadIdx.x >> 6);
  if (t >= tokens) return;
  TeacherRow r;
  r.read(teacher + t * k, ids + t * k, k, vocab, inv_tau, lane);
#pragma unroll
  for (int i = 0; i < TeacherRow::N; ++i) {
    const int j = lane + 64 * i;
    if (j < k) {
      id[t * k + j] = r.at[i];
      q[t * k + j] = r.q[i];
    }
  }
  if (lane == 0) term[t] = r.live ? r.term : NAN;   // NaN: no entry
}

// The live rows in their order, in one block, where there are too many for k_rows to
// count them itself: each wave has a segment, counts it, and writes it behind those
// before.  TEACHER: term tells them; else targets, which are written by slot.  Rows
// that do not count get loss and lse 0; slot: -1.
constexpr int kLiveThreads = 1024;
template <class I, bool TEACHER>
__global__ __launch_bounds__(kLiveThreads) void k_live(const I* __restrict__ targets, const float* __restrict__ term,
                                                       int32_t tokens, int32_t vocab, int32_t* __restrict__ id,
                                                       int32_t* __restrict__ rows, int32_t* __restrict__ slot,
                                                       int32_t* __restrict__ count, float* __restrict__ loss,
                                                       float* __restrict__ lse) {
  __shared__ int32_t sums[16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t segment = ((int64_t)tokens + kLiveThreads - 1) / kLiveThreads * 64;
  const int64_t first = w * segment < tokens ? w * segment : tokens;
  const int64_t last = first + segment < tokens ? first + segment : tokens;
  int32_t mine = 0;
  for (int64_t i = first; i < last; i += 512) {
    bool in[8];   // loads without conditions, so that they are in flight together
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t t = i + 64 * u + lane < last ? i + 64 * u + lane : last - 1;
      in[u] = TEACHER ? term[t] <= INFINITY : read_index(targets, t, vocab) >= 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += __popcll(__ballot(in[u] && i + 64 * u + lane < last));
  }
  if (lane == 0) sums[w] = mine;
  __syncthreads();
  int32_t at = 0, all = 0;
  for (int i = 0; i < 16; ++i) {
    at += i < w ? sums[i] : 0;
    all += sums[i];
  }
  if (threadIdx.x == 0) *count = all;
  for (int64_t i = first; i < last; i += 64) {
    const int64_t t = i + lane;
    int32_t v = -1;
    if (t < last) v = TEACHER ? (term[t] <= INFINITY ? 0 : -1) : read_index(targets, t, vocab);
    const uint64_t in = __ballot(v >= 0);
    if (t < last) {
      const int32_t to = at + __popcll(in & ((uint64_t(1) << lane) - 1));
      slot[t] = v >= 0 ? to : -1;
      if (!TEACHER && v >= 0) id[to] = v;
      if (v >= 0) rows[to] = (int32_t)t;
      else if (loss) loss[t] = lse[t] = 0.f;
    }
    at += __popcll(in);
  }
}

struct RowsArgs {
  const int32_t* slot;     // by k_live, or, where k_rows counts, what it writes:
  const float* term;
  int32_t* rows;
  int32_t* count;
  float* loss;
  float* lse_out;
  const int32_t* teacher_id;   // tokens x k
  const float* teacher_q;
  int32_t* id;             // by slot of the call, kp each
  float* q;
  const float* lse;        // tokens, or null: base, scale and g are k_join's
  const float* dloss;
  float* base;             // by slot of the call
  float* scale;
  float* g;
  float tau;
};

// Every row by itself, a wave each: a live one, and its teacher's entries, go to its
// slot; another's dx is zeros.  COUNT: blocks count the live rows before theirs
// themselves, and do what k_live does elsewhere: up to kCountRows rows, whose marks all
// blocks read from L2.  Against a launch of k_live before this one, a call over 150 rows
// is 1.4 us shorter, one over 4096 2 us, one over 8192 3.6 us; here they take 11 us.
constexpr int kRowsWaves = 16;
constexpr int64_t kCountRows = 16384;
template <class T, class I, bool TEACHER, bool COUNT>
__global__ __launch_bounds__(64 * kRowsWaves) void k_rows(LossArgs a, RowsArgs o, const I* __restrict__ targets,
                                                          T* __restrict__ xs, T* __restrict__ xd, T* __restrict__ dx) {
  __shared__ int32_t counts[kRowsWaves];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t0 = block_index() * kRowsWaves, t = t0 + w;
  int32_t s;
  if constexpr (COUNT) {
    auto marked = [&](int64_t i) { return TEACHER ? o.term[i] <= INFINITY : read_index(targets, i, a.vocab) >= 0; };
    int32_t mine = 0;
    const int64_t others = t0 < a.tokens ? t0 : a.tokens;
    for (int64_t i = threadIdx.x; i - threadIdx.x < others; i += 64 * kRowsWaves * 8) {
      bool in[8];   // loads without conditions, so that they are in flight together
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t at = i + 64 * kRowsWaves * u;
        in[u] = marked(at < others ? at : others - 1);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) mine += __popcll(__ballot(in[u] && i + 64 * kRowsWaves * u < others));
    }
    const int64_t own = t0 + (lane & (kRowsWaves - 1));
    const uint64_t here = __ballot(lane < kRowsWaves && own < a.tokens && marked(own < a.tokens ? own : a.tokens - 1));
    if (lane == 0) counts[w] = mine;
    __syncthreads();
    int32_t before = 0;
#pragma unroll
    for (int i = 0; i < kRowsWaves; ++i) before += counts[i];
    if (t0 < a.tokens && t0 + kRowsWaves >= a.tokens && threadIdx.x == 0) *o.count = before + __popcll(here);
    before += __popcll(here & ((uint64_t(1) << w) - 1));
    s = here >> w & 1 ? before : -1;
    if (a.twice && s < 0 && t < whole_slots((int32_t)a.tokens)) {   // a slot behind the live ones
      const float zero[8] = {};
      T* row = xd + twice_row(t < a.tokens ? a.tokens - 1 - (t - before) : t) * a.ld;
      for (int32_t c = lane * 8; c < a.ld; c += 512) {
        const int cnt = a.ld - c < 8 ? a.ld - c : 8;
        store8(row + c, cnt, zero);
        store8(row + 32 * (int64_t)a.ld + c, cnt, zero);
      }
    }
    if (t >= a.tokens) return;
    if (lane == 0) {
      if (s >= 0) {
        o.rows[s] = (int32_t)t;
        if (!TEACHER) o.id[s] = read_index(targets, t, a.vocab);
      } else if (o.loss) {
        o.loss[t] = o.lse_out[t] = 0.f;
      }
    }
  } else {
    if (t >= a.tokens) return;
    s = o.slot[t];
  }
  const T* x = static_cast<const T*>(a.x) + t * a.dim;
  if (s < 0) {
    const float zero[8] = {};
    if (dx)
      for (int32_t c = lane * 8; c < a.dim; c += 512) store8(dx + t * a.dim + c, a.dim - c < 8 ? a.dim - c : 8, zero);
    return;
  }
  for (int32_t c = lane * 8; c < a.dim; c += 2048) {
    float p[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int32_t at = c + 512 * u, left = a.dim - at;
      load8(x + at, left < 0 ? 0 : left < 8 ? left : 8, p[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {   // past dim: zeros
      const int32_t at = c + 512 * u, left = a.ld - at, cnt = left < 8 ? left : 8;
      if (left > 0) store8(xs + (int64_t)s * a.ld + at, cnt, p[u]);
      if (left > 0 && COUNT && a.twice) {
        T* row = xd + twice_row(s) * a.ld + at;
        store8(row, cnt, p[u]);
        store8(row + 32 * (int64_t)a.ld, cnt, p[u]);
      }
    }
  }
  if (TEACHER)
    for (int32_t i = lane; i < a.kp; i += 64) {
      o.id[(int64_t)s * a.kp + i] = i < a.k ? o.teacher_id[t * a.k + i] : -1;
      o.q[(int64_t)s * a.kp + i] = i < a.k ? o.teacher_q[t * a.k + i] : 0.f;
    }
  if (o.lse && lane == 0) {   // exp(-lse) = 2^-base scale, base a whole number
    const float lse = o.lse[t], base = rintf(lse * kLog2e);
    o.base[s] = base;
    o.scale[s] = __builtin_amdgcn_exp2f(-fmaf(lse, kLog2eLow, fmaf(lse, kLog2e, -base)));
    o.g[s] = o.dloss[t] * o.tau;
  }
}

// Rows of dim to rows of ld, zeros behind them: a wave has 512 columns of one.
__global__ __launch_bounds__(256) void k_pad(const bf16_t* __restrict__ w, int64_t rows, int32_t dim, int32_t ld,
                                             int32_t units, bf16_t* __restrict__ out) {
  const int64_t unit = block_index() * 4 + (threadIdx.x >> 6);
  const int64_t r = unit / units;
  const int32_t c = (int32_t)(unit - r * units) * 512 + (threadIdx.x & 63) * 8;
  if (r >= rows || c >= ld) return;
  float v[8];
  load8(w + r * dim + c, dim - c < 8 ? dim - c : 8, v);
  store8(out + r * ld + c, 8, v);
}

// The unit of dl; one where the largest g is zero, far from one or not a number.  Of
// a call that is given lse, g too (else k_join's).
__global__ __launch_bounds__(1024) void k_unit(LossArgs a, const float* __restrict__ dloss, float tau,
                                               float* __restrict__ unit, float* __restrict__ given) {
  __shared__ float tops[16];
  const int32_t live = __builtin_amdgcn_readfirstlane(*a.ch.count);
  float top = 0.f;
  for (int32_t i = threadIdx.x; i < live; i += 4096) {
    float g[4];   // loads without conditions, so that they are in flight together
#pragma unroll
    for (int u = 0; u < 4; ++u) g[u] = dloss[a.ch.rows[i + 1024 * u < live ? i + 1024 * u : live - 1]];
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, fabsf(g[u] * tau));
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  for (int i = 0; i < 16; ++i) top = fmaxf(top, tops[i]);
  if (!(top > 0x1p-100f && top < 0x1p100f)) top = 1.f;
  const float inverse = 1.f / top;
  if (threadIdx.x == 0) {
    unit[0] = inverse;
    unit[1] = top;
  }
  if (given)
    for (int32_t i = threadIdx.x; i < live; i += 1024) given[i] *= inverse;
}

// ------------------------------------------------------------------- targets

struct JoinArgs {
  const float* q;          // [chunk][kp], or null: 1
  const float* term;       // tokens, or null: 0
  const float* dloss;      // tokens, or null
  float* base;             // [chunk], these three: LossArgs; g null without gradients
  float* scale;
  float* g;
  float* loss;             // tokens
  float* lse;              // tokens
  int32_t slabs;
  float tau;
};

// Rows' sums over their slabs, and their losses.  A block has 16 slots (128 bytes
// of each slab's pairs) and 64 groups that go through the slabs side by side, then
// a wave for each slot.  8192 rows of 500 slabs (33 MB): 14 us; one row: 4.5 us.
constexpr int kJoinRows = 16;
template <class T>
__global__ __launch_bounds__(1024) void k_join(LossArgs a, JoinArgs j) {
  __shared__ float tops[16][kJoinRows + 1], sums[16][kJoinRows + 1];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int32_t live = live_slots(a.ch);
  const int64_t s0 = (int64_t)blockIdx.x * kJoinRows;
  if (s0 >= live) return;
  {
    const int r = threadIdx.x % kJoinRows;
    const int64_t s = s0 + r < live ? s0 + r : live - 1;
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    const f32x2* p = reinterpret_cast<const f32x2*>(a.stats) + s;
    float n = -INFINITY, sum = 0.f;
    int32_t i = threadIdx.x / kJoinRows;
    for (; i + 192 < j.slabs; i += 256) {
      f32x2 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = p[(int64_t)(i + 64 * u) * a.ch.size];
#pragma unroll
      for (int u = 0; u < 4; ++u) merge_sums(n, sum, v[u][0], v[u][1]);
    }
    for (; i < j.slabs; i += 64) {
      const f32x2 v = p[(int64_t)i * a.ch.size];
      merge_sums(n, sum, v[0], v[1]);
    }
#pragma unroll
    for (int o = kJoinRows; o < 64; o <<= 1) merge_sums(n, sum, __shfl_xor(n, o, 64), __shfl_xor(sum, o, 64));
    if (lane < kJoinRows) {
      tops[w][r] = n;
      sums[w][r] = sum;
    }
  }
  __syncthreads();
  const int64_t s = s0 + w;
  if (s >= live) return;
  float n = tops[lane & 15][w], sum = sums[lane & 15][w];
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) merge_sums(n, sum, __shfl_xor(n, o, 64), __shfl_xor(sum, o, 64));
  const int64_t t = a.ch.rows[a.ch.slot0 + s];
  const float log_sum = logf(sum);
  float off = 0.f;
  for (int32_t i = lane; i < a.kp; i += 64)
    if (a.ids[s * a.kp + i] >= 0)
      off += (j.q ? j.q[s * a.kp + i] : 1.f) *
             loss_term<T>(a, a.z ? a.z[s * a.dl_ld + a.ids[s * a.kp + i]] : a.picked[s * a.kp + i], n, log_sum);
  off = wave_sum(off);
  if (lane) return;
  j.loss[t] = j.tau * j.tau * ((j.term ? j.term[t] : 0.f) + off);
  j.lse[t] = log_of(n, log_sum);
  if (j.g) {
    j.base[s] = n;
    j.scale[s] = 1.f / sum;
    j.g[s] = a.unit ? j.dloss[t] * j.tau * a.unit[0] : j.dloss[t] * j.tau;
  }
}

// A target's entry of dl: an id that comes more than once counts with the sum of
// its weights.  All lanes bring the same slot and id.
__device__ __forceinline__ float weight_of(const LossArgs& a, const JoinArgs& j, int64_t s, int32_t v, int lane) {
  if (!j.q) return 1.f;   // k is 1
  float q = 0.f;
  for (int32_t i = lane; i < a.kp; i += 64) q += a.ids[s * a.kp + i] == v ? j.q[s * a.kp + i] : 0.f;
  return wave_sum(q);
}
template <class T>
__device__ __forceinline__ float target_entry(const LossArgs& a, float picked, float q, float base, float scale,
                                              float g) {
  return (__builtin_amdgcn_exp2f(exponent(a, picked, base, T())) * scale - q) * g;
}

__device__ __forceinline__ void load_exps(const bf16_t* p, int cnt, float (&v)[8]) {
  u32x4 t = {0u, 0u, 0u, 0u};
  if (cnt >= 8) {
    t = *reinterpret_cast<const u32x4_any*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) t[i / 2] |= (uint32_t)p[i].bits << (16 * (i % 2));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_exps(t[i], v[2 * i], v[2 * i + 1]);
}
__device__ __forceinline__ void load_exps(const float* p, int cnt, float (&v)[8]) { load8(p, cnt, v); }

// Gradients from 2^(exponent - n of its slab), in place where a slot has one row, or
// from logits (Z), and the targets' entries: a wave has 1024 columns of a slot, zeros
// past the vocabulary.
// 8192 x 32000 bf16, 1.05 GB: 176 us.
constexpr int kScaleRuns = 2, kScaleCols = 512 * kScaleRuns;
template <class T, bool Z>
__global__ __launch_bounds__(256) void k_rescale(LossArgs a, JoinArgs j, const T* exps, int32_t units) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = block_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t s = unit / units;
  const int32_t first = (int32_t)(unit - s * units) * kScaleCols;
  T* p = static_cast<T*>(a.dl) + (a.twice ? twice_row(s) : s) * a.dl_ld;
  auto store = [&](T* to, const float (&v)[kScaleRuns][8]) {
#pragma unroll
    for (int u = 0; u < kScaleRuns; ++u) {
      const int32_t c = first + 512 * u + lane * 8;
      if (c < a.dl_ld) store8(to + c, 8, v[u]);
    }
  };
  float v[kScaleRuns][8] = {};
  if (s >= live_slots(a.ch)) {
    if (a.twice && s < whole_slots(a.ch.size)) {
      store(p, v);
      store(p + 32 * a.dl_ld, v);
    }
    return;
  }
  const float base = a.base[s], scale = a.scale[s], g = a.g[s];
#pragma unroll
  for (int u = 0; u < kScaleRuns; ++u) {
    const int32_t c = first + 512 * u + lane * 8, left = a.vocab - c, cnt = left <= 0 ? 0 : left < 8 ? left : 8;
    if constexpr (Z) {
      load8(a.z + s * a.dl_ld + c, cnt, v[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[u][i] = i < cnt ? __builtin_amdgcn_exp2f(exponent(a, v[u][i], base, T())) * scale * g : 0.f;
    } else {
      load_exps(exps + s * a.dl_ld + c, cnt, v[u]);
      // past the vocabulary: zeros by a finite factor, whatever the row's base (NaN where the row's scale is)
      const float n = cnt ? a.stats[2 * ((int64_t)(c / Slab<T>::kCols) * a.ch.size + s)] : base;
      const float by = __builtin_amdgcn_exp2f(n - base) * (scale * g);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[u][i] *= by;
    }
  }
  for (int32_t j0 = 0; j0 < a.kp; j0 += 64) {
    const int32_t at = j0 + lane;
    const int32_t id = at < a.kp ? a.ids[s * a.kp + at] : -1;
    uint64_t hits = __ballot(id >= first && id - first < kScaleCols);
    while (hits) {
      const int h = __ffsll((unsigned long long)hits) - 1;
      hits &= hits - 1;
      const int32_t e = __builtin_amdgcn_readlane(id, h), c = e - first;
      const float l = Z ? a.z[s * a.dl_ld + e] : a.picked[s * a.kp + j0 + h];
      const float d = target_entry<T>(a, l, weight_of(a, j, s, e, lane), base, scale, g);
#pragma unroll
      for (int u = 0; u < kScaleRuns; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = c == 512 * u + lane * 8 + i ? d : v[u][i];
    }
  }
  store(p, v);
  if constexpr (sizeof(T) == 2) {
    if (a.twice) {
#pragma unroll
      for (int u = 0; u < kScaleRuns; ++u)
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const uint32_t first_row = pack2(v[u][i], v[u][i + 1]);
          v[u][i] -= __uint_as_float(first_row << 16);
          v[u][i + 1] -= __uint_as_float(first_row & 0xffff0000u);
        }
      store(p + 32 * a.dl_ld, v);
    }
  }
}

// The targets' entries of dl where the logits' gradients are there, a wave a slot.
template <class T>
__global__ __launch_bounds__(256) void k_targets(LossArgs a, JoinArgs j) {
  const int lane = threadIdx.x & 63;
  const int64_t s = block_index() * 4 + (threadIdx.x >> 6);
  if (s >= live_slots(a.ch)) return;
  const float base = a.base[s], scale = a.scale[s], g = a.g[s];
  T* dl = static_cast<T*>(a.dl) + s * a.dl_ld;
  for (int32_t i = 0; i < a.k; ++i) {
    const int32_t v = __builtin_amdgcn_readfirstlane(a.ids[s * a.kp + i]);
    if (v < 0) continue;
    const float d = target_entry<T>(a, a.picked[s * a.kp + i], weight_of(a, j, s, v, lane), base, scale, g);
    if (lane == 0) store1(dl + v, d);
  }
}

// ----------------------------------------------------------------------- host

struct Call {
  const void* x;
  const void* w;
  int dtype;
  int64_t tokens, vocab, dim;
  const void* targets;     // tokens x k
  int index_bytes;
  const void* teacher;     // tokens x k, or null: targets alone
  int teacher_dtype, k;
  float tau;
  const float* dloss;
  const float* lse_in;     // or null: the losses come with them
  float* loss;
  float* lse;
  void* dx;
  void* dw;                // or null: no gradients
};

// Slots of a chunk: as many as keep dl within 2 GiB and the slabs' sums within
// 256 MiB (whole batches of most models; a chunk more costs another pass over the
// sums of dw, 8 bytes an element of w).
int64_t chunk_slots(int dtype, int64_t tokens, int64_t vocab, bool grads, bool stats) {
  int64_t most = tokens;
  auto cap = [&](int64_t bytes, int64_t each) {
    int64_t n = bytes / each / 64 * 64;
    if (n < 64) n = 64;
    if (n < most) most = n;
  };
  if (grads) cap(int64_t(1) << 31, ceil_div(vocab, 64) * 64 * (dtype == MUON_BF16 ? 2 : 4));
  if (stats) cap(int64_t(1) << 28, ceil_div(vocab, slab_cols(dtype)) * 8);
  return most < 1 ? 1 : most;
}

// Places of a slot's targets: whole 16-byte fours, or one.
int32_t places(int32_t k) { return k == 1 ? 1 : (k + 3) / 4 * 4; }

struct LossSpace {
  bool few, twice, keeps;   // keeps: z, of few rows
  int64_t chunk, slabs, dl_ld;
  ProductParts parts;
  int32_t ld;
  uint64_t xs, xd, w, sums_of_parts, teacher_id, teacher_q, id, q, term, rows, slot, count, unit, stats, picked, base, scale, g, dl, z, sums, bytes;
};
LossSpace loss_space(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k, bool teacher, bool grads,
                     bool given) {
  Pieces p;
  LossSpace l = {};
  l.few = few_rows(dtype, tokens, vocab, dim);
  if (l.few && !grads) {
    l.stats = p.take((uint64_t)few_blocks(dtype, tokens, vocab, dim) * tokens * 8);
    const bool z = few_keeps(dtype, tokens, vocab, dim, k);
    l.dl_ld = ceil_div(vocab, 64) * 64;
    l.picked = p.take(z ? 0 : (uint64_t)tokens * 4);
    l.z = p.take(z ? (uint64_t)tokens * l.dl_ld * 4 : 0);
    l.keeps = z;
    l.bytes = p.used;
    return l;
  }
  const int64_t es = dtype == MUON_BF16 ? 2 : 4;
  l.chunk = chunk_slots(dtype, tokens, vocab, grads, !given);
  l.slabs = l.few ? few_blocks(dtype, tokens, vocab, dim) : ceil_div(vocab, slab_cols(dtype));
  l.dl_ld = ceil_div(vocab, 64) * 64;
  const bool large = large_sizes(dtype, tokens, vocab, dim);
  l.twice = grads && dtype == MUON_BF16 && l.chunk == tokens && tokens <= kTwiceRows;
  const int64_t rows = l.twice ? 2 * whole_slots((int32_t)l.chunk) : l.chunk;   // of dl
  l.parts = grads ? product_parts(dtype, rows, vocab, dim, large) : ProductParts{1, 1};
  l.ld = (int32_t)(large ? ceil_div(dim, 8) * 8 : dim);
  l.xs = p.take((uint64_t)tokens * l.ld * es);
  l.xd = p.take(l.twice ? (uint64_t)rows * l.ld * es : 0);
  l.w = p.take(l.ld != dim ? (uint64_t)vocab * l.ld * 2 : 0);
  const uint64_t of_dx = l.parts.dx > 1 ? (uint64_t)l.parts.dx * l.chunk * l.ld * 4 : 0;
  const uint64_t of_dw = l.parts.dw > 1 ? (uint64_t)l.parts.dw * vocab * l.ld * 4 : 0;
  l.sums_of_parts = p.take(of_dx > of_dw ? of_dx : of_dw);   // one after the other
  l.teacher_id = p.take(teacher ? (uint64_t)tokens * k * 4 : 0);
  l.teacher_q = p.take(teacher ? (uint64_t)tokens * k * 4 : 0);
  l.id = p.take((uint64_t)tokens * places(k) * 4);
  l.q = p.take(teacher ? (uint64_t)tokens * places(k) * 4 : 0);
  l.term = p.take(teacher ? (uint64_t)tokens * 4 : 0);
  l.rows = p.take((uint64_t)tokens * 4);
  l.slot = p.take((uint64_t)tokens * 4);
  l.count = p.take(4);
  l.unit = p.take(8);
  l.stats = p.take(given && (l.few || !l.twice) ? 0 : (uint64_t)l.slabs * l.chunk * 8);
  l.picked = p.take((uint64_t)tokens * places(k) * 4);
  l.base = p.take((uint64_t)tokens * 4);
  l.scale = p.take((uint64_t)tokens * 4);
  l.g = p.take((uint64_t)tokens * 4);
  l.dl = p.take(grads ? (uint64_t)rows * l.dl_ld * es : 0);
  l.keeps = l.few;
  l.z = p.take(l.few || l.twice ? (uint64_t)l.chunk * l.dl_ld * (l.few ? 4 : es) : 0);   // or exponentials
  l.sums = p.take(grads && l.chunk < tokens ? (uint64_t)vocab * l.ld * 4 : 0);
  l.bytes = p.used;
  return l;
}

// Live rows by slot, with their targets; no rows: their number alone.
template <class T, class I, bool TEACHER>
void launch_rows(const Call& c, const LossSpace& l, const LossArgs& a, char* ws, hipStream_t s) {
  const I* ids = static_cast<const I*>(c.targets);
  RowsArgs o = {};
  int32_t* slot = reinterpret_cast<int32_t*>(ws + l.slot);
  float* term = reinterpret_cast<float*>(ws + l.term);
  o.slot = slot;
  o.term = term;
  o.rows = reinterpret_cast<int32_t*>(ws + l.rows);
  o.count = reinterpret_cast<int32_t*>(ws + l.count);
  o.loss = c.loss;
  o.lse_out = c.lse;
  o.id = reinterpret_cast<int32_t*>(ws + l.id);
  o.q = reinterpret_cast<float*>(ws + l.q);
  o.lse = c.lse_in;
  o.dloss = c.dloss;
  o.base = reinterpret_cast<float*>(ws + l.base);
  o.scale = reinterpret_cast<float*>(ws + l.scale);
  o.g = reinterpret_cast<float*>(ws + l.g);
  o.tau = c.tau;
  if (TEACHER && c.tokens) {
    int32_t* teacher_id = reinterpret_cast<int32_t*>(ws + l.teacher_id);
    float* teacher_q = reinterpret_cast<float*>(ws + l.teacher_q);
    o.teacher_id = teacher_id;
    o.teacher_q = teacher_q;
    const dim3 grid = grid_of_blocks(ceil_div(c.tokens, 4), 256);
    if (c.teacher_dtype == MUON_BF16)
      hipLaunchKernelGGL((k_teacher<bf16_t, I>), grid, dim3(256), 0, s, static_cast<const bf16_t*>(c.teacher), ids,
                         c.tokens, c.k, (int32_t)c.vocab, 1.f / c.tau, teacher_id, teacher_q, term);
    else
      hipLaunchKernelGGL((k_teacher<float, I>), grid, dim3(256), 0, s, static_cast<const float*>(c.teacher), ids,
                         c.tokens, c.k, (int32_t)c.vocab, 1.f / c.tau, teacher_id, teacher_q, term);
  }
  const bool count = c.tokens > 0 && c.tokens <= kCountRows;
  if (!count)
    hipLaunchKernelGGL((k_live<I, TEACHER>), dim3(1), dim3(kLiveThreads), 0, s, ids, term, (int32_t)c.tokens,
                       (int32_t)c.vocab, o.id, o.rows, slot, o.count, c.loss, c.lse);
  if (!c.tokens) return;
  auto* kernel = count ? &k_rows<T, I, TEACHER, true> : &k_rows<T, I, TEACHER, false>;
  const int64_t rows = a.twice ? whole_slots((int32_t)c.tokens) : c.tokens;
  hipLaunchKernelGGL(kernel, grid_of_blocks(ceil_div(rows, kRowsWaves), 64 * kRowsWaves), dim3(64 * kRowsWaves), 0, s,
                     a, o, ids, reinterpret_cast<T*>(ws + l.xs), reinterpret_cast<T*>(ws + l.xd), c.dw ? static_cast<T*>(c.dx) : nullptr);
}

template <class T>
int find_rows(const Call& c, const LossSpace& l, const LossArgs& a, char* ws, hipStream_t s) {
  if (c.index_bytes == 8) {
    if (c.teacher_dtype >= 0) launch_rows<T, int64_t, true>(c, l, a, ws, s);
    else launch_rows<T, int64_t, false>(c, l, a, ws, s);
  } else {
    if (c.teacher_dtype >= 0) launch_rows<T, int32_t, true>(c, l, a, ws, s);
    else launch_rows<T, int32_t, false>(c, l, a, ws, s);
  }
  return launch_status("target launch");
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <class T>
int run(const Call& c, const LossSpace& l, char* ws, hipStream_t s) {
  const bool grads = c.dw != nullptr, given = c.lse_in != nullptr;
  int rc;
  // w in rows that the large tiles read: as it is, or copied
  const bool large = large_sizes(c.dtype, c.tokens, c.vocab, c.dim) && (l.ld != c.dim || aligned16(c.w));
  LossArgs a = {};
  a.ch.rows = reinterpret_cast<int32_t*>(ws + l.rows);
  a.ch.count = reinterpret_cast<int32_t*>(ws + l.count);
  a.ch.size = (int32_t)l.chunk;
  a.x = c.x;
  a.w = c.w;
  a.tokens = c.tokens;
  a.vocab = (int32_t)c.vocab;
  a.dim = (int32_t)c.dim;
  const double to_log2 = 1.4426950408889634 / (double)c.tau;
  a.to_log2 = (float)to_log2;
  if (sizeof(T) == 4) {   // from below, so that the low part is positive: a logit of -inf times it is -inf
    if ((double)a.to_log2 > to_log2) a.to_log2 = nextafterf(a.to_log2, 0.f);
    a.to_log2_low = fmaxf((float)(to_log2 - (double)a.to_log2), 0x1p-126f);
  }
  a.twice = l.twice;
  a.stats = given && (l.few || !a.twice) ? nullptr : reinterpret_cast<float*>(ws + l.stats);
  a.picked = reinterpret_cast<float*>(ws + l.picked);
  a.ld = l.few && !grads ? a.dim : l.ld;
  a.dl_ld = l.dl_ld;
  a.z = l.keeps ? reinterpret_cast<float*>(ws + l.z) : nullptr;
  if (l.few && !grads)
    return few_loss(a, c.dtype, FewCall{c.targets, c.index_bytes, c.teacher, c.teacher_dtype, c.k, c.tau, c.loss, c.lse},
                    s);
  a.k = c.k;
  a.kp = places(c.k);
  a.xs = ws + l.xs;
  a.xd = ws + l.xd;
  a.large = large;
  a.chunked = l.ld == c.dim && aligned16(c.dx) && aligned16(c.dw);
  if (l.ld != c.dim) {
    const int64_t units = ceil_div(l.ld, 512);
    hipLaunchKernelGGL(k_pad, grid_of_blocks(ceil_div(c.vocab * units, 4), 256), dim3(256), 0, s,
                       static_cast<const bf16_t*>(c.w), c.vocab, (int32_t)c.dim, l.ld, (int32_t)units,
                       reinterpret_cast<bf16_t*>(ws + l.w));
    a.w = ws + l.w;
  }
  a.sums_of_parts = reinterpret_cast<float*>(ws + l.sums_of_parts);
  a.parts = l.parts;
  a.dl = grads ? ws + l.dl : nullptr;
  a.dx = c.dx;
  a.dw = c.dw;
  a.sums = l.chunk < c.tokens ? reinterpret_cast<float*>(ws + l.sums) : nullptr;
  if ((rc = find_rows<T>(c, l, a, ws, s))) return rc;
  if (!c.tokens) {   // no rows: dw is zeros
    a.first = a.last = true;
    return grads ? dw_product(a, c.dtype, s) : MUON_OK;
  }
  if (grads && c.dtype == MUON_BF16 && !a.twice) {
    float* unit = reinterpret_cast<float*>(ws + l.unit);
    hipLaunchKernelGGL(k_unit, dim3(1), dim3(1024), 0, s, a, c.dloss, c.tau, unit,
                       given ? reinterpret_cast<float*>(ws + l.g) : nullptr);
    a.unit = unit;
  }
  float* base = reinterpret_cast<float*>(ws + l.base);
  float* scale = reinterpret_cast<float*>(ws + l.scale);
  float* g = reinterpret_cast<float*>(ws + l.g);
  float* picked = reinterpret_cast<float*>(ws + l.picked);
  int32_t* id = reinterpret_cast<int32_t*>(ws + l.id);
  float* q = reinterpret_cast<float*>(ws + l.q);
  JoinArgs j = {};
  j.term = c.teacher ? reinterpret_cast<float*>(ws + l.term) : nullptr;
  j.dloss = c.dloss;
  j.loss = c.loss;
  j.lse = c.lse;
  j.slabs = (int32_t)l.slabs;
  j.tau = c.tau;
  const int64_t chunks = ceil_div(c.tokens, l.chunk), slots = l.chunk;
  for (int64_t i = 0; i < chunks; ++i) {
    a.ch.slot0 = i * l.chunk;
    a.first = i == 0;
    a.last = i + 1 == chunks;
    a.base = j.base = base + a.ch.slot0;
    a.scale = j.scale = scale + a.ch.slot0;
    a.g = g + a.ch.slot0;
    j.g = grads ? g + a.ch.slot0 : nullptr;
    a.ids = id + a.ch.slot0 * a.kp;
    a.picked = picked + a.ch.slot0 * a.kp;
    j.q = c.teacher ? q + a.ch.slot0 * a.kp : nullptr;
    const bool at_once = given && !l.few && !a.twice;   // dl from the logits' product
    const Epilogue e = at_once ? kGradient : grads ? kStatsExp : kStats;
    void* const dl = a.dl;
    if (a.twice) a.dl = ws + l.z;   // the exponentials
    if ((rc = l.few ? few_logits(a, c.dtype, s) : logits_product(a, c.dtype, e, s))) return rc;
    const T* exps = static_cast<const T*>(a.dl);
    a.dl = dl;
    if (!given) hipLaunchKernelGGL((k_join<T>), dim3((uint32_t)ceil_div(slots, kJoinRows)), dim3(1024), 0, s, a, j);
    if (!grads) continue;
    if (at_once) {
      hipLaunchKernelGGL((k_targets<T>), grid_of_blocks(ceil_div(slots, 4), 256), dim3(256), 0, s, a, j);
    } else {
      const int64_t units = ceil_div(c.vocab, kScaleCols), rows = a.twice ? whole_slots((int32_t)slots) : slots;
      auto* kernel = l.few ? &k_rescale<T, true> : &k_rescale<T, false>;
      hipLaunchKernelGGL(kernel, grid_of_blocks(ceil_div(rows * units, 4), 256), dim3(256), 0, s, a, j, exps,
                         (int32_t)units);
    }
    if ((rc = launch_status("classifier loss launch"))) return rc;
    if ((rc = dx_product(a, c.dtype, s)) || (rc = dw_product(a, c.dtype, s))) return rc;
  }
  return launch_status("classifier loss launch");
}

int check_loss(const Call& c) {
  const int rc = check_sizes(c.dtype, c.index_bytes, c.tokens, c.vocab, c.dim);
  if (rc) return rc;
  if (c.teacher_dtype >= 0) {
    if (!good_dtype(c.teacher_dtype)) return fail(MUON_EUNSUPPORTED, "unsupported teacher dtype");
    if (c.k < 1) return fail(MUON_EINVAL, "k must be >= 1");
    if (c.k > kMaxTeacher) return fail(MUON_EUNSUPPORTED, "more than 256 teacher entries");
    if (c.tokens * c.k > kMaxCount) return fail(MUON_EUNSUPPORTED, "2^31 teacher entries or more");
    if (!(c.tau > 0.f && c.tau < INFINITY)) return fail(MUON_EINVAL, "temperature must be positive and finite");
    // its square, which scales the loss, and its inverse, which scales logits, are normal fp32 numbers
    if (!(c.tau >= 0x1p-63f && c.tau <= 0x1p63f))
      return fail(MUON_EUNSUPPORTED, "temperature must be in [2^-63, 2^63]");
  }
  return MUON_OK;
}

int loss_bytes(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k, int gradients, uint64_t* bytes) {
  muon::report_error(MUON_OK, "");
  if (!bytes) return fail(MUON_EINVAL, "NULL bytes");
  Call c = {};
  c.dtype = dtype;
  c.index_bytes = 4;
  c.tokens = tokens;
  c.vocab = vocab;
  c.dim = dim;
  c.k = k ? k : 1;
  c.teacher_dtype = k ? MUON_F32 : -1;
  c.tau = 1.f;
  const int rc = check_loss(c);
  if (rc) return rc;
  if (gradients < 0 || gradients > 2) return fail(MUON_EINVAL, "gradients must be 0, 1 or 2");
  *bytes = loss_space(dtype, tokens, vocab, dim, c.k, k != 0, gradients != 0, gradients == 2).bytes;
  return MUON_OK;
}

int launch_loss(const Call& c, void* workspace, uint64_t workspace_bytes, void* stream) {
  int rc;
  const bool teacher = c.teacher_dtype >= 0, grads = c.dw != nullptr;
  const LossSpace l = loss_space(c.dtype, c.tokens, c.vocab, c.dim, c.k, teacher, grads, c.lse_in != nullptr);
  if ((rc = check_workspace(workspace, workspace_bytes, l.bytes))) return rc;
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  return c.dtype == MUON_BF16 ? run<bf16_t>(c, l, ws, s) : run<float>(c, l, ws, s);
}

}  // namespace
}  // namespace vo
}  // namespace muon

using namespace muon::vo;

namespace {

Call targets_call(const void* x, const void* w, const void* targets, int index_bytes, int dtype, int64_t tokens,
                  int64_t vocab, int64_t dim) {
  Call c = {};
  c.x = x;
  c.w = w;
  c.dtype = dtype;
  c.tokens = tokens;
  c.vocab = vocab;
  c.dim = dim;
  c.targets = targets;
  c.index_bytes = index_bytes;
  c.teacher_dtype = -1;
  c.k = 1;
  c.tau = 1.f;
  return c;
}

Call teacher_call(const void* x, const void* w, const void* teacher, int teacher_dtype, const void* ids,
                  int index_bytes, int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k, float temperature) {
  Call c = targets_call(x, w, ids, index_bytes, dtype, tokens, vocab, dim);
  c.teacher = teacher;
  c.teacher_dtype = teacher_dtype < 0 ? 1 << 20 : teacher_dtype;   // negative: no dtype either
  c.k = k;
  c.tau = temperature;
  return c;
}

bool inputs(const Call& c) { return c.x && c.w && c.targets && (c.teacher_dtype < 0 || c.teacher); }

int forward(Call c, float* loss, float* lse, void* workspace, uint64_t workspace_bytes, void* stream) {
  const int rc = check_loss(c);
  if (rc || c.tokens == 0) return rc;
  if (!inputs(c) || !loss || !lse) return fail(MUON_EINVAL, "NULL pointer");
  c.loss = loss;
  c.lse = lse;
  return launch_loss(c, workspace, workspace_bytes, stream);
}

int with_gradients(Call c, const float* dloss, float* loss, float* lse, const float* lse_in, void* dx, void* dw,
                   void* workspace, uint64_t workspace_bytes, void* stream) {
  const int rc = check_loss(c);
  if (rc) return rc;
  if (!dw || (c.tokens > 0 && (!inputs(c) || !dloss || !dx || (lse_in ? false : !loss || !lse))))
    return fail(MUON_EINVAL, "NULL pointer");
  c.dloss = dloss;
  c.loss = loss;
  c.lse = lse;
  c.lse_in = lse_in;
  c.dx = dx;
  c.dw = dw;
  return launch_loss(c, workspace, workspace_bytes, stream);
}

}  // namespace

extern "C" {

int muon_classifier_loss_workspace(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int gradients,
                                   uint64_t* bytes) {
  return loss_bytes(dtype, tokens, vocab, dim, 0, gradients, bytes);
}

int muon_classifier_loss(const void* x, const void* w, const void* targets, int index_bytes, int dtype, int64_t tokens,
                         int64_t vocab, int64_t dim, float* loss, float* lse, void* workspace,
                         uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  return forward(targets_call(x, w, targets, index_bytes, dtype, tokens, vocab, dim), loss, lse, workspace,
                 workspace_bytes, stream);
}

int muon_classifier_loss_grads(const float* dloss, const void* x, const void* w, const void* targets, int index_bytes,
                               int dtype, int64_t tokens, int64_t vocab, int64_t dim, float* loss, float* lse,
                               void* dx, void* dw, void* workspace, uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  return with_gradients(targets_call(x, w, targets, index_bytes, dtype, tokens, vocab, dim), dloss, loss, lse, nullptr,
                        dx, dw, workspace, workspace_bytes, stream);
}

int muon_classifier_loss_backward(const float* dloss, const void* x, const void* w, const void* targets,
                                  const float* lse, int index_bytes, int dtype, int64_t tokens, int64_t vocab,
                                  int64_t dim, void* dx, void* dw, void* workspace, uint64_t workspace_bytes,
                                  void* stream) {
  muon::report_error(MUON_OK, "");
  if (tokens > 0 && !lse) return fail(MUON_EINVAL, "NULL pointer");
  static const float none = 0.f;   // no rows: lse is not read
  return with_gradients(targets_call(x, w, targets, index_bytes, dtype, tokens, vocab, dim), dloss, nullptr, nullptr,
                        lse ? lse : &none, dx, dw, workspace, workspace_bytes, stream);
}

int muon_distill_loss_workspace(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k, int gradients,
                                uint64_t* bytes) {
  if (k < 1) return fail(MUON_EINVAL, "k must be >= 1");
  return loss_bytes(dtype, tokens, vocab, dim, k, gradients, bytes);
}

int muon_distill_loss(const void* x, const void* w, const void* teacher, int teacher_dtype, const void* ids,
                      int index_bytes, int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k, float temperature,
                      float* loss, float* lse, void* workspace, uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  return forward(teacher_call(x, w, teacher, teacher_dtype, ids, index_bytes, dtype, tokens, vocab, dim, k, temperature),
                 loss, lse, workspace, workspace_bytes, stream);
}

int muon_distill_loss_grads(const float* dloss, const void* x, const void* w, const void* teacher, int teacher_dtype,
                            const void* ids, int index_bytes, int dtype, int64_t tokens, int64_t vocab, int64_t dim,
                            int k, float temperature, float* loss, float* lse, void* dx, void* dw, void* workspace,
                            uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  return with_gradients(teacher_call(x, w, teacher, teacher_dtype, ids, index_bytes, dtype, tokens, vocab, dim, k,
                                     temperature),
                        dloss, loss, lse, nullptr, dx, dw, workspace, workspace_bytes, stream);
}

int muon_distill_loss_backward(const float* dloss, const void* x, const void* w, const void* teacher,
                               int teacher_dtype, const void* ids, const float* lse, int index_bytes, int dtype,
                               int64_t tokens, int64_t vocab, int64_t dim, int k, float temperature, void* dx,
                               void* dw, void* workspace, uint64_t workspace_bytes, void* stream) {
  muon::report_error(MUON_OK, "");
  if (tokens > 0 && !lse) return fail(MUON_EINVAL, "NULL pointer");
  static const float none = 0.f;
  return with_gradients(teacher_call(x, w, teacher, teacher_dtype, ids, index_bytes, dtype, tokens, vocab, dim, k,
                                     temperature),
                        dloss, nullptr, nullptr, lse ? lse : &none, dx, dw, workspace, workspace_bytes, stream);
}

}  // extern "C"
