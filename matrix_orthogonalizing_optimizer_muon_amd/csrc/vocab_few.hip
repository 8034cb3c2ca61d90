// The classifier's losses of few rows without gradients (scoring token by token):
// what counts is how fast w comes from memory, once for all rows.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "expert_few.hpp"
#include "vocab_loss.hpp"

namespace muon {
namespace vo {
namespace {

constexpr int kFewWaves = 8, kFewLds = 140 * 1024;

// LDS of one row of x: its columns in whole steps of k, and 16 bytes so that 16
// rows read at one chunk lie on different banks.
template <class T>
__host__ __device__ constexpr int64_t few_row_bytes(int64_t dim) {
  constexpr int64_t STEP = 4 * Few<T>::PER;
  return (dim + STEP - 1) / STEP * STEP * (int64_t)sizeof(T) + 16;
}

// The exponents' sums of up to 16 NB rows (of x, whole in LDS) over w: a wave has
// 16 rows of w at a time, which come straight into the MFMA operands (lane l: 16
// bytes of row l % 16), eight loads in flight; lane l gets row l % 16 of x and rows
// 4 (l / 16) + 0..3 of w.  Bound by w's way from memory: 32000 x 1024 bf16, 66 MB, one row: 14 us.
// stats: [block][row] pairs.
template <class T, int NB>
__global__ __launch_bounds__(64 * kFewWaves) void k_few_logits(LossArgs a) {
  constexpr int PER = Few<T>::PER, STEP = 4 * PER, U = 8;
  __shared__ __attribute__((aligned(16))) char lds[kFewLds];
  __shared__ float tops[kFewWaves][16 * NB], sums[kFewWaves][16 * NB];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ld = (int)few_row_bytes<T>(a.dim), chunks = ld / 16 - 1, rows = (int)a.tokens;
  for (int i = tid; i < 16 * NB * chunks; i += 64 * kFewWaves) {
    const int r = i / chunks, c = i - r * chunks, left = a.dim - c * PER;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (r < rows && left > 0) v = load16(static_cast<const T*>(a.x) + (int64_t)r * a.dim + c * PER, left);
    *reinterpret_cast<u32x4*>(lds + r * ld + c * 16) = v;
  }
  __syncthreads();
  const char* xp = lds + (lane & 15) * ld + (lane >> 4) * 16;
  const int32_t groups = (int32_t)(((int64_t)a.vocab + 15) / 16), steps = a.dim / STEP, at = PER * (lane >> 4);
  float n[NB], sum[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    n[b] = -INFINITY;
    sum[b] = 0.f;
  }
  for (int32_t grp = blockIdx.x * kFewWaves + w; grp < groups; grp += gridDim.x * kFewWaves) {
    const int32_t r0 = grp * 16, r = r0 + (lane & 15);
    const T* wp = static_cast<const T*>(a.w) + (int64_t)(r < a.vocab ? r : a.vocab - 1) * a.dim + at;
    Acc16 acc[NB] = {};
    int s = 0;
    for (; s + U <= steps; s += U) {
      u32x4 f[U];
#pragma unroll
      for (int u = 0; u < U; ++u) f[u] = *reinterpret_cast<const u32x4_any*>(wp + (s + u) * STEP);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int b = 0; b < NB; ++b)
          acc[b] = multiply16(f[u], *reinterpret_cast<const u32x4*>(xp + b * 16 * ld + (s + u) * 64), acc[b], T());
    }
    for (; s * STEP < a.dim; ++s) {
      const int left = a.dim - at - s * STEP;
      const u32x4 f = left > 0 ? load16(wp + s * STEP, left) : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int b = 0; b < NB; ++b)
        acc[b] = multiply16(f, *reinterpret_cast<const u32x4*>(xp + b * 16 * ld + s * 64), acc[b], T());
    }
    const int32_t left = a.vocab - r0 - 4 * (lane >> 4);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float top = -INFINITY, add = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) top = fmaxf(top, acc[b][i]);
      const float m = whole_exponent(a, top);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) add += __builtin_amdgcn_exp2f(exponent(a, acc[b][i], m, T()));
      merge_sums(n[b], sum[b], m, add);
    }
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
#pragma unroll
    for (int o = 16; o < 64; o <<= 1) merge_sums(n[b], sum[b], __shfl_xor(n[b], o, 64), __shfl_xor(sum[b], o, 64));
    if (lane < 16) {
      tops[w][16 * b + lane] = n[b];
      sums[w][16 * b + lane] = sum[b];
    }
  }
  __syncthreads();
  if (tid >= rows) return;   // rows <= 16 NB <= 64
  float top = tops[0][tid], all = sums[0][tid];
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) merge_sums(top, all, tops[i][tid], sums[i][tid]);
  float* st = a.stats + 2 * ((int64_t)blockIdx.x * rows + tid);
  st[0] = top;
  st[1] = all;
}

// A row's loss from the blocks' sums, by one block: its targets' logits are dot
// products of its waves.  TT: the teacher's type, or void: targets alone.
template <class T, class I, class TT>
__global__ __launch_bounds__(512) void k_few_join(LossArgs a, const I* __restrict__ ids, const TT* __restrict__ teacher,
                                                  int32_t k, int32_t blocks, float tau, float* __restrict__ loss,
                                                  float* __restrict__ lse) {
  constexpr bool kTeacher = !std::is_same<TT, void>::value;
  __shared__ float tops[8], sums[8], picked[kMaxTeacher];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t = blockIdx.x;
  float n = -INFINITY, sum = 0.f;
  for (int i = tid; i < blocks; i += 512) {
    const float* st = a.stats + 2 * ((int64_t)i * a.tokens + t);
    merge_sums(n, sum, st[0], st[1]);
  }
  TeacherRow r;
  if constexpr (kTeacher) {
    r.read(teacher + t * k, ids + t * k, k, a.vocab, 1.f / tau, lane);
  } else {
    r.at[0] = lane == 0 ? read_index(ids, t, a.vocab) : -1;
    r.q[0] = 1.f;
    r.term = 0.f;
    r.live = __builtin_amdgcn_readfirstlane(r.at[0]) >= 0;
  }
  if (!r.live) {   // of the whole block
    if (tid == 0) loss[t] = lse[t] = 0.f;
    return;
  }
  const T* x = static_cast<const T*>(a.x) + t * a.dim;
  if constexpr (kTeacher) {   // entries w, w + 8, .. two at a time
#pragma unroll
    for (int i = 0; i < TeacherRow::N; ++i)
      for (int j = w; j < 64 && j + 64 * i < k; j += 16) {
        const int32_t v0 = __builtin_amdgcn_readlane(r.at[i], j);
        const int32_t v1 = __builtin_amdgcn_readlane(r.at[i], j + 8 < 64 ? j + 8 : j);
        const T* w0 = static_cast<const T*>(a.w) + (int64_t)(v0 < 0 ? 0 : v0) * a.dim;
        const T* w1 = static_cast<const T*>(a.w) + (int64_t)(v1 < 0 ? 0 : v1) * a.dim;
        float d0 = 0.f, d1 = 0.f;
#pragma unroll 2
        for (int32_t c = lane * 8; c < a.dim; c += 512) {
          const int cnt = a.dim - c < 8 ? a.dim - c : 8;
          float p[8], q0[8], q1[8];
          load8(x + c, cnt, p);
          load8(w0 + c, cnt, q0);
          load8(w1 + c, cnt, q1);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            d0 += p[u] * q0[u];
            d1 += p[u] * q1[u];
          }
        }
        d0 = wave_sum(d0);
        d1 = wave_sum(d1);
        if (lane == 0) {   // an entry that is not there is not read
          picked[j + 64 * i] = d0;
          if (j + 8 < 64) picked[j + 8 + 64 * i] = d1;
        }
      }
  } else if (w == 0) {
    const float d = row_dot(x, static_cast<const T*>(a.w) + (int64_t)__builtin_amdgcn_readfirstlane(r.at[0]) * a.dim,
                            a.dim, lane);
    if (lane == 0) picked[0] = d;
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) merge_sums(n, sum, __shfl_xor(n, o, 64), __shfl_xor(sum, o, 64));
  if (lane == 0) {
    tops[w] = n;
    sums[w] = sum;
  }
  __syncthreads();
  if (w) return;
  n = tops[0];
  sum = sums[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) merge_sums(n, sum, tops[i], sums[i]);
  const float log_sum = logf(sum);
  float off = 0.f;
#pragma unroll
  for (int i = 0; i < (kTeacher ? TeacherRow::N : 1); ++i)
    if (r.at[i] >= 0) off += r.q[i] * loss_term(a, picked[lane + 64 * i], n, log_sum);
  off = wave_sum(off);
  if (lane) return;
  loss[t] = tau * tau * (r.term + off);
  lse[t] = log_of(n, log_sum);
}

template <class T>
int launch(const LossArgs& a, const FewCall& c, hipStream_t s) {
  const dim3 grid((uint32_t)few_blocks(a.vocab)), block(64 * kFewWaves);
  const int nb = (int)((a.tokens + 15) / 16);
  if (nb == 1) hipLaunchKernelGGL((k_few_logits<T, 1>), grid, block, 0, s, a);
  else if (nb == 2) hipLaunchKernelGGL((k_few_logits<T, 2>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((k_few_logits<T, 4>), grid, block, 0, s, a);
  const dim3 rows((uint32_t)a.tokens);
  const int32_t blocks = (int32_t)grid.x;
  auto join = [&](auto index, auto* teacher) {
    typedef decltype(index) I;
    typedef typename std::remove_const<typename std::remove_pointer<decltype(teacher)>::type>::type TT;
    hipLaunchKernelGGL((k_few_join<T, I, TT>), rows, dim3(512), 0, s, a, static_cast<const I*>(c.ids), teacher, c.k,
                       blocks, c.tau, c.loss, c.lse);
  };
  auto by_teacher = [&](auto index) {
    if (!c.teacher) join(index, static_cast<const void*>(nullptr));
    else if (c.teacher_dtype == MUON_BF16) join(index, static_cast<const bf16_t*>(c.teacher));
    else join(index, static_cast<const float*>(c.teacher));
  };
  if (c.index_bytes == 8) by_teacher(int64_t(0));
  else by_teacher(int32_t(0));
  return launch_status("classifier loss launch");
}

}  // namespace

// 256 blocks of one CU each go through w; fewer where there is not a wave's work for each.
int64_t few_blocks(int64_t vocab) {
  const int64_t blocks = ceil_div(vocab, 16 * kFewWaves);
  return blocks < 256 ? blocks : 256;
}

bool few_rows(int dtype, int64_t tokens, int64_t dim) {
  if (tokens < 1 || tokens > 64) return false;
  const int64_t row = dtype == MUON_BF16 ? few_row_bytes<bf16_t>(dim) : few_row_bytes<float>(dim);
  return (tokens <= 16 ? 16 : tokens <= 32 ? 32 : 64) * row <= kFewLds;
}

int few_loss(const LossArgs& a, int dtype, const FewCall& c, hipStream_t s) {
  return dtype == MUON_BF16 ? launch<bf16_t>(a, c, s) : launch<float>(a, c, s);
}

}  // namespace vo
}  // namespace muon
