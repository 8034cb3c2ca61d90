// The classifier's losses of few rows (scoring token by token), and their logits for
// the gradients: what counts is how fast w comes from memory, once for all rows.
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

int row_blocks(int64_t tokens) { return tokens <= 16 ? 1 : tokens <= 32 ? 2 : tokens <= 64 ? 4 : 8; }

bool fits(int dtype, int64_t tokens, int64_t dim) {
  const int64_t row = dtype == MUON_BF16 ? few_row_bytes<bf16_t>(dim) : few_row_bytes<float>(dim);
  return tokens <= 64 && 16 * row_blocks(tokens) * row <= kFewLds;
}

// Whether a block has 16 entries of the vocabulary and reads x for them from L2: up to
// one for each CU, and where x is larger than LDS as long as that is less than the
// large tiles take for few rows (k-tiles of 0.9 us on few CUs).  Losses, us, so and by
// those: 24 rows of 4551 x 2624 19, 46; 64 of 8192 x 4096 42, 65; 32 of 16384 x 2560
// 34, 48; 100 of 4000 x 2048 22, 40; 420 of 20 x 3200 31, 58; 50 of 8000 x 1536 in
// fp32 31, 67; 4000 of 100 x 2048 in fp32 53, 93.
bool narrow(int dtype, int64_t tokens, int64_t vocab, int64_t dim) {
  return fits(dtype, tokens, dim) ? vocab <= 16 * 256 : vocab * (ceil_div(tokens, 16) * 16) <= (1 << 19);
}

// What a wave does with the logits of 16 entries of the vocabulary from r0 on and NB
// times 16 rows from 16 b0 on: lane l has those of row l % 16 and of entries
// 4 (l / 16) + 0..3.  They are kept in z, or, where that is null, those of the up to 64
// rows' targets go to picked as they come by.
template <class T, int NB, class I>
__device__ __forceinline__ void take_logits(const LossArgs& a, const I* targets, int rows, int32_t r0, int b0,
                                            int lane, const Acc16 (&acc)[NB], float (&n)[NB], float (&sum)[NB]) {
  if (!a.z) {
    const uint64_t id = lane < rows ? (uint64_t)(int64_t)targets[lane] : ~uint64_t(0);
    const uint64_t off = id - (uint64_t)r0;   // below: huge
    uint64_t hits = __ballot(off < 16 && id < (uint64_t)a.vocab);
    while (hits) {
      const int t = __ffsll((unsigned long long)hits) - 1;
      hits &= hits - 1;
      const int c = __builtin_amdgcn_readlane((int32_t)off, t);
      float x = 0.f;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < 4; ++i) x = t >> 4 == b0 + b && (c & 3) == i ? acc[b][i] : x;
      if (lane == (t & 15) + 16 * (c >> 2)) a.picked[t] = x;
    }
  }
  const int32_t left = a.vocab - r0 - 4 * (lane >> 4);
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const int t = 16 * (b0 + b) + (lane & 15);
    if (a.z && t < rows) *reinterpret_cast<Acc16*>(a.z + t * a.dl_ld + r0 + 4 * (lane >> 4)) = acc[b];
    float top = -INFINITY, add = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) top = fmaxf(top, acc[b][i]);
    const float m = whole_exponent<T>(a, top);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) add += __builtin_amdgcn_exp2f(exponent(a, acc[b][i], m, T()));
    merge_sums(n[b], sum[b], m, add);
  }
}

// The exponents' sums of up to 16 NB rows (of x, whole in LDS) over w: a wave has
// 16 rows of w at a time, which come straight into the MFMA operands (lane l: 16
// bytes of row l % 16), eight loads in flight; lane l gets row l % 16 of x and rows
// 4 (l / 16) + 0..3 of w.  Bound by w's way from memory: 32000 x 1024 bf16, 66 MB, one row: 14 us.
// stats: [block][row] pairs.  GRADS: rows are slots.
template <class T, int NB, class I, bool GRADS>
__global__ __launch_bounds__(64 * kFewWaves) void k_few_logits(LossArgs a, const I* __restrict__ targets) {
  constexpr int PER = Few<T>::PER, STEP = 4 * PER, U = 8;
  __shared__ __attribute__((aligned(16))) char lds[kFewLds];
  __shared__ float tops[kFewWaves][16 * NB], sums[kFewWaves][16 * NB];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ld = (int)few_row_bytes<T>(a.dim), chunks = ld / 16 - 1, rows = GRADS ? live_slots(a.ch) : (int)a.tokens;
  const T* x = static_cast<const T*>(GRADS ? a.xs : a.x);
  for (int i0 = tid; i0 < 16 * NB * chunks; i0 += 64 * kFewWaves * U) {
    u32x4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 64 * kFewWaves * u, r = i / chunks, c = i - r * chunks, left = a.dim - c * PER;
      v[u] = u32x4{0u, 0u, 0u, 0u};
      if (r < rows && left > 0) v[u] = load16(x + (int64_t)r * a.ld + c * PER, left);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 64 * kFewWaves * u, r = i / chunks;
      if (r < 16 * NB) *reinterpret_cast<u32x4*>(lds + r * ld + (i - r * chunks) * 16) = v[u];
    }
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
    const T* wp = static_cast<const T*>(a.w) + (int64_t)(r < a.vocab ? r : a.vocab - 1) * a.ld + at;
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
    take_logits<T, NB, I>(a, targets, rows, r0, 0, lane, acc, n, sum);
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
  if (tid >= rows || !a.stats) return;   // rows <= 16 NB <= 64
  float top = tops[0][tid], all = sums[0][tid];
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) merge_sums(top, all, tops[i][tid], sums[i][tid]);
  float* st = a.stats + 2 * ((int64_t)blockIdx.x * (GRADS ? a.ch.size : rows) + tid);
  st[0] = top;
  st[1] = all;
}

// The same with a block for 16 entries of the vocabulary (narrow): its waves have a
// piece of the columns each, of w and of x straight from memory, and the results are
// added up in LDS, 16 rows by a wave.  24 rows, 500 x 2048 bf16: 8.5 us, by waves
// with all columns 20.
template <class T, int NB, bool GRADS>
__global__ __launch_bounds__(64 * kFewWaves) void k_few_narrow(LossArgs a) {
  constexpr int PER = Few<T>::PER, STEP = 4 * PER, U = NB == 8 ? 2 : NB == 4 ? 4 : 8;
  __shared__ Acc16 pieces[kFewWaves][NB][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row0 = blockIdx.y * 128, rows = GRADS ? live_slots(a.ch) : (int)a.tokens;
  if (rows <= row0) return;
  const int32_t r0 = blockIdx.x * 16, r = r0 + (lane & 15), at = PER * (lane >> 4);
  const T* wp = static_cast<const T*>(a.w) + (int64_t)(r < a.vocab ? r : a.vocab - 1) * a.ld + at;
  const T* xp[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {   // rows past the last: its results are not kept
    const int t = row0 + 16 * b + (lane & 15);
    xp[b] = static_cast<const T*>(GRADS ? a.xs : a.x) + (int64_t)(t < rows ? t : rows - 1) * a.ld + at;
  }
  const int32_t steps = (a.dim + STEP - 1) / STEP, per = (steps + kFewWaves - 1) / kFewWaves;
  const int32_t end = (w + 1) * per < steps ? (w + 1) * per : steps, full = end < a.dim / STEP ? end : a.dim / STEP;
  Acc16 acc[NB] = {};
  int32_t s = w * per;
  for (; s + U <= full; s += U) {
    u32x4 f[U], g[U][NB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      f[u] = *reinterpret_cast<const u32x4_any*>(wp + (s + u) * STEP);
#pragma unroll
      for (int b = 0; b < NB; ++b) g[u][b] = *reinterpret_cast<const u32x4_any*>(xp[b] + (s + u) * STEP);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[b] = multiply16(f[u], g[u][b], acc[b], T());
  }
  for (; s < end; ++s) {
    const int left = a.dim - at - s * STEP;
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const u32x4 f = left > 0 ? load16(wp + s * STEP, left) : zero;
#pragma unroll
    for (int b = 0; b < NB; ++b) acc[b] = multiply16(f, left > 0 ? load16(xp[b] + s * STEP, left) : zero, acc[b], T());
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) pieces[w][b][lane] = acc[b];
  __syncthreads();
  if (w >= NB || row0 + 16 * w >= rows) return;
  Acc16 all[1] = {pieces[0][w][lane]};
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) all[0] += pieces[i][w][lane];
  float n[1] = {-INFINITY}, sum[1] = {0.f};
  take_logits<T, 1, int32_t>(a, nullptr, rows, r0, row0 / 16 + w, lane, all, n, sum);
#pragma unroll
  for (int o = 16; o < 64; o <<= 1) merge_sums(n[0], sum[0], __shfl_xor(n[0], o, 64), __shfl_xor(sum[0], o, 64));
  const int t = row0 + 16 * w + lane;
  if (lane >= 16 || t >= rows || !a.stats) return;
  float* st = a.stats + 2 * ((int64_t)blockIdx.x * (GRADS ? a.ch.size : rows) + t);
  st[0] = n[0];
  st[1] = sum[0];
}

// A row's loss from the blocks' sums, by one block.  TT: the teacher's type, or void:
// targets alone.
template <class T, class I, class TT>
__global__ __launch_bounds__(512) void k_few_join(LossArgs a, const I* __restrict__ ids, const TT* __restrict__ teacher,
                                                  int32_t k, int32_t blocks, float tau, float* __restrict__ loss,
                                                  float* __restrict__ lse) {
  constexpr bool kTeacher = !std::is_same<TT, void>::value;
  __shared__ float tops[8], sums[8];
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
    if (r.at[i] >= 0) off += r.q[i] * loss_term<T>(a, a.z ? a.z[t * a.dl_ld + r.at[i]] : a.picked[t], n, log_sum);
  off = wave_sum(off);
  if (lane) return;
  loss[t] = tau * tau * (r.term + off);
  lse[t] = log_of(n, log_sum);
}

template <class T, class I, bool GRADS>
void launch_logits(const LossArgs& a, const I* targets, hipStream_t s) {
  constexpr int kType = sizeof(T) == 2 ? MUON_BF16 : MUON_F32;
  const dim3 block(64 * kFewWaves);
  const uint32_t blocks = (uint32_t)few_blocks(kType, a.tokens, a.vocab, a.dim);
  const int nb = row_blocks(a.tokens);
  if (narrow(kType, a.tokens, a.vocab, a.dim)) {
    auto* kernel = nb == 1   ? &k_few_narrow<T, 1, GRADS>
                   : nb == 2 ? &k_few_narrow<T, 2, GRADS>
                   : nb == 4 ? &k_few_narrow<T, 4, GRADS>
                             : &k_few_narrow<T, 8, GRADS>;
    hipLaunchKernelGGL(kernel, dim3(blocks, (uint32_t)ceil_div(a.tokens, 128)), block, 0, s, a);
    return;
  }
  auto* kernel = nb == 1 ? &k_few_logits<T, 1, I, GRADS> : nb == 2 ? &k_few_logits<T, 2, I, GRADS>
                                                                  : &k_few_logits<T, 4, I, GRADS>;
  hipLaunchKernelGGL(kernel, dim3(blocks), block, 0, s, a, targets);
}

template <class T>
int launch(const LossArgs& a, const FewCall& c, hipStream_t s) {
  const dim3 rows((uint32_t)a.tokens);
  const int32_t blocks = (int32_t)few_blocks(sizeof(T) == 2 ? MUON_BF16 : MUON_F32, a.tokens, a.vocab, a.dim);
  auto by_index = [&](auto index) {
    typedef decltype(index) I;
    const I* ids = static_cast<const I*>(c.ids);
    launch_logits<T, I, false>(a, ids, s);
    auto join = [&](auto* teacher) {
      typedef typename std::remove_const<typename std::remove_pointer<decltype(teacher)>::type>::type TT;
      hipLaunchKernelGGL((k_few_join<T, I, TT>), rows, dim3(512), 0, s, a, ids, teacher, c.k, blocks, c.tau, c.loss, c.lse);
    };
    if (!c.teacher) join(static_cast<const void*>(nullptr));
    else if (c.teacher_dtype == MUON_BF16) join(static_cast<const bf16_t*>(c.teacher));
    else join(static_cast<const float*>(c.teacher));
  };
  if (c.index_bytes == 8) by_index(int64_t(0));
  else by_index(int32_t(0));
  return launch_status("classifier loss launch");
}

}  // namespace

// 256 blocks of one CU each go through w; fewer where there is not a wave's work for each.
int64_t few_blocks(int dtype, int64_t tokens, int64_t vocab, int64_t dim) {
  if (narrow(dtype, tokens, vocab, dim)) return ceil_div(vocab, 16);
  const int64_t blocks = ceil_div(vocab, 16 * kFewWaves);
  return blocks < 256 ? blocks : 256;
}

bool few_rows(int dtype, int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens < 1) return false;
  return fits(dtype, tokens, dim) || narrow(dtype, tokens, vocab, dim);
}

int few_logits(const LossArgs& a, int dtype, hipStream_t s) {
  if (dtype == MUON_BF16) launch_logits<bf16_t, int32_t, true>(a, nullptr, s);
  else launch_logits<float, int32_t, true>(a, nullptr, s);
  return launch_status("classifier product launch");
}

// k 1: the targets' logits are picked as they come by, unless blocks' waves share columns.
bool few_keeps(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k) {
  return k > 1 || narrow(dtype, tokens, vocab, dim);
}

int few_loss(const LossArgs& a, int dtype, const FewCall& c, hipStream_t s) {
  return dtype == MUON_BF16 ? launch<bf16_t>(a, c, s) : launch<float>(a, c, s);
}

}  // namespace vo
}  // namespace muon
