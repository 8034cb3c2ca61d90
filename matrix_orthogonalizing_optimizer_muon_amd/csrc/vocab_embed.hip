// The embedding of tokens and its gradient.
//
//   embed           out[t] = scale table[tokens[t]]
//   embed_backward  dtable[v] = scale sum over the t with tokens[t] = v of dout[t]
//
// Both are bound by memory: rows of a table read or written once.  The gradient
// has no atomics on values: the places of each token come sorted by token, then
// place, and each table row is summed by one wave (rows of many places in parts
// that are added in their order), so equal inputs give equal bits.
#include <hip/hip_runtime.h>

#include "vocab.hpp"

namespace muon {
namespace vo {
namespace {

constexpr int kCols = 512;   // columns of a wave: eight a lane

// Rows written past the caches, where a call writes more than a part of the last
// one that leaves room for what it reads (kStream): 32000 x 2048 bf16 of the
// gradient, 131 MB, 88 us by plain stores, 60 so; 16384 x 2048 of the embedding
// 18.2 and 16.5.
__device__ __forceinline__ void store8_past(bf16_t* p, int cnt, const float (&v)[8]) {
  if (cnt >= 8)
    __builtin_nontemporal_store(u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])},
                                reinterpret_cast<u32x4_any*>(p));
  else store8(p, cnt, v);
}
__device__ __forceinline__ void store8_past(float* p, int cnt, const float (&v)[8]) {
  if (cnt >= 8) {
    __builtin_nontemporal_store(u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])},
                                reinterpret_cast<u32x4_any*>(p));
    __builtin_nontemporal_store(u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])},
                                reinterpret_cast<u32x4_any*>(p + 4));
  } else {
    store8(p, cnt, v);
  }
}
constexpr int64_t kStream = int64_t(48) << 20;

// A wave has 512 columns of one token's row.
template <class T, class I, bool PAST>
__global__ __launch_bounds__(256) void k_embed(const I* __restrict__ tokens, const T* __restrict__ table, int64_t n,
                                               int32_t vocab, int64_t dim, int32_t slabs, float scale,
                                               T* __restrict__ out) {
  const int64_t unit = block_index() * 4 + (threadIdx.x >> 6);
  const int64_t t = unit / slabs;
  if (t >= n) return;
  const int64_t c = (unit - t * slabs) * kCols + (threadIdx.x & 63) * 8;
  if (c >= dim) return;
  const int cnt = dim - c < 8 ? (int)(dim - c) : 8;
  const int32_t v = read_index(tokens, t, vocab);
  float x[8] = {};
  if (v >= 0) load8(table + (int64_t)v * dim + c, cnt, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v >= 0 ? x[i] * scale : 0.f;
  if (PAST) store8_past(out + t * dim + c, cnt, x);
  else store8(out + t * dim + c, cnt, x);
}

// ------------------------------------------------------------ order of tokens

// Places sorted by token, then place, in one launch without any exchange
// between blocks: a block has `width` entries of the vocabulary, reads all
// tokens, counts those below its entries (where its places start) and those of
// each entry, and reads them again to write their places.  The tokens are cut
// into a segment for each of the 16 waves; a count for each (entry, wave), added
// up in that order, tells where a wave's places of an entry go, so each wave
// goes through its own segment in order and alone.  250 blocks read 16384
// tokens of 8 bytes from L2 in a few microseconds.
// start: vocab + 1 first places of the entries; pos and key: places, their tokens.
constexpr int kOrderThreads = 1024, kOrderWaves = 16, kOrderWidth = 512, kOrderRound = 16;

// Tokens i + 64 u, -1 from `last` on; the loads have no conditions, so that they
// are in flight together.
template <class I>
__device__ __forceinline__ void read_round(const I* __restrict__ tokens, int64_t i, int64_t last, int32_t vocab,
                                           int32_t (&v)[kOrderRound]) {
  I t[kOrderRound];
#pragma unroll
  for (int u = 0; u < kOrderRound; ++u) t[u] = tokens[i + 64 * u < last ? i + 64 * u : last - 1];
#pragma unroll
  for (int u = 0; u < kOrderRound; ++u)
    v[u] = i + 64 * u < last && t[u] >= 0 && t[u] < (I)vocab ? (int32_t)t[u] : -1;
}

template <class I>
__global__ __launch_bounds__(kOrderThreads) void k_order(const I* __restrict__ tokens, int32_t n, int32_t vocab,
                                                         int32_t width, int32_t* __restrict__ start,
                                                         int32_t* __restrict__ pos, int32_t* __restrict__ key) {
  __shared__ int32_t count[kOrderWidth * kOrderWaves];
  __shared__ int32_t sums[kOrderWaves + 1];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int32_t lo = (int32_t)((int64_t)blockIdx.x * width);
  const int32_t hi = vocab - lo < width ? vocab : lo + width;
  const int32_t cells = width * kOrderWaves, per = (cells + kOrderThreads - 1) / kOrderThreads;   // width: up to 64, or a multiple of it
  for (int i = tid; i < cells; i += kOrderThreads) count[i] = 0;
  __syncthreads();
  const int64_t segment = ((int64_t)n + kOrderThreads - 1) / kOrderThreads * 64;
  const int64_t first = w * segment < n ? w * segment : n, last = first + segment < n ? first + segment : n;
  int32_t below = 0;
  int32_t v[kOrderRound];   // the last round's tokens
  for (int64_t i = first + lane; i - lane < last; i += 64 * kOrderRound) {
    read_round(tokens, i, last, vocab, v);
#pragma unroll
    for (int u = 0; u < kOrderRound; ++u) {
      below += v[u] >= 0 && v[u] < lo;
      if (v[u] >= lo && v[u] < hi) atomicAdd(&count[(v[u] - lo) * kOrderWaves + w], 1);   // whole numbers: any order
    }
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) below += __shfl_xor(below, o, 64);
  if (lane == 0) sums[w] = below;
  __syncthreads();
  int32_t base = 0;
  for (int i = 0; i < kOrderWaves; ++i) base += sums[i];
  // exclusive sums over (entry, wave)
  int32_t mine = 0;
  const int last_cell = tid * per + per < cells ? tid * per + per : cells;
  for (int i = tid * per; i < last_cell; ++i) mine += count[i];
  const int32_t upto = wave_scan_add(mine, lane);
  __syncthreads();
  if (lane == 63) sums[w] = upto;
  __syncthreads();
  int32_t run = base + upto - mine;
  for (int i = 0; i < w; ++i) run += sums[i];
  for (int i = tid * per; i < last_cell; ++i) {
    const int32_t c = count[i];
    count[i] = run;
    run += c;
  }
  __syncthreads();
  for (int i = tid; i < hi - lo; i += kOrderThreads) start[lo + i] = count[i * kOrderWaves];
  if (hi == vocab && tid == kOrderThreads - 1) start[vocab] = run;   // cells past vocab are empty
  __syncthreads();
  const bool once = last - first <= 64 * kOrderRound;   // v still holds them
  for (int64_t i = first; i < last; i += 64 * kOrderRound) {
    if (!once) read_round(tokens, i + lane, last, vocab, v);
#pragma unroll
    for (int u = 0; u < kOrderRound; ++u) {
      const bool in = v[u] >= lo && v[u] < hi;
      uint64_t left = __ballot(in);
      while (left) {
        const int at = __ffsll((unsigned long long)left) - 1;
        const int32_t e = __builtin_amdgcn_readlane(v[u], at);
        const uint64_t same = __ballot(in && v[u] == e);
        const int32_t from = count[(e - lo) * kOrderWaves + w];
        if (in && v[u] == e) {
          const int32_t to = from + __popcll(same & ((uint64_t(1) << lane) - 1));
          pos[to] = (int32_t)(i + 64 * u + lane);
          key[to] = e;
          if (lane == at) count[(e - lo) * kOrderWaves + w] = from + __popcll(same);
        }
        left &= ~same;
      }
    }
  }
}

// ------------------------------------------------------------------- gradient

// Rows of up to kWindow places are summed by the wave that writes them, four rows
// one after the other (their places come in one load).  The
// sorted places are also cut into windows of kWindow; the places of a longer row
// are summed window by window, at most two such rows meeting in one (the row of
// its first place: part 0, and one that starts behind it: part 1), and the wave
// of the window where the row starts adds these sums up in the next launch.
// Windows of 16, 32 and 64 places: 49, 46 and 45 us for 16384 places of 32000 x 2048
// bf16 (198 MB), 20.8, 21.6 and 26.4 for 5003 of 4099 x 515 fp32.
constexpr int kWindow = 32, kGradRows = 4;   // kGradRows rows a wave

// Adds N of dout's rows, at places held one a lane.
template <class T, int N, bool WHOLE>
__device__ __forceinline__ void add_rows(const T* __restrict__ dout, int64_t dim, int32_t place, int j, int64_t c,
                                         int cnt, float (&sum)[8]) {
  float x[N][8];
#pragma unroll
  for (int u = 0; u < N; ++u)
    load8(dout + (int64_t)__builtin_amdgcn_readlane(place, j + u) * dim + c, WHOLE ? 8 : cnt, x[u]);
#pragma unroll
  for (int u = 0; u < N; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[i] += x[u][i];
}

// Sum of dout's rows at places [from, to), in their order.
template <class T, bool WHOLE>
__device__ __forceinline__ void sum_run(const T* __restrict__ dout, int64_t dim, int32_t place, int from, int to,
                                        int64_t c, int cnt, float (&sum)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = 0.f;
  int j = from;
  for (; j + 8 <= to; j += 8) add_rows<T, 8, WHOLE>(dout, dim, place, j, c, cnt, sum);
  for (; j + 2 <= to; j += 2) add_rows<T, 2, WHOLE>(dout, dim, place, j, c, cnt, sum);
  if (j < to) add_rows<T, 1, WHOLE>(dout, dim, place, j, c, cnt, sum);
}
template <class T>
__device__ __forceinline__ void sum_rows(const T* __restrict__ dout, int64_t dim, int32_t place, int from, int to,
                                         int64_t c, int cnt, float (&sum)[8]) {
  if (__all(cnt == 8)) sum_run<T, true>(dout, dim, place, from, to, c, 8, sum);
  else sum_run<T, false>(dout, dim, place, from, to, c, cnt, sum);
}

template <class T, bool PAST>
__global__ __launch_bounds__(256) void k_embed_grad(const T* __restrict__ dout, const int32_t* __restrict__ start,
                                                    const int32_t* __restrict__ pos, const int32_t* __restrict__ key,
                                                    int32_t n, int32_t vocab, int64_t dim, int32_t slabs, float scale,
                                                    T* __restrict__ dtable, float* __restrict__ parts) {
  const int lane = threadIdx.x & 63;
  const int64_t windows = ((int64_t)n + kWindow - 1) / kWindow;
  const int64_t unit = block_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t item = unit / slabs;
  const int64_t c = (unit - item * slabs) * kCols + lane * 8;
  const int cnt = c >= dim ? 0 : dim - c < 8 ? (int)(dim - c) : 8;
  float sum[8];
  if (item >= windows) {   // rows
    const int64_t v0 = (item - windows) * kGradRows;
    if (v0 >= vocab) return;
    const int32_t bound = start[v0 + lane < vocab ? v0 + lane : vocab];
    const int32_t first = __builtin_amdgcn_readlane(bound, 0);
    const bool together = __builtin_amdgcn_readlane(bound, kGradRows) - first <= 64;   // their places in one load
    int32_t place = together && first + lane < __builtin_amdgcn_readlane(bound, kGradRows) ? pos[first + lane] : 0;
#pragma unroll
    for (int r = 0; r < kGradRows; ++r) {
      if (v0 + r >= vocab) return;
      const int32_t s = __builtin_amdgcn_readlane(bound, r), e = __builtin_amdgcn_readlane(bound, r + 1);
      if (e - s > kWindow) continue;
      if (!together) place = lane < e - s ? pos[s + lane] : 0;
      const int from = together ? s - first : 0;
      sum_rows(dout, dim, place, from, from + (e - s), c, cnt, sum);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] *= scale;
      if (PAST) store8_past(dtable + (v0 + r) * dim + c, cnt, sum);
      else store8(dtable + (v0 + r) * dim + c, cnt, sum);
    }
    return;
  }
  const int32_t total = start[vocab];
  const int64_t begin = item * kWindow;
  if (begin >= total) return;
  const int here = total - begin < kWindow ? (int)(total - begin) : kWindow;
  const int32_t place = lane < here ? pos[begin + lane] : 0;
  const int32_t row = lane < here ? key[begin + lane] : 0;
  const int32_t head = __builtin_amdgcn_readlane(row, 0), tail = __builtin_amdgcn_readlane(row, here - 1);
  const int32_t head_end = start[head + 1], tail_start = start[tail];
  if (head_end - start[head] > kWindow) {
    const int to = head_end - begin < here ? (int)(head_end - begin) : here;
    sum_rows(dout, dim, place, 0, to, c, cnt, sum);
    if (cnt) store8(parts + item * 2 * dim + c, cnt, sum);
  }
  if (tail != head && start[tail + 1] - tail_start > kWindow) {
    sum_rows(dout, dim, place, (int)(tail_start - begin), here, c, cnt, sum);
    if (cnt) store8(parts + (item * 2 + 1) * dim + c, cnt, sum);
  }
}

// The long rows, each by the waves of the window where it starts.
template <class T>
__global__ __launch_bounds__(256) void k_embed_join(const int32_t* __restrict__ start, const int32_t* __restrict__ key,
                                                    int32_t n, int32_t vocab, int64_t dim, int32_t slabs, float scale,
                                                    const float* __restrict__ parts, T* __restrict__ dtable) {
  const int lane = threadIdx.x & 63;
  const int64_t unit = block_index() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t item = unit / slabs, begin = item * kWindow;
  const int32_t total = start[vocab];
  if (begin >= total) return;
  const int here = total - begin < kWindow ? (int)(total - begin) : kWindow;
  const int32_t v = key[begin + here - 1];   // a long row that starts here reaches the window's end
  const int32_t s = start[v], e = start[v + 1];
  if (e - s <= kWindow || s < begin) return;
  const int64_t c = (unit - item * slabs) * kCols + lane * 8;
  if (c >= dim) return;
  const int cnt = dim - c < 8 ? (int)(dim - c) : 8;
  float sum[8];
  load8(parts + (item * 2 + (s > begin ? 1 : 0)) * dim + c, cnt, sum);
  const int64_t upto = ((int64_t)e - 1) / kWindow;
#pragma unroll 4
  for (int64_t i = item + 1; i <= upto; ++i) {
    float x[8];
    load8(parts + i * 2 * dim + c, cnt, x);
#pragma unroll
    for (int u = 0; u < 8; ++u) sum[u] += x[u];
  }
#pragma unroll
  for (int u = 0; u < 8; ++u) sum[u] *= scale;
  store8(dtable + (int64_t)v * dim + c, cnt, sum);
}

// ----------------------------------------------------------------------- host

int64_t blocks_of(int64_t items, int64_t slabs) { return ceil_div(items * slabs, 4); }

struct GradSpace {
  uint64_t start, pos, key, parts, bytes;
};
GradSpace grad_space(int64_t tokens, int64_t vocab, int64_t dim) {
  Pieces p;
  GradSpace g;
  g.start = p.take((uint64_t)(vocab + 1) * 4);
  g.pos = p.take((uint64_t)tokens * 4);
  g.key = p.take((uint64_t)tokens * 4);
  g.parts = p.take(tokens > kWindow ? (uint64_t)ceil_div(tokens, kWindow) * 2 * dim * 4 : 0);
  g.bytes = p.used;
  return g;
}

template <class T, class I>
void launch_embed(const void* tokens, const void* table, int64_t n, int64_t vocab, int64_t dim, float scale, void* out,
                  hipStream_t s) {
  const int64_t slabs = ceil_div(dim, kCols);
  const auto kernel = n * dim * (int64_t)sizeof(T) > kStream ? &k_embed<T, I, true> : &k_embed<T, I, false>;
  hipLaunchKernelGGL(kernel, grid_of_blocks(blocks_of(n, slabs), 256), dim3(256), 0, s, static_cast<const I*>(tokens),
                     static_cast<const T*>(table), n, (int32_t)vocab, dim, (int32_t)slabs, scale, static_cast<T*>(out));
}

template <class T>
int launch_grad(const void* dout, const int32_t* start, const int32_t* pos, const int32_t* key, int64_t n,
                int64_t vocab, int64_t dim, float scale, float* parts, void* dtable, hipStream_t s) {
  const int64_t slabs = ceil_div(dim, kCols), windows = n > kWindow ? ceil_div(n, kWindow) : 0;
  // without windows no row is long
  const auto kernel = vocab * dim * (int64_t)sizeof(T) > kStream ? &k_embed_grad<T, true> : &k_embed_grad<T, false>;
  hipLaunchKernelGGL(kernel, grid_of_blocks(blocks_of(windows + ceil_div(vocab, kGradRows), slabs), 256), dim3(256), 0, s,
                     static_cast<const T*>(dout), start, pos, key, (int32_t)(windows ? n : 0), (int32_t)vocab, dim,
                     (int32_t)slabs, scale, static_cast<T*>(dtable), parts);
  if (windows)
    hipLaunchKernelGGL((k_embed_join<T>), grid_of_blocks(blocks_of(windows, slabs), 256), dim3(256), 0, s, start, key,
                       (int32_t)n, (int32_t)vocab, dim, (int32_t)slabs, scale, parts, static_cast<T*>(dtable));
  return launch_status("embedding gradient launch");
}

}  // namespace
}  // namespace vo
}  // namespace muon

using namespace muon::vo;

extern "C" {

int muon_embed(const void* tokens, int index_bytes, const void* table, int dtype, int64_t n, int64_t vocab, int64_t dim,
               float scale, void* out, void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_sizes(dtype, index_bytes, n, vocab, dim))) return rc;
  if (n == 0) return MUON_OK;
  if (!tokens || !table || !out) return fail(MUON_EINVAL, "NULL pointer");
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (dtype == MUON_BF16) {
    if (index_bytes == 8) launch_embed<bf16_t, int64_t>(tokens, table, n, vocab, dim, scale, out, s);
    else launch_embed<bf16_t, int32_t>(tokens, table, n, vocab, dim, scale, out, s);
  } else {
    if (index_bytes == 8) launch_embed<float, int64_t>(tokens, table, n, vocab, dim, scale, out, s);
    else launch_embed<float, int32_t>(tokens, table, n, vocab, dim, scale, out, s);
  }
  return launch_status("embedding launch");
}

int muon_embed_backward_workspace(int64_t n, int64_t vocab, int64_t dim, uint64_t* bytes) {
  muon::report_error(MUON_OK, "");
  if (!bytes) return fail(MUON_EINVAL, "NULL bytes");
  const int rc = check_sizes(MUON_F32, 4, n, vocab, dim);
  if (rc) return rc;
  *bytes = grad_space(n, vocab, dim).bytes;
  return MUON_OK;
}

int muon_embed_backward(const void* dout, const void* tokens, int index_bytes, int dtype, int64_t n, int64_t vocab,
                        int64_t dim, float scale, void* dtable, void* workspace, uint64_t workspace_bytes,
                        void* stream) {
  muon::report_error(MUON_OK, "");
  int rc;
  if ((rc = check_sizes(dtype, index_bytes, n, vocab, dim))) return rc;
  if (!dtable || (n > 0 && (!dout || !tokens))) return fail(MUON_EINVAL, "NULL pointer");
  const GradSpace g = grad_space(n, vocab, dim);
  if ((rc = check_workspace(workspace, workspace_bytes, g.bytes))) return rc;
  if ((rc = check_device())) return rc;
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  int32_t* start = reinterpret_cast<int32_t*>(ws + g.start);
  int32_t* pos = reinterpret_cast<int32_t*>(ws + g.pos);
  int32_t* key = reinterpret_cast<int32_t*>(ws + g.key);
  // few entries a block: tokens of one of them are placed one after the other (a call with 28569 tokens of 116: 49 us,
  // by 64 entries a block 128)
  int64_t width = ceil_div(vocab, 256);
  width = width > 64 ? ceil_div(width, 64) * 64 : width < 4 ? 4 : width;
  if (width > kOrderWidth) width = kOrderWidth;
  const dim3 grid((uint32_t)ceil_div(vocab, width));
  if (index_bytes == 8)
    hipLaunchKernelGGL((k_order<int64_t>), grid, dim3(kOrderThreads), 0, s, static_cast<const int64_t*>(tokens),
                       (int32_t)n, (int32_t)vocab, (int32_t)width, start, pos, key);
  else
    hipLaunchKernelGGL((k_order<int32_t>), grid, dim3(kOrderThreads), 0, s, static_cast<const int32_t*>(tokens),
                       (int32_t)n, (int32_t)vocab, (int32_t)width, start, pos, key);
  if ((rc = launch_status("token order launch"))) return rc;
  float* parts = reinterpret_cast<float*>(ws + g.parts);
  if (dtype == MUON_BF16) return launch_grad<bf16_t>(dout, start, pos, key, n, vocab, dim, scale, parts, dtable, s);
  return launch_grad<float>(dout, start, pos, key, n, vocab, dim, scale, parts, dtable, s);
}

}  // extern "C"
