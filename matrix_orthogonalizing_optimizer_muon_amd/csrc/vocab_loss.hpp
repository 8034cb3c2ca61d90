// What the classifier's losses (vocab_loss.hip) and their products
// (vocab_products.hip) share.
//
// Rows that count ("live": a target or a teacher entry names something) are
// numbered by slots, in their order; the products run over slots, so that work
// goes with the live rows, and read rows[slot], their number and nothing else
// from the device.  Large calls go through chunks of slots.
#pragma once
#include "vocab.hpp"

namespace muon {
namespace vo {

enum Epilogue { kStats = 0, kStatsExp = 1, kGradient = 2 };

// A product of one chunk.  Slots [slot0, slot0 + chunk), of which the first
// live(count) exist.
struct Chunk {
  const int32_t* rows;     // row of each slot
  const int32_t* count;    // live slots of the call
  int64_t slot0;
  int32_t size;            // slots a chunk can hold: rows of stats and of dl
};

// Parts into which the long sums of dx (over the vocabulary) and dw (over the rows)
// are cut.
struct ProductParts {
  int32_t dx, dw;
};

struct LossArgs {
  Chunk ch;
  const void* x;           // tokens x dim
  const void* w;           // vocab x ld
  const void* xs;          // x's live rows by slot, of ld
  int64_t tokens;
  int32_t vocab, dim;
  int32_t ld;              // dim, or, for the large tiles, dim in whole 16-byte chunks, filled up with zeros
  bool large;              // the large tiles take the products (large_sizes, and w on 16 bytes where it is not copied)
  bool chunked;            // rows of dx and dw are whole chunks on borders of 16 bytes
  int64_t dl_ld;           // elements of a row of dl: vocab in whole slabs of 64
  // exp(l / temperature) = 2^(l (to_log2 + to_log2_low)): log2(e) / temperature in two parts (bf16: the first alone)
  float to_log2, to_log2_low;
  // logits: exponents of two come as a whole number n and a sum of 2^(l to_log2 - n), so that differences of
  // exponents are exact and nothing is rounded at a logit's size
  float* stats;            // [slab][chunk] pairs (n, the smallest at or above the largest exponent; sum), or null
  // the targets of a slot of the chunk, kp places each (k, in whole fours where more than one; -1: none), and their
  // logits, which the logits' product writes as it has them in its sums: a loss near zero, or a probability near
  // one, is a difference of the two
  const int32_t* ids;
  float* picked;
  int32_t k, kp;
  // by slot of the chunk: probabilities are 2^(l to_log2 - base) scale; g is dloss times temperature, in units
  const float* base;
  const float* scale;
  const float* g;
  // (1 / u, u), or null: dl is in units of u, the largest |g| of a live row.  Losses that are averaged have one g, whose
  // rounding to bf16 would be in all of the gradients; in units of itself it is one
  const float* unit;
  void* dl;                // [chunk][dl_ld], or null
  float* z;                // [chunk][dl_ld] logits of few rows, which dl is made from and targets read; else null
  // Whether a slot has two rows of dl, twice_row(slot) and, 32 behind it, what rounding to bf16 left of the first;
  // xd has its x in both.  Rows between the live slots and whole 32 are zeros.
  bool twice;
  const void* xd;
  // gradients
  void* dx;                // tokens x dim
  void* dw;                // vocab x dim
  ProductParts parts;
  float* sums_of_parts;    // [part][chunk][ld] of dx, then [part][vocab][ld] of dw, where there are more than one
  float* sums;             // vocab x ld: of the chunks so far, or null where there is one
  bool first, last;        // chunk
};

// Rows of dl that are kept twice: a slot's two are in the registers of one lane.
__host__ __device__ __forceinline__ int64_t twice_row(int64_t slot) { return slot + slot / 32 * 32; }
__host__ __device__ __forceinline__ int32_t whole_slots(int32_t slots) { return (slots + 31) / 32 * 32; }

// log2(e) and ln 2, each in two parts
constexpr float kLog2e = 1.4426950408889634f, kLog2eLow = (float)(1.4426950408889634 - (double)kLog2e);
constexpr float kLn2 = 0.6931471805599453f, kLn2Low = (float)(0.6931471805599453 - (double)kLn2);

__device__ __forceinline__ int32_t live_slots(const Chunk& c) {
  const int64_t left = *c.count - c.slot0;
  return left < 0 ? 0 : left < c.size ? (int32_t)left : c.size;
}

// The exponent of two of a logit, less n.  In fp32 with both parts of the factor; a
// target's has to be what its sum was made with.
__device__ __forceinline__ float exponent(const LossArgs& a, float l, float n, float) {
  return fmaf(l, a.to_log2_low, fmaf(l, a.to_log2, -n));
}
__device__ __forceinline__ float exponent(const LossArgs& a, float l, float n, bf16_t) { return fmaf(l, a.to_log2, -n); }
// n of a largest logit.  Where all are -inf, and exponentials 0, the lowest number, so that 2^(n - a row's) is 0 too
// and not infinite in a row far below zero.  From 2^23 on the product is rounded to a whole number, which can lie below
// the exponent by half the distance of fp32 numbers, and in fp32 the factor's low part adds as much: then n is a number
// that does not, since pack_exps has room for less than 2, and 2^ that distance can be infinite.
template <class T>
__device__ __forceinline__ float whole_exponent(const LossArgs& a, float top) {
  constexpr float kLowest = -3.402823466e38f;
  if (top == -INFINITY) return kLowest;
  float n = fmaxf(ceilf(top * a.to_log2), kLowest);
  if (fabsf(n) >= 0x1p23f) {
    const float over = exponent(a, top, n, T());
    if (over > 0.f) {
      n += over;
      if (exponent(a, top, n, T()) > 0.f) n = __int_as_float(__float_as_int(n) + (n > 0.f ? 1 : -1));
    }
  }
  return n;
}

// Joins two sums of 2^(exponent - n) with their n; a sum of zero (exponents of -inf
// alone) has none.
__device__ __forceinline__ void merge_sums(float& n, float& sum, float n2, float sum2) {
  if (sum2 == 0.f) n2 = -INFINITY;
  const float to = fmaxf(n, n2), base = to == -INFINITY ? 0.f : to;
  sum = sum * __builtin_amdgcn_exp2f(n - base) + sum2 * __builtin_amdgcn_exp2f(n2 - base);
  n = to;
}
// The log of sum 2^n, from that of sum; and lse - l / tau of a logit.
__device__ __forceinline__ float log_of(float n, float log_sum) { return fmaf(n, kLn2, fmaf(n, kLn2Low, log_sum)); }
template <class T>
__device__ __forceinline__ float loss_term(const LossArgs& a, float l, float n, float log_sum) {
  return log_sum - exponent(a, l, n, T()) * kLn2;
}

// A teacher's entries of a row, lane l those of l + 64 i: ids, -1 where there is
// none (an id outside the vocabulary, a logit of -inf or NaN), the softmax of their
// logits over tau, and the sum of q log q.
struct TeacherRow {
  static constexpr int N = kMaxTeacher / 64;
  int32_t at[N];
  float q[N];
  float term;
  bool live;
  template <class TT, class I>
  __device__ __forceinline__ void read(const TT* teacher, const I* ids, int32_t k, int32_t vocab, float inv_tau,
                                       int lane) {
    float v[N], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int j = lane + 64 * i;
      at[i] = -1;
      v[i] = -INFINITY;
      if (j < k) {
        at[i] = read_index(ids, j, vocab);
        const float l = to_f32(teacher[j]);
        if (!(l > -INFINITY)) at[i] = -1;
        if (at[i] >= 0) v[i] = fminf(l, 3.402823466e38f);
      }
      top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
    float total = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = at[i] >= 0 ? (v[i] - top) * inv_tau : 0.f;
      q[i] = at[i] >= 0 ? expf(v[i]) : 0.f;
      total += q[i];
    }
    total = wave_sum(total);
    live = total > 0.f;
    const float log_total = live ? logf(total) : 0.f;
    term = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      q[i] = at[i] >= 0 ? q[i] / total : 0.f;
      if (q[i] > 0.f) term += q[i] * (v[i] - log_total);
    }
    term = wave_sum(term);
  }
};

// 2^(exponent - n) of a slab's n, between the first product and k_rescale.
// In 16 bits: no sign and seven bits of the exponent, which values below 2 do
// without the rest of, leave nine of the fraction, so that this rounding (2^-10 at
// the most) hardly adds to that of the gradient in bf16 (2^-8): a row's sum of dw
// off by 1.03 of what one rounding gives, where two to bf16 give 1.4.  A NaN comes
// out as anything; its row's scale is NaN.
__device__ __forceinline__ uint32_t pack_exps(float lo, float hi) {
  return __builtin_amdgcn_perm((__float_as_uint(hi) << 2) + 0x8000u, (__float_as_uint(lo) << 2) + 0x8000u, 0x07060302u);
}
__device__ __forceinline__ void unpack_exps(uint32_t p, float& lo, float& hi) {
  lo = __uint_as_float((p & 0xffffu) << 14);
  hi = __uint_as_float(p >> 16 << 14);
}

// Columns whose n and sum are kept together.
template <class T>
struct Slab;
template <>
struct Slab<bf16_t> {
  static constexpr int kCols = 64;
};
template <>
struct Slab<float> {
  static constexpr int kCols = 32;
};
inline int slab_cols(int dtype) { return dtype == MUON_BF16 ? Slab<bf16_t>::kCols : Slab<float>::kCols; }

// Whether the large tiles take a call's sizes: bf16 rows of which 31 bits address
// 256.  They read rows of whole 16-byte chunks: w is copied where its are not.
inline bool large_sizes(int dtype, int64_t tokens, int64_t vocab, int64_t dim) {
  return dtype == MUON_BF16 && vocab < (1 << 21) && dim < (1 << 21) && tokens > 0;
}
ProductParts product_parts(int dtype, int64_t tokens, int64_t vocab, int64_t dim, bool large);

// Up to so many rows of bf16 dl are kept twice (LossArgs::twice).  The gradients of
// a few rows are sums of few large entries of dl, whose rounding to bf16 does not
// average out: off by up to 2^-8, over the 2^-9 or so that rounding the result gives.
// Both rows fit one tile's 256 (or two of 128), so that the products pass over w and dw once either way,
// and dx is added up in the tile.
constexpr int64_t kTwiceRows = 128;

// Logits of few rows: whether vocab_few.hip takes them, and its
// blocks, each of which has a pair for every row in stats.
struct FewCall {
  const void* ids;
  int index_bytes;
  const void* teacher;     // or null
  int teacher_dtype;
  int32_t k;
  float tau;
  float* loss;
  float* lse;
};
bool few_rows(int dtype, int64_t tokens, int64_t vocab, int64_t dim);
int64_t few_blocks(int dtype, int64_t tokens, int64_t vocab, int64_t dim);
int few_logits(const LossArgs& a, int dtype, hipStream_t s);
bool few_keeps(int dtype, int64_t tokens, int64_t vocab, int64_t dim, int k);   // z, without gradients
int few_loss(const LossArgs& a, int dtype, const FewCall& c, hipStream_t s);

// The products, of one chunk.
int logits_product(const LossArgs& a, int dtype, Epilogue e, hipStream_t s);
int dx_product(const LossArgs& a, int dtype, hipStream_t s);
int dw_product(const LossArgs& a, int dtype, hipStream_t s);

}  // namespace vo
}  // namespace muon
