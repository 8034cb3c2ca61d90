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

struct LossArgs {
  Chunk ch;
  const void* x;           // tokens x dim
  const void* w;           // vocab x dim
  const void* xs;          // x's live rows by slot, or null where the products gather them
  int64_t tokens;
  int32_t vocab, dim;
  int64_t dl_ld;           // elements of a row of dl: vocab in whole slabs of 64
  // exp(l / temperature) = 2^(l (to_log2 + to_log2_low)): log2(e) / temperature in two parts
  float to_log2, to_log2_low;
  // logits: exponents of two come as a whole number n and a sum of 2^(l to_log2 - n), so that differences of
  // exponents are exact and nothing is rounded at a logit's size
  float* stats;            // [slab][chunk] pairs (n, the smallest at or above the largest exponent; sum), or null
  // by slot of the chunk: probabilities are 2^(l to_log2 - base) scale; g is dloss times temperature
  const float* base;
  const float* scale;
  const float* g;
  void* dl;                // [chunk][dl_ld], or null
  // gradients
  void* dx;                // tokens x dim
  void* dw;                // vocab x dim
  float* dx_parts;         // [part][chunk][dim]: sums of parts of the vocabulary, where there are more than one
  int32_t parts;
  float* sums;             // vocab x dim: of the chunks so far, or null where there is one
  bool first, last;        // chunk
};

__device__ __forceinline__ int32_t live_slots(const Chunk& c) {
  const int64_t left = *c.count - c.slot0;
  return left < 0 ? 0 : left < c.size ? (int32_t)left : c.size;
}

// The exponent of two of a logit, less n.  In fp32 with both parts of the factor.
__device__ __forceinline__ float exponent(const LossArgs& a, float l, float n, float) {
  return fmaf(l, a.to_log2_low, fmaf(l, a.to_log2, -n));
}
__device__ __forceinline__ float exponent(const LossArgs& a, float l, float n, bf16_t) { return fmaf(l, a.to_log2, -n); }
// n of a largest logit (0 for one of -inf).
__device__ __forceinline__ float whole_exponent(const LossArgs& a, float top) {
  return top == -INFINITY ? 0.f : ceilf(top * a.to_log2);
}

// 2^(exponent - n) of a slab's n, between the first product and k_rescale.
// In 16 bits: no sign and seven bits of the exponent, which values up to 1 do
// without the rest of, leave nine of the fraction, so that this rounding (2^-10 at
// the most) hardly adds to that of the gradient in bf16 (2^-8): a row's sum of dw
// off by 1.03 of what one rounding gives, where two to bf16 give 1.4.  A NaN comes
// out as anything; its row's scale is NaN.
__device__ __forceinline__ uint32_t pack_exps(float lo, float hi) {
  return ((__float_as_uint(lo) + 0x2000u) >> 14 & 0xffffu) | ((__float_as_uint(hi) + 0x2000u) << 2 & 0xffff0000u);
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

// Whether the large tiles take a call's sizes: bf16 rows of whole 16-byte chunks
// that 31 bits address 256 of; and the rest of what they need of a call.
inline bool large_sizes(int dtype, int64_t tokens, int64_t vocab, int64_t dim) {
  return dtype == MUON_BF16 && dim % 8 == 0 && vocab < (1 << 21) && dim < (1 << 21) && tokens > 0;
}
int dx_parts(int64_t tokens, int64_t vocab, int64_t dim);

// The products, of one chunk.
int logits_product(const LossArgs& a, int dtype, Epilogue e, hipStream_t s);
int dx_product(const LossArgs& a, int dtype, hipStream_t s);
int dw_product(const LossArgs& a, int dtype, hipStream_t s);

}  // namespace vo
}  // namespace muon
