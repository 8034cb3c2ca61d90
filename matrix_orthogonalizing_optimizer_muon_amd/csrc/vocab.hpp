// What the vocabulary operators (vocab_*.hip) share: bounds of their arguments
// and the device helpers beyond those of the expert layer's.
#pragma once
#include "experts.hpp"

namespace muon {
namespace vo {

using namespace ex;

constexpr int64_t kMaxWidth = (int64_t(1) << 24) - 1;   // columns of a row
constexpr int kMaxTeacher = 256;                        // teacher entries of a row: four a lane

inline bool good_index(int bytes) { return bytes == 4 || bytes == 8; }

// Sizes that the operators have in common.
inline int check_sizes(int dtype, int index_bytes, int64_t tokens, int64_t vocab, int64_t dim) {
  if (!good_dtype(dtype)) return fail(MUON_EUNSUPPORTED, "unsupported dtype");
  if (!good_index(index_bytes)) return fail(MUON_EUNSUPPORTED, "indices must have 4 or 8 bytes");
  if (tokens < 0 || vocab < 1 || dim < 1) return fail(MUON_EINVAL, "tokens must be >= 0; vocab and dim >= 1");
  if (tokens > kMaxCount || vocab > kMaxCount) return fail(MUON_EUNSUPPORTED, "2^31 tokens or vocabulary entries or more");
  if (dim > kMaxWidth) return fail(MUON_EUNSUPPORTED, "rows of 2^24 columns or more");
  return MUON_OK;
}

inline int check_workspace(const void* workspace, uint64_t bytes, uint64_t need) {
  if (need && (!workspace || bytes < need))
    return fail(MUON_EINVAL, "workspace of " + std::to_string(need) + " bytes needed");
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 15)) return fail(MUON_EINVAL, "workspace must be 16-byte aligned");
  return MUON_OK;
}

// Pieces of a workspace, each on a border of 256 bytes from its start.
struct Pieces {
  uint64_t used = 0;
  uint64_t take(uint64_t bytes) {
    const uint64_t at = used;
    used += (bytes + 255) / 256 * 256;
    return at;
  }
};

// ------------------------------------------------------------------ device

// An index from a user's array: -1 where it names no entry of `n`.
template <class I>
__device__ __forceinline__ int32_t read_index(const I* p, int64_t i, int32_t n) {
  const I v = p[i];
  return v >= 0 && v < (I)n ? (int32_t)v : -1;
}

}  // namespace vo
}  // namespace muon
