// How a sequence is cut for attention: the arithmetic that needs no GPU to be checked.
#pragma once

#include <hip/hip_runtime.h>

namespace lh {

constexpr int kAttentionStep = 128;          // tokens a workgroup takes at a time
// Tokens below which a sequence is not split further: up to 512 one launch does (64 sequences of up to
// 500 tokens 12.3 us against 19.1 with 256, 301 tokens 7.0 against 9.7)
constexpr int kAttentionMinChunk = 512;

// An entry of a block table as a page of the cache: itself, or 0 outside it.  A negative one is outside caches of over
// 2^32 pages, too.
__host__ __device__ inline int64_t page_or_first(int page, int64_t n_pages) {
  return (uint64_t)(int64_t)page < (uint64_t)n_pages ? page : 0;
}

// A sequence of len >= 0 tokens in at most `splits` parts of one size, a multiple of the step: the size and how many
// there are (one of an empty sequence).  Unsigned, since len and a part add up to more than 2^31.
struct EvenParts {
  unsigned size, count;
};
__host__ __device__ inline EvenParts even_parts(int len, int splits) {
  const unsigned n = (unsigned)len, s = (unsigned)splits;
  const unsigned each = ((n + s - 1) / s + kAttentionStep - 1) / kAttentionStep * kAttentionStep;
  const unsigned size = each > (unsigned)kAttentionMinChunk ? each : (unsigned)kAttentionMinChunk;
  const unsigned count = (n + size - 1) / size;
  return {size, count > 0 ? count : 1};
}

}  // namespace lh
