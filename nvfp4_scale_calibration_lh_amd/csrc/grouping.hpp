// Rows that ask for one of several matrices, found by every workgroup for itself: the set of the matrices that up to 64 rows ask
// for as one bit each, 64 bits a lane, and its n-th member.  And fp32 numbers as bf16 pieces.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lh {
namespace {

constexpr int kTokens = 64;                  // rows of one pass over the weights: one a lane

// What a first kernel leaves of a slot for a second: the matrix, its number of rows, (adapters) its rank, one unused, and the rows (experts: choices,
// token * topk + j).
constexpr int kPlan = 4 + kTokens;

__device__ inline uint64_t lane_of(uint64_t v, int lane) {
  return (uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 | (unsigned)__builtin_amdgcn_readlane((int)v, lane);
}

// The slot-th of the experts whose bits are set, or -1.
__device__ inline int find_expert(const uint64_t* bits, int slot) {
  const int lane = threadIdx.x & 63;
  const uint64_t word = bits[lane];
  const int mine = __popcll(word);
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(upto, o, 64);
    if (lane >= o) upto += v;
  }
  const uint64_t there = __ballot(upto > slot);
  if (there == 0) return -1;
  const int owner = __ffsll((unsigned long long)there) - 1;
  uint64_t w = lane_of(word, owner);
  for (int k = slot - __builtin_amdgcn_readlane(upto - mine, owner); k > 0; --k) w &= w - 1;
  return 64 * owner + __ffsll((unsigned long long)w) - 1;
}

// Truncated pieces of 8 bits each, the last one rounded; an infinity or NaN is its first piece.
template <int P>
__device__ inline void split(float x, __bf16* out) {
#pragma unroll
  for (int p = 0; p + 1 < P; ++p) {
    const float hi = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    out[p] = __builtin_bit_cast(__bf16, (unsigned short)(__float_as_uint(x) >> 16));
    x = x == hi ? 0.0f : x - hi;
  }
  out[P - 1] = (__bf16)x;
}

}  // namespace
}  // namespace lh
