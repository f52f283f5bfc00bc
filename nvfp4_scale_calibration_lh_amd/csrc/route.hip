// The choice of experts: the topk largest of each token's logits, in descending order, ties to the lowest index, and
// their softmax weights, over all logits or over the chosen ones.
//
// A wave takes a token and holds its logits in registers as integers that order like the numbers (0: not to be
// chosen).  Each choice is the wave's largest, found by DPP steps, and its first place, found by ballots in the order of
// the indices.  32 tokens of 512 experts, ten chosen, 5.7 us: a launch and ten such searches, each waiting for the one before; 8192 tokens
// 10.5 us (17 MB: the searches of four waves a SIMD unit, not the loads).
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kWaves = 4;

struct Args {
  const void* logits;
  int* ids;
  float* weights;
  int64_t tokens;
  int experts, topk;
  float scale;
  bool renormalize;
};

__device__ inline unsigned key_of(float x) {
  if (!(x > -__builtin_inff())) return 0;    // masked, or NaN
  const unsigned u = __float_as_uint(x + 0.0f);      // the zeros are equal
  return (int)u < 0 ? ~u : u | 0x80000000u;
}
__device__ inline float value_of(unsigned k) { return __uint_as_float((int)k < 0 ? k & 0x7FFFFFFFu : ~k); }

__device__ inline unsigned wave_max(unsigned v) {
#define LH_STEP(ctrl) v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, false))
  LH_STEP(0x111);                            // row_shr 1, 2, 4, 8: the last lane of 16 has their largest
  LH_STEP(0x112);
  LH_STEP(0x114);
  LH_STEP(0x118);
  LH_STEP(0x142);                            // row_bcast 15, 31
  LH_STEP(0x143);
#undef LH_STEP
  return (unsigned)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

template <class T, int N>
__global__ __launch_bounds__(64 * kWaves) void k_route(const Args a) {
  const int lane = threadIdx.x & 63;
  const int64_t token = (int64_t)blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (token >= a.tokens) return;
  const T* row = (const T*)a.logits + token * a.experts;
  unsigned key[N];
  T x[N];
#pragma unroll
  for (int j = 0; j < N; ++j) x[j] = row[min(64 * j + lane, a.experts - 1)];
#pragma unroll
  for (int j = 0; j < N; ++j) key[j] = 64 * j + lane < a.experts ? key_of((float)x[j]) : 0;
  unsigned first = 0, mine = 0;
  int id = -1;
  float all = 0.0f;
  for (int t = 0; t < a.topk; ++t) {
    unsigned best = key[0];
#pragma unroll
    for (int j = 1; j < N; ++j) best = max(best, key[j]);
    best = wave_max(best);
    if (best == 0) break;                    // none is left
    if (t == 0) {
      first = best;
      if (!a.renormalize) {
        const float high = value_of(first);
#pragma unroll
        for (int j = 0; j < N; ++j) all += key[j] == 0 ? 0.0f : key[j] == first ? 1.0f : expf(value_of(key[j]) - high);
      }
    }
    bool open = true;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (!open) continue;
      const uint64_t at = __ballot(key[j] == best);
      if (at) {
        const int owner = __ffsll((unsigned long long)at) - 1;
        if (lane == owner) key[j] = 0;
        if (lane == t) mine = best, id = 64 * j + owner;
        open = false;
      }
    }
  }
  // an infinity that leads has weight 1 like everything equal to it
  const float e = mine == 0 ? 0.0f : mine == first ? 1.0f : expf(value_of(mine) - value_of(first));
  const float total = wave_sum(a.renormalize ? e : all);
  if (lane < a.topk) {
    a.ids[token * a.topk + lane] = id;
    a.weights[token * a.topk + lane] = mine == 0 ? 0.0f : e / total * a.scale;
  }
}

template <class T>
hipError_t go(const Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.tokens + kWaves - 1) / kWaves)), block(64 * kWaves);
  if (a.experts <= 64) return launch_kernel(k_route<T, 1>, grid, block, 0, stream, a);
  if (a.experts <= 128) return launch_kernel(k_route<T, 2>, grid, block, 0, stream, a);
  if (a.experts <= 256) return launch_kernel(k_route<T, 4>, grid, block, 0, stream, a);
  if (a.experts <= 512) return launch_kernel(k_route<T, 8>, grid, block, 0, stream, a);
  if (a.experts <= 1024) return launch_kernel(k_route<T, 16>, grid, block, 0, stream, a);
  if (a.experts <= 2048) return launch_kernel(k_route<T, 32>, grid, block, 0, stream, a);
  return launch_kernel(k_route<T, 64>, grid, block, 0, stream, a);
}

}  // namespace

hipError_t launch_route(const void* logits, bool bf16, int64_t tokens, int64_t experts, int64_t topk, bool renormalize,
                        float scale, int* ids, float* weights, hipStream_t stream) {
  const Args a{logits, ids, weights, tokens, (int)experts, (int)topk, scale, renormalize};
  return bf16 ? go<__bf16>(a, stream) : go<float>(a, stream);
}

}  // namespace lh
