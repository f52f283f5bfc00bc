// A mixture-of-experts layer for a few tokens, on NVFP4 expert weights as the scale sweep leaves them:
//   y[t] = sum_j w[t, j] D_e (silu(G_e x[t]) * U_e x[t]),  e = ids[t, j],  silu(g) = g / (1 + exp(-g))
//
// Bound by reading the weights of every expert that is hit once (0.5625 bytes each).  Ten experts of 1280x2560 and 2560x640 for one token 22 us
// (28 MB: three launches, each with its cold instructions, and the tail of the last weights); 32 tokens that hit 125 of 512 such experts 107 us (346 MB at 3.3 TB/s);
// 61 tokens over eight experts of 24576x4096 and 4096x12288 237 us (680 MB at 2.9 TB/s; 122 rows, whose products and staging
// share the wave slots with the loads).  Three kernels:
//   gate and up  the channels of all experts that (up to 64) tokens hit, in tiles, are shared out evenly over as many workgroups as
//                are resident; each finds the experts of its share and their rows from the ids by itself.  A wave has 8 gate rows
//                and the 8 up rows that belong to them as one 16-row operand, so that silu(g) * u needs no other wave.
//                h = silu(g) * u goes to the workspace in fp32.
//   down         the same walk over D_e with h for x, one fp32 row for each chosen expert of a token
//   sum          adds a token's rows times their weights, in the order of its choices
// The rows (x or h) are staged in LDS, as much of k as fits, and shared by the workgroup's waves; the weights stream through registers, each
// wave its own channels, or `split` waves a share of k each where that is needed to fill the chip.
//
// A weight's E2M1 value times its block's E4M3 scale has at most 6 significant bits in [2^-10, 2688], exact in fp16.  Rows are fp16
// with a factor for each 128 elements: E4M3 values exactly, with the scale they came with; bf16 and fp32 times the power of two that
// takes the largest of the 128 to [2^14, 2^15), fp32 in two pieces: bf16 exactly from 2^-31 of that largest element on and to within
// 2^-39 of it below, fp32 to 2^-23 of itself and 2^-39 of the largest.  h takes two pieces where y is fp32; where y is bf16, whose rounding is
// 2^-8, one (2^-11, eight times finer than that and than h in bf16 would be, at half the products).  Products are exact, sums fp32, in a fixed order.
#include "grouping.hpp"
#include "lh_internal.hpp"
#include "nvfp4_weights.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kLds = 80 * 1024;              // of a workgroup, so that two fit a compute unit
constexpr int kResident = 2 * 256;           // workgroups

constexpr int kXHalf = 3;                    // rows as k_rows leaves them

struct Args {
  const void* x;
  const float* x_scale;
  const int* ids;
  const float* weights;
  const uint8_t* code;
  const uint8_t* fp4;
  const float* amax;
  int* hits;                                 // experts hit by each 64 tokens
  int* plan;
  float* h;
  _Float16* half;                            // rows made ready for products, and their factors (see k_rows)
  float* factor;
  float* part;
  void* y;
  int64_t tokens;
  int hidden, inner, experts, topk, x_scales, slots;
  int split, each, rows;                     // waves that share k; chunks of a step of theirs; rows taken at a time
  int budget;                                // LDS of the rows
  int64_t all_rows;                          // that were made ready
  float gdiv;
};

// A step's weights of a lane: 32 nibbles of each chunk, and the 8 scales of its channel for the chunk of each four that is its quarter of
// the wave.  (Scales loaded chunk by chunk, 8 bytes a channel, made the reading of the weights take 69 us where this takes 43: 135 experts
// of 1280x2560, 249 MB, loads alone.)
template <int U>
struct Weights {
  v4u nib[U];
  v2u code[(U + 3) / 4];
};

__device__ inline unsigned row_max(unsigned v) {     // over 16 neighbouring lanes
#define LH_STEP(n) v = max(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + n, 0xf, 0xf, false))
  LH_STEP(8);
  LH_STEP(4);
  LH_STEP(2);
  LH_STEP(1);
#undef LH_STEP
  return v;
}

// Eight elements of a row, as loaded, in fp16 pieces, and their factor, which 16 neighbouring lanes with the 128 elements of a chunk share
// (E4M3 elements have one already).
template <int X, int P>
__device__ inline void make_ready(const v4u* got, bool in, h8* out, float& factor) {
  if constexpr (X == kXE4m3) {
    each<4>([&](auto pp) {
      constexpr int Q = decltype(pp)::value;
      const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)got[0][Q / 2], 1.0f, Q % 2 == 1);
      out[0][2 * Q] = v[0];
      out[0][2 * Q + 1] = v[1];
    });
  } else {
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      v[e] = X == kXF32 ? __uint_as_float(got[e / 4][e % 4]) : __uint_as_float(e % 2 ? got[0][e / 2] & 0xFFFF0000u : got[0][e / 2] << 16);
    unsigned most = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max(most, __float_as_uint(v[e]) & 0x7FFFFFFFu);
    const int top = min(max((int)(row_max(in ? most : 0) >> 23), 1), 254);       // beside an infinity, what is finite stays so
    factor = __builtin_ldexpf(1.0f, top - 141);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float y = __builtin_ldexpf(v[e], 141 - top);
      out[0][e] = (_Float16)y;
      if constexpr (P == 2) out[1][e] = y == (float)out[0][e] ? (_Float16)0.0f : (_Float16)(y - (float)out[0][e]);
    }
  }
}

// Rows of k elements made ready for the products once, where each would otherwise be made ready by many workgroups many times:
// half [piece][row][chunk][128], factor [row][chunk].  Chunks as in k_experts: the last one, if short, is the last 128 elements
// with 0 for those that the chunk before it has (k >= 128).
struct Rows {
  const void* x;
  const float* x_scale;
  _Float16* half;
  float* factor;
  int64_t rows;
  int x_scales, k_all;
};
template <int X, int P>
__global__ __launch_bounds__(256) void k_rows(const Rows a) {
  const int chunks = (a.k_all + kChunk - 1) / kChunk;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16, row = at / chunks;
  if (row >= a.rows) return;                  // 16 lanes together
  const int c = (int)(at - row * chunks), k = min(c * kChunk, a.k_all - kChunk) + (threadIdx.x & 15) * 8;
  const int64_t from = row * a.k_all + k;
  v4u got[2];
  float f;
  if constexpr (X == kXF32) {
    got[0] = *(const v4u*)((const float*)a.x + from), got[1] = *(const v4u*)((const float*)a.x + from + 4);
  } else if constexpr (X == kXBf16) {
    got[0] = *(const v4u*)((const __bf16*)a.x + from);
  } else {
    const v2u v = *(const v2u*)((const uint8_t*)a.x + from);
    got[0] = v4u{v[0], v[1], 0, 0};
    f = a.x_scale[row * a.x_scales + (a.x_scales > 1 ? c : 0)];
  }
  const bool in = k >= c * kChunk;
  h8 out[P];
  make_ready<X, P>(got, in, out, f);
#pragma unroll
  for (int p = 0; p < P; ++p) *(v4u*)(a.half + (p * a.rows * chunks + at) * kChunk + (threadIdx.x & 15) * 8) = in ? __builtin_bit_cast(v4u, out[p]) : v4u{0, 0, 0, 0};
  if ((threadIdx.x & 15) == 0) a.factor[at] = f;
}

// n / d for n < 2^21, by the reciprocal of d (a quotient is at least 0.5 / d away from the next whole number).
__device__ inline int quotient(int n, float reciprocal) { return (int)(((float)n + 0.5f) * reciprocal); }

// LDS accesses of this wave before and after stay in that order, for lanes that read what others have written.  A wave's LDS accesses are carried out in
// order, so this holds the compiler and costs no wait.
__device__ inline void wave_turn() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// g / (1 + exp(-g)) * u; the power of two from the exact product's two halves.  Where exp(-g) nears the end of fp32, 96 powers of two of it, beside
// which the 1 is nothing, are taken off the product instead: g from -76 down to -155.
__device__ inline float silu_times(float g, float u) {
  constexpr float kHigh = -1.4426950216293335f, kLow = -1.9259629911e-8f;       // -log2(e)
  const float t = g * kHigh, rest = fmaf(g, kHigh, -t) + g * kLow;
  const bool far = t > 110.0f;
  const float e = __builtin_amdgcn_exp2f(far ? t - 96.0f : t) * (fabsf(t) < 1e30f ? 1.0f + rest * 0.6931471824645996f : 1.0f);     // exp(-g)
  return __builtin_ldexpf(g / (far ? e : 1.0f + e) * u, far ? -96 : 0);
}

// X: type of the rows, in P pieces.  DOWN: the second product, whose rows are h.  MT: 16-row tiles taken at a time at most.  U: chunks of k
// a wave holds or has on their way; a chunk's registers are loaded again as soon as it has been multiplied.  U = 1: k is less than a chunk.
//
// Instructions are fetched from cold caches at each launch (0.6 us a KB was seen), which a call for one token feels: so the code is short, its
// loops are not unrolled further than the registers ask for, and there are no 64-bit divisions.
template <int X, int P, bool DOWN, int MT, int U>
__global__ __launch_bounds__(kThreads, 4) void k_experts(const Args a) {
  constexpr int kRows = DOWN ? 16 : 8;       // channels of a tile
  constexpr bool SMALL = U == 1, READY = X == kXHalf;
  constexpr int kBatch = READY ? 4 : 2;      // 16-byte units of rows that a thread loads together
  constexpr int kSets = (U + 3) / 4;
  __shared__ uint64_t bits[64];
  __shared__ int rows[kTokens], source[kTokens];                     // an expert's rows: choices, and rows of x
  __shared__ int found;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ __attribute__((aligned(16))) uint8_t codes[kWaves][kSets][16][32];
  short* chosen = (short*)(lds + a.budget);
  float* red = (float*)(lds + a.budget + (DOWN ? 0 : kTokens * 2 * a.topk));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, quarter = lane >> 4;
  const int shift = __builtin_ctz(a.split), ks = wave & (a.split - 1), mine = wave >> shift, together = kWaves >> shift;    // tiles of the workgroup
  const int tiles = (DOWN ? a.hidden : a.inner) / kRows, groups = (tiles + together - 1) >> (3 - shift);
  const int64_t token0 = (int64_t)blockIdx.y * kTokens;
  const int tokens = (int)min((int64_t)kTokens, a.tokens - token0);
  int hits;
  if constexpr (DOWN) {
    hits = a.hits[blockIdx.y];
  } else {
    const int* ids = a.ids + token0 * a.topk;
    if (threadIdx.x < 64) bits[threadIdx.x] = 0;
    __syncthreads();
#pragma clang loop unroll(disable)
    for (int c = threadIdx.x; c < tokens * a.topk; c += kThreads) {
      const int id = ids[c];
      const bool in = id >= 0 && id < a.experts;
      if (in) atomicOr((unsigned long long*)&bits[id >> 6], 1ull << (id & 63));
      chosen[c] = in ? (short)id : (short)-1;
    }
    __syncthreads();
    hits = __popcll(bits[lane]);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) hits += __shfl_xor(hits, o, 64);
    hits = __builtin_amdgcn_readfirstlane(hits);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.hits[blockIdx.y] = hits;
  }
  // the tiles of all experts, shared out evenly
  const unsigned all = (unsigned)hits * groups, per = all / gridDim.x, over = all - per * gridDim.x;
  unsigned at = per * blockIdx.x + min(blockIdx.x, over);
  const unsigned end = at + per + (blockIdx.x < over);

  const int k_all = DOWN ? a.inner : a.hidden, chunks = (k_all + kChunk - 1) / kChunk;
  const unsigned row_bytes = (unsigned)k_all / 2, row_codes = (unsigned)k_all / 16;
  // the last chunk, if short, is the last 128 elements, and those that the one before it has are 0 in the rows
  const int last_start = k_all - kChunk;
  auto start_of = [&](int c) { return SMALL ? 0 : min(c * kChunk, last_start); };
  const int turn = a.each * a.split, steps = (chunks + turn - 1) / turn;       // of every wave; past the last chunk it multiplies nothing
  const unsigned channel = DOWN ? i : (i < 8 ? i : a.inner + i - 8);
  const unsigned w_at = channel * row_bytes + quarter * 16, c_at = channel * row_codes;

  while (at < end) {                          // the share's part of one expert
    const int slot = at / (unsigned)groups, first = at - slot * groups, count = min(groups - first, (int)(end - at));
    at += count;
    int* plan = a.plan + ((int64_t)blockIdx.y * a.slots + slot) * kPlan;
    const int expert = DOWN ? __builtin_amdgcn_readfirstlane(plan[0]) : find_expert(bits, slot);
    const int64_t channel0 = (int64_t)expert * (DOWN ? a.hidden : 2 * a.inner);
    // where a step's weights of a wave are, tile `mine` of a group and its chunks of k; past the last step all lanes load one place
    // again, so that the loads in flight are the same number on every path
    struct Place {
      const uint8_t *nib, *code;
      int chunk;
      unsigned mask;
    };
    auto place_of = [&](int group, int step, bool any) __attribute__((always_inline)) {
      const int64_t c0 = channel0 + min((first + group) * together + mine, tiles - 1) * kRows;
      return Place{a.fp4 + c0 * row_bytes, a.code + c0 * row_codes, (step * a.split + ks) * a.each, any ? ~0u : 0u};
    };
    Weights<U> w;
    auto load_nib = [&](const Place& p, int u) __attribute__((always_inline)) {
      if constexpr (SMALL) {                  // 16 elements at a time
        const int left = k_all - quarter * 32;
        w.nib[0] = v4u{0, 0, 0, 0};
        if (left >= 16) {
          const v2u v = *(const v2u*)(p.nib + w_at);
          w.nib[0][0] = v[0], w.nib[0][1] = v[1];
        }
        if (left >= 32) {
          const v2u v = *(const v2u*)(p.nib + w_at + 8);
          w.nib[0][2] = v[0], w.nib[0][3] = v[1];
        }
      } else {
        w.nib[u] = *(const v4u_a8*)(p.nib + (unsigned)start_of(p.chunk + u) / 2 + (w_at & (u < a.each ? p.mask : 0u)));
      }
    };
    auto load_code = [&](const Place& p, int s) __attribute__((always_inline)) {
      if constexpr (SMALL) {
        w.code[0] = v2u{0, 0};
#pragma unroll
        for (int b = 0; b < 7; ++b)
          if (16 * b < k_all) w.code[0][b / 4] |= (unsigned)p.code[c_at + b] << (8 * (b % 4));
      } else {
        w.code[s] = *(const v2u_a1*)(p.code + (((unsigned)start_of(p.chunk + 4 * s + quarter) / 16 + c_at) & p.mask));
      }
    };
    auto load_all = [&]() __attribute__((always_inline)) {
      const Place p = place_of(0, 0, true);
#pragma unroll
      for (int s = 0; s < kSets; ++s) load_code(p, s);
#pragma unroll
      for (int u = 0; u < U; ++u) load_nib(p, u);
    };
    // few rows come soon enough behind the first weights; many are asked for first (32 tokens 113 us with the weights first)
    bool fresh = MT > 1;                      // no weights are on their way
    if constexpr (MT == 1) load_all();
    __syncthreads();                          // the rows before have been used
    int n;
    if constexpr (DOWN) {
      n = __builtin_amdgcn_readfirstlane(plan[1]);
      if (threadIdx.x < kTokens) rows[threadIdx.x] = source[threadIdx.x] = plan[4 + threadIdx.x];
    } else if (wave == 0) {                   // a token's first choice of the expert stands for all of them
      int pick = -1;
      if (lane < tokens)
#pragma clang loop unroll_count(2)
        for (int j = a.topk - 1; j >= 0; --j) pick = chosen[lane * a.topk + j] == expert ? j : pick;
      const uint64_t hit = __ballot(pick >= 0);
      const int rank = __popcll(hit & ((1ull << lane) - 1)), number = (int)(token0 + lane) * a.topk + pick;
      if (pick >= 0) rows[rank] = number, source[rank] = (int)token0 + lane;
      if (lane == 0) found = __popcll(hit);
      if (first == 0) {                       // for the second product
        if (lane == 0) plan[0] = expert, plan[1] = __popcll(hit);
        if (pick >= 0) plan[4 + rank] = number;
      }
    }
    __syncthreads();
    if constexpr (!DOWN) n = __builtin_amdgcn_readfirstlane(found);
    const float g = a.amax[expert] / a.gdiv;

#pragma clang loop unroll(disable)
    for (int r0 = 0; r0 < n; r0 += a.rows) {
      const int live = min(a.rows, n - r0);
      // chunks of the rows that LDS holds at a time
      const int fit = (a.budget - live * P * 16) / (live * turn * (P * kChunk * 2 + 4));
      const int panel = min(max(fit, 1), steps) * turn, panels = (chunks + panel - 1) / panel;
      const unsigned stride = panel * (kChunk * 2) + 16;             // bytes of a row's piece; 16 rows begin in different banks
      float* scales = (float*)(lds + live * P * stride);             // [row][chunk]
      int begin = -1;                                                // of what is held, in chunks
      fresh = fresh || r0 > 0;
      auto hold = [&](int from) __attribute__((always_inline)) {
        begin = from;
        __syncthreads();
        constexpr int kSame = READY ? P : 1;                         // rows made ready: their pieces like rows of their own
        const int units = min(panel, chunks - begin) * (kChunk / 8), total = kSame * live * units;
        const float reciprocal = 1.0f / (float)units;
#pragma clang loop unroll(disable)
        for (int done = 0; done < total; done += kBatch * kThreads) {
          const int at0 = done + threadIdx.x;
          v4u got[kBatch][X == kXF32 ? 2 : 1];
          float scale[kBatch];
          int r[kBatch], u[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int unit = min(at0 + b * kThreads, total - 16 + (int)(threadIdx.x & 15));    // 16 lanes have a chunk of a row
            r[b] = quotient(unit, reciprocal), u[b] = unit - r[b] * units;
            const int c = begin + u[b] / 16;
            if constexpr (READY) {
              const int p = P > 1 && r[b] >= live;
              const int64_t chunk = ((int64_t)source[r0 + r[b] - p * live] + (p ? a.all_rows : 0)) * chunks + c;
              got[b][0] = *(const v4u*)(a.half + chunk * kChunk + u[b] % 16 * 8);
              if (u[b] % 16 == 0 && !p) scale[b] = a.factor[chunk];
              continue;
            }
            const int k = min(start_of(c) + u[b] % 16 * 8, k_all - 8);
            const int64_t row = source[r0 + r[b]], from = row * k_all + k;
            if constexpr (X == kXF32) {
              const float* p = (DOWN ? (const float*)a.h : (const float*)a.x) + from;
              got[b][0] = *(const v4u*)p, got[b][1] = *(const v4u*)(p + 4);
            } else if constexpr (X == kXBf16) {
              got[b][0] = *(const v4u*)((const __bf16*)a.x + from);
            } else if constexpr (X == kXE4m3) {
              const v2u v = *(const v2u*)((const uint8_t*)a.x + from);
              got[b][0] = v4u{v[0], v[1], 0, 0};
              scale[b] = a.x_scale[row * a.x_scales + (a.x_scales > 1 ? c : 0)];
            }
          }
          if (fresh) load_all(), fresh = false;      // behind the first rows, which are needed first
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            if constexpr (READY) {
              if (at0 + b * kThreads >= total) continue;
              *(v4u*)(lds + (unsigned)r[b] * stride + u[b] * 16) = got[b][0];
              if (u[b] % 16 == 0 && r[b] < live) scales[r[b] * panel + u[b] / 16] = scale[b];
            } else {
              const int c = begin + u[b] / 16, k = start_of(c) + u[b] % 16 * 8;
              const bool in = k >= c * kChunk && k < k_all;          // otherwise it counts in another chunk
              h8 out[P];
              make_ready<X, P>(got[b], in, out, scale[b]);
              if (at0 + b * kThreads >= total) continue;
#pragma unroll
              for (int p = 0; p < P; ++p)
                *(v4u*)(lds + (unsigned)(p * live + r[b]) * stride + u[b] * 16) = in ? __builtin_bit_cast(v4u, out[p]) : v4u{0, 0, 0, 0};
              if (u[b] % 16 == 0) scales[r[b] * panel + u[b] / 16] = scale[b];
            }
          }
        }
        __syncthreads();
      };
      v4f acc[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[t] = v4f{0, 0, 0, 0};
      // the rows of this lane, as places in LDS
      int x_at[MT], s_at[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const int row = min(16 * t + i, live - 1);
        x_at[t] = row * stride + quarter * 64, s_at[t] = row * panel;
      }
      // chunk u of a step that begins `c` chunks into what is held
      auto multiply = [&](const v4u& nib, auto uu, int c) __attribute__((always_inline)) {
        constexpr int u = decltype(uu)::value;
        const h2 scale = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)*(const uint16_t*)&codes[wave][u / 4][i][8 * (u % 4) + 2 * quarter], 1.0f, false);
        h8 f[4];
        each<4>([&](auto st) __attribute__((always_inline)) {
          constexpr int S = decltype(st)::value;
          const h2 s = {scale[S / 2], scale[S / 2]};
          each<4>([&](auto pp) {
            constexpr int Q = decltype(pp)::value;
            const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(nib[S], 1.0f, Q) * s;
            f[S][2 * Q] = v[0];
            f[S][2 * Q + 1] = v[1];
          });
        });
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          if (MT > 1 && t > 0 && 16 * t >= live) break;
          const char* from = lds + (x_at[t] + c * (kChunk * 2)) + u * (kChunk * 2);
          v4f sum = {0, 0, 0, 0};
#pragma unroll
          for (int p = 0; p < P; ++p)
#pragma unroll
            for (int s = 0; s < 4; ++s) sum = mfma(f[s], __builtin_bit_cast(h8, *(const v4u*)(from + p * live * stride + s * 16)), sum);
          acc[t] += *(scales + (s_at[t] + c) + u) * sum;
        }
      };
      int group = 0, step = 0;
#pragma clang loop unroll(disable)
      for (int left = count * steps; left > 0; --left) {
        const int now = step, here = panels == 1 ? 0 : now * turn / panel * panel;
        if (here != begin) hold(here);        // the same step of all waves
        const bool last = ++step == steps;
        if (last) step = 0;
        const Place p = place_of(group + (last && left > 1), step, left > 1);
        wave_turn();                          // what was in codes has been read
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
          *(v2u*)&codes[wave][s][i][8 * quarter] = w.code[s];
          load_code(p, s);
        }
        wave_turn();
        const int c = (now * a.split + ks) * a.each;
        each<U>([&](auto uu) __attribute__((always_inline)) {
          constexpr int u = decltype(uu)::value;
          if (u < a.each && c + u < chunks) multiply(w.nib[u], uu, c - begin);
          load_nib(p, u);
        });
        if (!last) continue;
        const int tile = (first + group) * together + mine;
        const bool own = tile < tiles && ks == 0;
        ++group;
#pragma clang loop unroll(disable)
        for (int t = 0; 16 * t < live; ++t) {
          v4f v = acc[0];
#pragma unroll
          for (int m = 0; m + 1 < MT; ++m) acc[m] = acc[m + 1];
          acc[MT - 1] = v4f{0, 0, 0, 0};
          if (a.split > 1) {                  // the shares of k, in their order
            *(v4f*)(red + (wave * 64 + lane) * 4) = v;
            __syncthreads();
            if (ks == 0)
#pragma clang loop unroll(disable)
              for (int s = 1; s < a.split; ++s) v += *(const v4f*)(red + ((wave + s) * 64 + lane) * 4);
            __syncthreads();
          }
          const int row = 16 * t + i;
          v *= g;
          if constexpr (DOWN) {
            if (own && row < live) *(v4f*)(a.part + (int64_t)rows[r0 + row] * a.hidden + 16 * tile + 4 * quarter) = v;
          } else {                            // a lane of the lower half has gate rows, 32 lanes on are their up rows
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float up = __shfl_xor(v[r], 32, 64);
              v[r] = silu_times(v[r], up);
            }
            if (own && row < live && quarter < 2) *(v4f*)(a.h + (int64_t)rows[r0 + row] * a.inner + 8 * tile + 4 * quarter) = v;
          }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[t] = v4f{0, 0, 0, 0};
      }
    }
  }
}

// y[t] from the rows of its choices, four channels a thread; a choice that repeats an earlier one has no row of its own.
template <bool BF16>
__global__ __launch_bounds__(256) void k_experts_sum(const Args a) {
  const unsigned blocks = ((unsigned)a.hidden / 4 + 255) / 256;
  const int64_t t = blockIdx.x / blocks;
  const int c = 4 * ((int)(blockIdx.x % blocks) * 256 + (int)threadIdx.x);
  const int lane = threadIdx.x & 63;
  const int* ids = a.ids + t * a.topk;
  const int id = lane < a.topk ? ids[lane] : -1;
  const float given = lane < a.topk ? a.weights[t * a.topk + lane] : 0.0f;
  float weight = 0.0f;                        // the sum of those of its expert
  bool first = id >= 0 && id < a.experts;
#pragma clang loop unroll(disable)
  for (int j = 0; j < a.topk; ++j) {
    const bool same = __builtin_amdgcn_readlane(id, j) == id;
    weight += same ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(given), j)) : 0.0f;
    first = first && !(same && j < lane);
  }
  const uint64_t mask = __ballot(first);
  if (c >= a.hidden) return;
  v4f y = {0, 0, 0, 0};
  const float* from = a.part + t * a.topk * a.hidden + c;
  for (uint64_t m = mask; m;) {
    v4f v[4];
    float w[4];
    bool have[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {              // independent loads
      have[k] = m != 0;
      const int j = have[k] ? __ffsll((unsigned long long)m) - 1 : __ffsll((unsigned long long)mask) - 1;
      v[k] = *(const v4f*)(from + (int64_t)j * a.hidden);
      w[k] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), j));
      m &= m - 1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (have[k]) y += w[k] * v[k];
  }
  if constexpr (BF16) {
    __bf16 out[4] = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
    v2u v;
    __builtin_memcpy(&v, out, sizeof v);
    *(v2u*)((__bf16*)a.y + t * a.hidden + c) = v;
  } else {
    *(v4f*)((float*)a.y + t * a.hidden + c) = y;
  }
}

struct Layout {
  int64_t slots, chunks, hits, plan, h, half, factor, part, all;     // chunks of tokens; bytes
  bool many;                                  // rows are made ready first
};
Layout layout(const MoeView& v) {
  Layout l{};
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  l.slots = std::min(v.experts, std::min<int64_t>(v.tokens, kTokens) * v.topk);
  l.chunks = (v.tokens + kTokens - 1) / kTokens;
  l.hits = up(l.chunks * 4);
  l.plan = up(l.slots * l.chunks * kPlan * 4);
  l.h = up(v.tokens * v.topk * v.inner * 4);
  l.part = v.tokens * v.topk * v.hidden * 4;
  // From four rows an expert on: eight experts of 4096x12288 with two for each of 61 tokens 237 us, 280 without; 64 of 2560x1280 with eight for
  // each of 40 tokens 125 us, 138 without; with eight for each of 20 87 us, 84 without, and two of the eight wide ones for 17 158 and 157.
  l.many = v.tokens > 16 && v.tokens * v.topk > 4 * v.experts && v.hidden >= kChunk && v.inner >= kChunk;
  if (l.many) {
    const int64_t x = v.tokens * ((v.hidden + kChunk - 1) / kChunk), h = v.tokens * v.topk * ((v.inner + kChunk - 1) / kChunk);
    l.half = up(std::max(x, h) * kChunk * 2 * (v.x_type == kXF32 ? 2 : 1));
    l.factor = up(std::max(x, h) * 4);
  }
  l.all = l.hits + l.plan + l.h + l.half + l.factor + l.part;
  return l;
}

template <int X, int P, bool DOWN, int MT, int U>
hipError_t go(const MoeView& v, Args a, const Layout& l, hipStream_t stream) {
  const int64_t k = DOWN ? v.inner : v.hidden, tiles = DOWN ? v.hidden / 16 : v.inner / 8, chunks = (k + kChunk - 1) / kChunk;
  const int64_t lds = kLds - 1536 - kWaves * 512 * ((U + 3) / 4) - (DOWN ? 0 : kTokens * 2 * v.topk), most = std::min<int64_t>(v.tokens, 16);
  // rows whose chunks of a step LDS holds
  auto fits = [&](int64_t turn, bool shared) { return (lds - (shared ? kWaves * 1024 : 0)) / (P * (turn * kChunk * 2 + 16) + 4 * turn); };
  // Waves that share k: until some 1500 have work, or all that are resident where each would still take 6000 elements of k.  One token of
  // ten experts of 1280x2560 and 2560x640 22.2 us, 23.3 with 2048 or 3000 waves, 24.9 with 4096.  Eight experts, all resident and not: of
  // 4096x12288 with 61 tokens 237 and 247 us, with 20 161 and 166, with 12 146 and 149, 40 of fp32 261 and 274; of 4096x6144, 2048x24576 and
  // 12288x2048 with 61 141 and 145, 293 and 303, 148 and 157.
  auto more = [&](int64_t waves) { return waves < 1536 || (waves < kResident * kWaves && chunks / a.split >= 48); };
  a.split = 1;
  while (a.split < kWaves && 2 * a.split <= chunks && more(l.slots * tiles * a.split) && fits(2 * a.split, true) >= most) a.split *= 2;
  const bool shared = a.split > 1;
  const int64_t steps = (chunks + U * a.split - 1) / (U * a.split);
  a.each = (int)((chunks + steps * a.split - 1) / (steps * a.split));
  while (fits(a.each * a.split, shared) < most) --a.each;
  a.rows = (int)std::min<int64_t>(16 * MT, fits(a.each * a.split, shared) / 16 * 16);
  if (X == kXHalf) a.all_rows = DOWN ? v.tokens * v.topk : v.tokens;
  if (a.rows < 16) a.rows = (int)most;        // fewer than 16 tokens
  a.budget = (int)((lds - (shared ? kWaves * 1024 : 0)) / 16 * 16);
  const int64_t groups = (tiles + kWaves / a.split - 1) / (kWaves / a.split);
  if (l.slots * groups >= int64_t(1) << 31) return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)std::min<int64_t>(kResident, l.slots * groups), (unsigned)l.chunks);
  return launch_kernel(k_experts<X, P, DOWN, MT, U>, grid, dim3(kThreads), (size_t)(a.budget + (DOWN ? 0 : kTokens * 2 * v.topk) + (shared ? kWaves * 1024 : 0)), stream, a);
}

template <int X, int P, bool DOWN>
hipError_t go_rows(const MoeView& v, const Args& a, const Layout& l, hipStream_t stream) {
  if (l.many) {                               // experts have many rows each
    const int64_t rows = DOWN ? v.tokens * v.topk : v.tokens, k = DOWN ? v.inner : v.hidden, blocks = (rows * ((k + kChunk - 1) / kChunk) + 15) / 16;
    if (blocks >= int64_t(1) << 24) return hipErrorInvalidConfiguration;
    // (its own status: the thread's last error may be an older call's)
    const hipError_t e = launch_kernel(k_rows<X, P>, dim3((unsigned)blocks), dim3(256), 0, stream, Rows{DOWN ? a.h : a.x, a.x_scale, a.half, a.factor, rows, a.x_scales, (int)k});
    if (e != hipSuccess) return e;
    return go<kXHalf, P, DOWN, P == 1 ? 4 : 2, 4>(v, a, l, stream);
  }
  // Up to 16 tokens an expert has at most one tile of rows.  24 tokens over 512 experts of 2560x640 86 us, 100 in tiles of one; 16 tokens 69.5 either
  // way, 5 tokens over eight wide experts 116.8 us, 117.9 in two.
  if ((DOWN ? v.inner : v.hidden) < kChunk) return v.tokens <= 16 ? go<X, P, DOWN, 1, 1>(v, a, l, stream) : go<X, P, DOWN, 2, 1>(v, a, l, stream);
  return v.tokens <= 16 ? go<X, P, DOWN, 1, 4>(v, a, l, stream) : go<X, P, DOWN, 2, 4>(v, a, l, stream);
}

hipError_t go_all(const MoeView& v, Args a, const Layout& l, hipStream_t stream) {
  const int64_t blocks = (v.hidden / 4 + 255) / 256 * v.tokens;
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;
  a.code = v.gate_up_code;
  a.fp4 = v.gate_up_fp4;
  a.amax = v.gate_up_amax;
  hipError_t e = v.x_type == kXBf16 ? go_rows<kXBf16, 1, false>(v, a, l, stream)
                 : v.x_type == kXF32 ? go_rows<kXF32, 2, false>(v, a, l, stream) : go_rows<kXE4m3, 1, false>(v, a, l, stream);
  if (e != hipSuccess) return e;
  a.code = v.down_code;
  a.fp4 = v.down_fp4;
  a.amax = v.down_amax;
  e = v.x_type == kXF32 ? go_rows<kXF32, 2, true>(v, a, l, stream) : go_rows<kXF32, 1, true>(v, a, l, stream);
  if (e != hipSuccess) return e;
  return v.x_type == kXF32 ? launch_kernel(k_experts_sum<false>, dim3((unsigned)blocks), dim3(256), 0, stream, a)
                           : launch_kernel(k_experts_sum<true>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

}  // namespace

int64_t moe_workspace(const MoeView& v) { return layout(v).all; }

hipError_t launch_moe(const MoeView& v, void* work, hipStream_t stream) {
  const Layout l = layout(v);
  Args a{};
  a.x = v.x;
  a.x_scale = v.x_scale;
  a.ids = v.ids;
  a.weights = v.weights;
  a.hits = (int*)work;
  a.plan = (int*)((char*)work + l.hits);
  a.h = (float*)((char*)work + l.hits + l.plan);
  a.half = (_Float16*)((char*)work + l.hits + l.plan + l.h);
  a.factor = (float*)((char*)work + l.hits + l.plan + l.h + l.half);
  a.part = (float*)((char*)work + l.hits + l.plan + l.h + l.half + l.factor);
  a.y = v.y;
  a.tokens = v.tokens;
  a.hidden = (int)v.hidden;
  a.inner = (int)v.inner;
  a.experts = (int)v.experts;
  a.topk = (int)v.topk;
  a.x_scales = (int)v.x_scales;
  a.slots = (int)l.slots;
  a.gdiv = v.gdiv;
  return go_all(v, a, l, stream);
}

}  // namespace lh
