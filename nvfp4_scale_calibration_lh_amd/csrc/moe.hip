// A mixture-of-experts layer for a few tokens, on NVFP4 expert weights as the scale sweep leaves them:
//   y[t] = sum_j w[t, j] D_e (silu(G_e x[t]) * U_e x[t]),  e = ids[t, j],  silu(g) = g / (1 + exp(-g))
//
// Bound by reading the weights of every expert that is hit once (0.5625 bytes each).  Three kernels:
//   gate and up  a workgroup takes the n-th expert that the (up to 64) tokens hit, which it finds from the ids by itself, and some
//                of its channels; a wave has 8 gate rows and the 8 up rows that belong to them as one 16-row operand, so that
//                silu(g) * u needs no other wave.  h = w * silu(g) * u goes to the workspace as two (fp32: three) bf16 pieces.
//   down         the same walk over D_e with h for x, one fp32 row for each chosen expert of a token
//   sum          adds a token's rows in the order of its choices
// The rows (x or h) are staged in LDS and shared by the workgroup's waves; the weights stream through registers, each
// wave its own channels, or KS waves a share of k each where that is needed to fill the chip.
//
// Values of weights and rows are exact as in the products of few rows (see nvfp4_weights.hpp); h is held to 2^-17 of itself
// (its second piece rounds to 8 bits; fp32 rows: to 2^-24 by a third), so that nothing but y rounds to 8 bits.  Sums are fp32, in a fixed order.
#include "grouping.hpp"
#include "lh_internal.hpp"
#include "nvfp4_weights.hpp"

#include <algorithm>

namespace lh {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kU = 2;                        // chunks of k a wave takes at a time: whole 128-byte lines of a channel
constexpr int kD = 3;                        // steps whose weights are held or on their way
constexpr int kBudget = 52 * 1024;           // LDS of the rows, so that three workgroups fit a compute unit
constexpr int kComputeUnits = 256;

struct Args {
  const void* x;
  const float* x_scale;
  const int* ids;
  const float* weights;
  const uint8_t* code;
  const uint8_t* fp4;
  const float* amax;
  int* plan;
  __bf16* h;
  float* part;
  void* y;
  int64_t tokens;
  int hidden, inner, experts, topk, x_scales, slots, split;
  float gdiv;
};

struct Weights {
  v4u nib;
  v2u code;
};

// X: type of x.  DOWN: the second product, whose rows are h.  P: bf16 (E4M3: fp16) pieces of a row's element.  HP: pieces of h.
// CT: 16-row tiles of rows taken at a time; an expert with more rows has its weights read again.
template <int X, bool DOWN, int P, int HP, int CT>
__global__ __launch_bounds__(kThreads) void k_experts(const Args a) {
  constexpr bool EIGHT = X == kXE4m3 && !DOWN;
  constexpr int WX = EIGHT ? kXE4m3 : kXBf16;
  using frag = typename Frag<WX>::type;
  __shared__ uint64_t bits[64];
  __shared__ int rows[kTokens];
  __shared__ float share[kTokens];
  __shared__ int found;
  extern __shared__ char lds[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, quarter = lane >> 4;
  const int ks = wave % a.split, together = kWaves / a.split;      // tiles of the workgroup
  const int tiles = DOWN ? a.hidden / 16 : a.inner / 8, groups = (tiles + together - 1) / together;
  const int slot = blockIdx.x / (unsigned)groups, group = blockIdx.x % (unsigned)groups;
  const int tile = min(group * together + wave / a.split, tiles - 1);
  const bool own = group * together + wave / a.split < tiles && ks == 0;
  int* plan = a.plan + ((int64_t)blockIdx.y * a.slots + slot) * kPlan;
  int expert, n;
  if constexpr (DOWN) {
    expert = __builtin_amdgcn_readfirstlane(plan[0]);
    n = __builtin_amdgcn_readfirstlane(plan[1]);
    if (n == 0) return;
  } else {
    const int64_t first = (int64_t)blockIdx.y * kTokens;
    const int count = (int)min((int64_t)kTokens, a.tokens - first) * a.topk;
    const int* ids = a.ids + first * a.topk;
    if (threadIdx.x < 64) bits[threadIdx.x] = 0;
    __syncthreads();
    for (int c = threadIdx.x; c < count; c += kThreads) {
      const int id = ids[c];
      if (id >= 0 && id < a.experts) atomicOr((unsigned long long*)&bits[id >> 6], 1ull << (id & 63));
    }
    __syncthreads();
    expert = find_expert(bits, slot);
    if (expert < 0) {
      if (group == 0 && threadIdx.x == 0) plan[1] = 0;
      return;
    }
  }
  const int k_all = DOWN ? a.inner : a.hidden, full = k_all / kChunk, chunks = (k_all + kChunk - 1) / kChunk;
  const unsigned row_bytes = (unsigned)k_all / 2, row_codes = (unsigned)k_all / 16;
  const int64_t channel0 = (int64_t)expert * (DOWN ? a.hidden : 2 * a.inner) + (DOWN ? 16 : 8) * tile;
  const unsigned channel = DOWN ? i : (i < 8 ? i : a.inner + i - 8);
  const uint8_t* nib = a.fp4 + channel0 * row_bytes;
  const uint8_t* code = a.code + channel0 * row_codes;
  const unsigned w_at = channel * row_bytes + quarter * 16, c_at = channel * row_codes;
  const int steps = (full + kU - 1) / kU;
  const int mine = ks < steps ? (steps - ks + a.split - 1) / a.split : 0;      // steps of this wave
  Weights w[kD][kU];
  auto load_w = [&](Weights (&w)[kU], int m) __attribute__((always_inline)) {
    const int g = min(m, mine - 1) * a.split + ks;
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int c = min(g * kU + u, full - 1);
      w[u].nib = *(const v4u_a8*)(nib + (size_t)c * (kChunk / 2) + w_at);
      w[u].code = *(const v2u_a1*)(code + (size_t)c * (kChunk / 16) + c_at);
    }
  };
  const bool all_held = mine <= kD;           // then nothing is loaded in the loop
  if (mine > 0) {
#pragma unroll
    for (int d = 0; d < kD - 1; ++d) load_w(w[d], d);
    if (all_held) load_w(w[kD - 1], kD - 1);
  }
  if constexpr (DOWN) {
    if (threadIdx.x < kTokens) rows[threadIdx.x] = plan[4 + threadIdx.x];
  } else {
    if (wave == 0) {                          // a token's first choice of the expert stands for all of them
      const int64_t t = (int64_t)blockIdx.y * kTokens + lane;
      int at = -1;
      float sum = 0.0f;
      if (t < a.tokens)
        for (int j = 0; j < a.topk; ++j)
          if (a.ids[t * a.topk + j] == expert) {
            at = at < 0 ? j : at;
            sum += a.weights[t * a.topk + j];
          }
      const uint64_t hit = __ballot(at >= 0);
      const int rank = __popcll(hit & ((1ull << lane) - 1));
      if (at >= 0) {
        rows[rank] = (int)(t * a.topk) + at;
        share[rank] = sum;
      }
      if (group == 0) {
        if (lane == 0) plan[0] = expert, plan[1] = __popcll(hit);
        if (at >= 0) plan[4 + rank] = (int)(t * a.topk) + at;
      }
      if (lane == 0) found = __popcll(hit);
    }
  }
  __syncthreads();
  if constexpr (!DOWN) n = found;

  for (int r0 = 0; r0 < n; r0 += 16 * CT) {
    const int live = min(16 * CT, n - r0);
    // chunks of the rows that LDS holds at a time
    const int fit = kBudget / (live * P * (kChunk * 2) + live * P * 16 / kU + (EIGHT ? live * 4 : 0)) / kU * kU;
    const int panel = min(max(fit, kU), (chunks + kU - 1) / kU * kU);
    const unsigned stride = panel * (kChunk * 2) + 16;               // bytes of a row's piece
    float* scales = (float*)(lds + live * P * stride);               // [chunk][row]
    int begin = -panel;                                              // of the panel, in chunks
    auto next_panel = [&]() __attribute__((always_inline)) {
      begin += panel;
      __syncthreads();
      const int held = min(panel, chunks - begin), units = held * (kChunk / 8), total = live * units;
      for (int at0 = threadIdx.x; at0 < total; at0 += 4 * kThreads) {
        v4u got[4][DOWN ? P : (X == kXF32 ? 2 : 1)];
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = min(at0 + b * kThreads, total - 1), r = at / units, k = begin * kChunk + (at - r * units) * 8;
          const int k_in = min(k, k_all - 8);                        // rows are multiples of 16
          if constexpr (DOWN) {
#pragma unroll
            for (int p = 0; p < P; ++p) got[b][p] = *(const v4u*)(a.h + ((int64_t)rows[r0 + r] * P + p) * a.inner + k_in);
          } else {
            const int64_t from = (int64_t)(rows[r0 + r] / a.topk) * a.hidden + k_in;
            if constexpr (X == kXBf16) got[b][0] = *(const v4u*)((const __bf16*)a.x + from);
            if constexpr (X == kXF32) got[b][0] = *(const v4u*)((const float*)a.x + from), got[b][1] = *(const v4u*)((const float*)a.x + from + 4);
            if constexpr (X == kXE4m3) {
              const v2u v = *(const v2u*)((const uint8_t*)a.x + from);
              got[b][0] = v4u{v[0], v[1], 0, 0};
            }
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int at = at0 + b * kThreads, r = at / units, u = at - r * units;
          if (at >= total) continue;
          const bool in = begin * kChunk + u * 8 < k_all;
          v4u out[P];
          if constexpr (DOWN || X == kXBf16) {
#pragma unroll
            for (int p = 0; p < P; ++p) out[p] = got[b][p];
          } else if constexpr (X == kXE4m3) {
            h8 f;
            each<4>([&](auto pp) {
              constexpr int Q = decltype(pp)::value;
              const h2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)got[b][0][Q / 2], 1.0f, Q % 2 == 1);
              f[2 * Q] = v[0];
              f[2 * Q + 1] = v[1];
            });
            out[0] = __builtin_bit_cast(v4u, f);
          } else {
            __bf16 f[3][8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              __bf16 three[3];
              split<3>(__uint_as_float(got[b][e / 4][e % 4]), three);
              f[0][e] = three[0], f[1][e] = three[1], f[2][e] = three[2];
            }
            __builtin_memcpy(out, f, sizeof f);
          }
#pragma unroll
          for (int p = 0; p < P; ++p) *(v4u*)(lds + (unsigned)(p * live + r) * stride + u * 16) = in ? out[p] : v4u{0, 0, 0, 0};
        }
      }
      if constexpr (EIGHT)
        for (int at = threadIdx.x; at < held * live; at += kThreads) {
          const int c = at / live, r = at - c * live;
          scales[at] = a.x_scale[(int64_t)(rows[r0 + r] / a.topk) * a.x_scales + (a.x_scales > 1 ? begin + c : 0)];
        }
      __syncthreads();
    };
    v4f acc[CT];
    unsigned x_at[CT];
    int row_of[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      acc[c] = v4f{0, 0, 0, 0};
      row_of[c] = min(16 * c + i, live - 1);
      x_at[c] = row_of[c] * stride + quarter * 16;
    }
    // chunk c of k (of the panel's) with these weights
    auto multiply = [&](const Weights& w, int c) __attribute__((always_inline)) {
      v4f part[CT];
#pragma unroll
      for (int t = 0; t < CT; ++t) part[t] = v4f{0, 0, 0, 0};
      auto& sum = *(EIGHT ? &part : &acc);
      const v4u words = exchange<kXBf16>(w.nib);
      const v2u codes = lane_codes<kXBf16>(w.code, quarter);
      const char* from = lds + (unsigned)(c - begin) * (kChunk * 2);
      each<4>([&](auto st) __attribute__((always_inline)) {
        constexpr int S = decltype(st)::value;
        const auto fw = weights<WX, 2 * (S % 2)>(words[S], codes[S / 2]);
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
          for (int p = 0; p < P; ++p)
            sum[t] = mfma(fw, __builtin_bit_cast(frag, *(const v4u*)(from + x_at[t] + p * live * stride + S * 64)), sum[t]);
      });
      if constexpr (EIGHT) {
#pragma unroll
        for (int t = 0; t < CT; ++t) acc[t] += scales[(c - begin) * live + row_of[t]] * part[t];
      }
    };
    auto one = [&](int m, const Weights (&w)[kU]) __attribute__((always_inline)) {
      const int c = (m * a.split + ks) * kU;
      while (c >= begin + panel) next_panel();
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (c + u < full) multiply(w[u], c + u);
    };
    next_panel();
    if (r0 > 0 && mine > 0) {                  // the weights once more
#pragma unroll
      for (int d = 0; d < kD - 1; ++d) load_w(w[d], d);
      if (all_held) load_w(w[kD - 1], kD - 1);
    }
    if (all_held) {
      each<kD>([&](auto dd) __attribute__((always_inline)) {
        constexpr int d = decltype(dd)::value;
        if (d < mine) one(d, w[d]);
      });
    } else {
      for (int m = 0; m < mine; m += kD)
        each<kD>([&](auto dd) __attribute__((always_inline)) {
          constexpr int d = decltype(dd)::value;
          if (m + d < mine) {
            load_w(w[(d + kD - 1) % kD], m + d + kD - 1);
            one(m + d, w[d]);
          }
        });
    }
    while (begin + panel < chunks) next_panel();
    if (full < chunks && ks == 0) {            // the last, short chunk: 16 elements at a time
      const int left = k_all - full * kChunk, own_k = left - quarter * 32;
      const uint8_t* pn = nib + (size_t)full * (kChunk / 2) + w_at;
      const uint8_t* pq = code + (size_t)full * (kChunk / 16) + c_at;
      Weights t{};
      if (own_k >= 16) {
        const v2u v = *(const v2u*)pn;
        t.nib[0] = v[0], t.nib[1] = v[1];
      }
      if (own_k >= 32) {
        const v2u v = *(const v2u*)(pn + 8);
        t.nib[2] = v[0], t.nib[3] = v[1];
      }
#pragma unroll
      for (int b = 0; b < 7; ++b)
        if (16 * b < left) t.code[b / 4] |= (unsigned)pq[b] << (8 * (b % 4));
      multiply(t, full);
    }
    if (a.split > 1) {                         // the shares of k, in their order
      __syncthreads();
      float* red = (float*)lds;
#pragma unroll
      for (int t = 0; t < CT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[((wave * CT + t) * 4 + r) * 64 + lane] = acc[t][r];
      __syncthreads();
      if (ks == 0)
        for (int s = 1; s < a.split; ++s)
#pragma unroll
          for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[t][r] += red[(((wave + s) * CT + t) * 4 + r) * 64 + lane];
    }
    const float g = a.amax[expert] / a.gdiv;
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const int row = 16 * t + i;
      if constexpr (DOWN) {
        if (own && row < live) *(v4f*)(a.part + (int64_t)rows[r0 + row] * a.hidden + 16 * tile + 4 * quarter) = acc[t] * g;
      } else {                                 // a lane of the lower half has gate rows, 32 lanes on are their up rows
        __bf16 out[HP][4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float gate = acc[t][r] * g, up = __shfl_xor(gate, 32, 64);
          __bf16 pieces[HP];
          split<HP>(gate / (1.0f + expf(-gate)) * up * share[min(r0 + row, kTokens - 1)], pieces);
#pragma unroll
          for (int p = 0; p < HP; ++p) out[p][r] = pieces[p];
        }
        if (own && row < live && quarter < 2) {
#pragma unroll
          for (int p = 0; p < HP; ++p) {
            v2u v;
            __builtin_memcpy(&v, out[p], sizeof v);
            *(v2u*)(a.h + ((int64_t)rows[r0 + row] * HP + p) * a.inner + 8 * tile + 4 * quarter) = v;
          }
        }
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
  bool first = id >= 0 && id < a.experts;
  for (int j = 0; j + 1 < a.topk; ++j)
    if (j < lane && __builtin_amdgcn_readlane(id, j) == id) first = false;
  const uint64_t mask = __ballot(first);
  if (c >= a.hidden) return;
  v4f y = {0, 0, 0, 0};
  const float* from = a.part + t * a.topk * a.hidden + c;
  for (uint64_t m = mask; m;) {
    v4f v[4];
    bool have[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {              // independent loads
      have[k] = m != 0;
      const int j = have[k] ? __ffsll((unsigned long long)m) - 1 : __ffsll((unsigned long long)mask) - 1;
      v[k] = *(const v4f*)(from + (int64_t)j * a.hidden);
      m &= m - 1;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (have[k]) y += v[k];
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
  int64_t slots, chunks, plan, h, part, all;  // bytes; chunks of tokens
};
Layout layout(const MoeView& v) {
  Layout l{};
  auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
  l.slots = std::min(v.experts, std::min<int64_t>(v.tokens, kTokens) * v.topk);
  l.chunks = (v.tokens + kTokens - 1) / kTokens;
  l.plan = up(l.slots * l.chunks * kPlan * 4);
  l.h = up(v.tokens * v.topk * v.inner * (v.x_type == kXF32 ? 3 : 2) * 2);
  l.part = v.tokens * v.topk * v.hidden * 4;
  l.all = l.plan + l.h + l.part;
  return l;
}

template <int X, int CT>
hipError_t go(const MoeView& v, Args a, const Layout& l, hipStream_t stream) {
  constexpr int P = Frag<X>::pieces, HP = X == kXF32 ? 3 : 2;
  // waves that share k, so that some 2000 waves have work
  auto split = [&](int64_t tiles, int64_t k) {
    int s = 1;
    while (s < kWaves && l.slots * tiles * s < 8 * kComputeUnits && s * kChunk * kU < k) s *= 2;
    return s;
  };
  auto grid = [&](int64_t tiles) { return (tiles + kWaves / a.split - 1) / (kWaves / a.split) * l.slots; };
  constexpr size_t kLds = kBudget + 1024;
  a.code = v.gate_up_code;
  a.fp4 = v.gate_up_fp4;
  a.amax = v.gate_up_amax;
  a.split = split(v.inner / 8, v.hidden);
  int64_t n = grid(v.inner / 8);
  if (n >= (int64_t(1) << 32) / kThreads) return hipErrorInvalidConfiguration;
  hipError_t e = launch_kernel(k_experts<X, false, P, HP, CT>, dim3((unsigned)n, (unsigned)l.chunks), dim3(kThreads), kLds, stream, a);
  if (e != hipSuccess) return e;
  a.code = v.down_code;
  a.fp4 = v.down_fp4;
  a.amax = v.down_amax;
  a.split = split(v.hidden / 16, v.inner);
  n = grid(v.hidden / 16);
  if (n >= (int64_t(1) << 32) / kThreads) return hipErrorInvalidConfiguration;
  e = launch_kernel(k_experts<X == kXF32 ? kXF32 : kXBf16, true, HP, HP, CT>, dim3((unsigned)n, (unsigned)l.chunks), dim3(kThreads), kLds, stream, a);
  if (e != hipSuccess) return e;
  const int64_t blocks = (v.hidden / 4 + 255) / 256 * v.tokens;
  if (blocks >= (int64_t(1) << 24)) return hipErrorInvalidConfiguration;
  return launch_kernel(k_experts_sum<X != kXF32>, dim3((unsigned)blocks), dim3(256), 0, stream, a);
}

template <int X>
hipError_t go_x(const MoeView& v, const Args& a, const Layout& l, hipStream_t stream) {
  return v.tokens <= 16 || v.tokens * v.topk <= 4 * v.experts ? go<X, 1>(v, a, l, stream) : go<X, 2>(v, a, l, stream);
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
  a.plan = (int*)work;
  a.h = (__bf16*)((char*)work + l.plan);
  a.part = (float*)((char*)work + l.plan + l.h);
  a.y = v.y;
  a.tokens = v.tokens;
  a.hidden = (int)v.hidden;
  a.inner = (int)v.inner;
  a.experts = (int)v.experts;
  a.topk = (int)v.topk;
  a.x_scales = (int)v.x_scales;
  a.slots = (int)l.slots;
  a.gdiv = v.gdiv;
  if (v.x_type == kXBf16) return go_x<kXBf16>(v, a, l, stream);
  return v.x_type == kXF32 ? go_x<kXF32>(v, a, l, stream) : go_x<kXE4m3>(v, a, l, stream);
}

}  // namespace lh
