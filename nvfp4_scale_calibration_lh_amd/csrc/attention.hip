// Attention of one new token per sequence over the paged, quantised key-value cache:
//   o[h] = sum_t p_t v_t,  p = softmax over the sequence's tokens of scale * (q[h] . k_t),
// head h reading the keys and values of key-value head h / share.  An empty sequence gives 0.
//
// Bound by reading the cache once, so one workgroup serves up to 16 of the query heads that share a
// key-value head (the column side of a 16-wide matrix instruction), and a long sequence is split
// over workgroups whose partial (maximum, sum, output) a second kernel joins.  Within a workgroup
// the four waves take 32-token tiles in turn, each with a running maximum and sum of its own, and
// meet in LDS at the end.  NVFP4, head dimension 128: 4 sequences of 131001 tokens, 64 heads on 8,
// 115 us (604 MB, 5.2 TB/s) and 5 us for the join; 48 sequences of up to 8191 tokens, 32 heads on 8, 54
// us (234 MB, 4.3 TB/s) and 5 us; 301 tokens of one sequence in E4M3 6.6 us.  Whole calls of the two long cases: 59 and
// 120 us in NVFP4, 89 and 193 in E4M3; with fp32 q and o 64 and 127, 89 and 193, off the 64-bit result by 4.5e-7 and
// 6.4e-7 of it (products and sums in plain fp32: 8.8e-7 and 2.3e-6), with bf16 by its rounding, 1.7e-3.
//
// A tile is two matrix products without any exchange between lanes:
//   S^T = K Q^T   A = 16 tokens of K, B = the heads' q; the result's lane (head, quarter) holds
//                 tokens 4*quarter + r of each 16
//   O^T = V^T P^T B = P^T in exactly that lane layout, A = V^T with its tokens taken in the same order
// Every code is exact in fp16: E2M1 times its E4M3 block scale has at most 6 significant bits in
// [2^-10, 2688], E4M3 has 4 in [2^-9, 448]; the heads' global scales multiply scores and outputs.
// q is multiplied by the power of two that brings its head's largest element to [2^14, 2^15):
// bf16 then fits fp16 exactly down to 2^-31 of that element and to within 2^-39 of it below, fp32 is held as
// two fp16 pieces.
// p is made as 2^(s - m + 10) with m within 4 of the running maximum, so it stays under 2^14 and
// tokens 2^-24 below the largest keep all fp16 bits; for fp32 it is two pieces as well.  Sums,
// maxima and outputs are fp32.
#include "attention_cut.hpp"
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 32;                    // tokens a wave takes at a time
constexpr int kStep = kAttentionStep;        // tokens a workgroup takes at a time
static_assert(kStep == kTile * kWaves, "a step is a tile of every wave");
static_assert(2 * kStep <= (int64_t(1) << 31) - kMaxContext, "positions fit 32 bits a step past the last token");
constexpr int kHeads = 16;                   // query heads of one workgroup
constexpr int kMinChunk = kAttentionMinChunk;
constexpr int kResident = 1024;              // workgroups that the registers let run at a time
constexpr float kPBits = 10.0f;              // p = 2^(s - m + kPBits)

struct Args {
  const void* q;
  int64_t q_stride;
  const uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_amax, *v_amax;
  const int* table;
  const int* lengths;
  void* o;
  float* part;                               // [unit][pair][2 + D][16]: m, l, then the outputs
  float scale_log2;                          // softmax scale * log2(e)
  int heads, share, tiles, batch, width;
  int splits;                                // parts of each sequence; 0: all are cut to one length, by
  unsigned budget_mul, least_mul;            // 2^32 / budget rounded up; that of the budget for which `units` suffice
  int units;                                 // parts of all sequences, at most
  int64_t n_pages;
  unsigned page_size, page_mul, page_shift;  // n / page_size = n * page_mul >> page_shift, n < 2^31
};

template <int N, class F>
__device__ inline void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// B bytes as 32-bit words.
template <int B>
struct Bytes {
  unsigned w[B < 4 ? 1 : B / 4];
};
template <int B>
__device__ inline Bytes<B> load(const uint8_t* p) {
  Bytes<B> r;
  if constexpr (B == 1) {
    r.w[0] = *p;
  } else if constexpr (B == 2) {
    r.w[0] = *(const unsigned short*)p;
  } else if constexpr (B == 4) {
    r.w[0] = *(const unsigned*)p;
  } else if constexpr (B == 8) {
    const uint2 v = *(const uint2*)p;
    r.w[0] = v.x, r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < B / 16; ++i) {
      const uint4 v = ((const uint4*)p)[i];
      r.w[4 * i] = v.x, r.w[4 * i + 1] = v.y, r.w[4 * i + 2] = v.z, r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}

// Elements 2P and 2P + 1 of a run of codes.
template <bool FOUR, int P, int B>
__device__ inline h2 pair_of(const Bytes<B>& b) {
  if constexpr (FOUR)
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(b.w[P / 4], 1.0f, P % 4);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b.w[P / 2], 1.0f, P % 2 == 1);
}

// The E4M3 block scale in byte I, in both halves.
template <int I, int B>
__device__ inline h2 scale_of(const Bytes<B>& b) {
  const h2 s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)b.w[I / 4], 1.0f, (I & 2) != 0);
  return h2{s[I & 1], s[I & 1]};
}

__device__ inline int length_of(const Args& a, int64_t b) {
  const int64_t most = (int64_t)a.width * a.page_size;
  const int len = a.lengths[b];
  return len < 0 ? 0 : (len > most ? (int)most : len);
}

// Inclusive sum over the lanes up to this one: within rows of 16, then the rows before.
__device__ inline unsigned scan(unsigned v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);     // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);     // lane 15 of rows 0, 2 to rows 1, 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);     // lane 31 to rows 2, 3
  return v;
}

// One unit of work: the tokens [from, to) of sequence b, one of its `splits` parts, whose first is unit `base`.
struct Unit {
  int b, len, from, to, splits, base;
};

// The unit-th part over all sequences in order, or sequence b if b >= 0; splits is 0 past the last part.
// Up to 64 sequences are cut to parts of one length, from the tokens of all of them, so that uneven
// sequences keep the compute units evenly busy (48 of up to 8191 tokens in NVFP4 59 us, in E4M3 89, against
// 68 and 100 where each was cut into as many parts as the others); every wave finds its part by a
// scan over its lanes.  More sequences get the same number of parts each: they even out, and a scan
// would be several dependent loads (300 sequences of one head 57 us with one, 53 without).
__device__ inline Unit find_unit(const Args& a, int unit, int b) {
  if (a.splits == 1) {                                  // without the divisions below
    const int seq = b >= 0 ? b : unit, len = length_of(a, seq);
    return {seq, len, 0, len, 1, seq};
  }
  if (a.splits > 0) {
    const int seq = b >= 0 ? b : unit / a.splits, base = seq * a.splits, len = length_of(a, seq);
    const EvenParts parts = even_parts(len, a.splits);
    const int splits = (int)parts.count, at = unit - base;
    if (b < 0 && at >= splits) return {0, 0, 0, 0, 0, 0};
    const int64_t from = (int64_t)at * parts.size, to = from + parts.size;
    return {seq, len, (int)min(from, (int64_t)len), (int)min(to, (int64_t)len), splits, base};
  }
  const int lane = threadIdx.x & 63;
  const int len = lane < a.batch ? length_of(a, lane) : 0;
  const unsigned steps = ((unsigned)len + kStep - 1) / kStep;
  const unsigned all = (unsigned)__builtin_amdgcn_readlane((int)scan(steps), 63);
  unsigned most, n, upto;
  auto cut = [&](unsigned budget_mul) __attribute__((always_inline)) {
    // steps of a part: all / budget rounded up (or one more), so that the parts are at most budget and one a sequence
    most = max(__umulhi(all - 1, budget_mul) + 1, (unsigned)(kMinChunk / kStep));
    // steps / most rounded up: the quotient is at most budget < 2^12, so the product is less than one away from it
    n = (unsigned)((float)steps * __builtin_amdgcn_rcpf((float)most));
    const int left = (int)(steps - n * most);
    n = n + (left > 0) + (left > 0 && (unsigned)left > most);
    n = lane < a.batch ? max(n, 1u) : 0;
    upto = scan(n);
  };
  cut(a.budget_mul);
  if (__builtin_amdgcn_readlane((int)upto, 63) > a.units) cut(a.least_mul);
  if (b < 0 && unit >= __builtin_amdgcn_readlane((int)upto, 63)) return {0, 0, 0, 0, 0, 0};
  const int owner = b >= 0 ? b : __ffsll((unsigned long long)__ballot((unsigned)unit < upto)) - 1;
  const int seq_len = __builtin_amdgcn_readlane(len, owner), splits = __builtin_amdgcn_readlane((int)n, owner);
  const int base = __builtin_amdgcn_readlane((int)upto, owner) - splits;
  const int64_t from = (int64_t)(unit - base) * most * kStep, to = from + (int64_t)most * kStep;
  return {owner, seq_len, (int)min(from, (int64_t)seq_len), (int)min(to, (int64_t)seq_len), splits, base};
}

// Where the 16 tokens of a group lie: in one page (16 | page_size), in at most two (page_size > 16), the
// page numbers being scalar loads, or anywhere, with a lookup for each token (pages of 24: 34 us by
// lookups of two pages against 40 by one for each token).
enum { kOnePage = 0, kTwoPages = 1, kAnyPages = 2 };

// FOUR: NVFP4 codes, otherwise E4M3.  F32: fp32 q and o.  128 registers leave room for four waves of a SIMD.
template <bool FOUR, int D, bool F32, int PAGES>
__global__ __launch_bounds__(kThreads, D <= 128 && !F32 ? 4 : 1) void k_attention(const Args a) {
  constexpr int kSteps = D / 32;                        // 32-deep matrix instructions of q . k
  constexpr int kOut = D / 16;                          // 16-row tiles of the output
  constexpr int kPieces = F32 ? 2 : 1;
  constexpr int kRow = FOUR ? D / 2 : D;                // code bytes of one token
  constexpr int kKB = kRow / 4, kVB = kRow / 16;        // code bytes a lane takes of a K / V token
  constexpr int kKS = D / 64;                           // K block scales of a lane
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, quarter = lane >> 4;

  // heads fastest: a compute die has the same share of every sequence
  const unsigned pairs = (unsigned)(a.heads * a.tiles), unit = blockIdx.x / pairs, pair = blockIdx.x % pairs;
  const int kvh = pair % a.heads, tile = pair / a.heads;
  const Unit rg = find_unit(a, (int)unit, -1);
  if (rg.splits == 0) return;                           // an empty sequence has one part, which writes zeros
  const int64_t b = rg.b;
  const int len = rg.len;

  const int head = tile * kHeads + i;                   // of this lane's column, within the share
  const bool live_head = head < a.share;
  const int64_t qh = (int64_t)kvh * a.share + head;

  // q, its power of two, and the factor of the scores
  h8 qf[kSteps][kPieces];
  float factor;
  {
    float x[D / 4];
    if constexpr (F32) {
      const uint4* p = (const uint4*)((const float*)a.q + b * a.q_stride + qh * D + quarter * (D / 4));
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        const uint4 v = live_head ? p[j] : uint4{0, 0, 0, 0};
        x[4 * j] = __uint_as_float(v.x), x[4 * j + 1] = __uint_as_float(v.y);
        x[4 * j + 2] = __uint_as_float(v.z), x[4 * j + 3] = __uint_as_float(v.w);
      }
    } else {
      const uint4* p = (const uint4*)((const unsigned short*)a.q + b * a.q_stride + qh * D + quarter * (D / 4));
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        const uint4 v = live_head ? p[j] : uint4{0, 0, 0, 0};
        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[8 * j + 2 * k] = __uint_as_float(w[k] << 16);
          x[8 * j + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
    }
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < D / 4; ++j) top = fmaxf(top, fabsf(x[j]));
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const int e = min(14 - (int)((__float_as_uint(top) >> 23) & 255u) + 127, 126);
    const float up = copysignf(ldexpf(1.0f, e), a.scale_log2);        // so that the factor is not negative
    factor = fabsf(a.scale_log2) * cache_unit(a.k_amax[kvh], FOUR) * ldexpf(1.0f, -e);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = x[8 * s + k] * up;
        qf[s][0][k] = (_Float16)f;
        if constexpr (F32) qf[s][1][k] = (_Float16)(f - (float)qf[s][0][k]);
      }
  }

  const int* table = a.table + b * a.width;
  const int last = len - 1;
  // The first row of a page in the codes, in tokens of one head; a page outside the cache is page 0.
  auto page_base = [&](int page) {
    return (page_or_first(page, a.n_pages) * a.heads + kvh) * a.page_size;
  };
  auto divide = [&](unsigned n) { return (unsigned)(((uint64_t)n * a.page_mul) >> a.page_shift); };
  // 16 tokens from t16 on: the row of the first, how many follow it up to the sequence's last token, and
  // with two pages the first token of the second and how much further its row lies.  Tokens past the
  // last repeat it, so every load is of the sequence.
  struct Group {
    int64_t row, jump;
    int rest, cut;
  };
  auto group_at = [&](int t16) {
    const int first = __builtin_amdgcn_readfirstlane(min(t16, last & ~15));
    const unsigned p = divide((unsigned)first);
    const unsigned in = first - p * a.page_size;
    Group g{page_base(table[p]) + in, 0, last - first, 16};
    if constexpr (PAGES == kTwoPages) {
      g.cut = min((int)(a.page_size - in), 16);
      const bool second = g.cut <= min(g.rest, 15);      // the sequence has tokens there
      g.jump = page_base(table[second ? p + 1 : p]) - g.row - g.cut;
    }
    return g;
  };
  auto row_at = [&](int t) {
    const int tc = min(t, last);
    const unsigned p = divide((unsigned)tc);
    return page_base(table[p]) + (unsigned)(tc - (int)(p * a.page_size));
  };
  // Pointer to element `each` * row + `in` of a token, the j-th of group g at t16.
  auto find = [&](const uint8_t* base, const Group& g, int t16, int j, int each, int in) {
    if constexpr (PAGES == kAnyPages) {
      return base + row_at(t16 + j) * each + in;
    } else {
      const unsigned at = min(j, g.rest);
      const uint8_t* p = base + g.row * each;
      if constexpr (PAGES == kTwoPages) p += (int)at >= g.cut ? g.jump * each : 0;
      return p + (at * each + in);
    }
  };

  Bytes<kKB> kc[2];
  Bytes<kKS> ks[2];
  Bytes<kVB> vc[8];
  unsigned vs[8];
  auto load_k = [&](const Group* g, int t0) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      kc[x] = load<kKB>(find(a.k, g[x], t0 + 16 * x, i, kRow, quarter * kKB));
      if constexpr (FOUR) ks[x] = load<kKS>(find(a.k_scale, g[x], t0 + 16 * x, i, D / 16, quarter * kKS));
    }
  };
  auto load_v = [&](const Group* g, int t0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int x = e / 4, j = 4 * quarter + e % 4;
      vc[e] = load<kVB>(find(a.v, g[x], t0 + 16 * x, j, kRow, i * kVB));
      if constexpr (FOUR) vs[e] = *find(a.v_scale, g[x], t0 + 16 * x, j, D / 16, i * kOut / 16);
    }
  };

  v4f acc[kOut];
#pragma unroll
  for (int n = 0; n < kOut; ++n) acc[n] = v4f{0, 0, 0, 0};
  // m is within 4 of the running maximum (0 before the first tile); the sum of p is a product with ones,
  // which also adds up the quarters' tokens
  float m = -INFINITY;
  v4f total = {0, 0, 0, 0};
  h8 ones;
#pragma unroll
  for (int e = 0; e < 8; ++e) ones[e] = (_Float16)1.0f;

  int t0 = rg.from + wave * kTile;
  Group g[2];
  if (t0 < rg.to) {
    if constexpr (PAGES != kAnyPages) g[0] = group_at(t0), g[1] = group_at(t0 + 16);
    load_k(g, t0);
    load_v(g, t0);
  }
  for (; t0 < rg.to; t0 += kStep) {
    // The next tile's loads are not conditional, so that the waits for this one's count exactly; past
    // the end they repeat the sequence's last token.
    const int next = t0 + kStep;
    Group gn[2];
    if constexpr (PAGES != kAnyPages) gn[0] = group_at(next), gn[1] = group_at(next + 16);
    // scores
    v4f s[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      each<kSteps>([&](auto st) {
        constexpr int S = decltype(st)::value;
        h8 kf;
        each<4>([&](auto pp) {
          constexpr int P = decltype(pp)::value;
          h2 v = pair_of<FOUR, 4 * S + P>(kc[x]);
          if constexpr (FOUR) v *= scale_of<S / 2>(ks[x]);
          kf[2 * P] = v[0];
          kf[2 * P + 1] = v[1];
        });
#pragma unroll
        for (int pc = 0; pc < kPieces; ++pc)
          s[x] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[S][pc], s[x], 0, 0, 0);
      });
    }
    load_k(gn, next);
    // p, with the running maximum moved only when a score passes it by more than 4; a repeated token
    // has the last one's score, so it does not disturb the maximum
    float tmax = s[0][0];
#pragma unroll
    for (int e = 1; e < 8; ++e) tmax = fmaxf(tmax, s[e / 4][e % 4]);
    tmax *= factor;
    if (__any(tmax > m + 4.0f)) {
      tmax = fmaxf(tmax, __shfl_xor(tmax, 16, 64));
      tmax = fmaxf(tmax, __shfl_xor(tmax, 32, 64));
      const float mn = fmaxf(m, tmax);
      const float alpha = __builtin_amdgcn_exp2f(m - mn);         // 0 at the first tile
      m = mn;
      total *= alpha;
#pragma unroll
      for (int n = 0; n < kOut; ++n) acc[n] *= alpha;
    }
    const float shift = kPBits - m;
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(fmaf(s[e / 4][e % 4], factor, shift));
    if (t0 + kTile > rg.to) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = t0 + 16 * (e / 4) + 4 * quarter + e % 4 < rg.to ? p[e] : 0.0f;
    }
    h8 pf[kPieces];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pf[0][e] = (_Float16)p[e];
      if constexpr (F32) pf[1][e] = (_Float16)(p[e] - (float)pf[0][e]);
    }
#pragma unroll
    for (int pc = 0; pc < kPieces; ++pc) total = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, pf[pc], total, 0, 0, 0);
    // output
    each<kOut / 2>([&](auto nn) {
      constexpr int P = decltype(nn)::value;
      h8 lo, hi;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h2 v = pair_of<FOUR, P>(vc[e]);
        if constexpr (FOUR) {
          const h2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)vs[e], 1.0f, false);
          v *= h2{sc[0], sc[0]};
        }
        lo[e] = v[0];
        hi[e] = v[1];
      }
#pragma unroll
      for (int pc = 0; pc < kPieces; ++pc) {
        acc[2 * P] = __builtin_amdgcn_mfma_f32_16x16x32_f16(lo, pf[pc], acc[2 * P], 0, 0, 0);
        acc[2 * P + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(hi, pf[pc], acc[2 * P + 1], 0, 0, 0);
      }
    });
    load_v(gn, next);
    g[0] = gn[0], g[1] = gn[1];
  }
  float l = total[0];

  // the four waves: a common maximum, then sums of the outputs in two halving steps
  __shared__ float sh_m[kWaves][kHeads], sh_l[kWaves][kHeads];
  __shared__ float sh_o[kWaves / 2][kHeads][D + 4];
  if (quarter == 0) sh_m[wave][i] = m;
  __syncthreads();
  float top = sh_m[0][i];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) top = fmaxf(top, sh_m[w][i]);
  const float alpha = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - top);
  if (quarter == 0) sh_l[wave][i] = l * alpha;
#pragma unroll
  for (int n = 0; n < kOut; ++n) acc[n] *= alpha;
  auto at = [&](int w, int n, int r) -> float& { return sh_o[w][i][(4 * quarter + r) * kOut + n]; };
#pragma unroll
  for (int half = kWaves / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int n = 0; n < kOut; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) at(wave - half, n, r) = acc[n][r];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int n = 0; n < kOut; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[n][r] += at(wave, n, r);
    }
    __syncthreads();
  }
  if (wave != 0 || !live_head) return;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) l += sh_l[w][i];
  const int d0 = 4 * quarter * kOut;                    // this lane's D / 4 outputs are contiguous
  if (rg.splits <= 1) {
    const float f = l > 0.0f ? cache_unit(a.v_amax[kvh], FOUR) / l : 0.0f;
    const int64_t to = (b * a.heads * a.share + qh) * D + d0;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int n = 0; n < kOut; n += 4) {
        const v4f v = {acc[n][r] * f, acc[n + 1][r] * f, acc[n + 2][r] * f, acc[n + 3][r] * f};
        if constexpr (F32) {
          *(v4f*)((float*)a.o + to + r * kOut + n) = v;
        } else {
          const v2bf x = __builtin_convertvector((v2f){v[0], v[1]}, v2bf), y = __builtin_convertvector((v2f){v[2], v[3]}, v2bf);
          *(uint2*)((unsigned short*)a.o + to + r * kOut + n) = uint2{__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y)};
        }
      }
    return;
  }
  float* part = a.part + (int64_t)blockIdx.x * (kHeads * (D + 2));
  if (quarter == 0) part[i] = top, part[kHeads + i] = l;
  float* out = part + 2 * kHeads + i * D + d0;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int n = 0; n < kOut; n += 4) *(v4f*)(out + r * kOut + n) = v4f{acc[n][r], acc[n + 1][r], acc[n + 2][r], acc[n + 3][r]};
}

// Joins the partial results of a sequence's splits; one workgroup a query head.  The splits' maxima
// and sums are turned into weights in LDS, then D / 4 threads take four elements each and the
// workgroup's kRuns such sets take the splits in turn, so that many loads are in flight; sums go in
// a fixed order.  Sequences with one split were finished by it.
template <bool FOUR, int D, bool F32>
__global__ __launch_bounds__(kThreads) void k_attention_join(const Args a) {
  constexpr int kPart = kHeads * (D + 2), kRuns = kThreads / (D / 4);
  __shared__ float weight[2 * kResident];               // a sequence has at most `budget` parts
  __shared__ float red[2][kWaves];
  __shared__ v4f sum[kRuns][D / 4];
  const int64_t b = blockIdx.x / (unsigned)(a.heads * a.share);
  const int h = blockIdx.x % (unsigned)(a.heads * a.share), kvh = h / a.share, head = h % a.share;
  const Unit rg = find_unit(a, 0, (int)b);
  const int splits = rg.splits;
  if (splits <= 1) return;
  const int tile = head / kHeads, i = head % kHeads, pairs = a.heads * a.tiles;
  const float* part = a.part + ((int64_t)rg.base * pairs + tile * a.heads + kvh) * kPart + i;
  const int64_t next = (int64_t)pairs * kPart;          // from one part of the sequence to the next
  float top = -INFINITY;
  for (int s = threadIdx.x; s < splits; s += kThreads) top = fmaxf(top, weight[s] = part[s * next]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((threadIdx.x & 63) == 0) red[0][threadIdx.x >> 6] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, red[0][w]);
  float l = 0.0f;
  for (int s = threadIdx.x; s < splits; s += kThreads) {        // this thread's own entries
    const float f = weight[s] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(weight[s] - top);
    weight[s] = f;
    l = fmaf(part[s * next + kHeads], f, l);
  }
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) l += __shfl_xor(l, o, 64);
  if ((threadIdx.x & 63) == 0) red[1][threadIdx.x >> 6] = l;
  __syncthreads();
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) l += red[1][w];
  const int run = threadIdx.x / (D / 4), d4 = threadIdx.x % (D / 4);
  const v4f* out = (const v4f*)(part - i + 2 * kHeads + i * D) + d4;
  v4f o = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = run; s < splits; s += kRuns) o += weight[s] * out[s * (next / 4)];
  sum[run][d4] = o;
  __syncthreads();
  if (run != 0) return;
#pragma unroll
  for (int r = 1; r < kRuns; ++r) o += sum[r][d4];
  o *= l > 0.0f ? cache_unit(a.v_amax[kvh], FOUR) / l : 0.0f;
  const int64_t to = (int64_t)blockIdx.x * D + 4 * d4;
  if constexpr (F32) {
    *(v4f*)((float*)a.o + to) = o;
  } else {
    const v2bf x = __builtin_convertvector((v2f){o[0], o[1]}, v2bf), y = __builtin_convertvector((v2f){o[2], o[3]}, v2bf);
    *(uint2*)((unsigned short*)a.o + to) = uint2{__builtin_bit_cast(unsigned, x), __builtin_bit_cast(unsigned, y)};
  }
}

// How the sequences are cut: `splits` parts each, or 0 and all to one length, into `budget` parts and up to
// one more a sequence, or if those are more than `units`, into `least` and one a sequence.  A part that is alone on its sequence is finished by its workgroup, so sequences that
// fill the card are not cut (128 of up to 3000 tokens on 8 heads 56 us, cut 68).  Few long sequences are
// cut to what is resident at a time, more of them to half of that, so that the last parts end together (7 of up
// to 60000 tokens 61 us against 65, 48 of up to 8191 59 against 66).
struct Cut {
  int splits, budget, least;
  int64_t units;                             // parts for each head, at most
};
Cut cut_for(const CacheView& c, int64_t batch, int64_t share, int64_t width) {
  const int64_t pairs = c.heads * ((share + kHeads - 1) / kHeads), most = std::max<int64_t>((width * c.page_size + kMinChunk - 1) / kMinChunk, 1);
  if (batch > 64 || batch * pairs >= kResident || most == 1) {
    const int64_t all = std::max<int64_t>(batch * pairs, 1), splits = std::min((kResident + all - 1) / all, most);
    return {(int)splits, 0, 0, batch * splits};
  }
  const int64_t one = kResident / pairs;
  if (batch * 8 <= one) return {0, (int)one, (int)(one - batch), std::min(one, batch * most)};
  return {0, (int)(2 * one), (int)(2 * one), std::min(2 * one + batch, batch * most)};
}

template <bool FOUR, int D, bool F32>
hipError_t launch_typed(const Args& a, unsigned grid, unsigned join, hipStream_t stream) {
  const auto kernel = a.page_size % 16 == 0 ? k_attention<FOUR, D, F32, kOnePage>
                      : a.page_size > 16    ? k_attention<FOUR, D, F32, kTwoPages>
                                            : k_attention<FOUR, D, F32, kAnyPages>;
  const hipError_t e = launch_kernel(kernel, dim3(grid), dim3(kThreads), 0, stream, a);
  if (e != hipSuccess || a.splits == 1) return e;
  return launch_kernel(k_attention_join<FOUR, D, F32>, dim3(join), dim3(kThreads), 0, stream, a);
}

template <int D>
hipError_t launch_dim(const Args& a, bool four, bool f32, unsigned grid, unsigned join, hipStream_t stream) {
  if (four) return f32 ? launch_typed<true, D, true>(a, grid, join, stream) : launch_typed<true, D, false>(a, grid, join, stream);
  return f32 ? launch_typed<false, D, true>(a, grid, join, stream) : launch_typed<false, D, false>(a, grid, join, stream);
}

}  // namespace

int64_t attention_grid(const CacheView& c, int64_t batch, int64_t share, int64_t width) {
  return c.heads * ((share + kHeads - 1) / kHeads) * cut_for(c, batch, share, width).units;
}

int64_t attention_workspace(const CacheView& c, int64_t batch, int64_t share, int64_t width) {
  if (cut_for(c, batch, share, width).splits == 1) return 0;
  return attention_grid(c, batch, share, width) * kHeads * (c.dim + 2) * (int64_t)sizeof(float);
}

hipError_t launch_attention(const CacheView& c, const void* q, bool bf16, int64_t batch, int64_t share, int64_t q_stride,
                            const int* table, int64_t width, const int* lengths, float scale, void* o, void* work,
                            hipStream_t stream) {
  Args a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k = c.k, a.v = c.v, a.k_scale = c.k_scale, a.v_scale = c.v_scale;
  a.k_amax = c.k_amax, a.v_amax = c.v_amax;
  a.table = table;
  a.lengths = lengths;
  a.o = o;
  a.part = (float*)work;
  a.scale_log2 = scale * 1.44269504088896340736f;
  a.heads = (int)c.heads;
  a.share = (int)share;
  a.tiles = (int)((share + kHeads - 1) / kHeads);
  a.batch = (int)batch;
  const Cut cut = cut_for(c, batch, share, width);
  a.splits = cut.splits;
  auto inverse = [](int n) { return (unsigned)(((uint64_t(1) << 32) + n - 1) / n); };
  if (cut.splits == 0) a.budget_mul = inverse(cut.budget), a.least_mul = inverse(cut.least), a.units = (int)cut.units;
  a.width = (int)width;
  a.n_pages = c.n_pages;
  a.page_size = (unsigned)c.page_size;
  unsigned lg = 0;
  while ((uint64_t(1) << lg) < a.page_size) ++lg;
  a.page_shift = 31 + lg;
  a.page_mul = (unsigned)(((uint64_t(1) << a.page_shift) + a.page_size - 1) / a.page_size);
  const unsigned grid = (unsigned)attention_grid(c, batch, share, width);
  const unsigned join = (unsigned)(batch * c.heads * share);
  if (c.dim == 64) return launch_dim<64>(a, c.four, !bf16, grid, join, stream);
  if (c.dim == 128) return launch_dim<128>(a, c.four, !bf16, grid, join, stream);
  return launch_dim<256>(a, c.four, !bf16, grid, join, stream);
}

}  // namespace lh
