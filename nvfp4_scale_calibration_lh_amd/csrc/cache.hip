// The quantised key-value cache: writing new tokens' keys and values to their slots, and reading
// slots back.
//
// A page holds page_size tokens of every key-value head, head by head: element (page, head, token,
// i) of the codes is at ((page * heads + head) * page_size + token) * dim + i, so attention reads
// one head's tokens of a page as one run of memory.  With one amax per head,
//   E4M3:  byte = sign, E4M3 value nearest to |x| / s, s = fp32(amax * fp32(1/448)) (ties to the
//          even code, saturating at 448); the value is fp32(E4M3 * s)
//   NVFP4: per 16 elements v = E4M3 nearest to max|x| / (6 g), g = fp32(amax * fp32(1/2688)), and
//          nibbles E2M1 nearest to |x| / s, s = fp32(v g): the input quantizer's rule on this g
// Every rounding decision is the one of the exact quotient.  Infinities saturate like any large element; a NaN is
// held as a NaN code, in E2M1, which has none, as a NaN scale of its block.
//
// A lane writes its block's codes and scale by two plain stores, unordered against those of other lanes: slots of
// one call are different ones, or their contents are unspecified.
//
// Bound by memory where the instructions allow it: a lane owns a 16-element block (32 bytes of bf16),
// consecutive lanes own consecutive blocks, and keys and values go in one launch (blockIdx.y).  Indices
// are split by multiplications with reciprocals from the host: with 32-bit divisions and 8 elements a
// lane, 8191 tokens of 8 x 128 took 16 us to write, bound by instructions.  Now 12.3 us (43 MB, 3.5
// TB/s) and 11.8 us to read back; 30011 tokens of 4 x 64 in E4M3 11.4 and 11.8 us (traced medians).
#include "acc_stream.hpp"
#include "e4m3.hpp"
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

using stream::v2bf;
using stream::v2f;
using stream::v4u;
typedef unsigned v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

// Division by d of n < 2^31: (2 n * mul) >> 32 >> lg with mul = ceil(2^(31 + lg) / d), lg = ceil(log2 d).
struct Divisor {
  unsigned d, mul, lg;
};
__device__ inline unsigned divide(unsigned n, const Divisor& by) { return __umulhi(2 * n, by.mul) >> by.lg; }
Divisor divisor(int64_t d) {
  Divisor r{(unsigned)d, 0, 0};
  while ((int64_t(1) << r.lg) < d) ++r.lg;
  r.mul = (unsigned)(((uint64_t(1) << (31 + r.lg)) + (uint64_t)d - 1) / (uint64_t)d);
  return r;
}

constexpr unsigned kTokens = 16;

struct Args {
  const void* in[2];          // K, V (write)
  int64_t in_stride[2];       // elements between tokens
  void* out[2];               // K, V (read)
  uint8_t* codes[2];
  uint8_t* scales[2];
  const float* amax[2];
  const int64_t* slots;
  int64_t tokens, n_blocks;   // n_blocks: tokens rounded up to kTokens, * heads * dim / 16
  int64_t n_slots;
  unsigned heads;
  Divisor dim16, group, page; // blocks of one head's row, of kTokens tokens, tokens of a page
};

// The first block of (token, head) in the paged codes, in 16-element blocks, or -1 for a slot outside
// the cache.
__device__ inline int64_t place(const Args& a, int64_t token, unsigned head) {
  const int64_t slot = a.slots[token];
  if (slot < 0 || slot >= a.n_slots) return -1;
  int64_t page;
  unsigned at;
  if (a.n_slots <= 0x7FFFFFFFll) {
    const unsigned p = divide((unsigned)slot, a.page);
    page = p;
    at = (unsigned)slot - p * a.page.d;
  } else {
    page = slot / a.page.d;
    at = (unsigned)(slot - page * a.page.d);
  }
  return ((page * a.heads + head) * a.page.d + at) * a.dim16.d;
}

// (token, head, block) of linear block i: 16 tokens of a head, then the next head's, then the next 16
// tokens, so that neighbouring slots' codes and scales, which lie side by side per head, are written
// as whole lines by one workgroup.  A token past the last is none.
__device__ inline void split(const Args& a, int64_t i, int64_t* token, unsigned* head, unsigned* u) {
  int64_t group;
  unsigned rest;
  if (a.n_blocks <= 0x7FFFFFFFll) {
    const unsigned g = divide((unsigned)i, a.group);
    group = g;
    rest = (unsigned)i - g * a.group.d;
  } else {
    group = i / a.group.d;
    rest = (unsigned)(i - group * a.group.d);
  }
  const unsigned row = divide(rest, a.dim16);
  *u = rest - row * a.dim16.d;
  *head = row / kTokens;
  *token = group * kTokens + row % kTokens;
}

// E4M3 code of a block's scale, top / (6 g); g in [2^-100, 2^100].
__device__ inline unsigned block_code(float top, float g) {
  const float t = top * __builtin_amdgcn_rcpf(6.0f * g);
  const unsigned c = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(fminf(t * kUp, 448.0f), fminf(t * kDown, 448.0f), 0, false);
  const unsigned up = c & 255u, dn = (c >> 8) & 255u;
  return up == dn ? up : e4m3_resolve6(top, g, dn);
}

// Sixteen signed E4M3 bytes of x / s.  s outside [2^-100, 2^100] (not fast) decides on float64 quotients.
__device__ inline v4u e4m3_codes(const float* x, float s, bool fast) {
  v4u out = {0, 0, 0, 0};
  if (fast) {
    const float is = __builtin_amdgcn_rcpf(s);
#pragma unroll
    for (int w = 0; w < 4; ++w) out[w] = e4m3_word(x + 4 * w, s, is);
  } else {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float v = s > 0.0f ? stream::e4m3_nearest((double)fabsf(x[k]) / (double)s) : 0.0f;
      const unsigned c = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(copysignf(v, x[k]), 0.0f, 0, false) & 255u;
      out[k / 4] |= c << (8 * (k % 4));
    }
  }
  return out;
}

// Eight E2M1 nibbles of x / s (element 2j in the low half of byte j), decided as in the fake-quant.
__device__ inline unsigned e2m1_nibbles(const float* x, float s, bool fast) {
  if (fast) {
    const float is = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
    const float iu = is * kUp, id = is * kDown;
    unsigned up = 0u, dn = 0u;
    auto pack = [&](auto sel) {
      constexpr int p = decltype(sel)::value;
      up = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(up, x[2 * p] * iu, x[2 * p + 1] * iu, 1.0f, p);
      dn = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(dn, x[2 * p] * id, x[2 * p + 1] * id, 1.0f, p);
    };
    pack(std::integral_constant<int, 0>{});
    pack(std::integral_constant<int, 1>{});
    pack(std::integral_constant<int, 2>{});
    pack(std::integral_constant<int, 3>{});
    if (up != dn) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int cu = (up >> (4 * k)) & 7, cd = (dn >> (4 * k)) & 7;
        if (cu != cd)
          up = (up & ~(7u << (4 * k))) | ((unsigned)stream::e2m1_resolve(fabsf(x[k]), s, cd) << (4 * k));
      }
    }
    return up;
  }
  unsigned out = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int c = s == 0.0f ? 0 : stream::e2m1_index_f64((double)fabsf(x[k]) / (double)s);
    out |= ((unsigned)c | (__float_as_uint(x[k]) >> 31 << 3)) << (4 * k);
  }
  return out;
}

template <bool BF16, bool FOUR>
__global__ __launch_bounds__(kThreads) void k_cache_write(const Args a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int kv = blockIdx.y;
  if (i >= a.n_blocks) return;
  int64_t token;
  unsigned head, u;
  split(a, i, &token, &head, &u);
  if (token >= a.tokens) return;
  const int64_t from = token * a.in_stride[kv] + (int64_t)(head * a.dim16.d + u) * 16;
  float x[16];
#pragma unroll
  for (int h = 0; h < (BF16 ? 2 : 4); ++h) {
    if constexpr (BF16) {
      const v4u v = ((const v4u*)((const unsigned short*)a.in[kv] + from))[h];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        x[8 * h + 2 * p] = stream::bf16_lo(v[p]);
        x[8 * h + 2 * p + 1] = stream::bf16_hi(v[p]);
      }
    } else {
      const v4u v = ((const v4u*)((const float*)a.in[kv] + from))[h];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = __uint_as_float(v[k]);
    }
  }
  const float amax = a.amax[kv][head];
  const int64_t row = place(a, token, head);
  if (row < 0) return;
  const int64_t to = row + u;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 16; k += 2) nan |= __builtin_isunordered(x[k], x[k + 1]);
  if constexpr (FOUR) {
    const float g = cache_unit(amax, true);
    const bool fast = g >= 0x1p-100f && g <= 0x1p100f;
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));
    unsigned code = 0;
    if (fast) code = block_code(top, g);
    else if (g > 0.0f) code = (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(stream::e4m3_nearest((double)top / (6.0 * (double)g)), 0.0f, 0, false) & 255u;
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)code, 0) * g;
    const v2u nib = {e2m1_nibbles(x, s, fast), e2m1_nibbles(x + 8, s, fast)};
    ((v2u*)a.codes[kv])[to] = nib;
    a.scales[kv][to] = nan ? 0x7F : (uint8_t)code;
  } else {
    const float s = cache_unit(amax, false);
    v4u codes = e4m3_codes(x, s, s >= 0x1p-100f && s <= 0x1p100f);
    if (nan) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (x[k] != x[k]) codes[k / 4] |= 0x7Fu << (8 * (k % 4));
    }
    ((v4u*)a.codes[kv])[to] = codes;
  }
}

template <bool BF16, bool FOUR>
__global__ __launch_bounds__(kThreads) void k_cache_read(const Args a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int kv = blockIdx.y;
  if (i >= a.n_blocks) return;
  int64_t token;
  unsigned head, u;
  split(a, i, &token, &head, &u);
  if (token >= a.tokens) return;
  const int64_t to = (token * a.heads + head) * a.dim16.d + u;
  const int64_t row = place(a, token, head);
  float x[16];
  if (row < 0) {
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = 0.0f;
  } else if constexpr (FOUR) {
    const v2u nib = ((const v2u*)a.codes[kv])[row + u];
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)a.scales[kv][row + u], 0) * cache_unit(a.amax[kv][head], true);
    auto dec = [&](auto sel) {
      constexpr int p = decltype(sel)::value;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(nib[w], 1.0f, p);
        x[8 * w + 2 * p] = v[0] * s;
        x[8 * w + 2 * p + 1] = v[1] * s;
      }
    };
    dec(std::integral_constant<int, 0>{});
    dec(std::integral_constant<int, 1>{});
    dec(std::integral_constant<int, 2>{});
    dec(std::integral_constant<int, 3>{});
  } else {
    const v4u c = ((const v4u*)a.codes[kv])[row + u];
    const float s = cache_unit(a.amax[kv][head], false);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], true);
      x[4 * w] = lo[0] * s;
      x[4 * w + 1] = lo[1] * s;
      x[4 * w + 2] = hi[0] * s;
      x[4 * w + 3] = hi[1] * s;
    }
  }
#pragma unroll
  for (int h = 0; h < (BF16 ? 2 : 4); ++h) {
    v4u o;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if constexpr (BF16) o[p] = __builtin_bit_cast(unsigned, __builtin_convertvector((v2f){x[8 * h + 2 * p], x[8 * h + 2 * p + 1]}, v2bf));
      else o[p] = __float_as_uint(x[4 * h + p]);
    }
    ((v4u*)a.out[kv])[to * (BF16 ? 2 : 4) + h] = o;
  }
}

Args args_of(const CacheView& c, int64_t tokens, const int64_t* slots) {
  Args a{};
  for (int kv = 0; kv < 2; ++kv) {
    a.codes[kv] = kv ? c.v : c.k;
    a.scales[kv] = kv ? c.v_scale : c.k_scale;
    a.amax[kv] = kv ? c.v_amax : c.k_amax;
  }
  a.slots = slots;
  a.heads = (unsigned)c.heads;
  a.dim16 = divisor(c.dim / 16);
  a.group = divisor(kTokens * c.heads * (c.dim / 16));
  a.page = divisor(c.page_size);
  a.n_slots = c.n_pages * c.page_size;
  a.tokens = tokens;
  a.n_blocks = (tokens + kTokens - 1) / kTokens * a.group.d;
  return a;
}

}  // namespace

hipError_t launch_cache_write(const CacheView& c, const void* k, const void* v, bool bf16, int64_t tokens,
                              int64_t k_stride, int64_t v_stride, const int64_t* slots, hipStream_t stream) {
  Args a = args_of(c, tokens, slots);
  a.in[0] = k;
  a.in[1] = v;
  a.in_stride[0] = k_stride;
  a.in_stride[1] = v_stride;
  const dim3 grid((unsigned)((a.n_blocks + kThreads - 1) / kThreads), 2);
  if (c.four)
    return launch_kernel(bf16 ? k_cache_write<true, true> : k_cache_write<false, true>, grid, dim3(kThreads), 0, stream, a);
  return launch_kernel(bf16 ? k_cache_write<true, false> : k_cache_write<false, false>, grid, dim3(kThreads), 0, stream, a);
}

hipError_t launch_cache_read(const CacheView& c, const int64_t* slots, int64_t tokens, void* k, void* v, bool bf16,
                             hipStream_t stream) {
  Args a = args_of(c, tokens, slots);
  a.out[0] = k;
  a.out[1] = v;
  const dim3 grid((unsigned)((a.n_blocks + kThreads - 1) / kThreads), 2);
  if (c.four)
    return launch_kernel(bf16 ? k_cache_read<true, true> : k_cache_read<false, true>, grid, dim3(kThreads), 0, stream, a);
  return launch_kernel(bf16 ? k_cache_read<true, false> : k_cache_read<false, false>, grid, dim3(kThreads), 0, stream, a);
}

}  // namespace lh
