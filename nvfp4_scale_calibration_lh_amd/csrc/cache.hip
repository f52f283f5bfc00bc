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
// Every rounding decision is the one of the exact quotient.
//
// HBM-bound: a lane owns 8 elements (16 bytes of bf16, half of a 16-element block, whose other half
// is in the neighbouring lane), consecutive lanes own consecutive elements, and keys and values go
// in one launch (blockIdx.y).
#include "acc_stream.hpp"
#include "lh_internal.hpp"

#include <algorithm>

namespace lh {
namespace {

using stream::v2bf;
using stream::v2f;
using stream::v4u;
typedef unsigned v2u __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;

struct Args {
  const void* in[2];          // K, V (write)
  int64_t in_stride[2];       // elements between tokens
  void* out[2];               // K, V (read)
  uint8_t* codes[2];
  uint8_t* scales[2];
  const float* amax[2];
  const int64_t* slots;
  int64_t n_units;            // tokens * heads * dim / 8
  int64_t n_slots;
  unsigned heads, dim8, page_size;
};

// First element of unit (token, head, u) in the paged codes, or -1 for a slot outside the cache.
__device__ inline int64_t place(const Args& a, int64_t token, unsigned head, unsigned u) {
  const int64_t slot = a.slots[token];
  if (slot < 0 || slot >= a.n_slots) return -1;
  int64_t page;
  unsigned at;
  if (a.n_slots <= 0xFFFFFFFFll) {
    page = (unsigned)slot / a.page_size;
    at = (unsigned)slot % a.page_size;
  } else {
    page = slot / a.page_size;
    at = (unsigned)(slot % a.page_size);
  }
  return (((page * a.heads + head) * a.page_size + at) * a.dim8 + u) * 8;
}

// (token, head, unit) of linear unit i; 32-bit divisions where the total allows them.
__device__ inline void split(const Args& a, int64_t i, int64_t* token, unsigned* head, unsigned* u) {
  const unsigned per = a.heads * a.dim8;
  unsigned rest;
  if (a.n_units <= 0xFFFFFFFFll) {
    *token = (unsigned)i / per;
    rest = (unsigned)i % per;
  } else {
    *token = i / per;
    rest = (unsigned)(i % per);
  }
  *head = rest / a.dim8;
  *u = rest % a.dim8;
}

// E4M3 code of |x| / s between codes lo and lo + 1: the sign of m s - |x| (m their midpoint, 5
// significant bits) is exact in one fma; a tie goes to the even code.
__device__ inline unsigned e4m3_resolve(float ax, float s, unsigned lo) {
  const float a = __builtin_amdgcn_cvt_f32_fp8((int)lo, 0), b = __builtin_amdgcn_cvt_f32_fp8((int)lo + 1, 0);
  const float d = fmaf(0.5f * (a + b), s, -ax);
  return d < 0.0f ? lo + 1 : (d > 0.0f ? lo : lo + (lo & 1));
}

// Eight signed E4M3 bytes of x / s.  As in the fake-quant: the quotient through the 1-ulp hardware
// reciprocal, pushed up and down by 2^-19, brackets the exact one; where the two round apart, the
// exact decision is taken.  s outside [2^-100, 2^100] (not fast) decides on float64 quotients.
__device__ inline v2u e4m3_codes(const float* x, float s, bool fast) {
  v2u out = {0, 0};
  if (fast) {
    const float is = __builtin_amdgcn_rcpf(s);
    const float iu = is * 1.0000019073486328125f, id = is * 0.9999980926513671875f;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      auto pack = [&](float f) {
        float t[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) t[k] = fminf(fmaxf(x[4 * w + k] * f, -448.0f), 448.0f);
        const int v = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
        return (unsigned)__builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], v, true);
      };
      unsigned up = pack(iu);
      const unsigned dn = pack(id);
      if (up != dn) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const unsigned cu = (up >> (8 * k)) & 127u, cd = (dn >> (8 * k)) & 127u;
          if (cu != cd)
            up = (up & ~(127u << (8 * k))) | (e4m3_resolve(fabsf(x[4 * w + k]), s, cd) << (8 * k));
        }
      }
      out[w] = up;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
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
    const float iu = is * 1.0000019073486328125f, id = is * 0.9999980926513671875f;
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
  // units past the end repeat the last one, so that both lanes of a block exist; they store nothing
  int64_t token;
  unsigned head, u;
  split(a, std::min(i, a.n_units - 1), &token, &head, &u);
  const int64_t from = token * a.in_stride[kv] + (int64_t)(head * a.dim8 + u) * 8;
  float x[8];
  if constexpr (BF16) {
    const v4u v = __builtin_nontemporal_load((const v4u*)((const unsigned short*)a.in[kv] + from));
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      x[2 * p] = stream::bf16_lo(v[p]);
      x[2 * p + 1] = stream::bf16_hi(v[p]);
    }
  } else {
    const v4u* p = (const v4u*)((const float*)a.in[kv] + from);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const v4u v = __builtin_nontemporal_load(p + h);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * h + k] = __uint_as_float(v[k]);
    }
  }
  const float amax = a.amax[kv][head];
  const int64_t to = place(a, token, head, u);
  const bool live = i < a.n_units && to >= 0;
  if constexpr (FOUR) {
    const float g = cache_unit(amax, true);
    const bool fast = g >= 0x1p-100f && g <= 0x1p100f;
    const double inv6g = 1.0 / (6.0 * (double)g);
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, __float_as_uint(x[k]) & 0x7FFFFFFFu);
    m = max(m, stream::dpp_u<0xB1>(m));               // the lane pair: the whole block
    const float top = __uint_as_float(m);
    const float v = fast ? stream::e4m3_nearest_f32(top, inv6g)
                         : (g > 0.0f ? stream::e4m3_nearest((double)top * inv6g) : 0.0f);
    const unsigned nib = e2m1_nibbles(x, v * g, fast);
    if (!live) return;
    *(unsigned*)(a.codes[kv] + to / 2) = nib;
    if (u % 2 == 0) a.scales[kv][to / 16] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(v, 0.0f, 0, false);
  } else {
    const float s = cache_unit(amax, false);
    const v2u c = e4m3_codes(x, s, s >= 0x1p-100f && s <= 0x1p100f);
    if (live) *(v2u*)(a.codes[kv] + to) = c;
  }
}

template <bool BF16, bool FOUR>
__global__ __launch_bounds__(kThreads) void k_cache_read(const Args a) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int kv = blockIdx.y;
  if (i >= a.n_units) return;
  int64_t token;
  unsigned head, u;
  split(a, i, &token, &head, &u);
  const int64_t from = place(a, token, head, u);
  float x[8];
  if (from < 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = 0.0f;
  } else if constexpr (FOUR) {
    const unsigned nib = *(const unsigned*)(a.codes[kv] + from / 2);
    const float s = __builtin_amdgcn_cvt_f32_fp8((int)a.scales[kv][from / 16], 0) * cache_unit(a.amax[kv][head], true);
    auto dec = [&](auto sel) {
      constexpr int p = decltype(sel)::value;
      const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(nib, 1.0f, p);
      x[2 * p] = v[0] * s;
      x[2 * p + 1] = v[1] * s;
    };
    dec(std::integral_constant<int, 0>{});
    dec(std::integral_constant<int, 1>{});
    dec(std::integral_constant<int, 2>{});
    dec(std::integral_constant<int, 3>{});
  } else {
    const v2u c = *(const v2u*)(a.codes[kv] + from);
    const float s = cache_unit(a.amax[kv][head], false);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], false), hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)c[w], true);
      x[4 * w] = lo[0] * s;
      x[4 * w + 1] = lo[1] * s;
      x[4 * w + 2] = hi[0] * s;
      x[4 * w + 3] = hi[1] * s;
    }
  }
  if constexpr (BF16) {
    v4u o;
#pragma unroll
    for (int p = 0; p < 4; ++p)
      o[p] = __builtin_bit_cast(unsigned, __builtin_convertvector((v2f){x[2 * p], x[2 * p + 1]}, v2bf));
    __builtin_nontemporal_store(o, (v4u*)a.out[kv] + i);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      v4u o;
#pragma unroll
      for (int k = 0; k < 4; ++k) o[k] = __float_as_uint(x[4 * h + k]);
      __builtin_nontemporal_store(o, (v4u*)a.out[kv] + 2 * i + h);
    }
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
  a.dim8 = (unsigned)(c.dim / 8);
  a.page_size = (unsigned)c.page_size;
  a.n_slots = c.n_pages * c.page_size;
  a.n_units = tokens * c.heads * (c.dim / 8);
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
  const dim3 grid((unsigned)((a.n_units + kThreads - 1) / kThreads), 2);
  if (c.four) {
    if (bf16) hipLaunchKernelGGL((k_cache_write<true, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_cache_write<false, true>), grid, dim3(kThreads), 0, stream, a);
  } else {
    if (bf16) hipLaunchKernelGGL((k_cache_write<true, false>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_cache_write<false, false>), grid, dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheView& c, const int64_t* slots, int64_t tokens, void* k, void* v, bool bf16,
                             hipStream_t stream) {
  Args a = args_of(c, tokens, slots);
  a.out[0] = k;
  a.out[1] = v;
  const dim3 grid((unsigned)((a.n_units + kThreads - 1) / kThreads), 2);
  if (c.four) {
    if (bf16) hipLaunchKernelGGL((k_cache_read<true, true>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_cache_read<false, true>), grid, dim3(kThreads), 0, stream, a);
  } else {
    if (bf16) hipLaunchKernelGGL((k_cache_read<true, false>), grid, dim3(kThreads), 0, stream, a);
    else hipLaunchKernelGGL((k_cache_read<false, false>), grid, dim3(kThreads), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace lh
