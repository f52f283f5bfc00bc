// C ABI of the decode-step operators (declarations and contracts in include/lh.h): RMS norm with
// 8-bit output, products with NVFP4 weights, the quantized key-value cache and attention over it.
//
// Every entry point validates its arguments, selects the device that owns the pointers and launches
// on the caller's stream.  There is no state besides the thread's error message.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/lh.h"
#include "lh_host.hpp"
#include "lh_internal.hpp"

using namespace lh::host;

namespace {

constexpr int64_t kMaxInt = 2147483647LL;
constexpr int64_t kMaxCin = int64_t(1) << 24;

lh_status check_rows(int64_t rows, int64_t cin) {
  if (rows < 0 || rows > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "rows must be in [0, 2^31-1] (got %lld)", (long long)rows);
  if (cin <= 0 || cin % 16 || cin > kMaxCin)
    return fail(LH_ERR_INVALID_ARGUMENT, "cin must be a positive multiple of 16 up to 2^24 (got %lld)", (long long)cin);
  return LH_OK;
}

lh_status check_cache(const lh_cache* c, lh::CacheView* out) {
  if (!c) return fail(LH_ERR_INVALID_ARGUMENT, "cache is NULL");
  if (c->format != LH_CACHE_E4M3 && c->format != LH_CACHE_FP4) return fail(LH_ERR_UNSUPPORTED, "unknown cache format %d", (int)c->format);
  const bool four = c->format == LH_CACHE_FP4;
  if (c->n_pages < 1 || c->page_size < 1 || c->n_heads < 1 || c->head_dim < 1)
    return fail(LH_ERR_INVALID_ARGUMENT, "n_pages, page_size, n_heads and head_dim must be positive");
  if (c->head_dim % 16 || c->head_dim > 65536) return fail(LH_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 16 up to 65536 (got %lld)", (long long)c->head_dim);
  if (c->page_size > kMaxInt || c->n_heads > (int64_t(1) << 27) / c->head_dim || c->n_pages > (int64_t(1) << 40) / c->page_size)
    return fail(LH_ERR_INVALID_ARGUMENT, "the cache is too large");
  if (!c->k || !c->v || !c->k_amax || !c->v_amax) return fail(LH_ERR_INVALID_ARGUMENT, "k, v, k_amax and v_amax are required");
  if (four != (c->k_scale != nullptr) || four != (c->v_scale != nullptr))
    return fail(LH_ERR_INVALID_ARGUMENT, four ? "k_scale and v_scale are required" : "k_scale and v_scale must be NULL for E4M3");
  for (const PtrCheck& p : {PtrCheck{c->k, "k"}, PtrCheck{c->v, "v"}}) {
    const lh_status st = check_aligned(p.p, p.name);
    if (st != LH_OK) return st;
  }
  if (((reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale)) & 3) != 0)
    return fail(LH_ERR_INVALID_ARGUMENT, "k_scale and v_scale must be 4-byte aligned");
  *out = lh::CacheView{c->k, c->v, c->k_scale, c->v_scale, c->k_amax, c->v_amax,
                       c->n_pages, c->page_size, c->n_heads, c->head_dim, four};
  return LH_OK;
}

// Workgroups of the cache kernels (256 lanes of 16 elements, tokens in sixteens), which must fit a launch.
lh_status check_tokens(const lh::CacheView& c, int64_t tokens) {
  if (tokens < 0) return fail(LH_ERR_INVALID_ARGUMENT, "tokens must be >= 0 (got %lld)", (long long)tokens);
  if (tokens > kMaxInt * 256 / (c.heads * (c.dim / 16)) - 16) return fail(LH_ERR_INVALID_ARGUMENT, "too many tokens for one call");
  return LH_OK;
}

}  // namespace

extern "C" {

lh_status lh_rms_norm_quant(const void* X, const void* R, lh_dtype dtype, int64_t rows, int64_t cin,
                            const void* gamma, float eps, int64_t group, void* summed, uint8_t* q,
                            float* q_scale, void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  lh_status st = check_rows(rows, cin);
  if (st != LH_OK) return st;
  if (group != 0 && group != 128) return fail(LH_ERR_INVALID_ARGUMENT, "group must be 0 or 128 (got %lld)", (long long)group);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(LH_ERR_INVALID_ARGUMENT, "eps must be >= 0 and finite");
  if ((R == nullptr) != (summed == nullptr)) return fail(LH_ERR_INVALID_ARGUMENT, "R and summed must be given together");
  if (!gamma) return fail(LH_ERR_INVALID_ARGUMENT, "gamma is required");
  if (rows == 0) return ok();
  if (!X || !q || !q_scale) return fail(LH_ERR_INVALID_ARGUMENT, "X, q and q_scale are required");
  for (const PtrCheck& p : {PtrCheck{X, "X"}, PtrCheck{R, "R"}, PtrCheck{gamma, "gamma"}, PtrCheck{summed, "summed"}, PtrCheck{q, "q"}})
    if ((st = check_aligned(p.p, p.name)) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{X, "X"}, {R, "R"}, {gamma, "gamma"}, {summed, "summed"}, {q, "q"}, {q_scale, "q_scale"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const hipError_t e = lh::launch_rms_norm(X, R, dtype == LH_DTYPE_BF16, rows, cin, gamma, eps, group != 0, summed, q, q_scale,
                                           reinterpret_cast<hipStream_t>(stream));
  return launched(e, "norm launch");
}

lh_status lh_matvec(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t rows,
                    int64_t cin, const int64_t* group_offsets, int64_t n_groups, int64_t cout,
                    const uint8_t* scale_code, const uint8_t* fp4, const float* global_amax,
                    float scale_norm, void* Y, void* stream) {
  const bool eight = x_dtype == LH_DTYPE_E4M3;
  if (!eight && !dtype_ok(x_dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)x_dtype);
  lh_status st = check_rows(rows, cin);
  if (st != LH_OK) return st;
  if (n_groups < 1 || n_groups > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "n_groups must be >= 1 (got %lld)", (long long)n_groups);
  if (!group_offsets && n_groups != 1) return fail(LH_ERR_INVALID_ARGUMENT, "group_offsets is required when n_groups > 1");
  if (cout < 0 || cout > 65535LL * 32) return fail(LH_ERR_INVALID_ARGUMENT, "cout must be in [0, 2097120] (got %lld)", (long long)cout);
  if (!e4m3_value(scale_norm)) return fail(LH_ERR_INVALID_ARGUMENT, "scale_norm must be a positive finite E4M3 value such as 448 or 256 (got %g)", (double)scale_norm);
  if (x_group != 0 && (x_group != 128 || !eight)) return fail(LH_ERR_INVALID_ARGUMENT, "x_group must be 0, or 128 for E4M3 rows (got %lld)", (long long)x_group);
  if (eight ? (!x_scale && rows > 0) : x_scale != nullptr)
    return fail(LH_ERR_INVALID_ARGUMENT, eight ? "x_scale is required for E4M3 rows" : "x_scale must be NULL for rows that are not E4M3");
  if (rows == 0 || cout == 0) return ok();
  if (!X || !Y || !scale_code || !fp4 || !global_amax) return fail(LH_ERR_INVALID_ARGUMENT, "X, scale_code, fp4, global_amax and Y are required");
  // at most one workgroup per 16 channels for every 4 rows and, with several groups, for every group with rows
  const int64_t pieces = (rows + 3) / 4 + (n_groups > 1 ? std::min(n_groups, rows) : 0);
  if (pieces > kMaxInt / ((cout + 15) / 16)) return fail(LH_ERR_INVALID_ARGUMENT, "too many rows for one call");
  if ((st = check_aligned(X, "X")) != LH_OK) return st;
  if (reinterpret_cast<uintptr_t>(fp4) % 8 != 0) return fail(LH_ERR_INVALID_ARGUMENT, "fp4 must be 8-byte aligned");
  int dev = -1;
  st = check_pointers({{X, "X"}, {x_scale, "x_scale"}, {group_offsets, "group_offsets"}, {scale_code, "scale_code"}, {fp4, "fp4"}, {global_amax, "global_amax"}, {Y, "Y"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const hipError_t e = lh::launch_matvec(X, eight ? 2 : (x_dtype == LH_DTYPE_F32 ? 1 : 0), x_scale, x_group ? (cin + 127) / 128 : 1, rows,
                                         cin, cout, n_groups > 1 ? group_offsets : nullptr, n_groups, scale_code, fp4, global_amax,
                                         6.0f * scale_norm, Y, reinterpret_cast<hipStream_t>(stream));
  return launched(e, "matvec launch");
}

lh_status lh_cache_write(const lh_cache* cache, const void* K, int64_t k_stride, const void* V,
                         int64_t v_stride, lh_dtype dtype, int64_t tokens, const int64_t* slots,
                         void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  lh::CacheView c;
  lh_status st = check_cache(cache, &c);
  if (st != LH_OK) return st;
  if ((st = check_tokens(c, tokens)) != LH_OK) return st;
  if ((st = check_stride(k_stride, c.heads * c.dim, dtype, "k_stride")) != LH_OK) return st;
  if ((st = check_stride(v_stride, c.heads * c.dim, dtype, "v_stride")) != LH_OK) return st;
  if (tokens == 0) return ok();
  if (!K || !V || !slots) return fail(LH_ERR_INVALID_ARGUMENT, "K, V and slots are required");
  if ((st = check_aligned(K, "K")) != LH_OK) return st;
  if ((st = check_aligned(V, "V")) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{K, "K"}, {V, "V"}, {slots, "slots"}, {c.k, "k"}, {c.v, "v"}, {c.k_scale, "k_scale"}, {c.v_scale, "v_scale"}, {c.k_amax, "k_amax"}, {c.v_amax, "v_amax"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const hipError_t e = lh::launch_cache_write(c, K, V, dtype == LH_DTYPE_BF16, tokens, k_stride, v_stride, slots,
                                              reinterpret_cast<hipStream_t>(stream));
  return launched(e, "cache write launch");
}

lh_status lh_cache_read(const lh_cache* cache, const int64_t* slots, int64_t tokens, lh_dtype dtype,
                        void* K, void* V, void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  lh::CacheView c;
  lh_status st = check_cache(cache, &c);
  if (st != LH_OK) return st;
  if ((st = check_tokens(c, tokens)) != LH_OK) return st;
  if (tokens == 0) return ok();
  if (!K || !V || !slots) return fail(LH_ERR_INVALID_ARGUMENT, "K, V and slots are required");
  if ((st = check_aligned(K, "K")) != LH_OK) return st;
  if ((st = check_aligned(V, "V")) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{slots, "slots"}, {K, "K"}, {V, "V"}, {c.k, "k"}, {c.v, "v"}, {c.k_scale, "k_scale"}, {c.v_scale, "v_scale"}, {c.k_amax, "k_amax"}, {c.v_amax, "v_amax"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const hipError_t e = lh::launch_cache_read(c, slots, tokens, K, V, dtype == LH_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream));
  return launched(e, "cache read launch");
}

}  // extern "C"

namespace {

lh_status check_attention(const lh::CacheView& c, int64_t batch, int64_t n_q_heads, int64_t max_pages) {
  if (c.dim != 64 && c.dim != 128 && c.dim != 256) return fail(LH_ERR_UNSUPPORTED, "head_dim must be 64, 128 or 256 for attention (got %lld)", (long long)c.dim);
  if (n_q_heads < 1 || n_q_heads % c.heads) return fail(LH_ERR_INVALID_ARGUMENT, "n_q_heads must be a positive multiple of the cache's %lld heads (got %lld)", (long long)c.heads, (long long)n_q_heads);
  if (batch < 0) return fail(LH_ERR_INVALID_ARGUMENT, "batch must be >= 0 (got %lld)", (long long)batch);
  if (max_pages < 0 || max_pages > lh::kMaxContext / c.page_size) return fail(LH_ERR_INVALID_ARGUMENT, "max_pages * page_size must be in [0, 2^31-4096]");
  if (batch > kMaxInt / n_q_heads || lh::attention_grid(c, batch, n_q_heads / c.heads, max_pages) > kMaxInt)
    return fail(LH_ERR_INVALID_ARGUMENT, "too many sequences for one call");
  return LH_OK;
}

}  // namespace

extern "C" {

int64_t lh_paged_attention_workspace(const lh_cache* cache, int64_t batch, int64_t n_q_heads, int64_t max_pages) {
  lh::CacheView c;
  if (check_cache(cache, &c) != LH_OK || check_attention(c, batch, n_q_heads, max_pages) != LH_OK) return 0;
  (void)ok();
  return lh::attention_workspace(c, batch, n_q_heads / c.heads, max_pages);
}

lh_status lh_paged_attention(const lh_cache* cache, const void* Q, int64_t q_stride, lh_dtype dtype,
                             int64_t batch, int64_t n_q_heads, const int32_t* block_table,
                             int64_t max_pages, const int32_t* lengths, float scale, void* O,
                             void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  lh::CacheView c;
  lh_status st = check_cache(cache, &c);
  if (st != LH_OK) return st;
  if ((st = check_attention(c, batch, n_q_heads, max_pages)) != LH_OK) return st;
  if ((st = check_stride(q_stride, n_q_heads * c.dim, dtype, "q_stride")) != LH_OK) return st;
  if (!std::isfinite(scale)) return fail(LH_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (batch == 0) return ok();
  if (!Q || !O || !lengths || (!block_table && max_pages > 0)) return fail(LH_ERR_INVALID_ARGUMENT, "Q, block_table, lengths and O are required");
  const int64_t share = n_q_heads / c.heads, need = lh::attention_workspace(c, batch, share, max_pages);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(LH_ERR_INVALID_ARGUMENT, "workspace must hold %lld bytes (got %lld)", (long long)need, (long long)(workspace ? workspace_bytes : 0));
  for (const PtrCheck& p : {PtrCheck{Q, "Q"}, PtrCheck{O, "O"}, PtrCheck{workspace, "workspace"}})
    if ((st = check_aligned(p.p, p.name)) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{Q, "Q"}, {O, "O"}, {block_table, "block_table"}, {lengths, "lengths"}, {workspace, "workspace"}, {c.k, "k"}, {c.v, "v"}, {c.k_scale, "k_scale"}, {c.v_scale, "v_scale"}, {c.k_amax, "k_amax"}, {c.v_amax, "v_amax"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const hipError_t e = lh::launch_attention(c, Q, dtype == LH_DTYPE_BF16, batch, share, q_stride, block_table, max_pages, lengths, scale, O,
                                            workspace, reinterpret_cast<hipStream_t>(stream));
  return launched(e, "attention launch");
}

}  // extern "C"
