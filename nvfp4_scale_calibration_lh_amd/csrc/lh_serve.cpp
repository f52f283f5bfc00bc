// C ABI of the operators around a decode step (declarations and contracts in include/lh.h): growth of the cache's
// sequences, rotary positions, the choice of experts, the expert layer and low-rank adapters.
//
// As for the decode-step operators: arguments are checked, the device that owns the pointers is selected, and the kernels are
// launched on the caller's stream.  There is no state besides the thread's error message.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/lh.h"
#include "lh_host.hpp"
#include "lh_internal.hpp"

using namespace lh::host;

namespace {

constexpr int64_t kMaxInt = 2147483647LL;

lh_status check_extend(int64_t batch, int64_t max_pages, int64_t page_size, int64_t max_tokens) {
  if (batch < 0 || batch > kMaxInt / 8) return fail(LH_ERR_INVALID_ARGUMENT, "batch must be in [0, 2^28-1] (got %lld)", (long long)batch);
  if (page_size < 1 || page_size > lh::kMaxContext) return fail(LH_ERR_INVALID_ARGUMENT, "page_size must be in [1, 2^31-4096] (got %lld)", (long long)page_size);
  if (max_pages < 0 || max_pages > lh::kMaxContext / page_size) return fail(LH_ERR_INVALID_ARGUMENT, "max_pages * page_size must be in [0, 2^31-4096]");
  if (max_tokens < 0 || max_tokens > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "max_tokens must be in [0, 2^31-1] (got %lld)", (long long)max_tokens);
  return LH_OK;
}

// tokens * topk choices and their rows' offsets; hidden * inner keeps a matrix's offsets within 32 bits.
lh_status check_moe(int64_t tokens, int64_t hidden, int64_t inner, int64_t n_experts, int64_t topk) {
  if (tokens < 0 || tokens > 65535 * 64) return fail(LH_ERR_INVALID_ARGUMENT, "tokens must be in [0, 4194240] (got %lld)", (long long)tokens);
  if (hidden < 1 || hidden % 16 || hidden > (int64_t(1) << 24)) return fail(LH_ERR_INVALID_ARGUMENT, "hidden must be a positive multiple of 16 up to 2^24 (got %lld)", (long long)hidden);
  if (inner < 1 || inner % 16 || inner > (int64_t(1) << 24)) return fail(LH_ERR_INVALID_ARGUMENT, "inner must be a positive multiple of 16 up to 2^24 (got %lld)", (long long)inner);
  if (hidden * inner > int64_t(1) << 32) return fail(LH_ERR_INVALID_ARGUMENT, "hidden * inner must be at most 2^32");
  if (n_experts < 1 || n_experts > lh::kMaxExperts) return fail(LH_ERR_INVALID_ARGUMENT, "n_experts must be in [1, 4096] (got %lld)", (long long)n_experts);
  if (topk < 1 || topk > 64) return fail(LH_ERR_INVALID_ARGUMENT, "topk must be in [1, 64] (got %lld)", (long long)topk);
  return LH_OK;
}

lh_status check_adapter(int64_t rows, int64_t cin, int64_t cout, int64_t n_adapters, int64_t rank) {
  if (rows < 0 || rows > 65535 * 64) return fail(LH_ERR_INVALID_ARGUMENT, "rows must be in [0, 4194240] (got %lld)", (long long)rows);
  if (cin <= 0 || cin % 16 || cin > (int64_t(1) << 24)) return fail(LH_ERR_INVALID_ARGUMENT, "cin must be a positive multiple of 16 up to 2^24 (got %lld)", (long long)cin);
  if (cout < 0 || cout > (int64_t(1) << 24)) return fail(LH_ERR_INVALID_ARGUMENT, "cout must be in [0, 2^24] (got %lld)", (long long)cout);
  if (n_adapters < 1 || n_adapters > lh::kMaxExperts) return fail(LH_ERR_INVALID_ARGUMENT, "n_adapters must be in [1, 4096] (got %lld)", (long long)n_adapters);
  if (rank < 8 || rank % 8 || rank > 256) return fail(LH_ERR_INVALID_ARGUMENT, "rank must be a multiple of 8 in [8, 256] (got %lld)", (long long)rank);
  return LH_OK;
}

// Rows of a product: their type (E4M3 with scales, as lh_matvec takes them).
lh_status check_rows_type(lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t rows) {
  const bool eight = x_dtype == LH_DTYPE_E4M3;
  if (!eight && !dtype_ok(x_dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)x_dtype);
  if (x_group != 0 && (x_group != 128 || !eight)) return fail(LH_ERR_INVALID_ARGUMENT, "x_group must be 0, or 128 for E4M3 rows (got %lld)", (long long)x_group);
  if (eight ? (!x_scale && rows > 0) : x_scale != nullptr)
    return fail(LH_ERR_INVALID_ARGUMENT, eight ? "x_scale is required for E4M3 rows" : "x_scale must be NULL for rows that are not E4M3");
  return LH_OK;
}

int type_of_rows(lh_dtype t) { return t == LH_DTYPE_E4M3 ? 2 : (t == LH_DTYPE_F32 ? 1 : 0); }

}  // namespace

extern "C" {

int64_t lh_cache_extend_workspace(int64_t batch, int64_t max_tokens) {
  if (check_extend(batch, 0, 1, max_tokens) != LH_OK) return 0;
  (void)ok();
  return lh::extend_workspace(batch, max_tokens);
}

lh_status lh_cache_extend(int32_t* block_table, int64_t batch, int64_t max_pages, int64_t page_size, const int32_t* lengths,
                          const int32_t* new_tokens, int32_t* free_pages, int64_t capacity, const int32_t* free_count,
                          int64_t max_tokens, int64_t* slots, int32_t* positions, int32_t* sequence, int32_t* offsets,
                          int32_t* new_lengths, int32_t* new_count, void* workspace, int64_t workspace_bytes, void* stream) {
  lh_status st = check_extend(batch, max_pages, page_size, max_tokens);
  if (st != LH_OK) return st;
  if (capacity < 0 || capacity > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "capacity must be in [0, 2^31-1] (got %lld)", (long long)capacity);
  if (!free_count || !new_count || !offsets) return fail(LH_ERR_INVALID_ARGUMENT, "free_count, new_count and offsets are required");
  if (batch > 0 && (!lengths || !new_lengths || (!block_table && max_pages > 0)))
    return fail(LH_ERR_INVALID_ARGUMENT, "block_table, lengths and new_lengths are required");
  if (capacity > 0 && !free_pages) return fail(LH_ERR_INVALID_ARGUMENT, "free_pages is required");
  if (max_tokens > 0 && (!slots || !positions || !sequence)) return fail(LH_ERR_INVALID_ARGUMENT, "slots, positions and sequence are required");
  const int64_t need = lh::extend_workspace(batch, max_tokens);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(LH_ERR_INVALID_ARGUMENT, "workspace must hold %lld bytes (got %lld)", (long long)need, (long long)(workspace ? workspace_bytes : 0));
  if ((st = check_aligned(workspace, "workspace")) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{free_count, "free_count"}, {new_count, "new_count"}, {offsets, "offsets"}, {block_table, "block_table"}, {lengths, "lengths"}, {new_tokens, "new_tokens"}, {free_pages, "free_pages"}, {slots, "slots"}, {positions, "positions"}, {sequence, "sequence"}, {new_lengths, "new_lengths"}, {need > 0 ? workspace : nullptr, "workspace"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const lh::ExtendView v{block_table, lengths, new_tokens, free_pages, free_count, slots, positions, sequence, offsets, new_lengths, new_count,
                         batch, max_pages, page_size, capacity, max_tokens};
  return launched(lh::launch_extend(v, workspace, reinterpret_cast<hipStream_t>(stream)), "extend launch");
}

lh_status lh_rotary_frequencies(double theta, int64_t rot_dim, lh_rotary_scaling scaling, double factor, int64_t original_context,
                                double low_turns, double high_turns, float* frequencies, float* scale) {
  if (!(theta > 0) || !std::isfinite(theta)) return fail(LH_ERR_INVALID_ARGUMENT, "theta must be positive and finite");
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > 65536) return fail(LH_ERR_INVALID_ARGUMENT, "rot_dim must be an even number up to 65536 (got %lld)", (long long)rot_dim);
  if (scaling != LH_ROTARY_PLAIN && scaling != LH_ROTARY_LINEAR && scaling != LH_ROTARY_BASE && scaling != LH_ROTARY_PARTS)
    return fail(LH_ERR_UNSUPPORTED, "unknown scaling %d", (int)scaling);
  const bool scaled = scaling != LH_ROTARY_PLAIN, parts = scaling == LH_ROTARY_PARTS;
  if (scaled && (!(factor >= 1) || !std::isfinite(factor))) return fail(LH_ERR_INVALID_ARGUMENT, "factor must be at least 1 and finite");
  if (scaling == LH_ROTARY_BASE && rot_dim == 2) return fail(LH_ERR_INVALID_ARGUMENT, "rot_dim must be at least 4 for the base to be scaled");
  if (parts && original_context < 1) return fail(LH_ERR_INVALID_ARGUMENT, "original_context must be positive (got %lld)", (long long)original_context);
  if (parts && (!(low_turns >= 0) || !(high_turns > low_turns) || !std::isfinite(high_turns)))
    return fail(LH_ERR_INVALID_ARGUMENT, "low_turns and high_turns must be an ascending pair of finite numbers >= 0");
  if (!frequencies || !scale) return fail(LH_ERR_INVALID_ARGUMENT, "frequencies and scale are required");
  const double base = scaling == LH_ROTARY_BASE ? theta * std::pow(factor, (double)rot_dim / (double)(rot_dim - 2)) : theta;
  for (int64_t j = 0; j < rot_dim / 2; ++j) {
    double f = std::pow(base, -2.0 * (double)j / (double)rot_dim);
    if (scaling == LH_ROTARY_LINEAR) f /= factor;
    if (parts) {
      const double turns = (double)original_context * f / 6.283185307179586;
      const double keep = std::min(std::max((turns - low_turns) / (high_turns - low_turns), 0.0), 1.0);
      f *= keep + (1.0 - keep) / factor;
    }
    frequencies[j] = (float)f;
  }
  *scale = parts ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return ok();
}

lh_status lh_rotary(const void* Q, int64_t q_stride, int64_t n_q_heads, const void* K, int64_t k_stride, int64_t n_k_heads, lh_dtype dtype,
                    int64_t tokens, int64_t head_dim, int64_t rot_dim, const int32_t* positions, const float* frequencies,
                    int32_t interleaved, int32_t inverse, float scale, void* Q_out, int64_t q_out_stride, void* K_out,
                    int64_t k_out_stride, void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (tokens < 0 || tokens > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "tokens must be in [0, 2^31-1] (got %lld)", (long long)tokens);
  if (head_dim < 1 || head_dim % 16 || head_dim > 65536) return fail(LH_ERR_INVALID_ARGUMENT, "head_dim must be a multiple of 16 up to 65536 (got %lld)", (long long)head_dim);
  if (rot_dim < 2 || rot_dim % 2 || rot_dim > head_dim) return fail(LH_ERR_INVALID_ARGUMENT, "rot_dim must be an even number up to head_dim (got %lld)", (long long)rot_dim);
  const int64_t most = (int64_t(1) << 27) / head_dim;
  if (n_q_heads < 1 || n_q_heads > most || n_k_heads < 0 || n_k_heads > most)
    return fail(LH_ERR_INVALID_ARGUMENT, "n_q_heads must be positive, n_k_heads >= 0, and heads * head_dim at most 2^27");
  if (!std::isfinite(scale)) return fail(LH_ERR_INVALID_ARGUMENT, "scale must be finite");
  lh_status st;
  if ((st = check_stride(q_stride, n_q_heads * head_dim, dtype, "q_stride")) != LH_OK) return st;
  if ((st = check_stride(q_out_stride, n_q_heads * head_dim, dtype, "q_out_stride")) != LH_OK) return st;
  if (n_k_heads > 0) {
    if ((st = check_stride(k_stride, n_k_heads * head_dim, dtype, "k_stride")) != LH_OK) return st;
    if ((st = check_stride(k_out_stride, n_k_heads * head_dim, dtype, "k_out_stride")) != LH_OK) return st;
  } else if (K || K_out) {
    return fail(LH_ERR_INVALID_ARGUMENT, "K and K_out must be NULL without key heads");
  }
  if (Q == Q_out && q_stride != q_out_stride) return fail(LH_ERR_INVALID_ARGUMENT, "in place, q_stride and q_out_stride must be equal");
  if (K && K == K_out && k_stride != k_out_stride) return fail(LH_ERR_INVALID_ARGUMENT, "in place, k_stride and k_out_stride must be equal");
  if (tokens == 0) return ok();
  if (!Q || !Q_out || !positions || !frequencies || (n_k_heads > 0 && (!K || !K_out)))
    return fail(LH_ERR_INVALID_ARGUMENT, "Q, K, Q_out, K_out, positions and frequencies are required");
  for (const PtrCheck& p : {PtrCheck{Q, "Q"}, PtrCheck{K, "K"}, PtrCheck{Q_out, "Q_out"}, PtrCheck{K_out, "K_out"}})
    if ((st = check_aligned(p.p, p.name)) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{Q, "Q"}, {K, "K"}, {Q_out, "Q_out"}, {K_out, "K_out"}, {positions, "positions"}, {frequencies, "frequencies"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  const lh::RotaryView v{Q, K, Q_out, K_out, positions, frequencies, tokens, n_q_heads, n_k_heads, head_dim, rot_dim,
                         q_stride, k_stride, q_out_stride, k_out_stride, scale, interleaved != 0, inverse != 0};
  return launched(lh::launch_rotary(v, dtype == LH_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)), "rotary launch");
}

lh_status lh_route(const void* logits, lh_dtype dtype, int64_t tokens, int64_t n_experts, int64_t topk, int32_t renormalize,
                   float scale, int32_t* ids, float* weights, void* stream) {
  if (!dtype_ok(dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (tokens < 0 || tokens > kMaxInt) return fail(LH_ERR_INVALID_ARGUMENT, "tokens must be in [0, 2^31-1] (got %lld)", (long long)tokens);
  if (n_experts < 1 || n_experts > lh::kMaxExperts) return fail(LH_ERR_INVALID_ARGUMENT, "n_experts must be in [1, 4096] (got %lld)", (long long)n_experts);
  if (topk < 1 || topk > 64 || topk > n_experts) return fail(LH_ERR_INVALID_ARGUMENT, "topk must be in [1, 64] and at most n_experts (got %lld)", (long long)topk);
  if (!std::isfinite(scale)) return fail(LH_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (tokens == 0) return ok();
  if (!logits || !ids || !weights) return fail(LH_ERR_INVALID_ARGUMENT, "logits, ids and weights are required");
  int dev = -1;
  lh_status st = check_pointers({{logits, "logits"}, {ids, "ids"}, {weights, "weights"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  return launched(lh::launch_route(logits, dtype == LH_DTYPE_BF16, tokens, n_experts, topk, renormalize != 0, scale, ids, weights,
                                   reinterpret_cast<hipStream_t>(stream)), "route launch");
}

int64_t lh_moe_workspace(lh_dtype x_dtype, int64_t tokens, int64_t hidden, int64_t inner, int64_t n_experts, int64_t topk) {
  if (x_dtype != LH_DTYPE_E4M3 && !dtype_ok(x_dtype)) {
    (void)fail(LH_ERR_UNSUPPORTED, "unknown dtype %d", (int)x_dtype);
    return 0;
  }
  if (check_moe(tokens, hidden, inner, n_experts, topk) != LH_OK) return 0;
  (void)ok();
  lh::MoeView v{};
  v.x_type = type_of_rows(x_dtype);
  v.tokens = tokens;
  v.hidden = hidden;
  v.inner = inner;
  v.experts = n_experts;
  v.topk = topk;
  return lh::moe_workspace(v);
}

lh_status lh_moe(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t tokens, int64_t hidden, int64_t inner,
                 int64_t n_experts, int64_t topk, const int32_t* ids, const float* weights, const uint8_t* gate_up_code,
                 const uint8_t* gate_up_fp4, const float* gate_up_amax, const uint8_t* down_code, const uint8_t* down_fp4,
                 const float* down_amax, float scale_norm, void* Y, void* workspace, int64_t workspace_bytes, void* stream) {
  lh_status st = check_rows_type(x_dtype, x_scale, x_group, tokens);
  if (st != LH_OK) return st;
  if ((st = check_moe(tokens, hidden, inner, n_experts, topk)) != LH_OK) return st;
  if (!e4m3_value(scale_norm)) return fail(LH_ERR_INVALID_ARGUMENT, "scale_norm must be a positive finite E4M3 value such as 448 or 256 (got %g)", (double)scale_norm);
  if (tokens == 0) return ok();
  if (!X || !ids || !weights || !gate_up_code || !gate_up_fp4 || !gate_up_amax || !down_code || !down_fp4 || !down_amax || !Y)
    return fail(LH_ERR_INVALID_ARGUMENT, "X, ids, weights, gate_up_code, gate_up_fp4, gate_up_amax, down_code, down_fp4, down_amax and Y are required");
  const lh::MoeView v{X, type_of_rows(x_dtype), x_scale, x_group ? (hidden + 127) / 128 : 1, tokens, hidden, inner, n_experts, topk, ids, weights,
                      gate_up_code, gate_up_fp4, gate_up_amax, down_code, down_fp4, down_amax, 6.0f * scale_norm, Y};
  const int64_t need = lh::moe_workspace(v);
  if (!workspace || workspace_bytes < need)
    return fail(LH_ERR_INVALID_ARGUMENT, "workspace must hold %lld bytes (got %lld)", (long long)need, (long long)(workspace ? workspace_bytes : 0));
  for (const PtrCheck& p : {PtrCheck{X, "X"}, PtrCheck{Y, "Y"}, PtrCheck{workspace, "workspace"}})
    if ((st = check_aligned(p.p, p.name)) != LH_OK) return st;
  if (((reinterpret_cast<uintptr_t>(gate_up_fp4) | reinterpret_cast<uintptr_t>(down_fp4)) & 7) != 0)
    return fail(LH_ERR_INVALID_ARGUMENT, "gate_up_fp4 and down_fp4 must be 8-byte aligned");
  int dev = -1;
  st = check_pointers({{X, "X"}, {x_scale, "x_scale"}, {ids, "ids"}, {weights, "weights"}, {gate_up_code, "gate_up_code"}, {gate_up_fp4, "gate_up_fp4"}, {gate_up_amax, "gate_up_amax"}, {down_code, "down_code"}, {down_fp4, "down_fp4"}, {down_amax, "down_amax"}, {Y, "Y"}, {workspace, "workspace"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  return launched(lh::launch_moe(v, workspace, reinterpret_cast<hipStream_t>(stream)), "expert layer launch");
}

int64_t lh_adapter_workspace(int64_t rows, int64_t cin, int64_t n_adapters, int64_t rank) {
  if (check_adapter(rows, cin, 0, n_adapters, rank) != LH_OK) return 0;
  (void)ok();
  lh::AdapterView v{};
  v.rows = rows;
  v.cin = cin;
  v.adapters = n_adapters;
  v.rank = rank;
  return lh::adapter_workspace(v);
}

lh_status lh_adapter(const void* X, lh_dtype x_dtype, const float* x_scale, int64_t x_group, int64_t rows, int64_t cin, int64_t cout,
                     int64_t n_adapters, int64_t rank, const void* A, const void* B, lh_dtype w_dtype, const int32_t* index,
                     const float* scaling, const int32_t* ranks, const void* base, void* Y, void* workspace, int64_t workspace_bytes,
                     void* stream) {
  lh_status st = check_rows_type(x_dtype, x_scale, x_group, rows);
  if (st != LH_OK) return st;
  if (!dtype_ok(w_dtype)) return fail(LH_ERR_UNSUPPORTED, "unknown dtype %d of A and B", (int)w_dtype);
  if ((st = check_adapter(rows, cin, cout, n_adapters, rank)) != LH_OK) return st;
  if (rows == 0 || cout == 0) return ok();
  if (!X || !A || !B || !index || !base || !Y) return fail(LH_ERR_INVALID_ARGUMENT, "X, A, B, index, base and Y are required");
  const lh::AdapterView v{X, type_of_rows(x_dtype), x_scale, x_group ? (cin + 127) / 128 : 1, rows, cin, cout, n_adapters, rank, A, B,
                          w_dtype == LH_DTYPE_F32, index, scaling, ranks, base, Y};
  const int64_t need = lh::adapter_workspace(v);
  if (!workspace || workspace_bytes < need)
    return fail(LH_ERR_INVALID_ARGUMENT, "workspace must hold %lld bytes (got %lld)", (long long)need, (long long)(workspace ? workspace_bytes : 0));
  for (const PtrCheck& p : {PtrCheck{X, "X"}, PtrCheck{A, "A"}, PtrCheck{B, "B"}, PtrCheck{base, "base"}, PtrCheck{Y, "Y"}, PtrCheck{workspace, "workspace"}})
    if ((st = check_aligned(p.p, p.name)) != LH_OK) return st;
  int dev = -1;
  st = check_pointers({{X, "X"}, {x_scale, "x_scale"}, {A, "A"}, {B, "B"}, {index, "index"}, {scaling, "scaling"}, {ranks, "ranks"}, {base, "base"}, {Y, "Y"}, {workspace, "workspace"}}, &dev);
  if (st != LH_OK) return st;
  DeviceGuard guard;
  if ((st = guard.enter(dev)) != LH_OK) return st;
  return launched(lh::launch_adapter(v, workspace, reinterpret_cast<hipStream_t>(stream)), "adapter launch");
}

}  // extern "C"
