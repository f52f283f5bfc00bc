// Internal declarations shared by the C-ABI shim and the kernel translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace lh {

// The runtime takes fewer than 2^32 work-items a launch.
inline bool launch_fits(dim3 grid, dim3 block) { return (uint64_t)grid.x * block.x < (uint64_t(1) << 32); }

// kernel(args) on the stream and its launch status; hipErrorInvalidConfiguration for one that does not fit.  hipLaunchKernel itself: the <<<>>> form passes
// the grid through two more runtime calls (2.25 us of the host against 2.45).
template <class A>
inline hipError_t launch_kernel(void (*kernel)(A), dim3 grid, dim3 block, size_t lds, hipStream_t stream, A args) {
  if (!launch_fits(grid, block)) return hipErrorInvalidConfiguration;
  void* list[] = {&args};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, list, lds, stream);
}

// Scratch of one launch_accumulate call: a work area (partial sums of row ranges that are added
// across workgroups) and arrival counters.  The counters must be
// zero when a call starts and are zero again when it ends.  launch_accumulate checks the sizes it
// is given against this and launches nothing if they are short.
struct AccScratch {
  size_t work_bytes;
  size_t counters;
};
AccScratch accumulate_scratch(int64_t rows, int64_t nb, const int64_t* offsets, int64_t n_groups,
                              bool bf16, bool act_aware, bool imp_only);

// Sets n words at p to zero (a kernel, so that graph capture records no memset node).
hipError_t launch_zero_fill(unsigned* p, size_t n, hipStream_t stream);

hipError_t launch_absmax(const void* W, bool bf16, int64_t n_groups, int64_t elems, float* amax,
                         hipStream_t stream);

// Activation-aware: X and Xq given, or X and x_amax (X_q made from X in the kernel, Xq ==
// nullptr); H and P required.  Otherwise Xq == x_amax == nullptr and H and/or imp given.
hipError_t launch_accumulate(const void* X, const void* Xq, const float* x_amax, bool bf16,
                             int64_t rows, int64_t cin, const int64_t* offsets, int64_t n_groups,
                             float beta, float* H, float* P, float* imp, void* work,
                             size_t work_bytes, unsigned* counters, size_t n_counters,
                             hipStream_t stream);

// X_q = the activations' NVFP4 fake-quant (the one the FQ accumulation applies), written to Xq.
hipError_t launch_act_fake_quant(const void* X, bool bf16, int64_t rows, int64_t cin, const int64_t* offsets,
                                 int64_t n_groups, const float* x_amax, void* Xq, hipStream_t stream);

// Options of one sweep launch, passed to the kernels by value: the divisor of the global scale,
// g = fp32(amax / gdiv) with gdiv = 6 * norm (norm an E4M3 value, so gdiv is exact in fp32), and
// the amax-multiplier grid (nm = 0: every one of the 126 candidates; otherwise a block takes only
// the codes its nm multipliers propose).
constexpr int kMaxMultipliers = 128;
struct SweepOpts {
  float gdiv;
  int nm;
  float mult[kMaxMultipliers];
};

// mu: device scratch of n_groups * cin/16 floats (each block column's Hessian eigenvalue bound,
// written and read by the launch).
hipError_t launch_sweep(const void* W, bool bf16, int64_t n_groups, int64_t cout, int64_t cin,
                        const float* amax, const float* H, const float* P, uint8_t* code,
                        uint8_t* fp4, float* loss, const SweepOpts& opts, float* mu, hipStream_t stream);

hipError_t launch_sweep_diag(const void* W, bool bf16, int64_t n_groups, int64_t cout,
                             int64_t cin, const float* amax, const float* imp, uint8_t* code,
                             uint8_t* fp4, float* loss, const SweepOpts& opts, hipStream_t stream);

// Hessians of grouped rows (n_groups >= 1, offsets device int64[n_groups+1] or NULL for one
// group) made in LDS and swept at once; outputs as launch_sweep with P = NULL.  cout <= kFusedMaxCout.
constexpr int kFusedMaxCout = 8192;
hipError_t launch_accumulate_sweep(const void* X, const void* W, bool bf16, int64_t rows, int64_t cin,
                                   const int64_t* offsets, int64_t n_groups, int64_t cout, const float* amax,
                                   uint8_t* code, uint8_t* fp4, float* loss, const SweepOpts& opts,
                                   hipStream_t stream);

// Wq (bf16 or fp32, may be NULL) and block_amax (may be NULL) from scale codes and FP4 nibbles;
// g = fp32(amax / gdiv) as in the sweep.
hipError_t launch_dequantize(const uint8_t* code, const uint8_t* fp4, const float* amax, int64_t n_groups,
                             int64_t cout, int64_t cin, bool bf16, void* Wq, float* block_amax, float gdiv,
                             hipStream_t stream);

// h = round(x + r) (x without r), its RMS norm times gamma as E4M3 q and scales s: one per row, or
// one per 128 channels (grouped).  r and h are both given or both NULL; h may be x or r.
hipError_t launch_rms_norm(const void* x, const void* r, bool bf16, int64_t rows, int64_t cin, const void* gamma,
                           float eps, bool grouped, void* h, uint8_t* q, float* s, hipStream_t stream);

// y[t] = W_g x[t] for the rows t of each group; x_type 0 bf16, 1 fp32, 2 E4M3 with x_scales scales a
// row; y is fp32 for fp32 x, otherwise bf16.  offsets NULL with one group.
hipError_t launch_matvec(const void* x, int x_type, const float* x_scale, int64_t x_scales, int64_t rows, int64_t cin,
                         int64_t cout, const int64_t* offsets, int64_t n_groups, const uint8_t* code, const uint8_t* fp4,
                         const float* amax, float gdiv, void* y, hipStream_t stream);

// Global scale of one key-value head from its amax.  A product with the rounded reciprocal, as GPU
// tensor libraries evaluate amax / 448 and amax / 2688, so codes made there by that rule are the
// same bits.
__host__ __device__ inline float cache_unit(float amax, bool four) {
  return amax * (four ? 1.0f / 2688.0f : 1.0f / 448.0f);
}

// A paged key-value cache (four: NVFP4 codes with block scales, otherwise E4M3).
struct CacheView {
  uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_amax, *v_amax;
  int64_t n_pages, page_size, heads, dim;
  bool four;
};
hipError_t launch_cache_write(const CacheView& c, const void* k, const void* v, bool bf16, int64_t tokens,
                              int64_t k_stride, int64_t v_stride, const int64_t* slots, hipStream_t stream);
hipError_t launch_cache_read(const CacheView& c, const int64_t* slots, int64_t tokens, void* k, void* v, bool bf16,
                             hipStream_t stream);

// Tokens of a sequence that attention takes at most: its positions are 32-bit, and a wave looks up to a step past
// the last one.
constexpr int64_t kMaxContext = (int64_t(1) << 31) - 4096;

// Attention of one token per sequence; `share` query heads per key-value head.  attention_grid is
// the launch's workgroups, attention_workspace its scratch in bytes (0: none).
int64_t attention_grid(const CacheView& c, int64_t batch, int64_t share, int64_t width);
int64_t attention_workspace(const CacheView& c, int64_t batch, int64_t share, int64_t width);
hipError_t launch_attention(const CacheView& c, const void* q, bool bf16, int64_t batch, int64_t share, int64_t q_stride,
                            const int* table, int64_t width, const int* lengths, float scale, void* o, void* work,
                            hipStream_t stream);

// Growth of a paged cache's sequences (lh_cache_extend): pointers and sizes as there, asked may be NULL.
// extend_workspace is the scratch in bytes (0: none).
struct ExtendView {
  int* table;
  const int *lengths, *asked;
  int* stack;
  const int* count;
  int64_t* slots;
  int *positions, *sequence, *offsets, *new_lengths, *new_count;
  int64_t batch, width, page, capacity, rows;
};
int64_t extend_workspace(int64_t batch, int64_t rows);
hipError_t launch_extend(const ExtendView& v, void* work, hipStream_t stream);

// Rotary positions of q (and k with k_heads > 0) into qo, ko, which may be q and k.
struct RotaryView {
  const void *q, *k;
  void *qo, *ko;
  const int* positions;
  const float* frequencies;
  int64_t tokens, q_heads, k_heads, dim, rot, q_stride, k_stride, qo_stride, ko_stride;
  float scale;
  bool interleaved, inverse;
};
hipError_t launch_rotary(const RotaryView& v, bool bf16, hipStream_t stream);

// The topk largest logits of each token and their softmax weights; experts <= kMaxExperts, topk <= 64.
constexpr int64_t kMaxExperts = 4096;
hipError_t launch_route(const void* logits, bool bf16, int64_t tokens, int64_t experts, int64_t topk, bool renormalize,
                        float scale, int* ids, float* weights, hipStream_t stream);

// The expert layer (lh_moe): x_type as launch_matvec, gdiv the divisor of the global scales.  moe_workspace is its scratch in bytes.
struct MoeView {
  const void* x;
  int x_type;
  const float* x_scale;
  int64_t x_scales, tokens, hidden, inner, experts, topk;
  const int* ids;
  const float* weights;
  const uint8_t *gate_up_code, *gate_up_fp4;
  const float* gate_up_amax;
  const uint8_t *down_code, *down_fp4;
  const float* down_amax;
  float gdiv;
  void* y;
};
int64_t moe_workspace(const MoeView& v);
hipError_t launch_moe(const MoeView& v, void* work, hipStream_t stream);

// Low-rank adapters (lh_adapter): x_type as launch_matvec, w_f32 the type of a and b; scaling and ranks may be NULL, y may be base.
// adapter_workspace is its scratch in bytes.
struct AdapterView {
  const void* x;
  int x_type;
  const float* x_scale;
  int64_t x_scales, rows, cin, cout, adapters, rank;
  const void *a, *b;
  bool w_f32;
  const int* index;
  const float* scaling;
  const int* ranks;
  const void* base;
  void* y;
};
int64_t adapter_workspace(const AdapterView& v);
hipError_t launch_adapter(const AdapterView& v, void* work, hipStream_t stream);

}  // namespace lh
