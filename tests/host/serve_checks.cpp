// Host-side checks of the operators around a decode step, built with AddressSanitizer and UndefinedBehaviorSanitizer on the
// host code (tests/test_serve_abi.py): every argument check that needs no GPU.  Each call must return the documented
// code with a message and launch nothing.
#include <cmath>
#include <cstdio>
#include <cstring>

#include "../../include/lh.h"
#include "../../nvfp4_scale_calibration_lh_amd/csrc/lh_host.hpp"

extern "C" const char* lh_last_error(void) { return lh::host::g_last_error; }

static int failures = 0;

static void expect(lh_status got, lh_status want, const char* what, const char* needle = nullptr) {
  const char* msg = lh_last_error();
  const bool ok = got == want && (!needle || std::strstr(msg, needle) != nullptr) && (want == LH_OK ? msg[0] == 0 : msg[0] != 0);
  if (!ok) {
    std::fprintf(stderr, "FAIL %s: got %d (%s), want %d%s%s\n", what, (int)got, msg, (int)want, needle ? " with " : "", needle ? needle : "");
    ++failures;
  }
}
static void holds(bool b, const char* what) {
  if (!b) std::fprintf(stderr, "FAIL %s\n", what), ++failures;
}

int main() {
  alignas(16) static unsigned char host[1 << 12];        // host memory: never a valid device pointer
  void* h = host;
  float* f = reinterpret_cast<float*>(host);
  uint8_t* b = host;
  int64_t* l = reinterpret_cast<int64_t*>(host);
  int32_t* i = reinterpret_cast<int32_t*>(host);
  const lh_dtype F32 = LH_DTYPE_F32, BF = LH_DTYPE_BF16, F8 = LH_DTYPE_E4M3, BAD = static_cast<lh_dtype>(9);
  const lh_status INV = LH_ERR_INVALID_ARGUMENT, UNS = LH_ERR_UNSUPPORTED;
  const int64_t HUGE = INT64_MAX, LOTS = int64_t(1) << 40;

  // growth of the cache's sequences
  auto ex = [&](int32_t* table, int64_t batch, int64_t pages, int64_t page, int32_t* lens, int32_t* stack, int64_t cap, int32_t* count, int64_t rows,
                int64_t* slots, int32_t* offsets, void* work, int64_t bytes) {
    return lh_cache_extend(table, batch, pages, page, lens, nullptr, stack, cap, count, rows, slots, i, i, offsets, i, i, work, bytes, nullptr);
  };
  expect(ex(i, -1, 4, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend batch", "batch");
  expect(ex(i, HUGE, 4, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend many", "batch");
  expect(ex(i, 2, 4, 0, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend page", "page_size");
  expect(ex(i, 2, 4, HUGE, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend large page", "page_size");
  expect(ex(i, 2, -1, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend pages", "max_pages");
  expect(ex(i, 2, HUGE, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend many pages", "max_pages");
  expect(ex(i, 2, (int64_t(1) << 27) - 256 + 1, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend one page too many", "max_pages");
  expect(ex(i, 2, (int64_t(1) << 27) - 256, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend the most pages", "device");
  expect(ex(i, 2, 4, 16, i, i, 8, i, -1, l, i, nullptr, 0), INV, "extend rows", "max_tokens");
  expect(ex(i, 2, 4, 16, i, i, 8, i, LOTS, l, i, h, HUGE), INV, "extend many rows", "max_tokens");
  expect(ex(i, 2, 4, 16, i, i, -1, i, 8, l, i, nullptr, 0), INV, "extend capacity", "capacity");
  expect(ex(i, 2, 4, 16, i, i, LOTS, i, 8, l, i, nullptr, 0), INV, "extend large capacity", "capacity");
  expect(ex(nullptr, 2, 4, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend table", "required");
  expect(ex(i, 2, 4, 16, nullptr, i, 8, i, 8, l, i, nullptr, 0), INV, "extend lengths", "required");
  expect(ex(i, 2, 4, 16, i, nullptr, 8, i, 8, l, i, nullptr, 0), INV, "extend stack", "required");
  expect(ex(i, 2, 4, 16, i, i, 8, nullptr, 8, l, i, nullptr, 0), INV, "extend count", "required");
  expect(ex(i, 2, 4, 16, i, i, 8, i, 8, nullptr, i, nullptr, 0), INV, "extend slots", "required");
  expect(ex(i, 2, 4, 16, i, i, 8, i, 8, l, nullptr, nullptr, 0), INV, "extend offsets", "required");
  const int64_t need = lh_cache_extend_workspace(5000, 100);
  holds(need > 0 && lh_cache_extend_workspace(64, 64) == 0, "extend workspace sizes");
  holds(lh_cache_extend_workspace(-1, 8) == 0 && lh_cache_extend_workspace(8, LOTS) == 0, "extend workspace of what is refused");
  expect(ex(i, 5000, 4, 16, i, i, 8, i, 100, l, i, nullptr, 0), INV, "extend workspace", "workspace");
  expect(ex(i, 5000, 4, 16, i, i, 8, i, 100, l, i, h, need - 1), INV, "extend short workspace", "workspace");
  expect(ex(i, 5000, 4, 16, i, i, 8, i, 100, l, i, host + 8, need), INV, "extend workspace aligned", "aligned");
  expect(ex(i, 2, 4, 16, i, i, 8, i, 8, l, i, nullptr, 0), INV, "extend host", "device");

  // frequencies
  float out[8], s = 0;
  auto fr = [&](double theta, int64_t rot, lh_rotary_scaling sc, double factor, int64_t context, double lo, double hi, float* to, float* scale) {
    return lh_rotary_frequencies(theta, rot, sc, factor, context, lo, hi, to, scale);
  };
  expect(fr(10000, 16, LH_ROTARY_PLAIN, NAN, 0, 0, 0, out, &s), LH_OK, "frequencies");
  holds(out[0] == 1.0f && s == 1.0f && std::fabs(out[4] - 0.01f) < 1e-8f, "plain frequencies");
  expect(fr(10000, 16, LH_ROTARY_LINEAR, 4, 0, 0, 0, out, &s), LH_OK, "linear");
  holds(out[0] == 0.25f && s == 1.0f, "linear frequencies");
  expect(fr(10000, 16, LH_ROTARY_BASE, 8, 0, 0, 0, out, &s), LH_OK, "base");
  holds(out[0] == 1.0f && std::fabs(out[7] * std::pow(10000.0, 0.875) - 0.125) < 1e-6, "the slowest angle of a scaled base");
  expect(fr(10000, 16, LH_ROTARY_PARTS, 8, 4096, 1, 32, out, &s), LH_OK, "parts");
  holds(out[0] == 1.0f && std::fabs(out[7] * std::pow(10000.0, 0.875) - 0.125) < 1e-6 && std::fabs(s - 1.2079442f) < 1e-6f, "frequencies in parts");
  expect(fr(0, 16, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "theta", "theta");
  expect(fr(NAN, 16, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "theta NaN", "theta");
  expect(fr(INFINITY, 16, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "theta inf", "theta");
  expect(fr(1e4, 15, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "odd", "rot_dim");
  expect(fr(1e4, 0, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "none", "rot_dim");
  expect(fr(1e4, HUGE - 1, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, &s), INV, "large", "rot_dim");
  expect(fr(1e4, 16, static_cast<lh_rotary_scaling>(4), 1, 0, 0, 0, out, &s), UNS, "scaling", "scaling");
  expect(fr(1e4, 16, LH_ROTARY_LINEAR, 0.5, 0, 0, 0, out, &s), INV, "factor", "factor");
  expect(fr(1e4, 16, LH_ROTARY_LINEAR, NAN, 0, 0, 0, out, &s), INV, "factor NaN", "factor");
  expect(fr(1e4, 2, LH_ROTARY_BASE, 2, 0, 0, 0, out, &s), INV, "base of one pair", "rot_dim");
  expect(fr(1e4, 16, LH_ROTARY_PARTS, 2, 0, 1, 32, out, &s), INV, "context", "original_context");
  expect(fr(1e4, 16, LH_ROTARY_PARTS, 2, 64, 32, 32, out, &s), INV, "turns", "turns");
  expect(fr(1e4, 16, LH_ROTARY_PARTS, 2, 64, NAN, 32, out, &s), INV, "turns NaN", "turns");
  expect(fr(1e4, 16, LH_ROTARY_PARTS, 2, 64, 1, INFINITY, out, &s), INV, "turns inf", "turns");
  expect(fr(1e4, 16, LH_ROTARY_PLAIN, 1, 0, 0, 0, nullptr, &s), INV, "frequencies NULL", "required");
  expect(fr(1e4, 16, LH_ROTARY_PLAIN, 1, 0, 0, 0, out, nullptr), INV, "scale NULL", "required");

  // rotary positions
  auto ro = [&](const void* q, int64_t qs, int64_t nq, const void* k, int64_t ks, int64_t nk, lh_dtype t, int64_t tokens, int64_t dim, int64_t rot,
                float scale, void* qo, int64_t qos, void* ko, int64_t kos) {
    return lh_rotary(q, qs, nq, k, ks, nk, t, tokens, dim, rot, i, f, 0, 0, scale, qo, qos, ko, kos, nullptr);
  };
  expect(ro(h, 256, 4, h, 128, 2, F8, 3, 64, 64, 1, h, 256, h, 128), UNS, "rotary dtype", "dtype");
  expect(ro(h, 256, 4, h, 128, 2, BF, -3, 64, 64, 1, h, 256, h, 128), INV, "rotary tokens", "tokens");
  expect(ro(h, 256, 4, h, 128, 2, BF, LOTS, 64, 64, 1, h, 256, h, 128), INV, "rotary many tokens", "tokens");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 56, 56, 1, h, 256, h, 128), INV, "rotary dim", "head_dim");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 63, 1, h, 256, h, 128), INV, "rotary odd", "rot_dim");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 66, 1, h, 256, h, 128), INV, "rotary past the head", "rot_dim");
  expect(ro(h, 256, 0, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary heads", "n_q_heads");
  expect(ro(h, 256, 4, h, 128, -2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary key heads", "n_k_heads");
  expect(ro(h, 256, HUGE / 32, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary many heads", "2^27");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 64, NAN, h, 256, h, 128), INV, "rotary scale", "scale");
  expect(ro(h, 255, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary q stride", "q_stride");
  expect(ro(h, 260, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary q stride aligned", "q_stride");
  expect(ro(h, 256, 4, h, 64, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary k stride", "k_stride");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 128, h, 128), INV, "rotary q out", "q_out_stride");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 64), INV, "rotary k out", "k_out_stride");
  expect(ro(h, 256, 4, h, 0, 0, BF, 3, 64, 64, 1, h, 256, nullptr, 0), INV, "rotary k without heads", "NULL");
  expect(ro(h, 256, 4, nullptr, 0, 0, BF, 3, 64, 64, 1, h, 264, nullptr, 0), INV, "rotary in place strides", "equal");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, host + 16, 256, h, 136), INV, "rotary k in place strides", "equal");
  expect(ro(nullptr, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary Q", "required");
  expect(ro(h, 256, 4, nullptr, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary K", "required");
  expect(ro(host + 8, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary aligned", "aligned");
  expect(ro(h, 256, 4, h, 128, 2, BF, 3, 64, 64, 1, h, 256, h, 128), INV, "rotary host", "device");
  expect(ro(nullptr, 256, 4, nullptr, 0, 0, F32, 0, 64, 64, 1, nullptr, 256, nullptr, 0), LH_OK, "rotary no tokens");

  // the choice of experts
  auto rt = [&](const void* x, lh_dtype t, int64_t tokens, int64_t experts, int64_t k, float scale, int32_t* ids) {
    return lh_route(x, t, tokens, experts, k, 1, scale, ids, f, nullptr);
  };
  expect(rt(h, F8, 4, 16, 2, 1, i), UNS, "route dtype", "dtype");
  expect(rt(h, BF, -4, 16, 2, 1, i), INV, "route tokens", "tokens");
  expect(rt(h, BF, 4, 0, 2, 1, i), INV, "route experts", "n_experts");
  expect(rt(h, BF, 4, 4097, 2, 1, i), INV, "route many experts", "n_experts");
  expect(rt(h, BF, 4, 16, 0, 1, i), INV, "route topk", "topk");
  expect(rt(h, BF, 4, 16, 17, 1, i), INV, "route large topk", "topk");
  expect(rt(h, BF, 4, 160, 65, 1, i), INV, "route topk over 64", "topk");
  expect(rt(h, BF, 4, 16, 2, INFINITY, i), INV, "route scale", "scale");
  expect(rt(nullptr, BF, 4, 16, 2, 1, i), INV, "route logits", "required");
  expect(rt(h, BF, 4, 16, 2, 1, nullptr), INV, "route ids", "required");
  expect(rt(h, BF, 4, 16, 2, 1, i), INV, "route host", "device");
  expect(rt(nullptr, F32, 0, 16, 2, 1, nullptr), LH_OK, "route no tokens");

  // the expert layer
  auto mo = [&](const void* x, lh_dtype t, const float* xs, int64_t xg, int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int64_t k,
                const int32_t* ids, const uint8_t* fp4, float norm, void* y, void* work, int64_t bytes) {
    return lh_moe(x, t, xs, xg, tokens, hidden, inner, experts, k, ids, f, b, fp4, f, b, b, f, norm, y, work, bytes, nullptr);
  };
  expect(mo(h, BAD, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), UNS, "moe dtype", "dtype");
  expect(mo(h, BF, f, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe scale of bf16", "x_scale");
  expect(mo(h, F8, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe no scale", "x_scale");
  expect(mo(h, F8, f, 64, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe group", "x_group");
  expect(mo(h, BF, nullptr, 128, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe group of bf16", "x_group");
  expect(mo(h, BF, nullptr, 0, -4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe tokens", "tokens");
  expect(mo(h, BF, nullptr, 0, 4194241, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe many tokens", "tokens");
  expect(mo(h, BF, nullptr, 0, 4, 72, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe hidden", "hidden");
  expect(mo(h, BF, nullptr, 0, 4, 64, 40, 8, 2, i, b, 448, h, h, HUGE), INV, "moe inner", "inner");
  expect(mo(h, BF, nullptr, 0, 4, HUGE - 15, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe large hidden", "hidden");
  expect(mo(h, BF, nullptr, 0, 4, 1 << 20, 1 << 14, 8, 2, i, b, 448, h, h, HUGE), INV, "moe large matrices", "2^32");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 0, 2, i, b, 448, h, h, HUGE), INV, "moe experts", "n_experts");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 4097, 2, i, b, 448, h, h, HUGE), INV, "moe many experts", "n_experts");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 0, i, b, 448, h, h, HUGE), INV, "moe topk", "topk");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 65, i, b, 448, h, h, HUGE), INV, "moe large topk", "topk");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 300, h, h, HUGE), INV, "moe norm", "scale_norm");
  expect(mo(nullptr, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, HUGE), INV, "moe X", "required");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, nullptr, b, 448, h, h, HUGE), INV, "moe ids", "required");
  const int64_t mw = lh_moe_workspace(BF, 4, 64, 32, 8, 2);
  holds(mw > 0 && lh_moe_workspace(F32, 4, 64, 32, 8, 2) >= mw, "moe workspace sizes");
  holds(lh_moe_workspace(BF, 4, 60, 32, 8, 2) == 0, "moe workspace of what is refused");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, mw - 1), INV, "moe short workspace", "workspace");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, nullptr, mw), INV, "moe workspace", "workspace");
  expect(mo(host + 8, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, mw), INV, "moe X aligned", "aligned");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, host + 4, h, mw), INV, "moe Y aligned", "aligned");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b + 4, 448, h, h, mw), INV, "moe fp4 aligned", "aligned");
  expect(mo(h, BF, nullptr, 0, 4, 64, 32, 8, 2, i, b, 448, h, h, mw), INV, "moe host", "device");
  expect(mo(nullptr, F8, nullptr, 0, 0, 64, 32, 8, 2, nullptr, b, 448, nullptr, nullptr, 0), LH_OK, "moe no tokens");

  // adapters
  auto ad = [&](const void* x, lh_dtype t, const float* xs, int64_t xg, int64_t rows, int64_t cin, int64_t cout, int64_t n, int64_t rank, const void* a,
                lh_dtype wt, const int32_t* index, const void* base, void* y, void* work, int64_t bytes) {
    return lh_adapter(x, t, xs, xg, rows, cin, cout, n, rank, a, h, wt, index, nullptr, nullptr, base, y, work, bytes, nullptr);
  };
  expect(ad(h, BAD, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), UNS, "adapter dtype", "dtype");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, F8, i, h, h, h, HUGE), UNS, "adapter weights", "dtype");
  expect(ad(h, F8, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter no scale", "x_scale");
  expect(ad(h, F8, f, 16, 4, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter group", "x_group");
  expect(ad(h, BF, nullptr, 0, -4, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter rows", "rows");
  expect(ad(h, BF, nullptr, 0, 4194241, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter many rows", "rows");
  expect(ad(h, BF, nullptr, 0, 4, 60, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter cin", "cin");
  expect(ad(h, BF, nullptr, 0, 4, 64, -8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter cout", "cout");
  expect(ad(h, BF, nullptr, 0, 4, 64, HUGE, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter large cout", "cout");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 0, 16, h, BF, i, h, h, h, HUGE), INV, "adapter none", "n_adapters");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 4097, 16, h, BF, i, h, h, h, HUGE), INV, "adapter many", "n_adapters");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 12, h, BF, i, h, h, h, HUGE), INV, "adapter rank", "rank");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 264, h, BF, i, h, h, h, HUGE), INV, "adapter large rank", "rank");
  expect(ad(nullptr, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, HUGE), INV, "adapter X", "required");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, nullptr, BF, i, h, h, h, HUGE), INV, "adapter A", "required");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, nullptr, h, h, h, HUGE), INV, "adapter index", "required");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, nullptr, h, h, HUGE), INV, "adapter base", "required");
  const int64_t aw = lh_adapter_workspace(4, 64, 2, 16);
  holds(aw > 0 && lh_adapter_workspace(4, 64, 2, 12) == 0, "adapter workspace sizes");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, aw - 1), INV, "adapter short workspace", "workspace");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, nullptr, aw), INV, "adapter workspace", "workspace");
  expect(ad(host + 8, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, aw), INV, "adapter X aligned", "aligned");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, host + 8, h, h, aw), INV, "adapter base aligned", "aligned");
  expect(ad(h, BF, nullptr, 0, 4, 64, 8, 2, 16, h, BF, i, h, h, h, aw), INV, "adapter host", "device");
  expect(ad(nullptr, BF, nullptr, 0, 0, 64, 8, 2, 16, nullptr, BF, nullptr, nullptr, nullptr, nullptr, 0), LH_OK, "adapter no rows");
  expect(ad(nullptr, BF, nullptr, 0, 4, 64, 0, 2, 16, nullptr, BF, nullptr, nullptr, nullptr, nullptr, 0), LH_OK, "adapter no channels");

  std::printf(failures ? "%d failures\n" : "ok: %d failures\n", failures);
  return failures != 0;
}
