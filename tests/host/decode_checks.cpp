// Host-side checks of the decode-step entry points, built with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code (tests/test_decode_abi.py): every argument check that
// needs no GPU.  Each call must return the documented code with a message and launch nothing.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <vector>

#include "../../include/lh.h"

static int failures = 0;

static void expect(lh_status got, lh_status want, const char* what, const char* needle = nullptr) {
  const char* msg = lh_last_error();
  const bool ok = got == want && (!needle || std::strstr(msg, needle) != nullptr) && (want == LH_OK ? msg[0] == 0 : msg[0] != 0);
  if (!ok) {
    std::fprintf(stderr, "FAIL %s: got %d (%s), want %d%s%s\n", what, (int)got, msg, (int)want, needle ? " with " : "",
                 needle ? needle : "");
    ++failures;
  }
}

int main() {
  alignas(16) static unsigned char host[1 << 12];        // host memory: never a valid device pointer
  void* h = host;
  float* hf = reinterpret_cast<float*>(host);
  uint8_t* hb = host;
  int64_t* ho = reinterpret_cast<int64_t*>(host);
  int32_t* hi = reinterpret_cast<int32_t*>(host);
  const lh_dtype BF = LH_DTYPE_BF16, F8 = LH_DTYPE_E4M3, BAD = static_cast<lh_dtype>(9);
  const lh_status INV = LH_ERR_INVALID_ARGUMENT, UNS = LH_ERR_UNSUPPORTED;
  const int64_t HUGE = INT64_MAX;

  // norm
  expect(lh_rms_norm_quant(h, nullptr, F8, 4, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), UNS, "norm E4M3 input", "dtype");
  expect(lh_rms_norm_quant(h, nullptr, BAD, 4, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), UNS, "norm dtype", "dtype");
  expect(lh_rms_norm_quant(h, nullptr, BF, -1, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm rows", "rows");
  expect(lh_rms_norm_quant(h, nullptr, BF, HUGE, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm many rows", "rows");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 40, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm cin", "cin");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, HUGE - 15, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm long rows", "cin");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, 0.f, 32, nullptr, hb, hf, nullptr), INV, "norm group", "group");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, -1.f, 0, nullptr, hb, hf, nullptr), INV, "norm eps", "eps");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, NAN, 0, nullptr, hb, hf, nullptr), INV, "norm eps NaN", "eps");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, INFINITY, 0, nullptr, hb, hf, nullptr), INV, "norm eps inf", "eps");
  expect(lh_rms_norm_quant(h, h, BF, 4, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm R alone", "together");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, 0.f, 0, h, hb, hf, nullptr), INV, "norm summed alone", "together");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, nullptr, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm gamma", "gamma");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, 0.f, 0, nullptr, nullptr, hf, nullptr), INV, "norm q", "required");
  expect(lh_rms_norm_quant(host + 8, nullptr, BF, 4, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm aligned", "aligned");
  expect(lh_rms_norm_quant(h, nullptr, BF, 4, 64, h, 0.f, 0, nullptr, hb, hf, nullptr), INV, "norm host", "device");
  expect(lh_rms_norm_quant(nullptr, nullptr, BF, 0, 64, h, 0.f, 0, nullptr, nullptr, nullptr, nullptr), LH_OK, "norm no rows");

  // products
  auto mv = [&](const void* x, lh_dtype t, const float* xs, int64_t xg, int64_t rows, int64_t cin, const int64_t* off, int64_t G,
                int64_t cout, const uint8_t* fp4, float norm) {
    return lh_matvec(x, t, xs, xg, rows, cin, off, G, cout, hb, fp4, hf, norm, h, nullptr);
  };
  expect(mv(h, BAD, nullptr, 0, 4, 64, nullptr, 1, 8, hb, 448.f), UNS, "matvec dtype", "dtype");
  expect(mv(h, BF, nullptr, 0, -4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec rows", "rows");
  expect(mv(h, BF, nullptr, 0, 4, 72, nullptr, 1, 8, hb, 448.f), INV, "matvec cin", "cin");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 0, 8, hb, 448.f), INV, "matvec groups", "n_groups");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 2, 8, hb, 448.f), INV, "matvec offsets", "group_offsets");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, -8, hb, 448.f), INV, "matvec cout", "cout");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, HUGE, hb, 448.f), INV, "matvec large cout", "cout");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, 8, hb, 300.f), INV, "matvec norm", "scale_norm");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, 8, hb, NAN), INV, "matvec norm NaN", "scale_norm");
  expect(mv(h, BF, hf, 0, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec scale of bf16", "x_scale");
  expect(mv(h, F8, nullptr, 0, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec no scale", "x_scale");
  expect(mv(h, BF, nullptr, 128, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec group of bf16", "x_group");
  expect(mv(h, F8, hf, 64, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec group", "x_group");
  expect(mv(h, BF, nullptr, 0, 2147483647, 64, nullptr, 1, 1 << 20, hb, 448.f), INV, "matvec launch", "too many rows");
  expect(mv(nullptr, BF, nullptr, 0, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec X", "required");
  expect(mv(host + 8, BF, nullptr, 0, 4, 64, nullptr, 1, 8, hb, 448.f), INV, "matvec X aligned", "aligned");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, 8, hb + 4, 448.f), INV, "matvec fp4 aligned", "aligned");
  expect(mv(h, BF, nullptr, 0, 4, 64, ho, 2, 8, hb, 256.f), INV, "matvec host", "device");
  expect(mv(nullptr, F8, nullptr, 0, 0, 64, nullptr, 1, 8, hb, 448.f), LH_OK, "matvec no rows");
  expect(mv(h, BF, nullptr, 0, 4, 64, nullptr, 1, 0, hb, 448.f), LH_OK, "matvec no channels");

  // the cache
  const lh_cache good{LH_CACHE_FP4, 4, 16, 2, 64, hb, hb, hb, hb, hf, hf};
  auto write = [&](const lh_cache* c, lh_dtype t = LH_DTYPE_BF16, int64_t ks = 128, int64_t vs = 128, int64_t n = 3) {
    return lh_cache_write(c, h, ks, h, vs, t, n, ho, nullptr);
  };
  expect(write(nullptr), INV, "no cache", "cache");
  expect(write(&good, F8), UNS, "cache E4M3 input", "dtype");
  lh_cache c = good;
  c.format = static_cast<lh_cache_format>(5);
  expect(write(&c), UNS, "cache format", "format");
  for (int k = 0; k < 4; ++k)
    for (int64_t bad : {int64_t(0), int64_t(-3)}) {
      c = good;
      (k == 0 ? c.n_pages : k == 1 ? c.page_size : k == 2 ? c.n_heads : c.head_dim) = bad;
      expect(write(&c), INV, "cache size", "positive");
    }
  c = good, c.head_dim = 72;
  expect(write(&c), INV, "cache head_dim", "head_dim");
  c = good, c.head_dim = 65552;
  expect(write(&c), INV, "cache long head_dim", "head_dim");
  c = good, c.n_pages = HUGE;
  expect(write(&c), INV, "cache pages", "large");
  c = good, c.page_size = HUGE;
  expect(write(&c), INV, "cache page size", "large");
  c = good, c.n_heads = HUGE;
  expect(write(&c), INV, "cache heads", "large");
  c = good, c.k = nullptr;
  expect(write(&c), INV, "cache k", "required");
  c = good, c.v_amax = nullptr;
  expect(write(&c), INV, "cache amax", "required");
  c = good, c.v_scale = nullptr;
  expect(write(&c), INV, "cache scales", "required");
  c = good, c.format = LH_CACHE_E4M3;
  expect(write(&c), INV, "cache E4M3 scales", "NULL");
  c = good, c.v = hb + 8;
  expect(write(&c), INV, "cache aligned", "aligned");
  c = good, c.k_scale = hb + 2;
  expect(write(&c), INV, "cache scales aligned", "aligned");
  expect(write(&good, BF, 120), INV, "k stride", "k_stride");
  expect(write(&good, BF, 128, 129), INV, "v stride", "v_stride");
  expect(write(&good, BF, -128, 128), INV, "negative stride", "k_stride");
  expect(write(&good, BF, 128, 128, -1), INV, "tokens", "tokens");
  expect(write(&good, BF, 128, 128, HUGE), INV, "many tokens", "too many");
  expect(write(&good), INV, "cache host", "device");
  expect(write(&good, BF, 128, 128, 0), LH_OK, "no tokens");
  expect(lh_cache_write(&good, h, 128, nullptr, 128, BF, 3, ho, nullptr), INV, "no V", "required");
  expect(lh_cache_write(&good, host + 8, 128, h, 128, BF, 3, ho, nullptr), INV, "K aligned", "aligned");
  expect(lh_cache_read(&good, nullptr, 3, BF, h, h, nullptr), INV, "no slots", "required");
  expect(lh_cache_read(&good, ho, -3, BF, h, h, nullptr), INV, "read tokens", "tokens");
  expect(lh_cache_read(&good, ho, 3, F8, h, h, nullptr), UNS, "read dtype", "dtype");
  expect(lh_cache_read(&good, ho, 3, BF, h, host + 8, nullptr), INV, "read aligned", "aligned");
  expect(lh_cache_read(&good, ho, 3, BF, h, h, nullptr), INV, "read host", "device");
  expect(lh_cache_read(&good, nullptr, 0, BF, nullptr, nullptr, nullptr), LH_OK, "read nothing");

  // attention
  auto att = [&](const lh_cache* cc, lh_dtype t, int64_t qs, int64_t batch, int64_t heads, int64_t pages, float scale, void* work,
                 int64_t bytes) {
    return lh_paged_attention(cc, h, qs, t, batch, heads, hi, pages, hi, scale, h, work, bytes, nullptr);
  };
  expect(att(nullptr, BF, 512, 2, 8, 4, 1.f, h, 1 << 20), INV, "attention cache", "cache");
  expect(att(&good, F8, 512, 2, 8, 4, 1.f, h, 1 << 20), UNS, "attention dtype", "dtype");
  c = good, c.head_dim = 96;
  expect(att(&c, BF, 512, 2, 8, 4, 1.f, h, 1 << 20), UNS, "attention head_dim", "head_dim");
  expect(att(&good, BF, 512, 2, 7, 4, 1.f, h, 1 << 20), INV, "attention heads", "multiple");
  expect(att(&good, BF, 512, 2, 0, 4, 1.f, h, 1 << 20), INV, "attention no heads", "multiple");
  expect(att(&good, BF, 512, -2, 8, 4, 1.f, h, 1 << 20), INV, "attention batch", "batch");
  expect(att(&good, BF, 512, HUGE, 8, 4, 1.f, h, 1 << 20), INV, "attention large batch", "too many");
  expect(att(&good, BF, 512, 2, 8, -4, 1.f, h, 1 << 20), INV, "attention pages", "max_pages");
  expect(att(&good, BF, 512, 2, 8, HUGE, 1.f, h, 1 << 20), INV, "attention many pages", "max_pages");
  expect(att(&good, BF, 511, 2, 8, 4, 1.f, h, 1 << 20), INV, "attention stride", "q_stride");
  expect(att(&good, BF, 512, 2, 8, 4, INFINITY, h, 1 << 20), INV, "attention scale", "scale");
  expect(att(&good, BF, 512, 2, 8, 4096, 1.f, nullptr, 1 << 20), INV, "attention no workspace", "workspace");
  expect(att(&good, BF, 512, 2, 8, 4096, 1.f, h, 64), INV, "attention short workspace", "workspace");
  expect(att(&good, BF, 512, 2, 8, 4, 1.f, host + 4, 1 << 20), INV, "attention workspace aligned", "aligned");
  expect(att(&good, BF, 512, 2, 8, 4, 1.f, h, 1 << 20), INV, "attention host", "device");
  expect(att(&good, BF, 512, 0, 8, 4, 1.f, nullptr, 0), LH_OK, "attention no sequences");
  if (lh_paged_attention_workspace(&good, 2, 8, 4096) <= 0 || lh_paged_attention_workspace(&good, 2, 7, 4096) != 0 ||
      lh_paged_attention_workspace(nullptr, 2, 8, 4096) != 0 || lh_paged_attention_workspace(&good, 2, 8, 1) != 0 ||
      lh_paged_attention_workspace(&good, HUGE, 8, 4096) != 0) {
    std::fprintf(stderr, "FAIL workspace\n");
    ++failures;
  }
  std::printf("ok: %d failures\n", failures);
  return failures != 0;
}
