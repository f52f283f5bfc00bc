// Host checks of how attention cuts a sequence into parts of one size and reads its table, built with UndefinedBehaviorSanitizer
// (tests/test_decode_limits.py).
#include <cstdint>
#include <cstdio>

#include "../../nvfp4_scale_calibration_lh_amd/csrc/attention_cut.hpp"

int main() {
  int failures = 0;
  const int64_t most = (int64_t(1) << 31) - 4096;
  for (int splits : {2, 3, 7, 16, 100, 1000, 1024})
    for (int64_t len : {int64_t(0), int64_t(1), int64_t(511), int64_t(512), int64_t(513), int64_t(1024), int64_t(40001),
                        int64_t(131001), int64_t(1) << 24, int64_t(1073741824), int64_t(1431655766), int64_t(1500000000),
                        most - 129, most - 1, most}) {
      const lh::EvenParts p = lh::even_parts((int)len, splits);
      const int64_t size = p.size, count = p.count;
      const bool ok = size >= lh::kAttentionMinChunk && size % lh::kAttentionStep == 0 && count >= 1 && count <= splits &&
                      size * count >= len && (len == 0 || size * (count - 1) < len);
      if (!ok) {
        std::fprintf(stderr, "FAIL %lld tokens in %d: %lld of %lld\n", (long long)len, splits, (long long)count, (long long)size);
        ++failures;
      }
    }
  for (int64_t pages : {int64_t(1), int64_t(3), int64_t(2147483647), int64_t(1) << 32, int64_t(1) << 40})
    for (int64_t page : {int64_t(0), int64_t(1), int64_t(2), int64_t(3), int64_t(2147483647), int64_t(-1), int64_t(-7), -(int64_t(1) << 31)}) {
      const int64_t got = lh::page_or_first((int)page, pages), want = page >= 0 && page < pages ? page : 0;
      if (got != want) {
        std::fprintf(stderr, "FAIL page %lld of %lld: %lld\n", (long long)page, (long long)pages, (long long)got);
        ++failures;
      }
    }
  std::printf("ok: %d failures\n", failures);
  return failures != 0;
}
