// Host-side driver for the sanitizer build of the validation of AdamW with
// 8-bit states: every call fails validation or has nothing to do, which returns
// before the first HIP call.  Built and run by tests/test_adamw8_sanitizers.py.
#include <cstdint>
#include <cstdio>
#include <vector>

#include "muon.h"

static int failures = 0;
static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}
static uint8_t* at(int i) { return reinterpret_cast<uint8_t*>(uintptr_t(0x100000000000ull) * (i + 1)); }
static muon_adamw8_state state(int64_t n, int base = 0) {
  return {at(base), at(base + 1), at(base + 2), at(base + 3), n};
}

int main() {
  const int64_t most = MUON_ADAMW8_MAX_ELEMENTS;
  for (int64_t n : {INT64_MIN, int64_t(-1), int64_t(0), int64_t(1), int64_t(31), int64_t(33), most,
                    most + 1, INT64_MAX})
    for (int dtype : {0, 1, 2}) {
      muon_adamw8_tensor t{at(4), nullptr, state(n), 0.1, 0.1, 7};
      const bool ok = n >= 0 && n <= most;
      const int want = dtype == 2 ? MUON_ERR_UNSUPPORTED_DTYPE
                       : !ok      ? MUON_ERR_INVALID_SHAPE
                       : n == 0   ? MUON_OK
                                  : MUON_ERR_INVALID_ARGUMENT;
      expect(muon_adamw_byte_step_grouped(&t, 1, dtype, 0.9, 0.99, 1e-8, 1, nullptr), want, "step");
      const muon_adamw8_state s = state(n);
      expect(muon_adamw_byte_moments(&s, 1, nullptr, at(5), dtype, nullptr), want, "moments");
    }
  // many tensors, the last one overlapping the first
  std::vector<muon_adamw8_tensor> many;
  for (int i = 0; i < 1000; ++i) {
    uint8_t* b = at(0) + size_t(i) * 0x100000;
    many.push_back({b, b + 0x10000, {b + 0x20000, b + 0x30000, b + 0x40000, b + 0x50000, 1000}, 0.1,
                    0.0, uint32_t(i)});
  }
  many.back().G = static_cast<uint8_t*>(many.front().P) + 3996;
  expect(muon_adamw_byte_step_grouped(many.data(), 1000, 0, 0.9, 0.99, 1e-8, 1, nullptr),
         MUON_ERR_INVALID_ARGUMENT, "overlap");
  std::vector<muon_adamw8_state> huge(40, state(most));
  expect(muon_adamw_byte_moments(huge.data(), 40, at(10), at(12), 0, nullptr), MUON_ERR_INVALID_SHAPE, "total");
  expect(muon_adamw_byte_moments(huge.data(), INT64_MIN, at(10), at(12), 0, nullptr),
         MUON_ERR_INVALID_ARGUMENT, "count");
  if (failures) return 1;
  std::puts("ALL_VALIDATION_CASES_OK");
  return 0;
}
