// Host-side driver for the sanitizer build of the validation of the linear
// products: every call fails validation or has nothing to do, which returns
// before the first HIP call.  Built and run by tests/test_linear_sanitizers.py.
#include <cstdint>
#include <cstdio>

#include "muon.h"

static int failures = 0;
static void expect(bool ok, const char* what) {
  if (!ok) {
    std::fprintf(stderr, "%s\n", what);
    ++failures;
  }
}
static char* at(int i) { return reinterpret_cast<char*>(uintptr_t(0x100000000000ull) * (i + 1)); }

int main() {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 127, 129, MUON_MAX_DIM, MUON_MAX_DIM + 1,
                           MUON_MAX_TOKENS, MUON_MAX_TOKENS + 1, INT64_MAX};
  const int64_t counts[] = {INT64_MIN, -1, 0, 1, 2, MUON_LINEAR_MAX_COUNT, MUON_LINEAR_MAX_COUNT + 1, INT64_MAX};
  const int64_t* offsets = reinterpret_cast<const int64_t*>(at(9));
  for (int64_t tokens : sizes)
    for (int64_t rows : sizes)
      for (int64_t cols : sizes)
        for (int64_t count : counts)
          for (int dtype : {0, 1, 5}) {
            // no output: refused, or there is nothing to do
            int st = muon_linear_forward(at(0), cols, dtype, at(1), offsets, count, tokens, rows, cols, nullptr, nullptr);
            expect(st != MUON_OK || tokens == 0, "forward");
            st = muon_linear_input_grad(at(0), rows, dtype, at(1), offsets, count, tokens, rows, cols, nullptr, nullptr);
            expect(st != MUON_OK || tokens == 0, "input grad");
            const muon_weight8 w{at(2), at(3), reinterpret_cast<uint8_t*>(at(4)), count, rows, cols};
            const muon_ckpt x{at(5), reinterpret_cast<uint8_t*>(at(6)), tokens, cols, MUON_CKPT_E4M3};
            st = muon_linear_forward_quantized(&x, &w, offsets, nullptr, dtype, nullptr);
            expect(st != MUON_OK || tokens == 0, "forward quantized");
            st = muon_weight_quantize(nullptr, dtype, &w, nullptr);
            expect(st != MUON_OK || count == 0, "quantize");
          }
  if (failures) return 1;
  std::puts("ALL_VALIDATION_CASES_OK");
  return 0;
}
