// Host-side driver for the sanitizer build of the layer operators' validation
// layer: every call below fails validation or has nothing to do, which
// returns before the first HIP call, so it runs without a GPU.  Built and run
// by tests/test_layer_sanitizers.py with AddressSanitizer and
// UndefinedBehaviorSanitizer on the host code; any report fails the test.
#include <cstdint>
#include <cstdio>

#include "muon.h"

static int failures = 0;

static void expect(int got, int want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "%s: status %d, expected %d\n", what, got, want);
    ++failures;
  }
}

static char* at(int i) { return reinterpret_cast<char*>(uintptr_t(0x1000000000ull) * (i + 1)); }
static float* f(int i) { return reinterpret_cast<float*>(at(i)); }

static muon_ckpt ck(int64_t tokens, int64_t cols, int format = MUON_CKPT_E4M3) {
  return {at(10), reinterpret_cast<uint8_t*>(at(11)), tokens, cols, format};
}

int main() {
  const int64_t big = INT64_MAX, most = MUON_MAX_TOKENS;
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 31, 33, 4097, MUON_MAX_DIM, MUON_MAX_DIM + 1, most,
                           most + 1, big};
  // workspace sizes over every combination, overflowing ones included
  int64_t sum = 0;
  for (int64_t t : sizes)
    for (int64_t c : sizes) {
      sum += int64_t(muon_layernorm_workspace_bytes(t, c) & 1);
      for (int64_t r : sizes)
        for (int64_t n : {int64_t(-1), int64_t(0), int64_t(1), int64_t(64),
                          int64_t(MUON_WEIGHT_GRAD_MAX_COUNT), big})
          for (int dtype : {int(MUON_DTYPE_F32), int(MUON_DTYPE_BF16), 7})
            for (int with : {0, 1})
              sum += int64_t(muon_weight_grad_workspace_bytes(n, with, t, r, c, dtype) & 1);
    }
  expect(int(sum), 0, "workspace sizes are whole words");

  for (int64_t t : sizes)
    for (int64_t c : sizes) {
      const bool ok = t >= 0 && t <= most && c >= 1 && c <= MUON_MAX_DIM;
      const muon_ckpt k = ck(t, c), odd = ck(t, c, 5);
      // a null x: refused by its size, or as a null pointer, or nothing to do
      const int want = !ok ? MUON_ERR_INVALID_SHAPE : t == 0 ? MUON_OK : MUON_ERR_INVALID_ARGUMENT;
      expect(muon_checkpoint_save(nullptr, c, 0, &k, nullptr), want, "save");
      expect(muon_checkpoint_restore(&k, nullptr, 1, nullptr), want, "restore");
      expect(muon_checkpoint_save(at(0), c, 0, &odd, nullptr), MUON_ERR_INVALID_ARGUMENT, "format");
      expect(muon_layernorm_forward(nullptr, c, at(1), at(2), t, c, 0, 0, 1e-5, at(3), f(4), f(5),
                                    nullptr, nullptr, nullptr), want, "forward");
      if (ok && t > 0)
        expect(muon_layernorm_forward(at(0), c - 1, at(1), at(2), t, c, 0, 0, 1e-5, at(3), f(4), f(5),
                                      &k, &k, nullptr), MUON_ERR_INVALID_ARGUMENT, "forward stride");
      if (ok && t > 0)
        expect(muon_layernorm_backward(at(0), c, at(1), c, nullptr, at(2), f(3), f(4), t, c, 0, 1,
                                       at(0), at(6), at(7), 0, at(8), SIZE_MAX / 2, nullptr),
               MUON_ERR_INVALID_ARGUMENT, "backward overlap");
      expect(muon_layernorm_backward(at(0), c, nullptr, 0, nullptr, at(2), f(3), f(4), t, c, 0, 1,
                                     at(5), at(6), nullptr, 1, at(8), 16, nullptr),
             want, "backward without x");
      for (int64_t r : sizes) {
        const bool fine = ok && r >= 1 && r <= MUON_MAX_DIM;
        const int st = muon_weight_grad(nullptr, r, 1, &k, nullptr, 1, r, at(1), 1, 1, at(2), 1 << 20, nullptr);
        expect(st, !fine ? MUON_ERR_INVALID_SHAPE : t == 0 ? MUON_OK : MUON_ERR_INVALID_ARGUMENT, "weight");
        for (int64_t n : {int64_t(2), int64_t(MUON_WEIGHT_GRAD_MAX_COUNT), big})
          if (muon_weight_grad(at(0), r, 1, &k, nullptr, n, r, at(1), 1, 0, at(2), 64, nullptr) == MUON_OK)
            expect(1, 0, "several matrices without offsets");
      }
    }
  // a G whose bytes pass 64 bits of address space, and one that wraps onto dy
  const muon_ckpt wide = ck(16, MUON_MAX_DIM);
  expect(muon_weight_grad(at(0), MUON_MAX_DIM, 0, &wide, reinterpret_cast<int64_t*>(at(3)),
                          MUON_WEIGHT_GRAD_MAX_COUNT, MUON_MAX_DIM, at(1), 0, 0, at(2), 64, nullptr),
         MUON_ERR_INVALID_ARGUMENT, "G over other buffers");
  expect(muon_checkpoint_save(at(0), 64, 0, nullptr, nullptr), MUON_ERR_INVALID_ARGUMENT, "null");
  if (failures) return 1;
  std::puts("ALL_VALIDATION_CASES_OK");
  return 0;
}
