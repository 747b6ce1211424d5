// What the host files of the layer operators, of the linear products and of
// AdamW with 8-bit states share: checks of arguments and launch results.
#pragma once

#include <cstdio>

#include "layer_internal.h"

namespace muon {
namespace {

constexpr size_t kAlign = 256;

bool dtype_ok(int dtype) { return dtype == MUON_DTYPE_F32 || dtype == MUON_DTYPE_BF16; }
size_t elem_size(int dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

bool sizes_ok(int64_t tokens, int64_t cols) {
  return tokens >= 0 && tokens <= MUON_MAX_TOKENS && cols >= 1 && cols <= MUON_MAX_DIM;
}

// The buffers of one call.  Outputs must not overlap anything else.
struct Buffers {
  struct Range {
    uintptr_t at;
    size_t bytes;
    bool out;
  };
  Range r[20];
  int n = 0;
  void add(const void* p, size_t bytes, bool out) {
    if (p && bytes) r[n++] = {reinterpret_cast<uintptr_t>(p), bytes, out};
  }
  // rows of `len` elements, `ld` apart
  void add_matrix(const void* p, int64_t rows, int64_t len, int64_t ld, size_t es, bool out) {
    if (rows > 0) add(p, (size_t(rows - 1) * size_t(ld) + size_t(len)) * es, out);
  }
  void add_ckpt(const muon_ckpt* c, bool out) {
    if (!c) return;
    add(c->q, size_t(c->tokens) * size_t(MUON_CKPT_Q_PITCH(c->cols)), out);
    add(c->scale, size_t(c->tokens) * size_t(MUON_CKPT_SCALE_PITCH(c->cols)), out);
  }
  bool clash() const {
    for (int i = 0; i < n; ++i)
      for (int j = i + 1; j < n; ++j)
        if ((r[i].out || r[j].out) && r[i].at < r[j].at + r[j].bytes &&
            r[j].at < r[i].at + r[i].bytes)
          return true;
    return false;
  }
};

// A row stride: at least the row, and small enough that the matrix's bytes
// stay far from overflow.
bool stride_ok(int64_t ld, int64_t len) { return ld >= len && ld <= (int64_t(1) << 24); }

// A checkpoint descriptor of tokens x cols (its pointers may be null when
// there are no tokens).
int check_ckpt(const muon_ckpt* c, int64_t tokens, int64_t cols) {
  if (c->format != MUON_CKPT_E4M3 && c->format != MUON_CKPT_INT8) return MUON_ERR_INVALID_ARGUMENT;
  if (!sizes_ok(c->tokens, c->cols) || c->tokens != tokens || c->cols != cols)
    return MUON_ERR_INVALID_SHAPE;
  if (tokens > 0 && (!c->q || !c->scale)) return MUON_ERR_INVALID_ARGUMENT;
  if (!aligned(c->q, 16) || !aligned(c->scale, 4)) return MUON_ERR_INVALID_ARGUMENT;
  return MUON_OK;
}

Ckpt view(const muon_ckpt* c) {
  Ckpt v{};
  v.fmt = -1;
  if (c) {
    v.q = static_cast<uint8_t*>(c->q);
    v.scale = c->scale;
    v.q_pitch = MUON_CKPT_Q_PITCH(c->cols);
    v.s_pitch = MUON_CKPT_SCALE_PITCH(c->cols);
    v.fmt = c->format;
  }
  return v;
}

struct Trace {
  explicit Trace(const char* name) { trace_push(name); }
  ~Trace() { trace_pop(); }
};

// After each launch: keeps the error, and synchronises under MUON_DEBUG.
int launched(hipError_t e, const char* what, hipStream_t s) {
  if (e == hipSuccess && debug_sync_enabled()) e = hipStreamSynchronize(s);
  if (e == hipSuccess) return MUON_OK;
  note_hip_error(e);
  if (debug_sync_enabled())
    std::fprintf(stderr, "muon: %s failed: %s\n", what, hipGetErrorString(e));
  return MUON_ERR_HIP;
}

size_t align_up(size_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

char* align_ptr(void* p) {
  return reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(p) + kAlign - 1) / kAlign * kAlign);
}

}  // namespace
}  // namespace muon
