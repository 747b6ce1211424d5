// C ABI of AdamW with 8-bit states: argument validation and the launches on
// the caller's stream.  Every argument is checked before the first HIP call.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "abi_util.h"
#include "adamw8_internal.h"

using namespace muon;

namespace {

constexpr uint32_t kMaxBlocks = (uint32_t(1) << 24) - 1;   // of one launch

int64_t state_blocks(int64_t n) { return (n + MUON_CKPT_BLOCK - 1) / MUON_CKPT_BLOCK; }
int64_t chunks(int64_t n) { return (n + kAdam8Chunk - 1) / kAdam8Chunk; }
static_assert(MUON_ADAMW8_MAX_ELEMENTS / kAdam8Chunk <= kMaxBlocks, "a tensor fits a launch");

// The buffers of a call of many tensors, none of which may overlap another.
// Ranges that may are inputs only (the states of a read).
class Ranges {
 public:
  // Room for those of `count` tensors, up to 6 each and 2 more: false where the host
  // has none, for no C++ exception may leave a C entry point.
  bool reserve(int64_t count) {
    if (count > int64_t(1) << 40) return false;
    try {
      r_.reserve(size_t(count) * 6 + 2);
      return true;
    } catch (const std::exception&) {
      return false;
    }
  }
  void add(const void* p, size_t bytes, bool out = true) {
    if (bytes) r_.push_back({reinterpret_cast<uintptr_t>(p), bytes, out});
  }
  // Sorted by their start, each output must lie behind everything before it,
  // and each input behind the outputs before it.
  bool clash() {
    std::sort(r_.begin(), r_.end(), [](const Range& a, const Range& b) { return a.at < b.at; });
    uintptr_t any = 0, outs = 0;   // ends so far
    for (const Range& x : r_) {
      if (x.at < outs || (x.out && x.at < any)) return true;
      any = std::max(any, x.at + x.bytes);
      if (x.out) outs = std::max(outs, x.at + x.bytes);
    }
    return false;
  }

 private:
  struct Range {
    uintptr_t at;
    size_t bytes;
    bool out;
  };
  std::vector<Range> r_;
};

int check_state(const muon_adamw8_state& x) {
  if (x.n < 0 || x.n > MUON_ADAMW8_MAX_ELEMENTS) return MUON_ERR_INVALID_SHAPE;
  if (x.n == 0) return MUON_OK;
  if (!x.m_q || !x.m_scale || !x.r_q || !x.r_scale || !aligned(x.m_q, 16) || !aligned(x.r_q, 16))
    return MUON_ERR_INVALID_ARGUMENT;
  return MUON_OK;
}

void add_state(Ranges& r, const muon_adamw8_state& x, bool out) {
  const size_t blocks = size_t(state_blocks(x.n));
  r.add(x.m_q, blocks * MUON_CKPT_BLOCK, out);
  r.add(x.r_q, blocks * MUON_CKPT_BLOCK, out);
  r.add(x.m_scale, blocks, out);
  r.add(x.r_scale, blocks, out);
}

// Collects tensors into launches.
struct Launches {
  Adam8Batch bt{};
  hipError_t (*launch)(const Adam8Batch&, bool, hipStream_t);
  const char* name;
  bool bf16;
  hipStream_t s;

  int flush() {
    if (bt.nseg == 0) return MUON_OK;
    const int st = launched(launch(bt, bf16, s), name, s);
    bt.nseg = 0;
    bt.blocks = 0;
    return st;
  }
  int add(const muon_adamw8_state& x, Adam8Seg g) {
    const uint32_t blocks = uint32_t(chunks(x.n));
    if (bt.nseg == kAdam8Segs || bt.blocks + blocks > kMaxBlocks)
      if (const int st = flush(); st != MUON_OK) return st;
    g.m_q = static_cast<uint8_t*>(x.m_q);
    g.m_scale = x.m_scale;
    g.r_q = x.r_q;
    g.r_scale = x.r_scale;
    g.n = x.n;
    g.begin = bt.blocks;
    bt.seg[bt.nseg++] = g;
    bt.blocks += blocks;
    return MUON_OK;
  }
};

}  // namespace

extern "C" {

int muon_adamw_byte_step_grouped(const muon_adamw8_tensor* tensors, int64_t count, int dtype,
                             double beta1, double beta2, double eps, int64_t step, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!(beta1 >= 0 && beta1 < 1 && beta2 >= 0 && beta2 < 1) || !std::isfinite(eps) || eps < 0 ||
      step < 1 || count < 0 || (count > 0 && !tensors))
    return MUON_ERR_INVALID_ARGUMENT;
  const size_t es = elem_size(dtype);
  Ranges r;
  if (!r.reserve(count)) return MUON_ERR_INVALID_ARGUMENT;
  for (int64_t i = 0; i < count; ++i) {
    const muon_adamw8_tensor& x = tensors[i];
    if (!std::isfinite(x.lr) || !std::isfinite(x.weight_decay)) return MUON_ERR_INVALID_ARGUMENT;
    if (const int st = check_state(x.state); st != MUON_OK) return st;
    if (x.state.n == 0) continue;
    if (!x.P || !x.G || !aligned(x.P, es) || !aligned(x.G, es)) return MUON_ERR_INVALID_ARGUMENT;
    r.add(x.P, size_t(x.state.n) * es);
    r.add(x.G, size_t(x.state.n) * es);
    add_state(r, x.state, true);
  }
  if (r.clash()) return MUON_ERR_INVALID_ARGUMENT;

  Trace t("muon_adamw_byte_step");
  // Bias corrections in double: 1 - beta^t.
  const double bc1 = 1.0 - std::pow(beta1, double(step));
  const double bc2 = 1.0 - std::pow(beta2, double(step));
  Launches l;
  l.launch = launch_adamw8;
  l.name = "adamw8";
  l.bf16 = dtype == MUON_DTYPE_BF16;
  l.s = static_cast<hipStream_t>(stream);
  l.bt.beta1 = float(beta1);
  l.bt.beta2 = float(beta2);
  l.bt.one_minus_beta1 = float(1.0 - beta1);
  l.bt.one_minus_beta2 = float(1.0 - beta2);
  l.bt.eps = float(eps);
  l.bt.inv_sqrt_bc2 = float(1.0 / std::sqrt(bc2));
  for (int64_t i = 0; i < count; ++i) {
    const muon_adamw8_tensor& x = tensors[i];
    if (x.state.n == 0) continue;
    Adam8Seg g{};
    g.P = x.P;
    g.G = x.G;
    g.decay = float(1.0 - x.lr * x.weight_decay);
    g.step_size = float(x.lr / bc1);
    g.seed = x.seed;
    if (const int st = l.add(x.state, g); st != MUON_OK) return st;
  }
  return l.flush();
}

int muon_adamw_byte_moments(const muon_adamw8_state* states, int64_t count, void* m, void* r,
                        int dtype, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (count < 0 || (count > 0 && !states)) return MUON_ERR_INVALID_ARGUMENT;
  const size_t es = elem_size(dtype);
  Ranges ranges;
  if (!ranges.reserve(count)) return MUON_ERR_INVALID_ARGUMENT;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (const int st = check_state(states[i]); st != MUON_OK) return st;
    if (states[i].n > 0) add_state(ranges, states[i], false);
    total += states[i].n;
    if (total > (int64_t(1) << 40)) return MUON_ERR_INVALID_SHAPE;
  }
  if (total == 0) return MUON_OK;
  if (!m || !r || !aligned(m, es) || !aligned(r, es)) return MUON_ERR_INVALID_ARGUMENT;
  ranges.add(m, size_t(total) * es);
  ranges.add(r, size_t(total) * es);
  if (ranges.clash()) return MUON_ERR_INVALID_ARGUMENT;

  Trace t("muon_adamw_byte_moments");
  Launches l;
  l.launch = launch_adamw8_moments;
  l.name = "adamw8_moments";
  l.bf16 = dtype == MUON_DTYPE_BF16;
  l.s = static_cast<hipStream_t>(stream);
  int64_t at = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (states[i].n == 0) continue;
    Adam8Seg g{};
    g.P = static_cast<char*>(m) + size_t(at) * es;
    g.G = static_cast<char*>(r) + size_t(at) * es;
    at += states[i].n;
    if (const int st = l.add(states[i], g); st != MUON_OK) return st;
  }
  return l.flush();
}

}  // extern "C"
