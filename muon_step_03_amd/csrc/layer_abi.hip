// C ABI of the layer operators: argument validation and the launches on the
// caller's stream.  Every argument is checked before the first HIP call, so
// every error status is returned without touching the device.
#include <cmath>

#include "abi_util.h"

using namespace muon;

namespace {

// Workspace of a weight gradient.
size_t weight_grad_bytes(const WeightGradPlan& plan) {
  const size_t n = align_up(plan.partial_bytes) + align_up(plan.table_bytes) + plan.repack_bytes;
  return plan.pieces > 0 && n > 0 ? n + kAlign : 0;
}

bool weight_grad_sizes_ok(int64_t count, int64_t tokens, int64_t rows, int64_t cols, int dtype) {
  return dtype_ok(dtype) && count >= 1 && count <= MUON_WEIGHT_GRAD_MAX_COUNT &&
         sizes_ok(tokens, cols) && rows >= 1 && rows <= MUON_MAX_DIM;
}

}  // namespace

extern "C" {

int muon_checkpoint_save(const void* x, int64_t ldx, int dtype, const muon_ckpt* ckpt,
                         void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!ckpt) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t tokens = ckpt->tokens, cols = ckpt->cols;
  int st = check_ckpt(ckpt, tokens, cols);
  if (st != MUON_OK) return st;
  if (tokens == 0) return MUON_OK;
  const size_t es = elem_size(dtype);
  if (!x || !aligned(x, es) || !stride_ok(ldx, cols)) return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_matrix(x, tokens, cols, ldx, es, false);
  b.add_ckpt(ckpt, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  Trace t("muon_checkpoint_save");
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(launch_ckpt_save(x, ldx, dtype == MUON_DTYPE_BF16, view(ckpt), tokens, int(cols), s),
                  "checkpoint_save", s);
}

int muon_checkpoint_restore(const muon_ckpt* ckpt, void* x, int dtype, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!ckpt) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t tokens = ckpt->tokens, cols = ckpt->cols;
  int st = check_ckpt(ckpt, tokens, cols);
  if (st != MUON_OK) return st;
  if (tokens == 0) return MUON_OK;
  const size_t es = elem_size(dtype);
  if (!x || !aligned(x, es)) return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_matrix(x, tokens, cols, cols, es, true);
  b.add_ckpt(ckpt, false);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  Trace t("muon_checkpoint_restore");
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(launch_ckpt_restore(view(ckpt), x, dtype == MUON_DTYPE_BF16, tokens, int(cols), s),
                  "checkpoint_restore", s);
}

int muon_layernorm_forward(const void* x, int64_t ldx, const void* gain, const void* bias,
                           int64_t tokens, int64_t cols, int dtype, int param_dtype, double eps,
                           void* y, float* mean, float* rstd, const muon_ckpt* x_ckpt,
                           const muon_ckpt* y_ckpt, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(tokens, cols)) return MUON_ERR_INVALID_SHAPE;
  if (!std::isfinite(eps) || eps < 0) return MUON_ERR_INVALID_ARGUMENT;
  for (const muon_ckpt* c : {x_ckpt, y_ckpt})
    if (c)
      if (const int st = check_ckpt(c, tokens, cols); st != MUON_OK) return st;
  if (tokens == 0) return MUON_OK;
  const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
  if (!x || !gain || !y || !mean || !rstd) return MUON_ERR_INVALID_ARGUMENT;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(gain, ps) || !aligned(bias, ps) ||
      !aligned(mean, 4) || !aligned(rstd, 4) || !stride_ok(ldx, cols))
    return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_matrix(x, tokens, cols, ldx, es, false);
  b.add(gain, size_t(cols) * ps, false);
  b.add(bias, size_t(cols) * ps, false);
  b.add_matrix(y, tokens, cols, cols, es, true);
  b.add(mean, size_t(tokens) * 4, true);
  b.add(rstd, size_t(tokens) * 4, true);
  b.add_ckpt(x_ckpt, true);
  b.add_ckpt(y_ckpt, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  LnForward p{};
  p.x = x;
  p.ldx = ldx;
  p.gain = gain;
  p.bias = bias;
  p.y = y;
  p.mean = mean;
  p.rstd = rstd;
  p.tokens = tokens;
  p.cols = int(cols);
  p.param_bf16 = param_dtype == MUON_DTYPE_BF16;
  p.eps = float(eps);
  p.xc = view(x_ckpt);
  p.yc = view(y_ckpt);
  Trace t("muon_layernorm_forward");
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(launch_ln_forward(p, dtype == MUON_DTYPE_BF16, s), "layernorm_forward", s);
}

size_t muon_layernorm_workspace_bytes(int64_t tokens, int64_t cols) {
  if (!sizes_ok(tokens, cols)) return 0;
  const int blocks = ln_backward_blocks(tokens, cols, true);   // enough for either type
  return blocks > 1 ? size_t(blocks) * 2 * size_t(cols) * 4 + kAlign : 0;
}

int muon_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                            const muon_ckpt* x_ckpt, const void* gain, const float* mean,
                            const float* rstd, int64_t tokens, int64_t cols, int dtype,
                            int param_dtype, void* dx, void* dgain, void* dbias, int accumulate,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(param_dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!sizes_ok(tokens, cols)) return MUON_ERR_INVALID_SHAPE;
  if (x_ckpt)
    if (const int st = check_ckpt(x_ckpt, tokens, cols); st != MUON_OK) return st;
  const size_t es = elem_size(dtype), ps = elem_size(param_dtype);
  if (!gain || !dgain || (x && x_ckpt)) return MUON_ERR_INVALID_ARGUMENT;
  if (tokens > 0) {
    if (!dy || !dx || !mean || !rstd || (!x && !x_ckpt)) return MUON_ERR_INVALID_ARGUMENT;
    if (!stride_ok(lddy, cols) || (x && !stride_ok(ldx, cols))) return MUON_ERR_INVALID_ARGUMENT;
  }
  if (!aligned(dy, es) || !aligned(x, es) || !aligned(dx, es) || !aligned(gain, ps) ||
      !aligned(dgain, ps) || !aligned(dbias, ps) || !aligned(mean, 4) || !aligned(rstd, 4))
    return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_matrix(dy, tokens, cols, lddy, es, false);
  b.add_matrix(x, tokens, cols, ldx, es, false);
  b.add_ckpt(x_ckpt, false);
  b.add(gain, size_t(cols) * ps, false);
  b.add(mean, size_t(tokens) * 4, false);
  b.add(rstd, size_t(tokens) * 4, false);
  b.add_matrix(dx, tokens, cols, cols, es, true);
  b.add(dgain, size_t(cols) * ps, true);
  b.add(dbias, size_t(cols) * ps, true);
  b.add(workspace, workspace_bytes, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  const size_t need = muon_layernorm_workspace_bytes(tokens, cols);
  if (need > 0 && !workspace) return MUON_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
  if (tokens == 0 && accumulate) return MUON_OK;
  LnBackward p{};
  p.dy = dy;
  p.lddy = lddy;
  p.x = x;
  p.ldx = ldx;
  p.xc = view(x_ckpt);
  p.gain = gain;
  p.mean = mean;
  p.rstd = rstd;
  p.dx = dx;
  p.dgain = dgain;
  p.dbias = dbias;
  p.partial = reinterpret_cast<float*>(align_ptr(workspace));
  p.tokens = tokens;
  p.cols = int(cols);
  p.param_bf16 = param_dtype == MUON_DTYPE_BF16;
  p.accumulate = accumulate != 0;
  p.blocks = ln_backward_blocks(tokens, cols, dtype == MUON_DTYPE_BF16);
  Trace t("muon_layernorm_backward");
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (p.blocks > 0) {
    const int st = launched(launch_ln_backward(p, dtype == MUON_DTYPE_BF16, s), "layernorm_backward", s);
    if (st != MUON_OK || p.blocks == 1) return st;
  }
  return launched(launch_ln_params(p, s), "layernorm_params", s);
}

size_t muon_weight_grad_workspace_bytes(int64_t count, int with_offsets, int64_t tokens,
                                        int64_t rows, int64_t cols, int dtype) {
  if (!weight_grad_sizes_ok(count, tokens, rows, cols, dtype)) return 0;
  return weight_grad_bytes(
      weight_grad_plan(count, tokens, rows, cols, with_offsets != 0, dtype == MUON_DTYPE_BF16));
}

int muon_weight_grad_tile(int64_t count, int with_offsets, int64_t tokens, int64_t rows,
                          int64_t cols, int dtype) {
  if (!weight_grad_sizes_ok(count, tokens, rows, cols, dtype)) return 0;
  const WeightGradPlan plan =
      weight_grad_plan(count, tokens, rows, cols, with_offsets != 0, dtype == MUON_DTYPE_BF16);
  return plan.pieces <= 0 ? 0 : plan.wide ? 256 : 128;
}

int muon_weight_grad(const void* dy, int64_t lddy, int dtype, const muon_ckpt* x,
                     const int64_t* offsets, int64_t count, int64_t rows, void* G, int g_dtype,
                     int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype) || !dtype_ok(g_dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (count < 0 || !x) return MUON_ERR_INVALID_ARGUMENT;
  const int64_t tokens = x->tokens, cols = x->cols;
  if (rows < 1 || rows > MUON_MAX_DIM || count > MUON_WEIGHT_GRAD_MAX_COUNT) return MUON_ERR_INVALID_SHAPE;
  if (const int st = check_ckpt(x, tokens, cols); st != MUON_OK) return st;
  if (count == 0) return MUON_OK;
  if (!offsets && count != 1) return MUON_ERR_INVALID_ARGUMENT;
  const size_t es = elem_size(dtype), gs = elem_size(g_dtype);
  if (!G || !aligned(G, gs) || !aligned(offsets, 8) || !aligned(dy, es))
    return MUON_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && (!dy || !stride_ok(lddy, rows))) return MUON_ERR_INVALID_ARGUMENT;
  size_t g_bytes;
  if (__builtin_mul_overflow(size_t(count), size_t(rows) * size_t(cols) * gs, &g_bytes))
    return MUON_ERR_INVALID_SHAPE;
  Buffers b;
  b.add_matrix(dy, tokens, rows, lddy, es, false);
  b.add_ckpt(x, false);
  b.add(offsets, offsets ? size_t(count + 1) * 8 : 0, false);
  b.add(G, g_bytes, true);
  b.add(workspace, workspace_bytes, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  const WeightGradPlan plan = weight_grad_plan(count, tokens, rows, cols, offsets != nullptr,
                                               dtype == MUON_DTYPE_BF16);
  if (plan.pieces <= 0) return MUON_ERR_INVALID_SHAPE;
  const size_t need = weight_grad_bytes(plan);
  if (need > 0 && !workspace) return MUON_ERR_INVALID_ARGUMENT;
  if (workspace_bytes < need) return MUON_ERR_WORKSPACE_TOO_SMALL;
  if (tokens == 0 && accumulate) return MUON_OK;
  WeightGrad p{};
  p.dy = dy;
  p.lddy = lddy;
  p.x = view(x);
  p.offsets = offsets;
  p.tokens = tokens;
  p.count = int(count);
  p.rows = int(rows);
  p.cols = int(cols);
  p.G = G;
  p.g_bf16 = g_dtype == MUON_DTYPE_BF16;
  p.accumulate = accumulate != 0;
  p.partial = reinterpret_cast<float*>(align_ptr(workspace));
  p.chunk = plan.chunk;
  p.pieces = plan.pieces;
  p.table = reinterpret_cast<char*>(p.partial) + align_up(plan.partial_bytes);
  p.repack = reinterpret_cast<uint16_t*>(static_cast<char*>(p.table) + align_up(plan.table_bytes));
  Trace t("muon_weight_grad");
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int st = launched(launch_weight_grad(p, plan, dtype == MUON_DTYPE_BF16, s), "weight_grad", s);
  if (st != MUON_OK || plan.slots == 0) return st;
  return launched(launch_weight_grad_join(p, plan, s), "weight_grad_join", s);
}

}  // extern "C"
