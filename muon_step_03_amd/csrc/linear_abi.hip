// C ABI of the linear products and of weights in 8 bits: argument validation
// and the launches on the caller's stream.  Every argument is checked before
// the first HIP call.
#include "abi_util.h"
#include "linear_internal.h"

using namespace muon;

namespace {

constexpr int64_t SIDE = MUON_WEIGHT_BLOCK;
int64_t blocks(int64_t n) { return (n + SIDE - 1) / SIDE; }

bool weight_sizes_ok(int64_t count, int64_t rows, int64_t cols) {
  return count >= 0 && count <= MUON_LINEAR_MAX_COUNT && rows >= 1 && rows <= MUON_MAX_DIM &&
         cols >= 1 && cols <= MUON_MAX_DIM;
}

int check_weight8(const muon_weight8* w) {
  if (!w) return MUON_ERR_INVALID_ARGUMENT;
  if (!weight_sizes_ok(w->count, w->rows, w->cols)) return MUON_ERR_INVALID_SHAPE;
  if (w->count > 0 && (!w->q || !w->q_t || !w->scale)) return MUON_ERR_INVALID_ARGUMENT;
  if (!aligned(w->q, 16) || !aligned(w->q_t, 16)) return MUON_ERR_INVALID_ARGUMENT;
  return MUON_OK;
}

void add_weight8(Buffers& b, const muon_weight8* w, bool out) {
  const size_t n = size_t(w->count), br = size_t(blocks(w->rows)), bc = size_t(blocks(w->cols));
  b.add(w->q, n * size_t(w->rows) * bc * SIDE, out);
  b.add(w->q_t, n * size_t(w->cols) * br * SIDE, out);
  b.add(w->scale, n * br * bc, out);
}

// Product of in [tokens][k] with the weights, into out [tokens][n]: the checks
// that both operand types share, and the launch.
struct Call {
  LinearType type;
  bool across;
  Linear p{};
  size_t out_es;
};
int run(Call& c, const int64_t* offsets, int64_t count, Buffers& b, const char* name, void* stream) {
  Linear& p = c.p;
  if (!offsets && count != 1) return MUON_ERR_INVALID_ARGUMENT;
  if (!aligned(offsets, 8)) return MUON_ERR_INVALID_ARGUMENT;
  if (p.tokens == 0) return MUON_OK;
  if (!p.y || !aligned(p.y, c.out_es)) return MUON_ERR_INVALID_ARGUMENT;
  b.add(offsets, offsets ? size_t(count + 1) * 8 : 0, false);
  b.add_matrix(p.y, p.tokens, p.n, p.n, c.out_es, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  p.offsets = offsets;
  p.count = int(count);
  p.y_bf16 = c.out_es == 2;
  const LinearPlan plan = linear_plan(c.type, c.across, count > 0 ? count : 1, p.tokens, p.k, p.n);
  if (plan == LIN_NONE) return MUON_ERR_INVALID_SHAPE;
  Trace t(name);
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(launch_linear(p, c.type, c.across, plan, s), name, s);
}

int run_plain(bool across, const void* x, int64_t ldx, int dtype, const void* W,
              const int64_t* offsets, int64_t count, int64_t tokens, int64_t rows, int64_t cols,
              void* y, const char* name, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (count < 0) return MUON_ERR_INVALID_ARGUMENT;
  if (!weight_sizes_ok(count, rows, cols) || !sizes_ok(tokens, cols)) return MUON_ERR_INVALID_SHAPE;
  const size_t es = elem_size(dtype);
  const int64_t k = across ? rows : cols, n = across ? cols : rows;
  if (!aligned(x, es) || !aligned(W, es)) return MUON_ERR_INVALID_ARGUMENT;
  if (tokens > 0 && (!x || !stride_ok(ldx, k) || (count > 0 && !W))) return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_matrix(x, tokens, k, ldx, es, false);
  b.add(W, size_t(count) * size_t(rows) * size_t(cols) * es, false);
  Call c{};
  c.type = dtype == MUON_DTYPE_BF16 ? LIN_BF16 : LIN_F32;
  c.across = across;
  c.out_es = es;
  c.p.x = x;
  c.p.ldx = ldx * int64_t(es);
  c.p.W = W;
  c.p.ldw = cols * int64_t(es);
  c.p.w_stride = rows * cols * int64_t(es);
  c.p.tokens = tokens;
  c.p.k = int(k);
  c.p.n = int(n);
  c.p.y = y;
  return run(c, offsets, count, b, name, stream);
}

int run_quantized(bool across, const muon_ckpt* x, const muon_weight8* W, const int64_t* offsets,
                  void* y, int dtype, const char* name, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (!x) return MUON_ERR_INVALID_ARGUMENT;
  if (const int st = check_weight8(W); st != MUON_OK) return st;
  const int64_t k = across ? W->rows : W->cols, n = across ? W->cols : W->rows;
  if (const int st = check_ckpt(x, x->tokens, k); st != MUON_OK) return st;
  if (x->format != MUON_CKPT_E4M3) return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add_ckpt(x, false);
  add_weight8(b, W, false);
  Call c{};
  c.type = dtype == MUON_DTYPE_BF16 ? LIN_E4M3 : LIN_E4M3_EXACT;
  c.across = false;      // either copy of the weight is read along its rows
  c.out_es = elem_size(dtype);
  const int64_t br = blocks(W->rows), bc = blocks(W->cols);
  c.p.x = x->q;
  c.p.ldx = MUON_CKPT_Q_PITCH(k);
  c.p.x_scale = x->scale;
  c.p.xs_pitch = MUON_CKPT_SCALE_PITCH(k);
  c.p.W = across ? W->q_t : W->q;
  c.p.ldw = (across ? br : bc) * SIDE;
  c.p.w_stride = n * c.p.ldw;
  c.p.w_scale = W->scale;
  c.p.ws_row = across ? 1 : bc;
  c.p.ws_col = across ? bc : 1;
  c.p.ws_stride = br * bc;
  c.p.tokens = x->tokens;
  c.p.k = int(k);
  c.p.n = int(n);
  c.p.y = y;
  return run(c, offsets, W->count, b, name, stream);
}

}  // namespace

extern "C" {

int muon_weight_quantize(const void* W, int dtype, const muon_weight8* out, void* stream) {
  if (!dtype_ok(dtype)) return MUON_ERR_UNSUPPORTED_DTYPE;
  if (const int st = check_weight8(out); st != MUON_OK) return st;
  if (out->count == 0) return MUON_OK;
  const size_t es = elem_size(dtype);
  if (!W || !aligned(W, es)) return MUON_ERR_INVALID_ARGUMENT;
  Buffers b;
  b.add(W, size_t(out->count) * size_t(out->rows) * size_t(out->cols) * es, false);
  add_weight8(b, out, true);
  if (b.clash()) return MUON_ERR_INVALID_ARGUMENT;
  // a grid of up to 2^24 - 1 blocks of threads
  if (out->count * blocks(out->rows) * blocks(out->cols) >= (int64_t(1) << 24)) return MUON_ERR_INVALID_SHAPE;
  Weight8 p{};
  p.W = W;
  p.q = static_cast<uint8_t*>(out->q);
  p.q_t = static_cast<uint8_t*>(out->q_t);
  p.scale = out->scale;
  p.count = out->count;
  p.rows = int(out->rows);
  p.cols = int(out->cols);
  Trace t("muon_weight_quantize");
  hipStream_t s = static_cast<hipStream_t>(stream);
  return launched(launch_weight_quantize(p, dtype == MUON_DTYPE_BF16, s), "weight_quantize", s);
}

int muon_linear_kernel(int input_grad, int quantized, int64_t count, int64_t tokens, int64_t rows,
                       int64_t cols, int dtype) {
  if (!dtype_ok(dtype) || count < 1 || !weight_sizes_ok(count, rows, cols) || !sizes_ok(tokens, cols) || tokens < 1)
    return -1;
  const LinearType type = !quantized ? (dtype == MUON_DTYPE_BF16 ? LIN_BF16 : LIN_F32)
                                     : (dtype == MUON_DTYPE_BF16 ? LIN_E4M3 : LIN_E4M3_EXACT);
  const LinearPlan plan = input_grad ? linear_plan(type, !quantized, count, tokens, rows, cols)
                                     : linear_plan(type, false, count, tokens, cols, rows);
  return plan == LIN_NONE ? -1 : int(plan);
}

int muon_linear_forward(const void* x, int64_t ldx, int dtype, const void* W, const int64_t* offsets,
                        int64_t count, int64_t tokens, int64_t rows, int64_t cols, void* y,
                        void* stream) {
  return run_plain(false, x, ldx, dtype, W, offsets, count, tokens, rows, cols, y,
                   "muon_linear_forward", stream);
}

int muon_linear_input_grad(const void* dy, int64_t lddy, int dtype, const void* W,
                           const int64_t* offsets, int64_t count, int64_t tokens, int64_t rows,
                           int64_t cols, void* dx, void* stream) {
  return run_plain(true, dy, lddy, dtype, W, offsets, count, tokens, rows, cols, dx,
                   "muon_linear_input_grad", stream);
}

int muon_linear_forward_quantized(const muon_ckpt* x, const muon_weight8* W, const int64_t* offsets,
                                  void* y, int dtype, void* stream) {
  return run_quantized(false, x, W, offsets, y, dtype, "muon_linear_forward_quantized", stream);
}

int muon_linear_input_grad_quantized(const muon_ckpt* dy, const muon_weight8* W,
                                     const int64_t* offsets, void* dx, int dtype, void* stream) {
  return run_quantized(true, dy, W, offsets, dx, dtype, "muon_linear_input_grad_quantized", stream);
}

}  // extern "C"
