// Entry points of the expert products and the 8-bit block operators:
// argument checks and launches.  Nothing is staged in memory (the arguments
// travel with the launch), so these calls may be captured into a graph.
#include <initializer_list>

#include "internal.h"

namespace dmuon {
namespace {

constexpr int64_t kMaxDim = int64_t(1) << 22;       // features, row strides
constexpr int64_t kMaxRows = int64_t(1) << 30;      // tokens
constexpr int64_t kMaxStride = int64_t(1) << 44;    // between experts' weights or a batch's matrices
constexpr int32_t kMaxExperts = 65536;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 4096;   // blocks of 256 threads in one launch

int bad(const std::string& msg) { return set_last_error(DMUON_ERR_INVALID_ARG, msg); }

bool real_dtype(int32_t dt) { return dt == DT_F32 || dt == DT_BF16; }
bool q8_dtype(int32_t dt) { return dt == DT_E4M3 || dt == DT_E5M2; }
int64_t size_of(int32_t dt) { return dt == DT_F32 ? 4 : dt == DT_BF16 ? 2 : 1; }
int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

struct Span {
  const void* p;
  int64_t bytes;      // from the first to one past the last
  const char* name;
};

// The written buffers (the first `nout`) must not overlap each other or anything read.
int check_spans(std::initializer_list<Span> spans, int nout) {
  int i = 0;
  for (const Span& a : spans) {
    if (i++ >= nout) break;
    if (!a.p || a.bytes <= 0) continue;
    int j = 0;
    for (const Span& b : spans) {
      if (j++ < i || !b.p || b.bytes <= 0) continue;
      const uintptr_t al = reinterpret_cast<uintptr_t>(a.p), bl = reinterpret_cast<uintptr_t>(b.p);
      if (al < bl + uintptr_t(b.bytes) && bl < al + uintptr_t(a.bytes))
        return set_last_error(DMUON_ERR_ALIASING, std::string(a.name) + " overlaps " + b.name);
    }
  }
  return DMUON_OK;
}

int hip_status(hipError_t e, const char* what) {
  return e == hipSuccess ? DMUON_OK
                         : set_last_error(DMUON_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
}

int64_t product_flops(int64_t m, int64_t n, int64_t k) {
  const double f = 2.0 * double(m) * double(n) * double(k);   // beyond int64 for the largest allowed sizes
  return f < 9e18 ? static_cast<int64_t>(f) : INT64_MAX;
}

int64_t rows_bytes(int64_t rows, int64_t ld, int64_t cols, int64_t size) {
  return rows <= 0 ? 0 : ((rows - 1) * ld + cols) * size;
}

int expert_product(int op, const dmuon_experts_t* d, const void* a, const void* b, const int32_t* offsets, void* c,
                   void* stream_) {
  set_last_error("");
  if (!d) return bad("experts descriptor is NULL");
  if (d->tokens < 0 || d->tokens > kMaxRows) return bad("tokens must be in 0..2^30");
  if (d->n < 1 || d->n > kMaxDim || d->k < 1 || d->k > kMaxDim) return bad("n and k must be in 1..2^22");
  if (d->experts < 1 || d->experts > kMaxExperts) return bad("experts must be in 1..65536");
  if (d->ld_k < d->k || d->ld_k > kMaxDim || d->ld_n < d->n || d->ld_n > kMaxDim || d->ldw < d->k ||
      d->ldw > kMaxDim)
    return bad("row strides must be at least the row and at most 2^22");
  if (d->experts > 1 && (d->w_stride < (d->n - 1) * d->ldw + d->k || d->w_stride > kMaxStride))
    return bad("w_stride must be at least one expert's weights and at most 2^44");
  if (d->accumulate != 0 && d->accumulate != 1) return bad("accumulate must be 0 or 1");
  if (d->accumulate && op != OP_WEIGHT) return bad("accumulate is for the weight gradient");
  if (!real_dtype(d->dtype)) return set_last_error(DMUON_ERR_UNSUPPORTED, "dtype must be F32 or BF16");
  const int32_t out = op == OP_WEIGHT ? d->out_dtype : d->dtype;
  if (!real_dtype(out) || (d->dtype == DT_F32 && out != DT_F32))
    return set_last_error(DMUON_ERR_UNSUPPORTED, "out_dtype must be F32, or BF16 with bf16 operands");
  if (d->tokens == 0 && (op != OP_WEIGHT || d->accumulate)) return DMUON_OK;
  if (!offsets || !c || (d->tokens > 0 && (!a || !b)) || (op != OP_WEIGHT && !b))
    return bad("a buffer or offsets is NULL");
  const int64_t sz = size_of(d->dtype), osz = size_of(out);
  if (!aligned(a, sz) || !aligned(b, sz) || !aligned(c, osz) || !aligned(offsets, 4))
    return bad("a buffer is not aligned to its element");
  const int64_t xk = rows_bytes(d->tokens, d->ld_k, d->k, 1), xn = rows_bytes(d->tokens, d->ld_n, d->n, 1);
  const int64_t wb = (d->experts - 1) * d->w_stride + (d->n - 1) * d->ldw + d->k;
  const int64_t ab = (op == OP_FORWARD ? xk : xn) * sz, bb = (op == OP_WEIGHT ? xk : wb) * sz;
  const int64_t cbytes = (op == OP_FORWARD ? xn : op == OP_INPUT ? xk : wb) * osz;
  int st = check_spans({{c, cbytes, "the result"}, {a, ab, "the first operand"}, {b, bb, "the second operand"},
                        {offsets, 4 * (int64_t(d->experts) + 1), "offsets"}}, 1);
  if (st) return st;
  int64_t blocks;
  if (op == OP_WEIGHT)
    blocks = d->experts * up(d->n, 128) * up(d->k, 128);
  else
    blocks = (d->tokens / 128 + (d->experts < d->tokens ? d->experts : d->tokens)) *
             up(op == OP_FORWARD ? d->n : d->k, 128);
  if (blocks > kMaxBlocks) return set_last_error(DMUON_ERR_UNSUPPORTED, "more than 2^24 tiles of 128 x 128");
  st = check_current_device();
  if (st) return st;
  ExpertArgs P;
  P.a = a; P.b = b; P.c = c; P.offsets = offsets;
  P.n = d->n; P.k = d->k;
  P.ld_k = d->ld_k; P.ld_n = d->ld_n; P.ldw = d->ldw; P.w_stride = d->w_stride;
  P.experts = d->experts; P.tokens = static_cast<int32_t>(d->tokens);
  P.accumulate = d->accumulate;
  // whole 16-byte chunks along every operand's contiguous dimension
  auto chunks = [&](const void* p, int64_t cols, int64_t ld) {
    return aligned(p, 16) && cols * sz % 16 == 0 && ld * sz % 16 == 0;
  };
  bool vec;
  if (op == OP_FORWARD) vec = chunks(a, d->k, d->ld_k) && chunks(b, d->k, d->ldw);
  else if (op == OP_INPUT) vec = chunks(a, d->n, d->ld_n) && chunks(b, d->k, d->ldw);
  else vec = chunks(a, d->n, d->ld_n) && chunks(b, d->k, d->ld_k);
  if (op != OP_WEIGHT) vec = vec && (d->w_stride * sz % 16 == 0 || d->experts == 1);
  const hipStream_t stream = static_cast<hipStream_t>(stream_);
  const int64_t flops = product_flops(d->tokens, d->n, d->k);
  return hip_status(profiled_launch(d->dtype == DT_F32 ? PK_EXPERT_F32 : PK_EXPERT_BF16, flops, ab + bb + cbytes, stream,
                                    [&] { return launch_expert_product(op, P, d->dtype, out, vec, stream); }),
                    "expert product");
}

int check_blocks(const dmuon_blocks_t* d) {
  if (!d) return bad("blocks descriptor is NULL");
  if (d->batch < 1 || d->batch > 65535) return bad("batch must be in 1..65535");
  if (d->rows < 0 || d->rows > kMaxRows) return bad("rows must be in 0..2^30");
  if (d->cols < 1 || d->cols > kMaxDim) return bad("cols must be in 1..2^22");
  if (d->ldx < d->cols || d->ldx > kMaxDim) return bad("ldx must be at least cols and at most 2^22");
  if (d->batch > 1 && (d->x_stride < (d->rows - 1) * d->ldx + d->cols || d->x_stride > kMaxStride))
    return bad("x_stride must be at least one matrix and at most 2^44");
  if (d->block_rows != 1 && d->block_rows != 128) return bad("block_rows must be 1 or 128");
  if (!real_dtype(d->x_dtype) || !q8_dtype(d->q_dtype))
    return set_last_error(DMUON_ERR_UNSUPPORTED, "x_dtype must be F32 or BF16, q_dtype E4M3 or E5M2");
  if (up(d->rows, 16) * up(d->cols, 128) * d->batch > kMaxBlocks)
    return set_last_error(DMUON_ERR_UNSUPPORTED, "more than 2^24 pieces of 16 x 128");
  return DMUON_OK;
}

void fill_quant(const dmuon_blocks_t* d, QuantArgs* P) {
  P->batch = d->batch; P->rows = d->rows; P->cols = d->cols; P->ldx = d->ldx; P->x_stride = d->x_stride;
  P->block_rows = d->block_rows;
}

}  // namespace
}  // namespace dmuon

using namespace dmuon;

extern "C" {

int dmuon_expert_matmul(const dmuon_experts_t* d, const void* x, const void* w, const int32_t* offsets, void* y,
                        void* stream) {
  return expert_product(OP_FORWARD, d, x, w, offsets, y, stream);
}

int dmuon_expert_input_grad(const dmuon_experts_t* d, const void* dy, const void* w, const int32_t* offsets, void* dx,
                            void* stream) {
  return expert_product(OP_INPUT, d, dy, w, offsets, dx, stream);
}

int dmuon_expert_weight_grad(const dmuon_experts_t* d, const void* dy, const void* x, const int32_t* offsets, void* dw,
                             void* stream) {
  return expert_product(OP_WEIGHT, d, dy, x, offsets, dw, stream);
}

int dmuon_quantize_blocks(const dmuon_blocks_t* d, const void* x, void* q, float* scale, void* qt, float* scale_t,
                          void* stream_) {
  set_last_error("");
  int st = check_blocks(d);
  if (st) return st;
  if ((q == nullptr) != (scale == nullptr) || (qt == nullptr) != (scale_t == nullptr))
    return bad("q and scale (and qt and scale_t) come together");
  if (d->rows == 0) return DMUON_OK;
  if (!x || (!q && !qt)) return bad("x, or every output, is NULL");
  const int64_t xs = size_of(d->x_dtype);
  if (!aligned(x, xs) || !aligned(scale, 4) || !aligned(scale_t, 4)) return bad("a buffer is not aligned to its element");
  const int64_t n = d->batch * d->rows * d->cols;
  const int64_t br = d->block_rows;
  const Span sx = {x, ((d->batch - 1) * d->x_stride + rows_bytes(d->rows, d->ldx, d->cols, 1)) * xs, "x"};
  st = check_spans({{q, n, "q"}, {scale, 4 * d->batch * up(d->rows, br) * up(d->cols, 128), "scale"}, {qt, n, "qt"},
                    {scale_t, 4 * d->batch * up(d->cols, br) * up(d->rows, 128), "scale_t"}, sx}, 4);
  if (st) return st;
  st = check_current_device();
  if (st) return st;
  QuantArgs P = {};
  fill_quant(d, &P);
  P.x = x;
  P.q = static_cast<uint8_t*>(q); P.scale = scale;
  P.qt = static_cast<uint8_t*>(qt); P.scale_t = scale_t;
  P.vec_x = aligned(x, 16) && d->cols % 8 == 0 && d->ldx * xs % 16 == 0 && (d->batch == 1 || d->x_stride * xs % 16 == 0);
  const hipStream_t stream = static_cast<hipStream_t>(stream_);
  return hip_status(profiled_launch(PK_QUANTIZE, 3 * n, n * (xs + (q ? 1 : 0) + (qt ? 1 : 0)), stream,
                                    [&] { return launch_quantize(P, d->x_dtype, d->q_dtype, stream); }),
                    "quantize_blocks");
}

int dmuon_dequantize_blocks(const dmuon_blocks_t* d, const void* q, const float* scale, void* x, void* stream_) {
  set_last_error("");
  int st = check_blocks(d);
  if (st) return st;
  if (d->rows == 0) return DMUON_OK;
  if (!q || !scale || !x) return bad("a buffer is NULL");
  const int64_t xs = size_of(d->x_dtype);
  if (!aligned(x, xs) || !aligned(scale, 4)) return bad("a buffer is not aligned to its element");
  const int64_t n = d->batch * d->rows * d->cols;
  st = check_spans({{x, ((d->batch - 1) * d->x_stride + rows_bytes(d->rows, d->ldx, d->cols, 1)) * xs, "x"}, {q, n, "q"},
                    {scale, 4 * d->batch * up(d->rows, d->block_rows) * up(d->cols, 128), "scale"}}, 1);
  if (st) return st;
  st = check_current_device();
  if (st) return st;
  QuantArgs P = {};
  fill_quant(d, &P);
  P.x_out = x;
  P.q = static_cast<uint8_t*>(const_cast<void*>(q));
  P.scale = const_cast<float*>(scale);
  const hipStream_t stream = static_cast<hipStream_t>(stream_);
  return hip_status(profiled_launch(PK_DEQUANTIZE, n, n * (xs + 1), stream,
                                    [&] { return launch_dequantize(P, d->x_dtype, d->q_dtype, stream); }),
                    "dequantize_blocks");
}

int dmuon_block_matmul(const dmuon_block_product_t* d, const void* a, const float* a_scale, const void* b,
                       const float* b_scale, const int32_t* offsets, void* c, void* stream_) {
  set_last_error("");
  if (!d) return bad("product descriptor is NULL");
  if (d->m < 0 || d->m > kMaxRows) return bad("m must be in 0..2^30");
  if (d->n < 1 || d->n > kMaxDim) return bad("n must be in 1..2^22");
  if (d->k < 1 || d->k > kMaxRows) return bad("k must be in 1..2^30");
  if (d->experts < 0 || d->experts > kMaxExperts) return bad("experts must be in 0..65536");
  if ((d->experts > 0) != (offsets != nullptr)) return bad("offsets go with experts > 0");
  if (d->lda < d->k || d->lda > kMaxRows || d->ldb < d->k || d->ldb > kMaxRows || d->ldc < d->n || d->ldc > kMaxDim)
    return bad("row strides must be at least the row and at most 2^30 (a, b) or 2^22 (c)");
  if (d->experts > 1 && (d->b_stride < (d->n - 1) * d->ldb + d->k || d->b_stride > kMaxStride))
    return bad("b_stride must be at least one expert's weights and at most 2^44");
  if (d->b_block_rows != 1 && d->b_block_rows != 128) return bad("b_block_rows must be 1 or 128");
  if (d->accumulate != 0 && d->accumulate != 1) return bad("accumulate must be 0 or 1");
  if (!q8_dtype(d->a_dtype) || !q8_dtype(d->b_dtype))
    return set_last_error(DMUON_ERR_UNSUPPORTED, "a_dtype and b_dtype must be E4M3 or E5M2");
  if (!real_dtype(d->out_dtype)) return set_last_error(DMUON_ERR_UNSUPPORTED, "out_dtype must be F32 or BF16");
  if (d->m == 0) return DMUON_OK;
  if (!a || !a_scale || !b || !b_scale || !c) return bad("a buffer is NULL");
  const int64_t osz = size_of(d->out_dtype), kb = up(d->k, 128), ne = d->experts > 0 ? d->experts : 1;
  if (!aligned(a_scale, 4) || !aligned(b_scale, 4) || !aligned(c, osz) || !aligned(offsets, 4))
    return bad("a buffer is not aligned to its element");
  const int64_t ab = rows_bytes(d->m, d->lda, d->k, 1);
  const int64_t bb = (ne - 1) * d->b_stride + rows_bytes(d->n, d->ldb, d->k, 1);
  const int64_t cbytes = rows_bytes(d->m, d->ldc, d->n, osz);
  int st = check_spans({{c, cbytes, "c"}, {a, ab, "a"}, {b, bb, "b"}, {a_scale, 4 * d->m * kb, "a_scale"},
                        {b_scale, 4 * ne * up(d->n, d->b_block_rows) * kb, "b_scale"},
                        {offsets, 4 * (int64_t(d->experts) + 1), "offsets"}}, 1);
  if (st) return st;
  const int64_t used = d->experts > 0 ? (d->experts < d->m ? d->experts : d->m) : 1;
  if ((d->m / 128 + used) * up(d->n, 128) > kMaxBlocks)
    return set_last_error(DMUON_ERR_UNSUPPORTED, "more than 2^24 tiles of 128 x 128");
  st = check_current_device();
  if (st) return st;
  BlockArgs P = {};
  P.a = a; P.b = b; P.a_scale = a_scale; P.b_scale = b_scale; P.c = c; P.offsets = offsets;
  P.m = d->m; P.n = d->n; P.k = d->k; P.lda = d->lda; P.ldb = d->ldb; P.ldc = d->ldc; P.b_stride = d->b_stride;
  P.experts = d->experts; P.accumulate = d->accumulate;
  const bool vec = aligned(a, 16) && aligned(b, 16) && d->k % 16 == 0 && d->lda % 16 == 0 && d->ldb % 16 == 0 &&
                   (ne == 1 || d->b_stride % 16 == 0);
  const hipStream_t stream = static_cast<hipStream_t>(stream_);
  return hip_status(profiled_launch(PK_BLOCK_MATMUL, product_flops(d->m, d->n, d->k), ab + bb + cbytes, stream,
                                    [&] {
                                      return launch_block_matmul(P, d->a_dtype, d->b_dtype, d->b_block_rows == 1,
                                                                 d->out_dtype == DT_F32, vec, stream);
                                    }),
                    "block_matmul");
}

}  // extern "C"
