// C-ABI of the operators around the layer: routing by scores, bias and groups,
// the norms of a block with its gate and residual, 8-bit linear products.
// Argument checks only; the kernels are in route.hip, block_norm.hip and
// int8_linear.hip.
#include <hip/hip_runtime.h>

#include <cmath>

#include "nvfp4_moe.h"
#include "kernels.hpp"
#include "moe_layout.hpp"

namespace nvfp4 {

namespace {

int64_t dtype_bytes(int32_t d) { return d == MOE_F32 ? 4 : d == MOE_BF16 || d == MOE_F16 ? 2 : 0; }

// Bytes from the first to the last element of rows of `cols` elements `ld`
// apart (the largest int64 where that is more).
int64_t span(int64_t rows, int64_t ld, int64_t cols, int64_t bytes) {
  if (rows <= 0 || cols <= 0) return 0;
  const __int128 n = (static_cast<__int128>(rows - 1) * ld + cols) * bytes;
  return n > INT64_MAX ? INT64_MAX : static_cast<int64_t>(n);
}

bool row_vectors(const void* p, int64_t ld, int64_t bytes) { return !p || (aligned(p, 16) && (ld * bytes) % 16 == 0); }

int check_norm(const moe_norm* n, const char* which, int64_t bytes) {
  if (n->kind != MOE_NORM_RMS && n->kind != MOE_NORM_LAYER)
    return api_fail(NVFP4_ERR_INVALID_ARG, "%s: unknown norm kind %d", which, n->kind);
  if (!std::isfinite(n->eps) || n->eps < 0.0f || !std::isfinite(n->offset))
    return api_fail(NVFP4_ERR_INVALID_ARG, "%s: eps must be finite and >= 0, offset finite", which);
  if ((n->weight_dev && !aligned(n->weight_dev, bytes)) || (n->bias_dev && !aligned(n->bias_dev, bytes)))
    return api_fail(NVFP4_ERR_INVALID_ARG, "%s: weight and bias must be aligned to their element", which);
  return NVFP4_OK;
}

NormParams norm_params(const moe_norm* n) {
  if (!n) return NormParams{-1, 0.0f, 0.0f, nullptr, nullptr};
  return NormParams{n->kind, n->eps, n->offset, n->weight_dev, n->bias_dev};
}

// Argument checks of the two 8-bit entry points (status; 0 rows pass early)
// and their launches.
int check_quantize(const void* x_dev, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_x, const void* codes_dev,
                   int64_t ld_codes, const float* scale_dev) {
  const int64_t bytes = dtype_bytes(dtype);
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (rows < 0 || rows > INT32_MAX)
    return api_fail(NVFP4_ERR_INVALID_ARG, "rows must be in [0, 2^31) (got %lld)", (long long)rows);
  if (cols < 1 || cols > (int64_t(1) << 30))
    return api_fail(NVFP4_ERR_INVALID_ARG, "cols must be in [1, 2^30] (got %lld)", (long long)cols);
  if (ld_x < cols) return api_fail(NVFP4_ERR_INVALID_ARG, "ld_x must be >= cols (got %lld)", (long long)ld_x);
  if (ld_codes < cols || ld_codes % 16 != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "ld_codes must be >= cols and a multiple of 16 (got %lld)",
                    (long long)ld_codes);
  if (rows == 0) return NVFP4_OK;
  if (!x_dev || !codes_dev || !scale_dev) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned(x_dev, bytes) || !aligned(codes_dev, 16) || !aligned(scale_dev, 4))
    return api_fail(NVFP4_ERR_INVALID_ARG, "codes must be 16-byte aligned, x and scale to their element");
  const int64_t nx = span(rows, ld_x, cols, bytes), nc = span(rows, ld_codes, (cols + 15) / 16 * 16, 1);
  if (overlap(codes_dev, nc, x_dev, nx) || overlap(scale_dev, rows * 4, x_dev, nx) ||
      overlap(scale_dev, rows * 4, codes_dev, nc))
    return api_fail(NVFP4_ERR_ALIAS, "codes and scale must not overlap x or each other");
  return NVFP4_OK;
}

int run_quantize(const void* x_dev, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_x, void* codes_dev,
                 int64_t ld_codes, float* scale_dev, void* stream) {
  hipError_t e = launch_int8_quantize_rows(x_dev, dtype, rows, cols, ld_x, static_cast<int8_t*>(codes_dev), ld_codes,
                                           scale_dev, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "int8_quantize_per_token launch");
  return api_ok();
}

int check_matmul_sizes(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb) {
  // (the last tile's row and channel numbers also stay below 2^31)
  if (M < 0 || N < 0 || M > INT32_MAX - 512 || N > INT32_MAX - 512)
    return api_fail(NVFP4_ERR_INVALID_ARG, "M and N must be in [0, 2^31 - 512) (got %lld, %lld)", (long long)M,
                    (long long)N);
  if (K < 1 || K > 131071)
    return api_fail(NVFP4_ERR_INVALID_ARG, "K must be in [1, 131071], the range of 32-bit sums (got %lld)",
                    (long long)K);
  if (lda < K || ldb < K || lda % 16 != 0 || ldb % 16 != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "lda and ldb must be >= K and multiples of 16 (got %lld, %lld)",
                    (long long)lda, (long long)ldb);
  if (lda > (int64_t(1) << 26) || ldb > (int64_t(1) << 26))
    return api_fail(NVFP4_ERR_INVALID_ARG, "lda and ldb must be <= 2^26 (got %lld, %lld)", (long long)lda,
                    (long long)ldb);
  return NVFP4_OK;
}

int check_matmul(const void* a_dev, int64_t lda, const float* scale_a_dev, const void* b_dev, int64_t ldb,
                 const float* scale_b_dev, const float* bias_dev, int64_t M, int64_t N, int64_t K, const void* out_dev,
                 int32_t dtype, int64_t ldo) {
  const int64_t bytes = dtype_bytes(dtype);
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  const int st = check_matmul_sizes(M, N, K, lda, ldb);
  if (st != NVFP4_OK) return st;
  if (ldo < N) return api_fail(NVFP4_ERR_INVALID_ARG, "ldo must be >= N (got %lld)", (long long)ldo);
  if (M == 0 || N == 0) return NVFP4_OK;
  if (!a_dev || !b_dev || !scale_a_dev || !scale_b_dev || !out_dev)
    return api_fail(NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned(a_dev, 16) || !aligned(b_dev, 16) || !aligned(scale_a_dev, 4) || !aligned(scale_b_dev, 4) ||
      !aligned(bias_dev, 4) || !aligned(out_dev, bytes))
    return api_fail(NVFP4_ERR_INVALID_ARG, "codes must be 16-byte aligned, scales, bias and out to their element");
  const int64_t K16 = (K + 15) / 16 * 16, no = span(M, ldo, N, bytes);
  if (overlap(out_dev, no, a_dev, span(M, lda, K16, 1)) || overlap(out_dev, no, b_dev, span(N, ldb, K16, 1)) ||
      overlap(out_dev, no, scale_a_dev, M * 4) || overlap(out_dev, no, scale_b_dev, N * 4) ||
      (bias_dev && overlap(out_dev, no, bias_dev, N * 4)))
    return api_fail(NVFP4_ERR_ALIAS, "out overlaps an input");
  return NVFP4_OK;
}

Int8GemmParams gemm_params(const void* a_dev, int64_t lda, const float* scale_a_dev, const void* b_dev, int64_t ldb,
                           const float* scale_b_dev, const float* bias_dev, int64_t M, int64_t N, int64_t K,
                           void* out_dev, int32_t dtype, int64_t ldo) {
  Int8GemmParams p{};
  p.a = static_cast<const int8_t*>(a_dev);
  p.b = static_cast<const int8_t*>(b_dev);
  p.sa = scale_a_dev;
  p.sb = scale_b_dev;
  p.bias = bias_dev;
  p.out = out_dev;
  p.lda = lda;
  p.ldb = ldb;
  p.ldo = ldo;
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.dtype = dtype;
  return p;
}

int run_matmul(const void* a_dev, int64_t lda, const float* scale_a_dev, const void* b_dev, int64_t ldb,
               const float* scale_b_dev, const float* bias_dev, int64_t M, int64_t N, int64_t K, void* out_dev,
               int32_t dtype, int64_t ldo, void* stream) {
  hipError_t e = launch_int8_matmul(
      gemm_params(a_dev, lda, scale_a_dev, b_dev, ldb, scale_b_dev, bias_dev, M, N, K, out_dev, dtype, ldo),
      static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "int8_matmul launch");
  return api_ok();
}

// int8_linear's workspace: the codes (rows of whole 16-byte pieces), then the
// scales; none for a single token, which one kernel quantizes and multiplies.
bool linear_in_one(int64_t M, int64_t K) { return (M == 1 && K <= kLinearTokenMaxK) || linear_few_tokens(M, K); }
int64_t linear_codes_bytes(int64_t M, int64_t K) { return M * ((K + 15) / 16 * 16); }

}  // namespace

int check_router(const moe_router* r, int64_t E, int64_t top_k) {
  if (!r) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL router");
  if (E < 1 || E > kMaxExperts) return api_fail(NVFP4_ERR_INVALID_ARG, "num_experts must be in [1, %d]", kMaxExperts);
  if (top_k < 1 || top_k > kMaxTopK || top_k > E)
    return api_fail(NVFP4_ERR_INVALID_ARG, "top_k must be in [1, min(%d, num_experts)]", kMaxTopK);
  if (r->score != MOE_SCORE_SOFTMAX && r->score != MOE_SCORE_SIGMOID)
    return api_fail(NVFP4_ERR_INVALID_ARG, "unknown router score %d", r->score);
  if (r->num_groups < 1 || r->num_groups > kMaxRouteGroups || E % r->num_groups != 0)
    return api_fail(NVFP4_ERR_INVALID_ARG, "num_groups must be in [1, %d] and divide num_experts (got %d)",
                    kMaxRouteGroups, r->num_groups);
  if (r->top_groups < 1 || r->top_groups > r->num_groups || r->top_groups * (E / r->num_groups) < top_k)
    return api_fail(NVFP4_ERR_INVALID_ARG,
                    "top_groups must be in [1, num_groups] and its groups hold top_k experts (got %d of %d)",
                    r->top_groups, r->num_groups);
  if (r->group_best != 1 && r->group_best != 2)
    return api_fail(NVFP4_ERR_INVALID_ARG, "group_best must be 1 or 2 (got %d)", r->group_best);
  if (r->renormalize != 0 && r->renormalize != 1)
    return api_fail(NVFP4_ERR_INVALID_ARG, "renormalize must be 0 or 1 (got %d)", r->renormalize);
  if (!std::isfinite(r->scale)) return api_fail(NVFP4_ERR_INVALID_ARG, "router scale must be finite");
  return NVFP4_OK;
}

RouteParams route_params(const moe_router& r, int64_t E, int64_t top_k) {
  RouteParams q{};
  q.E = static_cast<int>(E);
  q.k = static_cast<int>(top_k);
  q.score = r.score;
  q.groups = r.num_groups;
  q.top_groups = r.top_groups;
  q.group_best = r.group_best;
  q.renormalize = r.renormalize;
  q.scale = r.scale;
  const int64_t per_group = E / r.num_groups;
  q.group_magic = static_cast<uint32_t>(((int64_t(1) << 20) + per_group - 1) / per_group);
  return q;
}

}  // namespace nvfp4

using namespace nvfp4;

extern "C" {

int moe_route(const moe_router* r, const void* logits_dev, int32_t dtype, int64_t T, int64_t E, int64_t ld,
              int32_t top_k, const float* bias_dev, int32_t* ids_dev, float* weights_dev, void* stream) {
  int st = check_router(r, E, top_k);
  if (st != NVFP4_OK) return st;
  const int64_t bytes = dtype_bytes(dtype);
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d", dtype);
  if (T < 0 || T > INT32_MAX / top_k)
    return api_fail(NVFP4_ERR_INVALID_ARG, "T must be >= 0 and T * top_k < 2^31 (got T = %lld)", (long long)T);
  if (ld < E) return api_fail(NVFP4_ERR_INVALID_ARG, "ld must be >= num_experts (got %lld)", (long long)ld);
  if (T == 0) return api_ok();
  if (!logits_dev || !ids_dev || !weights_dev) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned(logits_dev, bytes) || !aligned(bias_dev, 4) || !aligned(ids_dev, 4) || !aligned(weights_dev, 4))
    return api_fail(NVFP4_ERR_INVALID_ARG, "logits, bias, ids and weights must be aligned to their element");
  const int64_t nl = span(T, ld, E, bytes), no = T * top_k * 4, nb = bias_dev ? E * 4 : 0;
  if (overlap(ids_dev, no, logits_dev, nl) || overlap(weights_dev, no, logits_dev, nl) ||
      overlap(ids_dev, no, bias_dev, nb) || overlap(weights_dev, no, bias_dev, nb) ||
      overlap(ids_dev, no, weights_dev, no))
    return api_fail(NVFP4_ERR_ALIAS, "ids and weights must not overlap the inputs or each other");
  RouteParams q = route_params(*r, E, top_k);
  q.logits = logits_dev;
  q.bias = bias_dev;
  q.ids = ids_dev;
  q.weights = weights_dev;
  q.ld = ld;
  q.T = static_cast<int>(T);
  q.dtype = dtype;
  hipError_t e = launch_route_scores(q, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "moe_route launch");
  return api_ok();
}

int moe_block_norm(const moe_block_norm_args* args, void* stream) {
  if (!args) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL arguments");
  const moe_block_norm_args a = *args;
  const int64_t bytes = dtype_bytes(a.dtype), rbytes = dtype_bytes(a.residual_dtype);
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d", a.dtype);
  if (a.residual_dtype != a.dtype && a.residual_dtype != MOE_F32)
    return api_fail(NVFP4_ERR_INVALID_ARG, "residual_dtype must be dtype or MOE_F32 (got %d)", a.residual_dtype);
  if (a.rows < 0 || a.rows > INT32_MAX)
    return api_fail(NVFP4_ERR_INVALID_ARG, "rows must be in [0, 2^31) (got %lld)", (long long)a.rows);
  if (a.cols < 1 || a.cols > 65536)
    return api_fail(NVFP4_ERR_INVALID_ARG, "cols must be in [1, 65536] (got %lld)", (long long)a.cols);
  if (a.ld_residual < a.cols || (a.y_dev && a.ld_y < a.cols) || (a.residual_out_dev && a.ld_residual_out < a.cols) ||
      (a.h_dev && a.ld_h < a.cols))
    return api_fail(NVFP4_ERR_INVALID_ARG, "leading dimensions must be >= cols");
  if (a.gate_dev && ((a.gate_cols != 1 && a.gate_cols != a.cols) || (a.ld_gate != 0 && a.ld_gate < a.gate_cols)))
    return api_fail(NVFP4_ERR_INVALID_ARG, "gate_cols must be 1 or cols, ld_gate 0 or >= gate_cols");
  if (a.gate_sigmoid != 0 && a.gate_sigmoid != 1)
    return api_fail(NVFP4_ERR_INVALID_ARG, "gate_sigmoid must be 0 or 1 (got %d)", a.gate_sigmoid);
  if (!std::isfinite(a.res_scale) || !std::isfinite(a.out_scale))
    return api_fail(NVFP4_ERR_INVALID_ARG, "res_scale and out_scale must be finite");
  int st = a.after ? check_norm(a.after, "after", bytes) : NVFP4_OK;
  if (st == NVFP4_OK && a.before) st = check_norm(a.before, "before", bytes);
  if (st != NVFP4_OK) return st;
  if (a.rows == 0) return api_ok();
  if (!a.y_dev && (a.after || a.gate_dev))
    return api_fail(NVFP4_ERR_INVALID_ARG, "a norm after the block and a gate need its output y");
  if (a.h_dev && !a.before) return api_fail(NVFP4_ERR_INVALID_ARG, "h needs a norm (before)");
  if (a.before && !a.h_dev) return api_fail(NVFP4_ERR_INVALID_ARG, "a norm before the next block needs h");
  if (!a.residual_dev || (!a.residual_out_dev && !a.h_dev))
    return api_fail(NVFP4_ERR_INVALID_ARG, "NULL pointer argument");
  if (!aligned(a.residual_dev, rbytes) || !aligned(a.residual_out_dev, rbytes) || !aligned(a.y_dev, bytes) ||
      !aligned(a.gate_dev, bytes) || !aligned(a.h_dev, bytes))
    return api_fail(NVFP4_ERR_INVALID_ARG, "tensors must be aligned to their element");

  const int64_t nr = span(a.rows, a.ld_residual, a.cols, rbytes);
  const int64_t ny = a.y_dev ? span(a.rows, a.ld_y, a.cols, bytes) : 0;
  const int64_t ng = a.gate_dev ? span(a.ld_gate ? a.rows : 1, a.ld_gate, a.gate_cols, bytes) : 0;
  const int64_t no = a.residual_out_dev ? span(a.rows, a.ld_residual_out, a.cols, rbytes) : 0;
  const int64_t nh = a.h_dev ? span(a.rows, a.ld_h, a.cols, bytes) : 0;
  const bool in_place_r = a.residual_out_dev == a.residual_dev && a.ld_residual_out == a.ld_residual;
  const bool in_place_y = a.h_dev == a.y_dev && a.ld_h == a.ld_y;
  bool bad = (!in_place_r && overlap(a.residual_out_dev, no, a.residual_dev, nr)) ||
             (!in_place_y && overlap(a.h_dev, nh, a.y_dev, ny)) || overlap(a.residual_out_dev, no, a.y_dev, ny) ||
             overlap(a.h_dev, nh, a.residual_dev, nr) || overlap(a.residual_out_dev, no, a.h_dev, nh) ||
             overlap(a.residual_out_dev, no, a.gate_dev, ng) || overlap(a.h_dev, nh, a.gate_dev, ng);
  for (const moe_norm* n : {a.after, a.before}) {
    if (!n) continue;
    for (const void* w : {n->weight_dev, n->bias_dev})
      bad = bad || (w && (overlap(a.residual_out_dev, no, w, a.cols * bytes) || overlap(a.h_dev, nh, w, a.cols * bytes)));
  }
  if (bad)
    return api_fail(NVFP4_ERR_ALIAS,
                    "an output overlaps another tensor (only residual_out = residual and h = y, with equal leading "
                    "dimensions, are in place)");

  BlockNormParams p{};
  p.rows = a.rows;
  p.cols = static_cast<int>(a.cols);
  p.r = a.residual_dev;
  p.y = a.y_dev;
  p.gate = a.gate_dev;
  p.ld_r = a.ld_residual;
  p.ld_y = a.ld_y;
  p.ld_gate = a.ld_gate;
  p.gate_cols = static_cast<int>(a.gate_cols);
  p.gate_sigmoid = a.gate_sigmoid;
  p.res_scale = a.res_scale;
  p.out_scale = a.out_scale;
  p.after = norm_params(a.after);
  p.before = norm_params(a.before);
  p.r_out = a.residual_out_dev;
  p.h = a.h_dev;
  p.ld_r_out = a.ld_residual_out;
  p.ld_h = a.ld_h;
  // whole 16-byte pieces where every row starts on one and cols fills them
  bool vec = a.cols % 8 == 0 && row_vectors(a.residual_dev, a.ld_residual, rbytes) &&
             row_vectors(a.y_dev, a.ld_y, bytes) && row_vectors(a.residual_out_dev, a.ld_residual_out, rbytes) &&
             row_vectors(a.h_dev, a.ld_h, bytes) &&
             (a.gate_cols == 1 || row_vectors(a.gate_dev, a.ld_gate, bytes));
  for (const NormParams* n : {&p.after, &p.before})
    vec = vec && row_vectors(n->weight, 0, bytes) && row_vectors(n->bias, 0, bytes);
  hipError_t e = launch_block_norm(p, a.dtype, a.residual_dtype, vec, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "moe_block_norm launch");
  return api_ok();
}

int int8_quantize_per_token(const void* x_dev, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_x,
                            void* codes_dev, int64_t ld_codes, float* scale_dev, void* stream) {
  const int st = check_quantize(x_dev, dtype, rows, cols, ld_x, codes_dev, ld_codes, scale_dev);
  if (st != NVFP4_OK) return st;
  if (rows == 0) return api_ok();
  return run_quantize(x_dev, dtype, rows, cols, ld_x, codes_dev, ld_codes, scale_dev, stream);
}

int int8_matmul(const void* a_dev, int64_t lda, const float* scale_a_dev, const void* b_dev, int64_t ldb,
                const float* scale_b_dev, const float* bias_dev, int64_t M, int64_t N, int64_t K, void* out_dev,
                int32_t dtype, int64_t ldo, void* stream) {
  const int st =
      check_matmul(a_dev, lda, scale_a_dev, b_dev, ldb, scale_b_dev, bias_dev, M, N, K, out_dev, dtype, ldo);
  if (st != NVFP4_OK) return st;
  if (M == 0 || N == 0) return api_ok();
  return run_matmul(a_dev, lda, scale_a_dev, b_dev, ldb, scale_b_dev, bias_dev, M, N, K, out_dev, dtype, ldo, stream);
}

int int8_matmul_kernel(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int32_t* kernel) {
  const int st = check_matmul_sizes(M, N, K, lda, ldb);
  if (st != NVFP4_OK) return st;
  if (M == 0 || N == 0 || !kernel) return api_fail(NVFP4_ERR_INVALID_ARG, "M and N must be >= 1, kernel not NULL");
  *kernel = choose_int8_kernel(M, N, K, lda, ldb);
  return api_ok();
}

int int8_linear_workspace(int64_t M, int64_t K, int64_t* bytes) {
  if (!bytes) return api_fail(NVFP4_ERR_INVALID_ARG, "NULL output");
  if (M < 0 || M > INT32_MAX || K < 1 || K > 131071)
    return api_fail(NVFP4_ERR_INVALID_ARG, "M must be in [0, 2^31) and K in [1, 131071] (got %lld, %lld)",
                    (long long)M, (long long)K);
  *bytes = linear_in_one(M, K) ? 0 : linear_codes_bytes(M, K) + M * 4;
  return api_ok();
}

int int8_linear(const void* x_dev, int32_t dtype, int64_t ld_x, const void* w_dev, int64_t ldw,
                const float* scale_w_dev, const float* bias_dev, int64_t M, int64_t N, int64_t K,
                void* workspace_dev, int64_t workspace_bytes, void* out_dev, int32_t out_dtype, int64_t ldo,
                void* stream) {
  const int64_t xb = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  if (!xb || !ob) return api_fail(NVFP4_ERR_INVALID_ARG, "unknown dtype %d or %d", dtype, out_dtype);
  int64_t need = 0;
  int st = int8_linear_workspace(M, K, &need);
  if (st != NVFP4_OK) return st;
  const int64_t ldc = (K + 15) / 16 * 16;
  if (need > 0 && (!workspace_dev || !aligned(workspace_dev, 16) || workspace_bytes < need))
    return api_fail(NVFP4_ERR_INVALID_ARG, "workspace must be 16-byte aligned, of at least %lld bytes (got %lld)",
                    (long long)need, (long long)workspace_bytes);
  // Both steps' checks first (nothing is enqueued on an error); where no codes
  // are kept, with addresses of their alignment that nothing reads or writes.
  const bool one = linear_in_one(M, K);
  char* const codes = one ? reinterpret_cast<char*>(uintptr_t{16}) : static_cast<char*>(workspace_dev);
  float* const scales = reinterpret_cast<float*>(codes + linear_codes_bytes(M, K));
  st = check_matmul(codes, ldc, scales, w_dev, ldw, scale_w_dev, bias_dev, M, N, K, out_dev, out_dtype, ldo);
  if (st != NVFP4_OK) return st;
  if (M == 0 || N == 0) return api_ok();
  st = check_quantize(x_dev, dtype, M, K, ld_x, codes, ldc, scales);
  if (st != NVFP4_OK) return st;
  if (overlap(out_dev, span(M, ldo, N, ob), x_dev, span(M, ld_x, K, xb)) ||
      overlap(codes, need, w_dev, span(N, ldw, ldc, 1)) || overlap(codes, need, scale_w_dev, N * 4) ||
      (bias_dev && overlap(codes, need, bias_dev, N * 4)))
    return api_fail(NVFP4_ERR_ALIAS, "out or workspace overlaps an input");
  if (one || linear_few_tiles(M, N, K)) {
    const Int8GemmParams p = gemm_params(nullptr, ldc, nullptr, w_dev, ldw, scale_w_dev, bias_dev, M, N, K, out_dev,
                                         out_dtype, ldo);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const hipError_t e = M == 1 ? launch_int8_token(p, x_dev, dtype, s) : launch_int8_few(p, x_dev, ld_x, dtype, s);
    if (e != hipSuccess) return hip_fail(e, "int8_linear launch");
    return api_ok();
  }
  st = run_quantize(x_dev, dtype, M, K, ld_x, codes, ldc, scales, stream);
  if (st != NVFP4_OK) return st;
  return run_matmul(codes, ldc, scales, w_dev, ldw, scale_w_dev, bias_dev, M, N, K, out_dev, out_dtype, ldo, stream);
}

}  // extern "C"
