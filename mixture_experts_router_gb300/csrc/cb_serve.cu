// Host side of the C ABI in cb_serve.h: argument validation and the launches.
#include "cb_serve.h"

#include <cmath>
#include <cstdlib>
#include <cstring>
#include <initializer_list>

#include "internal.h"

using namespace cbmoe;

namespace {

bool on(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool known_type(int32_t t) { return t == CB_T_BF16 || t == CB_T_F32; }
int size_of(int32_t type) { return type == CB_T_F32 ? 4 : 2; }

bool fault_injected() {  // testing only
  const char* v = std::getenv("CB_MOE_INJECT_FAULT");
  return v != nullptr && std::strcmp(v, "launch") == 0;
}

// Bytes that a call reads or writes.
struct Span {
  const void* p;
  uint64_t bytes;
};
Span rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int size) {
  return {p, rows > 0 ? (static_cast<uint64_t>(rows - 1) * ld + cols) * size : 0};
}
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p != nullptr && b.p != nullptr && a.bytes > 0 && b.bytes > 0 && x < y + b.bytes && y < x + a.bytes;
}
bool overlaps_any(const Span& a, std::initializer_list<Span> others) {
  for (const Span& o : others)
    if (overlap(a, o)) return true;
  return false;
}

cb_status_t ready(int* sms) {
  const cb_status_t st = static_cast<cb_status_t>(check_device(sms));
  if (st != CB_OK) return st;
  return fault_injected() ? CB_ERR_CUDA : CB_OK;
}

}  // namespace

extern "C" {

cb_status_t cb_rms_norm(const cb_rms_norm_t* p, void* stream) {
  if (p == nullptr || p->rows < 0 || p->cols <= 0 || !known_type(p->x_type) || !known_type(p->weight_type) ||
      !known_type(p->out_type) || !(p->eps >= 0.f) || std::isinf(p->eps) || (p->codes != nullptr) != (p->scales != nullptr))
    return CB_ERR_INVALID_ARG;
  if (p->ld_x < p->cols || (p->residual != nullptr && p->ld_residual < p->cols) ||
      (p->sum != nullptr && p->ld_sum < p->cols) || (p->out != nullptr && p->ld_out < p->cols))
    return CB_ERR_INVALID_ARG;
  const int64_t ld_most = (1ll << 61) / (p->rows + 1);
  if (p->cols > CB_NORM_MAX_COLS || p->rows >= (1ll << 31) - 1 || p->ld_x >= ld_most || p->ld_residual >= ld_most ||
      p->ld_sum >= ld_most || p->ld_out >= ld_most)
    return CB_ERR_UNSUPPORTED;
  if (p->rows == 0) return CB_OK;
  if (p->x == nullptr || p->weight == nullptr || (p->sum == nullptr && p->out == nullptr && p->codes == nullptr))
    return CB_ERR_INVALID_ARG;
  const int size = size_of(p->x_type);
  if (!on(p->x, size) || !on(p->residual, size) || !on(p->sum, size) || !on(p->weight, size_of(p->weight_type)) ||
      !on(p->out, size_of(p->out_type)) || !on(p->scales, 4))
    return CB_ERR_ALIGNMENT;
  const Span x = rows_of(p->x, p->rows, p->cols, p->ld_x, size);
  const Span r = rows_of(p->residual, p->rows, p->cols, p->ld_residual, size);
  const Span w = {p->weight, static_cast<uint64_t>(p->cols) * size_of(p->weight_type)};
  const Span sum = rows_of(p->sum, p->rows, p->cols, p->ld_sum, size);
  const Span out = rows_of(p->out, p->rows, p->cols, p->ld_out, size_of(p->out_type));
  const Span codes = rows_of(p->codes, p->rows, p->cols, p->cols, 1);
  const int64_t groups = (p->cols + CB_FP8_COLS - 1) / CB_FP8_COLS;
  const Span scales = rows_of(p->scales, p->rows, groups, groups, 4);
  // in place: every element is read by the thread that writes it, before any of its row is written
  const bool sum_is_x = p->sum == p->x && p->ld_sum == p->ld_x;
  const bool sum_is_r = p->sum == p->residual && p->ld_sum == p->ld_residual;
  const bool out_is_x = p->out == p->x && p->ld_out == p->ld_x && p->out_type == p->x_type;
  if ((!sum_is_x && overlap(sum, x)) || (!sum_is_r && overlap(sum, r)) || (!out_is_x && overlap(out, x)) ||
      overlaps_any(w, {sum, out, codes, scales}) || overlaps_any(out, {r, sum, codes, scales}) ||
      overlaps_any(sum, {codes, scales}) || overlaps_any(codes, {x, r, scales}) || overlaps_any(scales, {x, r}))
    return CB_ERR_INVALID_ARG;
  int sms;
  const cb_status_t st = ready(&sms);
  if (st != CB_OK) return st;
  NormArgs a{};
  a.rows = p->rows;
  a.cols = static_cast<int32_t>(p->cols);
  a.x = p->x;
  a.ld_x = p->ld_x;
  a.residual = p->residual;
  a.ld_residual = p->ld_residual;
  a.weight = p->weight;
  a.sum = p->sum;
  a.ld_sum = p->ld_sum;
  a.out = p->out;
  a.ld_out = p->ld_out;
  a.codes = p->codes;
  a.scales = p->scales;
  a.eps = p->eps;
  a.f32 = p->x_type == CB_T_F32;
  a.weight_f32 = p->weight_type == CB_T_F32;
  a.out_f32 = p->out_type == CB_T_F32;
  return launch_rms_norm(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

cb_status_t cb_route(const cb_route_t* p, void* stream) {
  if (p == nullptr || p->n_tokens < 0 || p->n_experts <= 0 || p->top_k <= 0 || !known_type(p->logits_type) ||
      (p->score != CB_SCORE_SIGMOID && p->score != CB_SCORE_SOFTMAX) ||
      (p->group_score != CB_GROUP_TOP2 && p->group_score != CB_GROUP_MAX) || p->n_groups <= 0 || p->top_groups <= 0 ||
      p->top_groups > p->n_groups || p->n_experts % p->n_groups != 0 || (p->renormalise != 0 && p->renormalise != 1) ||
      !std::isfinite(p->scale) || p->ld_logits < p->n_experts)
    return CB_ERR_INVALID_ARG;
  if (p->top_k > p->top_groups * (p->n_experts / p->n_groups)) return CB_ERR_INVALID_ARG;
  if (p->n_experts > 256 || p->top_k > 16 || p->n_groups > CB_ROUTE_MAX_GROUPS || p->n_tokens >= (1ll << 31) ||
      p->ld_logits >= (1ll << 61) / (p->n_tokens + 1))
    return CB_ERR_UNSUPPORTED;
  if (p->n_tokens == 0) return CB_OK;
  if (p->logits == nullptr || p->ids == nullptr || p->w == nullptr) return CB_ERR_INVALID_ARG;
  const int size = size_of(p->logits_type);
  if (!on(p->logits, size) || !on(p->bias, 4) || !on(p->ids, 4) || !on(p->w, 4)) return CB_ERR_ALIGNMENT;
  const Span l = rows_of(p->logits, p->n_tokens, p->n_experts, p->ld_logits, size);
  const Span b = {p->bias, static_cast<uint64_t>(p->n_experts) * 4};
  const Span ids = rows_of(p->ids, p->n_tokens, p->top_k, p->top_k, 4), w = rows_of(p->w, p->n_tokens, p->top_k, p->top_k, 4);
  if (overlaps_any(ids, {l, b, w}) || overlaps_any(w, {l, b})) return CB_ERR_INVALID_ARG;
  int sms;
  const cb_status_t st = ready(&sms);
  if (st != CB_OK) return st;
  RouteArgs a{};
  a.n_tokens = static_cast<int32_t>(p->n_tokens);
  a.n_experts = p->n_experts;
  a.top_k = p->top_k;
  a.logits = p->logits;
  a.ld = p->ld_logits;
  a.bias = p->bias;
  a.ids = p->ids;
  a.w = p->w;
  a.scale = p->scale;
  a.f32 = p->logits_type == CB_T_F32;
  a.softmax = p->score == CB_SCORE_SOFTMAX;
  a.n_groups = p->n_groups;
  a.top_groups = p->top_groups;
  a.group_max = p->group_score == CB_GROUP_MAX;
  a.renormalise = p->renormalise;
  return launch_route(a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

cb_status_t cb_int4_matmul_few(const cb_int4_matmul_t* p, void* stream) {
  if (p == nullptr || p->n_tokens < 0 || p->n <= 0 || p->k <= 0 || p->top_k <= 0 || p->n_experts <= 0 ||
      (p->group != 32 && p->group != 64 && p->group != 128) || !known_type(p->out_type))
    return CB_ERR_INVALID_ARG;
  const bool by_expert = p->ids != nullptr, swiglu = p->swiglu != 0;
  if (p->k % p->group != 0 || p->n % (swiglu ? 32 : 16) != 0) return CB_ERR_INVALID_ARG;
  if ((p->w != nullptr && (!by_expert || swiglu)) || (p->x_per_slot != 0 && !by_expert)) return CB_ERR_INVALID_ARG;
  if (!by_expert && (p->top_k != 1 || p->n_experts != 1)) return CB_ERR_INVALID_ARG;
  const int64_t cols = swiglu ? p->n / 2 : p->n;
  if (p->ld_x < p->k || p->ld_out < cols) return CB_ERR_INVALID_ARG;
  if (p->n_tokens > CB_INT4_MAX_ROWS || p->top_k > 16 || p->n_experts > 256 || p->n > (1 << 24) ||
      p->k > (by_expert ? CB_INT4_MAX_K : 8 * CB_INT4_MAX_K) ||
      p->ld_x > (1ll << 48) || p->ld_out > (1ll << 48))
    return CB_ERR_UNSUPPORTED;
  if (p->n_tokens == 0) return CB_OK;
  if (p->x == nullptr || p->codes == nullptr || p->scales == nullptr || p->out == nullptr) return CB_ERR_INVALID_ARG;
  const int x_size = p->x_scales != nullptr ? 1 : 2;
  const int64_t pairs = static_cast<int64_t>(p->n_tokens) * p->top_k, x_rows = p->x_per_slot ? pairs : p->n_tokens;
  if (!on(p->x, 16) || !on(p->codes, 16) || !on(p->scales, 16) || !on(p->zeros, 16) || !on(p->x_scales, 4) ||
      !on(p->ids, 4) || !on(p->w, 4) || !on(p->status, 4) || !on(p->out, size_of(p->out_type)) ||
      (p->ld_x % 8 != 0 && x_rows > 1))
    return CB_ERR_ALIGNMENT;
  const int64_t out_rows = p->w != nullptr ? p->n_tokens : pairs, blocks = (p->k + CB_FP8_COLS - 1) / CB_FP8_COLS;
  const uint64_t meta = static_cast<uint64_t>(p->n_experts) * (p->k / p->group) * p->n;
  const Span out = rows_of(p->out, out_rows, cols, p->ld_out, size_of(p->out_type));
  if (overlaps_any(out, {rows_of(p->x, x_rows, p->k, p->ld_x, x_size), rows_of(p->x_scales, x_rows, blocks, blocks, 4),
                         {p->codes, static_cast<uint64_t>(p->n_experts) * p->n * (p->k / 2)}, {p->scales, meta * 4},
                         {p->zeros, meta}, {p->ids, static_cast<uint64_t>(pairs) * 4},
                         {p->w, static_cast<uint64_t>(pairs) * 4}, {p->status, 4}}))
    return CB_ERR_INVALID_ARG;
  int sms;
  const cb_status_t st = ready(&sms);
  if (st != CB_OK) return st;
  Int4Args a{};
  a.pairs = static_cast<int32_t>(pairs);
  a.top = p->top_k;
  a.n_experts = p->n_experts;
  a.n = static_cast<int32_t>(p->n);
  a.k = static_cast<int32_t>(p->k);
  a.x = p->x;
  a.ld_x = p->ld_x;
  a.x_scales = p->x_scales;
  a.x_per_slot = p->x_per_slot != 0;
  a.codes = p->codes;
  a.scales = p->scales;
  a.zeros = p->zeros;
  a.ids = p->ids;
  a.w = p->w;
  a.swiglu = swiglu;
  a.out = p->out;
  a.ld_out = p->ld_out;
  a.out_f32 = p->out_type == CB_T_F32;
  a.status = p->status;
  return launch_int4_few(p->group, a, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? CB_OK : CB_ERR_CUDA;
}

}  // extern "C"
