// C entry points of the operators of a trained layer: argument checks, then
// the launches.  Nothing is enqueued before every check has passed, and
// nothing leaves an entry point as an exception.
#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "abi_checks.hpp"
#include "layer_ops.hpp"
#include "linear.hpp"
#include "linear_plan.hpp"
#include "muon.h"

using namespace muon;
using namespace muon::abi;

namespace {

// Threads that one grid takes, less a workgroup.
constexpr int64_t kThreads = ((int64_t)1 << 32) - 1024;

// A buffer that may be the output itself (same address and ld).
Span apart(const void *p, int64_t rows, int64_t cols, int64_t ld, uintptr_t e, const char *name, const void *out,
           int64_t out_ld) {
  if (p == out && (ld == out_ld || rows <= 1)) return {0, 0, name};
  return matrix(p, rows, cols, ld, e, name);
}

muon_status check_route(const char *me, const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype,
                        const muon_route_options *opt, const void *choices, int32_t choice_type, int64_t k) {
  static_assert(MUON_BALANCE_MAX_EXPERTS == ROUTE_MAX_EXPERTS && MUON_ROUTE_MAX_CHOICES == ROUTE_MAX_CHOICES &&
                    MUON_ROUTE_MAX_GROUPS == ROUTE_MAX_GROUPS,
                "the header's limits");
  if (tokens < 0 || experts < 1 || k < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs tokens >= 0, experts >= 1, k >= 1");
  if (!opt) return fail(MUON_ERR_INVALID_ARG, me, "NULL options");
  if (!known_dtype(dtype) || !known_index(choice_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype or choice type");
  if (opt->scoring != MUON_SCORE_SOFTMAX && opt->scoring != MUON_SCORE_SIGMOID)
    return fail(MUON_ERR_INVALID_ARG, me, "unknown scoring");
  if (!std::isfinite(opt->scale)) return fail(MUON_ERR_INVALID_ARG, me, "scale must be finite");
  if (tokens > 0 && (!logits || !choices)) return fail(MUON_ERR_INVALID_ARG, me, "NULL logits or choices");
  if (ld < experts) return fail(MUON_ERR_INVALID_ARG, me, "ld is below the experts");
  if (experts > ROUTE_MAX_EXPERTS || k > ROUTE_MAX_CHOICES)
    return fail(MUON_ERR_UNSUPPORTED, me, "at most 1024 experts and 32 choices");
  if (tokens >= kMax || tokens * k >= kMax || !fits(tokens, ld)) return fail(MUON_ERR_UNSUPPORTED, me, "tokens * k must be below 2^31");
  if (tokens >= (int64_t)1 << 26 && experts > 256)
    return fail(MUON_ERR_UNSUPPORTED, me, "tokens of more than 256 experts must be below 2^26");
  return MUON_OK;
}

// Whether the experts cut into groups; the gradient has no use of them.
muon_status check_groups(const char *me, int64_t experts, int64_t k, const muon_route_options *o) {
  if (k > experts) return fail(MUON_ERR_INVALID_ARG, me, "more choices than experts");
  if (o->groups < 1 || experts % o->groups != 0) return fail(MUON_ERR_INVALID_ARG, me, "the experts do not divide into the groups");
  if (o->keep_groups < 1 || o->keep_groups > o->groups) return fail(MUON_ERR_INVALID_ARG, me, "keep_groups must be in [1, groups]");
  if (o->group_top != 1 && o->group_top != 2) return fail(MUON_ERR_INVALID_ARG, me, "group_top must be 1 or 2");
  if (o->groups > ROUTE_MAX_GROUPS) return fail(MUON_ERR_UNSUPPORTED, me, "at most 32 groups");
  return MUON_OK;
}

muon_status check_rows(const char *me, int64_t tokens, int64_t k, int64_t rows, int64_t dim, int32_t dtype) {
  if (tokens < 0 || k < 1 || rows < 0 || dim < 1)
    return fail(MUON_ERR_INVALID_ARG, me, "needs tokens >= 0, k >= 1, rows >= 0, dim >= 1");
  if (!known_dtype(dtype)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype");
  if (tokens >= kMax || k >= kMax || tokens * k >= kMax || rows >= kMax || dim >= kMax)
    return fail(MUON_ERR_UNSUPPORTED, me, "tokens * k, rows and dim must be below 2^31");
  // a wave a token, or a thread a 16-byte vector
  if (tokens > kThreads / 64 || tokens > kThreads / ((dim + 3) / 4)) return fail(MUON_ERR_UNSUPPORTED, me, "too many elements");
  return MUON_OK;
}

constexpr int64_t kMaxGroups = 1024;
constexpr int64_t kMaxTiles = (int64_t)1 << 23;  // of 128 x 128 elements: a launch has fewer, and every grid its threads

muon_status check_linear(const char *me, int64_t rows, int64_t in, int64_t out, int64_t groups) {
  static_assert(MUON_LINEAR_MAX_GROUPS == kMaxGroups, "the header's limit");
  if (rows < 0 || in < 1 || out < 1 || groups < 1)
    return fail(MUON_ERR_INVALID_ARG, me, "needs rows >= 0, in >= 1, out >= 1, groups >= 1");
  if (rows >= kMax || in >= kMax || out >= kMax || groups > kMaxGroups)
    return fail(MUON_ERR_UNSUPPORTED, me, "rows, in and out must be below 2^31, groups at most 1024");
  const int64_t r = rows / 128 + groups, i = in / 128 + 1, o = out / 128 + 1;
  if (r * i >= kMaxTiles || r * o >= kMaxTiles || i * o * groups >= kMaxTiles)
    return fail(MUON_ERR_UNSUPPORTED, me, "2^23 tiles of 128 x 128 elements or more");
  return MUON_OK;
}

muon_status check_activation(const char *me, int32_t act) {
  if (act < MUON_ACT_NONE || act > MUON_ACT_GELU_TANH) return fail(MUON_ERR_INVALID_ARG, me, "unknown activation");
  return MUON_OK;
}

muon_status check_offsets(const char *me, const void *offsets, int32_t type, int64_t groups) {
  if (!known_index(type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown offset type");
  if (!offsets && groups != 1) return fail(MUON_ERR_INVALID_ARG, me, "NULL offsets of more than one group");
  return MUON_OK;
}

// The length of a row of a matrix of `in` x `out`, and the rows.
int64_t row_length(int32_t layout, int64_t in, int64_t out) { return layout == MUON_W_IN_OUT ? out : in; }

muon_status check_matrices(const char *me, int32_t layout, int64_t in, int64_t out, int64_t ld, int64_t stride, int64_t groups) {
  if (layout != MUON_W_IN_OUT && layout != MUON_W_OUT_IN) return fail(MUON_ERR_INVALID_ARG, me, "unknown layout of the weights");
  const int64_t cols = row_length(layout, in, out), rows = layout == MUON_W_IN_OUT ? in : out;
  if (ld < cols) return fail(MUON_ERR_INVALID_ARG, me, "ld of the weights is below their row length");
  if (!fits(rows, ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld of the weights is too large");
  if (groups > 1 && stride < (rows - 1) * ld + cols) return fail(MUON_ERR_INVALID_ARG, me, "the groups' weights overlap");
  if (groups > 1 && !fits(groups, stride)) return fail(MUON_ERR_UNSUPPORTED, me, "the stride of the weights is too large");
  return MUON_OK;
}

Span matrices(const void *p, int32_t layout, int64_t in, int64_t out, int64_t ld, int64_t stride, int64_t groups,
              uintptr_t e, const char *name) {
  const int64_t cols = row_length(layout, in, out), rows = layout == MUON_W_IN_OUT ? in : out;
  return flat(p, (groups - 1) * stride + (rows - 1) * ld + cols, e, name);
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of the weights' gradient.
struct WeightGradLayout {
  size_t partial, columns, total;
};
WeightGradLayout weight_grad_layout(int64_t rows, int64_t in, int64_t out, int64_t groups) {
  WeightGradLayout l{};
  // either layout of dw
  l.partial = rounded(sizeof(LinearQueue));
  l.columns = l.partial + rounded(std::max(linear_partial_bytes(in, out, rows, (int32_t)groups, true),
                               linear_partial_bytes(out, in, rows, (int32_t)groups, true)));
  l.total = l.columns + rounded((size_t)groups * (size_t)column_sum_splits(rows, out, (int32_t)groups) * (size_t)out * 4);
  return l;
}

muon_status check_weights(const char *me, const muon_weights *w, int64_t rows) {
  if (!w) return fail(MUON_ERR_INVALID_ARG, me, "NULL weights");
  muon_status st = check_linear(me, rows, w->in, w->out, w->groups);
  if (st != MUON_OK) return st;
  if (!known_dtype(w->dtype)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype");
  if (!w->w) return fail(MUON_ERR_INVALID_ARG, me, "NULL weights");
  if ((st = check_offsets(me, w->offsets, w->offset_type, w->groups)) != MUON_OK) return st;
  return check_matrices(me, w->layout, w->in, w->out, w->ld, w->stride, w->groups);
}

Span weight_span(const muon_weights *w) {
  return matrices(w->w, w->layout, w->in, w->out, w->ld, w->stride, w->groups, dtype_bytes(w->dtype), "weights");
}
Span offset_span(const void *offsets, int32_t type, int64_t groups) {
  return flat(offsets, groups + 1, index_bytes(type), "offsets");
}

}  // namespace

extern "C" {

muon_status muon_dropout(const void *x, int64_t rows, int64_t cols, int64_t ld, int32_t dtype, double p, uint64_t seed,
                         uint32_t site, uint32_t step, const int64_t *device_step, const void *residual,
                         int64_t residual_ld, void *out, int64_t out_ld, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_dropout";
    if (rows < 0 || cols < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs rows >= 0 and cols >= 1");
    if (!known_dtype(dtype)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype");
    const double threshold = std::nearbyint(p * 4294967296.0);
    if (!(p >= 0.0) || !(threshold < 4294967296.0)) return fail(MUON_ERR_INVALID_ARG, me, "p must be in [0, 1)");
    if (rows > 0 && (!x || !out)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (ld < cols || out_ld < cols || (residual && residual_ld < cols))
      return fail(MUON_ERR_INVALID_ARG, me, "ld is below the row length");
    if (rows >= kMax || cols >= kMax || rows > 4 * kThreads / ((cols + 3) / 4) || !fits(rows, ld) || !fits(rows, out_ld) ||
        (residual && !fits(rows, residual_ld)))
      return fail(MUON_ERR_UNSUPPORTED, me, "rows and cols must be below 2^31, and their vectors fit a grid");
    const uintptr_t e = dtype_bytes(dtype);
    const muon_status st =
        no_overlap(me, {matrix(out, rows, cols, out_ld, e, "out")},
                   {apart(x, rows, cols, ld, e, "x", out, out_ld), apart(residual, rows, cols, residual_ld, e, "residual", out, out_ld),
                    flat(device_step, 1, 8, "device_step")});
    if (st != MUON_OK) return st;
    const DropoutArgs a{x, residual, out, rows, cols, ld, residual_ld, out_ld, (uint32_t)threshold,
                        (float)(1.0 / (1.0 - p)), (uint32_t)seed, (uint32_t)(seed >> 32), site, step, device_step};
    return done(launch_dropout(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_route(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype, const float *bias,
                       const uint8_t *valid, const muon_route_options *opt, void *choices, int32_t choice_type,
                       int64_t k, float *weights, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_route";
    muon_status st = check_route(me, logits, tokens, experts, ld, dtype, opt, choices, choice_type, k);
    if (st != MUON_OK) return st;
    if ((st = check_groups(me, experts, k, opt)) != MUON_OK) return st;
    if (tokens > 0 && !weights) return fail(MUON_ERR_INVALID_ARG, me, "NULL weights");
    st = no_overlap(me, {flat(choices, tokens * k, index_bytes(choice_type), "choices"), flat(weights, tokens * k, 4, "weights")},
                    {matrix(logits, tokens, experts, ld, dtype_bytes(dtype), "logits"), flat(bias, experts, 4, "bias"),
                     flat(valid, tokens, 1, "valid")});
    if (st != MUON_OK) return st;
    RouteArgs a{};
    a.logits = logits;
    a.bias = bias;
    a.valid = valid;
    a.ld = ld;
    a.tokens = tokens;
    a.experts = (int32_t)experts;
    a.k = (int32_t)k;
    a.softmax = opt->scoring == MUON_SCORE_SOFTMAX;
    a.renormalize = opt->renormalize != 0;
    a.groups = opt->groups;
    a.keep = opt->keep_groups;
    a.top = opt->group_top;
    if (a.keep == a.groups) a.groups = a.keep = 1;  // every group stays
    a.scale = (float)opt->scale;
    a.choices = {choices, choice_type == MUON_IDX_INT64};
    a.weights = weights;
    return done(launch_route(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_route_backward(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype,
                                const uint8_t *valid, const muon_route_options *opt, const void *choices,
                                int32_t choice_type, int64_t k, const float *dweights, void *dlogits,
                                int64_t dlogits_ld, int32_t first, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_route_backward";
    muon_status st = check_route(me, logits, tokens, experts, ld, dtype, opt, choices, choice_type, k);
    if (st != MUON_OK) return st;
    if (tokens > 0 && (!dweights || !dlogits)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (dlogits_ld < experts) return fail(MUON_ERR_INVALID_ARG, me, "ld is below the experts");
    if (!fits(tokens, dlogits_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrix(dlogits, tokens, experts, dlogits_ld, e, "dlogits")},
                    {matrix(logits, tokens, experts, ld, e, "logits"), flat(valid, tokens, 1, "valid"),
                     flat(choices, tokens * k, index_bytes(choice_type), "choices"), flat(dweights, tokens * k, 4, "dweights")});
    if (st != MUON_OK) return st;
    RouteArgs a{};
    a.logits = logits;
    a.valid = valid;
    a.ld = ld;
    a.tokens = tokens;
    a.experts = (int32_t)experts;
    a.k = (int32_t)k;
    a.softmax = opt->scoring == MUON_SCORE_SOFTMAX;
    a.renormalize = opt->renormalize != 0;
    a.scale = (float)opt->scale;
    a.choices = {choices, choice_type == MUON_IDX_INT64};
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.dld = dlogits_ld;
    a.first = first != 0;
    return done(launch_route_backward(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_expert_order_workspace_bytes(int64_t tokens, int64_t k, int64_t experts, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_expert_order_workspace_bytes";
    if (!bytes || tokens < 0 || k < 1 || experts < 1) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument or bad size");
    if (experts > ROUTE_MAX_EXPERTS || tokens >= kMax || k >= kMax || tokens * k >= kMax)
      return fail(MUON_ERR_UNSUPPORTED, me, "at most 1024 experts, tokens * k below 2^31");
    *bytes = order_layout(tokens * k, (int32_t)experts).total;
    return MUON_OK;
  });
}

muon_status muon_expert_order(const void *choices, int32_t choice_type, int64_t tokens, int64_t k, int64_t experts,
                              int32_t *slot_tokens, int32_t *offsets, int32_t *place, void *ws, size_t ws_bytes,
                              void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_expert_order";
    if (tokens < 0 || k < 1 || experts < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs tokens >= 0, k >= 1, experts >= 1");
    if (!known_index(choice_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown choice type");
    if (!offsets || (tokens > 0 && (!choices || !slot_tokens || !place))) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (experts > ROUTE_MAX_EXPERTS || tokens >= kMax || k >= kMax || tokens * k >= kMax)
      return fail(MUON_ERR_UNSUPPORTED, me, "at most 1024 experts, tokens * k below 2^31");
    const int64_t n = tokens * k;
    const size_t need = order_layout(n, (int32_t)experts).total;
    muon_status st = check_workspace(me, ws, ws_bytes, need);
    if (st != MUON_OK) return st;
    st = no_overlap(me, {flat(slot_tokens, n, 4, "slot_tokens"), flat(offsets, experts + 1, 4, "offsets"),
                         flat(place, n, 4, "place"), flat(ws, (int64_t)need, 1, "workspace")},
                    {flat(choices, n, index_bytes(choice_type), "choices")});
    if (st != MUON_OK) return st;
    const OrderArgs a{{choices, choice_type == MUON_IDX_INT64}, n, (int32_t)k, (int32_t)experts, slot_tokens, offsets, place};
    return done(launch_order(a, static_cast<char *>(ws), static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_expert_combine(const void *y, int64_t rows, int64_t dim, int64_t y_ld, int32_t dtype,
                                const int32_t *place, int64_t tokens, int64_t k, const float *weights,
                                const void *residual, int64_t residual_ld, void *out, int64_t out_ld, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_expert_combine";
    muon_status st = check_rows(me, tokens, k, rows, dim, dtype);
    if (st != MUON_OK) return st;
    if ((rows > 0 && !y) || (tokens > 0 && (!place || !out))) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (y_ld < dim || out_ld < dim || (residual && residual_ld < dim)) return fail(MUON_ERR_INVALID_ARG, me, "ld is below dim");
    if (!fits(rows, y_ld) || !fits(tokens, out_ld) || (residual && !fits(tokens, residual_ld)))
      return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrix(out, tokens, dim, out_ld, e, "out")},
                    {matrix(y, rows, dim, y_ld, e, "y"), flat(place, tokens * k, 4, "place"),
                     flat(weights, tokens * k, 4, "weights"), apart(residual, tokens, dim, residual_ld, e, "residual", out, out_ld)});
    if (st != MUON_OK) return st;
    const CombineArgs a{y, residual, out, place, weights, rows, tokens, dim, k, y_ld, residual_ld, out_ld};
    return done(launch_combine(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_expert_combine_backward(const void *dout, int64_t tokens, int64_t dim, int64_t dout_ld, int32_t dtype,
                                         const int32_t *place, int64_t k, const float *weights, const void *y,
                                         int64_t y_ld, int64_t rows, void *dy, int64_t dy_ld, float *dweights,
                                         void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_expert_combine_backward";
    muon_status st = check_rows(me, tokens, k, rows, dim, dtype);
    if (st != MUON_OK) return st;
    if (tokens > 0 && rows > 0 && !dy && !dweights) return fail(MUON_ERR_INVALID_ARG, me, "neither dy nor dweights is asked for");
    if (tokens > 0 && (!dout || !place)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (dweights && rows > 0 && !y) return fail(MUON_ERR_INVALID_ARG, me, "dweights needs y");
    if (dout_ld < dim || (dweights && y_ld < dim) || (dy && dy_ld < dim)) return fail(MUON_ERR_INVALID_ARG, me, "ld is below dim");
    if (!fits(tokens, dout_ld) || (dweights && !fits(rows, y_ld)) || (dy && !fits(rows, dy_ld)))
      return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    if (!dweights) y = nullptr;
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrix(dy, rows, dim, dy_ld, e, "dy"), flat(dweights, tokens * k, 4, "dweights")},
                    {matrix(dout, tokens, dim, dout_ld, e, "dout"), flat(place, tokens * k, 4, "place"),
                     flat(weights, tokens * k, 4, "weights"), apart(y, rows, dim, y_ld, e, "y", dy, dy_ld)});
    if (st != MUON_OK) return st;
    const CombineBwdArgs a{dout, y, dy, place, weights, dweights, rows, tokens, dim, k, dout_ld, y_ld, dy_ld};
    return done(launch_combine_backward(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_linear_workspace_bytes(int64_t rows, int64_t in, int64_t out, int64_t groups, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_linear_workspace_bytes";
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    const muon_status st = check_linear(me, rows, in, out, groups);
    if (st != MUON_OK) return st;
    *bytes = 256 + rounded(linear_partial_bytes(rows, out, in, (int32_t)groups, false));
    return MUON_OK;
  });
}

muon_status muon_linear_forward(const void *x, int64_t rows, int64_t x_ld, const muon_weights *w, const void *bias,
                                int32_t activation, void *pre, int64_t pre_ld, const void *residual,
                                int64_t residual_ld, void *out, int64_t out_ld, void *ws, size_t ws_bytes,
                                void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_linear_forward";
    muon_status st = check_weights(me, w, rows);
    if (st != MUON_OK) return st;
    if ((st = check_activation(me, activation)) != MUON_OK) return st;
    if (rows > 0 && (!x || !out)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    const int64_t in = w->in, n = w->out;
    if (x_ld < in || out_ld < n || (pre && pre_ld < n) || (residual && residual_ld < n))
      return fail(MUON_ERR_INVALID_ARG, me, "ld is below the row length");
    if (!fits(rows, x_ld) || !fits(rows, out_ld) || (pre && !fits(rows, pre_ld)) || (residual && !fits(rows, residual_ld)))
      return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const size_t need = 256 + rounded(linear_partial_bytes(rows, n, in, w->groups, false));
    if ((st = check_workspace(me, ws, ws_bytes, need)) != MUON_OK) return st;
    const uintptr_t e = dtype_bytes(w->dtype);
    st = no_overlap(me, {matrix(out, rows, n, out_ld, e, "out"), matrix(pre, rows, n, pre_ld, e, "pre"),
                         flat(ws, (int64_t)need, 1, "workspace")},
                    {matrix(x, rows, in, x_ld, e, "x"), weight_span(w), flat(bias, w->groups * n, e, "bias"),
                     apart(residual, rows, n, residual_ld, e, "residual", out, out_ld),
                     offset_span(w->offsets, w->offset_type, w->groups)});
    if (st != MUON_OK) return st;
    if (rows == 0) return MUON_OK;
    LinearArgs a{};
    a.a = x;
    a.b = w->w;
    a.lda = x_ld;
    a.ldb = w->ld;
    a.bstride = w->stride;
    a.M = rows;
    a.N = n;
    a.K = in;
    a.offsets = {w->offsets, w->offset_type == MUON_IDX_INT64};
    a.groups = w->groups;
    a.mode = LIN_FORWARD;
    a.bias = bias;
    a.pre = pre;
    a.residual = residual;
    a.out = out;
    a.pre_ld = pre_ld;
    a.res_ld = residual_ld;
    a.out_ld = out_ld;
    a.act = activation;
    a.partial = static_cast<float *>(ws);
    return done(launch_linear(a, w->dtype == MUON_DT_BF16, LIN_K_ADJACENT,
                              w->layout == MUON_W_IN_OUT ? LIN_K_ACROSS : LIN_K_ADJACENT, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_linear_input_grad(const void *dy, int64_t rows, int64_t dy_ld, const muon_weights *w,
                                   int32_t activation, const void *pre, int64_t pre_ld, const void *residual,
                                   int64_t residual_ld, void *dx, int64_t dx_ld, void *ws, size_t ws_bytes,
                                   void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_linear_input_grad";
    muon_status st = check_weights(me, w, rows);
    if (st != MUON_OK) return st;
    if ((st = check_activation(me, activation)) != MUON_OK) return st;
    if (rows > 0 && (!dy || !dx)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (activation == MUON_ACT_NONE) pre = nullptr;
    else if (rows > 0 && !pre) return fail(MUON_ERR_INVALID_ARG, me, "an activation needs pre");
    const int64_t n = w->in, k = w->out;
    if (dy_ld < k || dx_ld < n || (pre && pre_ld < n) || (residual && residual_ld < n))
      return fail(MUON_ERR_INVALID_ARG, me, "ld is below the row length");
    if (!fits(rows, dy_ld) || !fits(rows, dx_ld) || (pre && !fits(rows, pre_ld)) || (residual && !fits(rows, residual_ld)))
      return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const size_t need = 256 + rounded(linear_partial_bytes(rows, n, k, w->groups, false));
    if ((st = check_workspace(me, ws, ws_bytes, need)) != MUON_OK) return st;
    const uintptr_t e = dtype_bytes(w->dtype);
    st = no_overlap(me, {matrix(dx, rows, n, dx_ld, e, "dx"), flat(ws, (int64_t)need, 1, "workspace")},
                    {matrix(dy, rows, k, dy_ld, e, "dy"), weight_span(w), matrix(pre, rows, n, pre_ld, e, "pre"),
                     apart(residual, rows, n, residual_ld, e, "residual", dx, dx_ld),
                     offset_span(w->offsets, w->offset_type, w->groups)});
    if (st != MUON_OK) return st;
    if (rows == 0) return MUON_OK;
    LinearArgs a{};
    a.a = dy;
    a.b = w->w;
    a.lda = dy_ld;
    a.ldb = w->ld;
    a.bstride = w->stride;
    a.M = rows;
    a.N = n;
    a.K = k;
    a.offsets = {w->offsets, w->offset_type == MUON_IDX_INT64};
    a.groups = w->groups;
    a.mode = LIN_INPUT;
    a.pre = const_cast<void *>(pre);
    a.residual = residual;
    a.out = dx;
    a.pre_ld = pre_ld;
    a.res_ld = residual_ld;
    a.out_ld = dx_ld;
    a.act = activation;
    a.partial = static_cast<float *>(ws);
    return done(launch_linear(a, w->dtype == MUON_DT_BF16, LIN_K_ADJACENT,
                              w->layout == MUON_W_IN_OUT ? LIN_K_ADJACENT : LIN_K_ACROSS, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_linear_weight_grad_workspace_bytes(int64_t rows, int64_t in, int64_t out, int64_t groups, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_linear_weight_grad_workspace_bytes";
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    const muon_status st = check_linear(me, rows, in, out, groups);
    if (st != MUON_OK) return st;
    *bytes = weight_grad_layout(rows, in, out, groups).total;
    return MUON_OK;
  });
}

muon_status muon_linear_weight_grad(const void *x, int64_t rows, int64_t in, int64_t x_ld, const void *dy, int64_t out,
                                    int64_t dy_ld, int32_t dtype, const void *offsets, int32_t offset_type,
                                    int64_t groups, float *dw, int64_t dw_ld, int64_t dw_stride, int32_t dw_layout,
                                    float *dbias, int32_t first, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_linear_weight_grad";
    muon_status st = check_linear(me, rows, in, out, groups);
    if (st != MUON_OK) return st;
    if (!known_dtype(dtype)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype");
    if ((st = check_offsets(me, offsets, offset_type, groups)) != MUON_OK) return st;
    if ((rows > 0 && (!x || !dy)) || !dw) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (x_ld < in || dy_ld < out) return fail(MUON_ERR_INVALID_ARG, me, "ld is below the row length");
    if (!fits(rows, x_ld) || !fits(rows, dy_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    if ((st = check_matrices(me, dw_layout, in, out, dw_ld, dw_stride, groups)) != MUON_OK) return st;
    const WeightGradLayout l = weight_grad_layout(rows, in, out, groups);
    if ((st = check_workspace(me, ws, ws_bytes, l.total)) != MUON_OK) return st;
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrices(dw, dw_layout, in, out, dw_ld, dw_stride, groups, 4, "dw"), flat(dbias, groups * out, 4, "dbias"),
                         flat(ws, (int64_t)l.total, 1, "workspace")},
                    {matrix(x, rows, in, x_ld, e, "x"), matrix(dy, rows, out, dy_ld, e, "dy"),
                     offset_span(offsets, offset_type, groups)});
    if (st != MUON_OK) return st;
    const bool plain = dw_layout == MUON_W_IN_OUT;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    LinearArgs a{};
    a.a = plain ? x : dy;
    a.b = plain ? dy : x;
    a.lda = plain ? x_ld : dy_ld;
    a.ldb = plain ? dy_ld : x_ld;
    a.M = plain ? in : out;
    a.N = plain ? out : in;
    a.K = rows;
    a.offsets = {offsets, offset_type == MUON_IDX_INT64};
    a.groups = (int32_t)groups;
    a.mode = LIN_WEIGHT;
    a.out = dw;
    a.out_ld = dw_ld;
    a.out_stride = dw_stride;
    a.first = first != 0;
    a.queue = static_cast<int32_t *>(ws);
    a.partial = reinterpret_cast<float *>(static_cast<char *>(ws) + l.partial);
    hipError_t err = launch_linear(a, dtype == MUON_DT_BF16, LIN_K_ACROSS, LIN_K_ACROSS, s);
    if (err == hipSuccess && dbias) {
      const ColumnSumArgs c{dy, rows, out, dy_ld, a.offsets, (int32_t)groups, a.first, dbias,
                            reinterpret_cast<float *>(static_cast<char *>(ws) + l.columns),
                            column_sum_splits(rows, out, (int32_t)groups)};
      err = launch_column_sums(c, dtype == MUON_DT_BF16, s);
    }
    return done(err, me);
  });
}

muon_status muon_activation_grad(const void *dy, int64_t rows, int64_t cols, int64_t dy_ld, int32_t dtype,
                                 int32_t activation, const void *pre, int64_t pre_ld, void *dpre, int64_t dpre_ld,
                                 void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_activation_grad";
    if (rows < 0 || cols < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs rows >= 0 and cols >= 1");
    if (!known_dtype(dtype)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype");
    muon_status st = check_activation(me, activation);
    if (st != MUON_OK) return st;
    if (rows > 0 && (!dy || !pre || !dpre)) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (dy_ld < cols || pre_ld < cols || dpre_ld < cols) return fail(MUON_ERR_INVALID_ARG, me, "ld is below the row length");
    if (rows >= kMax || cols >= kMax || rows > kThreads / ((cols + 7) / 8) || !fits(rows, dy_ld) || !fits(rows, pre_ld) || !fits(rows, dpre_ld))
      return fail(MUON_ERR_UNSUPPORTED, me, "rows and cols must be below 2^31, and their vectors fit a grid");
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrix(dpre, rows, cols, dpre_ld, e, "dpre")},
                    {apart(dy, rows, cols, dy_ld, e, "dy", dpre, dpre_ld), apart(pre, rows, cols, pre_ld, e, "pre", dpre, dpre_ld)});
    if (st != MUON_OK) return st;
    const ActivationGradArgs a{dy, pre, dpre, rows, cols, dy_ld, pre_ld, dpre_ld, activation};
    return done(launch_activation_grad(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

}  // extern "C"
