// C entry points of the operators of a trained layer: argument checks, then
// the launches.  Nothing is enqueued before every check has passed, and
// nothing leaves an entry point as an exception.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>

#include "abi_checks.hpp"
#include "layer_ops.hpp"
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
  // 64 lanes a token at the most
  if (tokens > kThreads / 64 && experts > 256) return fail(MUON_ERR_UNSUPPORTED, me, "too many tokens of more than 256 experts");
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

}  // extern "C"
