// C entry points of the training-step operators: argument checks, then the
// launches.  Nothing is enqueued before every check has passed, and nothing
// leaves an entry point as an exception.
#include <hip/hip_runtime_api.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <string>

#include "muon.h"
#include "plan.hpp"
#include "train_ops.hpp"

using namespace muon;

namespace {

constexpr int64_t kMax = (int64_t)1 << 31;  // sizes are below this

muon_status fail(muon_status st, const char *where, const char *what) {
  set_error(std::string(where) + ": " + what);
  return st;
}

muon_status done(hipError_t e, const char *where) {
  if (e == hipSuccess) return MUON_OK;
  return fail(MUON_ERR_HIP, where, hipGetErrorString(e));
}

// Runs an entry point's body; an exception (host memory for a message) ends
// as a status.
template <class F>
muon_status guarded(F body) {
  try {
    return body();
  } catch (...) {
    return MUON_ERR_INVALID_ARG;
  }
}

bool known_dtype(int32_t t) { return t == MUON_DT_FP32 || t == MUON_DT_BF16; }
bool known_index(int32_t t) { return t == MUON_IDX_INT32 || t == MUON_IDX_INT64; }
uintptr_t dtype_bytes(int32_t t) { return t == MUON_DT_BF16 ? 2 : 4; }
uintptr_t index_bytes(int32_t t) { return t == MUON_IDX_INT64 ? 8 : 4; }

// The addresses a buffer spans.
struct Span {
  uintptr_t lo, hi;
  const char *name;
};
Span flat(const void *p, int64_t n, uintptr_t e, const char *name) {
  return {(uintptr_t)p, (uintptr_t)p + (p ? (uintptr_t)n * e : 0), name};
}
Span matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, uintptr_t e, const char *name) {
  return flat(p, rows > 0 ? (rows - 1) * ld + cols : 0, e, name);
}

// Whether a rows x ld extent stays an address (2^62 bytes leave room).
bool fits(int64_t rows, int64_t ld) { return ld < ((int64_t)1 << 59) && (rows == 0 || ld < ((int64_t)1 << 59) / rows); }

// Every written buffer against every other buffer of the call.
muon_status no_overlap(const char *where, std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span *a = out.begin(); a != out.end(); ++a) {
    auto clash = [&](const Span &b) { return a->lo < a->hi && b.lo < b.hi && a->lo < b.hi && b.lo < a->hi; };
    for (const Span *b = a + 1; b != out.end(); ++b)
      if (clash(*b)) {
        set_error(std::string(where) + ": buffers overlap: " + a->name + " and " + b->name);
        return MUON_ERR_ALIAS;
      }
    for (const Span &b : in)
      if (clash(b)) {
        set_error(std::string(where) + ": buffers overlap: " + a->name + " and " + b.name);
        return MUON_ERR_ALIAS;
      }
  }
  return MUON_OK;
}

muon_status check_workspace(const char *where, const void *ws, size_t have, size_t need) {
  if (!ws) return fail(MUON_ERR_WORKSPACE, where, "workspace is NULL");
  if ((uintptr_t)ws % 256 != 0) return fail(MUON_ERR_WORKSPACE, where, "workspace must be 256-byte aligned");
  if (have < need) {
    set_error(std::string(where) + ": workspace too small: " + std::to_string(have) + " < " + std::to_string(need));
    return MUON_ERR_WORKSPACE;
  }
  return MUON_OK;
}

muon_status check_embed_sizes(const char *where, int64_t tokens, int64_t vocab, int64_t dim) {
  if (tokens < 0 || vocab < 1 || dim < 1) return fail(MUON_ERR_INVALID_ARG, where, "needs tokens >= 0, vocab >= 1, dim >= 1");
  if (tokens >= kMax || vocab >= kMax || dim >= kMax) return fail(MUON_ERR_UNSUPPORTED, where, "tokens, vocab and dim must be below 2^31");
  return MUON_OK;
}

muon_status check_logits(const char *where, const muon_logits *x) {
  if (!x) return fail(MUON_ERR_INVALID_ARG, where, "NULL logits description");
  if (x->rows < 0 || x->vocab < 1) return fail(MUON_ERR_INVALID_ARG, where, "needs rows >= 0 and vocab >= 1");
  if (!known_dtype(x->dtype) || !known_index(x->target_type)) return fail(MUON_ERR_INVALID_ARG, where, "unknown dtype or target type");
  if (x->rows > 0 && (!x->logits || !x->targets)) return fail(MUON_ERR_INVALID_ARG, where, "NULL logits or targets");
  if (x->ld < x->vocab) return fail(MUON_ERR_INVALID_ARG, where, "ld is below the vocabulary");
  if (x->rows >= kMax || x->vocab >= kMax / 4 || !fits(x->rows, x->ld))
    return fail(MUON_ERR_UNSUPPORTED, where, "rows must be below 2^31 and vocab below 2^29");
  return MUON_OK;
}

LogitArgs logit_args(const muon_logits *x) {
  return {x->logits, {x->targets, x->target_type == MUON_IDX_INT64}, x->ld, x->vocab, x->rows, 0};
}

// dlogits: the logits themselves, or apart from them
Span dlogits_span(const muon_logits *x, const void *d, int64_t dld) {
  return matrix(d, x->rows, x->vocab, dld, dtype_bytes(x->dtype), "dlogits");
}
Span logits_span(const muon_logits *x, const void *d, int64_t dld) {
  if (d == x->logits && dld == x->ld) return {0, 0, "logits"};
  return matrix(x->logits, x->rows, x->vocab, x->ld, dtype_bytes(x->dtype), "logits");
}

}  // namespace

extern "C" {

muon_status muon_embed_forward(const void *table, int64_t vocab, int64_t dim, int64_t table_ld, int32_t dtype,
                               const void *ids, int32_t id_type, int64_t tokens, float scale, void *out,
                               int64_t out_ld, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_embed_forward";
    muon_status st = check_embed_sizes(me, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    if (!known_dtype(dtype) || !known_index(id_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype or id type");
    if (!table || (tokens > 0 && (!ids || !out))) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (table_ld < dim || out_ld < dim) return fail(MUON_ERR_INVALID_ARG, me, "ld is below dim");
    if (!std::isfinite(scale)) return fail(MUON_ERR_INVALID_ARG, me, "scale is not finite");
    if (!fits(vocab, table_ld) || !fits(tokens, out_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const uintptr_t e = dtype_bytes(dtype);
    st = no_overlap(me, {matrix(out, tokens, dim, out_ld, e, "out")},
                    {matrix(table, vocab, dim, table_ld, e, "table"), flat(ids, tokens, index_bytes(id_type), "ids")});
    if (st != MUON_OK) return st;
    const EmbedFwdArgs a{table, out, {ids, id_type == MUON_IDX_INT64}, table_ld, out_ld, vocab, dim, tokens, scale, 0};
    return done(launch_embed_forward(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_embed_backward_workspace_bytes(int64_t tokens, int64_t vocab, int64_t dim, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_embed_backward_workspace_bytes";
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    muon_status st = check_embed_sizes(me, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    *bytes = embed_layout(tokens, vocab, dim).total;
    return MUON_OK;
  });
}

muon_status muon_embed_backward(const void *ids, int32_t id_type, int64_t tokens, const void *dout, int32_t dtype,
                                int64_t dout_ld, float scale, float *acc, int64_t vocab, int64_t dim, int64_t acc_ld,
                                int32_t first, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_embed_backward";
    muon_status st = check_embed_sizes(me, tokens, vocab, dim);
    if (st != MUON_OK) return st;
    if (!known_dtype(dtype) || !known_index(id_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype or id type");
    if (!acc || (tokens > 0 && (!ids || !dout))) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (dout_ld < dim || acc_ld < dim) return fail(MUON_ERR_INVALID_ARG, me, "ld is below dim");
    if (!std::isfinite(scale)) return fail(MUON_ERR_INVALID_ARG, me, "scale is not finite");
    if (!fits(vocab, acc_ld) || !fits(tokens, dout_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const EbLayout l = embed_layout(tokens, vocab, dim);
    if ((st = check_workspace(me, ws, ws_bytes, l.total)) != MUON_OK) return st;
    st = no_overlap(me, {matrix(acc, vocab, dim, acc_ld, 4, "acc"), flat(ws, (int64_t)l.total, 1, "workspace")},
                    {matrix(dout, tokens, dim, dout_ld, dtype_bytes(dtype), "dout"),
                     flat(ids, tokens, index_bytes(id_type), "ids")});
    if (st != MUON_OK) return st;
    char *w = static_cast<char *>(ws);
    EmbedBwdArgs a{};
    a.ids = {ids, id_type == MUON_IDX_INT64};
    a.dout = dout;
    a.acc = acc;
    a.dout_ld = dout_ld;
    a.acc_ld = acc_ld;
    a.vocab = vocab;
    a.dim = dim;
    a.tokens = tokens;
    a.scale = scale;
    a.first = first != 0;
    a.buckets = reinterpret_cast<EbBucket *>(w + l.buckets);
    a.perm = reinterpret_cast<int32_t *>(w + l.perm);
    a.key_a = reinterpret_cast<int32_t *>(w + l.key_a);
    a.key_b = reinterpret_cast<int32_t *>(w + l.key_b);
    a.tok_b = reinterpret_cast<int32_t *>(w + l.tok_b);
    a.chunks = reinterpret_cast<EbChunk *>(w + l.chunks);
    a.partials = reinterpret_cast<float *>(w + l.partials);
    a.arrive = reinterpret_cast<int32_t *>(w + l.arrive);
    return done(launch_embed_backward(a, dtype == MUON_DT_BF16, static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_token_logprob(const muon_logits *x, float *logp, float *lse, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_token_logprob";
    muon_status st = check_logits(me, x);
    if (st != MUON_OK) return st;
    if (x->rows > 0 && !logp) return fail(MUON_ERR_INVALID_ARG, me, "NULL logp");
    st = no_overlap(me, {flat(logp, x->rows, 4, "logp"), flat(lse, x->rows, 4, "lse")},
                    {logits_span(x, nullptr, 0), flat(x->targets, x->rows, index_bytes(x->target_type), "targets")});
    if (st != MUON_OK) return st;
    return done(launch_token_logprob(logit_args(x), x->dtype == MUON_DT_BF16, logp, lse,
                                     static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_policy_loss_workspace_bytes(int64_t rows, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_policy_loss_workspace_bytes";
    if (!bytes || rows < 0) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument or negative size");
    if (rows >= kMax) return fail(MUON_ERR_UNSUPPORTED, me, "rows must be below 2^31");
    *bytes = policy_layout(rows).total;
    return MUON_OK;
  });
}

muon_status muon_policy_loss(const muon_logits *x, const float *advantages, const float *weights,
                             const float *old_logp, const float *ref_logp, const muon_policy_options *opt,
                             float *stats, float *logp, void *dlogits, int64_t dlogits_ld, void *ws, size_t ws_bytes,
                             void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_policy_loss";
    muon_status st = check_logits(me, x);
    if (st != MUON_OK) return st;
    if (!opt || !stats || (x->rows > 0 && (!advantages || !weights || !logp || !dlogits)))
      return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (!std::isfinite(opt->clip_low) || !std::isfinite(opt->clip_high) || opt->clip_low < 0.0 || opt->clip_high < 0.0 ||
        !std::isfinite(opt->kl_coef))
      return fail(MUON_ERR_INVALID_ARG, me, "clip_low and clip_high must be finite and >= 0, kl_coef finite");
    if (dlogits_ld < x->vocab) return fail(MUON_ERR_INVALID_ARG, me, "ld of dlogits is below the vocabulary");
    if (!fits(x->rows, dlogits_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld of dlogits is too large");
    const size_t need = policy_layout(x->rows).total;
    if ((st = check_workspace(me, ws, ws_bytes, need)) != MUON_OK) return st;
    const int64_t n = x->rows;
    st = no_overlap(me, {dlogits_span(x, dlogits, dlogits_ld), flat(stats, 4, 4, "stats"), flat(logp, n, 4, "logp"),
                         flat(ws, (int64_t)need, 1, "workspace")},
                    {logits_span(x, dlogits, dlogits_ld), flat(x->targets, n, index_bytes(x->target_type), "targets"),
                     flat(advantages, n, 4, "advantages"), flat(weights, n, 4, "weights"),
                     flat(old_logp, n, 4, "old_logp"), flat(ref_logp, n, 4, "ref_logp")});
    if (st != MUON_OK) return st;
    const PolicyArgs p{advantages, weights, old_logp, ref_logp, opt->clip_low, opt->clip_high, opt->kl_coef, stats, logp};
    return done(launch_policy(logit_args(x), p, x->dtype == MUON_DT_BF16, dlogits, dlogits_ld, static_cast<char *>(ws),
                              static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_preference_loss_workspace_bytes(int64_t rows, int64_t pairs, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_preference_loss_workspace_bytes";
    if (!bytes || rows < 0 || pairs < 1) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument or bad size");
    if (rows >= kMax || pairs >= kMax / 2) return fail(MUON_ERR_UNSUPPORTED, me, "rows and 2 pairs must be below 2^31");
    *bytes = preference_layout(rows, pairs).total;
    return MUON_OK;
  });
}

muon_status muon_preference_loss(const muon_logits *x, const void *offsets, int32_t offset_type, int64_t pairs,
                                 const float *ref_logp, const muon_preference_options *opt, float *loss,
                                 float *rewards, void *dlogits, int64_t dlogits_ld, void *ws, size_t ws_bytes,
                                 void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_preference_loss";
    muon_status st = check_logits(me, x);
    if (st != MUON_OK) return st;
    if (!known_index(offset_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown offset type");
    if (pairs < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs pairs >= 1");
    if (pairs >= kMax / 2) return fail(MUON_ERR_UNSUPPORTED, me, "2 pairs must be below 2^31");
    if (!opt || !offsets || !ref_logp || !loss || !rewards || (x->rows > 0 && !dlogits))
      return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (!std::isfinite(opt->beta) || !(opt->label_smoothing >= 0.0 && opt->label_smoothing <= 1.0))
      return fail(MUON_ERR_INVALID_ARG, me, "beta must be finite, label_smoothing in [0, 1]");
    if (dlogits_ld < x->vocab) return fail(MUON_ERR_INVALID_ARG, me, "ld of dlogits is below the vocabulary");
    if (!fits(x->rows, dlogits_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld of dlogits is too large");
    const size_t need = preference_layout(x->rows, pairs).total;
    if ((st = check_workspace(me, ws, ws_bytes, need)) != MUON_OK) return st;
    st = no_overlap(me, {dlogits_span(x, dlogits, dlogits_ld), flat(loss, 1, 4, "loss"),
                         flat(rewards, 2 * pairs, 4, "rewards"), flat(ws, (int64_t)need, 1, "workspace")},
                    {logits_span(x, dlogits, dlogits_ld),
                     flat(x->targets, x->rows, index_bytes(x->target_type), "targets"),
                     flat(offsets, 2 * pairs + 1, index_bytes(offset_type), "offsets"),
                     flat(ref_logp, 2 * pairs, 4, "ref_logp")});
    if (st != MUON_OK) return st;
    const PreferenceArgs p{{offsets, offset_type == MUON_IDX_INT64}, pairs, ref_logp, opt->beta, opt->label_smoothing,
                           loss, rewards};
    return done(launch_preference(logit_args(x), p, x->dtype == MUON_DT_BF16, dlogits, dlogits_ld,
                                  static_cast<char *>(ws), static_cast<hipStream_t>(stream)), me);
  });
}

muon_status muon_balance_loss_workspace_bytes(int64_t tokens, int64_t experts, size_t *bytes) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_balance_loss_workspace_bytes";
    if (!bytes || tokens < 0 || experts < 1) return fail(MUON_ERR_INVALID_ARG, me, "NULL argument or bad size");
    if (experts > MUON_BALANCE_MAX_EXPERTS || tokens >= kMax) return fail(MUON_ERR_UNSUPPORTED, me, "at most 1024 experts and 2^31 - 1 tokens");
    *bytes = balance_layout(tokens, (int32_t)experts).total;
    return MUON_OK;
  });
}

muon_status muon_balance_loss(const void *logits, int64_t tokens, int64_t experts, int64_t ld, int32_t dtype,
                              const void *choices, int32_t choice_type, int64_t k, const uint8_t *valid,
                              const muon_balance_options *opt, int32_t *counts, float *stats, void *dlogits,
                              int64_t dlogits_ld, void *ws, size_t ws_bytes, void *stream) {
  return guarded([&]() -> muon_status {
    const char *const me = "muon_balance_loss";
    static_assert(MUON_BALANCE_MAX_EXPERTS == BAL_MAX_EXPERTS, "the header's limit");
    if (tokens < 0 || experts < 1 || k < 1) return fail(MUON_ERR_INVALID_ARG, me, "needs tokens >= 0, experts >= 1, k >= 1");
    if (experts > BAL_MAX_EXPERTS) return fail(MUON_ERR_UNSUPPORTED, me, "at most 1024 experts");
    if (tokens >= kMax || k >= kMax || tokens * k >= kMax) return fail(MUON_ERR_UNSUPPORTED, me, "tokens * k must be below 2^31");
    if (!known_dtype(dtype) || !known_index(choice_type)) return fail(MUON_ERR_INVALID_ARG, me, "unknown dtype or choice type");
    if (!opt || !counts || !stats || (tokens > 0 && (!logits || !choices || !dlogits)))
      return fail(MUON_ERR_INVALID_ARG, me, "NULL argument");
    if (!std::isfinite(opt->coef) || !std::isfinite(opt->z_coef)) return fail(MUON_ERR_INVALID_ARG, me, "coef and z_coef must be finite");
    if (ld < experts || dlogits_ld < experts) return fail(MUON_ERR_INVALID_ARG, me, "ld is below the experts");
    if (!fits(tokens, ld) || !fits(tokens, dlogits_ld)) return fail(MUON_ERR_UNSUPPORTED, me, "ld is too large");
    const size_t need = balance_layout(tokens, (int32_t)experts).total;
    muon_status st = check_workspace(me, ws, ws_bytes, need);
    if (st != MUON_OK) return st;
    const uintptr_t e = dtype_bytes(dtype);
    const bool in_place = dlogits == logits && dlogits_ld == ld;
    st = no_overlap(me, {matrix(dlogits, tokens, experts, dlogits_ld, e, "dlogits"), flat(counts, experts, 4, "counts"),
                         flat(stats, 3, 4, "stats"), flat(ws, (int64_t)need, 1, "workspace")},
                    {matrix(in_place ? nullptr : logits, tokens, experts, ld, e, "logits"),
                     flat(choices, tokens * k, index_bytes(choice_type), "choices"), flat(valid, tokens, 1, "valid")});
    if (st != MUON_OK) return st;
    const BalanceArgs a{logits, {choices, choice_type == MUON_IDX_INT64}, valid, ld, dlogits_ld, tokens,
                        (int32_t)experts, (int32_t)k, opt->coef, opt->z_coef, counts, stats, dlogits};
    return done(launch_balance(a, dtype == MUON_DT_BF16, static_cast<char *>(ws), static_cast<hipStream_t>(stream)), me);
  });
}

}  // extern "C"
