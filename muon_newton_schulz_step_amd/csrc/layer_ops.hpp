// The operators of a trained layer around the Muon step (dropout, routing to
// experts, the order of the tokens by expert, the experts' weighted sum):
// argument blocks and launchers shared by their C entry points
// (layer_abi.cpp) and kernels (k_dropout.hip, k_route.hip, k_order.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "train_ops.hpp"

namespace muon {

// -------------------------------------------------------------- dropout

struct DropoutArgs {
  const void *x, *residual;  // residual may be NULL
  void *out;
  int64_t rows, cols, ld, rld, old;
  uint32_t threshold;  // an element is kept if its random word is at least this
  float scale;
  uint32_t key0, key1, site, step;
  const int64_t *device_step;  // its low half replaces step, if not NULL
};
hipError_t launch_dropout(const DropoutArgs &a, bool bf16, hipStream_t s);

// -------------------------------------------------------------- routing

constexpr int ROUTE_MAX_EXPERTS = 1024;
constexpr int ROUTE_MAX_CHOICES = 32;
constexpr int ROUTE_MAX_GROUPS = 32;

struct RouteArgs {
  const void *logits;
  const float *bias;     // may be NULL
  const uint8_t *valid;  // may be NULL
  int64_t ld, tokens;
  int32_t experts, k;
  int32_t softmax, renormalize;
  int32_t groups, keep, top;
  float scale;
  IndexVec choices;  // written by the forward pass
  float *weights;
  const float *dweights;
  void *dlogits;
  int64_t dld;
  int32_t first;
};
hipError_t launch_route(const RouteArgs &a, bool bf16, hipStream_t s);
hipError_t launch_route_backward(const RouteArgs &a, bool bf16, hipStream_t s);

// --------------------------------------------- order of the tokens by expert

struct OrderArgs {
  IndexVec choices;
  int64_t n;  // tokens * k
  int32_t k, experts;
  int32_t *tokens, *offsets, *place;
};
struct OrderLayout {
  size_t hist, totals, total;
};
OrderLayout order_layout(int64_t n, int32_t experts);
hipError_t launch_order(const OrderArgs &a, char *ws, hipStream_t s);

// ------------------------------------------------ the experts' weighted sum

struct CombineArgs {
  const void *y, *residual;  // residual may be NULL
  void *out;
  const int32_t *place;
  const float *weights;  // may be NULL: 1
  int64_t rows, tokens, dim, k;
  int64_t yld, rld, old;
};
hipError_t launch_combine(const CombineArgs &a, bool bf16, hipStream_t s);

struct CombineBwdArgs {
  const void *dout, *y;  // y may be NULL without dweights
  void *dy;              // may be NULL
  const int32_t *place;
  const float *weights;  // may be NULL: 1
  float *dweights;       // may be NULL
  int64_t rows, tokens, dim, k;
  int64_t dold, yld, dyld;
};
hipError_t launch_combine_backward(const CombineBwdArgs &a, bool bf16, hipStream_t s);

}  // namespace muon
