// The product with a weight matrix, or with one a group of rows, and its
// gradients: argument blocks and launchers shared by the C entry points
// (layer_abi.cpp) and kernels (k_linear.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

#include "train_ops.hpp"

namespace muon {

// What becomes of a product's elements.
enum LinearMode : int32_t {
  LIN_FORWARD = 0,  // out = act(v + bias) + residual, pre = v + bias
  LIN_INPUT = 1,    // out = v act'(pre) + residual
  LIN_WEIGHT = 2,   // out = v (+ out), fp32
};

// C = A B of M x K and K x N elements, for every group of rows of A (and C)
// with a matrix B of its own; in LIN_WEIGHT for every group of the contracted
// rows, with a matrix C of its own.
struct LinearArgs {
  const void *a, *b;
  int64_t lda, ldb, bstride;  // bstride: from a group's B to the next one's
  int64_t M, N, K;
  IndexVec offsets;           // p NULL: one group of everything
  int32_t groups, mode;
  // what the product leaves
  const void *bias;           // groups x N, may be NULL
  void *pre;                  // written forwards (may be NULL), read for the gradient
  const void *residual;       // may be NULL
  void *out;
  int64_t pre_ld, res_ld, out_ld, out_stride;
  int32_t act, first;
  // the launch
  int32_t splits;             // parts of K, whose sums meet in `partial`
  int32_t tiles_m, tiles_n;   // output tiles (over all groups, at most)
  float *partial;             // splits x (rows of all groups' C) x N
  int32_t *queue;             // LIN_WEIGHT of groups: LinearQueue
};

// The order in which a grouped weight gradient's tiles are taken: groups from
// the longest to the shortest, and what each XCD's workgroups have taken, a
// line of 128 bytes an XCD.
struct LinearQueue {
  int32_t taken[8][32];
  int32_t group[1024];
};

// How operands lie: K adjacent (rows of A, columns of B), or the other way.
enum LinearOperand : int32_t { LIN_K_ADJACENT = 0, LIN_K_ACROSS = 1 };

hipError_t launch_linear_few(LinearArgs &a, bool bf16, bool bx, hipStream_t s);

hipError_t launch_linear(LinearArgs a, bool bf16, int la, int lb, hipStream_t s);

// dbias[g] (+)= the sums of dy's columns over the group's rows
struct ColumnSumArgs {
  const void *dy;
  int64_t rows, cols, ld;
  IndexVec offsets;
  int32_t groups, first;
  float *out;      // groups x cols
  float *partial;  // groups x splits x cols
  int32_t splits;
};
int32_t column_sum_splits(int64_t rows, int64_t cols, int32_t groups);
hipError_t launch_column_sums(const ColumnSumArgs &a, bool bf16, hipStream_t s);

struct ActivationGradArgs {
  const void *dy, *pre;
  void *out;
  int64_t rows, cols, dld, pld, old;
  int32_t act;
};
hipError_t launch_activation_grad(const ActivationGradArgs &a, bool bf16, hipStream_t s);

}  // namespace muon
