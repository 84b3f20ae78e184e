// The training-step operators around the Muon step: argument blocks and
// launchers shared by their C entry points (train_abi.cpp) and kernels
// (k_embed.hip, k_logits.hip, k_balance.hip).
#pragma once

#include <hip/hip_runtime_api.h>

#include <cstddef>
#include <cstdint>

namespace muon {

// A vector of whole numbers on the device, int32 or int64 (token ids,
// targets, sequence offsets, expert choices).
struct IndexVec {
  const void *p;
  int32_t is64;
};

// ------------------------------------------------------------ embedding

struct EmbedFwdArgs {
  const void *table;
  void *out;
  IndexVec ids;
  int64_t table_ld, out_ld;
  int64_t vocab, dim, tokens;
  float scale;
  int64_t token0;  // the first token of a launch
};
hipError_t launch_embed_forward(const EmbedFwdArgs &a, bool bf16, hipStream_t s);

constexpr int EB_BUCKETS = 256;  // bucket of a table row = row mod EB_BUCKETS
constexpr int EB_CHUNK = 32;     // tokens of a row that one wave adds up, at most
constexpr int EB_GROUP = 32;     // chunks whose sums are joined at a time
constexpr int EB_LIGHT = 2;      // a row of more tokens is added up before one of these
constexpr int EB_FEW = 1024;     // up to so many tokens need no sort

// What the sort leaves about one bucket.
struct EbBucket {
  int32_t first;   // its tokens' first position in the sorted order
  int32_t tokens;  // their count, and its chunk slots: [first, first + tokens)
  int32_t heavy;   // chunks of rows with more than EB_LIGHT tokens, from the first slot on
  int32_t light;   // the other chunks, from the last slot down
};

// At most EB_CHUNK consecutive sorted tokens of one table row.  A row with
// more tokens has several chunks, whose sums meet in the workspace: EB_GROUP
// chunks at a time, then the groups.
struct EbChunk {
  int32_t row, start;
  int32_t count;  // tokens of this chunk
  int32_t parts;  // chunks of the row (1: the chunk writes the row itself)
  int32_t index;  // this chunk's place among them
  int32_t slot0;  // the first chunk's slot in the partial sums, the others' follow
  int32_t tok0;   // the row's first token
  int32_t pad;
};

// Workspace of the gradient, carved in this order (256-byte aligned parts).
struct EbLayout {
  size_t buckets, perm, key_a, key_b, tok_b, chunks, partials, arrive, total;
};
EbLayout embed_layout(int64_t tokens, int64_t vocab, int64_t dim);

struct EmbedBwdArgs {
  IndexVec ids;
  const void *dout;
  float *acc;
  int64_t dout_ld, acc_ld;
  int64_t vocab, dim, tokens;
  float scale;
  int32_t first;
  // workspace parts
  EbBucket *buckets;
  int32_t *perm, *key_a, *key_b, *tok_b;
  EbChunk *chunks;
  float *partials;
  int32_t *arrive;
};
hipError_t launch_embed_backward(const EmbedBwdArgs &a, bool bf16, hipStream_t s);

// --------------------------------------------------- losses over logits

// A row's softmax statistics: its maximum, the sum of exp(x - max), the
// target's log-probability and expm1 of that.
struct RowStat {
  float max, total;
  double logp, share;
};

// What the gradient of a row's logits needs: d x_j = c exp(x_j - max) away from
// the target, dt at the target; all of it 0 where live is 0.
struct RowGrad {
  float max, c, dt;
  int32_t live;
};

struct LogitArgs {
  const void *logits;
  IndexVec targets;
  int64_t ld, vocab, rows;
  int64_t row0;  // the first row of a launch
};

struct PolicyArgs {
  const float *advantages, *weights;
  const float *old_logp, *ref_logp;  // may be NULL
  double clip_low, clip_high, kl_coef;
  float *stats, *logp;
};

struct PreferenceArgs {
  IndexVec offsets;
  int64_t pairs;
  const float *ref_logp;
  double beta, smoothing;
  float *loss, *rewards;
};

// lse may be NULL
hipError_t launch_token_logprob(const LogitArgs &a, bool bf16, float *logp, float *lse, hipStream_t s);

struct PolicyLayout {
  size_t done, part, terms, total;
};
PolicyLayout policy_layout(int64_t rows);
hipError_t launch_policy(const LogitArgs &a, const PolicyArgs &p, bool bf16, void *dlogits, int64_t dld, char *ws,
                         hipStream_t s);

constexpr int PREF_THREADS = 512;  // threads of a workgroup of the preference loss
constexpr int PREF_SLACK = 64;     // rows between a pair's last sum and its first gradient

// The state of a walk over the rows of the pairs.
struct PreferenceWalk {
  uint64_t ticket;
  int32_t pairs_done;
  int32_t rows;  // rows that belong to a sequence
  int32_t lag;   // rows whose sums are handed out before the first gradient
  alignas(128) int32_t late;  // a gradient gave up waiting (a line of its own: the first one takes the tickets)
};
// Workspace of the preference loss.
struct PreferenceWork {
  int32_t max_polls;     // of a gradient's wait
  PreferenceWalk *walk;
  RowStat *stat;         // a row
  double *losses, *coef; // a pair
  int32_t *bounds;       // 2 pairs + 1: the sequences' first rows
  int32_t *starts;       // pairs + 1: a pair's place in the walk
  int32_t *done, *ready; // a pair: rows summed, coefficient written
};
struct PreferenceLayout {
  size_t walk, stat, grad, losses, coef, bounds, starts, done, ready, total;
};
PreferenceLayout preference_layout(int64_t rows, int64_t pairs);
hipError_t launch_preference(const LogitArgs &a, const PreferenceArgs &p, bool bf16, void *dlogits, int64_t dld,
                             char *ws, hipStream_t s);

// ---------------------------------------------------------- balance loss

constexpr int BAL_MAX_EXPERTS = 1024;

struct BalanceArgs {
  const void *logits;
  IndexVec experts;
  const uint8_t *valid;  // may be NULL
  int64_t ld, dld, tokens;
  int32_t n_experts, k;
  double coef, z_coef;
  int32_t *counts;
  float *stats;
  void *dlogits;
};
struct BalanceLayout {
  size_t hist, sums, arrive, total;
};
BalanceLayout balance_layout(int64_t tokens, int32_t n_experts);
hipError_t launch_balance(const BalanceArgs &a, bool bf16, char *ws, hipStream_t s);

}  // namespace muon
