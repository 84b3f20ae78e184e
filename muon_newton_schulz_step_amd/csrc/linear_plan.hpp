// How a product is cut into tiles and parts, and the workspace that its parts
// need: host arithmetic alone, shared by the launches and the entry points
// that tell the workspace's size, so that neither can change without the other.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace muon {

// Tiles of 128 x 128 if they fill the chip, of 64 x 64 otherwise, and then K in
// parts: enough for four workgroups a CU, of 8 stages of 64 (bf16) or 4 (fp32,
// whose stages take twice as long) and more, as far as their sums take no more
// than 64 MB.  64 x 4096 x 4096 bf16: 15.0 us in parts of 8 stages, 17.8 of 4;
// 64 x 1024 x 1024 fp32: 13.1 in parts of 4, 19.1 of 8.  Where one tile a CU
// fills the chip, parts begin to pay at 24 stages (1021 x 1000 bf16, whole and
// in parts: K = 512 6.8 and 14.5 us, 1024 13.4 and 16.9, 2048 23.6 and 21.3).
// A product's rows count as one group's, though each group begins a tile of its
// own: 64 rows of 32 experts of 4096 x 4096 bf16 take 206 us in 8 parts (182 for
// the weights' bytes).
struct LinearPlan {
  int w;
  int32_t splits;
};
inline LinearPlan linear_plan(int64_t M, int64_t N, int64_t K, int32_t groups, bool weight, bool bf16) {
  const int64_t per = weight ? groups : 1;
  if ((M + 127) / 128 * ((N + 127) / 128) * per >= 256) return {4, 1};
  const int64_t tiles = (M + 63) / 64 * ((N + 63) / 64) * per;
  const int64_t stages = (K / (weight ? groups : 1) + 63) / 64;
  if (tiles >= 256 && stages < 24) return {2, 1};
  const int64_t bytes = std::max<int64_t>(1, M * per * N * 4);
  const int64_t parts = std::min<int64_t>({1024 / std::max<int64_t>(1, tiles), stages / (bf16 ? 8 : 4), ((int64_t)64 << 20) / bytes, 32});
  return {2, (int32_t)std::max<int64_t>(1, parts)};
}

// Products of up to FEW_ROWS rows take kl_few, whose workgroups take FEW_ACROSS
// columns where K is across and FEW_ADJACENT where it is adjacent, in parts of
// a multiple of FEW_PART.
constexpr int FEW_ROWS = 8, FEW_ACROSS = 64, FEW_ADJACENT = 8, FEW_PART = 512;

// Whether a product's rows are few enough for kl_few.  4096 x 11008, kl_few
// against 64 x 64 tiles: fp32 of 8 rows 38 and 53 us (K adjacent, across)
// against 70; bf16 of 4 rows 19 and 21 against 24, of 8 rows 26 and 29 against
// 24.  Where K is adjacent smaller weights still gain with 8 (4096 x 4096: 11
// against 17), and rows of groups are mostly of different ones.
inline bool few_rows(int64_t M, bool bf16, bool bx, bool grouped) { return M <= (bf16 && bx && !grouped ? 4 : FEW_ROWS); }

struct FewPlan {
  int32_t tiles_m, tiles_n, splits;
};
inline FewPlan few_plan(int64_t M, int64_t N, int64_t K, int32_t groups, bool bf16, bool bx) {
  const int64_t columns = bx ? FEW_ACROSS : FEW_ADJACENT;
  // groups that have rows: no more than the rows
  FewPlan p{(int32_t)std::min<int64_t>(M, groups), (int32_t)((N + columns - 1) / columns), 1};
  const int64_t tiles = (int64_t)p.tiles_m * p.tiles_n;
  // K across, in parts while there are CUs for them and K is long enough to pay
  // for the second launch, 3 us (2048 x 512 bf16: 5.7 us whole, 6.7 in 4 parts;
  // 2048 x 512 fp32: 8.7 in 2 parts, 7.9 in 4; 1024 x 4096 fp32: 7.5, 8.7 in 2)
  const int64_t bytes = K * (bf16 ? 2 : 4);
  if (bx && bytes >= 8192) p.splits = (int32_t)std::max<int64_t>(1, std::min<int64_t>({256 / tiles, bytes / 2048, 32}));
  return p;
}

// Workspace of a call's parts, of either type and layout of the weights:
// whichever kernel takes it.
inline size_t linear_partial_bytes(int64_t M, int64_t N, int64_t K, int32_t groups, bool weight) {
  int32_t parts = 1;
  for (bool bf16 : {false, true}) {
    parts = std::max(parts, linear_plan(M, N, K, groups, weight, bf16).splits);
    if (!weight && M > 0 && few_rows(M, bf16, true, true))
      parts = std::max(parts, few_plan(M, N, K, groups, bf16, true).splits);
  }
  return parts > 1 ? (size_t)parts * (size_t)(M * (weight ? groups : 1)) * (size_t)N * 4 : 0;
}

}  // namespace muon
