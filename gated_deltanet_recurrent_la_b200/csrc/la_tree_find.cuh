// la_tree_find.cuh -- the compiled (pool dtype, d_k, d_v, gate) combinations of the tree
// kernels for one io type.
#pragma once

#include "la_tree.cuh"
#include "la_tree_tc.cuh"

namespace la {
namespace tree {

template <typename IT, bool KDA>
TreeLaunchFn find_tree_io(int dk, int dv, int st) {
#define LA_TREE_CASE(ST_CODE, ST, DK, DV) \
  if (st == ST_CODE && dk == DK && dv == DV) return &launch_tree<ST, IT, DK, DV, KDA>;
#define LA_TREE_TC(ST_CODE, ST, DK, DV) \
  if (st == ST_CODE && dk == DK && dv == DV) return &launch_tree_tc<ST, IT, DK, DV, KDA>;
#define LA_TREE_SHAPES(ST_CODE, ST)      \
  LA_TREE_TC(ST_CODE, ST, 64, 64)        \
  LA_TREE_TC(ST_CODE, ST, 128, 64)       \
  LA_TREE_TC(ST_CODE, ST, 128, 128)
  LA_TREE_CASE(LA_F32, float, 16, 16)
  LA_TREE_CASE(LA_BF16, __nv_bfloat16, 16, 16)
  LA_TREE_SHAPES(LA_F32, float)
  LA_TREE_SHAPES(LA_BF16, __nv_bfloat16)
  LA_TREE_SHAPES(LA_Q8, q8_t)
  return nullptr;
#undef LA_TREE_SHAPES
#undef LA_TREE_TC
#undef LA_TREE_CASE
}

template <typename IT, bool KDA>
TreeCommitLaunchFn find_commit_io(int dk, int dv, int st) {
#define LA_TREE_CASE(ST_CODE, ST, DK, DV) \
  if (st == ST_CODE && dk == DK && dv == DV) return &launch_commit<ST, IT, DK, DV, KDA>;
#define LA_TREE_SHAPES(ST_CODE, ST)        \
  LA_TREE_CASE(ST_CODE, ST, 64, 64)        \
  LA_TREE_CASE(ST_CODE, ST, 128, 64)       \
  LA_TREE_CASE(ST_CODE, ST, 128, 128)
  LA_TREE_CASE(LA_F32, float, 16, 16)
  LA_TREE_CASE(LA_BF16, __nv_bfloat16, 16, 16)
  LA_TREE_SHAPES(LA_F32, float)
  LA_TREE_SHAPES(LA_BF16, __nv_bfloat16)
  LA_TREE_SHAPES(LA_Q8, q8_t)
  return nullptr;
#undef LA_TREE_SHAPES
#undef LA_TREE_CASE
}

}  // namespace tree
}  // namespace la
