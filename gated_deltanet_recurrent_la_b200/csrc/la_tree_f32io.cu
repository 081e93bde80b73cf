// Tree verification and commit with FP32 q, k, v, o.
#include "la_tree_find.cuh"

namespace la {
TreeLaunchFn find_tree_f32io(bool kda, int dk, int dv, int st) {
  return kda ? tree::find_tree_io<float, true>(dk, dv, st) : tree::find_tree_io<float, false>(dk, dv, st);
}
TreeCommitLaunchFn find_tree_commit_f32io(bool kda, int dk, int dv, int st) {
  return kda ? tree::find_commit_io<float, true>(dk, dv, st) : tree::find_commit_io<float, false>(dk, dv, st);
}
}  // namespace la
