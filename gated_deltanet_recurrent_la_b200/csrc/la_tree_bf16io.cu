// Tree verification and commit with BF16 q, k, v, o.
#include "la_tree_find.cuh"

namespace la {
TreeLaunchFn find_tree_bf16io(bool kda, int dk, int dv, int st) {
  return kda ? tree::find_tree_io<__nv_bfloat16, true>(dk, dv, st)
             : tree::find_tree_io<__nv_bfloat16, false>(dk, dv, st);
}
TreeCommitLaunchFn find_tree_commit_bf16io(bool kda, int dk, int dv, int st) {
  return kda ? tree::find_commit_io<__nv_bfloat16, true>(dk, dv, st)
             : tree::find_commit_io<__nv_bfloat16, false>(dk, dv, st);
}
}  // namespace la
