// la_tree.cu -- acceptance of drafted trees, and the dispatch of the tree kernels by io type.
#include "la_device.cuh"
#include "la_serving.h"

namespace la {

TreeLaunchFn find_tree_f32io(bool kda, int dk, int dv, int st);
TreeLaunchFn find_tree_bf16io(bool kda, int dk, int dv, int st);
TreeCommitLaunchFn find_tree_commit_f32io(bool kda, int dk, int dv, int st);
TreeCommitLaunchFn find_tree_commit_bf16io(bool kda, int dk, int dv, int st);

TreeLaunchFn find_tree(int rule, int dk, int dv, int st, int io) {
  const bool kda = rule == LA_RULE_KDA;
  return io == LA_F32 ? find_tree_f32io(kda, dk, dv, st) : find_tree_bf16io(kda, dk, dv, st);
}
TreeCommitLaunchFn find_tree_commit(int rule, int dk, int dv, int st, int io) {
  const bool kda = rule == LA_RULE_KDA;
  return io == LA_F32 ? find_tree_commit_f32io(kda, dk, dv, st) : find_tree_commit_bf16io(kda, dk, dv, st);
}

namespace {

// One warp per sequence, two nodes per lane: from the root, the lowest child of the current
// node whose drafted token is the one wanted there; a child lies behind its parent, so the
// walk ends after at most max_nodes steps.  Bound by latency (a few dependent ballots).
__global__ void __launch_bounds__(32) accept_kernel(const TreeAcceptParams p) {
  griddep_wait();
  const int b = blockIdx.x, lane = threadIdx.x;
  const int c0 = ld_coherent(p.cu + b), c1 = ld_coherent(p.cu + b + 1);
  if (c0 < 0 || c1 < c0 || c1 > p.total) {
    if (lane == 0) report(p.err, LA_DEVERR_CU_SEQLENS);
    return;
  }
  const int n = c1 - c0;
  if (n > p.max_nodes) {
    if (lane == 0) report(p.err, LA_DEVERR_TREE);
    return;
  }
  int par[2], tok[2], tgt[2];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int t = lane + 32 * e;
    par[e] = -2;
    tok[e] = tgt[e] = 0;
    if (t < n) {
      par[e] = ld_coherent(p.parent + c0 + t);
      tok[e] = ld_coherent(p.draft + c0 + t);
      tgt[e] = ld_coherent(p.target + c0 + t);
      bad |= par[e] < -1 || par[e] >= t;
    }
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (lane == 0) report(p.err, LA_DEVERR_TREE);
    return;
  }
  int cur = -1, want = ld_coherent(p.root + b), count = 0;
  for (int step = 0; step < n; ++step) {
    const uint32_t lo = __ballot_sync(0xffffffffu, par[0] == cur && tok[0] == want);
    const uint32_t hi = __ballot_sync(0xffffffffu, par[1] == cur && tok[1] == want);
    if (lo == 0u && hi == 0u) break;
    cur = lo ? __ffs(lo) - 1 : 31 + __ffs(hi);
    const int a = __shfl_sync(0xffffffffu, tgt[0], cur & 31), c = __shfl_sync(0xffffffffu, tgt[1], cur & 31);
    want = cur < 32 ? a : c;
    ++count;
  }
  if (lane == 0) {
    p.leaf[b] = cur;
    p.count[b] = count;
    p.next[b] = want;
  }
}

}  // namespace

cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t stream) {
  return launch_dependent(accept_kernel, p.n_seqs, 32, 0, stream, p);
}

}  // namespace la
