// la_serving.h -- host-side interfaces of the serving operators around the slot pool: tree
// verification and commit, beam selection, slot bookkeeping over the slabs of all layers.
// Not installed; not part of the ABI.
#pragma once

#include "la_internal.h"

namespace la {

struct TreeParams {
  const void* src;            // source pool data
  int32_t src_slots;
  int32_t src_n_hp;           // q8 pools: BF16 key channels per head and the channel masks
  const uint32_t* src_mask;
  const int32_t* read_slot;   // [n_seqs] or nullptr (slot b)
  int32_t n_seqs;
  const int32_t* cu;          // [n_seqs + 1]
  int32_t total;
  const int32_t* parent;      // [total]
  int32_t max_nodes;
  int32_t n_qk_heads;
  int32_t n_v_heads;
  int32_t use_beta;           // b = beta (else 1)
  int32_t predicts;           // the delta correction
  const void* q;
  const void* k;
  const void* v;
  const float* g;             // nullptr: no gate
  const float* beta;
  float scale;
  void* o;
  float* u;                   // [total, n_v_heads, d_v] or nullptr
  int32_t* err;
  // failure-path test hooks: the time limit of a wait for products (ns), and a tile (sequence *
  // n_v_heads + head) whose products with the state are not issued (-1: none)
  uint64_t wait_ns;
  int64_t withhold;
};

struct TreeCommitParams {
  const void* src;
  int32_t src_slots;
  const int32_t* read_slot;
  void* dst;
  int32_t dst_slots;
  const int32_t* write_slot;
  int32_t n_hp;               // q8 pools
  const uint32_t* src_mask;
  const uint32_t* dst_mask;
  int32_t n_seqs;
  const int32_t* cu;
  int32_t total;
  const int32_t* parent;
  const int32_t* leaf;        // [n_seqs]
  int32_t max_nodes;
  int32_t n_qk_heads;
  int32_t n_v_heads;
  const void* k;
  const float* g;
  const float* u;
  int32_t* err;
};

struct TreeAcceptParams {
  int32_t n_seqs;
  const int32_t* cu;
  int32_t total;
  const int32_t* parent;
  int32_t max_nodes;
  const int32_t* draft;
  const int32_t* target;
  const int32_t* root;
  int32_t* leaf;
  int32_t* count;
  int32_t* next;
  int32_t* err;
};

using TreeLaunchFn = cudaError_t (*)(const TreeParams&, cudaStream_t);
using TreeCommitLaunchFn = cudaError_t (*)(const TreeCommitParams&, cudaStream_t);
// st: la_dtype of the pool, io: la_dtype of q, k, v, o; nullptr when not compiled
TreeLaunchFn find_tree(int rule, int dk, int dv, int st, int io);
TreeCommitLaunchFn find_tree_commit(int rule, int dk, int dv, int st, int io);
cudaError_t launch_tree_accept(const TreeAcceptParams& p, cudaStream_t stream);

struct BeamParams {
  int32_t n_seqs, n_beams, vocab, n_out;
  const void* logits;
  int32_t io;
  int64_t row_stride;         // elements between the rows of two beams
  const float* cum;
  const int32_t* finished;    // or nullptr
  int32_t eos;
  int32_t* parent;
  int32_t* token;
  float* score;
  int32_t* finished_out;      // or nullptr
  void* workspace;
};
size_t beam_workspace_bytes(int64_t n_seqs, int64_t n_beams, int64_t vocab, int64_t n_out);
cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t stream);

constexpr int kMaxSlabs = LA_MAX_SLABS;
struct SlabList {
  int32_t n;
  void* data[kMaxSlabs];
  int64_t bytes[kMaxSlabs];   // of one slot, a multiple of 16
  int32_t first[kMaxSlabs + 1];  // pieces of a slot before slab l (the launcher's)
  // failure-path test hooks: the time limit of a wait for a piece (ns), and the piece of the first
  // warp whose load is not issued (-1: none)
  uint64_t wait_ns;
  int64_t withhold;
};
cudaError_t launch_pool_reorder(const SlabList& slabs, int32_t n_slots, int32_t n_seqs, int32_t n_beams,
                                const int32_t* slots, const int32_t* parent, int32_t* new_slots, int32_t* err,
                                cudaStream_t stream);
cudaError_t launch_pool_alloc(int32_t* ref, int32_t n_slots, int32_t n, int32_t* slots, int32_t* err,
                              cudaStream_t stream);
cudaError_t launch_pool_ref(int32_t* ref, int32_t n_slots, int32_t n, const int32_t* slots, int32_t delta, int32_t* err,
                            cudaStream_t stream);
cudaError_t launch_pool_fork(const SlabList& slabs, int32_t* ref, int32_t n_slots, int32_t n, const int32_t* src_slots,
                             int32_t* new_slots, int32_t* err, cudaStream_t stream);
cudaError_t launch_pool_compact(const SlabList& slabs, int32_t n_slots, const int32_t* ref, int32_t* new_ref,
                                int32_t* remap, int32_t* moves, int32_t* counts, int32_t* err, cudaStream_t stream);
cudaError_t launch_pool_remap(int64_t n, const int32_t* table, int32_t n_slots, const int32_t* remap,
                              int32_t* new_table, int32_t* err, cudaStream_t stream);

// Launch that may start before the stream's previous kernel has drained: the kernel itself waits
// for it (griddep_wait) before it touches memory, so only the launch's own latency overlaps.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*fn)(P...), int grid, int threads, int smem, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fn, P(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace la
