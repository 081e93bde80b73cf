// la_slots.cu -- slot bookkeeping on the device, over the slabs of all layers at once: beam
// reordering, allocation by reference counts, forking, freeing, compaction.
//
// Each call is a small kernel that decides which slots move (whole numbers only, the same
// answer whatever the order of the threads) and one copy kernel for the slabs of all layers.
// Sources and destinations of the copies of one call never meet, so they run in any order.
#include <algorithm>

#include "la_device.cuh"
#include "la_serving.h"

namespace la {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;
constexpr int64_t kCopyVecs = (int64_t)kCopyThreads * kCopyUnroll;  // 16 KiB

struct Pairs {
  int32_t n;                 // upper bound
  const int32_t* n_dev;      // nullptr, or the number on the device
  const int32_t* src;        // slot of pair i: src[i], or src[group base + via[i]]
  const int32_t* via;
  int32_t group;
  const int32_t* dst;        // dst[i], or dst[src[i]] with dst_by_src
  int32_t dst_by_src;
  int32_t n_slots;
  int32_t chunks_per_slot;
};

__global__ void __launch_bounds__(kCopyThreads) slab_copy_kernel(const SlabList slabs, const Pairs q) {
  const int n = q.n_dev ? min(q.n, __ldg(q.n_dev)) : q.n;
  const int64_t work = (int64_t)n * q.chunks_per_slot;
  for (int64_t w = blockIdx.x; w < work; w += gridDim.x) {
    const int i = (int)(w / q.chunks_per_slot);
    int chunk = (int)(w % q.chunks_per_slot);
    int s;
    if (q.via) {
      const int v = __ldg(q.via + i);
      if (v < 0 || v >= q.group) continue;  // reported by the planning kernel
      s = __ldg(q.src + i / q.group * q.group + v);
    } else {
      s = __ldg(q.src + i);
    }
    if (s < 0 || s >= q.n_slots) continue;
    const int d = __ldg(q.dst + (q.dst_by_src ? s : i));
    if (d < 0 || d >= q.n_slots || d == s) continue;
    int l = 0;
    for (; l < slabs.n; ++l) {
      const int c = (int)((slabs.bytes[l] / 16 + kCopyVecs - 1) / kCopyVecs);
      if (chunk < c) break;
      chunk -= c;
    }
    const int64_t vecs = slabs.bytes[l] / 16;
    const uint4* from = reinterpret_cast<const uint4*>(static_cast<unsigned char*>(slabs.data[l]) + s * slabs.bytes[l]);
    uint4* to = reinterpret_cast<uint4*>(static_cast<unsigned char*>(slabs.data[l]) + d * slabs.bytes[l]);
    const int64_t v0 = chunk * kCopyVecs + threadIdx.x;
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e)
      if (v0 + e * kCopyThreads < vecs) x[e] = __ldcs(from + v0 + e * kCopyThreads);
#pragma unroll
    for (int e = 0; e < kCopyUnroll; ++e)
      if (v0 + e * kCopyThreads < vecs) to[v0 + e * kCopyThreads] = x[e];
  }
}

int chunks_per_slot(const SlabList& slabs) {
  int64_t c = 0;
  for (int l = 0; l < slabs.n; ++l) c += (slabs.bytes[l] / 16 + kCopyVecs - 1) / kCopyVecs;
  return (int)c;
}

cudaError_t copy_pairs(const SlabList& slabs, const Pairs& q, cudaStream_t stream) {
  if (q.n == 0 || q.chunks_per_slot == 0) return cudaSuccess;
  const int per_sm = prepare_kernel(reinterpret_cast<const void*>(&slab_copy_kernel), kCopyThreads, 0);
  if (per_sm <= 0) return cudaErrorInvalidConfiguration;
  const int64_t work = (int64_t)q.n * q.chunks_per_slot;
  const int grid = (int)std::min<int64_t>(work, (int64_t)device_sm_count() * per_sm);
  slab_copy_kernel<<<grid, kCopyThreads, 0, stream>>>(slabs, q);
  return cudaGetLastError();
}

// ---- planning ------------------------------------------------------------------------------

// One CTA of 64 threads per sequence, thread j = new beam j: the first child of a beam keeps
// its slot, the k-th other child takes the slot of the k-th beam without a child.
__global__ void __launch_bounds__(64) reorder_plan_kernel(int K, int n_slots, const int32_t* slots, const int32_t* parent,
                                                          int32_t* new_slots, int32_t* err) {
  __shared__ int par[64];
  __shared__ uint32_t has[2], other[2];
  const int j = threadIdx.x;
  const int64_t base = (int64_t)blockIdx.x * K;
  bool bad = false;
  int slot = 0;
  if (j < K) {
    par[j] = parent[base + j];
    slot = slots[base + j];
    bad = slot < 0 || slot >= n_slots;
  }
  if (j < 2) has[j] = 0u;
  const bool bad_parent = j < K && (par[j] < 0 || par[j] >= K);
  const bool any_slot = __syncthreads_or(bad), any_parent = __syncthreads_or(bad_parent);
  if (any_slot || any_parent) {  // this sequence stays as it is
    if (j == 0) report(err, (any_slot ? LA_DEVERR_READ_SLOT : 0u) | (any_parent ? LA_DEVERR_TREE : 0u));
    if (j < K) new_slots[base + j] = -1;
    return;
  }
  bool first = true;
  if (j < K) {
    for (int i = 0; i < j; ++i) first &= par[i] != par[j];
    atomicOr(&has[par[j] >> 5], 1u << (par[j] & 31));
  }
  const uint32_t rest = __ballot_sync(0xffffffffu, j < K && !first);
  if ((j & 31) == 0) other[j >> 5] = rest;
  __syncthreads();
  if (j >= K) return;
  int from = par[j];
  if (!first) {
    int k = __popc(other[j >> 5] & ((1u << (j & 31)) - 1u)) + (j >= 32 ? __popc(other[0]) : 0);
    for (from = 0; from < K; ++from) {  // the k-th beam without a child
      if (has[from >> 5] >> (from & 31) & 1u) continue;
      if (k-- == 0) break;
    }
  }
  new_slots[base + j] = slots[base + from];
}

constexpr int kPlanThreads = 1024;

// Exclusive rank of `flag` among the CTA's threads in order, and the total.
__device__ __forceinline__ int block_rank(bool flag, int* warp_count, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) warp_count[warp] = __popc(m);
  __syncthreads();
  int before = 0;
  total = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    before += w < warp ? warp_count[w] : 0;
    total += warp_count[w];
  }
  return before + __popc(m & ((1u << lane) - 1u));
}

// The n lowest slots with ref 0, in order; -1 behind the last free one.  With sources (fork):
// one for each source that is held, -1 for the others.
__global__ void __launch_bounds__(kPlanThreads) alloc_kernel(int32_t* ref, int n_slots, int n, int32_t* slots,
                                                             const int32_t* src, int32_t* err) {
  __shared__ int warp_count[kPlanThreads / 32];
  int want = n, total;
  uint32_t bad = 0u;
  auto held = [&](int i) {  // before any count changes
    const int s = src[i];
    if (s < 0 || s >= n_slots) {
      bad |= LA_DEVERR_READ_SLOT;
      return false;
    }
    if (ref[s] <= 0) bad |= LA_DEVERR_REF;
    return ref[s] > 0;
  };
  if (src) {
    want = 0;
    for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
      const int i = i0 + threadIdx.x;
      block_rank(i < n && held(i), warp_count, total);
      want += total;
    }
    if (bad) report(err, bad);
    __syncthreads();
  }
  int found = 0;
  for (int s0 = 0; s0 < n_slots && found < want; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const bool free = s < n_slots && ref[s] == 0;
    const int rank = found + block_rank(free, warp_count, total);
    if (free && rank < want) slots[rank] = s;
    found += total;
  }
  __syncthreads();
  if (found < want && threadIdx.x == 0) report(err, LA_DEVERR_NO_SLOT);
  if (!src) {
    for (int i = threadIdx.x; i < n; i += kPlanThreads) {
      if (i < found) ref[slots[i]] = 1;
      else slots[i] = -1;
    }
    return;
  }
  // spread the list over the held sources from the back: entry i reads a place at or before
  // it; the counts change last, when no source is looked up any more
  int behind = 0;
  for (int i0 = (n - 1) / kPlanThreads * kPlanThreads; i0 >= 0; i0 -= kPlanThreads) {
    const int i = i0 + threadIdx.x;
    const bool ok = i < n && held(i);
    const int rank = block_rank(ok, warp_count, total);
    const int at = want - behind - total + rank;
    const int s = ok && at < found ? slots[at] : -1;
    __syncthreads();
    if (i < n) slots[i] = s;
    behind += total;
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n; i += kPlanThreads)
    if (slots[i] >= 0) ref[slots[i]] = 1;
}

__global__ void __launch_bounds__(256) ref_kernel(int32_t* ref, int n_slots, int n, const int32_t* slots, int delta,
                                                  int32_t* err) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int s = slots[i];
  if (s == -1) return;
  if (s < 0 || s >= n_slots) {
    report(err, LA_DEVERR_READ_SLOT);
    return;
  }
  // counted up or down only while it is held, whatever else this call does to the same slot
  int old = *reinterpret_cast<volatile int32_t*>(ref + s);
  while (old > 0) {
    const int seen = atomicCAS(ref + s, old, old + delta);
    if (seen == old) return;
    old = seen;
  }
  report(err, LA_DEVERR_REF);
}

// One CTA: live slots behind the first n_live go to the free ones before, both in order.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(int n_slots, const int32_t* ref, int32_t* new_ref,
                                                                    int32_t* remap, int32_t* moves, int32_t* counts) {
  __shared__ int warp_count[kPlanThreads / 32];
  int n_live = 0, total;
  for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    block_rank(s < n_slots && ref[s] > 0, warp_count, total);
    n_live += total;
  }
  // new_ref holds the free places, in order, until the moves are known
  int holes = 0, moved = 0;
  for (int s0 = 0; s0 < n_live; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const bool hole = s < n_live && !(ref[s] > 0);
    const int rank = holes + block_rank(hole, warp_count, total);
    if (hole) new_ref[rank] = s;
    holes += total;
  }
  __syncthreads();
  for (int s0 = 0; s0 < n_slots; s0 += kPlanThreads) {
    const int s = s0 + threadIdx.x;
    const bool live = s < n_slots && ref[s] > 0;
    const bool tail = live && s >= n_live;
    const int rank = moved + block_rank(tail, warp_count, total);
    if (s < n_slots) remap[s] = tail ? new_ref[rank] : live ? s : -1;
    if (tail) moves[rank] = s;
    moved += total;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n_slots; s += kPlanThreads) {
    if (s >= moved) moves[s] = -1;
    new_ref[s] = 0;
  }
  __syncthreads();
  for (int s = threadIdx.x; s < n_slots; s += kPlanThreads)
    if (remap[s] >= 0) new_ref[remap[s]] = ref[s];
  if (threadIdx.x == 0) {
    counts[0] = n_live;
    counts[1] = moved;
  }
}

__global__ void __launch_bounds__(256) remap_kernel(int64_t n, const int32_t* table, int n_slots, const int32_t* remap,
                                                    int32_t* new_table, int32_t* err) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int s = table[i];
  int d = s;
  if (s != -1) {
    if (s < 0 || s >= n_slots) report(err, LA_DEVERR_READ_SLOT);
    else d = remap[s];
  }
  new_table[i] = d;
}

}  // namespace

cudaError_t launch_pool_reorder(const SlabList& slabs, int32_t n_slots, int32_t n_seqs, int32_t n_beams,
                                const int32_t* slots, const int32_t* parent, int32_t* new_slots, int32_t* err,
                                cudaStream_t stream) {
  reorder_plan_kernel<<<n_seqs, 64, 0, stream>>>(n_beams, n_slots, slots, parent, new_slots, err);
  Pairs q{};
  q.n = n_seqs * n_beams;
  q.src = slots;
  q.via = parent;
  q.group = n_beams;
  q.dst = new_slots;
  q.n_slots = n_slots;
  q.chunks_per_slot = chunks_per_slot(slabs);
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_alloc(int32_t* ref, int32_t n_slots, int32_t n, int32_t* slots, int32_t* err,
                              cudaStream_t stream) {
  alloc_kernel<<<1, kPlanThreads, 0, stream>>>(ref, n_slots, n, slots, nullptr, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_ref(int32_t* ref, int32_t n_slots, int32_t n, const int32_t* slots, int32_t delta, int32_t* err,
                            cudaStream_t stream) {
  ref_kernel<<<(n + 255) / 256, 256, 0, stream>>>(ref, n_slots, n, slots, delta, err);
  return cudaGetLastError();
}

cudaError_t launch_pool_fork(const SlabList& slabs, int32_t* ref, int32_t n_slots, int32_t n, const int32_t* src_slots,
                             int32_t* new_slots, int32_t* err, cudaStream_t stream) {
  alloc_kernel<<<1, kPlanThreads, 0, stream>>>(ref, n_slots, n, new_slots, src_slots, err);
  Pairs q{};
  q.n = n;
  q.src = src_slots;
  q.dst = new_slots;
  q.n_slots = n_slots;
  q.chunks_per_slot = chunks_per_slot(slabs);
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_compact(const SlabList& slabs, int32_t n_slots, const int32_t* ref, int32_t* new_ref,
                                int32_t* remap, int32_t* moves, int32_t* counts, int32_t* err, cudaStream_t stream) {
  compact_plan_kernel<<<1, kPlanThreads, 0, stream>>>(n_slots, ref, new_ref, remap, moves, counts);
  Pairs q{};
  q.n = n_slots / 2;  // at most as many moves as free places
  q.n_dev = counts + 1;
  q.src = moves;
  q.dst = remap;
  q.dst_by_src = 1;
  q.n_slots = n_slots;
  q.chunks_per_slot = chunks_per_slot(slabs);
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_remap(int64_t n, const int32_t* table, int32_t n_slots, const int32_t* remap,
                              int32_t* new_table, int32_t* err, cudaStream_t stream) {
  remap_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(n, table, n_slots, remap, new_table, err);
  return cudaGetLastError();
}

}  // namespace la
