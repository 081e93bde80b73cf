// la_slots.cu -- slot bookkeeping on the device, over the slabs of all layers at once: beam
// reordering, allocation by reference counts, forking, freeing, compaction.
//
// Which slots move is decided by whole numbers, the same whatever the order of the threads: by a
// kernel of one CTA (allocation, compaction) or by the copying warps themselves (reordering).
// One copy kernel moves them in the slabs of all layers.
// Sources and destinations of the copies of one call never meet, so they run in any order.
#include <algorithm>

#include "la_device.cuh"
#include "la_serving.h"

namespace la {

namespace {

// ---- copies ---------------------------------------------------------------------------------
// Slots of many slabs, bound by HBM (each byte read and written once).  A slot is cut into
// pieces of at most kPiece bytes.  Every CTA of a persistent grid lists the pairs that move, a
// thread per pair (the same list in all of them); every warp takes the listed pairs' pieces a
// grid apart, so that all warps copy equally much to within a piece.  Its lanes work out 32
// pieces at a time (source, destination, bytes), and one lane moves them with bulk copies
// through a ring of kStages buffers in shared memory: loads kLead ahead of the stores, no
// registers in between.  Of 4 to 16 KiB pieces with 192 KiB of buffers, 16 KiB and three warps
// are fastest by up to 5 % (64 slots over eight layers, 1.15 GB moved: 193 us, 195 with 6 warps
// and 8 KiB, 211 with 16-byte loads and stores through registers).
constexpr int kCopyWarps = 3;
constexpr int kStages = 4;
constexpr int kLead = 2;
constexpr int kPiece = 16384;
constexpr int kCopySmem = kCopyWarps * kStages * kPiece + kCopyWarps * kStages * 8;

enum PairKind { kPairsList, kPairsMoves, kPairsBeams };

struct Pairs {
  int32_t kind;
  int32_t n;                // pairs (list, beams), their upper bound (moves)
  int32_t n_slots;
  // list: src[i] -> dst[i].  moves: src[i] -> dst[src[i]], i < *count.  beams: see beam_pair
  const int32_t* src;
  const int32_t* dst;
  const int32_t* count;
  int32_t n_beams;
  const int32_t* parent;
  int32_t* new_slots;
  int32_t* err;
};

// New beam i = (sequence, j) of a reordering: its slot, and the slot it is copied from (-1: it
// stays where its parent was).  The first child of a beam keeps its slot, the k-th other child
// takes the slot of the k-th beam without a child.  Whole numbers, the same in every warp.
__device__ __forceinline__ int beam_pair(const Pairs& q, int i, int& from, uint32_t& bad) {
  const int K = q.n_beams, j = i % K;
  const int32_t* slots = q.src + (i - j);
  const int32_t* par = q.parent + (i - j);
  uint64_t has = 0, others = 0;  // beams with a child; new beams that are not a first child
  bad = 0u;
  for (int e = 0; e < K; ++e) {
    const int s = ld_coherent(slots + e), pe = ld_coherent(par + e);
    if (s < 0 || s >= q.n_slots) bad |= LA_DEVERR_READ_SLOT;
    if (pe < 0 || pe >= K) {
      bad |= LA_DEVERR_TREE;
    } else {
      if (has >> pe & 1) others |= 1ull << e;
      has |= 1ull << pe;
    }
  }
  from = -1;
  if (bad) return -1;  // this sequence stays as it is
  const int mine = ld_coherent(par + j);
  if (!(others >> j & 1)) return ld_coherent(slots + mine);
  uint64_t spare = ~has;
  for (int k = __popcll(others & ((1ull << j) - 1)); k > 0; --k) spare &= spare - 1;
  from = ld_coherent(slots + mine);
  return ld_coherent(slots + __ffsll((long long)spare) - 1);
}

__global__ void __launch_bounds__(kCopyWarps * 32) slab_copy_kernel(const SlabList slabs, const Pairs q) {
  extern __shared__ __align__(128) unsigned char sm[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kCopyWarps * kStages * kPiece);
  __shared__ int from_slot[kCopyWarps * 32], to_slot[kCopyWarps * 32], count[kCopyWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = sm + warp * kStages * kPiece;
  uint64_t* full = bars + warp * kStages;
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(full + s, 1);
    mbar_init_fence();
  }
  __syncwarp();
  griddep_wait();
  const int n = q.kind == kPairsMoves ? min(q.n, ld_coherent(q.count)) : q.n;
  const int per = slabs.first[slabs.n];
  const int me = warp * (int)gridDim.x + (int)blockIdx.x, step = (int)gridDim.x * kCopyWarps;
  uint32_t loaded = 0, stored = 0;  // lane 0: pieces so far
  bool ok = true;
  uint32_t bytes_of[kStages];       // of the pieces in the ring
  unsigned char* to_of[kStages];
  auto store = [&] {
    const uint32_t s = stored % kStages;
    ok = mbar_wait(full + s, (stored / kStages) & 1u, slabs.wait_ns);
    if (!ok) return;
    unsigned char* to = nullptr;
    uint32_t nb = 0;
#pragma unroll
    for (int e = 0; e < kStages; ++e)
      if (s == (uint32_t)e) {
        to = to_of[e];
        nb = bytes_of[e];
      }
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_addr(ring + s * kPiece)),
                 "r"(nb)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    ++stored;
  };
  int64_t next = me;  // this warp's next piece, counted from the batch's first
  for (int64_t i0 = 0; i0 < n; i0 += kCopyWarps * 32) {
    int src = -1, dst = -1;
    if (i0 + threadIdx.x < n) {
      const int i = (int)i0 + (int)threadIdx.x;
      if (q.kind == kPairsBeams) {
        uint32_t bad;
        dst = beam_pair(q, i, src, bad);
        if (blockIdx.x == 0) {
          q.new_slots[i] = dst;
          if (bad && i % q.n_beams == 0) report(q.err, bad);
        }
      } else {
        src = ld_coherent(q.src + i);
        if (src >= 0 && src < q.n_slots) dst = ld_coherent(q.dst + (q.kind == kPairsMoves ? src : i));
      }
    }
    const bool moves = src >= 0 && src < q.n_slots && dst >= 0 && dst < q.n_slots && dst != src;
    const uint32_t among = __ballot_sync(0xffffffffu, moves);
    if (lane == 0) count[warp] = __popc(among);
    __syncthreads();
    int at = __popc(among & ((1u << lane) - 1u)), listed = 0;
#pragma unroll
    for (int w = 0; w < kCopyWarps; ++w) {
      at += w < warp ? count[w] : 0;
      listed += count[w];
    }
    if (moves) {
      from_slot[at] = src;
      to_slot[at] = dst;
    }
    __syncthreads();
    const int64_t work = (int64_t)listed * per;
    for (int64_t w0 = next; w0 < work; w0 += 32ll * step) {
      const int64_t w = w0 + (int64_t)lane * step;
      const unsigned char* from = nullptr;
      unsigned char* to = nullptr;
      uint32_t bytes = 0;
      if (w < work) {
        const int e = (int)(w / per), piece = (int)(w % per);
        const int s = from_slot[e], d = to_slot[e];
        int l = 0, hi = slabs.n - 1;
        while (l < hi) {  // the slab of the piece
          const int mid = (l + hi + 1) / 2;
          if (slabs.first[mid] <= piece) l = mid;
          else hi = mid - 1;
        }
        const int64_t size = slabs.bytes[l], off = (int64_t)(piece - slabs.first[l]) * kPiece;
        from = static_cast<const unsigned char*>(slabs.data[l]) + s * size + off;
        to = static_cast<unsigned char*>(slabs.data[l]) + d * size + off;
        bytes = (uint32_t)(size - off < kPiece ? size - off : kPiece);
      }
      for (uint32_t left = __ballot_sync(0xffffffffu, bytes != 0u); left; left &= left - 1) {
        const int e = __ffs(left) - 1;
        const uint64_t f = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(from), e);
        const uint64_t t = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(to), e);
        const uint32_t nb = __shfl_sync(0xffffffffu, bytes, e);
        if (lane == 0 && ok) {
          // the buffer's last store has been read out: at most kStages - 1 - kLead younger ones are not
          asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kStages - 1 - kLead) : "memory");
          const uint32_t s = loaded % kStages;
#pragma unroll
          for (int c = 0; c < kStages; ++c)
            if (s == (uint32_t)c) {
              to_of[c] = reinterpret_cast<unsigned char*>(t);
              bytes_of[c] = nb;
            }
          if (me != 0 || loaded != slabs.withhold) {
            mbar_arrive_expect_tx(full + s, nb);
            bulk_g2s(ring + s * kPiece, reinterpret_cast<const void*>(f), nb, full + s);
          }
          ++loaded;
          if (loaded - stored > kLead) store();
        }
      }
    }
    next = next < work ? next + (work - next + step - 1) / step * step - work : next - work;
  }
  if (lane == 0) {
    while (ok && stored < loaded) store();
    if (!ok) {
      report(q.err, LA_DEVERR_TIMEOUT);
      // no load may be in flight when the CTA ends: the one that was late gets its limit once more
      for (uint32_t e = stored; e < loaded; ++e)
        if (me != 0 || e != slabs.withhold) mbar_wait(full + e % kStages, (e / kStages) & 1u, slabs.wait_ns);
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
}

cudaError_t copy_pairs(const SlabList& in, const Pairs& q, cudaStream_t stream) {
  if (q.n == 0) return cudaSuccess;
  SlabList slabs = in;
  int64_t per = 0;
  for (int l = 0; l < slabs.n; ++l) {
    slabs.first[l] = (int32_t)per;
    per += (slabs.bytes[l] + kPiece - 1) / kPiece;
  }
  if (per > INT32_MAX) return cudaErrorInvalidValue;
  slabs.first[slabs.n] = (int32_t)per;
  if (prepare_kernel(reinterpret_cast<const void*>(&slab_copy_kernel), kCopyWarps * 32, kCopySmem) <= 0)
    return cudaErrorInvalidConfiguration;
  const int grid = (int)std::min<int64_t>((int64_t)q.n * per, device_sm_count());
  return launch_dependent(slab_copy_kernel, grid, kCopyWarps * 32, kCopySmem, stream, slabs, q);
}

// ---- planning ------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
static_assert(kPlanThreads == 32 * 32, "block_rank reads one count per lane");

// Exclusive rank of `flag` among the CTA's threads in order, and the total.
__device__ __forceinline__ int block_rank(bool flag, int* warp_count, int& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, flag);
  __syncthreads();
  if (lane == 0) warp_count[warp] = __popc(m);
  __syncthreads();
  const int c = warp_count[lane];
  total = __reduce_add_sync(0xffffffffu, c);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? c : 0);
  return before + __popc(m & ((1u << lane) - 1u));
}

// The n lowest slots with ref 0, in order; -1 behind the last free one.  With sources (fork):
// one for each source that is held, -1 for the others.
__global__ void __launch_bounds__(kPlanThreads) alloc_kernel(int32_t* ref, int n_slots, int n, int32_t* slots,
                                                             const int32_t* src, int32_t* err) {
  __shared__ int warp_count[kPlanThreads / 32];
  griddep_wait();
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
  griddep_wait();
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
  griddep_wait();
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
  griddep_wait();
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
  Pairs q{};
  q.kind = kPairsBeams;
  q.n = n_seqs * n_beams;
  q.n_slots = n_slots;
  q.src = slots;
  q.n_beams = n_beams;
  q.parent = parent;
  q.new_slots = new_slots;
  q.err = err;
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_alloc(int32_t* ref, int32_t n_slots, int32_t n, int32_t* slots, int32_t* err,
                              cudaStream_t stream) {
  return launch_dependent(alloc_kernel, 1, kPlanThreads, 0, stream, ref, n_slots, n, slots, (const int32_t*)nullptr, err);
}

cudaError_t launch_pool_ref(int32_t* ref, int32_t n_slots, int32_t n, const int32_t* slots, int32_t delta, int32_t* err,
                            cudaStream_t stream) {
  return launch_dependent(ref_kernel, (n - 1) / 256 + 1, 256, 0, stream, ref, n_slots, n, slots, delta, err);
}

cudaError_t launch_pool_fork(const SlabList& slabs, int32_t* ref, int32_t n_slots, int32_t n, const int32_t* src_slots,
                             int32_t* new_slots, int32_t* err, cudaStream_t stream) {
  const cudaError_t e = launch_dependent(alloc_kernel, 1, kPlanThreads, 0, stream, ref, n_slots, n, new_slots, src_slots, err);
  if (e != cudaSuccess) return e;
  Pairs q{};
  q.kind = kPairsList;
  q.n = n;
  q.n_slots = n_slots;
  q.src = src_slots;
  q.dst = new_slots;
  q.err = err;
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_compact(const SlabList& slabs, int32_t n_slots, const int32_t* ref, int32_t* new_ref,
                                int32_t* remap, int32_t* moves, int32_t* counts, int32_t* err, cudaStream_t stream) {
  const cudaError_t e = launch_dependent(compact_plan_kernel, 1, kPlanThreads, 0, stream, n_slots, ref, new_ref, remap, moves, counts);
  if (e != cudaSuccess) return e;
  Pairs q{};
  q.kind = kPairsMoves;
  q.n = n_slots / 2;  // at most as many moves as free places
  q.n_slots = n_slots;
  q.src = moves;
  q.dst = remap;
  q.count = counts + 1;
  q.err = err;
  return copy_pairs(slabs, q, stream);
}

cudaError_t launch_pool_remap(int64_t n, const int32_t* table, int32_t n_slots, const int32_t* remap,
                              int32_t* new_table, int32_t* err, cudaStream_t stream) {
  return launch_dependent(remap_kernel, (int)((n - 1) / 256 + 1), 256, 0, stream, n, table, n_slots, remap, new_table, err);
}

}  // namespace la
