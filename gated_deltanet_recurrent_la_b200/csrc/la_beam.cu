// la_beam.cu -- beam search's selection over beams and vocabulary (la_beam_select).
//
// Candidate (i, v) of a sequence has the score cum_i + x_iv - logsumexp(x_i).  Within a beam
// the order of the candidates is the order of the logits, so each beam's best n_out come from
// its logits alone (ties to the lower index), and the sequence's best n_out are among them.
// Scores are formed of the log-sum and compared in FP64: neighbouring candidates can lie closer
// than an FP32 rounding of a sum of their size, and their order decides whole numbers.  A
// log-sum is that of FP32 exponentials, four or eight of them added in FP32 and those sums in
// FP64: an exponential is off by at most 2^-22 and 2^-22.8 per unit of the distance to its
// reference, a sum of eight by 2^-21, which leaves about 2^-20 and decides how beams of almost
// equal scores are ordered.  The sums depend on the row's values alone, not on where it lies, so
// beams with equal logits and cum_score tie.
//
// beam_row_kernel reads a row (or a part of it, where rows are few) once from memory: each
// thread keeps the place of its best piece of 16 bytes and a sum of exponentials against a
// reference that follows the maximum loosely (they stay below e^8, and it seldom moves).  NaN and
// +inf show in a piece's maximum or sum and send it to a slower form, so nothing is cleaned
// element by element: about 50 instructions a piece of eight.  The threads form 128 groups; the
// n_out-th best of the groups' best elements is at or below the row's n_out-th best element, and
// elements at or above it lie in n_out groups only, so a second look (from L2) at those few per
// cent of the row finds every candidate: n_out of them and a handful more, which are ranked by
// counting.  beam_merge_kernel joins the sorted lists.
// 384 rows of 50257 BF16 logits take 27 us (24 of 50256), of which their bytes are 6 and the
// exponentials 4: bound by the phases of a single wave of two or three CTAs per SM (reading,
// groups, ranks, second look), which all pass at the same time.
#include <type_traits>

#include "la_device.cuh"
#include "la_serving.h"

namespace la {

namespace {

constexpr int kRowThreads = 512;
constexpr int kGroups = 128;    // of threads tid, tid + 128, ..; at least LA_BEAM_MAX
constexpr int kCand = 512;      // candidates kept of one part
constexpr int kMaxParts = 16;
static_assert(kGroups >= LA_BEAM_MAX && kCand <= kRowThreads && kRowThreads % kGroups == 0, "sizes");

struct BeamPart {   // of one part of a row: then n_out keys (order of the logit, ~index), best first; 0 = none
  double sum;       // of exp(x - ref)
  float ref;        // -inf: nothing
  float pad;
};
__host__ __device__ constexpr int64_t beam_part_bytes(int n_out) { return (int64_t)sizeof(BeamPart) + 8 * (int64_t)n_out; }

// Parts of a row: enough of them for two CTAs on each of a B200's 148 SMs, of 4096 elements at
// least (below that the merge costs more than the reading).  A number of the sizes alone, so that
// a row's sums are the same on every device and in every workspace.
int beam_parts(int64_t rows, int64_t vocab) {
  int64_t s = (2 * 148 + rows - 1) / rows;
  if (s > vocab / 4096) s = vocab / 4096;
  return (int)(s < 1 ? 1 : s > kMaxParts ? kMaxParts : s);
}

// FP32 order as an unsigned key; -0 counts as +0, NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float beam_clean(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f) + 0.0f; }
__device__ __forceinline__ uint32_t beam_order(float x) {
  const uint32_t w = __float_as_uint(x);
  return w & 0x80000000u ? ~w : w | 0x80000000u;
}
__device__ __forceinline__ float beam_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t beam_key(float x, int v) {
  return ((uint64_t)beam_order(x) << 32) | (0xffffffffu - (uint32_t)v);
}

// Elements [lo, hi) of a row in pieces of four 4-byte words.  A chunk is 128 words; piece j holds
// words lane, lane + 32, + 64, + 96 (lane = j % 32) of chunk j / 32, counted from lo wherever the
// row lies in memory: what a thread adds up, and in which order, depends on the row's values
// alone, so equal rows have equal sums.  A warp reads a chunk with four coalesced loads.  BF16
// rows that begin in the middle of a word (`odd`) are turned by a half word between neighbours.
template <typename IT>
struct RowPieces {
  static constexpr int W = 4 / (int)sizeof(IT), E = 4 * W, kChunk = 128 * W;  // elements of a word, a piece, a chunk
  const uint32_t* words;  // the word with element lo
  int lo, len, odd, chunks;
  __device__ __forceinline__ RowPieces(const IT* row, int lo_, int hi_) : lo(lo_), len(hi_ - lo_) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(row + lo_);
    odd = W == 2 ? (int)(at >> 1 & 1u) : 0;
    words = reinterpret_cast<const uint32_t*>(at & ~(uintptr_t)3);
    chunks = (len + kChunk - 1) / kChunk;
  }
  // element e of piece j counted from lo (those of a piece rise with e), and whether the row has it
  static __device__ __forceinline__ int place(int j, int e) { return ((j >> 5) * 128 + (j & 31) + e / W * 32) * W + e % W; }
  __device__ __forceinline__ bool has(int j, int e) const { return place(j, e) < len; }
  // whether every word of chunk c, and the one behind it, lies within the elements
  __device__ __forceinline__ bool inner(int c) const { return c >= odd && (c + 1) * kChunk + odd <= len; }
  // word i; elements outside are not read and count as -inf
  __device__ __forceinline__ uint32_t word(int i) const {
    if constexpr (W == 1) {
      return i < len ? ld_coherent(words + i) : 0xff800000u;
    } else {
      const int a = 2 * i - odd;
      if (a >= 0 && a + 1 < len) return ld_coherent(words + i);
      const unsigned short* h = reinterpret_cast<const unsigned short*>(words + i);
      return (a >= 0 && a < len ? (uint32_t)h[0] : 0xff80u) | (a + 1 < len ? (uint32_t)h[1] : 0xff80u) << 16;
    }
  }
  __device__ __forceinline__ uint4 words_at(int i) const { return make_uint4(word(i), word(i + 32), word(i + 64), word(i + 96)); }
  static __device__ __forceinline__ uint4 turn(const uint4& w, const uint4& b) {
    return make_uint4(__funnelshift_r(w.x, b.x, 16), __funnelshift_r(w.y, b.y, 16), __funnelshift_r(w.z, b.z, 16),
                      __funnelshift_r(w.w, b.w, 16));
  }
  __device__ __forceinline__ uint4 load(int j) const {
    const int i = (j >> 5) * 128 + (j & 31);
    return odd ? turn(words_at(i), words_at(i + 1)) : words_at(i);
  }
  // of the piece's values f = unpack(w): NaN counts as nothing unless all are
  static __device__ __forceinline__ float largest(const uint4& w, const float* f) {
    if constexpr (sizeof(IT) == 4) {
      return fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3]));
    } else {
      const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&w);
      const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
      return fmaxf(__low2float(m), __high2float(m));
    }
  }
  static __device__ __forceinline__ void values(const uint4& w, float* f) {
    StateVec<IT>::unpack(w, f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = beam_clean(f[e]);
  }
};

// 2^x to about 2^-22 of its value, 0 for results below 2^-126
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename IT>
__global__ void __launch_bounds__(kRowThreads, 3) beam_row_kernel(const BeamParams p, int parts) {
  constexpr int E = RowPieces<IT>::E;
  __shared__ uint64_t keys[kRowThreads];  // the threads' best, then the groups', then the candidates
  __shared__ double sums[kRowThreads / 32];
  __shared__ float tops[kRowThreads / 32];
  __shared__ int ranks[kGroups];
  __shared__ int winners[LA_BEAM_MAX];
  __shared__ uint64_t tau;
  __shared__ int n_win, n_cand;
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x / parts, part = blockIdx.x % parts, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const float cum = p.cum[row];
  const bool dead = !(cum > -INFINITY);
  const bool done = p.finished && p.finished[row] != 0;
  unsigned char* out = static_cast<unsigned char*>(p.workspace) + (int64_t)blockIdx.x * beam_part_bytes(p.n_out);
  uint64_t* best = reinterpret_cast<uint64_t*>(out + sizeof(BeamPart));
  BeamPart* head = reinterpret_cast<BeamPart*>(out);
  const int take = min(p.n_out, p.vocab);
  if (dead || done) {  // no logits: eos at the beam's own score, everything else -inf
    for (int r = tid; r < take; r += kRowThreads) {
      uint64_t k = 0;
      if (part == 0) {
        if (dead) k = beam_key(-INFINITY, r);
        else k = r == 0 ? beam_key(0.0f, p.eos) : beam_key(-INFINITY, r - 1 < p.eos ? r - 1 : r);
      }
      best[r] = k;
    }
    if (tid == 0) *head = BeamPart{0.0, -INFINITY, 0.0f};
    return;
  }
  const int span = (p.vocab + parts - 1) / parts, lo = part * span, hi = min(p.vocab, lo + span);
  const RowPieces<IT> pieces(static_cast<const IT*>(p.logits) + (int64_t)row * p.row_stride, lo, hi);

  float ref = -INFINITY, at = -INFINITY;
  int where = -1;  // piece with the thread's first largest element, `at`
  double sum = 0.0;
  auto follow = [&](float m, int j) {  // m: the piece's maximum, finite or -inf
    if (m > at || where < 0) {
      at = m;
      where = j;
    }
    if (m > ref + 8.0f) {
      sum *= (double)expf(ref - m);
      ref = m;
    }
  };
  // of x - ref, rounded once before 2^.. (an offset of all logits cancels exactly)
  auto exponential = [&](float x) { return exp2_approx((x - ref) * 1.44269504f); };
  auto visit = [&](const uint4& w, int j) -> float {  // the piece's exponentials
    float f[E], s = 0.0f;
    StateVec<IT>::unpack(w, f);
    const float m = RowPieces<IT>::largest(w, f);
    if (m < INFINITY) {
      follow(m, j);
#pragma unroll
      for (int e = 0; e < E; ++e) s += exponential(f[e]);
      if (s < INFINITY) return s;
    }
    RowPieces<IT>::values(w, f);  // a NaN or +inf among them, or nothing finite so far
    float c = f[0];
#pragma unroll
    for (int e = 1; e < E; ++e) c = fmaxf(c, f[e]);
    follow(c, j);
    s = 0.0f;
    if (ref > -INFINITY)
#pragma unroll
      for (int e = 0; e < E; ++e) s += exponential(f[e]);
    return s;
  };
  constexpr int kWarps = kRowThreads / 32;
  auto walk = [&](auto odd) {  // a warp reads its chunks
    auto words = [&](int c, int i) {  // of an inner chunk, from word lane + i
      const uint32_t* at = pieces.words + c * 128 + lane + i;
      return make_uint4(ld_coherent(at), ld_coherent(at + 32), ld_coherent(at + 64), ld_coherent(at + 96));
    };
    auto turned = [&](const uint4& w, int c) {  // (the words behind lie in L1 by then)
      if constexpr (decltype(odd)::value) return pieces.turn(w, words(c, 1));
      else return w;
    };
    for (int c = warp; c < pieces.chunks; c += 4 * kWarps) {
      if (pieces.inner(c) && pieces.inner(c + 3 * kWarps)) {  // four of them in flight
        uint4 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = words(c + e * kWarps, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) sum += (double)visit(turned(w[e], c + e * kWarps), (c + e * kWarps) * 32 + lane);
      } else {
#pragma unroll 1
        for (int d = c; d < min(c + 4 * kWarps, pieces.chunks); d += kWarps) {
          const int j = d * 32 + lane;
          sum += (double)visit(pieces.inner(d) ? turned(words(d, 0), d) : pieces.load(j), j);
        }
      }
    }
  };
  if (pieces.odd) walk(std::true_type{});
  else walk(std::false_type{});

  keys[tid] = 0ull;
  if (where >= 0) {  // the first of the piece's largest elements
    float f[E];
    RowPieces<IT>::values(pieces.load(where), f);
    int first = -1;
#pragma unroll
    for (int e = E - 1; e >= 0; --e)
      if (f[e] == at && pieces.has(where, e)) first = lo + pieces.place(where, e);
    if (first >= 0) keys[tid] = beam_key(at + 0.0f, first);  // (-0 as +0)
  }
  // the sums against the largest reference of a warp, then of the CTA
  auto join = [&](float& r, double& x) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const float r2 = __shfl_xor_sync(0xffffffffu, r, off), to = fmaxf(r, r2);
      const double x2 = __shfl_xor_sync(0xffffffffu, x, off);
      if (to > -INFINITY) x = x * (double)expf(r - to) + x2 * (double)expf(r2 - to);
      r = to;
    }
  };
  join(ref, sum);
  if (lane == 0) {
    tops[warp] = ref;
    sums[warp] = sum;
  }
  if (tid < kGroups) ranks[tid] = 0;
  if (tid == 0) {
    tau = 0ull;
    n_cand = n_win = 0;
  }
  __syncthreads();
  uint64_t mine = 0ull;
  if (tid < kGroups) {
#pragma unroll
    for (int e = 0; e < kRowThreads / kGroups; ++e) mine = max(mine, keys[tid + e * kGroups]);
  } else if (warp == kGroups / 32) {
    float r = lane < kRowThreads / 32 ? tops[lane] : -INFINITY;
    double x = lane < kRowThreads / 32 ? sums[lane] : 0.0;
    join(r, x);
    if (lane == 0) *head = BeamPart{x, r, 0.0f};
  }
  __syncthreads();
  if (tid < kGroups) keys[tid] = mine;
  __syncthreads();
  {  // ranks of the groups' best: every thread compares with a quarter of them
    constexpr int kShare = kGroups * kGroups / kRowThreads;
    const uint64_t k = keys[tid % kGroups];
    int rank = 0;
#pragma unroll 8
    for (int g = 0; g < kShare; ++g) rank += keys[tid / kGroups * kShare + g] > k;
    if (rank) atomicAdd(&ranks[tid % kGroups], rank);
  }
  __syncthreads();
  if (tid < kGroups && mine) {
    const int rank = ranks[tid];
    if (rank < take) {
      winners[rank] = tid;
      atomicAdd(&n_win, 1);
      if (rank == take - 1) tau = mine;
    }
  }
  __syncthreads();
  // (fewer groups than n_out: the part has no more than 64 pieces, and all of it is taken)
  const uint64_t border = tau;
  const int wins = n_win, n_pieces = pieces.chunks * 32, per = (n_pieces + kGroups - 1) / kGroups;
  for (int e = tid; e < wins * per; e += kRowThreads) {
    const int jj = winners[e % wins] + e / wins * kGroups;
    if (jj >= n_pieces) continue;
    float f[E];
    RowPieces<IT>::values(pieces.load(jj), f);
#pragma unroll
    for (int c = 0; c < E; ++c) {
      const uint64_t k = beam_key(f[c], lo + pieces.place(jj, c));
      if (pieces.has(jj, c) && k >= border) {
        const int i = atomicAdd(&n_cand, 1);
        if (i < kCand) keys[i] = k;
      }
    }
  }
  __syncthreads();
  const int cand = n_cand;
  if (cand <= kCand) {
    for (int r = cand + tid; r < take; r += kRowThreads) best[r] = 0ull;
    if (tid < cand) {
      const uint64_t k = keys[tid];
      int rank = 0;
      for (int i = 0; i < cand; ++i) rank += keys[i] > k;
      if (rank < take) best[rank] = k;
    }
    return;
  }
  // Many of the best in few groups (values laid out with the groups' stride): one pass each.
  uint64_t last = ~0ull;
  for (int r = 0; r < take; ++r) {
    uint64_t k = 0;
    for (int q = tid; q < n_pieces; q += kRowThreads) {
      float f[E];
      RowPieces<IT>::values(pieces.load(q), f);
#pragma unroll
      for (int c = 0; c < E; ++c) {
        const uint64_t x = beam_key(f[c], lo + pieces.place(q, c));
        if (pieces.has(q, c) && x < last && x > k) k = x;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, off));
    __syncthreads();
    if (lane == 0) keys[warp] = k;
    __syncthreads();
    for (int w = 0; w < kRowThreads / 32; ++w) k = max(k, keys[w]);
    if (tid == 0) best[r] = k;
    last = k;
  }
}

// FP64 order as an unsigned key (no NaN; -0 as +0); every value's is above 0
__device__ __forceinline__ uint64_t score_key(double s) {
  const long long w = __double_as_longlong(s + 0.0);
  return w < 0 ? ~(uint64_t)w : (uint64_t)w | 0x8000000000000000ull;
}

// The largest key of a warp; 64 bits by two 32-bit reductions.
__device__ __forceinline__ uint64_t warp_max(uint64_t k) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return (uint64_t)hi << 32 | lo;
}

constexpr int kMergeThreads = 512;

// One CTA per sequence.  A warp per beam joins the lists of its parts (a lane per part, n_out
// rounds of a maximum over their heads), then one warp joins the beams' lists the same way
// (two beams a lane) by score, ties to the lower beam.
__global__ void __launch_bounds__(kMergeThreads) beam_merge_kernel(const BeamParams p, int parts) {
  extern __shared__ uint64_t sm[];
  const int b = blockIdx.x, K = p.n_beams, take = min(p.n_out, p.vocab);
  // score = offset + (x - ref): cum - log(sum) and the reference apart, so that neither is lost
  // beside logits of 1e38 (a row masked by the type's lowest value is a uniform one)
  double* offset = reinterpret_cast<double*>(sm);  // [K]
  double* refs = offset + K;                       // [K]
  uint64_t* lists = sm + 2 * K;                    // [K][take]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t pb = beam_part_bytes(p.n_out);
  const unsigned char* first = static_cast<const unsigned char*>(p.workspace) + (int64_t)b * K * parts * pb;
  __shared__ bool done[LA_BEAM_MAX];  // read before anything is written: finished_out may be finished
  griddep_wait();
  if (tid < K) {
    done[tid] = p.finished && p.finished[(int64_t)b * K + tid] != 0;
    const float cum = p.cum[(int64_t)b * K + tid];
    const unsigned char* w = first + (int64_t)tid * parts * pb;
    float ref = -INFINITY;
    for (int s = 0; s < parts; ++s) ref = fmaxf(ref, reinterpret_cast<const BeamPart*>(w + s * pb)->ref);
    double off = cum > -INFINITY ? (double)fminf(cum, 3.402823466e38f) : 0.0;
    if (ref > -INFINITY) {  // (a dead or finished beam, or one with every token masked, has none)
      double sum = 0.0;
      for (int s = 0; s < parts; ++s) {
        const BeamPart* q = reinterpret_cast<const BeamPart*>(w + s * pb);
        sum += q->sum * (double)expf(q->ref - ref);
      }
      off -= log(sum);
    }
    offset[tid] = off;
    refs[tid] = ref > -INFINITY ? (double)ref : 0.0;
  }
  if (parts == 1) {
    for (int e = tid; e < K * take; e += kMergeThreads)
      lists[e] = reinterpret_cast<const uint64_t*>(first + e / take * pb + sizeof(BeamPart))[e % take];
  } else {
    for (int i = warp; i < K; i += kMergeThreads / 32) {
      const uint64_t* mine = reinterpret_cast<const uint64_t*>(first + ((int64_t)i * parts + min(lane, parts - 1)) * pb +
                                                               sizeof(BeamPart));
      int at = 0;
      uint64_t k = lane < parts ? mine[0] : 0ull;
      uint64_t next = lane < parts && take > 1 ? mine[1] : 0ull;
      for (int r = 0; r < take; ++r) {
        const uint64_t m = warp_max(k);
        if (lane == 0) lists[i * take + r] = m;
        if (k == m && m) {
          ++at;
          k = next;
          next = at + 1 < take ? mine[at + 1] : 0ull;
        }
      }
    }
  }
  __syncthreads();
  if (warp != 0) return;
  int at[2] = {0, 0};
  uint64_t score[2];
  auto value = [&](int i, uint64_t k) { return offset[i] + ((double)beam_value((uint32_t)(k >> 32)) - refs[i]); };
  auto load = [&](int e) {
    const int i = lane + 32 * e;
    const uint64_t k = i < K && at[e] < take ? lists[i * take + at[e]] : 0ull;
    score[e] = k ? score_key(value(i, k)) : 0ull;
  };
  load(0);
  load(1);
  for (int r = 0; r < p.n_out; ++r) {
    const int e = score[1] > score[0];
    const uint64_t m = warp_max(score[e]);
    const uint32_t beam = __reduce_min_sync(0xffffffffu, score[0] == m ? lane : score[1] == m ? lane + 32 : 255);
    if ((beam & 31) == lane) {
      const int i = (int)beam, w = i >> 5;
      const uint64_t k = lists[i * take + (w ? at[1] : at[0])];
      const int64_t to = (int64_t)b * p.n_out + r;
      const int token = (int)(0xffffffffu - (uint32_t)k);
      p.parent[to] = i;
      p.token[to] = token;
      p.score[to] = (float)value(i, k);
      if (p.finished_out) p.finished_out[to] = done[i] || token == p.eos;
      if (w) {
        ++at[1];
        load(1);
      } else {
        ++at[0];
        load(0);
      }
    }
  }
}

}  // namespace

size_t beam_workspace_bytes(int64_t n_seqs, int64_t n_beams, int64_t vocab, int64_t n_out) {
  const int64_t rows = n_seqs * n_beams;
  return rows ? (size_t)(rows * beam_parts(rows, vocab) * beam_part_bytes((int)n_out)) : 0;
}

cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t stream) {
  const int rows = p.n_seqs * p.n_beams, parts = beam_parts(rows, p.vocab);
  const cudaError_t e = launch_dependent(p.io == LA_F32 ? beam_row_kernel<float> : beam_row_kernel<__nv_bfloat16>,
                                         rows * parts, kRowThreads, 0, stream, p, parts);
  if (e != cudaSuccess) return e;
  const int take = p.n_out < p.vocab ? p.n_out : p.vocab;
  return launch_dependent(beam_merge_kernel, p.n_seqs, kMergeThreads, 8 * p.n_beams * (2 + take), stream, p, parts);
}

}  // namespace la
