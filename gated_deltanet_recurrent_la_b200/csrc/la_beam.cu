// la_beam.cu -- beam search's selection over beams and vocabulary (la_beam_select).
//
// Candidate (i, v) of a sequence has the score cum_i + x_iv - logsumexp(x_i).  Within a beam
// the order of the candidates is the order of the logits, so each beam's best n_out come from
// its logits alone (ties to the lower index), and the sequence's best n_out are among them.
// Scores are formed and compared in FP64: neighbouring candidates can lie closer than an FP32
// rounding of a sum of their size, and their order decides whole numbers.
#include "la_device.cuh"
#include "la_serving.h"

namespace la {

namespace {

constexpr int kRowThreads = 256;

struct BeamRow {     // of one beam: the scores' offset cum - logsumexp, then n_out (logit, index) pairs
  double offset;
};
__host__ __device__ constexpr int64_t beam_row_bytes(int n_out) { return 8 + 8 * (int64_t)n_out; }

// FP32 order as an unsigned key; -0 counts as +0, NaN as -inf, +inf as the largest finite value
__device__ __forceinline__ float beam_clean(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f) + 0.0f; }
__device__ __forceinline__ uint32_t beam_order(float x) {
  const uint32_t w = __float_as_uint(x);
  return w & 0x80000000u ? ~w : w | 0x80000000u;
}
__device__ __forceinline__ float beam_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

template <typename IT>
__global__ void __launch_bounds__(kRowThreads) beam_row_kernel(const BeamParams p) {
  const int row = blockIdx.x, tid = threadIdx.x;
  const float cum = p.cum[row];
  const bool dead = !(cum > -INFINITY);
  const bool done = p.finished && p.finished[row] != 0;
  const IT* x = static_cast<const IT*>(p.logits) + (int64_t)row * p.row_stride;
  auto value = [&](int v) {
    if (dead) return -INFINITY;
    if (done) return v == p.eos ? 0.0f : -INFINITY;
    return beam_clean(io_load(x + v));
  };
  __shared__ uint64_t best[kRowThreads / 32];
  __shared__ double sums[kRowThreads / 32];
  unsigned char* out = static_cast<unsigned char*>(p.workspace) + row * beam_row_bytes(p.n_out);
  const int take = min(p.n_out, p.vocab);
  uint64_t last = ~0ull;
  float top = -INFINITY;
  for (int r = 0; r < take; ++r) {
    uint64_t k = 0;
    for (int v = tid; v < p.vocab; v += kRowThreads) {
      const uint64_t c = ((uint64_t)beam_order(value(v)) << 32) | (0xffffffffu - (uint32_t)v);
      if (c < last && c > k) k = c;
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) k = max(k, __shfl_xor_sync(0xffffffffu, k, off));
    if ((tid & 31) == 0) best[tid >> 5] = k;
    __syncthreads();
    k = best[0];
    for (int w = 1; w < kRowThreads / 32; ++w) k = max(k, best[w]);
    __syncthreads();
    if (r == 0) top = beam_value((uint32_t)(k >> 32));
    if (tid == 0) reinterpret_cast<uint64_t*>(out + 8)[r] = k;
    last = k;
  }
  double sum = 0.0;
  if (!dead && !done && top > -INFINITY)
    for (int v = tid; v < p.vocab; v += kRowThreads) sum += (double)expf(value(v) - top);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if ((tid & 31) == 0) sums[tid >> 5] = sum;
  __syncthreads();
  if (tid == 0) {
    sum = 0.0;
    for (int w = 0; w < kRowThreads / 32; ++w) sum += sums[w];
    double off = (double)fminf(cum, 3.402823466e38f);
    if (dead) off = 0.0;
    else if (!done && top > -INFINITY) off -= (double)top + log(sum);
    reinterpret_cast<BeamRow*>(out)->offset = off;
  }
}

// One CTA per sequence: every beam's list is in order, so a candidate's rank is the number of
// better ones in each list, by bisection.
__global__ void __launch_bounds__(kRowThreads) beam_merge_kernel(const BeamParams p) {
  const int b = blockIdx.x, K = p.n_beams, take = min(p.n_out, p.vocab);
  const unsigned char* rows = static_cast<const unsigned char*>(p.workspace) + (int64_t)b * K * beam_row_bytes(p.n_out);
  for (int c = threadIdx.x; c < K * take; c += kRowThreads) {
    const int i = c / take, e = c % take;
    const unsigned char* mine = rows + i * beam_row_bytes(p.n_out);
    const uint64_t k = reinterpret_cast<const uint64_t*>(mine + 8)[e];
    const double s = reinterpret_cast<const BeamRow*>(mine)->offset + (double)beam_value((uint32_t)(k >> 32));
    int rank = e;
    for (int o = 0; o < K; ++o) {
      if (o == i) continue;
      const unsigned char* other = rows + o * beam_row_bytes(p.n_out);
      const double off = reinterpret_cast<const BeamRow*>(other)->offset;
      int lo = 0, hi = take;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        const double so = off + (double)beam_value((uint32_t)(reinterpret_cast<const uint64_t*>(other + 8)[mid] >> 32));
        const bool better = so > s || (so == s && o < i);
        if (better) lo = mid + 1;
        else hi = mid;
      }
      rank += lo;
    }
    if (rank < p.n_out) {
      const int64_t at = (int64_t)b * p.n_out + rank;
      const int token = (int)(0xffffffffu - (uint32_t)k);
      p.parent[at] = i;
      p.token[at] = token;
      p.score[at] = (float)s;
      if (p.finished_out) p.finished_out[at] = (p.finished && p.finished[b * K + i] != 0) || token == p.eos;
    }
  }
}

}  // namespace

size_t beam_workspace_bytes(int64_t n_seqs, int64_t n_beams, int64_t vocab, int64_t n_out) {
  return (size_t)(n_seqs * n_beams * beam_row_bytes((int)n_out));
}

cudaError_t launch_beam_select(const BeamParams& p, cudaStream_t stream) {
  const int rows = p.n_seqs * p.n_beams;
  if (p.io == LA_F32) beam_row_kernel<float><<<rows, kRowThreads, 0, stream>>>(p);
  else beam_row_kernel<__nv_bfloat16><<<rows, kRowThreads, 0, stream>>>(p);
  beam_merge_kernel<<<p.n_seqs, kRowThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace la
