// la_tree.cuh -- drafted token trees over the slot pool (la_state_tree, la_state_tree_commit).
//
// A request's drafted tokens form a tree below its current state S0.  Node t with parent p
// continues S_p:  S_t = a_t S_p + k_t u_t^T,  u_t = b_t (v_t - c_t S_p^T k_t),  o_t = scale
// S_t^T q_t.  No S_t is ever formed.  With D_ts the product of the gates on the path from s
// (exclusive) down to t and Gamma_t that from the root (kda: one product per key channel),
// unrolling the recurrence along the path gives
//   u_t = b_t (v_t - [S0^T (Gamma_t k_t) + sum_{s above t} (k_t . D_ts k_s) u_s])    (delta rules)
//   o_t = scale (S0^T (Gamma_t q_t) + sum_{s above or at t} (q_t . D_ts k_s) u_s)
// so S0 is read once and nothing is written but the outputs (and u, for the commit).  The
// products D_ts are taken step by step along the path, never as ratios, so a gate of zero or
// of either sign is exact, and sums run over a node's own path only, so a non-finite value in
// one branch does not reach another.
#pragma once

#include "la_device.cuh"
#include "la_serving.h"

namespace la {
namespace tree {

constexpr int kMaxNodes = LA_TREE_MAX_NODES;

// A state tile of a pool.
template <typename ST>
struct TileReader {
  const ST* tile;
  __device__ __forceinline__ void init(const void* pool, int64_t tile_index, int dk, int dv, int, const int*) {
    tile = static_cast<const ST*>(pool) + tile_index * dk * dv;
  }
  template <int DV>
  __device__ __forceinline__ float at(int i, int j) const { return io_load(tile + i * DV + j); }
};
template <>
struct TileReader<q8_t> {
  const unsigned char* tile;
  int n8;
  const int* row_info;  // of row i: its rank in its block, times two, plus one for a BF16 row
  __device__ __forceinline__ void init(const void* pool, int64_t tile_index, int dk, int dv, int n_hp, const int* info) {
    tile = static_cast<const unsigned char*>(pool) + tile_index * q8_tile_bytes(dk, dv, n_hp);
    n8 = dk - n_hp;
    row_info = info;
  }
};

// Ranks of a q8 head's rows (threads of the CTA, dk <= blockDim.x); false for a mask that does not hold n_hp rows.
__device__ __forceinline__ bool q8_rows(const uint32_t* mask, int dk, int n_hp, int* row_info) {
  int count = 0;
  for (int w = 0; w < dk / 32; ++w) count += __popc(ld_coherent(mask + w));
  if (count != n_hp) return false;
  for (int i = threadIdx.x; i < dk; i += blockDim.x) {
    int below = 0;
    for (int w = 0; w < i / 32; ++w) below += __popc(ld_coherent(mask + w));
    const uint32_t m = ld_coherent(mask + i / 32);
    below += __popc(m & ((1u << (i & 31)) - 1u));
    const bool hp = (m >> (i & 31)) & 1u;
    row_info[i] = hp ? 2 * below + 1 : 2 * (i - below);
  }
  return true;
}

// The nodes of sequence b: c0 and their number, -1 when the offsets or the count are wrong.
__device__ __forceinline__ int tree_span(const int32_t* cu, int total, int max_nodes, int b, int& c0) {
  c0 = ld_coherent(cu + b);
  const int c1 = ld_coherent(cu + b + 1);
  if (c0 < 0 || c1 < c0 || c1 > total) return -1;
  return c1 - c0 > max_nodes ? -2 : c1 - c0;
}
__device__ __forceinline__ uint32_t span_error(int n) { return n == -1 ? LA_DEVERR_CU_SEQLENS : LA_DEVERR_TREE; }

// Piece c (16 bytes; of INT8 rows 8, with their scale) of row i of a tile as it lies in memory, and its values.
template <typename ST>
struct RawPiece {
  uint4 w;
};
template <>
struct RawPiece<q8_t> {
  uint4 w;      // BF16 values, or codes in w.x, w.y
  float scale;  // negative: BF16
};
template <typename ST, int DV>
__device__ __forceinline__ RawPiece<ST> raw_piece(const TileReader<ST>& S, int i, int c) {
  RawPiece<ST> r;
  if constexpr (std::is_same<ST, q8_t>::value) {
    constexpr int NG = DV / 32;
    const int e = S.row_info[i], idx = e >> 1;
    if (e & 1) {
      r.w = __ldcs(reinterpret_cast<const uint4*>(S.tile + S.n8 * DV + S.n8 * NG * 4 + (idx * DV + 8 * c) * 2));
      r.scale = -1.0f;
    } else {
      const uint2 w = __ldcs(reinterpret_cast<const uint2*>(S.tile + idx * DV + 8 * c));
      r.w = make_uint4(w.x, w.y, 0u, 0u);
      r.scale = reinterpret_cast<const float*>(S.tile + S.n8 * DV)[idx * NG + (c >> 2)];
    }
  } else {
    r.w = __ldcs(reinterpret_cast<const uint4*>(S.tile + i * DV) + c);
  }
  return r;
}
template <typename ST>
__device__ __forceinline__ void unpack_piece(const RawPiece<ST>& r, float* x) {
  if constexpr (std::is_same<ST, q8_t>::value) {
    if (r.scale < 0.0f) {
      StateVec<__nv_bfloat16>::unpack(r.w, x);
    } else {
      const uint32_t words[2] = {r.w.x, r.w.y};
      q8_unpack<8>(words, r.scale, x);
    }
  } else {
    StateVec<ST>::unpack(r.w, x);
  }
}

// eight consecutive state values (columns 8 c ..) of row i in FP32
template <typename ST, int DV>
__device__ __forceinline__ void state_eight(const TileReader<ST>& S, int i, int c, float* x) {
  if constexpr (std::is_same<ST, float>::value) {
    unpack_piece(raw_piece<ST, DV>(S, i, 2 * c), x);
    unpack_piece(raw_piece<ST, DV>(S, i, 2 * c + 1), x + 4);
  } else {
    unpack_piece(raw_piece<ST, DV>(S, i, c), x);
  }
}

// ---- verification ------------------------------------------------------------------------

constexpr int kTreeThreads = 128;
constexpr int kBlock = 16;  // nodes whose products with S0 are formed in one pass over it

template <int DK, int DV>
__host__ __device__ constexpr int tree_smem(int rows, bool kda) {
  return 4 * (rows * DK * (kda ? 3 : 2) + 2 * rows * rows + rows * DV + 2 * kBlock * DV + 3 * rows);
}

// The form for heads too narrow for the tensor cores (16 x 16).  One CTA per (sequence, state
// head), FP32 throughout.  The pair coefficients are one warp per node walking to the root; the
// products with S0 one column of d_v per thread (kBlock nodes per pass); the substitution one
// column per thread, node after node.
template <typename ST, typename IT, int DK, int DV, bool KDA>
__global__ void __launch_bounds__(kTreeThreads) tree_kernel(const TreeParams p, int rows) {
  extern __shared__ __align__(16) float sm[];
  float* K = sm;                        // [rows][DK]
  float* Q = K + rows * DK;             // [rows][DK] (kda: scaled by Gamma after the pair pass)
  float* KG = Q + rows * DK;            // [rows][DK] kda: K scaled by Gamma
  float* KK = KDA ? KG + rows * DK : KG;  // [rows][rows]
  float* QK = KK + rows * rows;
  float* U = QK + rows * rows;          // [rows][DV]
  float* buf = U + rows * DV;           // [kBlock][2][DV]
  float* gamma = buf + 2 * kBlock * DV; // [rows]
  float* gate = gamma + rows;           // [rows] (scalar gates)
  int* par = reinterpret_cast<int*>(gate + rows);  // [rows]

  griddep_wait();
  const int H = p.n_v_heads;
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int hq = h / (H / p.n_qk_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int c0;
  const int n = tree_span(p.cu, p.total, p.max_nodes, b, c0);
  if (n < 0) {
    if (tid == 0) report(p.err, span_error(n));
    return;
  }
  if (n == 0) return;
  const int slot = p.read_slot ? ld_coherent(p.read_slot + b) : b;
  if (slot < 0 || slot >= p.src_slots) {
    if (tid == 0) report(p.err, LA_DEVERR_READ_SLOT);
    return;
  }
  bool bad = false;
  for (int t = tid; t < n; t += kTreeThreads) {
    const int pt = ld_coherent(p.parent + c0 + t);
    bad |= pt < -1 || pt >= t;
    par[t] = pt;
    if (!KDA) gate[t] = p.g ? ld_coherent(p.g + (int64_t)(c0 + t) * H + h) : 1.0f;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0) report(p.err, LA_DEVERR_TREE);
    return;
  }
  const IT* gq = static_cast<const IT*>(p.q);
  const IT* gk = static_cast<const IT*>(p.k);
  const IT* gv = static_cast<const IT*>(p.v);
  for (int e = tid; e < n * DK; e += kTreeThreads) {
    const int64_t at = ((int64_t)(c0 + e / DK) * p.n_qk_heads + hq) * DK + e % DK;
    K[e] = io_load(gk + at);
    Q[e] = io_load(gq + at);
  }
  __syncthreads();

  // pair coefficients and Gamma: one warp per node, lane = DK / 32 key channels
  constexpr int CH = DK / 32 > 0 ? DK / 32 : 1;
  const bool on = lane * CH < DK;
  for (int t = warp; t < n; t += kTreeThreads / 32) {
    float kt[CH], qt[CH], d[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      kt[c] = on ? K[t * DK + lane * CH + c] : 0.0f;
      qt[c] = on ? Q[t * DK + lane * CH + c] : 0.0f;
      d[c] = 1.0f;
    }
    int s = t;
    while (true) {
      float kk = 0.0f, qk = 0.0f;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float x = on ? d[c] * K[s * DK + lane * CH + c] : 0.0f;
        kk = fmaf(kt[c], x, kk);
        qk = fmaf(qt[c], x, qk);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        kk += __shfl_xor_sync(0xffffffffu, kk, off);
        qk += __shfl_xor_sync(0xffffffffu, qk, off);
      }
      if (lane == 0) {
        KK[t * rows + s] = kk;
        QK[t * rows + s] = qk;
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if constexpr (KDA) {
          if (on) d[c] *= ld_coherent(p.g + ((int64_t)(c0 + s) * H + h) * DK + lane * CH + c);
        } else {
          d[c] *= gate[s];
        }
      }
      s = par[s];
      if (s < 0) break;
    }
    if constexpr (KDA) {
      if (on) {
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          KG[t * DK + lane * CH + c] = kt[c] * d[c];
          Q[t * DK + lane * CH + c] = qt[c] * d[c];  // read by this warp only
        }
      }
    } else if (lane == 0) {
      gamma[t] = d[0];
    }
  }
  __syncthreads();

  TileReader<ST> S;
  S.init(p.src, (int64_t)slot * H + h, DK, DV, 0, nullptr);
  const float* KS = KDA ? KG : K;
  constexpr int NPT = kBlock * DV / kTreeThreads;  // nodes of a thread in one pass
  const int j = tid % DV, grp = tid / DV;
  for (int t0 = 0; t0 < n; t0 += kBlock) {
    float ak[NPT], aq[NPT];
#pragma unroll
    for (int m = 0; m < NPT; ++m) ak[m] = aq[m] = 0.0f;
    for (int i = 0; i < DK; i += 4) {
      float s[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) s[e] = S.template at<DV>(i + e, j);
#pragma unroll
      for (int m = 0; m < NPT; ++m) {
        const float4 kk = *reinterpret_cast<const float4*>(KS + (t0 + grp * NPT + m) * DK + i);
        const float4 qq = *reinterpret_cast<const float4*>(Q + (t0 + grp * NPT + m) * DK + i);
        ak[m] = fmaf(kk.x, s[0], fmaf(kk.y, s[1], fmaf(kk.z, s[2], fmaf(kk.w, s[3], ak[m]))));
        aq[m] = fmaf(qq.x, s[0], fmaf(qq.y, s[1], fmaf(qq.z, s[2], fmaf(qq.w, s[3], aq[m]))));
      }
    }
#pragma unroll
    for (int m = 0; m < NPT; ++m) {
      buf[(2 * (grp * NPT + m)) * DV + j] = ak[m];
      buf[(2 * (grp * NPT + m) + 1) * DV + j] = aq[m];
    }
    __syncthreads();
    if (tid < DV) {
      for (int t = t0; t < min(t0 + kBlock, n); ++t) {
        const float G = KDA ? 1.0f : gamma[t];
        float pred = G * buf[(2 * (t - t0)) * DV + j], out = G * buf[(2 * (t - t0) + 1) * DV + j];
        for (int s = par[t]; s >= 0; s = par[s]) {
          pred = fmaf(KK[t * rows + s], U[s * DV + j], pred);
          out = fmaf(QK[t * rows + s], U[s * DV + j], out);
        }
        const int64_t at = ((int64_t)(c0 + t) * H + h) * DV + j;
        float x = io_load(gv + at);
        if (p.predicts) x -= pred;
        if (p.use_beta) x *= ld_coherent(p.beta + (int64_t)(c0 + t) * H + h);
        U[t * DV + j] = x;
        if (p.u) p.u[at] = x;
        io_store(static_cast<IT*>(p.o) + at, p.scale * fmaf(QK[t * rows + t], x, out));
      }
    }
    __syncthreads();
  }
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
cudaError_t launch_tree(const TreeParams& p, cudaStream_t stream) {
  const int rows = (p.max_nodes + kBlock - 1) / kBlock * kBlock;
  auto fn = &tree_kernel<ST, IT, DK, DV, KDA>;
  if (prepare_kernel(reinterpret_cast<const void*>(fn), kTreeThreads, tree_smem<DK, DV>(kMaxNodes, KDA)) <= 0)
    return cudaErrorInvalidConfiguration;
  return launch_dependent(fn, p.n_seqs * p.n_v_heads, kTreeThreads, tree_smem<DK, DV>(rows, KDA), stream, p, rows);
}

// ---- commit ------------------------------------------------------------------------------------
// S <- Gamma_leaf S0 + sum over the path's nodes s of (D_leaf,s k_s) u_s^T, rounded once at the
// store.  Bound by the state's bytes (read and written once): one CTA per (sequence, state
// head) reads its whole tile into registers before it looks at the path, so that the loads
// cover the dependent reads of leaf, parents, k and u; a thread's pieces lie in one column
// group, so a path node costs it one piece of u and one factor per row.

constexpr int kCommitThreads = 256;
constexpr int kCommitPieces = 2;  // unpacked at a time

// Eight (q8, BF16) or four (FP32) consecutive values of a row.
template <typename ST>
struct CommitVec {
  static constexpr int kElems = std::is_same<ST, float>::value ? 4 : 8;
};

template <int DK, int DV>
__host__ __device__ constexpr int commit_smem(int rows) {
  return 4 * (rows * (DK + DV) + DK + 2 * DK + 4 * rows + 4);
}

// CTAs of an SM whose raw pieces and working registers fit
template <typename ST, int SIZE>
constexpr int commit_ctas() {
  return SIZE <= 128 * 64 ? 4 : std::is_same<ST, float>::value ? 2 : std::is_same<ST, q8_t>::value ? 3 : 4;
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
__global__ void __launch_bounds__(kCommitThreads, (commit_ctas<ST, DK * DV>())) commit_kernel(const TreeCommitParams p, int rows) {
  constexpr bool Q8 = std::is_same<ST, q8_t>::value;
  constexpr int E = CommitVec<ST>::kElems, PR = DV / E;            // pieces of a row
  constexpr int NP = DK * PR;
  constexpr int ACT = NP < kCommitThreads ? NP : kCommitThreads;   // threads that hold pieces
  constexpr int NPT = NP / ACT, RS = ACT / PR;                     // pieces of a thread, rows between them
  extern __shared__ __align__(16) float sm[];
  float* kc = sm;                 // [path][DK]: D_leaf,s k_s
  float* us = kc + rows * DK;     // [path][DV]
  float* G = us + rows * DV;      // [DK]
  int* src_info = reinterpret_cast<int*>(G + DK);  // [DK] (q8)
  int* dst_info = src_info + DK;
  int* par = dst_info + DK;       // [rows]
  int* path = par + rows;         // [rows]: leaf first
  float* gate = reinterpret_cast<float*>(path + rows);  // [rows]: of the path's nodes
  float* dec = gate + rows;       // [rows]: D_leaf,s (scalar gates)
  int* n_path = reinterpret_cast<int*>(dec + rows);
  griddep_wait();
  const int H = p.n_v_heads;
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int hq = h / (H / p.n_qk_heads);
  const int tid = threadIdx.x;
  const int rs = p.read_slot ? ld_coherent(p.read_slot + b) : b, ws = p.write_slot ? ld_coherent(p.write_slot + b) : b;
  int c0;
  const int n = tree_span(p.cu, p.total, p.max_nodes, b, c0);
  const int leaf = ld_coherent(p.leaf + b);
  if (n < 0) {
    if (tid == 0) report(p.err, span_error(n));
    return;
  }
  const bool r_ok = rs >= 0 && rs < p.src_slots, w_ok = ws >= 0 && ws < p.dst_slots;
  if (!r_ok || !w_ok) {
    if (tid == 0) report(p.err, (r_ok ? 0u : LA_DEVERR_READ_SLOT) | (w_ok ? 0u : LA_DEVERR_WRITE_SLOT));
    return;
  }
  if constexpr (Q8) {
    if (!q8_rows(p.src_mask + h * (DK / 32), DK, p.n_hp, src_info) ||
        !q8_rows(p.dst_mask + h * (DK / 32), DK, p.n_hp, dst_info)) {
      if (tid == 0) report(p.err, LA_DEVERR_Q8_MASK);
      return;
    }
    __syncthreads();
  }
  const int row0 = tid / PR, col = tid % PR;
  TileReader<ST> S;
  S.init(p.src, (int64_t)rs * H + h, DK, DV, p.n_hp, src_info);
  RawPiece<ST> raw[NPT];
  if (tid < ACT) {
#pragma unroll
    for (int k = 0; k < NPT; ++k) raw[k] = raw_piece<ST, DV>(S, row0 + k * RS, col);
  }
  for (int t = tid; t < n; t += kCommitThreads) par[t] = ld_coherent(p.parent + c0 + t);
  __syncthreads();
  if (tid == 0) {
    int m = 0, s = leaf;
    bool ok = s >= -1 && s < n;
    while (ok && s >= 0) {
      path[m++] = s;
      const int up = par[s];
      ok = up >= -1 && up < s;
      s = up;
    }
    *n_path = ok ? m : -1;
  }
  __syncthreads();
  const int m = *n_path;
  if (m < 0) {
    if (tid == 0) report(p.err, LA_DEVERR_TREE);
    return;
  }
  if constexpr (Q8) {
    bool same = m == 0;  // nothing accepted, and the rows of one kind in both pools: the tile as it is
    for (int w = 0; same && w < DK / 32; ++w)
      same = ld_coherent(p.src_mask + h * (DK / 32) + w) == ld_coherent(p.dst_mask + h * (DK / 32) + w);
    if (same) {
      const int64_t bytes = q8_tile_bytes(DK, DV, p.n_hp);
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(p.src) + ((int64_t)rs * H + h) * bytes);
      uint4* d = reinterpret_cast<uint4*>(static_cast<unsigned char*>(p.dst) + ((int64_t)ws * H + h) * bytes);
      for (int i = tid; i < bytes / 16; i += kCommitThreads) d[i] = s[i];
      return;
    }
  }
  const IT* gk = static_cast<const IT*>(p.k);
  if constexpr (KDA) {
    for (int i = tid; i < DK; i += kCommitThreads) {
      float d = 1.0f;
#pragma unroll 4
      for (int a = 0; a < m; ++a) {
        const int64_t t = c0 + path[a];
        kc[a * DK + i] = d * io_load(gk + (t * p.n_qk_heads + hq) * DK + i);
        d *= ld_coherent(p.g + (t * H + h) * DK + i);
      }
      G[i] = d;
    }
  } else if (m > 0) {
    if (p.g) {
      for (int a = tid; a < m; a += kCommitThreads) gate[a] = ld_coherent(p.g + (int64_t)(c0 + path[a]) * H + h);
      __syncthreads();
      for (int a = tid; a <= m; a += kCommitThreads) {
        float d = 1.0f;
        for (int e = 0; e < a; ++e) d *= gate[e];
        if (a < m) dec[a] = d;
        else G[0] = d;
      }
      __syncthreads();
    }
    for (int e = tid; e < m * DK; e += kCommitThreads) {
      const int a = e / DK;
      const float k = io_load(gk + ((int64_t)(c0 + path[a]) * p.n_qk_heads + hq) * DK + e % DK);
      kc[e] = p.g ? dec[a] * k : k;
    }
  }
  for (int e = tid; e < m * (DV / 4); e += kCommitThreads)
    *reinterpret_cast<float4*>(us + 4 * e) = ld_coherent(reinterpret_cast<const float4*>(
        p.u + ((int64_t)(c0 + path[e / (DV / 4)]) * H + h) * DV + e % (DV / 4) * 4));
  __syncthreads();
  if (tid >= ACT) return;
  // CH pieces at a time: few registers, so that four CTAs of an SM have their tiles in flight (two
  // for FP32 128 x 128).  64 sequences x 32 heads BF16: 26.4 us, 33.8 with all pieces unpacked at
  // once and two CTAs.
  constexpr int CH = NPT < kCommitPieces ? NPT : kCommitPieces;
#pragma unroll
  for (int k0 = 0; k0 < NPT; k0 += CH) {
    float x[CH][E];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      unpack_piece(raw[k0 + k], x[k]);
      if (m > 0 && (KDA || p.g)) {
        const float g = G[KDA ? row0 + (k0 + k) * RS : 0];
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] *= g;
      }
    }
#pragma unroll 1
    for (int a = 0; a < m; ++a) {
      float y[E];
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 w = *reinterpret_cast<const float4*>(us + a * DV + col * E + e);
        y[e] = w.x; y[e + 1] = w.y; y[e + 2] = w.z; y[e + 3] = w.w;
      }
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const float f = kc[a * DK + row0 + (k0 + k) * RS];
#pragma unroll
        for (int e = 0; e < E; ++e) x[k][e] = fmaf(f, y[e], x[k][e]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int row = row0 + (k0 + k) * RS;
      if constexpr (Q8) {
        constexpr int NG = DV / 32;
        const int n8 = DK - p.n_hp;
        unsigned char* tile = static_cast<unsigned char*>(p.dst) + ((int64_t)ws * H + h) * q8_tile_bytes(DK, DV, p.n_hp);
        const int e = dst_info[row], idx = e >> 1;
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(x[k][c]));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));  // 32 columns: four threads
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        if (e & 1) {
          reinterpret_cast<uint4*>(tile + n8 * DV + n8 * NG * 4)[idx * PR + col] = StateVec<__nv_bfloat16>::pack(x[k]);
        } else {
          float s, inv;
          q8_scales(amax, s, inv);
          uint32_t words[2];
          q8_pack<8>(x[k], inv, words);
          reinterpret_cast<uint2*>(tile)[idx * PR + col] = make_uint2(words[0], words[1]);
          if ((col & 3) == 0) reinterpret_cast<float*>(tile + n8 * DV)[idx * NG + (col >> 2)] = s;
        }
      } else {
        uint4* tile = reinterpret_cast<uint4*>(static_cast<ST*>(p.dst) + ((int64_t)ws * H + h) * DK * DV);
        __stcs(tile + row * PR + col, StateVec<ST>::pack(x[k]));
      }
    }
  }
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
cudaError_t launch_commit(const TreeCommitParams& p, cudaStream_t stream) {
  auto fn = &commit_kernel<ST, IT, DK, DV, KDA>;
  if (prepare_kernel(reinterpret_cast<const void*>(fn), kCommitThreads, commit_smem<DK, DV>(kMaxNodes)) <= 0)
    return cudaErrorInvalidConfiguration;
  const int rows = (p.max_nodes + 3) / 4 * 4;
  return launch_dependent(fn, p.n_seqs * p.n_v_heads, kCommitThreads, commit_smem<DK, DV>(rows), stream, p, rows);
}

}  // namespace tree
}  // namespace la
