// la_tree_tc.cuh -- verification of drafted trees (la_state_tree) on the fifth-generation
// tensor cores, for the 64 and 128 wide heads.
//
// With K, Q the nodes' rows (n <= 64) and S0 the sequence's state, the dense parts of
//   u_t = b_t (v_t - [S0^T (Gamma_t k_t) + sum_{s above t} (k_t . D_ts k_s) u_s])
//   o_t = scale (S0^T (Gamma_t q_t) + sum_{s above or at t} (q_t . D_ts k_s) u_s)
// are two products of the stacked rows A = [K; Q] (2 R of the M = 128 rows, R = n rounded up to
// 16):  A K^T  [128 x R], whose entries on a node's path, times D_ts, are the pair coefficients,
// and A S0  [128 x d_v].  Rows and columns of absent nodes hold what shared memory held: an MMA
// row depends on its own row of A only, and off-path coefficients are never read, so nothing
// of them (nor a non-finite value of another branch) reaches a result.
//
// Precision: the accumulators are FP32.  BF16 operands are multiplied exactly; an FP32 operand
// (FP32 q and k, an FP32 or q8 state, the kda rows scaled by Gamma) is cut into three BF16
// terms of 8 significand bits each, exact together, and the products of terms i + j <= 2 are
// summed: what is left out is below 2^-23 of the product.
//
// The substitution along the paths stays in FP32 on the CUDA cores, eight nodes at a time: a
// warp per node adds the nodes above of earlier blocks, then one thread per column solves the
// block in registers, then a warp per node adds the block's own part to the output.  It takes
// 2 (path length) d_v FMAs a node whatever the tree; only ancestors are touched.
//
// One CTA of 8 warps per (sequence, state head); the MMA results live in 128 tensor-memory
// columns (the pair product first, the state product over it once it is read) and then go to
// shared memory over the operands, so four CTAs fit an SM for small trees, two at 64 nodes.
#pragma once

#include "la_tree.cuh"
#include "la_umma.cuh"

namespace la {
namespace tree {

constexpr int kTcThreads = 256;
constexpr uint32_t kTcCols = 128;

template <typename ST, typename IT, int DK, int DV, bool KDA>
struct TcCfg {
  static constexpr int TA = (KDA || sizeof(IT) == 4) ? 3 : 1;       // BF16 terms of A
  static constexpr int TS = std::is_same<ST, __nv_bfloat16>::value ? 1 : 3;  // and of S0
  static constexpr int PA = DK / 64, PV = DV / 64;                  // panels of 64 columns
  static constexpr int kRows = TS == 1 ? DK : 64;                   // rows of S0 staged at a time
  static constexpr int kStagesS = DK / kRows;
  static constexpr int kXs = DV + 4;                                // padded row of X (floats)
  __host__ __device__ static constexpr int panel_a(int R) { return 2 * R * 128; }
  __host__ __device__ static constexpr int bytes_a(int R) { return TA * PA * panel_a(R); }
  static constexpr int kTermS = PV * kRows * 128;
  static constexpr int kBytesS = TS * kTermS;
  // operands, under them the results X [2 R][kXs]; an MMA reads 128 rows from any panel of A
  __host__ __device__ static constexpr int region(int R) {
    int x = bytes_a(R) + kBytesS;
    if (KDA && bytes_a(R) + R * DK * 8 > x) x = bytes_a(R) + R * DK * 8;  // K and g in FP32
    if (2 * R * kXs * 4 > x) x = 2 * R * kXs * 4;
    if (bytes_a(R) - panel_a(R) + 16384 > x) x = bytes_a(R) - panel_a(R) + 16384;
    return (x + 15) / 16 * 16;
  }
  __host__ __device__ static constexpr int cs(int R) { return R + 4; }  // padded row of the coefficients
  // + coefficients KK, QK [R][R + 4], path lists [R][R] bytes, 6 arrays of R words, q8 rows, misc
  __host__ __device__ static constexpr int smem(int R) {
    return 1024 + region(R) + 2 * R * (R + 4) * 4 + R * R + 6 * R * 4 + DK * 4 + 32;
  }
};

// x = hi + mid + lo, each a BF16 (by truncation, exact while nothing underflows; a non-finite x
// gives non-finite terms)
__device__ __forceinline__ void split3(float x, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffff0000u;
  const float r = x - __uint_as_float(hi);
  mid = __float_as_uint(r) & 0xffff0000u;
  lo = __float_as_uint(r - __uint_as_float(mid));
}
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

// N (2, 4 or 8) values as three terms at dst, dst + stride, dst + 2 stride
template <int N>
__device__ __forceinline__ void store_terms(unsigned char* dst, int stride, const float* x) {
  uint32_t w[3][N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    uint32_t h0, m0, l0, h1, m1, l1;
    split3(x[2 * e], h0, m0, l0);
    split3(x[2 * e + 1], h1, m1, l1);
    w[0][e] = pack_hi(h0, h1);
    w[1][e] = pack_hi(m0, m1);
    w[2][e] = pack_hi(l0, l1);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if constexpr (N == 8) *reinterpret_cast<uint4*>(dst + i * stride) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    else if constexpr (N == 4) *reinterpret_cast<uint2*>(dst + i * stride) = make_uint2(w[i][0], w[i][1]);
    else *reinterpret_cast<uint32_t*>(dst + i * stride) = w[i][0];
  }
}

template <int VEC>
__device__ __forceinline__ void lds_vec(const float* p, float* x) {
  if constexpr (VEC == 4) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(p);
    x[0] = v.x; x[1] = v.y;
  }
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
__global__ void __launch_bounds__(kTcThreads, 2) tree_tc_kernel(const TreeParams p, int R) {
  using C = TcCfg<ST, IT, DK, DV, KDA>;
  constexpr int TA = C::TA, TS = C::TS, PA = C::PA;
  extern __shared__ __align__(16) unsigned char raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int bytesA = C::bytes_a(R), panelA = C::panel_a(R), cs = C::cs(R);
  unsigned char* smA = sm;
  unsigned char* smS = sm + bytesA;
  float* X = reinterpret_cast<float*>(sm);                       // [2 R][kXs], after the products
  float* KK = reinterpret_cast<float*>(sm + C::region(R));       // [R][cs]
  float* QK = KK + R * cs;
  unsigned char* list = reinterpret_cast<unsigned char*>(QK + R * cs);  // [R][R]: nodes above, of earlier blocks
  float* gate = reinterpret_cast<float*>(list + R * R);          // [R]
  float* gamma = gate + R;
  float* bta = gamma + R;
  int* par = reinterpret_cast<int*>(bta + R);
  int* len = par + R;                                            // entries of the node's list
  int* own = len + R;                                            // nodes above in its own block, a bit each
  int* row_info = own + R;                                       // [DK] (q8)
  uint64_t* bar = reinterpret_cast<uint64_t*>(row_info + DK);
  uint32_t* tm = reinterpret_cast<uint32_t*>(bar + 1);

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
  const int slot = p.read_slot ? __ldg(p.read_slot + b) : b;
  if (slot < 0 || slot >= p.src_slots) {
    if (tid == 0) report(p.err, LA_DEVERR_READ_SLOT);
    return;
  }
  bool bad = false;
  for (int t = tid; t < n; t += kTcThreads) {
    const int pt = __ldg(p.parent + c0 + t);
    bad |= pt < -1 || pt >= t;
    par[t] = pt;
    gate[t] = !KDA && p.g ? __ldg(p.g + (int64_t)(c0 + t) * H + h) : 1.0f;
    bta[t] = p.use_beta ? __ldg(p.beta + (int64_t)(c0 + t) * H + h) : 1.0f;
  }
  // BF16 operands straight to shared memory: the rows of K and Q first, the state behind them
  const IT* gk = static_cast<const IT*>(p.k);
  const IT* gq = static_cast<const IT*>(p.q);
  const int64_t row0 = ((int64_t)c0 * p.n_qk_heads + hq) * DK, row_step = (int64_t)p.n_qk_heads * DK;
  if constexpr (TA == 1) {
    for (int e = tid; e < 2 * n * (DK / 8); e += kTcThreads) {
      const int r = e / (DK / 8), ch = e % (DK / 8), t = r < n ? r : r - n;
      cp_async_16(smA + umma::panel_piece(2 * R, r < n ? t : R + t, ch), (r < n ? gk : gq) + row0 + t * row_step + ch * 8);
    }
    cp_async_commit();
  }
  TileReader<ST> S;
  S.init(p.src, (int64_t)slot * H + h, DK, DV, p.src_n_hp, row_info);
  if constexpr (TS == 1 && !KDA) {
    for (int e = tid; e < DK * (DV / 8); e += kTcThreads)
      cp_async_16(smS + umma::panel_piece(C::kRows, e / (DV / 8), e % (DV / 8)), S.tile + e * 8);
    cp_async_commit();
  }
  bool mask_ok = true;
  if constexpr (std::is_same<ST, q8_t>::value) mask_ok = q8_rows(p.src_mask + h * (DK / 32), DK, p.src_n_hp, row_info);
  if (__syncthreads_or(bad) || !mask_ok) {
    cp_async_wait<0>();
    if (tid == 0) report(p.err, !mask_ok ? LA_DEVERR_Q8_MASK : LA_DEVERR_TREE);
    return;
  }
  if (warp == 7) umma::alloc(tm, kTcCols);
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init_fence();
  }
  // v of a warp's node is read a block ahead
  constexpr int VEC = DV / 32;
  const IT* gv = static_cast<const IT*>(p.v);
  auto value_at = [&](int t) { return ((int64_t)(c0 + t) * H + h) * DV + lane * VEC; };
  float vnext[VEC];
  if (warp < n) load_f32<IT, VEC>(gv + value_at(warp), vnext);

  // lists of the nodes above, and the decays on the way to them
  if (tid < 2 * R) {
    const int t = tid < R ? tid : tid - R;
    if (t < n) {
      float* D = (tid < R ? KK : QK) + t * cs;
      int m = 0, bits = 0;
      float d = 1.0f;
      const int t0 = t & ~7;
      for (int s = t; s >= 0; s = par[s]) {
        if constexpr (!KDA) {
          D[s] = d;
          d *= gate[s];
        }
        if (tid < R && s != t) {
          if (s >= t0) bits |= 1 << (s - t0);
          else list[t * R + m++] = (unsigned char)s;
        }
      }
      if (tid < R) {
        len[t] = m;
        own[t] = bits;
        gamma[t] = d;
      }
    }
  }

  if constexpr (KDA) {
    // K and g in FP32 behind A; a warp per node walks its path with one decay per channel, forms
    // the pair coefficients, and writes its rows of A scaled by Gamma
    constexpr int CH = DK / 32;
    float* Kf = reinterpret_cast<float*>(smS);
    float* Gf = Kf + R * DK;
    for (int e = tid; e < n * (DK / 4); e += kTcThreads) {
      const int t = e / (DK / 4), c = e % (DK / 4) * 4;
      load_f32<IT, 4>(gk + row0 + t * row_step + c, Kf + t * DK + c);
      *reinterpret_cast<float4*>(Gf + t * DK + c) =
          __ldg(reinterpret_cast<const float4*>(p.g + ((int64_t)(c0 + t) * H + h) * DK + c));
    }
    __syncthreads();
    for (int t = warp; t < n; t += kTcThreads / 32) {
      float kt[CH], qt[CH], d[CH];
      load_f32<IT, CH>(gq + row0 + t * row_step + lane * CH, qt);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        kt[c] = Kf[t * DK + lane * CH + c];
        d[c] = 1.0f;
      }
      for (int s = t; s >= 0;) {  // two nodes of the path at a time: their reductions overlap
        const int s2 = par[s];
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const float x = d[c] * Kf[s * DK + lane * CH + c];
          v[0] = fmaf(kt[c], x, v[0]);
          v[1] = fmaf(qt[c], x, v[1]);
          d[c] *= Gf[s * DK + lane * CH + c];
        }
        if (s2 >= 0) {
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const float x = d[c] * Kf[s2 * DK + lane * CH + c];
            v[2] = fmaf(kt[c], x, v[2]);
            v[3] = fmaf(qt[c], x, v[3]);
            d[c] *= Gf[s2 * DK + lane * CH + c];
          }
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], off);
        if (lane == 0) {
          KK[t * cs + s] = v[0];
          QK[t * cs + s] = v[1];
          if (s2 >= 0) {
            KK[t * cs + s2] = v[2];
            QK[t * cs + s2] = v[3];
          }
        }
        s = s2 >= 0 ? par[s2] : -1;
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        kt[c] *= d[c];
        qt[c] *= d[c];
      }
      store_terms<CH>(smA + umma::panel_off(2 * R, t, lane * CH), PA * panelA, kt);
      store_terms<CH>(smA + umma::panel_off(2 * R, R + t, lane * CH), PA * panelA, qt);
    }
    if constexpr (TS == 1) {  // the state goes over K and g
      __syncthreads();
      for (int e = tid; e < DK * (DV / 8); e += kTcThreads)
        cp_async_16(smS + umma::panel_piece(C::kRows, e / (DV / 8), e % (DV / 8)), S.tile + e * 8);
      cp_async_commit();
    }
  } else if constexpr (TA == 3) {
    for (int e = tid; e < 2 * n * (DK / 8); e += kTcThreads) {
      const int r = e / (DK / 8), ch = e % (DK / 8), t = r < n ? r : r - n;
      float x[8];
      load_f32<IT, 8>((r < n ? gk : gq) + row0 + t * row_step + ch * 8, x);
      store_terms<8>(smA + umma::panel_piece(2 * R, r < n ? t : R + t, ch), PA * panelA, x);
    }
  } else {
    cp_async_wait<TS == 1 ? 1 : 0>();
  }
  umma::fence_smem();
  umma::fence_before();
  __syncthreads();
  umma::fence_after();
  const uint32_t tmem = *tm;
  const uint64_t dA = umma::sdesc(smem_addr(smA), 16, 1024);
  const uint64_t dS = umma::sdesc(smem_addr(smS), C::kRows * 128, 1024);
  bool ok = true;
  uint32_t phase = 0;
  auto done = [&] {  // every MMA issued so far
    ok &= mbar_wait(bar, phase & 1u);
    ++phase;
    umma::fence_after();
  };
  const uint32_t quarter = umma::taddr(tmem, (warp & 3) * 32, 0);
  const int row = (warp & 3) * 32 + lane;
  const bool mine = (warp & 3) * 32 < 2 * R;  // the warp's lanes hold rows of A

  if constexpr (!KDA) {
    if (tid == 0) {
      const uint32_t id = umma::idesc_bf16(128, R, false, false);
      uint32_t acc = 0;
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TA - i; ++j)
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t ko = (kk >> 2) * panelA + (kk & 3) * 32;
            umma::mma(tmem, umma::sdesc_add(dA, i * PA * panelA + ko), umma::sdesc_add(dA, j * PA * panelA + ko), id, acc);
            acc = 1;
          }
      umma::commit(bar);
    }
    done();
    if (mine)
      for (int c = (warp >> 2) * 16; c < R; c += 32) {
        uint32_t w[16];
        umma::ld16(quarter + c, w);
        umma::wait_ld();
        if (row < 2 * R) {
          float4* D = reinterpret_cast<float4*>((row < R ? KK + row * cs : QK + (row - R) * cs) + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4 x = D[e];
            x.x *= __uint_as_float(w[4 * e]);
            x.y *= __uint_as_float(w[4 * e + 1]);
            x.z *= __uint_as_float(w[4 * e + 2]);
            x.w *= __uint_as_float(w[4 * e + 3]);
            D[e] = x;
          }
        }
      }
  }
  // the state product, over the pair product's columns
  uint32_t acc = 0;
  for (int st = 0; st < C::kStagesS; ++st) {
    if constexpr (TS == 1) {
      cp_async_wait<0>();
    } else {
      constexpr int kPieces = C::kRows * (DV / 8) / kTcThreads;
      float x[kPieces][8];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int at = tid + e * kTcThreads;
        state_piece<8, ST, DV>(S, st * C::kRows + at / (DV / 8), at % (DV / 8), x[e]);
      }
      if (st > 0) done();  // the stage's buffer is free
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int at = tid + e * kTcThreads;
        store_terms<8>(smS + umma::panel_piece(C::kRows, at / (DV / 8), at % (DV / 8)), C::kTermS, x[e]);
      }
    }
    umma::fence_smem();
    umma::fence_before();
    __syncthreads();
    if (tid == 0) {
      umma::fence_after();
      constexpr uint32_t id = umma::idesc_bf16(128, DV, false, true);
#pragma unroll
      for (int i = 0; i < TA; ++i)
#pragma unroll
        for (int j = 0; j < TS; ++j)
          if (i + j <= 2)
#pragma unroll
            for (int kk = 0; kk < C::kRows / 16; ++kk) {
              const int ka = st * (C::kRows / 16) + kk;
              umma::mma(tmem, umma::sdesc_add(dA, i * PA * panelA + (ka >> 2) * panelA + (ka & 3) * 32),
                        umma::sdesc_add(dS, j * C::kTermS + kk * 2048), id, acc);
              acc = 1;
            }
      umma::commit(bar);
    }
  }
  done();
  // the results over the operands; a scalar gate's Gamma is a factor of the row
  if (mine)
    for (int c = (warp >> 2) * 16; c < DV; c += 32) {
      uint32_t w[16];
      umma::ld16(quarter + c, w);
      umma::wait_ld();
      if (row < 2 * R) {
        float G = 1.0f;
        if (!KDA) G = gamma[row < R ? row : row - R];
        float4* D = reinterpret_cast<float4*>(X + row * C::kXs + c);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          D[e] = make_float4(G * __uint_as_float(w[4 * e]), G * __uint_as_float(w[4 * e + 1]),
                             G * __uint_as_float(w[4 * e + 2]), G * __uint_as_float(w[4 * e + 3]));
      }
    }
  umma::fence_before();
  const bool failed = __syncthreads_or(!ok);
  if (warp == 7) {
    umma::fence_after();
    umma::dealloc(tmem, kTcCols);
  }
  if (failed) {
    if (tid == 0) report(p.err, LA_DEVERR_TIMEOUT);
    return;
  }

  for (int t0 = 0; t0 < n; t0 += 8) {
    const int t = t0 + warp;
    float out[VEC];
    if (t < n) {
      float pred[VEC];
      lds_vec<VEC>(X + t * C::kXs + lane * VEC, pred);
      lds_vec<VEC>(X + (R + t) * C::kXs + lane * VEC, out);
      const float* KKr = KK + t * cs;
      const float* QKr = QK + t * cs;
      const int m = len[t];
      for (int i = 0; i < m; i += 4) {
        const uint32_t four = *reinterpret_cast<const uint32_t*>(list + t * R + i);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (i + e < m) {
            const int s = (four >> (8 * e)) & 255;
            float x[VEC];
            lds_vec<VEC>(X + s * C::kXs + lane * VEC, x);
            const float kk = KKr[s], qk = QKr[s];
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
              pred[c] = fmaf(kk, x[c], pred[c]);
              out[c] = fmaf(qk, x[c], out[c]);
            }
          }
      }
#pragma unroll
      for (int c = 0; c < VEC; ++c) X[t * C::kXs + lane * VEC + c] = p.predicts ? vnext[c] - pred[c] : vnext[c];
    }
    if (t + 8 < n) load_f32<IT, VEC>(gv + value_at(t + 8), vnext);
    __syncthreads();
    if (p.predicts) {
      if (tid < DV) {
        float x[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          if (t0 + r < n) {
            float y = X[(t0 + r) * C::kXs + tid];
            const int bits = own[t0 + r];
            const float4 a = *reinterpret_cast<const float4*>(KK + (t0 + r) * cs + t0);
            const float4 z = *reinterpret_cast<const float4*>(KK + (t0 + r) * cs + t0 + 4);
            const float coef[8] = {a.x, a.y, a.z, a.w, z.x, z.y, z.z, z.w};
#pragma unroll
            for (int s = 0; s < r; ++s)
              if (bits >> s & 1) y = fmaf(-coef[s], x[s], y);
            x[r] = bta[t0 + r] * y;
            X[(t0 + r) * C::kXs + tid] = x[r];
          }
        }
      }
      __syncthreads();
    }
    if (t < n) {
      const float* QKr = QK + t * cs;
      for (int bits = own[t]; bits; bits &= bits - 1) {
        const int s = t0 + __ffs(bits) - 1;
        float x[VEC];
        lds_vec<VEC>(X + s * C::kXs + lane * VEC, x);
        const float qk = QKr[s];
#pragma unroll
        for (int c = 0; c < VEC; ++c) out[c] = fmaf(qk, x[c], out[c]);
      }
      float x[VEC];
      lds_vec<VEC>(X + t * C::kXs + lane * VEC, x);
      const float qk = QKr[t];
#pragma unroll
      for (int c = 0; c < VEC; ++c) out[c] = p.scale * fmaf(qk, x[c], out[c]);
      const int64_t at = value_at(t);
      store_f32<IT, VEC>(static_cast<IT*>(p.o) + at, out);
      if (p.u) store_f32<float, VEC>(p.u + at, x);
    }
  }
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t stream) {
  using C = TcCfg<ST, IT, DK, DV, KDA>;
  const int R = (p.max_nodes + 15) / 16 * 16;
  auto fn = &tree_tc_kernel<ST, IT, DK, DV, KDA>;
  static_assert(C::smem(kMaxNodes) <= 227 * 1024, "shared memory");
  if (prepare_kernel(reinterpret_cast<const void*>(fn), kTcThreads, C::smem(kMaxNodes)) <= 0)
    return cudaErrorInvalidConfiguration;
  fn<<<p.n_seqs * p.n_v_heads, kTcThreads, C::smem(R), stream>>>(p, R);
  return cudaGetLastError();
}

}  // namespace tree
}  // namespace la
