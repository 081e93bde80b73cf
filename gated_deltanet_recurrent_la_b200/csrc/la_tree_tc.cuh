// la_tree_tc.cuh -- verification of drafted trees (la_state_tree) on the fifth-generation
// tensor cores, for the 64 and 128 wide heads.
//
// With K, Q the nodes' rows (n <= 64) and S0 the sequence's state, the dense parts of
//   u_t = b_t (v_t - [S0^T (Gamma_t k_t) + sum_{s above t} (k_t . D_ts k_s) u_s])
//   o_t = scale (S0^T (Gamma_t q_t) + sum_{s above or at t} (q_t . D_ts k_s) u_s)
// are two products with the stacked rows A = [K; Q] (2 R rows, R = n rounded up to 16):
//   A K^T     [128 x R], a node per tensor-memory lane: the pair coefficients, of which a lane
//             keeps those on its node's path, times D_ts, packed along the path;
//   S0^T A^T  [128 x 2 R], a column of d_v per lane.
// Rows and columns of absent nodes hold what shared memory held: they reach only results that
// nothing reads, and off-path coefficients are dropped, so a non-finite value of another branch
// reaches nothing either.
//
// Precision: the accumulators are FP32.  BF16 operands are multiplied exactly; an FP32 operand
// (FP32 q and k, an FP32 or q8 state, the kda rows scaled by Gamma) is cut into three BF16
// terms of 8 significand bits each, exact together, and the products of terms i + j <= 2 are
// summed: what is left out is below 2^-23 of the product.  An MMA truncates its sum to the FP32
// accumulator's last place, so the number of MMAs that add to a full-sized accumulator counts:
// smaller products come first (A K^T) or go to an accumulator of their own (S0^T A^T, whose
// rows come in stages), which leaves the d_k / 16 of the leading terms.
//
// The substitution along the paths is FP32 on the CUDA cores with one thread per column of d_v:
// it takes S0^T k_t and S0^T q_t from its own tensor-memory lane and keeps its column of V, then
// U, in shared memory (over the operands), so the nodes follow one another without a barrier;
// only ancestors are touched, two FMAs for each.  Two nodes at a time: a warp's instructions
// come about 5 cycles apart when each waits for the one before.  Paths are padded to fours with
// entries that point to a row of zeros, so the loop has no predicates, and it is kept rolled:
// unrolled over eight nodes it ran out of the instruction caches (570 cycles a node).
//
// One CTA of 4 warps per (sequence, state head), 8 where operands are cut into terms (the cutting
// and the kda decays use them).  Bound by latency within a CTA (loads, MMA, path), which the
// other CTAs of the SM cover: four fit for trees of up to 32 nodes; above that a BF16 state comes
// in two halves of its rows, so that three fit.
#pragma once

#include "la_tree.cuh"
#include "la_umma.cuh"

namespace la {
namespace tree {

template <typename ST, typename IT, int DK, int DV, bool KDA>
struct TcCfg {
  static constexpr int TA = (KDA || sizeof(IT) == 4) ? 3 : 1;       // BF16 terms of A
  static constexpr int TS = std::is_same<ST, __nv_bfloat16>::value ? 1 : 3;  // and of S0
  static constexpr int kThreads = TA == 1 && TS == 1 ? 128 : 256;
  static constexpr int kMinCtas = kThreads == 128 ? 4 : 2;          // 128 registers a thread
  static constexpr int PA = DK / 64;                                // panels of 64 columns
  __host__ __device__ static constexpr int rows_s(int R) { return TS == 1 && R <= 32 ? DK : 64; }  // of S0, at a time
  __host__ __device__ static constexpr int panel_s(int R) { return rows_s(R) * 128; }
  __host__ __device__ static constexpr int term_s(int R) { return DV / 64 * panel_s(R); }
  __host__ __device__ static constexpr int panel_a(int R) { return 2 * R * 128; }
  __host__ __device__ static constexpr int bytes_a(int R) { return TA * PA * panel_a(R); }
  // operands; over them U [R][DV] and a row of zeros.  A K^T reads 128 rows from any panel of A,
  // S0^T A^T two panels of 64 columns from any term of S0.
  __host__ __device__ static constexpr int region(int R) {
    int x = bytes_a(R) + (TS - 1) * term_s(R) + 2 * panel_s(R);
    if (KDA && bytes_a(R) + R * DK * 8 > x) x = bytes_a(R) + R * DK * 8;  // K and g in FP32
    if ((R + 1) * DV * 4 > x) x = (R + 1) * DV * 4;
    if (bytes_a(R) - panel_a(R) + 16384 > x) x = bytes_a(R) - panel_a(R) + 16384;
    return (x + 15) / 16 * 16;
  }
  // paths: entries (at most t for node t, rounded up to fours, four for node 0) as two
  // coefficients and a place (the count is a multiple of 8)
  __host__ __device__ static constexpr int entries(int R) { return R * (R + 2) / 2 + 8; }
  static constexpr int kRowInfo = std::is_same<ST, q8_t>::value ? DK : 0;
  static constexpr int smem(int R) { return region(R) + entries(R) * 9 + R * 64 + R * 8 + kRowInfo * 4 + 32; }
  // tensor memory: S0^T A^T [2 R], before it A K^T [R]; with terms, behind it the products of the
  // smaller ones [2 R]
  static constexpr bool kTerms = TA * TS > 1;
  __host__ __device__ static constexpr uint32_t cols(int R) {
    const int n = kTerms ? 4 * R : 2 * R;
    return n <= 32 ? 32 : n <= 64 ? 64 : n <= 128 ? 128 : 256;
  }
};
// m entries rounded up to fours, at least one four; the first entry kept for node t
__device__ __forceinline__ int path_size(int m) { return max(4, (m + 3) & ~3); }
__device__ __forceinline__ int path_at(int t) {
  const int a = (t + 3) >> 2;  // of the nodes 1 .. t - 1, four each have 1, 2, .. fours
  return t == 0 ? 0 : 4 + 8 * a * (a - 1) + 4 * a * (t - 4 * a + 3);
}

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

// The thread sleeps in the test itself, up to 20 us.
__device__ __forceinline__ bool tree_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return done != 0;
}
// Waits for a phase of `bar`, without reading a timer where it comes soon.  False when the time
// limit ran out: then it has waited as long once more, so that the products the phase stands for
// have ended before their operands and their tensor memory are given up.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (tree_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  bool late = false;
  for (uint32_t polls = 1; polls < kWaitMaxPolls; ++polls) {
    if (tree_try_wait(bar, parity)) return !late;
    const uint64_t t = global_timer_ns() - t0;
    late = t > limit_ns;
    if (t > 2 * limit_ns) return false;
  }
  return false;
}

// What the solve reads of a node: one record, so that its loads need one address.
struct NodeRecord {
  float gamma, b, self;   // product of the path's gates, write strength, q . k
  int path;               // length | (number of the first four entries) << 16 | (more than four) << 31
  uint32_t at[4];         // the nearest four: byte offset of their row of U,
  float coef[2][4];       // and their coefficients for u and o
};

// two columns of this thread's tensor-memory lane (wait_ld before they are used)
__device__ __forceinline__ void tmem_ld2(uint32_t taddr, uint32_t& a, uint32_t& b) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(a), "=r"(b) : "r"(taddr) : "memory");
}

// if (bit): x at shared address `at`.  Predicated, with the addresses formed outside: as branches
// the 64 columns of a row took 4 times as long.
__device__ __forceinline__ void store_if(uint32_t bit, uint32_t at, float x) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p st.shared.f32 [%1], %2;\n\t}" ::"r"(bit), "r"(at), "f"(x)
               : "memory");
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
__global__ void __launch_bounds__((TcCfg<ST, IT, DK, DV, KDA>::kThreads), (TcCfg<ST, IT, DK, DV, KDA>::kMinCtas))
    tree_tc_kernel(const TreeParams p, int R) {
  using C = TcCfg<ST, IT, DK, DV, KDA>;
  constexpr int TA = C::TA, TS = C::TS, PA = C::PA, NT = C::kThreads;
  // (not a rounded pointer: the compiler has to see that it is shared memory)
  extern __shared__ __align__(1024) unsigned char tc_smem[];
  unsigned char* sm = tc_smem;
  const int bytesA = C::bytes_a(R), panelA = C::panel_a(R);
  unsigned char* smA = sm;
  unsigned char* smS = sm + bytesA;
  float* U = reinterpret_cast<float*>(sm);                           // [R][DV], after the products
  const int plane = C::entries(R);
  float* coef = reinterpret_cast<float*>(sm + C::region(R));         // [2][entries]: of u, of o; nearest node first
  NodeRecord* node = reinterpret_cast<NodeRecord*>(coef + 2 * plane);  // [R]
  unsigned char* place = reinterpret_cast<unsigned char*>(node + R);  // entries: the node above
  float* gate = reinterpret_cast<float*>(place + C::entries(R));     // [R]
  int* par = reinterpret_cast<int*>(gate + R);                       // [R]
  int* row_info = par + R;                                           // [DK] (q8)
  uint64_t* bar = reinterpret_cast<uint64_t*>(row_info + C::kRowInfo);  // A K^T, S0^T A^T
  uint32_t* tm = reinterpret_cast<uint32_t*>(bar + 2);

  griddep_wait();
  const int H = p.n_v_heads;
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int hq = h / (H / p.n_qk_heads);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slot = p.read_slot ? ld_coherent(p.read_slot + b) : b;
  int c0;
  const int n = tree_span(p.cu, p.total, p.max_nodes, b, c0);
  if (n < 0) {
    if (tid == 0) report(p.err, span_error(n));
    return;
  }
  if (n == 0) return;
  if (slot < 0 || slot >= p.src_slots) {
    if (tid == 0) report(p.err, LA_DEVERR_READ_SLOT);
    return;
  }
  if (smem_addr(sm) & 1023u) {  // the panels' alignment (the declaration asks for it)
    if (tid == 0) report(p.err, LA_DEVERR_TIMEOUT);
    return;
  }
  int my_par = -1;
  float my_gate = 1.0f, my_beta = 1.0f;
  if (tid < n) {
    my_par = ld_coherent(p.parent + c0 + tid);
    if (!KDA && p.g) my_gate = ld_coherent(p.g + (int64_t)(c0 + tid) * H + h);
    if (p.use_beta) my_beta = ld_coherent(p.beta + (int64_t)(c0 + tid) * H + h);
  }
  // BF16 operands straight to shared memory: the rows of K and Q first, the state behind them
  const IT* gk = static_cast<const IT*>(p.k);
  const IT* gq = static_cast<const IT*>(p.q);
  const int64_t row0 = ((int64_t)c0 * p.n_qk_heads + hq) * DK, row_step = (int64_t)p.n_qk_heads * DK;
  if constexpr (TA == 1) {
    // (a thread's rows lie a multiple of 8 apart: the swizzle is the same in all of them)
    constexpr int RS = NT / (DK / 8);
    const int t0 = tid / (DK / 8), ch = tid % (DK / 8);
    unsigned char* dst = smA + umma::panel_piece(2 * R, t0, ch);
    const IT* fk = gk + row0 + t0 * row_step + ch * 8;
    const IT* fq = gq + row0 + t0 * row_step + ch * 8;
    for (int t = t0; t < n; t += RS, dst += RS * 128, fk += RS * row_step, fq += RS * row_step) {
      cp_async_16(dst, fk);
      cp_async_16(dst + R * 128, fq);
    }
    cp_async_commit();
  }
  TileReader<ST> S;
  S.init(p.src, (int64_t)slot * H + h, DK, DV, p.src_n_hp, row_info);
  const int rows = C::rows_s(R), panelS = C::panel_s(R), termS = C::term_s(R), stages = DK / rows;
  auto state_async = [&](int st) {
    if constexpr (TS == 1) {
      constexpr int RS = NT / (DV / 8);
      unsigned char* dst = smS + umma::panel_piece(rows, tid / (DV / 8), tid % (DV / 8));
      const ST* src = S.tile + st * rows * DV + tid * 8;
#pragma unroll 8
      for (int i = 0; i < rows / RS; ++i) cp_async_16(dst + i * RS * 128, src + i * RS * DV);
      cp_async_commit();
    }
  };
  if constexpr (!KDA) state_async(0);
  bool mask_ok = true;
  if constexpr (std::is_same<ST, q8_t>::value) mask_ok = q8_rows(p.src_mask + h * (DK / 32), DK, p.src_n_hp, row_info);
  if (tid < n) {
    par[tid] = my_par;
    gate[tid] = my_gate;
    node[tid].gamma = 1.0f;
    node[tid].b = my_beta;
  }
  if (__syncthreads_or(tid < n && (my_par < -1 || my_par >= tid)) || !mask_ok) {
    cp_async_wait<0>();
    if (tid == 0) report(p.err, !mask_ok ? LA_DEVERR_Q8_MASK : LA_DEVERR_TREE);
    return;
  }
  if (warp == NT / 32 - 1) umma::alloc(tm, C::cols(R));
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 1, 1);
    mbar_init_fence();
  }
  if (TS == 1 && stages > 1 && tid == 0)  // the second half on its way to L2
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(S.tile + rows * DV), "r"((DK - rows) * DV * 2));
  // v waits in registers until the products are done with the operands
  constexpr int PV = DV * (int)sizeof(IT) / 16, VE = 16 / (int)sizeof(IT);  // pieces of a row of v, values of a piece
  constexpr int VN = kMaxNodes * PV / NT;
  const int64_t base_v = ((int64_t)c0 * H + h) * DV, step_v = (int64_t)H * DV;
  uint4 vr[VN];
#pragma unroll
  for (int e = 0; e < VN; ++e) {
    const int at = tid + e * NT;
    if (at < n * PV)
      vr[e] = ld_coherent(reinterpret_cast<const uint4*>(static_cast<const IT*>(p.v) + base_v + at / PV * step_v) + at % PV);
  }

  // the nodes above; thread t for the coefficients of u, R + t for those of o
  uint64_t above = 0;
  uint32_t four = 0x01010101u * R;  // the nearest four, R where there are fewer
  const bool is_q = tid >= R;
  const int t_own = is_q ? tid - R : tid;
  const bool own = tid < (KDA ? R : 2 * R) && t_own < n;  // (kda: the walk forms both)
  if (own) {
    uint32_t* words = reinterpret_cast<uint32_t*>(place + path_at(t_own));
    uint32_t word = 0x01010101u * R;
    int i = 0;
    for (int s = par[t_own]; s >= 0; s = par[s]) {
      above |= 1ull << s;
      word = word ^ (uint32_t)(R ^ s) << (8 * (i & 3));
      if ((++i & 3) == 0) {
        if (i == 4) four = word;
        if (!is_q) *words++ = word;
        word = 0x01010101u * R;
      }
    }
    if (i < 4) four = word;
    if (!is_q && ((i & 3) || i == 0)) *words = word;
  }
  // length and offsets of a record
  auto describe = [&](int t, int m, uint32_t w) {
    node[t].path = m | path_at(t) << 14 | (m > 4 ? INT32_MIN : 0);
    *reinterpret_cast<uint4*>(node[t].at) =
        make_uint4((w & 255u) * (DV * 4), (w >> 8 & 255u) * (DV * 4), (w >> 16 & 255u) * (DV * 4), (w >> 24) * (DV * 4));
  };
  if (own && !is_q) describe(t_own, __popcll(above), four);
  if (tid == 0 && (n & 1)) {  // the node behind an odd last one: no path
    describe(n, 0, 0x01010101u * R);
#pragma unroll
    for (int e = 0; e < 8; ++e) node[n].coef[e >> 2][e & 3] = 0.0f;
  }

  if constexpr (KDA) {
    // K and g in FP32 behind A; a warp per node walks its path with one decay per channel, forms
    // the pair coefficients, and writes its rows of A scaled by Gamma
    constexpr int CH = DK / 32;
    float* Kf = reinterpret_cast<float*>(smS);
    float* Gf = Kf + R * DK;
    for (int e = tid; e < n * (DK / 4); e += NT) {
      const int t = e / (DK / 4), c = e % (DK / 4) * 4;
      load_f32<IT, 4>(gk + row0 + t * row_step + c, Kf + t * DK + c);
      *reinterpret_cast<float4*>(Gf + t * DK + c) =
          ld_coherent(reinterpret_cast<const float4*>(p.g + ((int64_t)(c0 + t) * H + h) * DK + c));
    }
    __syncthreads();
    for (int t = warp; t < n; t += NT / 32) {
      float kt[CH], qt[CH], d[CH], self = 0.0f;
      load_f32<IT, CH>(gq + row0 + t * row_step + lane * CH, qt);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        kt[c] = Kf[t * DK + lane * CH + c];
        d[c] = Gf[t * DK + lane * CH + c];
        self = fmaf(qt[c], kt[c], self);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) self += __shfl_xor_sync(0xffffffffu, self, off);
      if (lane == 0) node[t].self = self;
      const int first = path_at(t), m = node[t].path & 255;
      int i = 0;
      do {  // four nodes of the path at a time (at least once: the record's coefficients)
        const uint32_t w = *reinterpret_cast<const uint32_t*>(place + first + i);
        float v[8];  // (k_t, q_t) . D k of the four
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = v[2 * e + 1] = 0.0f;
          if (i + e < m) {
            const int s = w >> (8 * e) & 255;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              const float x = d[c] * Kf[s * DK + lane * CH + c];
              v[2 * e] = fmaf(kt[c], x, v[2 * e]);
              v[2 * e + 1] = fmaf(qt[c], x, v[2 * e + 1]);
              d[c] *= Gf[s * DK + lane * CH + c];
            }
          }
        }
        // eight sums over the lanes with nine shuffles: each step hands half of the values over
#pragma unroll
        for (int half = 4, off = 16; half >= 1; half >>= 1, off >>= 1) {
          const bool up = lane & off;
#pragma unroll
          for (int e = 0; e < half; ++e) {
            const float give = up ? v[e] : v[e + half], keep = up ? v[e + half] : v[e];
            v[e] = keep + __shfl_xor_sync(0xffffffffu, give, off);
          }
        }
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 2);
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], 1);
        if ((lane & 3) == 0) {  // value lane / 4: entry lane / 8, of u or of o
          const int e = lane >> 3, o = lane >> 2 & 1;
          if (i == 0) node[t].coef[o][e] = v[0];
          else coef[o * plane + first + i + e] = v[0];
        }
        i += 4;
      } while (i < m);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        kt[c] *= d[c];
        qt[c] *= d[c];
      }
      store_terms<CH>(smA + umma::panel_off(2 * R, t, lane * CH), PA * panelA, kt);
      store_terms<CH>(smA + umma::panel_off(2 * R, R + t, lane * CH), PA * panelA, qt);
    }
    __syncthreads();  // the state goes over K and g
    state_async(0);
  } else if constexpr (TA == 3) {
    for (int e = tid; e < 2 * n * (DK / 8); e += NT) {
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
  const uint64_t dS = umma::sdesc(smem_addr(smS), panelS, 1024);
  bool ok = true;

  if constexpr (!KDA) {
    if (tid == 0) {
      const uint32_t id = umma::idesc_bf16(128, R, false, false);
      uint32_t acc = 0;
#pragma unroll
      for (int ij = TA - 1; ij >= 0; --ij)  // the smallest first
#pragma unroll
        for (int i = 0; i <= ij; ++i)
#pragma unroll
          for (int kk = 0; kk < DK / 16; ++kk) {
            const uint32_t ko = (kk >> 2) * panelA + (kk & 3) * 32;
            umma::mma(tmem, umma::sdesc_add(dA, i * PA * panelA + ko), umma::sdesc_add(dA, (ij - i) * PA * panelA + ko), id, acc);
            acc = 1;
          }
      umma::commit(bar);
    }
    ok = tree_wait(bar, 0, p.wait_ns);
    umma::fence_after();
    if (warp < 4 && warp * 32 < 2 * R) {
      // nearest first: the places fall as s rises
      uint32_t at = smem_addr(coef + is_q * plane + path_at(t_own) + __popcll(above));
      const uint32_t at_self = smem_addr(&node[t_own].self);
#pragma unroll 1
      for (int c = 0; c < R; c += 16) {
        const uint32_t bits = own ? (uint32_t)(above >> c) & 0xffffu : 0u;
        const uint32_t diag = own && is_q && t_own >> 4 == c >> 4 ? 1u << (t_own & 15) : 0u;
        if (!__any_sync(0xffffffffu, bits | diag)) continue;
        uint32_t w[16];
        umma::ld16(umma::taddr(tmem, warp * 32, c), w);
        umma::wait_ld();
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const uint32_t bit = bits >> e & 1u;
          at -= 4 * bit;
          store_if(bit, at, __uint_as_float(w[e]));
        }
        if (__any_sync(0xffffffffu, diag)) {
#pragma unroll
          for (int e = 0; e < 16; ++e) store_if(diag >> e & 1u, at_self, __uint_as_float(w[e]));
        }
      }
    }
    umma::fence_before();
  }
  // S0^T A^T, over the columns of A K^T
  auto issue = [&](int st) {
    umma::fence_after();
    const uint32_t id = umma::idesc_bf16(128, 2 * R, true, false);
    uint32_t small = st;  // whether something is in their accumulator
#pragma unroll
    for (int ij = 2; ij >= 0; --ij)
#pragma unroll
      for (int i = 0; i <= ij; ++i) {
        const int j = ij - i;
        if (i < TA && j < TS) {
          for (int kk = 0; kk < rows / 16; ++kk) {
            const int ka = st * (rows / 16) + kk;
            umma::mma(ij ? tmem + 2 * R : tmem, umma::sdesc_add(dS, j * termS + kk * 2048),
                      umma::sdesc_add(dA, (i * PA + (ka >> 2)) * panelA + (ka & 3) * 32), id, ij ? small : st | kk);
            if (ij) small = 1;
          }
        }
      }
    umma::commit(bar + 1);
  };
  // (a thread whose wait ran out leaves the operands alone and issues nothing more; all of them learn
  // of it at the last barrier, and nothing of the tile is written)
  for (int st = 0; st < stages; ++st) {
    if constexpr (TS == 1) {
      if (st > 0) {  // the buffer is free
        if (ok) ok = tree_wait(bar + 1, (st - 1) & 1, p.wait_ns);
        if (ok) state_async(st);
      }
    } else {
      constexpr int kPieces = 64 * (DV / 8) / NT;
      float x[kPieces][8];
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        const int at = tid + e * NT;
        state_eight<ST, DV>(S, st * 64 + at / (DV / 8), at % (DV / 8), x[e]);
      }
      if (st > 0 && ok) ok = tree_wait(bar + 1, (st - 1) & 1, p.wait_ns);
#pragma unroll
      for (int e = 0; e < kPieces; ++e) {
        if (!ok) break;
        const int at = tid + e * NT;
        store_terms<8>(smS + umma::panel_piece(64, at / (DV / 8), at % (DV / 8)), termS, x[e]);
      }
    }
    if (!KDA && st == stages - 1 && own) {  // the decays along the path, while the state is on its way
      float d = gate[t_own];
      const int m = __popcll(above), first = path_at(t_own);
      float4* c4 = reinterpret_cast<float4*>(coef + is_q * plane + first);
      auto scale4 = [&](float4 c, uint32_t w, int left) {  // the gates of absent entries are not taken
        const float g0 = gate[w & 255u], g1 = gate[w >> 8 & 255u], g2 = gate[w >> 16 & 255u], g3 = gate[w >> 24];
        c.x = left > 0 ? c.x * d : 0.0f;
        d = left > 0 ? d * g0 : d;
        c.y = left > 1 ? c.y * d : 0.0f;
        d = left > 1 ? d * g1 : d;
        c.z = left > 2 ? c.z * d : 0.0f;
        d = left > 2 ? d * g2 : d;
        c.w = left > 3 ? c.w * d : 0.0f;
        d = left > 3 ? d * g3 : d;
        return c;
      };
      *reinterpret_cast<float4*>(node[t_own].coef[is_q]) = scale4(c4[0], four, m);
      for (int i = 4; i < m; i += 4)
        c4[i >> 2] = scale4(c4[i >> 2], *reinterpret_cast<const uint32_t*>(place + first + i), m - i);
      if (!is_q) node[t_own].gamma = d;
    }
    if constexpr (TS == 1) cp_async_wait<0>();
    umma::fence_smem();
    __syncthreads();
    if (tid == 0 && ok && (st > 0 || blockIdx.x != p.withhold)) issue(st);
  }

  // v in FP32 where U will be
  if (ok) ok = tree_wait(bar + 1, (stages - 1) & 1, p.wait_ns);
  umma::fence_after();
#pragma unroll
  for (int e = 0; e < VN; ++e) {
    const int at = tid + e * NT;
    if (at < n * PV) {
      float x[VE];
      StateVec<IT>::unpack(vr[e], x);
#pragma unroll
      for (int c = 0; c < VE; c += 4)
        *reinterpret_cast<float4*>(U + at / PV * DV + at % PV * VE + c) = make_float4(x[c], x[c + 1], x[c + 2], x[c + 3]);
    }
  }
  if (tid < DV) U[R * DV + tid] = 0.0f;
  const bool failed = __syncthreads_or(!ok);

  if (!failed && tid < DV) {
    uint32_t mine_k = umma::taddr(tmem, warp * 32, 0), mine_q = mine_k + R;
    const float4* entry_u = reinterpret_cast<const float4*>(coef);           // four entries each
    const float4* entry_o = reinterpret_cast<const float4*>(coef + plane);
    const uint32_t* places = reinterpret_cast<const uint32_t*>(place);
    const unsigned char* rows_u = reinterpret_cast<const unsigned char*>(U + tid);
    float* mine = U + tid;
    IT* go = static_cast<IT*>(p.o) + base_v + tid;
    float* gu = p.u + base_v + tid;
    uint32_t off = 0;
    const uint32_t step = (uint32_t)step_v;  // (the host has checked that 64 rows of all heads fit 32 bits)
    const bool store_u = p.u != nullptr;
    const NodeRecord* rec = node;
    uint32_t k0, k1, q0, q1, kl0 = 0, kl1 = 0, ql0 = 0, ql1 = 0;  // (l: of the smaller terms)
    auto products = [&] {
      tmem_ld2(mine_k, k0, k1);
      tmem_ld2(mine_q, q0, q1);
      if constexpr (C::kTerms) {
        tmem_ld2(mine_k + 2 * R, kl0, kl1);
        tmem_ld2(mine_q + 2 * R, ql0, ql1);
      }
    };
    products();
    auto row = [&](uint32_t at) { return *reinterpret_cast<const float*>(rows_u + at); };
    auto further = [&](int path, float& pred, float& out) {
      const int m = path & 255;
      const int first = path >> 16 & 0x7fff, last = first + ((m - 1) >> 2);
#pragma unroll 1
      for (int i = first + 1; i <= last; ++i) {
        const float4 cu = entry_u[i], co = entry_o[i];
        const uint32_t s = places[i];
        const float x0 = row((s & 255u) * (DV * 4)), x1 = row((s >> 8 & 255u) * (DV * 4));
        const float x2 = row((s >> 16 & 255u) * (DV * 4)), x3 = row((s >> 24) * (DV * 4));
        pred = fmaf(cu.x, x0, pred), out = fmaf(co.x, x0, out);
        pred = fmaf(cu.y, x1, pred), out = fmaf(co.y, x1, out);
        pred = fmaf(cu.z, x2, pred), out = fmaf(co.z, x2, out);
        pred = fmaf(cu.w, x3, pred), out = fmaf(co.w, x3, out);
      }
    };
    umma::wait_ld();
#pragma unroll 1
    for (int t = 0; t < n; t += 2) {
      asm volatile("" : "+r"(k0), "+r"(k1), "+r"(q0), "+r"(q1));  // not before the wait
      if constexpr (C::kTerms) {
        asm volatile("" : "+r"(kl0), "+r"(kl1), "+r"(ql0), "+r"(ql1));
        k0 = __float_as_uint(__uint_as_float(k0) + __uint_as_float(kl0));
        k1 = __float_as_uint(__uint_as_float(k1) + __uint_as_float(kl1));
        q0 = __float_as_uint(__uint_as_float(q0) + __uint_as_float(ql0));
        q1 = __float_as_uint(__uint_as_float(q1) + __uint_as_float(ql1));
      }
      const float4 ia = reinterpret_cast<const float4*>(rec)[0], ib = reinterpret_cast<const float4*>(rec)[4];
      const uint4 oa = reinterpret_cast<const uint4*>(rec)[1], ob = reinterpret_cast<const uint4*>(rec)[5];
      const float4 ua = reinterpret_cast<const float4*>(rec)[2], oa4 = reinterpret_cast<const float4*>(rec)[3];
      const float4 ub = reinterpret_cast<const float4*>(rec)[6], ob4 = reinterpret_cast<const float4*>(rec)[7];
      const float va = mine[0], vb = mine[DV];
      const float xa0 = row(oa.x), xa1 = row(oa.y), xa2 = row(oa.z), xa3 = row(oa.w);
      const float xb0 = row(ob.x), xb1 = row(ob.y), xb2 = row(ob.z), xb3 = row(ob.w);
      float preda = ia.x * __uint_as_float(k0), outa = ia.x * __uint_as_float(q0);
      float predb = ib.x * __uint_as_float(k1), outb = ib.x * __uint_as_float(q1);
      preda = fmaf(ua.x, xa0, preda), outa = fmaf(oa4.x, xa0, outa);
      predb = fmaf(ub.y, xb1, predb), outb = fmaf(ob4.y, xb1, outb);
      preda = fmaf(ua.y, xa1, preda), outa = fmaf(oa4.y, xa1, outa);
      predb = fmaf(ub.z, xb2, predb), outb = fmaf(ob4.z, xb2, outb);
      preda = fmaf(ua.z, xa2, preda), outa = fmaf(oa4.z, xa2, outa);
      predb = fmaf(ub.w, xb3, predb), outb = fmaf(ob4.w, xb3, outb);
      preda = fmaf(ua.w, xa3, preda), outa = fmaf(oa4.w, xa3, outa);
      const int pa = __float_as_int(ia.w), pb = __float_as_int(ib.w);
      if ((pa | pb) < 0) {
        further(pa, preda, outa);
        further(pb, predb, outb);
      }
      const float xa = p.predicts ? ia.y * (va - preda) : va;
      // the second node may continue the first
      const float xp = ob.x == (uint32_t)t * (DV * 4) ? xa : xb0;
      predb = fmaf(ub.x, xp, predb), outb = fmaf(ob4.x, xp, outb);
      const float xb = p.predicts ? ib.y * (vb - predb) : vb;
      mine_k += 2;
      mine_q += 2;
      if (t + 2 < n) products();  // a pair ahead of its use
      mine[0] = xa;
      mine[DV] = xb;
      // (behind an odd last node: that node once more, instead of a branch)
      const bool both = t + 1 < n;
      const float ya = p.scale * fmaf(ia.z, xa, outa), yb = both ? p.scale * fmaf(ib.z, xb, outb) : ya;
      const uint32_t off_b = both ? off + step : off;
      io_store(go + off, ya);
      io_store(go + off_b, yb);
      if (store_u) {
        gu[off] = xa;
        gu[off_b] = both ? xb : xa;
      }
      off += 2 * step;
      mine += 2 * DV;
      rec += 2;
      umma::wait_ld();
    }
  }
  umma::fence_before();
  __syncthreads();
  if (warp == NT / 32 - 1) {
    umma::fence_after();
    umma::dealloc(tmem, C::cols(R));
  }
  if (failed && tid == 0) report(p.err, LA_DEVERR_TIMEOUT);
}

template <typename ST, typename IT, int DK, int DV, bool KDA>
cudaError_t launch_tree_tc(const TreeParams& p, cudaStream_t stream) {
  using C = TcCfg<ST, IT, DK, DV, KDA>;
  const int R = (p.max_nodes + 15) / 16 * 16;
  auto fn = &tree_tc_kernel<ST, IT, DK, DV, KDA>;
  static_assert(C::smem(kMaxNodes) <= 227 * 1024, "shared memory");
  if (prepare_kernel(reinterpret_cast<const void*>(fn), C::kThreads, C::smem(kMaxNodes)) <= 0)
    return cudaErrorInvalidConfiguration;
  return launch_dependent(fn, p.n_seqs * p.n_v_heads, C::kThreads, C::smem(R), stream, p, R);
}

}  // namespace tree
}  // namespace la
