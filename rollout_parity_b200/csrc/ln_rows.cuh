// Layer norm row kernels of librn, forward and backward, for B200 (sm_100a):
//   mean = sum_j x_j / H,  c = x - mean,  rstd = rsqrt(sum_j c_j^2 / H + eps)
//   y = c * rstd * w + b
//   g = w * dy,  xh = c * rstd
//   dx = rstd * (g - mean_j(g) - xh * mean_j(g * xh))
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
// A team of T threads owns a row, each thread K 16-byte vectors staged with
// cp.async S-1 rows ahead, as in the RMS norm (rn_rows.cuh).  Rows of up to 128
// vectors belong to teams of at most a warp; the backward of wider ones has a
// kernel of its own (k_ln_bwd_wide).  (T, K) is a function of the width and
// element format only, so a row's y, mean, rstd and dx are bitwise the same
// alone or inside any batch.
//
// The variance is the mean of the squared differences from the mean, taken
// from the row held in registers (a second reduction instead of E[x^2] - mean^2,
// which cancels when the mean is large).
#pragma once

#include "ln_common.cuh"
#include "rn_rows.cuh"

namespace rn_detail {

// ---- backward launch shapes ---------------------------------------------------
__host__ __device__ constexpr int ln_bwd_block_of(int T) { return T <= 8 ? 128 : 256; }
// CTAs per SM the kernel is built for
__host__ __device__ constexpr int ln_bwd_ctas_of(int T) { return T <= 8 ? 4 : 2; }
// rows in flight per team: what the SM's shared memory takes at that many CTAs,
// two to four
__host__ __device__ constexpr int ln_bwd_stages_of(int T, int K, int VE) {
  const int per = 2 * K * ln_bwd_block_of(T) * 16;
  const int room = 200 * 1024 / ln_bwd_ctas_of(T) -
                   (gain_src_of(T, K, VE) == kGainSmem ? K * T * VE * 4 : 0);
  return room / per >= 4 ? 4 : room / per;
}

// ---- wide rows ---------------------------------------------------------------
// Backward, rows of more than 128 vectors: one CTA to an SM, holding NT teams
// of T threads that walk rows independently of one another, each with a named
// barrier of its own.  What bounds a row is the chain load - sums - barrier -
// store, so rows in flight count for more than threads to a row: a thread
// holds 24 to 40 elements (their dw and db sums take up to 80 registers).
constexpr int kWideThreads = 512;
constexpr size_t kWideSmem = 227 * 1024;
struct WideShape {
  int teams, stages;   // teams to a CTA, rows staged to a team
  size_t smem;
};
// As many teams as the threads allow with two rows of each in shared memory, one at
// least, then as many rows as fit, up to four (fp32 rows from 12288 elements on: one
// team and one row, so that its load, sums and store take turns).
__host__ __device__ constexpr WideShape wide_shape(int T, int K, int VE) {
  const size_t params = size_t(K) * VE * T * 4;                 // w
  const size_t row = size_t(2 * K * 16 + 2 * 4) * T;            // x, dy, mean, rstd
  const size_t team = 256;                                      // reduction scratch
  const size_t room = kWideSmem - params;
  int teams = kWideThreads / T;
  if (T > 32 && teams > 15) teams = 15;                         // named barriers 1 to 15
  while (teams > 1 && teams * (2 * row + team) > room) --teams;
  const size_t fit = (room - teams * team) / (teams * row);
  const int stages = fit > 4 ? 4 : int(fit);
  return WideShape{teams, stages, params + teams * (stages * row + team)};
}

// The two-lane fp32 addition.  (The RMS norm keeps its additions scalar so that
// a product before one is never fused into it; here either form is as good, and
// every row runs the same instructions.)
__device__ __forceinline__ float2 addp(float2 a, float2 b) { return __fadd2_rn(a, b); }

// Sum of a thread's elements: a vector's even and odd elements ascending from
// -0.0, the two joined, the K vectors by the pairwise tree; a vector the row does
// not reach is the identity.
template <int VE, int T, int K, bool EXACT, bool SQUARE>
__device__ __forceinline__ float thread_sum(const float2 (&a)[K][VE / 2], int nv, int t) {
  float p[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 c = bc2(-0.0f);
#pragma unroll
    for (int q = 0; q < VE / 2; ++q) c = SQUARE ? fma2(a[k][q], a[k][q], c) : addp(c, a[k][q]);
    p[k] = (EXACT || k * T + t < nv) ? __fadd_rn(c.x, c.y) : -0.0f;
  }
  return pairwise_tree<K>(p);
}

// sum / H, correctly rounded: the product with the rounded reciprocal and one
// correction by its residual (P. Markstein, "Computation of elementary functions on
// the IBM RISC System/6000 processor", 1990).  The product alone is off in the last
// place for some widths (776 among them): a constant row was not its bias then, but
// off by that times 1 / sqrt(eps).  The other means stay products: their last place
// is the last place of an output.  (__fdiv_rn here: 16384 x 5120 bf16 60.2 to 61.1
// us, 8192 x 1544 fp32 17 to 19; in the backward 88.9 to 100.6.)
__device__ __forceinline__ float row_mean(float sum, float h, float inv_h) {
  const float q = __fmul_rn(sum, inv_h);
  return fabsf(q) < INFINITY ? fmaf(fmaf(-q, h, sum), inv_h, q) : q;
}

template <int DT, int T, int K, bool EXACT>
__global__ void __launch_bounds__(fwd_block_of(T, K), fwd_min_blocks_of(T, K))
k_ln_fwd(const LnFwdArgs a) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  constexpr int S = fwd_stages_of(T, false, false, VE);
  constexpr int B = fwd_block_of(T, K);
  constexpr int NT = B / T;
  constexpr int W = T > 32 ? T / 32 : 1;
  constexpr int GS = gain_src_of(T, K, VE);
  // dynamic shared memory: reduction scratch [2][NT][W] (T > 32) | gain and bias
  // [2][K*T*VE] (where the gain is kept there) | stages [S][K][B] uint4
  extern __shared__ float dsm[];
  float* red = dsm;
  float* gsm = red + (T > 32 ? 2 * NT * W : 0);
  float* bsm = gsm + (GS == kGainSmem ? K * T * VE : 0);
  uint4* stg = reinterpret_cast<uint4*>(bsm + (GS == kGainSmem ? K * T * VE : 0));
  const int tid = threadIdx.x, team = tid / T, t = tid % T;
  const int nv = a.nv;
  const bool biased = a.b != nullptr;
  int phase = 0;

  griddep_trigger();
  griddep_wait();
  Gain<VE, K, T, GS> gain, bias;
  gain.init(a.w, 0.0f, nv, t, gsm);
  if (biased) bias.init(a.b, 0.0f, nv, t, bsm);   // uniform branch

  auto slot = [&](int sl, int k) -> uint4* { return stg + (sl * K + k) * B + tid; };
  const int64_t nblk = (a.rows + NT - 1) / NT;
  const int64_t iters = nblk > blockIdx.x ? (nblk - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
  auto row_of = [&](int64_t i) { return (int64_t(blockIdx.x) + i * gridDim.x) * NT + team; };
  auto issue = [&](int64_t i, int sl) {
    if (i < iters) {
      const int64_t row = row_of(i);
      if (row < a.rows) {
        const int64_t off = row * nv + t;
#pragma unroll
        for (int k = 0; k < K; ++k)
          if (EXACT || k * T + t < nv) cp_async16(slot(sl, k), a.x + off + k * T);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i, i);
  int sl = 0;
  for (int64_t i = 0; i < iters; ++i) {
    {
      int sa = sl + S - 1;
      if (sa >= S) sa -= S;
      issue(i + S - 1, sa);
    }
    cp_async_wait<S - 1>();
    const int64_t row = row_of(i);
    const bool act = row < a.rows;
    float2 xf[K][VE / 2];
#pragma unroll
    for (int k = 0; k < K; ++k) F::unpack2(*slot(sl, k), xf[k]);
    float sum[1] = {thread_sum<VE, T, K, EXACT, false>(xf, nv, t)};
    team_sum<T, 1>(sum, red, phase, team, NT, 0xffffffffu);
    const float mu = row_mean(sum[0], float(a.H), a.inv_h);
    const float2 mu2 = bc2(-mu);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) xf[k][q] = addp(xf[k][q], mu2);   // x - mean
    float ss[1] = {thread_sum<VE, T, K, EXACT, true>(xf, nv, t)};
    team_sum<T, 1>(ss, red, phase, team, NT, 0xffffffffu);
    const float r = rsqrtf(__fadd_rn(__fmul_rn(ss[0], a.inv_h), a.eps));
    const float2 r2 = bc2(r);
    const int64_t off = row * nv + t;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (act && (EXACT || k * T + t < nv)) {
        float2 yv[VE / 2], gk[VE / 2];
        gain.get2(k, gk);
        if (biased) {
          float2 bk[VE / 2];
          bias.get2(k, bk);
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) yv[q] = fma2(mul2(xf[k][q], r2), gk[q], bk[q]);
        } else {
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) yv[q] = mul2(mul2(xf[k][q], r2), gk[q]);
        }
        st_stream(a.y + off + k * T, F::pack2v(yv));
      }
    }
    if (act && t == 0) {
      if (a.mean != nullptr) a.mean[row] = mu;
      if (a.rstd != nullptr) a.rstd[row] = r;
    }
    if (++sl == S) sl = 0;
  }
  cp_async_wait<0>();
}

// Backward.  CTA c owns the contiguous rows [c*block_rows, (c+1)*block_rows);
// its NT teams take consecutive rows of it step by step, so a step reads and
// writes one contiguous block of memory.  A team keeps the dw and db sums of
// its rows, in ascending order from -0.0, in registers (2*K*VE floats a
// thread); at the end the CTA's teams are joined by the pairwise tree in shared
// memory and the CTA writes one partial row of each, which k_ln_fold joins with the
// same tree.  block_rows depends on the sizes and the format only.
// The two row sums (of g and g*xh) go through one team reduction.  x and dy stay
// staged in shared memory across it and xh and g are formed again after it: the
// accumulators leave no registers to keep them.
template <int DT, int T, int K, bool EXACT>
__global__ void __launch_bounds__(ln_bwd_block_of(T), ln_bwd_ctas_of(T))
k_ln_bwd(const LnBwdArgs a) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  constexpr int B = ln_bwd_block_of(T);
  constexpr int S = ln_bwd_stages_of(T, K, VE);
  constexpr int NT = B / T;
  constexpr int GS = gain_src_of(T, K, VE);
  static_assert(T <= 32, "a team within a warp: its sums need no shared memory");
  // dynamic shared memory: gain [K*T*VE] | stages [S][2][K][B] uint4 (afterwards
  // the teams' partials [NT][2H] floats) | mean and rstd stages [S][2][B]
  extern __shared__ float dsm[];
  float* gsm = dsm;
  uint4* stg = reinterpret_cast<uint4*>(gsm + (GS == kGainSmem ? K * T * VE : 0));
  float* ssm = reinterpret_cast<float*>(stg + S * 2 * K * B);
  const int tid = threadIdx.x, team = tid / T, t = tid % T;
  const int nv = a.nv;
  int phase = 0;

  griddep_trigger();
  griddep_wait();
  Gain<VE, K, T, GS> gain;
  gain.init(a.w, 0.0f, nv, t, gsm);

  auto slot = [&](int sl, int ten, int k) -> uint4* { return stg + ((sl * 2 + ten) * K + k) * B + tid; };
  const int64_t r0 = int64_t(blockIdx.x) * a.block_rows;
  const int64_t r1 = r0 + a.block_rows < a.rows ? r0 + a.block_rows : a.rows;
  const int steps = int((r1 - r0 + NT - 1) / NT);
  auto issue = [&](int i, int sl) {
    const int64_t row = r0 + int64_t(i) * NT + team;
    if (i < steps && row < r1) {
      const int64_t off = row * nv + t;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (EXACT || k * T + t < nv) {
          cp_async16(slot(sl, 0, k), a.x + off + k * T);
          cp_async16(slot(sl, 1, k), a.dy + off + k * T);
        }
      }
      cp_async4(ssm + (sl * 2) * B + tid, a.mean + row);
      cp_async4(ssm + (sl * 2 + 1) * B + tid, a.rstd + row);
    }
    cp_async_commit();
  };
  float2 aw[K][VE / 2], ab[K][VE / 2];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int q = 0; q < VE / 2; ++q) aw[k][q] = ab[k][q] = bc2(-0.0f);

#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(i, i);
  int sl = 0;
  for (int i = 0; i < steps; ++i) {
    {
      int sa = sl + S - 1;
      if (sa >= S) sa -= S;
      issue(i + S - 1, sa);
    }
    cp_async_wait<S - 1>();
    const int64_t row = r0 + int64_t(i) * NT + team;
    const bool act = row < r1;
    const bool counts = act && (a.mask == nullptr || __ldg(a.mask + row) != 0);
    const float2 mu2 = bc2(-ssm[(sl * 2) * B + tid]), rs2 = bc2(ssm[(sl * 2 + 1) * B + tid]);
    float p1[K], p2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 xf[VE / 2], df[VE / 2], gk[VE / 2];
      F::unpack2(*slot(sl, 0, k), xf);
      F::unpack2(*slot(sl, 1, k), df);
      gain.get2(k, gk);
      float2 c1 = bc2(-0.0f), c2 = bc2(-0.0f);   // even and odd elements
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) {
        const float2 gd = mul2(gk[q], df[q]);
        c1 = addp(c1, gd);
        c2 = fma2(gd, mul2(addp(xf[q], mu2), rs2), c2);
      }
      const bool in = EXACT || k * T + t < nv;
      p1[k] = in ? __fadd_rn(c1.x, c1.y) : -0.0f;
      p2[k] = in ? __fadd_rn(c2.x, c2.y) : -0.0f;
    }
    float s[2] = {pairwise_tree<K>(p1), pairwise_tree<K>(p2)};
    team_sum<T, 2>(s, nullptr, phase, team, NT, 0xffffffffu);
    __syncwarp();   // (a team of one warp too: the staged row is read again, not kept in registers)
    const float2 m1 = bc2(-__fmul_rn(s[0], a.inv_h));
    const float2 m2 = bc2(-__fmul_rn(s[1], a.inv_h));
    const int64_t off = row * nv + t;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (act && (EXACT || k * T + t < nv)) {
        float2 xf[VE / 2], df[VE / 2], gk[VE / 2], dxv[VE / 2];
        F::unpack2(*slot(sl, 0, k), xf);
        F::unpack2(*slot(sl, 1, k), df);
        gain.get2(k, gk);
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) {
          const float2 xh = mul2(addp(xf[q], mu2), rs2);
          // rstd * ((g - mean(g)) - xh * mean(g*xh))
          dxv[q] = mul2(rs2, fma2(xh, m2, addp(mul2(gk[q], df[q]), m1)));
          if (counts) {
            aw[k][q] = fma2(df[q], xh, aw[k][q]);
            ab[k][q] = addp(ab[k][q], df[q]);
          }
        }
        st_stream(a.dx + off + k * T, F::pack2v(dxv));
      }
    }
    if (++sl == S) sl = 0;
  }
  cp_async_wait<0>();

  const bool biased = a.pb != nullptr;
  float4* ow = reinterpret_cast<float4*>(a.pw + int64_t(blockIdx.x) * a.H);
  float4* ob = reinterpret_cast<float4*>(a.pb + (biased ? int64_t(blockIdx.x) * a.H : 0));
  const int H4 = a.H / 4;
  float4* lb = reinterpret_cast<float4*>(stg);   // [NT][2 * H4]
  __syncthreads();   // every team is done with its staged rows
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int v = k * T + t;
    if (EXACT || v < nv) {
#pragma unroll
      for (int q = 0; q < VE / 4; ++q) {
        float4* at = lb + team * 2 * H4 + v * (VE / 4) + q;
        at[0] = make_float4(aw[k][2 * q].x, aw[k][2 * q].y, aw[k][2 * q + 1].x, aw[k][2 * q + 1].y);
        at[H4] = make_float4(ab[k][2 * q].x, ab[k][2 * q].y, ab[k][2 * q + 1].x, ab[k][2 * q + 1].y);
      }
    }
  }
  __syncthreads();
  // a team without rows holds -0.0, the identity, so every team joins
  for (int c = tid; c < (biased ? 2 : 1) * H4; c += B) {
    constexpr int LB = NT == 8 ? 3 : (NT == 16 ? 4 : (NT == 32 ? 5 : (NT == 64 ? 6 : 7)));
    static_assert(NT == 1 << LB, "8 to 128 teams");
    TreeCounter<LB, float4> tc;
#pragma unroll 8
    for (int j = 0; j < NT; ++j) tc.push(j, lb[j * 2 * H4 + c]);
    const float4 r = tc.finish(NT);
    if (c < H4) ow[c] = r;
    else ob[c - H4] = r;
  }
}

// ---------------------------------------------------------------------------
// Wide rows
// ---------------------------------------------------------------------------
__device__ __forceinline__ void team_barrier(int team, int T) {
  asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(T) : "memory");
}
// U sums over a team of T threads: the xor butterfly over the lanes, then the
// pairwise tree over the warps' results, which every thread forms, so that all
// end with the same bits.  `red` is the team's scratch, [2][U][16] floats.
template <int U, int T>
__device__ __forceinline__ void wide_sum(float (&v)[U], float* red, int& phase, int team) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __fadd_rn(v[u], __shfl_xor_sync(0xffffffffu, v[u], o));
  }
  if constexpr (T > 32) {
    constexpr int W = T / 32;
    float* buf = red + phase * (U * 16);
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) buf[u * 16 + (threadIdx.x % T) / 32] = v[u];
    }
    team_barrier(team, T);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float p[W];
#pragma unroll
      for (int i = 0; i < W; ++i) p[i] = buf[u * 16 + i];
      v[u] = pairwise_tree<W>(p);
    }
  }
}
// a thread's vector of fp32 parameters, [vectors][quarters][T] float4 in shared
// memory: consecutive threads read consecutive 16-byte words
template <int VE, int T>
__device__ __forceinline__ void read_param(const float4* p, int k, float2 (&f)[VE / 2]) {
#pragma unroll
  for (int q = 0; q < VE / 4; ++q) {
    const float4 u = p[(k * (VE / 4) + q) * T];
    f[2 * q] = make_float2(u.x, u.y);
    f[2 * q + 1] = make_float2(u.z, u.w);
  }
}

// As k_ln_bwd: CTA c owns the rows [c*block_rows, ...), its teams take consecutive
// ones, and the teams' partials are joined at the end.
template <int DT, int T, int K, bool EXACT>
__global__ void __launch_bounds__(kWideThreads, 1)
k_ln_bwd_wide(const LnBwdArgs a) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  constexpr WideShape kShape = wide_shape(T, K, VE);
  constexpr int NT = kShape.teams, S = kShape.stages, B = NT * T;
  static_assert(S >= 1, "a row fits");
  // dynamic shared memory: w [K][VE/4][T] float4 | stages [S][2][K][B] uint4
  // (afterwards the teams' partials [NT][H] floats, dw then db) | mean and rstd
  // stages [S][2][B] | reduction scratch [teams][2][2][16]
  extern __shared__ float dsm[];
  const int tid = threadIdx.x, team = tid / T, t = tid % T;
  float4* wsm = reinterpret_cast<float4*>(dsm);
  uint4* stg = reinterpret_cast<uint4*>(wsm + K * (VE / 4) * T);
  float* ssm = reinterpret_cast<float*>(stg + S * 2 * K * B);
  float* red = ssm + S * 2 * B + team * 64;
  const int nv = a.nv;
  int phase = 0;
  griddep_trigger();
  griddep_wait();
  uint4* mine = stg + tid;
  if constexpr (!EXACT) {   // past the row: zeros
    for (int i = 0; i < S * 2 * K; ++i)
      if ((i % K) * T + t >= nv) mine[i * B] = make_uint4(0, 0, 0, 0);
  }
  const int64_t r0 = int64_t(blockIdx.x) * a.block_rows;
  const int64_t r1 = r0 + a.block_rows < a.rows ? r0 + a.block_rows : a.rows;
  auto issue = [&](int64_t row, int sl) {
    if (row < r1) {
      const uint4* xp = a.x + row * nv + t;
      const uint4* dp = a.dy + row * nv + t;
      uint4* sp = mine + sl * (2 * K * B);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (EXACT || k * T + t < nv) {
          cp_async16(sp + k * B, xp + k * T);
          cp_async16(sp + (K + k) * B, dp + k * T);
        }
      }
      cp_async4(ssm + (sl * 2) * B + tid, a.mean + row);
      cp_async4(ssm + (sl * 2 + 1) * B + tid, a.rstd + row);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue(r0 + i * NT + team, i);
  for (int i = tid; i < K * (VE / 4) * T; i += B) {
    const int v = (i / T / (VE / 4)) * T + i % T;
    wsm[i] = EXACT || v < nv ? __ldg(reinterpret_cast<const float4*>(a.w) + v * (VE / 4) + i / T % (VE / 4))
                             : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float4* wp = wsm + t;
  float2 aw[K][VE / 2], ab[K][VE / 2];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int q = 0; q < VE / 2; ++q) aw[k][q] = ab[k][q] = bc2(-0.0f);
  __syncthreads();

  int sl = 0;
  for (int64_t row = r0 + team; row < r1; row += NT) {
    {
      int sa = sl + S - 1;
      if (sa >= S) sa -= S;
      issue(row + int64_t(S - 1) * NT, sa);
    }
    cp_async_wait<S - 1>();
    const bool counts = a.mask == nullptr || __ldg(a.mask + row) != 0;   // uniform in the team
    // with c = x - mean:  xh = rstd * c,  dx = rstd * ((g - mean(g)) - c * (rstd * mean(g * xh)))
    // (no power of rstd stands alone: every value is of the size of dy or of dx)
    const uint4* sp = mine + sl * (2 * K * B);
    const float rs = ssm[(sl * 2 + 1) * B + tid];
    const float2 mu2 = bc2(-ssm[(sl * 2) * B + tid]), rs2 = bc2(rs);
    float p1[K], p2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 xf[VE / 2], df[VE / 2], g[VE / 2];
      F::unpack2(sp[k * B], xf);
      F::unpack2(sp[(K + k) * B], df);
      read_param<VE, T>(wp, k, g);
      float2 c1 = bc2(-0.0f), c2 = bc2(-0.0f);   // even and odd elements
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) {
        const float2 xh = mul2(addp(xf[q], mu2), rs2), gd = mul2(g[q], df[q]);
        c1 = addp(c1, gd);
        c2 = fma2(gd, xh, c2);
        if (counts) {   // dw and db need no row sum: taken before the barrier
          aw[k][q] = fma2(df[q], xh, aw[k][q]);
          ab[k][q] = addp(ab[k][q], df[q]);
        }
      }
      p1[k] = __fadd_rn(c1.x, c1.y);
      p2[k] = __fadd_rn(c2.x, c2.y);
    }
    float s[2] = {pairwise_tree<K>(p1), pairwise_tree<K>(p2)};
    wide_sum<2, T>(s, red, phase, team);
    __syncwarp();   // (a team of one warp too: the staged row is read again, not kept in registers)
    const float2 m1 = bc2(-__fmul_rn(s[0], a.inv_h));
    const float2 m2 = bc2(-__fmul_rn(rs, __fmul_rn(s[1], a.inv_h)));
    uint4* op = a.dx + row * nv + t;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (EXACT || k * T + t < nv) {   // c and g again from the staged row: no registers to keep them
        float2 xf[VE / 2], df[VE / 2], g[VE / 2];
        F::unpack2(sp[k * B], xf);
        F::unpack2(sp[(K + k) * B], df);
        read_param<VE, T>(wp, k, g);
#pragma unroll
        for (int q = 0; q < VE / 2; ++q)
          xf[q] = mul2(rs2, fma2(addp(xf[q], mu2), m2, addp(mul2(g[q], df[q]), m1)));
        st_stream(op + k * T, F::pack2v(xf));
      }
    }
    if (++sl == S) sl = 0;
  }
  cp_async_wait<0>();

  // the teams' partials, dw then db: written by the teams, joined by the CTA's
  // threads with the pairwise tree (a team without rows holds the identity)
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    if (part == 1 && a.pb == nullptr) break;
    float4* out = reinterpret_cast<float4*>((part == 0 ? a.pw : a.pb) + int64_t(blockIdx.x) * a.H);
    const int H4 = a.H / 4;
    float4* lb = NT == 1 ? out : reinterpret_cast<float4*>(stg) + team * H4;
    if (NT > 1) __syncthreads();   // the staging buffer, or its last use, is done with
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * T + t;
      if (EXACT || v < nv) {
#pragma unroll
        for (int q = 0; q < VE / 4; ++q) {
          const float2 lo = part == 0 ? aw[k][2 * q] : ab[k][2 * q];
          const float2 hi = part == 0 ? aw[k][2 * q + 1] : ab[k][2 * q + 1];
          lb[v * (VE / 4) + q] = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
      }
    }
    if (NT > 1) {
      __syncthreads();
      const float4* all = reinterpret_cast<const float4*>(stg);
      for (int c = tid; c < H4; c += B) {
        float4 p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) p[j] = j < NT ? all[j * H4 + c] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
#pragma unroll
          for (int j = 0; j + d < 16; j += 2 * d)
            if (j + d < NT) p[j] = add4(p[j], p[j + d]);
        }
        out[c] = p[0];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host: launch one instantiation, dispatch over the shapes that row_sched and ln_bwd_sched give
// ---------------------------------------------------------------------------
template <int DT, int T, int K, bool EXACT>
rn_status launch_ln_fwd_tk(const LnFwdArgs& a, cudaStream_t st) {
  constexpr int VE = Fmt<DT>::VE, B = fwd_block_of(T, K), NT = B / T;
  constexpr size_t smem = (T > 32 ? 2 * NT * (T / 32) * sizeof(float) : 0) +
                          (gain_src_of(T, K, VE) == kGainSmem ? 2 * K * T * VE * sizeof(float) : 0) +
                          size_t(fwd_stages_of(T, false, false, VE)) * K * B * 16;
  static KernelPrep prep;
  const int nb = prepare_kernel(k_ln_fwd<DT, T, K, EXACT>, B, smem, prep);
  const int64_t nblk = (a.rows + NT - 1) / NT;
  const int64_t wave = int64_t(nb) * sm_count();
  return launch_pdl(k_ln_fwd<DT, T, K, EXACT>, dim3(grid_cap(nblk < wave ? nblk : wave)), dim3(B),
                    smem, st, a);
}

template <int DT, int T, int K, bool EXACT>
rn_status launch_ln_bwd_tk(const LnBwdArgs& a, int ctas, cudaStream_t st) {
  constexpr int VE = Fmt<DT>::VE, B = ln_bwd_block_of(T), NT = B / T;
  constexpr int S = ln_bwd_stages_of(T, K, VE);
  constexpr size_t stages = size_t(S) * 2 * K * B * 16;
  static_assert(size_t(NT) * 2 * T * K * VE * 4 <= stages + size_t(S) * 2 * B * 4,
                "the teams' partials reuse the staging buffer");
  constexpr size_t smem = (gain_src_of(T, K, VE) == kGainSmem ? K * T * VE * sizeof(float) : 0) +
                          stages + size_t(S) * 2 * B * sizeof(float);
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static KernelPrep prep;
  (void)prepare_kernel(k_ln_bwd<DT, T, K, EXACT>, B, smem, prep);
  return launch_pdl(k_ln_bwd<DT, T, K, EXACT>, dim3(ctas), dim3(B), smem, st, a);
}

template <int DT, int T, int K, bool EXACT>
rn_status launch_ln_bwd_wide(const LnBwdArgs& a, int ctas, cudaStream_t st) {
  constexpr WideShape w = wide_shape(T, K, Fmt<DT>::VE);
  static KernelPrep prep;
  (void)prepare_kernel(k_ln_bwd_wide<DT, T, K, EXACT>, w.teams * T, w.smem, prep);
  return launch_pdl(k_ln_bwd_wide<DT, T, K, EXACT>, dim3(ctas), dim3(w.teams * T), w.smem, st, a);
}

// Rows per backward CTA: about one wave of CTAs on a 148-SM B200 (the number is
// a constant of the operator, not the device's, so dw does not depend on the
// device), and at least four steps of the CTA's teams: few rows make fewer CTAs than
// SMs (1000 rows of width 1032 16 of them, of 5120 63).
inline int64_t ln_rows_of_block(int64_t rows, int teams, int ctas_per_sm) {
  const int64_t wave = int64_t(148) * ctas_per_sm;
  const int64_t per = (rows + wave - 1) / wave;
  const int64_t steps = (per + teams - 1) / teams;
  return (steps < 4 ? 4 : steps) * teams;
}

// teams of at most a warp (rows of up to 128 vectors): the RMS norm's (T, K)
#define RN_LN_SHAPES_16(X)                                                                      \
  X(1, 1, true) X(1, 2, true) X(1, 3, true) X(1, 4, true) X(8, 2, true)                         \
  X(2, 3, false) X(2, 3, true) X(2, 4, false) X(2, 4, true)                                     \
  X(4, 3, false) X(4, 3, true) X(4, 4, false) X(4, 4, true)                                     \
  X(8, 3, false) X(8, 3, true) X(8, 4, false) X(8, 4, true)                                     \
  X(32, 2, false) X(32, 2, true) X(32, 3, false) X(32, 3, true) X(32, 4, false) X(32, 4, true)
#define RN_LN_SHAPES_32(X)                                                                      \
  X(1, 2, true) X(1, 4, true) X(2, 3, true) X(2, 4, true)                                       \
  X(4, 3, false) X(4, 3, true) X(4, 4, false) X(4, 4, true)                                     \
  X(8, 3, false) X(8, 3, true) X(8, 4, false) X(8, 4, true)                                     \
  X(32, 2, false) X(32, 2, true) X(32, 3, false) X(32, 3, true) X(32, 4, false) X(32, 4, true)

// wide backward teams, (T, eights of elements a thread); at 32 threads fewer than
// five only in fp32, whose 128 vectors are half as many elements
#define RN_LN_WIDE_32(X) X(32, 3) X(32, 4)
#define RN_LN_WIDE(X)                                                                     \
  X(32, 5) X(64, 3) X(64, 4) X(64, 5) X(128, 3) X(128, 4) X(128, 5) X(256, 3) X(256, 4)   \
  X(256, 5) X(512, 3) X(512, 4)

template <int DT>
rn_status launch_ln_fwd(const Sched& s, const LnFwdArgs& a, cudaStream_t st) {
  const bool ex = a.nv == s.T * s.K;
#define RN_LN_CASE(T_, K_, EX_) \
  if (s.T == T_ && s.K == K_ && ex == EX_) return launch_ln_fwd_tk<DT, T_, K_, EX_>(a, st);
  if constexpr (DT == RN_F32) {
    RN_SHAPES_32(RN_LN_CASE)
  } else {
    RN_SHAPES_16(RN_LN_CASE)
  }
#undef RN_LN_CASE
  return RN_E_WIDTH;
}

template <int DT>
int64_t ln_bwd_block_rows(const Sched& s, int64_t rows, bool wide) {
  constexpr int VE = Fmt<DT>::VE;
  if (wide) return ln_rows_of_block(rows, wide_shape(s.T, s.K, VE).teams, 1);
  return ln_rows_of_block(rows, ln_bwd_block_of(s.T) / s.T, ln_bwd_ctas_of(s.T));
}

template <int DT>
rn_status launch_ln_bwd(const Sched& s, const LnBwdArgs& a, int ctas, cudaStream_t st) {
  constexpr int M = 8 / Fmt<DT>::VE;
  const bool ex = a.nv == s.T * s.K;
  if (a.nv > 128) {
#define RN_LN_CASE(T_, E_)                                                                     \
  if (s.T == T_ && s.K == E_ * M)                                                              \
    return ex ? launch_ln_bwd_wide<DT, T_, E_ * M, true>(a, ctas, st)                          \
              : launch_ln_bwd_wide<DT, T_, E_ * M, false>(a, ctas, st);
    if constexpr (DT == RN_F32) {
      RN_LN_WIDE_32(RN_LN_CASE)
    }
    RN_LN_WIDE(RN_LN_CASE)
#undef RN_LN_CASE
    return RN_E_WIDTH;
  }
#define RN_LN_CASE(T_, K_, EX_)            \
  if (s.T == T_ && s.K == K_ && ex == EX_) \
    return launch_ln_bwd_tk<DT, T_, K_, EX_>(a, ctas, st);
  if constexpr (DT == RN_F32) {
    RN_LN_SHAPES_32(RN_LN_CASE)
  } else {
    RN_LN_SHAPES_16(RN_LN_CASE)
  }
#undef RN_LN_CASE
  return RN_E_WIDTH;
}

}  // namespace rn_detail
