// Layer norm row kernels of librn, forward and backward, for B200 (sm_100a):
//   mean = sum_j x_j / H,  c = x - mean,  rstd = rsqrt(sum_j c_j^2 / H + eps)
//   y = c * rstd * w + b
//   g = w * dy,  xh = c * rstd
//   dx = rstd * (g - mean_j(g) - xh * mean_j(g * xh))
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
// The rows' layout, staging and team reductions are the RMS norm's
// (rn_rows.cuh): a team of T threads owns a row, each thread K 16-byte vectors
// staged with cp.async S-1 rows ahead, (T, K) a function of the width and
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
__host__ __device__ constexpr int ln_bwd_block_of(int T) { return T <= 8 ? 128 : (T == 32 ? 256 : T); }
// CTAs per SM the kernel is built for
__host__ __device__ constexpr int ln_bwd_ctas_of(int T, int K, int VE) {
  return T <= 8 ? 4 : (T <= 128 ? 2 : 1);
}
// rows in flight per team: what the SM's shared memory takes at that many CTAs,
// one to four (one where two rows of the widest fp32 teams pass 227 KB)
__host__ __device__ constexpr int ln_bwd_stages_of(int T, int K, int VE) {
  const int per = 2 * K * ln_bwd_block_of(T) * 16;
  const int room = 200 * 1024 / ln_bwd_ctas_of(T, K, VE) -
                   (gain_src_of(T, K, VE) == kGainSmem ? K * T * VE * 4 : 0);
  return room / per >= 4 ? 4 : (room / per >= 1 ? room / per : 1);
}

// K per-vector sums, ascending from -0.0, joined by the pairwise tree; a vector
// the row does not reach is the identity
template <int VE, int T, int K, bool EXACT>
__device__ __forceinline__ float thread_sum(const float2 (&a)[K][VE / 2], int nv, int t) {
  float p[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float acc = -0.0f;
#pragma unroll
    for (int q = 0; q < VE / 2; ++q) {
      acc = __fadd_rn(acc, a[k][q].x);
      acc = __fadd_rn(acc, a[k][q].y);
    }
    p[k] = (EXACT || k * T + t < nv) ? acc : -0.0f;
  }
  return pairwise_tree<K>(p);
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
    float sum[1] = {thread_sum<VE, T, K, EXACT>(xf, nv, t)};
    team_sum<T, 1>(sum, red, phase, team, NT, 0xffffffffu);
    const float mu = mean_of(sum[0], a.H, a.inv_h, a.h_pow2);
    const float2 mu2 = bc2(-mu);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) xf[k][q] = add2(xf[k][q], mu2);   // x - mean
    float ss[1];
    {
      float p[K];
      vector_dots<VE, T, K, EXACT>(xf, xf, nv, t, p);
      ss[0] = pairwise_tree<K>(p);
    }
    team_sum<T, 1>(ss, red, phase, team, NT, 0xffffffffu);
    const float r = rsqrtf(__fadd_rn(mean_of(ss[0], a.H, a.inv_h, a.h_pow2), a.eps));
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
__global__ void __launch_bounds__(ln_bwd_block_of(T), ln_bwd_ctas_of(T, K, Fmt<DT>::VE))
k_ln_bwd(const LnBwdArgs a) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  constexpr int B = ln_bwd_block_of(T);
  constexpr int S = ln_bwd_stages_of(T, K, VE);
  constexpr int NT = B / T;
  constexpr int W = T > 32 ? T / 32 : 1;
  constexpr int GS = gain_src_of(T, K, VE);
  // dynamic shared memory: reduction scratch [2][NT][2][W] (T > 32) | gain
  // [K*T*VE] | stages [S][2][K][B] uint4 (afterwards the teams' partials
  // [NT][2H] floats) | mean and rstd stages [S][2][B]
  extern __shared__ float dsm[];
  float* red = dsm;
  float* gsm = red + (T > 32 ? 2 * NT * 2 * W : 0);
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
        c1 = add2(c1, gd);
        c2 = fma2(gd, mul2(add2(xf[q], mu2), rs2), c2);
      }
      const bool in = EXACT || k * T + t < nv;
      p1[k] = in ? __fadd_rn(c1.x, c1.y) : -0.0f;
      p2[k] = in ? __fadd_rn(c2.x, c2.y) : -0.0f;
    }
    float s[2] = {pairwise_tree<K>(p1), pairwise_tree<K>(p2)};
    team_sum<T, 2>(s, red, phase, team, NT, 0xffffffffu);
    const float2 m1 = bc2(-mean_of(s[0], a.H, a.inv_h, a.h_pow2));
    const float2 m2 = bc2(-mean_of(s[1], a.H, a.inv_h, a.h_pow2));
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
          const float2 xh = mul2(add2(xf[q], mu2), rs2);
          // rstd * ((g - mean(g)) - xh * mean(g*xh))
          dxv[q] = mul2(rs2, fma2(xh, m2, add2(mul2(gk[q], df[q]), m1)));
          if (counts) {
            aw[k][q] = fma2(df[q], xh, aw[k][q]);
            ab[k][q] = add2(ab[k][q], df[q]);
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
  if constexpr (NT == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int v = k * T + t;
      if (EXACT || v < nv) {
#pragma unroll
        for (int q = 0; q < VE / 4; ++q) {
          ow[v * (VE / 4) + q] = make_float4(aw[k][2 * q].x, aw[k][2 * q].y, aw[k][2 * q + 1].x, aw[k][2 * q + 1].y);
          if (biased)
            ob[v * (VE / 4) + q] = make_float4(ab[k][2 * q].x, ab[k][2 * q].y, ab[k][2 * q + 1].x, ab[k][2 * q + 1].y);
        }
      }
    }
  } else {
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
      constexpr int LB = NT <= 4 ? 2 : (NT == 8 ? 3 : (NT == 16 ? 4 : (NT == 32 ? 5 : (NT == 64 ? 6 : 7))));
      TreeCounter<LB, float4> tc;
#pragma unroll 8
      for (int j = 0; j < NT; ++j) tc.push(j, lb[j * 2 * H4 + c]);
      const float4 r = tc.finish(NT);
      if (c < H4) ow[c] = r;
      else ob[c - H4] = r;
    }
  }
}

// ---------------------------------------------------------------------------
// host: launch one instantiation, dispatch over the (T, K, exact) shapes
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

// Rows per backward CTA: about one wave of CTAs on a 148-SM B200 (the number is
// a constant of the operator, not the device's, so dw does not depend on the
// device), and at least four steps of the CTA's teams.
template <int DT, int T, int K>
constexpr int64_t ln_block_rows(int64_t rows) {
  constexpr int NT = ln_bwd_block_of(T) / T;
  constexpr int64_t wave = int64_t(148) * ln_bwd_ctas_of(T, K, Fmt<DT>::VE);
  const int64_t per = (rows + wave - 1) / wave;
  const int64_t steps = (per + NT - 1) / NT;
  return (steps < 4 ? 4 : steps) * NT;
}

template <int DT, int T, int K, bool EXACT>
rn_status launch_ln_bwd_tk(LnBwdArgs a, int64_t block_rows, int ctas, cudaStream_t st) {
  constexpr int VE = Fmt<DT>::VE, B = ln_bwd_block_of(T), NT = B / T;
  constexpr int S = ln_bwd_stages_of(T, K, VE);
  constexpr size_t stages = size_t(S) * 2 * K * B * 16;
  static_assert(NT == 1 || size_t(NT) * 2 * T * K * VE * 4 <= stages + size_t(S) * 2 * B * 4,
                "the teams' partials reuse the staging buffer");
  constexpr size_t smem = (T > 32 ? 2 * NT * 2 * (T / 32) * sizeof(float) : 0) +
                          (gain_src_of(T, K, VE) == kGainSmem ? K * T * VE * sizeof(float) : 0) +
                          stages + size_t(S) * 2 * B * sizeof(float);
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  static KernelPrep prep;
  (void)prepare_kernel(k_ln_bwd<DT, T, K, EXACT>, B, smem, prep);
  a.block_rows = block_rows;
  return launch_pdl(k_ln_bwd<DT, T, K, EXACT>, dim3(ctas), dim3(B), smem, st, a);
}

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
int64_t ln_bwd_block_rows(const Sched& s, int64_t rows) {
#define RN_LN_CASE(T_, K_, EX_) \
  if (s.T == T_ && s.K == K_) return ln_block_rows<DT, T_, K_>(rows);
  if constexpr (DT == RN_F32) {
    RN_SHAPES_32(RN_LN_CASE)
  } else {
    RN_SHAPES_16(RN_LN_CASE)
  }
#undef RN_LN_CASE
  return 0;
}

template <int DT>
rn_status launch_ln_bwd(const Sched& s, const LnBwdArgs& a, int64_t block_rows, int ctas,
                        cudaStream_t st) {
  const bool ex = a.nv == s.T * s.K;
#define RN_LN_CASE(T_, K_, EX_)            \
  if (s.T == T_ && s.K == K_ && ex == EX_) \
    return launch_ln_bwd_tk<DT, T_, K_, EX_>(a, block_rows, ctas, st);
  if constexpr (DT == RN_F32) {
    RN_SHAPES_32(RN_LN_CASE)
  } else {
    RN_SHAPES_16(RN_LN_CASE)
  }
#undef RN_LN_CASE
  return RN_E_WIDTH;
}

}  // namespace rn_detail
