// Linear cross entropy of librn (include/rn.h, "Linear cross entropy"): the
// projection of x [rows, H] onto the vocabulary W [V, H] and the softmax loss
// of one target per row, without ever storing the logits of the whole
// vocabulary:
//   z = x W^T,  s = z or cap * tanh(z / cap),  lse = log sum_v exp(s_v)
//   nll = lse - s[target]
//   dz_v = g * (exp(s_v - lse) - [v == target]) * (1 - (s_v / cap)^2)
//   dx = dz W,  dW = dz^T x
//
// Four matrix products on the tensor cores run through one kernel,
// k_xent_tile: the logits of the forward (their epilogue keeps, per row and
// 256 columns, the maximum and the sum of exponentials), the logits again in
// the backward (the epilogue writes dz, rounded to the element format), dx and
// dW.  The backward takes the vocabulary in pieces whose dz fits the
// workspace.
//
// Order of the sums: a row's statistics are taken over its 256-column tiles
// and joined in an order that depends on V only; dx is summed over chunks of
// the vocabulary whose size depends on V only, in ascending order.  So nll,
// lse and dx of a row are bitwise the same alone or inside any batch.  dW sums
// the kept rows in order, in the tensor cores' fp32 accumulator.
#include <cuda.h>

#include <cmath>
#include <mutex>

#include "rn_checks.cuh"
#include "rn_rows.cuh"
#include "rn_tc.cuh"

using namespace rn_detail;

namespace {

constexpr int64_t kMaxXentRows = int64_t(1) << 22;
constexpr int64_t kMaxXentVocab = int64_t(1) << 24;
constexpr int kIgnored = -1;

// ---------------------------------------------------------------------------
// the tile kernel
// ---------------------------------------------------------------------------
constexpr int kTileM = 256, kTileN = 256, kTileK = 64;   // of a pair of CTAs
constexpr int kStages = 6;                               // 32 KB each
constexpr int kStageBytes = 32768, kHalf = 16384;        // A and B halves of a CTA
constexpr int kThreads = 192;                            // loader, MMA, four epilogue warps
constexpr int kTileSmem = kStages * kStageBytes + 1024 + 256;

enum TileMode { kFwd, kDz, kDx, kDw };

struct XentArgs {
  int rows;          // kFwd: all rows; else the rows of the workspace's capacity
  int rows_pad;      // rows rounded up to 256
  int H;
  int vocab;
  int v0;            // first column of this piece of the vocabulary
  int chunk;         // columns of a chunk (a multiple of 256)
  int chunks;        // chunks of this piece
  int ld;            // columns of dz: chunk * chunks
  float cap;         // 0: none
  float inv_cap;
  const int64_t* target;   // kFwd
  const float* head;       // backward: [0] kept rows (int), [1] dz scale, [2] 1 / scale
  const int* tgt_k;        // backward, by kept row: target,
  const float* lse_k;      //   lse
  const float* g_k;        //   dnll * scale
  float2* part;            // kFwd: [tiles][rows_pad] (max, sum)
  float* zt;               // kFwd: [rows_pad] the target's s
  void* dz;                // kDz: [rows_pad][ld]
  float* slab;             // kDx: [chunks][rows_pad][H]
  void* dw;                // kDw: [vocab][H]
};

// Set when a wait in k_xent_tile ran out: from then on the operator's results
// on this device are NaN (see k_xent_join and k_xent_fold).
__device__ uint32_t g_wait_failed;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {   // 2 units in the last place
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// r = 1 / (1 + e^(2u)): tanh(u) = 1 - 2r and 1 - tanh(u)^2 = 4r(1 - r); the
// absolute error of both is a few 2^-24
__device__ __forceinline__ float half_tail(float u) {
  float r;
  const float d = 1.0f + exp2_approx(u * (2.0f * kLog2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d));
  return r;
}

struct TileAt {
  int m0, n0, kblocks, k0;   // k0: first K coordinate of A; kb0 of B differs by mode
  int chunk;
};

template <int MODE>
__device__ __forceinline__ int tile_count(const XentArgs& a, int kept, int& mt, int& nt) {
  if (MODE == kFwd) {
    mt = (a.rows + kTileM - 1) / kTileM;
    nt = (a.vocab + kTileN - 1) / kTileN;
    return mt * nt;
  }
  if (MODE == kDz) {
    const int cols = a.vocab - a.v0 < a.ld ? a.vocab - a.v0 : a.ld;
    mt = (kept + kTileM - 1) / kTileM;
    // every chunk's K blocks are read whole: columns up to the next multiple of
    // 256 are written (zeros past the vocabulary)
    nt = (cols + kTileN - 1) / kTileN;
    return mt * nt;
  }
  if (MODE == kDx) {
    mt = (kept + kTileM - 1) / kTileM;
    nt = (a.H + kTileN - 1) / kTileN;
    return mt * nt * a.chunks;
  }
  const int cols = a.vocab - a.v0 < a.ld ? a.vocab - a.v0 : a.ld;
  mt = (cols + kTileM - 1) / kTileM;
  nt = (a.H + kTileN - 1) / kTileN;
  return mt * nt;
}

template <int MODE>
__device__ __forceinline__ TileAt tile_at(const XentArgs& a, int t, int kept, int mt, int nt) {
  TileAt p;
  p.chunk = 0;
  p.k0 = 0;
  if (MODE == kFwd || MODE == kDz) {   // the row tiles of one column tile follow each other
    p.m0 = (t % mt) * kTileM;
    p.n0 = (t / mt) * kTileN;
    p.kblocks = (a.H + kTileK - 1) / kTileK;
  } else if (MODE == kDx) {
    p.n0 = (t % nt) * kTileN;
    p.m0 = (t / nt % mt) * kTileM;
    p.chunk = t / nt / mt;
    p.k0 = p.chunk * a.chunk;
    const int left = a.vocab - a.v0 - p.k0;
    p.kblocks = ((left < a.chunk ? left : a.chunk) + kTileK - 1) / kTileK;
  } else {
    p.n0 = (t % nt) * kTileN;
    p.m0 = (t / nt) * kTileM;
    p.kblocks = (kept + kTileK - 1) / kTileK;
  }
  return p;
}

// Warp 0 loads the operands' tiles by TMA into a ring of stages, warp 1 of the
// even CTA issues the MMAs of the pair, warps 2 to 5 read the accumulator (256
// columns of tensor memory, two of them so that the next tile's products run
// meanwhile) and finish the tile.  One pair of CTAs per two SMs walks the tiles
// with a fixed stride.
template <int DT, int MODE, bool CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_xent_tile(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const XentArgs a) {
  using F = Fmt<DT>;
  constexpr bool kAmn = MODE == kDw, kBmn = MODE == kDx || MODE == kDw;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kStages * kStageBytes;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto acc_full = [&](int b) { return bars + 8 * (2 * kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };
  const uint32_t tmem_slot = bars + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  uint32_t* err = &g_wait_failed;

  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 8);   // the epilogue warps of both CTAs
    }
    mbar_init_fence();
  }
  __syncwarp();
  if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  uint32_t tmem;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(tmem) : "r"(tmem_slot));
  griddep_trigger();
  griddep_wait();

  const int kept = MODE == kFwd ? a.rows : __float_as_int(__ldcg(a.head));
  int mt, nt;
  const int tiles = tile_count<MODE>(a, kept, mt, nt);

  if (warp == 0) {
    if (lane == 0) {
      int it = 0;   // K blocks loaded so far
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs) {
        const TileAt p = tile_at<MODE>(a, t, kept, mt, nt);
        const int am = p.m0 + int(rank) * 128, bn = p.n0 + int(rank) * 128;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % kStages;
          ok = mbar_wait(empty(s), ((it / kStages) & 1) ^ 1, err);
          if (!ok) break;
          if (rank == 0) mbar_expect_tx(full(s), 2 * kStageBytes);
          const uint32_t sa = base + s * kStageBytes, sb = sa + kHalf;
          const int k = kb * kTileK;
          if (MODE == kFwd) {
            tma_load_pair(sa, &map_a, k, am, full(s));
            tma_load_pair(sb, &map_b, k, bn, full(s));
          } else if (MODE == kDz) {
            tma_load_pair(sa, &map_a, k, am, full(s));
            tma_load_pair(sb, &map_b, k, a.v0 + bn, full(s));
          } else if (MODE == kDx) {   // A: dz by rows; B: W, H contiguous
            tma_load_pair(sa, &map_a, p.k0 + k, am, full(s));
            tma_load_pair(sb, &map_b, bn, a.v0 + p.k0 + k, full(s));
            tma_load_pair(sb + 8192, &map_b, bn + 64, a.v0 + p.k0 + k, full(s));
          } else {                    // A: dz, columns contiguous; B: x, H contiguous
            tma_load_pair(sa, &map_a, am, k, full(s));
            tma_load_pair(sa + 8192, &map_a, am + 64, k, full(s));
            tma_load_pair(sb, &map_b, bn, k, full(s));
            tma_load_pair(sb + 8192, &map_b, bn + 64, k, full(s));
          }
        }
      }
      // after a failed wait: no copy may be in flight when the CTA ends
      if (!ok && rank == 0)
        for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
          (void)mbar_wait(full(i % kStages), (i / kStages) & 1, err);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = mma_desc(DT == RN_BF16, kTileM, kTileN, kAmn, kBmn);
      int it = 0, n = 0;
      bool ok = true;
      for (int t = pair; t < tiles && ok; t += pairs, ++n) {
        const TileAt p = tile_at<MODE>(a, t, kept, mt, nt);
        const int b = n & 1;
        ok = mbar_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, err);
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % kStages;
          ok = mbar_wait(full(s), (it / kStages) & 1, err);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = base + s * kStageBytes;
          const uint64_t da = smem_desc(sa, kAmn), db = smem_desc(sa + kHalf, kBmn);
#pragma unroll
          for (int k = 0; k < kTileK / 16; ++k)   // 16 K: 32 bytes of a row, or 16 rows of 128
            mma_pair(tmem + b * kTileN, da + k * (kAmn ? 128 : 2), db + k * (kBmn ? 128 : 2), idesc,
                     kb > 0 || k > 0);
          mma_commit_pair(empty(s));
        }
        if (ok) mma_commit_pair(acc_full(b));
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;   // the quarter of tensor memory this warp may read
    const uint32_t lanes = tmem + (uint32_t(q * 32) << 16);
    const int my_row = int(rank) * 128 + q * 32 + lane;
    int n = 0;
    for (int t = pair; t < tiles; t += pairs, ++n) {
      const TileAt p = tile_at<MODE>(a, t, kept, mt, nt);
      const int b = n & 1;
      const int row = p.m0 + my_row;
      if (!__all_sync(0xffffffffu, mbar_wait(acc_full(b), (n >> 1) & 1, err))) break;
      tc_fence_after();
      const uint32_t acc = lanes + b * kTileN;

      if constexpr (MODE == kFwd) {
        const bool act = row < a.rows;
        const int64_t tg = act ? __ldg(a.target + row) : -1;
        const int at = tg >= p.n0 && tg < p.n0 + kTileN && tg < a.vocab ? int(tg - p.n0) : -1;
        const int cols = a.vocab - p.n0;   // valid columns when less than 256
        float m = -INFINITY, sum = 0.0f;
        for (int c = 0; c < kTileN; c += 32) {
          uint32_t r[32];
          tmem_ld32(acc + c, r);
          tmem_ld_wait();
          float z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            z[i] = __uint_as_float(r[i]);
            if (CAP) z[i] = a.cap * fmaf(-2.0f, half_tail(z[i] * a.inv_cap), 1.0f);
          }
          if (c + 32 > cols) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i >= cols) z[i] = -INFINITY;
          }
          if (unsigned(at - c) < 32u) {
            float zt = 0.0f;
#pragma unroll
            for (int i = 0; i < 32; ++i) zt = at - c == i ? z[i] : zt;
            a.zt[row] = zt;
          }
          float mc[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int i = 4; i < 32; ++i) mc[i & 3] = fmaxf(mc[i & 3], z[i]);
          const float mn = fmaxf(m, fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3])));
          float2 s2[2] = {bc2(0.0f), bc2(0.0f)};
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 e = mul2(add2(make_float2(z[i], z[i + 1]), bc2(-mn)), bc2(kLog2e));
            s2[(i >> 1) & 1] = add2(s2[(i >> 1) & 1], make_float2(exp2_approx(e.x), exp2_approx(e.y)));
          }
          const float sc = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
          // m is -inf before the first columns only: exp2 of -inf is 0
          sum = c == 0 ? sc : fmaf(sum, exp2_approx((m - mn) * kLog2e), sc);
          m = mn;
        }
        if (act) a.part[int64_t(p.n0 / kTileN) * a.rows_pad + row] = make_float2(m, sum);
      } else if constexpr (MODE == kDz) {
        const bool act = row < kept;
        const int tg = act ? __ldcg(a.tgt_k + row) - a.v0 - p.n0 : -1;
        const float lse = act ? __ldcg(a.lse_k + row) : 0.0f;
        const float g = act ? __ldcg(a.g_k + row) : 0.0f;
        const int cols = a.vocab - a.v0 - p.n0;
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dz) + int64_t(row) * a.ld + p.n0);
        for (int c = 0; c < kTileN; c += 32) {
          uint32_t r[32];
          tmem_ld32(acc + c, r);
          tmem_ld_wait();
          float d[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float z = __uint_as_float(r[i]), slope = g;
            if (CAP) {
              const float h = half_tail(z * a.inv_cap);
              z = a.cap * fmaf(-2.0f, h, 1.0f);
              slope *= 4.0f * h * (1.0f - h);
            }
            const float prob = exp2_approx((z - lse) * kLog2e);
            d[i] = slope * (tg == c + i ? prob - 1.0f : prob);
            if (!act || c + i >= cols) d[i] = 0.0f;   // no row, or no column: exactly nothing
          }
#pragma unroll
          for (int v = 0; v < 4; ++v)
            dst[c / 8 + v] = make_uint4(F::pack2(d[8 * v], d[8 * v + 1]), F::pack2(d[8 * v + 2], d[8 * v + 3]),
                                        F::pack2(d[8 * v + 4], d[8 * v + 5]), F::pack2(d[8 * v + 6], d[8 * v + 7]));
        }
      } else if constexpr (MODE == kDx) {
        float4* dst = reinterpret_cast<float4*>(a.slab + (int64_t(p.chunk) * a.rows_pad + row) * a.H + p.n0);
        for (int c = 0; c < kTileN && p.n0 + c < a.H; c += 32) {
          uint32_t r[32];
          tmem_ld32(acc + c, r);
          tmem_ld_wait();
          if (row < kept) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              if (p.n0 + c + 4 * v < a.H)
                dst[c / 4 + v] = make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                             __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
          }
        }
      } else {
        const int64_t v_row = int64_t(a.v0) + row;
        const bool act = row < a.ld && v_row < a.vocab;
        const float inv = __ldcg(a.head + 2);
        uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.dw) + v_row * a.H + p.n0);
        for (int c = 0; c < kTileN && p.n0 + c < a.H; c += 32) {
          uint32_t r[32];
          tmem_ld32(acc + c, r);
          tmem_ld_wait();
          if (p.kblocks == 0) {   // no kept row: the accumulator was never written
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = 0;
          }
          if (act) {
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(r[8 * v + i]) * inv;
              if (p.n0 + c + 8 * v < a.H)
                dst[c / 8 + v] = make_uint4(F::pack2(f[0], f[1]), F::pack2(f[2], f[3]), F::pack2(f[4], f[5]),
                                            F::pack2(f[6], f[7]));
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_at(acc_empty(b), 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // every product is read and every arrival made
  if (warp == 1) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// forward: joins a row's tile statistics.  32 rows of a CTA by eight groups of
// tiles (group j takes tiles j, j + 8, ...), joined by the pairwise tree.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {   // (max, sum)
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, a.y + b.y);
  return make_float2(m, fmaf(a.y, exp2_approx((a.x - m) * kLog2e), b.y * exp2_approx((b.x - m) * kLog2e)));
}

__global__ void __launch_bounds__(256)
k_xent_join(int rows, int rows_pad, int tiles, int vocab, const float2* __restrict__ part,
            const float* __restrict__ zt, const int64_t* __restrict__ target, float* __restrict__ nll,
            float* __restrict__ lse) {
  griddep_trigger();
  griddep_wait();
  __shared__ float2 sm[8][32];
  const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float2 s = make_float2(-INFINITY, 0.0f);
  if (row < rows) {
    for (int t0 = j; t0 < tiles; t0 += 8 * 8) {   // eight loads in flight
      float2 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = t0 + 8 * i < tiles ? __ldcg(part + int64_t(t0 + 8 * i) * rows_pad + row) : make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (t0 + 8 * i < tiles) s = join_stats(s, v[i]);
    }
  }
  sm[j][lane] = s;
  __syncthreads();
  if (j == 0 && row < rows) {
    float2 p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = sm[i][lane];
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
#pragma unroll
      for (int i = 0; i + d < 8; i += 2 * d) p[i] = join_stats(p[i], p[i + d]);
    const float l = logf(p[0].y);
    const int64_t t = target[row];
    const bool failed = __ldcg(&g_wait_failed) != 0;
    // (max - s[target]) + log(sum): no cancellation where the target is likely
    const float loss = t >= 0 && t < vocab ? (p[0].x - zt[row]) + l : 0.0f;
    if (nll) nll[row] = failed ? NAN : loss;
    if (lse) lse[row] = failed ? NAN : p[0].x + l;
  }
}

// ---------------------------------------------------------------------------
// backward: the rows that carry a loss, listed in order by one CTA, and the
// power of two that dz is scaled by (fp16 only: dz is at most max |dnll|, and
// 2^15 / that keeps small probabilities out of fp16's subnormals; bf16 has
// fp32's exponents and takes 1)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024)
k_xent_scan(int rows, int vocab, int fp16, const int64_t* __restrict__ target,
            const float* __restrict__ dnll, float* __restrict__ head, int* __restrict__ pos,
            int* __restrict__ kept_row) {
  griddep_trigger();
  griddep_wait();
  __shared__ int warp_sum[32];
  __shared__ float warp_max[32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  int done = 0;
  float top = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += 1024) {
    const int r = r0 + tid;
    bool keep = false;
    if (r < rows) {
      const int64_t t = __ldg(target + r);
      keep = t >= 0 && t < vocab;
      if (keep) top = fmaxf(top, fabsf(__ldg(dnll + r)));
    }
    const unsigned b = __ballot_sync(0xffffffffu, keep);
    if (lane == 0) warp_sum[w] = __popc(b);
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < 32; ++i) {
      const int n = warp_sum[i];
      before += i < w ? n : 0;
      all += n;
    }
    const int at = done + before + __popc(b & ((1u << lane) - 1u));
    if (r < rows) pos[r] = keep ? at : kIgnored;
    if (keep) kept_row[at] = r;
    done += all;
    __syncthreads();
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) warp_max[w] = top;
  __syncthreads();
  if (tid == 0) {
    for (int i = 1; i < 32; ++i) top = fmaxf(top, warp_max[i]);
    int e = 0;
    if (fp16 && top > 0.0f && top < INFINITY) {
      (void)frexpf(top, &e);               // top <= 2^e
      e = 15 - e;
      e = e < -100 ? -100 : (e > 100 ? 100 : e);
    }
    head[0] = __int_as_float(done);
    head[1] = ldexpf(1.0f, e);
    head[2] = ldexpf(1.0f, -e);
  }
}

// The kept rows of x next to each other, and their targets, lse and scaled
// gradients; the rows up to the next multiple of 256 are zero (they are read as
// parts of tiles).
__global__ void __launch_bounds__(256)
k_xent_gather(int rows_pad, int nv, const int* __restrict__ kept_row, const float* __restrict__ head,
              const uint4* __restrict__ x, const int64_t* __restrict__ target,
              const float* __restrict__ lse, const float* __restrict__ dnll, uint4* __restrict__ xk,
              int* __restrict__ tgt_k, float* __restrict__ lse_k, float* __restrict__ g_k) {
  griddep_trigger();
  griddep_wait();
  const int kept = __float_as_int(__ldcg(head));
  const float scale = __ldcg(head + 1);
  const int end = (kept + kTileM - 1) / kTileM * kTileM;
  for (int i = blockIdx.x * 8 + (threadIdx.x >> 5); i < end; i += gridDim.x * 8) {
    const int lane = threadIdx.x & 31;
    const int r = i < kept ? __ldcg(kept_row + i) : -1;
    for (int v0 = lane; v0 < nv; v0 += 32 * 4) {
      uint4 u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = r >= 0 && v0 + 32 * j < nv ? __ldg(x + int64_t(r) * nv + v0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v0 + 32 * j < nv) xk[int64_t(i) * nv + v0 + 32 * j] = u[j];
    }
    if (lane == 0 && r >= 0) {
      tgt_k[i] = int(target[r]);
      lse_k[i] = lse[r];
      g_k[i] = dnll[r] * scale;
    }
  }
}

// ---------------------------------------------------------------------------
// backward: dx from the chunks' products, added in ascending order.  Not the
// last piece: acc = (acc +) slab 0 + slab 1 + ... by kept row.  Last piece: the
// same sum, unscaled, rounded and put at the rows' own places, zeros for rows
// without a loss.
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(256)
k_xent_fold(int rows, int rows_pad, int H, int chunks, int first, int last, const float* __restrict__ slab,
            float* __restrict__ acc, const float* __restrict__ head, const int* __restrict__ pos,
            uint4* __restrict__ dx) {
  using F = Fmt<DT>;
  griddep_trigger();
  griddep_wait();
  const int kept = __float_as_int(__ldcg(head));
  const float inv = __ldcg(head + 2);
  const bool failed = __ldcg(&g_wait_failed) != 0;
  const int nv = H / 8;
  const int64_t n = int64_t(last ? rows : kept) * nv;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < n; i += int64_t(gridDim.x) * 256) {
    const int r = int(i / nv), v = int(i % nv);
    const int k = last ? __ldcg(pos + r) : r;
    float4 s[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    if (k >= 0) {
      const int64_t at = (int64_t(k) * H + v * 8) / 4, step = int64_t(rows_pad) * H / 4;
      const float4* p = reinterpret_cast<const float4*>(slab) + at;
      float4* q = reinterpret_cast<float4*>(acc) + at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s[h] = __ldcs(p + h);
        if (!first) s[h] = add4(q[h], s[h]);
        for (int c = 1; c < chunks; ++c) s[h] = add4(s[h], __ldcs(p + c * step + h));
        if (!last) q[h] = s[h];
      }
    }
    if (last) {
      float2 f[4] = {make_float2(s[0].x, s[0].y), make_float2(s[0].z, s[0].w), make_float2(s[1].x, s[1].y),
                     make_float2(s[1].z, s[1].w)};
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = failed ? bc2(NAN) : mul2(f[e], bc2(inv));
      dx[i] = F::pack2v(f);
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static std::atomic<void*> cached{nullptr};
  void* f = cached.load();
  if (f == nullptr) {
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      (void)cudaGetLastError();
      return nullptr;
    }
    cached.store(f);
  }
  return reinterpret_cast<EncodeTiled>(f);
}

// A row-major matrix of 16-bit elements read in boxes of 64 columns (128 bytes,
// swizzled) by `box_rows` rows; what lies outside reads as zero.
rn_status make_map(CUtensorMap* map, rn_dtype dt, const void* p, int64_t rows, int64_t cols, int64_t ld,
                   int box_rows) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return cuda_failed(int(cudaErrorNotSupported));
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * 2};
  const cuuint32_t box[2] = {64, cuuint32_t(box_rows)}, steps[2] = {1, 1};
  const CUresult e =
      enc(map, dt == RN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? RN_OK : cuda_failed(int(cudaErrorInvalidValue));
}

template <int DT, int MODE, bool CAP>
rn_status launch_tile(const CUtensorMap& ma, const CUtensorMap& mb, const XentArgs& a, int64_t most_tiles,
                      cudaStream_t st) {
  static KernelPrep prep;
  (void)prepare_kernel(k_xent_tile<DT, MODE, CAP>, kThreads, kTileSmem, prep);
  const int64_t pairs = sm_count() / 2;
  const int64_t want = most_tiles < pairs ? most_tiles : pairs;
  return launch_pdl(k_xent_tile<DT, MODE, CAP>, dim3(unsigned(2 * (want < 1 ? 1 : want))), dim3(kThreads),
                    kTileSmem, st, ma, mb, a);
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// carves a workspace into 256-byte aligned pieces
struct Carve {
  uintptr_t p, p0;
  explicit Carve(void* base) : p(reinterpret_cast<uintptr_t>(base)), p0(p) {}
  template <typename T>
  T* take(int64_t n) {
    T* q = reinterpret_cast<T*>(p);
    p += (size_t(n) * sizeof(T) + 255) & ~size_t(255);
    return q;
  }
  size_t bytes() const { return size_t(p - p0); }
};

struct FwdWs {
  float2* part;
  float* zt;
  size_t bytes;
};
FwdWs xent_fwd_ws(void* base, int64_t rows, int64_t vocab) {
  Carve c(base);
  FwdWs w;
  const int64_t rp = up(rows, kTileM);
  w.part = c.take<float2>(ceil_div(vocab, kTileN) * rp);
  w.zt = c.take<float>(rp);
  w.bytes = c.bytes();
  return w;
}

// The vocabulary in chunks of at most 16384 columns (dx is summed over them, so
// the size depends on V only); a piece is as many chunks as keep dz within
// 256 MB, at least one.
constexpr int64_t kMostChunk = 16384;
constexpr int64_t kDzBudget = int64_t(256) << 20;
struct BwdPlan {
  int64_t rows_pad;
  int chunk, chunks, per_piece, pieces;
};
BwdPlan xent_plan(int64_t rows, int64_t vocab) {
  BwdPlan p;
  p.rows_pad = up(rows, kTileM);
  p.chunk = int(up(ceil_div(vocab, ceil_div(vocab, kMostChunk)), 256));
  p.chunks = int(ceil_div(vocab, p.chunk));
  const int64_t fit = kDzBudget / (p.rows_pad * p.chunk * 2);
  const int64_t g = fit < 1 ? 1 : (fit < p.chunks ? fit : p.chunks);
  p.pieces = int(ceil_div(p.chunks, g));
  p.per_piece = int(ceil_div(p.chunks, p.pieces));
  p.pieces = int(ceil_div(p.chunks, p.per_piece));
  return p;
}
struct BwdWs {
  float* head;
  int* pos;
  int* kept_row;
  int* tgt_k;
  float* lse_k;
  float* g_k;
  uint16_t* xk;
  uint16_t* dz;
  float* slab;
  float* acc;
  size_t bytes;
};
BwdWs xent_bwd_ws(void* base, int64_t rows, int width, const BwdPlan& p) {
  Carve c(base);
  BwdWs w;
  w.head = c.take<float>(4);
  w.pos = c.take<int>(rows);
  w.kept_row = c.take<int>(rows);
  w.tgt_k = c.take<int>(p.rows_pad);
  w.lse_k = c.take<float>(p.rows_pad);
  w.g_k = c.take<float>(p.rows_pad);
  w.xk = c.take<uint16_t>(p.rows_pad * width);
  w.dz = c.take<uint16_t>(p.rows_pad * p.chunk * p.per_piece);
  w.slab = c.take<float>(p.rows_pad * width * p.per_piece);
  w.acc = c.take<float>(p.pieces > 1 ? p.rows_pad * width : 0);
  w.bytes = c.bytes();
  return w;
}

bool xent_sizes_ok(int64_t rows, int64_t vocab) {
  return rows >= 0 && rows <= kMaxXentRows && vocab >= 1 && vocab <= kMaxXentVocab;
}

template <int DT>
rn_status run_xent_fwd(int64_t rows, int width, int64_t vocab, const void* x, const void* w,
                       const int64_t* target, float cap, float* nll, float* lse, void* ws, cudaStream_t st) {
  const FwdWs f = xent_fwd_ws(ws, rows, vocab);
  CUtensorMap mx, mw;
  rn_status e = make_map(&mx, rn_dtype(DT), x, rows, width, width, 128);
  if (e == RN_OK) e = make_map(&mw, rn_dtype(DT), w, vocab, width, width, 128);
  if (e != RN_OK) return e;
  XentArgs a = {};
  a.rows = int(rows);
  a.rows_pad = int(up(rows, kTileM));
  a.H = width;
  a.vocab = int(vocab);
  a.cap = cap;
  a.inv_cap = cap > 0 ? 1.0f / cap : 0.0f;
  a.target = target;
  a.part = f.part;
  a.zt = f.zt;
  const int64_t tiles = ceil_div(rows, kTileM) * ceil_div(vocab, kTileN);
  e = cap > 0 ? launch_tile<DT, kFwd, true>(mx, mw, a, tiles, st) : launch_tile<DT, kFwd, false>(mx, mw, a, tiles, st);
  if (e != RN_OK) return e;
  return launch_pdl(k_xent_join, dim3(unsigned(ceil_div(rows, 32))), dim3(256), 0, st, a.rows, a.rows_pad,
                    int(ceil_div(vocab, kTileN)), a.vocab, f.part, f.zt, target, nll, lse);
}

template <int DT>
rn_status run_xent_bwd(int64_t rows, int width, int64_t vocab, const void* x, const void* w,
                       const int64_t* target, const float* lse, const float* dnll, float cap, void* dx, void* dw,
                       void* ws, cudaStream_t st) {
  const BwdPlan p = xent_plan(rows, vocab);
  const BwdWs b = xent_bwd_ws(ws, rows, width, p);
  rn_status e = launch_pdl(k_xent_scan, dim3(1), dim3(1024), 0, st, int(rows), int(vocab), int(DT == RN_F16),
                           target, dnll, b.head, b.pos, b.kept_row);
  if (e != RN_OK) return e;
  const int wave = 4 * sm_count();
  const int64_t groups = ceil_div(p.rows_pad, 8);
  e = launch_pdl(k_xent_gather, dim3(unsigned(groups < wave ? groups : wave)), dim3(256), 0, st,
                 int(p.rows_pad), width / 8, b.kept_row, b.head, static_cast<const uint4*>(x), target, lse, dnll,
                 reinterpret_cast<uint4*>(b.xk), b.tgt_k, b.lse_k, b.g_k);
  if (e != RN_OK) return e;
  const int64_t ld = int64_t(p.chunk) * p.per_piece;
  CUtensorMap mx, mw, mdz, mdz_t, mw_n, mx_n;
  e = make_map(&mx, rn_dtype(DT), b.xk, p.rows_pad, width, width, 128);
  if (e == RN_OK) e = make_map(&mw, rn_dtype(DT), w, vocab, width, width, 128);
  if (e == RN_OK) e = make_map(&mdz, rn_dtype(DT), b.dz, p.rows_pad, ld, ld, 128);
  if (e == RN_OK) e = make_map(&mdz_t, rn_dtype(DT), b.dz, p.rows_pad, ld, ld, 64);
  if (e == RN_OK) e = make_map(&mw_n, rn_dtype(DT), w, vocab, width, width, 64);
  if (e == RN_OK) e = make_map(&mx_n, rn_dtype(DT), b.xk, p.rows_pad, width, width, 64);
  if (e != RN_OK) return e;
  XentArgs a = {};
  a.rows = int(rows);
  a.rows_pad = int(p.rows_pad);
  a.H = width;
  a.vocab = int(vocab);
  a.chunk = p.chunk;
  a.ld = int(ld);
  a.cap = cap;
  a.inv_cap = cap > 0 ? 1.0f / cap : 0.0f;
  a.head = b.head;
  a.tgt_k = b.tgt_k;
  a.lse_k = b.lse_k;
  a.g_k = b.g_k;
  a.dz = b.dz;
  a.slab = b.slab;
  a.dw = dw;
  const int64_t mt = p.rows_pad / kTileM, ht = ceil_div(width, kTileN);
  for (int piece = 0; piece < p.pieces; ++piece) {
    const int c0 = piece * p.per_piece;
    a.chunks = p.chunks - c0 < p.per_piece ? p.chunks - c0 : p.per_piece;
    a.v0 = c0 * p.chunk;
    const int64_t vt = int64_t(a.chunks) * (p.chunk / kTileN);
    e = cap > 0 ? launch_tile<DT, kDz, true>(mx, mw, a, mt * vt, st) : launch_tile<DT, kDz, false>(mx, mw, a, mt * vt, st);
    if (e == RN_OK && dw) e = launch_tile<DT, kDw, false>(mdz_t, mx_n, a, vt * ht, st);
    if (e == RN_OK && dx) {
      e = launch_tile<DT, kDx, false>(mdz, mw_n, a, mt * ht * a.chunks, st);
      if (e != RN_OK) return e;
      const bool last = piece + 1 == p.pieces;
      const int64_t n = ceil_div(rows * (width / 8), 256);
      const int64_t cap_grid = int64_t(8) * sm_count();
      e = launch_pdl(k_xent_fold<DT>, dim3(unsigned(n < cap_grid ? n : cap_grid)), dim3(256), 0, st, int(rows),
                     a.rows_pad, width, a.chunks, int(piece == 0), int(last), b.slab, b.acc, b.head, b.pos,
                     static_cast<uint4*>(dx));
    }
    if (e != RN_OK) return e;
  }
  return RN_OK;
}

rn_status xent_checks(int64_t rows, int32_t width, int64_t vocab, rn_dtype dt, float cap) {
  if (!xent_sizes_ok(rows, vocab) || !std::isfinite(cap) || cap < 0.0f) return RN_E_ARG;
  if (dt != RN_BF16 && dt != RN_F16) return RN_E_DTYPE;
  if (!width_ok(width)) return RN_E_WIDTH;
  return RN_OK;
}

}  // namespace

extern "C" {

size_t linear_xent_fwd_workspace_bytes(int64_t rows, int64_t vocab) {
  if (!xent_sizes_ok(rows, vocab) || rows == 0) return 0;
  return xent_fwd_ws(nullptr, rows, vocab).bytes;
}

rn_status linear_xent_fwd(int64_t rows, int32_t width, int64_t vocab, rn_dtype dt, const void* x,
                          const void* w, const int64_t* target, float softcap, float* nll, float* lse,
                          void* ws, size_t ws_bytes, rn_stream stream) {
  begin_call();
  rn_status e = xent_checks(rows, width, vocab, dt, softcap);
  if (e != RN_OK) return e;
  if (!w || (rows > 0 && (!x || !target || (!nll && !lse)))) return RN_E_ARG;
  if (!aligned16(x) || !aligned16(w) || (uintptr_t(target) & 7u) || (uintptr_t(nll) & 3u) || (uintptr_t(lse) & 3u))
    return RN_E_ALIGN;
  const size_t need = linear_xent_fwd_workspace_bytes(rows, vocab);
  if (rows > 0 && (!ws || ws_bytes < need)) return RN_E_WORKSPACE;
  if (!aligned16(ws)) return RN_E_ALIGN;
  const size_t row = size_t(width) * 2, sb = size_t(rows) * 4;
  const Range in[] = {{x, size_t(rows) * row}, {w, size_t(vocab) * row}, {target, size_t(rows) * 8}};
  const Range out[] = {{nll, sb}, {lse, sb}, {ws, need}};
  e = check_ranges(in, 3, out, 3);
  if (e != RN_OK || validate_only() || rows == 0) return e;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dt == RN_BF16 ? run_xent_fwd<RN_BF16>(rows, width, vocab, x, w, target, softcap, nll, lse, ws, st)
                       : run_xent_fwd<RN_F16>(rows, width, vocab, x, w, target, softcap, nll, lse, ws, st);
}

size_t linear_xent_bwd_workspace_bytes(int64_t rows, int32_t width, int64_t vocab) {
  if (!xent_sizes_ok(rows, vocab) || rows == 0 || !width_ok(width)) return 0;
  return xent_bwd_ws(nullptr, rows, width, xent_plan(rows, vocab)).bytes;
}

rn_status linear_xent_bwd(int64_t rows, int32_t width, int64_t vocab, rn_dtype dt, const void* x,
                          const void* w, const int64_t* target, const float* lse, const float* dnll,
                          float softcap, void* dx, void* dw, void* ws, size_t ws_bytes, rn_stream stream) {
  begin_call();
  rn_status e = xent_checks(rows, width, vocab, dt, softcap);
  if (e != RN_OK) return e;
  if (!w || (!dx && !dw) || (rows > 0 && (!x || !target || !lse || !dnll))) return RN_E_ARG;
  if (!aligned16(x) || !aligned16(w) || !aligned16(dx) || !aligned16(dw) || (uintptr_t(target) & 7u) ||
      (uintptr_t(lse) & 3u) || (uintptr_t(dnll) & 3u))
    return RN_E_ALIGN;
  const size_t need = linear_xent_bwd_workspace_bytes(rows, width, vocab);
  if (rows > 0 && (!ws || ws_bytes < need)) return RN_E_WORKSPACE;
  if (!aligned16(ws)) return RN_E_ALIGN;
  const size_t row = size_t(width) * 2, sb = size_t(rows) * 4;
  const Range in[] = {{x, size_t(rows) * row}, {w, size_t(vocab) * row}, {target, size_t(rows) * 8}, {lse, sb}, {dnll, sb}};
  const Range out[] = {{dx, size_t(rows) * row}, {dw, size_t(vocab) * row}, {ws, need}};
  e = check_ranges(in, 5, out, 3);
  if (e != RN_OK || validate_only()) return e;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // no row, no gradient
    if (dw && cudaMemsetAsync(dw, 0, size_t(vocab) * row, st) != cudaSuccess) return cuda_failed(int(cudaGetLastError()));
    return RN_OK;
  }
  return dt == RN_BF16 ? run_xent_bwd<RN_BF16>(rows, width, vocab, x, w, target, lse, dnll, softcap, dx, dw, ws, st)
                       : run_xent_bwd<RN_F16>(rows, width, vocab, x, w, target, lse, dnll, softcap, dx, dw, ws, st);
}

}  // extern "C"
