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
// 128 columns, the maximum and the sum of exponentials), the logits again in
// the backward (the epilogue writes dz, rounded to the element format), dx and
// dW.  The backward takes the vocabulary in pieces whose dz fits the
// workspace.
//
// Order of the sums: a row's statistics are taken over 128 columns each
// and joined in an order that depends on V only; dx is summed over chunks of
// the vocabulary whose size depends on V only, in ascending order.  So nll,
// lse and dx of a row are bitwise the same alone or inside any batch.  dW sums
// the kept rows in order, 16384 at a time in the tensor cores' fp32 accumulator.
#include <cuda.h>

#include <algorithm>
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
// A pair of CTAs computes a tile of 256 x 256, 64 of K a stage.  (256 x 128 for
// shapes of few tiles was no faster a tile: 2048 x 7 rows 177 against 124 us.)
constexpr int kTileM = 256, kTileN = 256, kTileK = 64;
constexpr int kHalf = 16384;                             // a CTA's half of A or B, a stage
constexpr int kStages = 6, kStageBytes = 2 * kHalf;      // 192 KB
constexpr int kThreads = 384;                            // loader, MMA, two idle, eight epilogue warps
constexpr int kOtherRegs = 40, kEpilogueRegs = 224;      // a thread, of the first four warps and the others
constexpr int kOutBytes = 4096;                          // a warp's part of the result: 32 rows of 128 bytes
constexpr int kTileSmem = kStages * kStageBytes + 8 * kOutBytes + 1024 + 256;
constexpr int kRestRow = 32;                             // see kDz
constexpr int kStatCols = 128;                           // columns of one (max, sum) of the forward
// The logits sum K in segments of 1024: the tensor cores cut each addition to
// the accumulator off instead of rounding it, an error that grows with the
// partial sum and the number of steps; the segments' results are added with
// rounding.  Relative error of nll at H = 2048 in one segment 1.1e-6 to 1.5e-6,
// in two half of it, in four (of 512) 2.5e-7; but every accumulator read costs
// the products some 600 cycles (4096 rows: 1.90, 2.0 and 2.19 ms).
constexpr int kSegment = 16;                             // K blocks
// What is cut off is toward zero and so shortens every logit; over n additions
// of 16 products it measured 1.2e-8 to 1.4e-8 n (bf16) and 1.6e-8 n (fp16) of the
// logit for random terms, up to 3.5e-8 n and 9.7e-8 n for terms of one sign.  The
// segments are therefore lengthened by 2^-26 n: nll's relative error at H = 2048
// falls from 4e-7 to 5e-8.  A sum that loses nothing (one-hot rows) is too long by
// it, 64 x 2^-26 = 9.5e-7 of the logit at H >= 1024; one of terms of one sign stays
// too short by up to 1.3e-6 (bf16) or 5.3e-6 (fp16).  The backward forms its logits
// with the same segments and factor: they are the bits that lse was made of, so its
// probabilities add up to 1.  (In one segment without the factor all but the
// target's were too small by the same share: at H = 16384 and logits of 30 in fp16
// 3e-3 for terms of one sign.)
constexpr float kCutOff = 0x1p-26f;
// dW sums the kept rows in segments of 16384 for the same reason (2^19 rows of one
// sign in one segment: 3.3e-3 too small in fp16, 4.5e-3 with its rounding in bf16);
// dx's chunks of the vocabulary are no longer.
constexpr int kGradSegment = 256;                        // K blocks

// kFwd: logits and their statistics; kDz: logits and dz; kGrad: dx and dW of dz
enum TileMode { kFwd, kDz, kGrad };

struct XentArgs {
  int rows;          // kFwd: all rows; else the rows of the workspace's capacity
  int rows_pad;      // rows rounded up to 256
  int x_rows;        // kFwd, kDz: rows of x that a CTA loads for a tile (128, or fewer where there
                     // are fewer in all: the rest of the tile is never looked at)
  int x_odd;         // whether the odd CTA has any
  int H;
  int vocab;
  int v0;            // first column of this piece of the vocabulary
  int chunk;         // columns of a chunk (a multiple of 256)
  int chunks;        // chunks of this piece
  int ld;            // columns of dz: chunk * chunks
  float cap;         // 0: none
  float inv_cap;
  const int64_t* target;   // kFwd
  const float* head;       // backward: [0] kept rows (int), [1] 1 / dz's scale
  const int* tgt_k;        // backward, by kept row: target,
  const float* lse_k;      //   lse
  const float* g_k;        //   dnll * scale,
  const float* zt_k;       //   the target's logit, in fp32 (see warp_dot)
  float* lo_k;             // kDz: what the target's dz was rounded by
  void* dz;                // kDz: [rows_pad][ld]
  float2* part;            // kFwd: [ceil(vocab/128)][rows_pad] (max, sum)
  float* zt;               // kFwd: [rows_pad] the target's s, as the products give it
  float* slab;             // kGrad: [chunks][rows_pad][H], NULL: no dx
  void* dw;                // kGrad: [vocab][H], NULL: no dW
  int dw_32;               // the rows of dW start on 32 bytes
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
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// r = 1 / (1 + e^(2u)): tanh(u) = 1 - 2r and 1 - tanh(u)^2 = 4r(1 - r), the
// absolute error of both a few 2^-24.  For |u| < 1/8 tanh from its series (to u^7,
// the next term is 1.3e-9 of it), so that a cap far above the logits leaves them
// their digits.  Two arguments at a time.
__device__ __forceinline__ float2 tanh2(float2 u, float2* r_out) {
  float2 r;
  const float2 e = mul2(u, bc2(2.0f * kLog2e));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(1.0f + exp2_approx(e.x)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(1.0f + exp2_approx(e.y)));
  const float2 q = mul2(u, u);
  const float2 p = fma2(fma2(bc2(-17.0f / 315.0f), q, bc2(2.0f / 15.0f)), q, bc2(-1.0f / 3.0f));
  const float2 s = fma2(mul2(p, q), u, u), t = fma2(bc2(-2.0f), r, bc2(1.0f));
  *r_out = r;
  return make_float2(fabsf(u.x) < 0.125f ? s.x : t.x, fabsf(u.y) < 0.125f ? s.y : t.y);
}

struct TileAt {
  int m0, n0, kblocks;
  int chunk;      // kGrad: of a dx tile; -1 for a dW tile
};

// The tiles of one pair of CTAs, the j-th at at(j).  kFwd, kDz: every pairs-th, the
// row tiles of one column tile after each other.  kGrad: the dx tiles, whose K is
// a chunk of the vocabulary, are dealt out first; the dW tiles, whose K is the
// kept rows, fill up the pairs that got one dx tile less, so that all pairs have
// about the same number of K blocks (one more a tile for its epilogue, which takes
// as long as five).
template <int MODE>
struct TileWalk {
  int mt, nt, pair, pairs, tiles;
  int my_dx, dw_first, dw_step, my_dw, kept, cols;

  __device__ __forceinline__ TileWalk(const XentArgs& a, int kept_, int pair_, int pairs_)
      : pair(pair_), pairs(pairs_), my_dx(0), dw_first(0), dw_step(1), my_dw(0), kept(kept_) {
    cols = MODE == kFwd ? a.vocab : min(a.vocab - a.v0, a.ld);
    mt = ((MODE == kFwd ? a.rows : kept) + kTileM - 1) / kTileM;
    nt = ((MODE == kGrad ? a.H : cols) + kTileN - 1) / kTileN;   // kDz: the last tile is written whole
    tiles = mt * nt;
    if constexpr (MODE == kGrad) {
      const int dx_tiles = a.slab ? mt * nt * a.chunks : 0;
      const int dw_tiles = a.dw ? (cols + kTileM - 1) / kTileM * nt : 0;
      const int more = dx_tiles % pairs;   // pairs with one dx tile more
      my_dx = dx_tiles / pairs + (pair < more);
      const float lead = float(min(a.chunk, cols) / kTileK + 1) / float(max((kept + kTileK - 1) / kTileK, 5) + 1);
      // dW tiles of a pair with one dx tile more: that dx tile's worth (`lead`) below the others
      const float even = (float(dw_tiles) - float(pairs - more) * lead) / float(pairs);
      const int few = more > 0 && even > 0.0f ? int(even) : 0;
      // each kind of pair walks its part of the tiles side by side (the column
      // tiles of one vocabulary tile share dz, which then comes from L2)
      const int split = min(more * few, dw_tiles);
      const bool lower = pair < more;
      dw_first = lower ? pair : split + pair - more;
      dw_step = lower ? more : pairs - more;
      my_dw = max(0, ((lower ? split : dw_tiles) - dw_first + dw_step - 1) / dw_step);
    }
  }
  __device__ __forceinline__ int count() const {
    if constexpr (MODE == kGrad) return my_dx + my_dw;
    return tiles > pair ? (tiles - pair + pairs - 1) / pairs : 0;
  }
  __device__ __forceinline__ TileAt at(const XentArgs& a, int j) const {
    TileAt p;
    p.chunk = 0;
    if constexpr (MODE == kGrad) {
      if (j < my_dx) {   // the column tiles of one row tile after each other: they share dz
        const int t = pair + j * pairs;
        p.n0 = t % nt * kTileN;
        p.m0 = t / nt % mt * kTileM;
        p.chunk = t / nt / mt;
        p.kblocks = (min(cols - p.chunk * a.chunk, a.chunk) + kTileK - 1) / kTileK;
      } else {
        const int t = dw_first + (j - my_dx) * dw_step;
        p.n0 = t % nt * kTileN;
        p.m0 = t / nt * kTileM;
        p.chunk = -1;
        p.kblocks = (kept + kTileK - 1) / kTileK;
      }
    } else {
      const int t = pair + j * pairs;
      p.m0 = t % mt * kTileM;
      p.n0 = t / mt * kTileN;
      p.kblocks = (a.H + kTileK - 1) / kTileK;
    }
    return p;
  }
};

__device__ __forceinline__ void st_32(void* p, const uint32_t* r) {   // 32 bytes, aligned
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// x . w of two rows, fp32, by a warp; every lane gets it.  A target's logit is
// formed so, apart: the products' own value is short by what the tensor cores cut
// off, and that is what a likely target's loss and gradient consist of.
template <int DT>
__device__ __forceinline__ float warp_dot(const uint4* __restrict__ x, const uint4* __restrict__ w, int nv) {
  using F = Fmt<DT>;
  float2 s = bc2(0.0f);
  for (int v0 = threadIdx.x & 31; v0 < nv; v0 += 32 * 4) {
    uint4 a[4], b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = v0 + 32 * i < nv;
      a[i] = in ? __ldg(x + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
      b[i] = in ? __ldg(w + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f[4], g[4];
      F::unpack2(a[i], f);
      F::unpack2(b[i], g);
#pragma unroll
      for (int q = 0; q < 4; ++q) s = fma2(f[q], g[q], s);
    }
  }
  float t = s.x + s.y;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}
// Warp 0 loads the operands' tiles by TMA into a ring of stages, warp 1 of the
// even CTA issues the MMAs of the pair, and eight warps read the accumulators
// (two of 256 columns in tensor memory, so that the next products run
// meanwhile) and finish the tile, four warps the left half of the columns and
// four the right.
// Tensor maps: kFwd, kDz  a: x, b: W;  kGrad  a: dz (boxes of 128 rows), b: W (boxes
// of 64), c: dz again (boxes of 64), d: x (boxes of 64), e: dW, where it is written
// by TMA.
template <int DT, int MODE, bool CAP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
k_xent_tile(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
            const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_d,
            const __grid_constant__ CUtensorMap map_e, const XentArgs a) {
  using F = Fmt<DT>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kStages * kStageBytes + 8 * kOutBytes;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kStages + s); };
  auto acc_full = [&](int b) { return bars + 8 * (2 * kStages + b); };
  auto acc_empty = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };
  const uint32_t tmem_slot = bars + 8 * (2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cta_rank();
  uint32_t* err = &g_wait_failed;

  if (warp == 0 && lane == 0) {
    tma_prefetch_map(&map_a);
    tma_prefetch_map(&map_b);
    if (MODE == kGrad) {
      tma_prefetch_map(&map_c);
      tma_prefetch_map(&map_d);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(acc_full(b), 1);
      mbar_init(acc_empty(b), 16);   // the epilogue warps of both CTAs
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
  const TileWalk<MODE> walk(a, kept, blockIdx.x >> 1, gridDim.x >> 1);
  const int count = walk.count();
  // accumulators of one tile: segments of K (one where K is empty)
  constexpr int kSeg = MODE == kGrad ? kGradSegment : kSegment;
  auto segments = [](int kblocks) { return max((kblocks + kSeg - 1) / kSeg, 1); };

  // The epilogue holds the sums of 128 columns of its row: its two warpgroups take
  // 224 registers a thread from what the block was launched with (launch_tile checks
  // that these are enough: with fewer the warpgroups would wait for good).
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 0 && lane == 0) {
      const uint32_t bytes = MODE == kGrad ? 2 * kStageBytes
                                           : 2 * kHalf + a.x_rows * 128 * (1 + a.x_odd);   // of both CTAs
      int it = 0;   // K blocks loaded so far
      bool ok = true;
      for (int j = 0; j < count && ok; ++j) {
        const TileAt p = walk.at(a, j);
        const int am = p.m0 + int(rank) * 128, bn = p.n0 + int(rank) * 128;
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int s = it % kStages;
          ok = mbar_wait(empty(s), ((it / kStages) & 1) ^ 1, err);
          if (!ok) break;
          if (rank == 0) mbar_expect_tx(full(s), bytes);
          const uint32_t sa = base + s * kStageBytes, sb = sa + kHalf;
          const int k = kb * kTileK;
          if (MODE != kGrad) {         // x and W by rows
            if (rank == 0 || a.x_odd) tma_load_pair(sa, &map_a, k, am, full(s));
            tma_load_pair(sb, &map_b, k, (MODE == kDz ? a.v0 : 0) + bn, full(s));
          } else if (p.chunk >= 0) {   // dz by rows, W with H contiguous
            const int kc = p.chunk * a.chunk + k;
            tma_load_pair(sa, &map_a, kc, am, full(s));
            tma_load_pair(sb, &map_b, bn, a.v0 + kc, full(s));
            tma_load_pair(sb + 8192, &map_b, bn + 64, a.v0 + kc, full(s));
          } else {                     // dz with its columns contiguous, x with H contiguous
            tma_load_pair(sa, &map_c, am, k, full(s));
            tma_load_pair(sa + 8192, &map_c, am + 64, k, full(s));
            tma_load_pair(sb, &map_d, bn, k, full(s));
            tma_load_pair(sb + 8192, &map_d, bn + 64, k, full(s));
          }
        }
      }
      // after a failed wait: no copy may be in flight when the CTA ends
      if (!ok && rank == 0)
        for (int i = it > kStages ? it - kStages : 0; i < it; ++i)
          (void)mbar_wait(full(i % kStages), (i / kStages) & 1, err);
    } else if (warp == 1 && lane == 0 && rank == 0) {
      int it = 0, n = 0;   // K blocks, accumulators
      bool ok = true;
      for (int j = 0; j < count && ok; ++j) {
        const TileAt p = walk.at(a, j);
        const bool a_mn = MODE == kGrad && p.chunk < 0, b_mn = MODE == kGrad;
        const uint32_t idesc = mma_desc(DT == RN_BF16, kTileM, kTileN, a_mn, b_mn);
        const uint32_t a_step = a_mn ? 128 : 2;   // 16 K: 16 rows of 128 bytes, or 32 bytes of a row
        const int segs = segments(p.kblocks);
        int kb = 0;
        for (int sg = 0; sg < segs && ok; ++sg, ++n) {
          const int b = n & 1, end = sg + 1 < segs ? kb + kSeg : p.kblocks;
          ok = mbar_wait(acc_empty(b), ((n >> 1) & 1) ^ 1, err);
          if (!ok) break;
          tc_fence_after();
          for (bool fresh = true; kb < end; ++kb, ++it, fresh = false) {
            const int s = it % kStages;
            ok = mbar_wait(full(s), (it / kStages) & 1, err);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = base + s * kStageBytes;
            const uint64_t da = smem_desc(sa, a_mn), db = smem_desc(sa + kHalf, b_mn);
#pragma unroll
            for (int k = 0; k < kTileK / 16; ++k)
              mma_pair(tmem + b * kTileN, da + k * a_step, db + k * (b_mn ? 128 : 2), idesc, !fresh || k > 0);
            mma_commit_pair(empty(s));
          }
          if (ok) mma_commit_pair(acc_full(b));
        }
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegs));
    const int q = warp & 3;                 // the quarter of tensor memory this warp may read
    const int c0 = ((warp - 4) >> 2) * 128;
    const uint32_t lanes = tmem + (uint32_t(q * 32) << 16) + c0;
    const int my_row = int(rank) * 128 + q * 32 + lane;
    const uint32_t out = base + kStages * kStageBytes + (warp - 4) * kOutBytes;
    // A dz, dx or dW tile: a thread holds a row of it and stores 32 bytes at a time.
    // Where dW's rows start on 16 bytes only, it leaves through shared memory by
    // TMA instead (16-byte stores against it: 509 x 1032 x 32771 step 205 and 188 us;
    // for rows on 32 bytes TMA was up to 4% slower).
    // A row of the warp's 32 x 32 words, its 16-byte pieces swizzled as the tensor
    // map says, into the warp's buffer; then one lane stores the box at (c0, c1).
    auto store_box = [&](const CUtensorMap* map, const uint32_t (&w)[32], int c0, int c1, bool inside) {
      if (lane == 0) tma_store_wait_read();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(out + lane * 128 + ((i ^ (lane & 7)) << 4)),
                     "r"(w[4 * i]), "r"(w[4 * i + 1]), "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
      async_proxy_fence();
      __syncwarp();
      if (lane == 0 && inside) tma_store(map, out, c0, c1);
    };
    int n = 0;   // accumulators
    bool ok = true;
    for (int j = 0; j < count && ok; ++j) {
      const TileAt p = walk.at(a, j);
      const int segs = segments(p.kblocks);
      const int row = p.m0 + my_row, col0 = p.n0 + c0;   // this thread's row, its first column
      auto wait_acc = [&]() {
        ok = __all_sync(0xffffffffu, mbar_wait(acc_full(n & 1), (n >> 1) & 1, err));
        tc_fence_after();
        return ok;
      };
      auto free_acc = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_at(acc_empty(n & 1), 0);
        ++n;
      };

      // The logits stand in the accumulators over k0, the full segments' factor (of the
      // only one where there is one), the last one's over k0 / rest.
      const int last_k = a.H - (segs - 1) * kSegment * kTileK;
      const float k0 = 1.0f + kCutOff * float((segs > 1 ? kSegment * kTileK : a.H) / 16);
      const float rest = 1.0f - kCutOff * float((a.H - last_k > 0 ? kSegment * kTileK - last_k : 0) / 16);
      // z: the sum of the first `count` >= 1 of the tile's accumulators, this thread's
      // row and 128 columns
      auto read_sums = [&](float (&z)[kStatCols], int count) {
        if (!wait_acc()) return;
#pragma unroll
        for (int c = 0; c < kStatCols; c += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + (n & 1) * kTileN + c, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) z[c + i] = __uint_as_float(r[i]);
        }
        free_acc();
        for (int sg = 1; sg < count; ++sg) {
          if (!wait_acc()) return;
          const float f = MODE == kGrad || sg + 1 < segs ? 1.0f : rest;
#pragma unroll
          for (int c = 0; c < kStatCols; c += 32) {
            uint32_t r[32];
            tmem_ld32(lanes + (n & 1) * kTileN + c, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) z[c + i] = fmaf(__uint_as_float(r[i]), f, z[c + i]);
          }
          free_acc();
        }
      };

      if constexpr (MODE == kFwd) {
        float z[kStatCols];
        read_sums(z, segs);
        if (!ok) break;
        const int cols = a.vocab - col0;   // valid columns when less than 128
        if (CAP) {
#pragma unroll
          for (int i = 0; i < kStatCols; i += 2) {
            float2 r;
            const float2 s = mul2(bc2(a.cap), tanh2(mul2(make_float2(z[i], z[i + 1]), bc2(a.inv_cap * k0)), &r));
            z[i] = s.x;
            z[i + 1] = s.y;
          }
        }
        if (cols < kStatCols) {
#pragma unroll
          for (int i = 0; i < kStatCols; ++i)
            if (i >= cols) z[i] = -INFINITY;
        }
        const bool act = row < a.rows;
        const int64_t tg = act ? __ldg(a.target + row) : -1;
        if (tg >= col0 && tg < col0 + kStatCols && tg < a.vocab) {
          const int at = int(tg - col0);
          float zt = 0.0f;
#pragma unroll
          for (int i = 0; i < kStatCols; ++i) zt = at == i ? z[i] : zt;
          a.zt[row] = CAP ? zt : zt * k0;
        }
        if (act && cols > 0) {
          float mc[4] = {z[0], z[1], z[2], z[3]};
#pragma unroll
          for (int i = 4; i + 8 <= kStatCols; i += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k) mc[k] = max3(mc[k], z[i + k], z[i + 4 + k]);
#pragma unroll
          for (int k = 0; k < 4; ++k) mc[k] = fmaxf(mc[k], z[kStatCols - 4 + k]);
          const float m = fmaxf(fmaxf(mc[0], mc[1]), fmaxf(mc[2], mc[3]));
          // exp(z - m) as 2^(z log2e - t) with t = m log2e rounded: one multiply-add
          // an element; what t was rounded by, r, is common to all and taken out of
          // the sum (so the largest element counts as exactly 1)
          // (a maximum of -inf is put to 0: every exponential is of -inf)
          const float top = m == -INFINITY ? 0.0f : m;
          const float l2 = CAP ? kLog2e : kLog2e * k0;
          const float t = top * l2, r = fmaf(top, l2, -t);
          float2 s2[4] = {bc2(0.0f), bc2(0.0f), bc2(0.0f), bc2(0.0f)};
#pragma unroll
          for (int i = 0; i < kStatCols; i += 2) {
            const float2 e = fma2(make_float2(z[i], z[i + 1]), bc2(l2), bc2(-t));
            s2[(i >> 1) & 3] = __fadd2_rn(s2[(i >> 1) & 3], make_float2(exp2_approx(e.x), exp2_approx(e.y)));
          }
          const float2 u2 = __fadd2_rn(__fadd2_rn(s2[0], s2[1]), __fadd2_rn(s2[2], s2[3]));
          const float u = (u2.x + u2.y) * exp2_approx(-r);
          a.part[int64_t(col0 / kStatCols) * a.rows_pad + row] = make_float2(CAP ? m : m * k0, u);
        }
      } else if constexpr (MODE == kDz) {
        // With at most 32 kept rows, row 32 + k holds what the target's dz of row k
        // was rounded by (x stands there again): it costs nothing in dW's first 64
        // rows of K, where few rows would not average the rounding out.
        const bool act = row < kept, again = kept <= kRestRow && row >= kRestRow && row < kRestRow + kept;
        const int k = again ? row - kRestRow : row;
        const int target = act || again ? __ldcg(a.tgt_k + k) : -1, tg = target - a.v0 - col0;
        // exp(z - lse) as 2^(z log2e - lse2), and what lse2 was rounded by in the
        // factor (a likely target's p - 1 would lose digits to it)
        const float lse = act || again ? __ldcg(a.lse_k + k) : 0.0f, lse2 = lse * kLog2e;
        const float g = act || again ? __ldcg(a.g_k + k) : 0.0f;
        const float gp = g * exp2_approx(-fmaf(lse, kLog2e, -lse2));
        const int cols = a.vocab - a.v0 - col0;
        const bool here = target >= 0 && unsigned(tg) < 128u;
        uint16_t* dst = static_cast<uint16_t*>(a.dz) + int64_t(row) * a.ld + col0;
        // the target's dz, from its own logit, and what it is rounded by
        float dt = 0.0f, lo = 0.0f;
        if (here) {
          float2 z = bc2(__ldcg(a.zt_k + k)), f = bc2(1.0f);
          if (CAP) {
            float2 h;
            z = mul2(bc2(a.cap), tanh2(mul2(z, bc2(a.inv_cap)), &h));
            f = mul2(mul2(bc2(4.0f), h), fma2(h, bc2(-1.0f), bc2(1.0f)));
          }
          dt = (gp * exp2_approx(fmaf(z.x, kLog2e, -lse2)) - g) * f.x;
          lo = dt - F::pair(F::pack2(dt, 0.0f)).x;
          if (act) a.lo_k[row] = lo;
        }
        float zs[kStatCols];
        // the last accumulator is read as it is used: read whole, as the others and as in the
        // forward, 4096 x 1024 x 50000 took 344 us and not 281
        if (segs > 1) read_sums(zs, segs - 1);
        if (!ok || !wait_acc()) break;
        const float l2 = CAP ? kLog2e : kLog2e * k0;
#pragma unroll
        for (int c = 0; c < kStatCols; c += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + (n & 1) * kTileN + c, r);
          tmem_ld_wait();
          if (segs > 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(fmaf(__uint_as_float(r[i]), rest, zs[c + i]));
          }
          float2 d[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 z = make_float2(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1])), slope = bc2(gp);
            if (CAP) {
              float2 h;
              z = mul2(bc2(a.cap), tanh2(mul2(z, bc2(a.inv_cap * k0)), &h));
              slope = mul2(slope, mul2(mul2(bc2(4.0f), h), fma2(h, bc2(-1.0f), bc2(1.0f))));
            }
            const float2 e = fma2(z, bc2(l2), bc2(-lse2));
            d[i] = mul2(slope, make_float2(exp2_approx(e.x), exp2_approx(e.y)));
          }
          if (!act || cols < c + 32) {    // no row, or no column: exactly nothing
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (!act || c + 2 * i >= cols) d[i].x = 0.0f;
              if (!act || c + 2 * i + 1 >= cols) d[i].y = 0.0f;
            }
          }
          if (here && unsigned(tg - c) < 32u) {
            const float v = act ? dt : lo;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              if (tg == c + 2 * i) d[i].x = v;
              if (tg == c + 2 * i + 1) d[i].y = v;
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) r[i] = F::pack2(d[i].x, d[i].y);
          if (c == 96) free_acc();
          st_32(dst + c, r);
          st_32(dst + c + 16, r + 8);
        }
      } else if (p.chunk >= 0) {   // dx
        float* dst = a.slab + (int64_t(p.chunk) * a.rows_pad + row) * a.H + col0;
        if (!wait_acc()) break;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + (n & 1) * kTileN + c, r);
          tmem_ld_wait();
          if (c == 96) free_acc();
          if (row < kept) {
#pragma unroll
            for (int v = 0; v < 32; v += 8)
              if (col0 + c + v < a.H) st_32(dst + c + v, r + v);
          }
        }
      } else {                     // dW
        const float inv = __ldcg(a.head + 1);
        const int v_row = a.v0 + p.m0 + int(rank) * 128 + q * 32;   // the warp's first row
        uint16_t* dst = static_cast<uint16_t*>(a.dw) + int64_t(v_row + lane) * a.H + col0;
        float zs[kStatCols];
        if (segs > 1) read_sums(zs, segs - 1);
        if (!ok || !wait_acc()) break;
        uint32_t w[32];            // 64 columns
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t r[32];
          tmem_ld32(lanes + (n & 1) * kTileN + c, r);
          tmem_ld_wait();
          if (segs > 1) {
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__fadd_rn(__uint_as_float(r[i]), zs[c + i]));
          }
#pragma unroll
          for (int i = 0; i < 16; ++i)   // no kept row: the accumulator was never written
            w[c % 64 / 2 + i] = p.kblocks == 0 ? 0u : F::pack2(__uint_as_float(r[2 * i]) * inv, __uint_as_float(r[2 * i + 1]) * inv);
          if (c == 96) free_acc();
          if (c % 64 == 32 && col0 + c - 32 < a.H) {   // uniform
            if (a.dw_32) {
#pragma unroll
              for (int v = 0; v < 64; v += 16)
                if (v_row + lane < a.vocab && col0 + c - 32 + v < a.H) st_32(dst + c - 32 + v, w + v / 2);
            } else {
              store_box(&map_e, w, col0 + c - 32, v_row, v_row < a.vocab);
            }
          }
        }
      }
    }
    if (lane == 0) tma_store_wait();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // every product is read and every arrival made
  if (warp == 1) tmem_free_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// forward: joins a row's statistics.  32 rows of a CTA by 32 groups (group j
// takes tiles j, j + 32, ... in order), joined by the pairwise tree.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float2 join_stats(float2 a, float2 b) {   // (max, sum)
  const float m = fmaxf(a.x, b.x);
  if (m == -INFINITY) return make_float2(m, a.y + b.y);
  return make_float2(m, fmaf(a.y, exp2_approx((a.x - m) * kLog2e), b.y * exp2_approx((b.x - m) * kLog2e)));
}

// The target's logit is put right here: nll and lse as functions of it have the
// slopes p - 1 and p, and it moves by some 1e-6 of itself (so the second order
// is far below fp32).  A warp to a row; in the tile kernel, at the columns of the
// target, a small vocabulary waited for it (3000 x 400 x 5000 27.6 us, here 23.7; 4000 x 400 x
// 600 30.9 and 18.4).
template <int DT>
__global__ void __launch_bounds__(1024)
k_xent_join(int rows, int rows_pad, int tiles, int vocab, int nv, float cap, float inv_cap,
            const uint4* __restrict__ x, const uint4* __restrict__ w, const float2* __restrict__ part,
            const float* __restrict__ zt, const int64_t* __restrict__ target, float* __restrict__ nll,
            float* __restrict__ lse) {
  griddep_trigger();
  griddep_wait();
  __shared__ float2 sm[32][33];
  const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + lane;
  float2 s = make_float2(-INFINITY, 0.0f);
  if (row < rows) {
    constexpr int kAhead = 20;   // loads in flight, to one rescaling
    for (int t0 = j; t0 < tiles; t0 += 32 * kAhead) {
      float2 v[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        v[i] = t0 + 32 * i < tiles ? __ldcg(part + int64_t(t0 + 32 * i) * rows_pad + row) : make_float2(-INFINITY, 0.0f);
      float m = s.x;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) m = fmaxf(m, v[i].x);
      const float base = m == -INFINITY ? 0.0f : m;   // (then every exponential is of -inf)
      float sum = s.y * exp2_approx((s.x - base) * kLog2e);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) sum = fmaf(v[i].y, exp2_approx((v[i].x - base) * kLog2e), sum);
      s = make_float2(m, sum);
    }
  }
  sm[j][lane] = s;
  const int mine = blockIdx.x * 32 + j;
  const int64_t t = mine < rows ? __ldg(target + mine) : -1;
  const bool keep = t >= 0 && t < vocab;
  float move = 0.0f;   // what the target's logit is more than the products gave
  if (keep) {
    float2 z = bc2(warp_dot<DT>(x + int64_t(mine) * nv, w + t * nv, nv)), h;
    if (cap > 0.0f) z = mul2(bc2(cap), tanh2(mul2(z, bc2(inv_cap)), &h));
    move = z.x - __ldcg(zt + mine);
    if (!(fabsf(move) < INFINITY)) move = 0.0f;   // infinite either way
  }
  __syncthreads();
  // warp j joins row j's groups: lane l holds group l
  s = sm[lane][j];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const float2 o = make_float2(__shfl_down_sync(0xffffffffu, s.x, d), __shfl_down_sync(0xffffffffu, s.y, d));
    if ((lane & (2 * d - 1)) == 0) s = join_stats(s, o);
  }
  if (lane == 0 && mine < rows) {
    const float l = logf(s.y);
    const bool failed = __ldcg(&g_wait_failed) != 0;
    // (max - s[target]) + log(sum): no cancellation where the target is likely
    float loss = 0.0f, all = s.x + l;
    if (keep) {
      loss = (s.x - __ldcg(zt + mine)) + l;
      const float other = -expm1f(-loss);   // 1 - p
      all = fmaf(1.0f - other, move, all);
      loss = fmaf(-other, move, loss);
      // a certain target's sum may come out as 1 - 2^-24 (a NaN stays)
      loss = loss < 0.0f ? 0.0f : loss;
    }
    if (nll) nll[mine] = failed ? NAN : loss;
    if (lse) lse[mine] = failed ? NAN : all;
  }
}

// ---------------------------------------------------------------------------
// backward: the rows that carry a loss, next to each other and in order, with
// their targets, lse and scaled gradients, and the power of two that dz is scaled
// by (fp16 only: dz is at most max |dnll|, and 2^15 / that keeps small
// probabilities out of fp16's subnormals; bf16 has fp32's exponents and takes
// 1).  Every CTA looks at all targets (12 bytes a row, from L2) to know how many
// kept rows come before its own: one launch in place of a scan and a gather, 4 us
// less for few rows.
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(256)
k_xent_pack(int rows, int rows_per_cta, int vocab, int nv, int fp16, const uint4* __restrict__ x,
            const int64_t* __restrict__ target, const float* __restrict__ lse, const float* __restrict__ dnll,
            const uint4* __restrict__ weight, float* __restrict__ head, int* __restrict__ pos, uint4* __restrict__ xk,
            int* __restrict__ tgt_k, float* __restrict__ lse_k, float* __restrict__ g_k, float* __restrict__ zt_k) {
  griddep_trigger();
  griddep_wait();
  __shared__ int s_before[8], s_all[8], s_row[256];
  __shared__ float s_top[8];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int start = min(int64_t(blockIdx.x) * rows_per_cta, int64_t(rows));
  const int end = min(int64_t(start) + rows_per_cta, int64_t(rows));
  int before = 0, all = 0;
  float top = 0.0f;
  for (int64_t r0 = tid; r0 < rows; r0 += 256 * 8) {
    int64_t t[8];
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 256 * i;
      t[i] = r < rows ? __ldg(target + r) : -1;
      g[i] = r < rows ? __ldg(dnll + r) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t[i] >= 0 && t[i] < vocab) {
        ++all;
        before += r0 + 256 * i < start;
        top = fmaxf(top, fabsf(g[i]));
      }
    }
  }
  before = __reduce_add_sync(0xffffffffu, before);
  all = __reduce_add_sync(0xffffffffu, all);
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (lane == 0) {
    s_before[w] = before;
    s_all[w] = all;
    s_top[w] = top;
  }
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    before += s_before[i];
    all += s_all[i];
    top = fmaxf(top, s_top[i]);
  }
  int e = 0;
  if (fp16 && top > 0.0f && top < INFINITY) {
    (void)frexpf(top, &e);               // top <= 2^e
    e = 15 - e;
    e = e < -100 ? -100 : (e > 100 ? 100 : e);
  }
  const float scale = ldexpf(1.0f, e);
  if (blockIdx.x == 0 && tid == 0) {
    head[0] = __int_as_float(all);
    head[1] = ldexpf(1.0f, -e);
  }
  // a kept row (r >= 0), or zeros, to row `to` of xk; one warp
  auto copy_row = [&](int r, int to) {
    for (int v0 = lane; v0 < nv; v0 += 32 * 4) {
      uint4 u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = r >= 0 && v0 + 32 * j < nv ? __ldg(x + int64_t(r) * nv + v0 + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (v0 + 32 * j < nv) xk[int64_t(to) * nv + v0 + 32 * j] = u[j];
    }
  };
  for (int r0 = start; r0 < end; r0 += 256) {
    const int r = r0 + tid;
    const int64_t t = r < end ? __ldg(target + r) : -1;
    const bool keep = t >= 0 && t < vocab;
    const unsigned kept = __ballot_sync(0xffffffffu, keep);
    __syncthreads();   // the readers of s_before and s_row are done
    if (lane == 0) s_before[w] = __popc(kept);
    __syncthreads();
    int at = __popc(kept & ((1u << lane) - 1u)), here = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      at += i < w ? s_before[i] : 0;
      here += s_before[i];
    }
    if (r < end) pos[r] = keep ? before + at : kIgnored;
    if (keep) {
      s_row[at] = r;
      tgt_k[before + at] = int(t);
      lse_k[before + at] = lse[r];
      g_k[before + at] = dnll[r] * scale;
    }
    __syncthreads();
    for (int i = w; i < here; i += 8) {
      copy_row(s_row[i], before + i);
      if (all <= kRestRow) copy_row(s_row[i], kRestRow + before + i);   // see kDz
      const float z = warp_dot<DT>(x + int64_t(s_row[i]) * nv, weight + __ldg(target + s_row[i]) * nv, nv);
      if (lane == 0) zt_k[before + i] = z;
    }
    before += here;
  }
  // dW reads x in blocks of 64 rows: zeros to the end of the last one (dz is zero
  // there too, but what the workspace held might not be finite)
  for (int i = all + blockIdx.x * 8 + w; i < (all + kTileK - 1) / kTileK * kTileK; i += gridDim.x * 8)
    if (all > kRestRow || i < kRestRow || i >= kRestRow + all) copy_row(-1, i);
}

// ---------------------------------------------------------------------------
// backward: dx from the chunks' products, added in ascending order.  Not the
// last piece: acc = (acc +) slab 0 + slab 1 + ... by kept row.  Last piece: the
// same sum, unscaled, rounded and put at the rows' own places, zeros for rows
// without a loss.  After a wait that ran out the last piece's launch makes dx NaN, and
// dW, whose tiles may be anything then.  Either may be NULL: not wanted.
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(256)
k_xent_fold(int rows, int rows_pad, int H, int chunks, int first, int last, const float* __restrict__ slab,
            float* __restrict__ acc, const float* __restrict__ head, const int* __restrict__ pos,
            const int* __restrict__ tgt_k, const float* __restrict__ lo_k, const uint4* __restrict__ w,
            uint4* __restrict__ dx, int64_t dw_vecs, uint4* __restrict__ dw) {
  using F = Fmt<DT>;
  griddep_trigger();
  griddep_wait();
  const int kept = __float_as_int(__ldcg(head));
  const float inv = __ldcg(head + 1);
  const bool failed = __ldcg(&g_wait_failed) != 0;
  const int nv = H / 8;
  if (failed && last && dw != nullptr) {
    const float2 f[4] = {bc2(NAN), bc2(NAN), bc2(NAN), bc2(NAN)};
    for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < dw_vecs; i += int64_t(gridDim.x) * 256)
      dw[i] = F::pack2v(f);
  }
  const int64_t n = dx == nullptr ? 0 : int64_t(last ? rows : kept) * nv;
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
      if (k >= 0) {   // what the target's dz was rounded by
        float2 wt[4];
        F::unpack2(__ldg(w + int64_t(__ldcg(tgt_k + k)) * nv + v), wt);
        const float lo = __ldcg(lo_k + k);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = fma2(bc2(lo), wt[e], f[e]);
      }
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

// A row-major matrix read or written in boxes of 128 bytes (swizzled) by `box_rows`
// rows; what lies outside reads as zero.
rn_status make_map(CUtensorMap* map, rn_dtype dt, const void* p, int64_t rows, int64_t cols, int64_t ld,
                   int box_rows) {
  const EncodeTiled enc = encode_tiled();
  if (!enc) return cuda_failed(int(cudaErrorNotSupported));
  const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)};
  const cuuint64_t strides[1] = {cuuint64_t(ld) * elem_bytes(dt)};
  const cuuint32_t box[2] = {cuuint32_t(128 / elem_bytes(dt)), cuuint32_t(box_rows)}, steps[2] = {1, 1};
  const CUresult e =
      enc(map, dt == RN_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
               : dt == RN_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
          const_cast<void*>(p), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return e == CUDA_SUCCESS ? RN_OK : cuda_failed(int(cudaErrorInvalidValue));
}

// The tensor maps of a launch (see k_xent_tile); those it does not use are zeros.
struct TileMaps {
  CUtensorMap a, b, c, d, e;
};
template <int DT, int MODE, bool CAP>
rn_status launch_tile(const TileMaps& m, const XentArgs& a, int64_t most_tiles, cudaStream_t st) {
  static KernelPrep prep;
  (void)prepare_kernel(k_xent_tile<DT, MODE, CAP>, kThreads, kTileSmem, prep);
  static std::atomic<int> regs{0};   // a thread at launch, of this build
  if (regs.load() == 0) {
    cudaFuncAttributes fa;
    const cudaError_t e = cudaFuncGetAttributes(&fa, k_xent_tile<DT, MODE, CAP>);
    if (e != cudaSuccess) return cuda_failed(int(e));
    regs.store(fa.numRegs);
  }
  if (regs.load() * kThreads < 128 * kOtherRegs + (kThreads - 128) * kEpilogueRegs)
    return cuda_failed(int(cudaErrorLaunchOutOfResources));
  const int64_t pairs = sm_count() / 2;
  const int64_t want = most_tiles < pairs ? most_tiles : pairs;
  return launch_pdl(k_xent_tile<DT, MODE, CAP>, dim3(unsigned(2 * (want < 1 ? 1 : want))), dim3(kThreads),
                    kTileSmem, st, m.a, m.b, m.c, m.d, m.e, a);
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// carves a workspace into 256-byte aligned pieces (the caller's is 16-byte aligned)
struct Carve {
  uintptr_t p, p0;
  explicit Carve(void* base) : p((reinterpret_cast<uintptr_t>(base) + 255) & ~uintptr_t(255)), p0(p) {}
  template <typename T>
  T* take(int64_t n) {
    T* q = reinterpret_cast<T*>(p);
    p += (size_t(n) * sizeof(T) + 255) & ~size_t(255);
    return q;
  }
  size_t bytes() const { return size_t(p - p0) + 240; }   // and the alignment of the start
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
  w.part = c.take<float2>(ceil_div(vocab, kStatCols) * rp);
  w.zt = c.take<float>(rp);
  w.bytes = c.bytes();
  return w;
}

// The vocabulary in chunks that dx is summed over: at most 16384 columns, and
// down to 8192 while the chunks of one row tile make fewer than 64 tiles of dx, so
// that few rows have tiles for every pair of CTAs (100 x 1024 x 50000 step 142 us in
// chunks of 16384, 122 in 8192, 132 in 4096, 4096 rows of it 1419, 1401, 1498: a
// smaller chunk costs many rows the writing and reading of its product).  The
// number depends on V and H only, so a row's dx does not depend on the rows.
// A piece is as many chunks as keep dz within 512 MB, at least one (4096 x 2048 x
// 151936 step: 64 MB pieces 7.05 ms, 256 MB 6.50, 512 MB 6.41).
constexpr int64_t kMostChunk = 16384, kLeastChunk = 8192, kFewTiles = 64;
static_assert(kMostChunk <= kGradSegment * kTileK, "dx takes a chunk in one accumulator");
constexpr int64_t kDzBudget = int64_t(512) << 20;
struct BwdPlan {
  int64_t rows_pad;
  int chunk, chunks, per_piece, pieces;
};
BwdPlan xent_plan(int64_t rows, int width, int64_t vocab) {
  BwdPlan p;
  p.rows_pad = up(rows, kTileM);
  const int64_t spread = std::min(ceil_div(vocab, kLeastChunk), ceil_div(kFewTiles, ceil_div(width, kTileN)));
  p.chunk = int(up(ceil_div(vocab, std::max(ceil_div(vocab, kMostChunk), spread)), 256));
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
  int* tgt_k;
  float* lse_k;
  float* g_k;
  float* zt_k;
  float* lo_k;
  uint16_t* xk;
  uint16_t* dz;
  float* slab;
  float* acc;
  size_t bytes;
};
BwdWs xent_bwd_ws(void* base, int64_t rows, int width, const BwdPlan& p) {
  Carve c(base);
  BwdWs w;
  w.head = c.take<float>(2);
  w.pos = c.take<int>(rows);
  w.tgt_k = c.take<int>(p.rows_pad);
  w.lse_k = c.take<float>(p.rows_pad);
  w.g_k = c.take<float>(p.rows_pad);
  w.zt_k = c.take<float>(p.rows_pad);
  w.lo_k = c.take<float>(p.rows_pad);
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
  XentArgs a = {};
  a.rows = int(rows);
  a.rows_pad = int(up(rows, kTileM));
  a.x_rows = int(rows < 128 ? up(rows, 8) : 128);
  a.x_odd = rows > 128;
  a.H = width;
  a.vocab = int(vocab);
  a.cap = cap;
  a.inv_cap = cap > 0 ? 1.0f / cap : 0.0f;
  a.target = target;
  a.part = f.part;
  a.zt = f.zt;
  TileMaps m = {};
  rn_status e = make_map(&m.a, rn_dtype(DT), x, rows, width, width, a.x_rows);
  if (e == RN_OK) e = make_map(&m.b, rn_dtype(DT), w, vocab, width, width, 128);
  if (e != RN_OK) return e;
  const int64_t tiles = ceil_div(rows, kTileM) * ceil_div(vocab, kTileN);
  e = cap > 0 ? launch_tile<DT, kFwd, true>(m, a, tiles, st) : launch_tile<DT, kFwd, false>(m, a, tiles, st);
  if (e != RN_OK) return e;
  return launch_pdl(k_xent_join<DT>, dim3(unsigned(ceil_div(rows, 32))), dim3(1024), 0, st, a.rows, a.rows_pad,
                    int(ceil_div(vocab, kStatCols)), a.vocab, width / 8, a.cap, a.inv_cap,
                    static_cast<const uint4*>(x), static_cast<const uint4*>(w), f.part, f.zt, target, nll, lse);
}

template <int DT>
rn_status run_xent_bwd(int64_t rows, int width, int64_t vocab, const void* x, const void* w,
                       const int64_t* target, const float* lse, const float* dnll, float cap, void* dx, void* dw,
                       void* ws, cudaStream_t st) {
  const BwdPlan p = xent_plan(rows, width, vocab);
  const BwdWs b = xent_bwd_ws(ws, rows, width, p);
  // (eight CTAs at least: they share the zero rows)
  const int64_t most = 2 * sm_count(), per = up(ceil_div(rows, most), 8);
  rn_status e = launch_pdl(k_xent_pack<DT>, dim3(unsigned(std::max<int64_t>(8, ceil_div(rows, per)))), dim3(256), 0, st, int(rows), int(per),
                           int(vocab), width / 8, int(DT == RN_F16), static_cast<const uint4*>(x), target, lse, dnll,
                           static_cast<const uint4*>(w), b.head, b.pos, reinterpret_cast<uint4*>(b.xk), b.tgt_k, b.lse_k,
                           b.g_k, b.zt_k);
  if (e != RN_OK) return e;
  const int64_t ld = int64_t(p.chunk) * p.per_piece;
  XentArgs a = {};
  a.rows = int(rows);
  a.rows_pad = int(p.rows_pad);
  a.x_rows = int(rows <= 64 ? 64 : rows < 128 ? up(rows, 8) : 128);   // (rows 32 to 63 may hold rests)
  a.x_odd = rows > 128;
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
  a.zt_k = b.zt_k;
  a.lo_k = b.lo_k;
  a.dz = b.dz;
  a.slab = dx ? b.slab : nullptr;
  a.dw = dw;
  TileMaps logits = {}, grad = {};
  e = make_map(&logits.a, rn_dtype(DT), b.xk, p.rows_pad, width, width, a.x_rows);
  if (e == RN_OK) e = make_map(&logits.b, rn_dtype(DT), w, vocab, width, width, 128);
  if (e == RN_OK) e = make_map(&grad.a, rn_dtype(DT), b.dz, p.rows_pad, ld, ld, 128);
  if (e == RN_OK) e = make_map(&grad.b, rn_dtype(DT), w, vocab, width, width, 64);
  if (e == RN_OK) e = make_map(&grad.c, rn_dtype(DT), b.dz, p.rows_pad, ld, ld, 64);
  if (e == RN_OK) e = make_map(&grad.d, rn_dtype(DT), b.xk, p.rows_pad, width, width, 64);
  a.dw_32 = width % 16 == 0 && (uintptr_t(dw) & 31) == 0;
  if (e == RN_OK && dw && !a.dw_32) e = make_map(&grad.e, rn_dtype(DT), dw, vocab, width, width, 32);
  if (e != RN_OK) return e;
  const int64_t mt = p.rows_pad / kTileM, ht = ceil_div(width, kTileN);
  for (int piece = 0; piece < p.pieces; ++piece) {
    const int c0 = piece * p.per_piece;
    a.chunks = p.chunks - c0 < p.per_piece ? p.chunks - c0 : p.per_piece;
    a.v0 = c0 * p.chunk;
    const int64_t left = vocab - a.v0;
    const int64_t vt = ceil_div(left < int64_t(a.chunks) * p.chunk ? left : int64_t(a.chunks) * p.chunk, kTileN);
    e = cap > 0 ? launch_tile<DT, kDz, true>(logits, a, mt * vt, st)
                : launch_tile<DT, kDz, false>(logits, a, mt * vt, st);
    if (e == RN_OK)
      e = launch_tile<DT, kGrad, false>(grad, a, (dx ? mt * ht * a.chunks : 0) + (dw ? vt * ht : 0), st);
    const bool last = piece + 1 == p.pieces;
    if (e == RN_OK && (dx || last)) {
      const int64_t n = dx ? ceil_div(rows * (width / 8), 256) : 1;
      const int64_t cap_grid = int64_t(8) * sm_count();
      e = launch_pdl(k_xent_fold<DT>, dim3(unsigned(n < cap_grid ? n : cap_grid)), dim3(256), 0, st, int(rows),
                     a.rows_pad, width, a.chunks, int(piece == 0), int(last), b.slab, b.acc, b.head, b.pos, b.tgt_k,
                     b.lo_k, static_cast<const uint4*>(w), static_cast<uint4*>(dx), vocab * (width / 8),
                     static_cast<uint4*>(dw));
    }
    if (e != RN_OK) return e;
  }
  return RN_OK;
}

rn_status xent_checks(int64_t rows, int32_t width, int64_t vocab, rn_dtype dt, float cap) {
  // (the cap and its reciprocal far from fp32's ends)
  if (!xent_sizes_ok(rows, vocab) || !(cap == 0.0f || (cap >= 0x1p-100f && cap <= 0x1p100f))) return RN_E_ARG;
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
  return xent_bwd_ws(nullptr, rows, width, xent_plan(rows, width, vocab)).bytes;
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

rn_status rn_test_set_wait_failed(int32_t on) {
  if (validate_only()) return RN_OK;
  const uint32_t v = on ? 1u : 0u;
  const cudaError_t e = cudaMemcpyToSymbol(g_wait_failed, &v, sizeof v);
  return e == cudaSuccess ? RN_OK : cuda_failed(int(e));
}

}  // extern "C"
