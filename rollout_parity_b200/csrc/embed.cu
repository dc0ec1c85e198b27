// Embedding of librn and its gradient (include/rn.h, "Embedding"):
//   forward   y[t] = fmt(scale * E[ids[t]])
//   gradient  dE[v] = fmt(scale * sum over t with ids[t] == v of dy[t])
// A token whose id is outside [0, vocab) has a zero row and no gradient.
//
// The gradient uses no floating-point atomics.  The tokens are sorted by id,
// stably, so that the tokens of a vocabulary row (a run) lie next to each other
// in token order; a run is cut into leaves of 32 tokens counted from its own
// start, a leaf is summed in token order, and a run's leaves are joined by the
// level-by-level pairwise tree.  So a row of dE depends on its own tokens only,
// bitwise, wherever they stand in the batch and whatever the other tokens are.
// Three kernels: k_embed_sort (which also clears dE with the CTAs that do not
// sort), k_embed_reduce, k_embed_join.
#include <cooperative_groups.h>

#include <cmath>

#include "rn_checks.cuh"
#include "rn_rows.cuh"

namespace cg = cooperative_groups;
using namespace rn_detail;

namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 28;
constexpr int kMaxVocab = 1 << 27;

constexpr int kSortCtas = 8;         // one cluster sorts
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kDigitBits = 9;        // at most 512 bins a pass
constexpr int kLeaf = 32;            // tokens of one leaf

// ---------------------------------------------------------------------------
// forward: a warp per token, up to eight 16-byte vectors of a lane in flight
// ---------------------------------------------------------------------------
template <int DT>
__global__ void __launch_bounds__(128)
k_embed_fwd(int64_t tokens, int64_t vocab, int nv, float scale, const int64_t* __restrict__ ids,
            const uint4* __restrict__ table, uint4* __restrict__ y) {
  using F = Fmt<DT>;
  griddep_trigger();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t step = int64_t(gridDim.x) * 4;
  for (int64_t t = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5); t < tokens; t += step) {
    const int64_t id = __ldg(ids + t);
    const bool ok = id >= 0 && id < vocab;
    const uint4* src = table + (ok ? id : 0) * nv;
    uint4* dst = y + t * nv;
    for (int v0 = lane; v0 < nv; v0 += 32 * 8) {
      uint4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        u[i] = ok && v0 + 32 * i < nv ? __ldg(src + v0 + 32 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (v0 + 32 * i >= nv) break;
        if (ok) {
          float2 f[F::VE / 2];
          F::unpack2(u[i], f);
#pragma unroll
          for (int q = 0; q < F::VE / 2; ++q) f[q] = mul2(f[q], bc2(scale));
          u[i] = F::pack2v(f);
        }
        st_stream(dst + v0 + 32 * i, u[i]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// gradient, workspace
// ---------------------------------------------------------------------------
struct EmbedWs {
  uint32_t* key[2];      // [tokens] sorted ids (vocab: no row), ping and pong
  uint32_t* tok[2];      // [tokens] their tokens
  uint32_t* run_start;   // [tokens + 1] first position of each run
  uint32_t* run_of;      // [tokens/32 + 1] the run that holds position 32 e
  uint32_t* counts;      // [0] runs, [1] runs longer than a leaf
  uint32_t* long_runs;   // [tokens/32 + 1] those runs, in any order
  float* first_leaf;     // [tokens/32 + 1][H] leaf 0 of the run starting at s: row s/32
  float* more_leaves;    // [tokens/32 + 1][H] leaf j > 0: row ceil(s/32) + j - 1
  size_t bytes;
};

EmbedWs embed_ws(void* base, int64_t tokens, int width) {
  EmbedWs w;
  uintptr_t p = reinterpret_cast<uintptr_t>(base);
  const uintptr_t p0 = p;
  auto take = [&](size_t n) {
    const uintptr_t q = p;
    p += (n + 255) & ~size_t(255);
    return q;
  };
  const size_t n = size_t(tokens), b = n / kLeaf + 1;
  for (int i = 0; i < 2; ++i) {
    w.key[i] = reinterpret_cast<uint32_t*>(take(n * 4));
    w.tok[i] = reinterpret_cast<uint32_t*>(take(n * 4));
  }
  w.run_start = reinterpret_cast<uint32_t*>(take((n + 1) * 4));
  w.run_of = reinterpret_cast<uint32_t*>(take(b * 4));
  w.counts = reinterpret_cast<uint32_t*>(take(8));
  w.long_runs = reinterpret_cast<uint32_t*>(take(b * 4));
  w.first_leaf = reinterpret_cast<float*>(take(b * size_t(width) * 4));
  w.more_leaves = reinterpret_cast<float*>(take(b * size_t(width) * 4));
  w.bytes = size_t(p - p0);
  return w;
}

// ---------------------------------------------------------------------------
// gradient, pass 1: cluster 0 sorts the tokens by id (stable least-significant-
// digit radix sort) and lists the runs; the other clusters clear dE meanwhile.
// A warp owns a contiguous piece of the positions.  Per pass: a histogram of
// each warp's piece, prefix sums over the warps, the cluster's CTAs
// (distributed shared memory) and the bins, then the scatter in order.
// ---------------------------------------------------------------------------
struct SortShared {
  uint32_t hist[kSortWarps][1 << kDigitBits];
  uint32_t total[1 << kDigitBits];
  uint32_t base[1 << kDigitBits];
  uint32_t warp_sum[kSortWarps];
};

// exclusive prefix sum over the CTA's threads; every thread must call it
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* warp_sum, uint32_t* all) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += u;
  }
  __syncthreads();   // earlier readers of warp_sum are done
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  uint32_t s = warp_sum[lane];   // kSortWarps == 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  *all = __shfl_sync(0xffffffffu, s, 31);
  const uint32_t before = w == 0 ? 0 : __shfl_sync(0xffffffffu, s, w - 1);
  return before + x - v;
}

__global__ void __launch_bounds__(kSortThreads)
k_embed_sort(uint32_t tokens, uint32_t vocab, int passes, int bits, const int64_t* __restrict__ ids,
             EmbedWs ws, uint4* __restrict__ clear, int64_t clear_vecs) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  SortShared& sm = *reinterpret_cast<SortShared*>(smem_raw);
  griddep_trigger();
  griddep_wait();
  if (blockIdx.x >= kSortCtas) {
    const int64_t stride = int64_t(gridDim.x - kSortCtas) * kSortThreads;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = int64_t(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x; i < clear_vecs;
         i += stride)
      clear[i] = zero;
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const unsigned below = (1u << lane) - 1u;
  // this warp's positions: a multiple of 32 each, in order of (CTA, warp)
  const uint32_t groups = (tokens + 31) / 32;
  const uint32_t per = (groups + kSortCtas * kSortWarps - 1) / (kSortCtas * kSortWarps) * 32;
  const uint64_t lo64 = uint64_t(blockIdx.x * kSortWarps + w) * per;
  const uint32_t lo = lo64 < tokens ? uint32_t(lo64) : tokens;
  const uint32_t hi = tokens - lo < per ? tokens : lo + per;
  const int bins = 1 << bits;

  for (int pass = 0; pass < passes; ++pass) {
    const uint32_t* src_key = ws.key[(pass + 1) & 1];
    const uint32_t* src_tok = ws.tok[(pass + 1) & 1];
    uint32_t* dst_key = ws.key[pass & 1];
    uint32_t* dst_tok = ws.tok[pass & 1];
    const int shift = pass * bits;
    auto key_at = [&](uint32_t i) -> uint32_t {
      if (pass > 0) return __ldcg(src_key + i);
      const int64_t id = __ldg(ids + i);
      return id >= 0 && id < int64_t(vocab) ? uint32_t(id) : vocab;
    };
    for (int i = tid; i < kSortWarps * (1 << kDigitBits); i += kSortThreads) (&sm.hist[0][0])[i] = 0;
    __syncthreads();
    for (uint32_t p = lo; p < hi; p += 32) {
      const bool in = p + lane < hi;
      const uint32_t d = in ? (key_at(p + lane) >> shift) & (bins - 1) : 0xffffffffu;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (in && (same & below) == 0) sm.hist[w][d] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    uint32_t mine = 0;
    if (tid < bins) {   // prefix over the warps
#pragma unroll 8
      for (int i = 0; i < kSortWarps; ++i) {
        const uint32_t c = sm.hist[i][tid];
        sm.hist[i][tid] = mine;
        mine += c;
      }
      sm.total[tid] = mine;
    }
    cluster.sync();
    uint32_t all = 0, before = 0;
    if (tid < bins) {   // over the cluster's CTAs
#pragma unroll
      for (int c = 0; c < kSortCtas; ++c) {
        const uint32_t n = cluster.map_shared_rank(&sm.total[0], c)[tid];
        all += n;
        if (c < int(blockIdx.x)) before += n;
      }
    }
    uint32_t sum;
    const uint32_t start = block_prefix(all, sm.warp_sum, &sum);   // over the bins
    if (tid < bins) sm.base[tid] = start + before;
    __syncthreads();
    for (uint32_t p = lo; p < hi; p += 32) {
      const bool in = p + lane < hi;
      const uint32_t key = in ? key_at(p + lane) : 0;
      const uint32_t d = in ? (key >> shift) & (bins - 1) : 0xffffffffu;
      const uint32_t t = !in ? 0 : pass > 0 ? __ldcg(src_tok + p + lane) : p + lane;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      if (in) {
        const uint32_t at = sm.base[d] + sm.hist[w][d] + __popc(same & below);
        __stcg(dst_key + at, key);
        __stcg(dst_tok + at, t);
      }
      __syncwarp();
      if (in && (same & below) == 0) sm.hist[w][d] += __popc(same);
      __syncwarp();
    }
    __threadfence();
    cluster.sync();   // the scatter is complete; the totals may be overwritten
  }

  // the runs: positions whose id differs from the one before
  const uint32_t* key = ws.key[(passes + 1) & 1];
  auto starts = [&](uint32_t p) -> unsigned {   // one bit a position of [p, p + 32)
    const bool in = p + lane < hi;
    bool s = false;
    if (in) s = p + lane == 0 || __ldcg(key + p + lane) != __ldcg(key + p + lane - 1);
    return __ballot_sync(0xffffffffu, s);
  };
  uint32_t n = 0;
  for (uint32_t p = lo; p < hi; p += 32) n += __popc(starts(p));
  // prefix over the CTA's warps (a warp's count is carried by its lane 0)
  uint32_t cta_runs;
  uint32_t at = block_prefix(lane == 0 ? n : 0, sm.warp_sum, &cta_runs);
  at = __shfl_sync(0xffffffffu, at, 0);
  if (tid == 0) sm.total[0] = cta_runs;
  cluster.sync();
  uint32_t all = 0;
  for (int c = 0; c < kSortCtas; ++c) {
    const uint32_t m = *cluster.map_shared_rank(&sm.total[0], c);
    if (c < int(blockIdx.x)) at += m;
    all += m;
  }
  for (uint32_t p = lo; p < hi; p += 32) {
    const unsigned s = starts(p);
    if ((s >> lane) & 1u) ws.run_start[at + __popc(s & below)] = p + lane;
    if (lane == 0) ws.run_of[p / 32] = at + (s & 1u) - 1;   // the run that holds position p
    at += __popc(s);
  }
  if (blockIdx.x == 0 && tid == 0) {
    ws.run_start[all] = tokens;
    ws.counts[0] = all;
    ws.counts[1] = 0;
  }
  cluster.sync();   // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------------------
// gradient, pass 2: sums of the leaves.  A unit is one leaf and one slab of
// columns (two 16-byte vectors a lane, 1 KB of a row); a warp takes units in
// turn and has the tokens' rows of four steps in flight.  The unit of run u
// sums its leaf 0; leaf j > 0 of a run is summed by the unit of the j-th
// multiple of 32 among the run's positions (there are at least as many as
// leaves after the first).  A run of one leaf is written to dE at once.
// ---------------------------------------------------------------------------
template <int DT>
__device__ __forceinline__ void embed_store(uint4* at, const float2 (&s)[Fmt<DT>::VE / 2],
                                            float scale, bool add) {
  using F = Fmt<DT>;
  float2 f[F::VE / 2];
  if (add) {
    F::unpack2(*at, f);
#pragma unroll
    for (int q = 0; q < F::VE / 2; ++q) f[q] = fma2(s[q], bc2(scale), f[q]);
  } else {
#pragma unroll
    for (int q = 0; q < F::VE / 2; ++q) f[q] = mul2(s[q], bc2(scale));
  }
  *at = F::pack2v(f);
}

template <int DT>
__global__ void __launch_bounds__(256)
k_embed_reduce(uint32_t tokens, uint32_t vocab, int nv, float scale, int add, int last,
               EmbedWs ws, const uint4* __restrict__ dy, uint4* __restrict__ out) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE, C = 2, U = 4;   // vectors a lane, tokens in flight
  griddep_trigger();
  griddep_wait();
  const uint32_t* key = ws.key[last];
  const uint32_t* tok = ws.tok[last];
  const int lane = threadIdx.x & 31;
  const uint32_t slabs = (nv + 32 * C - 1) / (32 * C);
  const uint32_t blocks = (tokens + kLeaf - 1) / kLeaf;
  const uint64_t units = uint64_t(blocks + __ldcg(ws.counts)) * slabs;
  const uint64_t stride = uint64_t(gridDim.x) * (blockDim.x / 32);
  for (uint64_t u = uint64_t(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5); u < units;
       u += stride) {
    const uint32_t unit = uint32_t(u / slabs), slab = uint32_t(u % slabs);
    const bool first = unit >= blocks;
    const uint32_t run = first ? unit - blocks : __ldcg(ws.run_of + unit);
    const uint32_t s = __ldcg(ws.run_start + run), e = __ldcg(ws.run_start + run + 1);
    const uint32_t e0 = (s + kLeaf - 1) / kLeaf;          // the run's first multiple of 32
    const uint32_t leaf = first ? 0 : unit - e0 + 1;      // (unit >= e0: 32 unit is in the run)
    const uint32_t p0 = s + leaf * kLeaf;
    if (p0 >= e) continue;                                // no such leaf
    const uint32_t id = __ldcg(key + s);
    if (id >= vocab) continue;                            // tokens of no row
    const int cnt = e - p0 < kLeaf ? int(e - p0) : kLeaf;
    const uint32_t my_tok = lane < cnt ? __ldcg(tok + p0 + lane) : 0;
    const int v0 = int(slab) * 32 * C + lane;
    float2 acc[C][VE / 2];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int q = 0; q < VE / 2; ++q) acc[c][q] = bc2(-0.0f);
    for (int i = 0; i < cnt; i += U) {
      uint4 r[U][C];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const uint32_t t = __shfl_sync(0xffffffffu, my_tok, (i + j) & 31);
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (i + j < cnt && v0 + 32 * c < nv) r[j][c] = __ldcs(dy + int64_t(t) * nv + v0 + 32 * c);
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (i + j < cnt) {
#pragma unroll
          for (int c = 0; c < C; ++c) {
            float2 f[VE / 2];
            F::unpack2(r[j][c], f);
#pragma unroll
            for (int q = 0; q < VE / 2; ++q) acc[c][q] = add2(acc[c][q], f[q]);
          }
        }
      }
    }
    if (e - s <= kLeaf) {
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (v0 + 32 * c < nv) embed_store<DT>(out + int64_t(id) * nv + v0 + 32 * c, acc[c], scale, add);
    } else {
      const uint64_t row = first ? s / kLeaf : unit;
      float4* part = reinterpret_cast<float4*>(first ? ws.first_leaf : ws.more_leaves) + row * nv * (VE / 4);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (v0 + 32 * c < nv) {
#pragma unroll
          for (int q = 0; q < VE / 4; ++q)
            part[(v0 + 32 * c) * (VE / 4) + q] = make_float4(acc[c][2 * q].x, acc[c][2 * q].y,
                                                             acc[c][2 * q + 1].x, acc[c][2 * q + 1].y);
        }
      }
      if (first && slab == 0 && lane == 0) ws.long_runs[atomicAdd(ws.counts + 1, 1u)] = run;
    }
  }
}

// ---------------------------------------------------------------------------
// gradient, pass 3: the leaves of the long runs, joined by the level-by-level
// pairwise tree.  A CTA takes one run and 32 16-byte vectors' columns at a
// time; its eight warps stream aligned power-of-two blocks of leaves (perfect
// subtrees), joined in shared memory.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
template <int DT>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_embed_join(int nv, float scale, int add, int last, EmbedWs ws, uint4* __restrict__ out) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  griddep_trigger();
  griddep_wait();
  __shared__ float sm[kJoinWarps][32][VE + 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t cols = (nv + 31) / 32;
  const uint64_t items = uint64_t(__ldcg(ws.counts + 1)) * cols;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint32_t run = __ldcg(ws.long_runs + it / cols);
    const int v = int(it % cols) * 32 + lane;
    const uint32_t s = __ldcg(ws.run_start + run), e = __ldcg(ws.run_start + run + 1);
    const uint32_t leaves = (e - s + kLeaf - 1) / kLeaf;
    const uint32_t e0 = (s + kLeaf - 1) / kLeaf;
    uint32_t per = 1;                       // leaves per warp: a power of two
    while (per * kJoinWarps < leaves) per <<= 1;
    const uint32_t l0 = w * per;
    const uint32_t cnt = l0 >= leaves ? 0 : (leaves - l0 < per ? leaves - l0 : per);
    auto leaf_at = [&](uint32_t l, float2 (&f)[VE / 2]) {
      const float4* p = reinterpret_cast<const float4*>(l == 0 ? ws.first_leaf : ws.more_leaves) +
                        (uint64_t(l == 0 ? s / kLeaf : e0 + l - 1) * nv + v) * (VE / 4);
#pragma unroll
      for (int q = 0; q < VE / 4; ++q) {
        const float4 x = __ldcg(p + q);
        f[2 * q] = make_float2(x.x, x.y);
        f[2 * q + 1] = make_float2(x.z, x.w);
      }
    };
    // a stack of pending perfect subtrees, the j-th of 2^k leaves where bit k
    // of the leaves taken so far is set
    float2 stack[24][VE / 2];
    int top = 0;
    if (v < nv) {
      for (uint32_t i = 0; i < cnt; ++i) {
        float2 cur[VE / 2];
        leaf_at(l0 + i, cur);
        for (uint32_t k = i; k & 1u; k >>= 1) {
          --top;
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) cur[q] = add2(stack[top][q], cur[q]);
        }
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) stack[top][q] = cur[q];
        ++top;
      }
      float2 res[VE / 2];
      if (cnt > 0) {   // pending subtrees, smallest (rightmost) first
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) res[q] = stack[top - 1][q];
        for (int k = top - 2; k >= 0; --k)
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) res[q] = add2(stack[k][q], res[q]);
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) {
          sm[w][lane][2 * q] = res[q].x;
          sm[w][lane][2 * q + 1] = res[q].y;
        }
      }
    }
    __syncthreads();
    if (w == 0 && v < nv) {
      const int nw = int((leaves + per - 1) / per);
      float2 p[kJoinWarps][VE / 2];
#pragma unroll
      for (int i = 0; i < kJoinWarps; ++i)
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) p[i][q] = make_float2(sm[i][lane][2 * q], sm[i][lane][2 * q + 1]);
#pragma unroll
      for (int d = 1; d < kJoinWarps; d <<= 1) {
#pragma unroll
        for (int l = 0; l + d < kJoinWarps; l += 2 * d)
          if (l + d < nw) {
#pragma unroll
            for (int q = 0; q < VE / 2; ++q) p[l][q] = add2(p[l][q], p[l + d][q]);
          }
      }
      const uint32_t id = __ldcg(ws.key[last] + s);
      embed_store<DT>(out + int64_t(id) * nv + v, p[0], scale, add);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
bool embed_sizes_ok(int64_t tokens, int64_t vocab) {
  return tokens >= 0 && tokens <= kMaxTokens && vocab >= 1 && vocab <= kMaxVocab;
}

rn_status launch_sort(int64_t tokens, int64_t vocab, const int64_t* ids, const EmbedWs& ws,
                      void* clear, size_t clear_bytes, int* last, cudaStream_t st) {
  int bits = 1;
  while ((int64_t(1) << bits) <= vocab) ++bits;   // the largest key is vocab
  const int passes = (bits + kDigitBits - 1) / kDigitBits;
  const int digit = (bits + passes - 1) / passes;
  *last = (passes + 1) & 1;
  static KernelPrep prep;
  (void)prepare_kernel(k_embed_sort, kSortThreads, sizeof(SortShared), prep);
  // the clearing CTAs: two of the kernel's CTAs fit on an SM
  const int clusters = clear ? (2 * sm_count() - kSortCtas) / kSortCtas : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSortCtas * (1 + (clusters > 0 ? clusters : clear ? 1 : 0)));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = sizeof(SortShared);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSortCtas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  (void)cudaLaunchKernelEx(&cfg, k_embed_sort, uint32_t(tokens), uint32_t(vocab), passes, digit, ids,
                           ws, static_cast<uint4*>(clear), int64_t(clear_bytes / 16));
  return launch_status();
}

template <int DT>
rn_status run_embed_bwd(int64_t tokens, int64_t vocab, int width, float scale, bool add,
                        const int64_t* ids, const void* dy, void* dtable, const EmbedWs& ws,
                        cudaStream_t st) {
  const int nv = width / Fmt<DT>::VE;
  int last = 0;
  rn_status e = launch_sort(tokens, vocab, ids, ws, add ? nullptr : dtable,
                            size_t(vocab) * nv * 16, &last, st);
  if (e != RN_OK || tokens == 0) return e;
  static KernelPrep prep_reduce, prep_join;
  const uint64_t slabs = (nv + 63) / 64;
  const uint64_t most = (uint64_t(tokens) + tokens / kLeaf + 1) * slabs;   // units, at most
  const uint64_t want = (most + 7) / 8;
  const int fit = prepare_kernel(k_embed_reduce<DT>, 256, 0, prep_reduce) * sm_count();
  e = launch_pdl(k_embed_reduce<DT>, dim3(unsigned(want < uint64_t(fit) ? want : fit)), dim3(256), 0,
                 st, uint32_t(tokens), uint32_t(vocab), nv, scale, int(add), last, ws,
                 static_cast<const uint4*>(dy), static_cast<uint4*>(dtable));
  if (e != RN_OK || tokens <= kLeaf) return e;   // no run longer than a leaf
  const int jfit = prepare_kernel(k_embed_join<DT>, 32 * kJoinWarps, 0, prep_join) * sm_count();
  const uint64_t items = uint64_t(tokens / (kLeaf + 1)) * ((nv + 31) / 32);
  return launch_pdl(k_embed_join<DT>, dim3(unsigned(items < uint64_t(jfit) ? items : jfit)),
                    dim3(32 * kJoinWarps), 0, st, nv, scale, int(add), last, ws,
                    static_cast<uint4*>(dtable));
}

template <int DT>
rn_status run_embed_fwd(int64_t tokens, int64_t vocab, int width, float scale, const int64_t* ids,
                        const void* table, void* y, cudaStream_t st) {
  static KernelPrep prep;
  const int64_t fit = int64_t(prepare_kernel(k_embed_fwd<DT>, 128, 0, prep)) * sm_count();
  const int64_t want = (tokens + 3) / 4;
  return launch_pdl(k_embed_fwd<DT>, dim3(unsigned(want < fit ? want : fit)), dim3(128), 0, st,
                    tokens, vocab, width / Fmt<DT>::VE, scale, ids,
                    static_cast<const uint4*>(table), static_cast<uint4*>(y));
}

}  // namespace

extern "C" {

rn_status embed_fwd(int64_t tokens, int64_t vocab, int32_t width, float scale, rn_dtype dt,
                    const int64_t* ids, const void* table, void* y, rn_stream stream) {
  begin_call();
  if (!embed_sizes_ok(tokens, vocab) || !std::isfinite(scale)) return RN_E_ARG;
  if (!dtype_ok(dt)) return RN_E_DTYPE;
  if (!width_ok(width)) return RN_E_WIDTH;
  if (!table || (tokens > 0 && (!ids || !y))) return RN_E_ARG;
  if (!aligned16(table) || !aligned16(y) || (uintptr_t(ids) & 7u)) return RN_E_ALIGN;
  const size_t row = size_t(width) * elem_bytes(dt);
  const Range in[] = {{ids, size_t(tokens) * 8}, {table, size_t(vocab) * row}};
  const Range out[] = {{y, size_t(tokens) * row}};
  const rn_status e = check_ranges(in, 2, out, 1);
  if (e != RN_OK || validate_only() || tokens == 0) return e;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dt) {
    case RN_BF16: return run_embed_fwd<RN_BF16>(tokens, vocab, width, scale, ids, table, y, st);
    case RN_F16: return run_embed_fwd<RN_F16>(tokens, vocab, width, scale, ids, table, y, st);
    default: return run_embed_fwd<RN_F32>(tokens, vocab, width, scale, ids, table, y, st);
  }
}

size_t embed_bwd_workspace_bytes(int64_t tokens, int32_t width) {
  if (tokens < 0 || tokens > kMaxTokens || !width_ok(width)) return 0;
  return embed_ws(nullptr, tokens, width).bytes;
}

rn_status embed_bwd(int64_t tokens, int64_t vocab, int32_t width, float scale, rn_dtype dt,
                    const int64_t* ids, const void* dy, int32_t accumulate, void* dtable, void* ws,
                    size_t ws_bytes, rn_stream stream) {
  begin_call();
  if (!embed_sizes_ok(tokens, vocab) || !std::isfinite(scale)) return RN_E_ARG;
  if (!dtype_ok(dt)) return RN_E_DTYPE;
  if (!width_ok(width)) return RN_E_WIDTH;
  if (!dtable || (tokens > 0 && (!ids || !dy))) return RN_E_ARG;
  if (!aligned16(dtable) || !aligned16(dy) || (uintptr_t(ids) & 7u)) return RN_E_ALIGN;
  const size_t need = embed_bwd_workspace_bytes(tokens, width);
  if (!ws || ws_bytes < need) return RN_E_WORKSPACE;
  if (!aligned16(ws)) return RN_E_ALIGN;
  const size_t row = size_t(width) * elem_bytes(dt);
  const Range in[] = {{ids, size_t(tokens) * 8}, {dy, size_t(tokens) * row}};
  const Range out[] = {{dtable, size_t(vocab) * row}, {ws, need}};
  const rn_status e = check_ranges(in, 2, out, 2);
  if (e != RN_OK || validate_only()) return e;
  if (tokens == 0 && accumulate) return RN_OK;
  const EmbedWs w = embed_ws(ws, tokens, width);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool add = accumulate != 0;
  switch (dt) {
    case RN_BF16: return run_embed_bwd<RN_BF16>(tokens, vocab, width, scale, add, ids, dy, dtable, w, st);
    case RN_F16: return run_embed_bwd<RN_F16>(tokens, vocab, width, scale, add, ids, dy, dtable, w, st);
    default: return run_embed_bwd<RN_F32>(tokens, vocab, width, scale, add, ids, dy, dtable, w, st);
  }
}

}  // extern "C"
