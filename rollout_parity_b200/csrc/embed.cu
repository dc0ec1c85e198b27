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
// Three kernels: k_embed_sort (few tokens: k_embed_sort_few), k_embed_reduce and
// k_embed_join; the first two also clear the rows of dE that no token has.
#include <cooperative_groups.h>

#include <algorithm>
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
  uint32_t* long_count;  // runs longer than a leaf
  uint2* long_runs;      // [tokens/32 + 1] their positions [x, y), in any order
  // sums of the long runs' leaves: of the leaf that starts at position p, row p/32
  // (32 positions hold at most one first leaf of a long run and one later leaf)
  float* first_leaf;     // [tokens/32 + 1][H]
  float* more_leaves;    // [tokens/32 + 1][H]
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
  w.long_count = reinterpret_cast<uint32_t*>(take(4));
  w.long_runs = reinterpret_cast<uint2*>(take(b * 8));
  w.first_leaf = reinterpret_cast<float*>(take(b * size_t(width) * 4));
  w.more_leaves = reinterpret_cast<float*>(take(b * size_t(width) * 4));
  w.bytes = size_t(p - p0);
  return w;
}

// ---------------------------------------------------------------------------
// gradient, pass 1: cluster 0 sorts the tokens by id (stable least-significant-
// digit radix sort); the other clusters clear rows of dE meanwhile.
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

constexpr int kAhead = 4;   // groups of 32 keys a warp has in flight

// The lanes whose digit equals this lane's, among those that are `in`.
__device__ __forceinline__ unsigned same_digit(uint32_t d, bool in) {
  unsigned same = __ballot_sync(0xffffffffu, in);
#pragma unroll
  for (int b = 0; b < kDigitBits; ++b) {
    const bool bit = d & (1u << b);
    const unsigned m = __ballot_sync(0xffffffffu, bit);
    same &= bit ? m : ~m;
  }
  return same;
}

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
  cg::cluster_group cluster = cg::this_cluster();
  if (blockIdx.x >= kSortCtas) {
    const int64_t stride = int64_t(gridDim.x - kSortCtas) * kSortThreads;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int64_t i = int64_t(blockIdx.x - kSortCtas) * kSortThreads + threadIdx.x; i < clear_vecs;
         i += stride)
      clear[i] = zero;
    return;
  }
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
    for (uint32_t p0 = lo; p0 < hi; p0 += 32 * kAhead) {
      uint32_t k[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) k[i] = p0 + 32 * i + lane < hi ? key_at(p0 + 32 * i + lane) : 0;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (p0 + 32 * i >= hi) break;   // uniform
        const bool in = p0 + 32 * i + lane < hi;
        if (in) atomicAdd(&sm.hist[w][(k[i] >> shift) & (bins - 1)], 1u);   // (a count: no order)
      }
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
    for (uint32_t p0 = lo; p0 < hi; p0 += 32 * kAhead) {
      uint32_t k[kAhead], t[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const uint32_t p = p0 + 32 * i + lane;
        k[i] = p < hi ? key_at(p) : 0;
        t[i] = p < hi && pass > 0 ? __ldcg(src_tok + p) : p;
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (p0 + 32 * i >= hi) break;   // uniform
        const bool in = p0 + 32 * i + lane < hi;
        const uint32_t d = (k[i] >> shift) & (bins - 1);
        const unsigned same = same_digit(d, in);
        if (in) {
          const uint32_t at = sm.base[d] + sm.hist[w][d] + __popc(same & below);
          __stcg(dst_key + at, k[i]);
          __stcg(dst_tok + at, t[i]);
        }
        __syncwarp();
        if (in && (same & below) == 0) sm.hist[w][d] += __popc(same);
        __syncwarp();
      }
    }
    // the scatter is complete (the barrier releases this thread's stores to the
    // cluster and acquires the others'), and the totals may be overwritten
    cluster.sync();
  }

  if (blockIdx.x == 0 && tid == 0) *ws.long_count = 0;
}

// Up to 4096 tokens: CTA 0 sorts them in its shared memory, every key in a register
// over a pass.  The rank of a key in its warp's piece is taken once, with the
// count, and completed by the prefix sums; no cluster barrier, no pass through
// global memory.  Measured against the cluster, the whole call: 1000 tokens of 4 KB
// added to 50021 rows (and the old rows' copy) 98 and 105 us, 2000 of 1 KB to 1000
// rows 27 and 32; 8192 of 2 KB 82 and 79.
constexpr int kFewTokens = 4096, kFewGroups = kFewTokens / kSortThreads;
struct FewShared {
  uint16_t count[kSortWarps][1 << kDigitBits];
  uint32_t key[kFewTokens];
  uint16_t tok[kFewTokens];
  uint32_t warp_sum[kSortWarps];
};
__global__ void __launch_bounds__(kSortThreads)
k_embed_sort_few(uint32_t tokens, uint32_t vocab, int passes, const int64_t* __restrict__ ids, EmbedWs ws,
                 uint4* __restrict__ clear, int64_t clear_vecs) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FewShared& sm = *reinterpret_cast<FewShared*>(smem_raw);
  griddep_trigger();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if (blockIdx.x > 0) {
    const int64_t stride = int64_t(gridDim.x - 1) * kSortThreads;
    for (int64_t i = int64_t(blockIdx.x - 1) * kSortThreads + tid; i < clear_vecs; i += stride) clear[i] = zero;
    return;
  }
  const unsigned below = (1u << lane) - 1u;
  const int groups = (tokens + kSortThreads - 1) / kSortThreads;   // of 32 tokens, to a warp
  const uint32_t p0 = uint32_t(w * groups) * 32 + lane;            // this lane's first position
  uint32_t k[kFewGroups], off[kFewGroups];
  uint16_t t[kFewGroups];
#pragma unroll
  for (int i = 0; i < kFewGroups; ++i) {
    const uint32_t p = p0 + 32 * i;
    const int64_t id = i < groups && p < tokens ? __ldg(ids + p) : -1;
    k[i] = id >= 0 && id < int64_t(vocab) ? uint32_t(id) : vocab;
    t[i] = uint16_t(p);
  }
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * kDigitBits;
    uint4* count = reinterpret_cast<uint4*>(sm.count);
    for (int i = tid; i < int(sizeof(sm.count) / 16); i += kSortThreads) count[i] = zero;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewGroups; ++i) {
      if (i >= groups) break;   // uniform
      const bool in = p0 + 32 * i < tokens;
      const uint32_t d = (k[i] >> shift) & ((1u << kDigitBits) - 1);
      const unsigned same = same_digit(d, in);
      const uint32_t c = sm.count[w][d];
      off[i] = c + __popc(same & below);
      __syncwarp();
      if (in && (same & below) == 0) sm.count[w][d] = uint16_t(c + __popc(same));
      __syncwarp();
    }
    __syncthreads();
    // prefix sums in the order (digit, warp): a thread takes 16 warps of a digit
    const int d = tid >> 1, w0 = (tid & 1) * 16;
    uint32_t c[16], mine = 0, all;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      c[i] = mine;
      mine += sm.count[w0 + i][d];
    }
    const uint32_t start = block_prefix(mine, sm.warp_sum, &all);
#pragma unroll
    for (int i = 0; i < 16; ++i) sm.count[w0 + i][d] = uint16_t(start + c[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kFewGroups; ++i) {
      if (i < groups && p0 + 32 * i < tokens) {
        const uint32_t at = sm.count[w][(k[i] >> shift) & ((1u << kDigitBits) - 1)] + off[i];
        sm.key[at] = k[i];
        sm.tok[at] = t[i];
      }
    }
    __syncthreads();
    if (pass + 1 < passes) {
#pragma unroll
      for (int i = 0; i < kFewGroups; ++i) {
        const uint32_t p = p0 + 32 * i;
        if (i < groups && p < tokens) {
          k[i] = sm.key[p];
          t[i] = sm.tok[p];
        }
      }
    }
  }
  for (uint32_t p = tid; p < tokens; p += kSortThreads) {
    ws.key[0][p] = sm.key[p];
    ws.tok[0][p] = sm.tok[p];
  }
  if (tid == 0) *ws.long_count = 0;
}

// ---------------------------------------------------------------------------
// gradient, pass 2: sums of the leaves.  A warp takes 16 sorted positions and
// 512 bytes of their columns (16 a lane), and sums the leaves that start among
// them; the last one may reach up to 31 positions further.  The tokens' rows
// are read four at a time, across the ends of runs: most runs have one or two
// tokens, and a warp to a run had too few bytes in flight.  A run of one leaf is
// written to dE at once.  Measured, 32768 tokens of 4 KB rows over 151936, the
// whole gradient: a warp to a run and 1 KB 227 us, 32 positions 187, 16 170 (8: 177);
// with the clearing here too 180, then eight tokens in flight at 24 warps an SM
// against four at 32 warps 163.
// ---------------------------------------------------------------------------
// The first position of [lo, hi] whose key is at least k, one warp (key[hi] is, or
// hi is one past the last position): 32 probes a step.
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* key, uint32_t tokens, uint32_t lo, uint32_t hi,
                                                uint32_t k) {
  const uint32_t lane = threadIdx.x & 31;
  while (lo < hi) {   // uniform
    const uint32_t step = (hi - lo) / 32 + 1;
    const uint32_t at = min(lo + lane * step, hi);
    const unsigned b = __ballot_sync(0xffffffffu, at >= tokens || __ldcg(key + at) >= k);
    if (b & 1u) return lo;
    const uint32_t f = b ? __ffs(b) - 1 : 32;
    hi = min(lo + f * step, hi);
    lo = lo + (f - 1) * step + 1;
  }
  return lo;
}

// *at = fmt(scale * s), or with ADD fmt(old + scale * s)
template <int DT, bool ADD>
__device__ __forceinline__ void embed_store(uint4* at, const uint4& old, const float2 (&s)[Fmt<DT>::VE / 2],
                                            float scale) {
  using F = Fmt<DT>;
  float2 f[F::VE / 2];
  if constexpr (ADD) F::unpack2(old, f);
#pragma unroll
  for (int q = 0; q < F::VE / 2; ++q) f[q] = ADD ? fma2(s[q], bc2(scale), f[q]) : mul2(s[q], bc2(scale));
  *at = F::pack2v(f);
}

// Clears the rows of [v0, v1), at most 32, that no token has; one warp.
__device__ __forceinline__ void clear_rows(const uint32_t* key, uint32_t tokens, uint32_t v0, uint32_t v1,
                                           int nv, uint4* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  unsigned hit = 0;
  uint32_t p = lower_bound(key, tokens, 0, tokens, v0);
  while (true) {   // uniform; every turn finds a row of its own or is the last
    const uint32_t k = p + lane < tokens ? __ldcg(key + p + lane) : 0xffffffffu;
    const bool in = k < v1;
    hit |= __reduce_or_sync(0xffffffffu, in ? 1u << (k - v0) : 0u);
    if (!__all_sync(0xffffffffu, in)) break;
    p = lower_bound(key, tokens, p + 32, tokens, __shfl_sync(0xffffffffu, k, 31) + 1);   // past that row's run
  }
  for (uint32_t r = v0; r < v1; ++r) {
    if ((hit >> (r - v0)) & 1u) continue;
    for (int v = lane; v < nv; v += 32) out[int64_t(r) * nv + v] = make_uint4(0, 0, 0, 0);
  }
}

constexpr int kSpan = 16;   // sorted positions of a unit
template <int DT, bool ADD>
__global__ void __launch_bounds__(256, ADD ? 3 : 4)
k_embed_reduce(uint32_t tokens, uint32_t vocab, int nv, float scale, int last, EmbedWs ws, uint32_t cleared,
               uint32_t clear_step, uint32_t sum_blocks, const uint4* __restrict__ dy, uint4* __restrict__ out) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE, U = 4;   // tokens (and with ADD, old rows) in flight
  constexpr uint32_t kNone = 0xffffffffu;
  enum { kSkip = 0, kWhole = 1, kFirst = 2, kMore = 3 };   // where a leaf's sum goes
  griddep_trigger();
  griddep_wait();
  const uint32_t* key = ws.key[last];
  const uint32_t* tok = ws.tok[last];
  const int lane = threadIdx.x & 31;
  const uint32_t slabs = (nv + 31) / 32;
  // the blocks that sum and those that clear, spread evenly among one another
  const uint64_t sums_before = uint64_t(blockIdx.x) * sum_blocks / gridDim.x;
  if constexpr (!ADD) {
    if (uint64_t(blockIdx.x + 1) * sum_blocks / gridDim.x == sums_before) {
      const uint64_t v0 = cleared + ((uint64_t(blockIdx.x) - sums_before) * 8 + (threadIdx.x >> 5)) * clear_step;
      if (v0 < vocab) clear_rows(key, tokens, uint32_t(v0), uint32_t(min(v0 + clear_step, uint64_t(vocab))), nv, out);
      return;
    }
  }
  const uint64_t unit = sums_before * (blockDim.x / 32) + (threadIdx.x >> 5);
  const uint32_t slab = uint32_t(unit % slabs), p0 = uint32_t(unit / slabs) * kSpan;
  if (p0 >= tokens) return;
  const int v = int(slab) * 32 + lane;
  const bool col = v < nv;

  // positions p0 + lane and p0 + 32 + lane
  const uint32_t a0 = p0 + lane, a1 = a0 + 32;
  const uint32_t k0 = a0 < tokens ? __ldcg(key + a0) : kNone, k1 = a1 < tokens ? __ldcg(key + a1) : kNone;
  const uint32_t t0 = a0 < tokens ? __ldcg(tok + a0) : 0, t1 = a1 < tokens ? __ldcg(tok + a1) : 0;
  const uint32_t before = p0 > 0 ? __ldcg(key + p0 - 1) : kNone;
  // the start of position p0's run: p0 itself, or where its key first stands
  const uint32_t key0 = __shfl_sync(0xffffffffu, k0, 0);
  const uint32_t start0 = key0 == before ? lower_bound(key, tokens, 0, p0, key0) : p0;
  const uint32_t up = __shfl_up_sync(0xffffffffu, k0, 1);
  const bool valid = a0 < tokens;
  const unsigned upto = 0xffffffffu >> (31 - lane);         // lanes 0..lane
  const unsigned changes = __ballot_sync(0xffffffffu, valid && k0 != (lane == 0 ? before : up));
  const uint32_t start = changes & upto ? p0 + 31 - __clz(changes & upto) : start0;   // of the lane's run
  const bool leaf = valid && lane < kSpan && ((a0 - start) & (kLeaf - 1)) == 0;
  const unsigned leaves = __ballot_sync(0xffffffffu, leaf);
  if (leaves == 0) return;   // inside a long run's leaf
  const int first = __ffs(leaves) - 1, final = 31 - __clz(leaves);
  // the last leaf reaches to its run's end or 32 positions, past these ones
  const uint32_t key_f = __shfl_sync(0xffffffffu, k0, final);
  const unsigned same0 = __ballot_sync(0xffffffffu, k0 == key_f), same1 = __ballot_sync(0xffffffffu, k1 == key_f);
  const uint64_t same = (uint64_t(same1) << 32 | same0) >> final;
  const int length = ~same == 0 ? kLeaf : min(__ffsll(~same) - 1, kLeaf);
  const int end = final + length;   // the tokens to read: [first, end) counted from p0
  // what becomes of the leaf that starts at this lane
  const unsigned later = leaves & ~upto;
  const int to = later ? __ffs(later) - 1 : end;            // one past its last position
  const uint32_t next0 = __shfl_sync(0xffffffffu, k0, to & 31), next1 = __shfl_sync(0xffffffffu, k1, to & 31);
  const bool goes_on = to - lane == kLeaf && (to < 32 ? next0 : next1) == k0;
  const bool head = a0 == start;
  const uint32_t kind = !leaf || k0 >= vocab ? kSkip : !head ? kMore : goes_on ? kFirst : kWhole;
  const uint32_t dest = kind << 30 | (kind == kWhole ? k0 : a0 / kLeaf);
  if (slab == 0) {   // lists the long runs that start here
    for (unsigned m = __ballot_sync(0xffffffffu, kind == kFirst); m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const uint32_t id = __shfl_sync(0xffffffffu, k0, l);
      const uint32_t e = lower_bound(key, tokens, p0 + l + kLeaf, tokens, id + 1);
      if (lane == 0) ws.long_runs[atomicAdd(ws.long_count, 1u)] = make_uint2(p0 + l, e);
    }
  }

  float2 acc[VE / 2];
  uint32_t d = __shfl_sync(0xffffffffu, dest, first);       // of the leaf being summed
  uint4 old = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int q = 0; q < VE / 2; ++q) acc[q] = bc2(-0.0f);
  auto flush = [&]() {
    const uint32_t row = d & 0x3fffffffu;
    if (d >> 30 == kWhole) {
      if (col) embed_store<DT, ADD>(out + int64_t(row) * nv + v, old, acc, scale);
    } else if (d >> 30 != kSkip) {
      float4* part = reinterpret_cast<float4*>(d >> 30 == kFirst ? ws.first_leaf : ws.more_leaves) +
                     (uint64_t(row) * nv + v) * (VE / 4);
      if (col) {
#pragma unroll
        for (int q = 0; q < VE / 4; ++q)
          part[q] = make_float4(acc[2 * q].x, acc[2 * q].y, acc[2 * q + 1].x, acc[2 * q + 1].y);
      }
    }
  };
  for (int i = first; i < end; i += U) {
    uint4 r[U], o[ADD ? U : 1];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int x = i + j;
      const uint32_t lo = __shfl_sync(0xffffffffu, t0, x & 31), hi = __shfl_sync(0xffffffffu, t1, x & 31);
      if (x < end && col) r[j] = __ldcs(dy + int64_t(x < 32 ? lo : hi) * nv + v);
      if constexpr (ADD) {
        const uint32_t dx = __shfl_sync(0xffffffffu, dest, x & 31);
        if (x < kSpan && dx >> 30 == kWhole && col) o[j] = __ldcs(out + int64_t(dx & 0x3fffffffu) * nv + v);
      }
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int x = i + j;
      if (x < end) {   // uniform
        if (x < kSpan && ((leaves >> x) & 1u)) {
          if (x > first) {
            flush();
            d = __shfl_sync(0xffffffffu, dest, x);
#pragma unroll
            for (int q = 0; q < VE / 2; ++q) acc[q] = bc2(-0.0f);
          }
          if constexpr (ADD) old = o[j];
        }
        float2 f[VE / 2];
        F::unpack2(r[j], f);
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) acc[q] = add2(acc[q], f[q]);
      }
    }
  }
  flush();
}

// ---------------------------------------------------------------------------
// gradient, pass 3: the leaves of the long runs, joined by the level-by-level
// pairwise tree.  A CTA takes one run and 32 16-byte vectors' columns at a
// time; its eight warps stream aligned power-of-two blocks of leaves (perfect
// subtrees), joined in shared memory.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
template <int DT, bool ADD>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_embed_join(int nv, float scale, int last, EmbedWs ws, uint4* __restrict__ out) {
  using F = Fmt<DT>;
  constexpr int VE = F::VE;
  griddep_trigger();
  griddep_wait();
  __shared__ float sm[kJoinWarps][32][VE + 1];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t cols = (nv + 31) / 32;
  const uint32_t* key = ws.key[last];
  const uint64_t items = uint64_t(__ldcg(ws.long_count)) * cols;
  for (uint64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const uint2 run = __ldcg(ws.long_runs + it / cols);
    const uint32_t s = run.x, e = run.y, id = __ldcg(key + s);
    const int v = int(it % cols) * 32 + lane;
    const uint32_t leaves = (e - s + kLeaf - 1) / kLeaf;
    uint32_t per = 1;                       // leaves per warp: a power of two
    while (per * kJoinWarps < leaves) per <<= 1;
    const uint32_t l0 = w * per;
    const uint32_t cnt = l0 >= leaves ? 0 : (leaves - l0 < per ? leaves - l0 : per);
    auto leaf_at = [&](uint32_t l, float2 (&f)[VE / 2]) {
      const float4* p = reinterpret_cast<const float4*>(l == 0 ? ws.first_leaf : ws.more_leaves) +
                        (uint64_t(s / kLeaf + l) * nv + v) * (VE / 4);
#pragma unroll
      for (int q = 0; q < VE / 4; ++q) {
        const float4 x = __ldcg(p + q);
        f[2 * q] = make_float2(x.x, x.y);
        f[2 * q + 1] = make_float2(x.z, x.w);
      }
    };
    // leaves in fours (perfect subtrees, loaded at once), and a stack of pending
    // subtrees: one of 2^k fours for every bit k of the fours taken so far
    float2 stack[23][VE / 2], res[VE / 2];
    int top = 0;
    if (v < nv && cnt > 0) {
      for (uint32_t i = 0; i < cnt; i += 4) {
        float2 f[4][VE / 2];
        const int n = cnt - i < 4 ? int(cnt - i) : 4;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) leaf_at(l0 + i + j, f[j]);
        if (n > 1) {
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) f[0][q] = add2(f[0][q], f[1][q]);
        }
        if (n > 3) {
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) f[2][q] = add2(f[2][q], f[3][q]);
        }
        if (n > 2) {
#pragma unroll
          for (int q = 0; q < VE / 2; ++q) f[0][q] = add2(f[0][q], f[2][q]);
        }
        if (n == 4) {
          for (uint32_t k = i / 4; k & 1u; k >>= 1) {
            --top;
#pragma unroll
            for (int q = 0; q < VE / 2; ++q) f[0][q] = add2(stack[top][q], f[0][q]);
          }
        }
#pragma unroll
        for (int q = 0; q < VE / 2; ++q) stack[top][q] = f[0][q];
        ++top;
      }
      // pending subtrees, smallest (rightmost) first
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
      uint4* at = out + int64_t(id) * nv + v;
      embed_store<DT, ADD>(at, ADD ? *at : make_uint4(0, 0, 0, 0), p[0], scale);
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
  if (tokens <= kFewTokens) {
    *last = 0;
    static KernelPrep few;
    const int fit = prepare_kernel(k_embed_sort_few, kSortThreads, sizeof(FewShared), few) * sm_count();
    return launch_pdl(k_embed_sort_few, dim3(clear ? (fit > 1 ? fit : 2) : 1), dim3(kSortThreads), sizeof(FewShared), st,
                      uint32_t(tokens), uint32_t(vocab), passes, ids, ws, static_cast<uint4*>(clear),
                      int64_t(clear_bytes / 16));
  }
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

template <int DT, bool ADD>
rn_status run_embed_bwd(int64_t tokens, int64_t vocab, int width, float scale, const int64_t* ids,
                        const void* dy, void* dtable, const EmbedWs& ws,
                        cudaStream_t st) {
  const int nv = width / Fmt<DT>::VE;
  int last = 0;
  // Rows cleared beside the sort, which takes about 8 us and 1 us for every 4096
  // tokens, at 5 MB a us; the others are cleared beside the sums, where the rows
  // that a token has need no clearing.
  const int64_t beside = (int64_t(8) + tokens / 4096) * 5000000 / (int64_t(nv) * 16);
  const int64_t cleared = ADD ? vocab : tokens == 0 || beside > vocab ? vocab : beside;
  rn_status e = launch_sort(tokens, vocab, ids, ws, ADD ? nullptr : dtable,
                            size_t(cleared) * nv * 16, &last, st);
  if (e != RN_OK || tokens == 0) return e;
  static KernelPrep prep_join;
  const uint64_t units = uint64_t((tokens + kSpan - 1) / kSpan) * ((nv + 31) / 32);
  // a clearing warp takes about 32 KB, 32 rows at most
  const int64_t step = std::min<int64_t>(32, std::max<int64_t>(1, 32768 / (int64_t(nv) * 16)));
  const uint64_t sums = (units + 7) / 8, clears = (vocab - cleared + 8 * step - 1) / (8 * step);
  e = launch_pdl(k_embed_reduce<DT, ADD>, dim3(unsigned(sums + clears)), dim3(256), 0, st, uint32_t(tokens),
                 uint32_t(vocab), nv, scale, last, ws, uint32_t(cleared), uint32_t(step), uint32_t(sums),
                 static_cast<const uint4*>(dy), static_cast<uint4*>(dtable));
  if (e != RN_OK || tokens <= kLeaf) return e;   // no run longer than a leaf
  const int jfit = prepare_kernel(k_embed_join<DT, ADD>, 32 * kJoinWarps, 0, prep_join) * sm_count();
  const uint64_t items = uint64_t(tokens / (kLeaf + 1)) * ((nv + 31) / 32);
  const uint64_t wave = uint64_t(jfit < 4 * sm_count() ? jfit : 4 * sm_count());   // few runs are long
  return launch_pdl(k_embed_join<DT, ADD>, dim3(unsigned(items < wave ? items : wave)),
                    dim3(32 * kJoinWarps), 0, st, nv, scale, last, ws,
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
#define RN_EMBED_BWD(DT_)                                                                                   \
  return accumulate ? run_embed_bwd<DT_, true>(tokens, vocab, width, scale, ids, dy, dtable, w, st)        \
                    : run_embed_bwd<DT_, false>(tokens, vocab, width, scale, ids, dy, dtable, w, st)
  switch (dt) {
    case RN_BF16: RN_EMBED_BWD(RN_BF16);
    case RN_F16: RN_EMBED_BWD(RN_F16);
    default: RN_EMBED_BWD(RN_F32);
  }
#undef RN_EMBED_BWD
}

}  // extern "C"
