// Layer norm host unit: argument checks, workspace layout, launches
// (include/rn.h, "Layer norm").
#include <cmath>

#include "ln_common.cuh"
#include "rn_checks.cuh"

using namespace rn_detail;

namespace {

// dw and db from the CTAs' partials, n rows of each: the level-by-level
// pairwise tree, one CTA of W warps per 32 columns.  Warp w streams the aligned
// block of L rows [wL, (w+1)L), a perfect subtree, all of them in flight; the
// warps' results are joined by the tree in shared memory.
template <int LB, int W>
__global__ void __launch_bounds__(32 * W)
k_ln_fold(const float* __restrict__ pw, const float* __restrict__ pb, int n, int H,
          float* __restrict__ dw, float* __restrict__ db) {
  constexpr int L = 1 << LB;
  griddep_trigger();
  griddep_wait();
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const float* in = blockIdx.y == 0 ? pw : pb;
  float* out = blockIdx.y == 0 ? dw : db;
  const int c = blockIdx.x * 32 + lane;
  const int start = wid * L;
  const int cnt = c >= H || n <= start ? 0 : (n - start < L ? n - start : L);
  float v[L];
#pragma unroll
  for (int i = 0; i < L; ++i) v[i] = i < cnt ? __ldcg(in + int64_t(start + i) * H + c) : 0.0f;
  TreeCounter<LB, float> tc;
#pragma unroll
  for (int i = 0; i < L; ++i)
    if (i < cnt) tc.push(i, v[i]);
  __shared__ float sm[W][32];
  sm[wid][lane] = cnt > 0 ? tc.finish(cnt) : 0.0f;
  __syncthreads();
  if (wid == 0 && c < H) {
    const int nw = (n + L - 1) / L;
    float p[W];
#pragma unroll
    for (int i = 0; i < W; ++i) p[i] = sm[i][lane];
#pragma unroll
    for (int s = 1; s < W; s <<= 1) {
#pragma unroll
      for (int l = 0; l + s < W; l += 2 * s)
        if (l + s < nw) p[l] = __fadd_rn(p[l], p[l + s]);
    }
    out[c] = p[0];
  }
}

// Partial rows the backward writes: one per CTA (ln_bwd_block_rows).
struct LnPlan {
  Sched s;
  int64_t block_rows;
  int ctas;
};

LnPlan ln_plan(int64_t rows, int32_t width, rn_dtype dt) {
  LnPlan p;
  p.s = ln_bwd_sched(width, dt);
  const bool wide = width / vec_elems(dt) > 128;
  p.block_rows = dt == RN_F32    ? ln_bwd_block_rows<RN_F32>(p.s, rows, wide)
                 : dt == RN_BF16 ? ln_bwd_block_rows<RN_BF16>(p.s, rows, wide)
                                 : ln_bwd_block_rows<RN_F16>(p.s, rows, wide);
  p.ctas = int((rows + p.block_rows - 1) / p.block_rows);
  return p;
}

size_t ln_ws_bytes(int64_t rows, int32_t width, rn_dtype dt) {
  if (rows <= 0 || rows > kMaxRows || !width_ok(width) || !dtype_ok(dt)) return 0;
  const LnPlan p = ln_plan(rows, width, dt);
  return p.ctas > 1 ? size_t(p.ctas) * width * 2 * sizeof(float) : 0;
}

rn_status launch_ln_fold(const float* pw, const float* pb, int n, int H, float* dw, float* db,
                         cudaStream_t st) {
  const dim3 grid((H + 31) / 32, db ? 2 : 1);
  if (n <= 64) return launch_pdl(k_ln_fold<3, 8>, grid, dim3(256), 0, st, pw, pb, n, H, dw, db);
  if (n <= 256) return launch_pdl(k_ln_fold<3, 32>, grid, dim3(1024), 0, st, pw, pb, n, H, dw, db);
  if (n <= 512) return launch_pdl(k_ln_fold<4, 32>, grid, dim3(1024), 0, st, pw, pb, n, H, dw, db);
  if (n <= 1024) return launch_pdl(k_ln_fold<5, 32>, grid, dim3(1024), 0, st, pw, pb, n, H, dw, db);
  return RN_E_ARG;   // unreachable: at most 592 CTAs
}

}  // namespace

extern "C" {

rn_status layernorm_fwd(int64_t rows, int32_t width, float eps, rn_dtype dt, const void* x,
                        const float* w, const float* b, void* y, float* mean, float* rstd,
                        rn_stream stream) {
  begin_call();
  if (rows < 0 || rows > kMaxRows || !std::isfinite(eps) || eps < 0.0f) return RN_E_ARG;
  if (!dtype_ok(dt)) return RN_E_DTYPE;
  if (!width_ok(width)) return RN_E_WIDTH;
  if (!w || (rows > 0 && (!x || !y))) return RN_E_ARG;
  const size_t tb = size_t(rows) * size_t(width) * elem_bytes(dt);
  if (rows > 0 && (!aligned16(x) || !aligned16(w) || !aligned16(b) || !aligned16(y) ||
                   (uintptr_t(mean) & 3u) || (uintptr_t(rstd) & 3u)))
    return RN_E_ALIGN;
  const size_t vb = size_t(width) * 4, sb = size_t(rows) * 4;
  const Range in[] = {{x, tb}, {w, vb}, {b, vb}};
  const Range out[] = {{y, tb}, {mean, sb}, {rstd, sb}};
  const rn_status e = check_ranges(in, 3, out, 3, 0, 0);   // y may be x itself
  if (e != RN_OK) return e;
  if (validate_only() || rows == 0) return RN_OK;
  const LnFwdArgs a{rows, width, width / vec_elems(dt), eps, 1.0f / float(width),
                    static_cast<const uint4*>(x), w, b,
                    static_cast<uint4*>(y), mean, rstd};
  const Sched s = row_sched(width, dt);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (dt) {
    case RN_BF16: return launch_ln_fwd<RN_BF16>(s, a, st);
    case RN_F16: return launch_ln_fwd<RN_F16>(s, a, st);
    default: return launch_ln_fwd<RN_F32>(s, a, st);
  }
}

size_t layernorm_bwd_workspace_bytes(int64_t rows, int32_t width, rn_dtype dt) {
  return ln_ws_bytes(rows, width, dt);
}

rn_status layernorm_bwd(int64_t rows, int32_t width, rn_dtype dt, const void* x, const float* w,
                        const void* dy, const float* mean, const float* rstd,
                        const uint8_t* row_mask, void* dx, float* dw, float* db, void* ws,
                        size_t ws_bytes, rn_stream stream) {
  begin_call();
  if (rows < 0 || rows > kMaxRows) return RN_E_ARG;
  if (!dtype_ok(dt)) return RN_E_DTYPE;
  if (!width_ok(width)) return RN_E_WIDTH;
  if (!w || !dw || (rows > 0 && (!x || !dy || !mean || !rstd || !dx))) return RN_E_ARG;
  if (!aligned16(w) || !aligned16(dw) || !aligned16(db)) return RN_E_ALIGN;
  const size_t need = ln_ws_bytes(rows, width, dt);
  if (rows > 0) {
    if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || (uintptr_t(mean) & 3u) ||
        (uintptr_t(rstd) & 3u))
      return RN_E_ALIGN;
    if (need > 0 && (!ws || ws_bytes < need)) return RN_E_WORKSPACE;
    if (!aligned16(ws)) return RN_E_ALIGN;
  }
  const size_t tb = size_t(rows) * size_t(width) * elem_bytes(dt);
  const size_t vb = size_t(width) * 4, sb = size_t(rows) * 4;
  const Range in[] = {{x, tb}, {w, vb}, {dy, tb}, {mean, sb}, {rstd, sb}, {row_mask, size_t(rows)}};
  const Range out[] = {{dx, tb}, {dw, vb}, {db, vb}, {ws, need}};
  rn_status e = check_ranges(in, 6, out, 4, 0, 2);   // dx may be dy itself
  if (e != RN_OK) return e;
  if (validate_only()) return RN_OK;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // the empty sums
    e = fill_neg_zero(dw, width, st);
    return e == RN_OK && db ? fill_neg_zero(db, width, st) : e;
  }
  const LnPlan p = ln_plan(rows, width, dt);
  float* pw = p.ctas > 1 ? static_cast<float*>(ws) : dw;
  float* pb = !db ? nullptr : p.ctas > 1 ? pw + size_t(p.ctas) * width : db;
  const LnBwdArgs a{rows, p.block_rows, width, width / vec_elems(dt), 1.0f / float(width),
                    static_cast<const uint4*>(x), w,
                    static_cast<const uint4*>(dy), mean, rstd, row_mask, static_cast<uint4*>(dx),
                    pw, pb};
  switch (dt) {
    case RN_BF16: e = launch_ln_bwd<RN_BF16>(p.s, a, p.ctas, st); break;
    case RN_F16: e = launch_ln_bwd<RN_F16>(p.s, a, p.ctas, st); break;
    default: e = launch_ln_bwd<RN_F32>(p.s, a, p.ctas, st); break;
  }
  if (e != RN_OK || p.ctas == 1) return e;
  return launch_ln_fold(pw, pb, p.ctas, width, dw, db, st);
}

}  // extern "C"
