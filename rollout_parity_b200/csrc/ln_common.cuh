// Declarations shared by the layer norm's host unit (ln.cu) and its row-kernel
// units (ln_{bf16,f16,f32}.cu).  Not part of the public interface.
#pragma once

#include "rn_common.cuh"

namespace rn_detail {

struct LnFwdArgs {
  int64_t rows;
  int H, nv;
  float eps, inv_h;
  const uint4* x;
  const float* w;
  const float* b;   // NULL: no bias
  uint4* y;
  float* mean;      // NULL: not written
  float* rstd;      // NULL: not written
};

struct LnBwdArgs {
  int64_t rows;
  int64_t block_rows;    // rows per CTA, a multiple of its teams
  int H, nv;
  float inv_h;
  const uint4* x;
  const float* w;
  const uint4* dy;
  const float* mean;
  const float* rstd;
  const uint8_t* mask;   // rows with mask[r] == 0 add nothing to dw, db (NULL: every row)
  uint4* dx;
  float* pw;             // [CTAs][H] partials of dw (dw itself with one CTA)
  float* pb;             // [CTAs][H] partials of db, NULL: no db
};

// rows per backward CTA (its partial of dw and db), from the sizes and the
// element format only
template <int DT>
int64_t ln_bwd_block_rows(const Sched& s, int64_t rows, bool wide);
template <int DT>
rn_status launch_ln_fwd(const Sched& s, const LnFwdArgs& a, cudaStream_t st);
template <int DT>
rn_status launch_ln_bwd(const Sched& s, const LnBwdArgs& a, int ctas, cudaStream_t st);

// The backward's team of a row: the forward's (the RMS norm's) for up to 128
// vectors, else 24, 32 or 40 elements a thread and a power of two of warps,
// whichever leaves the fewest slots empty (the more elements at a tie).
inline Sched ln_bwd_sched(int32_t width, rn_dtype dt) {
  const int nv = width / vec_elems(dt);
  Sched s = row_sched(width, dt);
  if (nv <= 128) return s;
  int best = 0;
  for (int T = 32; T <= 512; T *= 2) {
    for (int e = 3; e <= 5; ++e) {
      const int k = e * 8 / vec_elems(dt);
      if (T * k < nv || (T == 512 && e == 5) || (best && T * k > best)) continue;
      if (best && T * k == best && k < s.K) continue;
      best = T * k;
      s.T = T;
      s.K = k;
    }
  }
  return s;
}

}  // namespace rn_detail
