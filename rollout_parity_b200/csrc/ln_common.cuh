// Declarations shared by the layer norm's host unit (ln.cu) and its row-kernel
// units (ln_{bf16,f16,f32}.cu).  Not part of the public interface.
#pragma once

#include "rn_common.cuh"

namespace rn_detail {

struct LnFwdArgs {
  int64_t rows;
  int H, nv;
  float eps, inv_h;
  int h_pow2;
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
  int h_pow2;
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
int64_t ln_bwd_block_rows(const Sched& s, int64_t rows);
template <int DT>
rn_status launch_ln_fwd(const Sched& s, const LnFwdArgs& a, cudaStream_t st);
template <int DT>
rn_status launch_ln_bwd(const Sched& s, const LnBwdArgs& a, int64_t block_rows, int ctas,
                        cudaStream_t st);

}  // namespace rn_detail
