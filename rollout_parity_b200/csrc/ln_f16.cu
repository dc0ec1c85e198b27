// Layer norm row kernels, forward and backward, for f16 rows (the kernels are in
// ln_rows.cuh; one unit per element format, so that they compile in parallel).
#include "ln_rows.cuh"

namespace rn_detail {
template rn_status launch_ln_fwd<RN_F16>(const Sched&, const LnFwdArgs&, cudaStream_t);
template int64_t ln_bwd_block_rows<RN_F16>(const Sched&, int64_t, bool);
template rn_status launch_ln_bwd<RN_F16>(const Sched&, const LnBwdArgs&, int, cudaStream_t);
}  // namespace rn_detail
