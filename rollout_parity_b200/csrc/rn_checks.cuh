// Argument-check helpers shared by librn's host units.  Not part of the public
// interface.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "rn.h"

namespace rn_detail {

struct Range {
  const void* p;
  size_t n;
};

inline bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = uintptr_t(a.p), b0 = uintptr_t(b.p);
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

inline bool aligned16(const void* p) { return (uintptr_t(p) & 15u) == 0; }

inline bool width_ok(int32_t width) { return width >= 8 && width <= 16384 && width % 8 == 0; }
inline bool dtype_ok(rn_dtype dt) { return dt == RN_F32 || dt == RN_BF16 || dt == RN_F16; }

// inputs: read-only ranges; outputs: written ranges.  Outputs must not overlap
// anything else; inputs may overlap one another.  alias_out / alias_in name
// one output that may be exactly the given input (same start, same size): an
// in-place update, which the kernels allow because a thread reads each element
// before it writes the same element and no other thread touches it.
inline rn_status check_ranges(const Range* in, int nin, const Range* out, int nout,
                              int alias_out = -1, int alias_in = -1) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j) {
      if (i == alias_out && j == alias_in && out[i].p == in[j].p && out[i].n == in[j].n) continue;
      if (overlap(out[i], in[j])) return RN_E_ARG;
    }
    for (int j = i + 1; j < nout; ++j)
      if (overlap(out[i], out[j])) return RN_E_ARG;
  }
  return RN_OK;
}

}  // namespace rn_detail
