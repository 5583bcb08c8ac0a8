// qcast_runs.h -- device helpers of the kernels that bring tokens' rows to
// their experts: a slot's row, and the padding rows of the experts' runs.
#pragma once

#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {

constexpr uint32_t kPadRows = 8;       // padding rows of a workgroup

// Workgroups that write the padding (behind those of the tokens).
inline uint64_t pad_groups(const ExpertRuns& r) {
  return r.offsets && r.align > 1
             ? (uint64_t)r.experts * ((r.align - 1 + kPadRows - 1) / kPadRows) : 0;
}

// Padding rows [first, last) of workgroup g; what the arrays say is held to
// the rows there are.
__device__ __forceinline__ void pad_range(const ExpertRuns& r, uint32_t g, uint32_t& first,
                                          uint32_t& last) {
  const uint32_t per = (r.align - 1 + kPadRows - 1) / kPadRows;
  const uint32_t e = g / per;
  const int64_t from = (int64_t)r.offsets[e] + r.counts[e] + (int64_t)(g - e * per) * kPadRows;
  const int64_t end = r.offsets[e + 1] < (int64_t)r.rows ? r.offsets[e + 1] : (int64_t)r.rows;
  first = last = 0;
  if (from < 0 || from >= end) return;
  first = (uint32_t)from;
  last = end - from < kPadRows ? (uint32_t)end : first + kPadRows;
}

}  // namespace qcast
