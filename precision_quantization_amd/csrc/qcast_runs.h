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

// The rows of a token's slots k0 .. k0 + 7, the same in every lane; kNoRow behind
// its last slot. One batch of loads, vector loads where the kernel's loop stores.
constexpr int kBatch = 8;
constexpr uint32_t kNoRow = 0xffffffffu;
__device__ __forceinline__ void slot_rows(const int32_t* dest, uint32_t k0, uint32_t top_k,
                                          uint32_t (&r)[kBatch]) {
#pragma unroll
  for (int j = 0; j < kBatch; ++j)
    r[j] = (uint32_t)dest[k0 + j < top_k ? k0 + j : top_k - 1];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) r[j] = k0 + j < top_k ? r[j] : kNoRow;
}

// The scale of a chunk's group as it is stored: the word and its place in a
// row, in the lane that stores it.
struct ChunkScale {
  float inv;
  uint32_t word, at;
  bool stores;
};
template <int kFmt>
__device__ __forceinline__ ChunkScale chunk_scale(const RowCast& rc, uint32_t c,
                                                  const float v[8]) {
  const uint32_t lane = threadIdx.x & 63, n = 1u << rc.shift;
  Scale s = group_scale<kFmt>(run_max(absmax8_of(v), rc.shift), rc.floor);
  if (rc.lay.flags & kSfRound) s = round_scale_pow2(s);
  ChunkScale o;
  o.inv = s.inv;
  o.word = __float_as_uint(s.sf);
  o.at = c >> rc.shift;
  o.stores = (lane & (n - 1)) == 0;
  if (rc.lay.flags & kSfPacked) {
    const uint32_t e = o.word >> 23;
    o.word = e | ((uint32_t)__shfl((int)e, (int)(lane + n)) << 8) |
             ((uint32_t)__shfl((int)e, (int)(lane + 2 * n)) << 16) |
             ((uint32_t)__shfl((int)e, (int)(lane + 3 * n)) << 24);
    o.at /= 4;
    o.stores = (lane & (4 * n - 1)) == 0;
  }
  return o;
}
__device__ __forceinline__ void put_scale(const RowCast& rc, uint32_t row, const ChunkScale& s) {
  if (!s.stores) return;
  const uint32_t words = rc.lay.flags & kSfPacked ? rc.lay.gpr / 4 : rc.lay.gpr;
  const bool col = (rc.lay.flags & kSfColMajor) != 0;
  uint32_t* to = static_cast<uint32_t*>(rc.sf) + (col ? row : (uint64_t)row * words);
  to[col ? s.at * rc.lay.rows_pad : s.at] = s.word;
}
// The codes of chunk c of a row from values already times the inverse scale.
template <int kFmt>
__device__ __forceinline__ void put_codes(const RowCast& rc, uint32_t row, uint32_t chunks,
                                          uint32_t c, const float y[8]) {
  store_chunk8<kFmt>(rc.q + (uint64_t)row * chunks * code_bytes<kFmt>(8), c, y);
}

}  // namespace qcast
