// dispatch.hip -- tokens' rows brought to the rows of their experts: stored
// codes with their scales, or the per-token cast of bf16 rows.
//
// A row is read once and written top_k times: bound by HBM writes.
//
// gfx950 design. A wave takes one piece of a token's row (64 chunks of 16
// bytes, or 512 columns to cast) and writes it to each of the token's rows,
// whose numbers are the same in every lane. Workgroups behind the tokens'
// write the padding of the runs.
#include "qcast_runs.h"

namespace qcast {
namespace {

constexpr uint32_t kWaves = kThreads / 64;

__device__ __forceinline__ uint32_t scale_index(uint32_t row, uint32_t w, uint32_t words,
                                                uint32_t pad) {
  return pad ? w * pad + row : row * words + w;
}

// Pieces of a token: one for each 64 chunks, then one for its scales.
__global__ __launch_bounds__(kThreads) void dispatch_codes_kernel(DispatchCodes p, uint32_t pieces,
                                                                  uint32_t groups,
                                                                  uint32_t first) {
  const uint32_t lane = threadIdx.x & 63, group = blockIdx.x + first;
  const uint32_t segs = (p.chunks + 63) / 64;
  if (group >= groups) {
    uint32_t r0, r1;
    pad_range(p.runs, group - groups, r0, r1);
    for (uint32_t r = r0; r < r1; ++r) {
      for (uint32_t c = threadIdx.x; c < p.chunks; c += kThreads)
        store_stream(p.out + (uint64_t)r * p.chunks + c, u32x4{0, 0, 0, 0});
      if (p.sf_out)
        for (uint32_t w = threadIdx.x; w < p.words; w += kThreads)
          p.sf_out[scale_index(r, w, p.words, p.pad_out)] = 0;
    }
    return;
  }
  const uint64_t item = (uint64_t)group * kWaves + (threadIdx.x >> 6);
  const uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / pieces));
  const uint32_t piece = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % pieces));
  if (t >= p.runs.tokens) return;
  const int32_t* dest = p.runs.dest + (uint64_t)t * p.runs.top_k;
  if (piece < segs) {
    const uint32_t c = piece * 64 + lane;
    if (c >= p.chunks) return;
    const u32x4 v = p.in[(uint64_t)t * p.chunks + c];
    for (uint32_t k = 0; k < p.runs.top_k; k += kBatch) {
      uint32_t r[kBatch];
      slot_rows(dest, k, p.runs.top_k, r);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (r[j] < p.runs.rows) store_stream(p.out + (uint64_t)r[j] * p.chunks + c, v);
    }
  } else {
    for (uint32_t w = lane; w < p.words; w += 64) {
      const uint32_t v = p.sf_in[scale_index(t, w, p.words, p.pad_in)];
      for (uint32_t k = 0; k < p.runs.top_k; k += kBatch) {
        uint32_t r[kBatch];
        slot_rows(dest, k, p.runs.top_k, r);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (r[j] < p.runs.rows) p.sf_out[scale_index(r[j], w, p.words, p.pad_out)] = v;
      }
    }
  }
}

// Without weights a row is cast once, whatever the number of its places (4096 x 8
// of 7168, runs of 128: 54 us). With weights each place is: its weight is loaded
// behind the stores of the place before, and its groups' maxima are formed again
// (65 to 84 us).
template <int kFmt, bool kWeighted>
__global__ __launch_bounds__(kThreads) void dispatch_cast_kernel(DispatchCast p, uint32_t segs,
                                                                 uint32_t groups, uint32_t first) {
  const uint32_t lane = threadIdx.x & 63, group = blockIdx.x + first;
  if (group >= groups) {
    uint32_t r0, r1;
    pad_range(p.runs, group - groups, r0, r1);
    const float zero[8] = {};
    for (uint32_t c = threadIdx.x; c < p.chunks; c += kThreads) {
      const ChunkScale s = chunk_scale<kFmt>(p.cast, c, zero);
      for (uint32_t r = r0; r < r1; ++r) {
        put_codes<kFmt>(p.cast, r, p.chunks, c, zero);
        put_scale(p.cast, r, s);
      }
    }
    return;
  }
  const uint64_t item = (uint64_t)group * kWaves + (threadIdx.x >> 6);
  const uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / segs));
  const uint32_t seg = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % segs));
  const uint32_t c = seg * 64 + lane;
  if (t >= p.runs.tokens || c >= p.chunks) return;      // a group's lanes leave together
  const u32x4 raw = reinterpret_cast<const u32x4*>(p.x)[(uint64_t)t * p.chunks + c];
  float x[8], y[8];
  unpack8(raw, x);
  ChunkScale s;
  if constexpr (!kWeighted) {
    s = chunk_scale<kFmt>(p.cast, c, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * s.inv;
  }
  const uint64_t slot = (uint64_t)t * p.runs.top_k;
  for (uint32_t k = 0; k < p.runs.top_k; k += kBatch) {
    uint32_t r[kBatch];
    slot_rows(p.runs.dest + slot, k, p.runs.top_k, r);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (r[j] >= p.runs.rows) continue;
      if constexpr (kWeighted) {
        const float w = p.weight[slot + k + j];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w * x[i];
        s = chunk_scale<kFmt>(p.cast, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * s.inv;
      }
      put_codes<kFmt>(p.cast, r[j], p.chunks, c, y);
      put_scale(p.cast, r[j], s);
    }
  }
}

template <int kFmt>
auto cast_kernel(bool weighted) {
  return weighted ? dispatch_cast_kernel<kFmt, true> : dispatch_cast_kernel<kFmt, false>;
}

}  // namespace

hipError_t launch_dispatch_codes(const DispatchCodes& p, hipStream_t stream) {
  const uint32_t pieces = (p.chunks + 63) / 64 + (p.sf_in ? 1 : 0);
  const uint64_t groups = ((uint64_t)p.runs.tokens * pieces + kWaves - 1) / kWaves;
  const uint64_t all = groups + pad_groups(p.runs);
  if (all >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  return launch_groups(dispatch_codes_kernel, all, kThreads, stream, p, pieces,
                       (uint32_t)groups);
}

hipError_t launch_dispatch_cast(const DispatchCast& p, hipStream_t stream) {
  const uint32_t segs = (p.chunks + 63) / 64;
  const uint64_t groups = ((uint64_t)p.runs.tokens * segs + kWaves - 1) / kWaves;
  const uint64_t all = groups + pad_groups(p.runs);
  if (all >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  const bool w = p.weight != nullptr;
  auto kernel = p.cast.fmt == kE4M3   ? cast_kernel<kE4M3>(w)
                : p.cast.fmt == kE5M2 ? cast_kernel<kE5M2>(w)
                : p.cast.fmt == kE2M1 ? cast_kernel<kE2M1>(w)
                                      : cast_kernel<kE5M6>(w);
  return launch_groups(kernel, all, kThreads, stream, p, segs, (uint32_t)groups);
}

}  // namespace qcast
