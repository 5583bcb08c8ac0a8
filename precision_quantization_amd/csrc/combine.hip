// combine.hip -- the experts' output rows brought back to their tokens,
// weighted and summed, and the gradient of that.
//
// Forward: out[t] = base[t] + sum_k w[t][k] y[dest[t][k]], one fma per value
// in fp32. Backward: dy[dest[t][k]] = w[t][k] dout[t], cast per token, and
// dw[t][k] = <dout[t], y[dest[t][k]]>. Every value of y is touched once: both
// are bound by HBM bandwidth.
#include "qcast_runs.h"

namespace qcast {
namespace {

constexpr uint32_t kWaves = kThreads / 64;

// A wave sums 512 columns of one token, eight rows in flight. A row is a buffer
// of its own (of no bytes for a slot without one: its loads give zeros without
// reading anything, and its weight is taken as 0).
__global__ __launch_bounds__(kThreads) void combine_kernel(Combine p, uint32_t segs) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / segs));
  const uint32_t seg = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % segs));
  if (t >= p.tokens) return;
  const uint32_t c = seg * 64 + lane, bytes = p.chunks * 16;
  const uint64_t slot = (uint64_t)t * p.top_k;
  float acc[8] = {};
  if (p.base)
    unpack8(buffer_load16<0>(row_buffer(p.base, (uint64_t)t * bytes, bytes), c * 16), acc);
  for (uint32_t k = 0; k < p.top_k; k += kBatch) {
    uint32_t r[kBatch];
    float w[kBatch];
    if (p.dest) {
      slot_rows(p.dest + slot, k, p.top_k, r);
    } else {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) r[j] = k + j < p.top_k ? (uint32_t)slot + k + j : kNoRow;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      w[j] = p.weight ? p.weight[slot + (k + j < p.top_k ? k + j : p.top_k - 1)] : 1.0f;
    u32x4 v[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const bool in = r[j] < p.rows;
      v[j] = buffer_load16(row_buffer(p.y, in ? (uint64_t)r[j] * bytes : 0, in ? bytes : 0),
                           c * 16);
      w[j] = in ? w[j] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float f[8];
      unpack8(v[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w[j], f[i], acc[i]);
    }
  }
  if (c < p.chunks)
    store_stream(reinterpret_cast<u32x4*>(p.out) + (uint64_t)t * p.chunks + c, pack8_bf16(acc));
}

// A wave takes kSlots slots of one token over all columns, 512 at a time, the
// next 512 asked for ahead. What is not asked for is a buffer of no bytes.
constexpr int kSlots = 2;
template <int kFmt>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(DispatchCast p,
                                                                    uint32_t pairs,
                                                                    uint32_t groups) {
  const uint32_t lane = threadIdx.x & 63;
  if (blockIdx.x >= groups) {
    uint32_t r0, r1;
    pad_range(p.runs, blockIdx.x - groups, r0, r1);
    const float zero[8] = {};
    for (uint32_t c = threadIdx.x; c < p.chunks; c += kThreads) {
      const ChunkScale s = chunk_scale<kFmt>(p.cast, c, zero);
      for (uint32_t r = r0; r < r1; ++r) {
        if (p.cast.q) {
          put_codes<kFmt>(p.cast, r, p.chunks, c, zero);
          put_scale(p.cast, r, s);
        }
        if (p.dy)
          store_stream(reinterpret_cast<u32x4*>(p.dy) + (uint64_t)r * p.chunks + c,
                       u32x4{0, 0, 0, 0});
      }
    }
    return;
  }
  const uint64_t item = (uint64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / pairs));
  const uint32_t k0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % pairs)) * kSlots;
  if (t >= p.runs.tokens) return;
  const uint32_t bytes = p.chunks * 16;
  const uint64_t slot = (uint64_t)t * p.runs.top_k + k0;
  uint32_t r[kSlots];
  float w[kSlots], dot[kSlots];
  RowBuffer y[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    const uint32_t s = k0 + j < p.runs.top_k ? j : 0;
    r[j] = k0 + j < p.runs.top_k ? (uint32_t)p.runs.dest[slot + s] : kNoRow;
    w[j] = p.weight ? p.weight[slot + s] : 1.0f;
    const bool reads = r[j] < p.runs.rows && p.dw;
    y[j] = row_buffer(p.y, reads ? (uint64_t)r[j] * bytes : 0, reads ? bytes : 0);
    dot[j] = 0.0f;
  }
  const RowBuffer x = row_buffer(p.x, (uint64_t)t * bytes, bytes);
  u32x4 xn = buffer_load16<0>(x, lane * 16), yn[kSlots];
#pragma unroll
  for (int j = 0; j < kSlots; ++j) yn[j] = buffer_load16(y[j], lane * 16);
  for (uint32_t c = lane; c - lane < p.chunks; c += 64) {
    float d[8], f[kSlots][8];
    unpack8(xn, d);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) unpack8(yn[j], f[j]);
    xn = buffer_load16<0>(x, (c + 64) * 16);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) yn[j] = buffer_load16(y[j], (c + 64) * 16);
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) dot[j] = __builtin_fmaf(d[i], f[j][i], dot[j]);
      if (r[j] < p.runs.rows && c < p.chunks) {         // a group's lanes leave together
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = w[j] * d[i];
        if (p.dy)
          store_stream(reinterpret_cast<u32x4*>(p.dy) + (uint64_t)r[j] * p.chunks + c,
                       pack8_bf16(v));
        if (p.cast.q) {
          const ChunkScale s = chunk_scale<kFmt>(p.cast, c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = v[i] * s.inv;
          put_codes<kFmt>(p.cast, r[j], p.chunks, c, v);
          put_scale(p.cast, r[j], s);
        }
      }
    }
  }
  if (p.dw) {
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const float sum = wave_sum(dot[j]);
      if (lane == 0 && k0 + j < p.runs.top_k) p.dw[slot + j] = r[j] < p.runs.rows ? sum : 0.0f;
    }
  }
}

}  // namespace

hipError_t launch_combine(const Combine& p, hipStream_t stream) {
  const uint32_t segs = (p.chunks + 63) / 64;
  const uint64_t groups = ((uint64_t)p.tokens * segs + kWaves - 1) / kWaves;
  if (groups >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  if (groups == 0) return hipSuccess;
  launch_kernel(combine_kernel, dim3((uint32_t)groups), dim3(kThreads), 0, stream, p, segs);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const DispatchCast& p, hipStream_t stream) {
  const uint32_t pairs = (p.runs.top_k + kSlots - 1) / kSlots;
  const uint64_t groups = ((uint64_t)p.runs.tokens * pairs + kWaves - 1) / kWaves;
  const uint64_t all = groups + (p.cast.q || p.dy ? pad_groups(p.runs) : 0);
  if (all >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  if (all == 0) return hipSuccess;
  auto kernel = p.cast.fmt == kE4M3   ? combine_backward_kernel<kE4M3>
                : p.cast.fmt == kE5M2 ? combine_backward_kernel<kE5M2>
                : p.cast.fmt == kE2M1 ? combine_backward_kernel<kE2M1>
                                      : combine_backward_kernel<kE5M6>;
  launch_kernel(kernel, dim3((uint32_t)all), dim3(kThreads), 0, stream, p, pairs,
                (uint32_t)groups);
  return hipGetLastError();
}

}  // namespace qcast
