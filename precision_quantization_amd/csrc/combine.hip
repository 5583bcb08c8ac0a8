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

// A wave sums 512 columns of one token.
__global__ __launch_bounds__(kThreads) void combine_kernel(Combine p, uint32_t segs) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const uint32_t t = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / segs));
  const uint32_t seg = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % segs));
  const uint32_t c = seg * 64 + lane;
  if (t >= p.tokens || c >= p.chunks) return;
  float acc[8] = {};
  if (p.base) unpack8(reinterpret_cast<const u32x4*>(p.base)[(uint64_t)t * p.chunks + c], acc);
  const uint64_t slot = (uint64_t)t * p.top_k;
  for (uint32_t k = 0; k < p.top_k; ++k) {
    const uint32_t r = p.dest ? (uint32_t)p.dest[slot + k] : (uint32_t)(slot + k);
    if (r >= p.rows) continue;
    const float w = p.weight ? p.weight[slot + k] : 1.0f;
    float v[8];
    unpack8(reinterpret_cast<const u32x4*>(p.y)[(uint64_t)r * p.chunks + c], v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = __builtin_fmaf(w, v[i], acc[i]);
  }
  reinterpret_cast<u32x4*>(p.out)[(uint64_t)t * p.chunks + c] = pack8_bf16(acc);
}

// A wave takes one slot.
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(DispatchCast p,
                                                                    uint32_t groups) {
  const uint32_t lane = threadIdx.x & 63;
  if (blockIdx.x >= groups) {
    uint32_t r0, r1;
    pad_range(p.runs, blockIdx.x - groups, r0, r1);
    const float zero[8] = {};
    for (uint32_t r = r0; r < r1; ++r)
      for (uint32_t c = threadIdx.x; c < p.chunks; c += kThreads) {
        if (p.cast.q) cast_chunk(p.cast, r, c, p.chunks, zero);
        if (p.dy) reinterpret_cast<u32x4*>(p.dy)[(uint64_t)r * p.chunks + c] = u32x4{0, 0, 0, 0};
      }
    return;
  }
  const uint32_t slot = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(blockIdx.x * kWaves + (threadIdx.x >> 6)));
  if (slot >= p.runs.tokens * p.runs.top_k) return;
  const uint32_t t = slot / p.runs.top_k;
  const uint32_t r = (uint32_t)p.runs.dest[slot];
  float dot = 0.0f;
  if (r < p.runs.rows) {
    const float w = p.weight ? p.weight[slot] : 1.0f;
    for (uint32_t c = lane; c < p.chunks; c += 64) {
      float d[8], v[8];
      unpack8(reinterpret_cast<const u32x4*>(p.x)[(uint64_t)t * p.chunks + c], d);
      if (p.dw) {
        float y[8];
        unpack8(reinterpret_cast<const u32x4*>(p.y)[(uint64_t)r * p.chunks + c], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(d[i], y[i], dot);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p.weight ? w * d[i] : d[i];
      if (p.cast.q) cast_chunk(p.cast, r, c, p.chunks, v);
      if (p.dy) reinterpret_cast<u32x4*>(p.dy)[(uint64_t)r * p.chunks + c] = pack8_bf16(v);
    }
  }
  if (p.dw) {
    dot = wave_sum(dot);
    if (lane == 0) p.dw[slot] = dot;
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
  const uint64_t groups = ((uint64_t)p.runs.tokens * p.runs.top_k + kWaves - 1) / kWaves;
  const uint64_t all = groups + (p.cast.q || p.dy ? pad_groups(p.runs) : 0);
  if (all >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  if (all == 0) return hipSuccess;
  launch_kernel(combine_backward_kernel, dim3((uint32_t)all), dim3(kThreads), 0, stream, p,
                (uint32_t)groups);
  return hipGetLastError();
}

}  // namespace qcast
