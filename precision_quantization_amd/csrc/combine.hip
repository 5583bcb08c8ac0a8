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

// A wave sums 512 columns of kTokens tokens, eight rows in flight. A row is a
// buffer of its own (of no bytes for a slot without one: its loads give zeros
// without reading anything, and its weight is taken as 0).
template <int kTokens>
__global__ __launch_bounds__(kThreads) void combine_kernel(Combine p, uint32_t segs,
                                                           uint32_t first) {
  constexpr uint32_t kSlots = kBatch / kTokens;        // of a token, at once
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)(blockIdx.x + first) * kWaves + (threadIdx.x >> 6);
  const uint32_t t0 = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item / segs)) * kTokens;
  const uint32_t seg = (uint32_t)__builtin_amdgcn_readfirstlane((int)(item % segs));
  if (t0 >= p.tokens) return;
  const uint32_t c = seg * 64 + lane, bytes = p.chunks * 16;
  float acc[kTokens][8] = {};
  if (p.base)
#pragma unroll
    for (uint32_t i = 0; i < kTokens; ++i) {
      const bool in = t0 + i < p.tokens;
      unpack8(buffer_load16<0>(row_buffer(p.base, in ? (uint64_t)(t0 + i) * bytes : 0,
                                          in ? bytes : 0), c * 16), acc[i]);
    }
  for (uint32_t k = 0; k < p.top_k; k += kSlots) {
    uint32_t r[kBatch];
    float w[kBatch];
    // a slot past the token's last or of no token: another's number, and no row
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
      const uint32_t t = t0 + j / kSlots < p.tokens ? t0 + j / kSlots : t0;
      const uint32_t at = k + j % kSlots < p.top_k ? k + j % kSlots : p.top_k - 1;
      const uint64_t slot = (uint64_t)t * p.top_k + at;
      r[j] = p.dest ? (uint32_t)p.dest[slot] : (uint32_t)slot;
      w[j] = p.weight ? p.weight[slot] : 1.0f;
    }
    u32x4 v[kBatch];
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
      const bool in = r[j] < p.rows && k + j % kSlots < p.top_k && t0 + j / kSlots < p.tokens;
      v[j] = buffer_load16(row_buffer(p.y, in ? (uint64_t)r[j] * bytes : 0, in ? bytes : 0),
                           c * 16);
      w[j] = in ? w[j] : 0.0f;
    }
#pragma unroll
    for (uint32_t j = 0; j < kBatch; ++j) {
      float f[8];
      unpack8(v[j], f);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        acc[j / kSlots][i] = __builtin_fmaf(w[j], f[i], acc[j / kSlots][i]);
    }
  }
  if (c < p.chunks)
#pragma unroll
    for (uint32_t i = 0; i < kTokens; ++i)
      if (t0 + i < p.tokens)
        store_stream(reinterpret_cast<u32x4*>(p.out) + (uint64_t)(t0 + i) * p.chunks + c,
                     pack8_bf16(acc[i]));
}

// A wave takes one slot over all columns, 512 at a time, with the next 512 asked
// for ahead (the loop's end waits for them and, as the number of stores is not
// known there, for this step's stores); the waves of a token's slots read its dout
// from the caches. What is not asked for is a buffer of no bytes. 4096 x 8 x 7168
// with codes and dw: 150 us (800 MB with the padding, 5.3 TB/s), as with two or
// four slots a wave (150 and 153), or a wave for 512 columns of all slots with a
// join of dw's parts (151); 257 x 6 x 2048: 6.0, 6.4, 8.7 and 9.2.
template <int kFmt>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(DispatchCast p,
                                                                    uint32_t groups,
                                                                    uint32_t first) {
  const uint32_t lane = threadIdx.x & 63, group = blockIdx.x + first;
  if (group >= groups) {
    uint32_t r0, r1;
    pad_range(p.runs, group - groups, r0, r1);
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
  const uint32_t slot = (uint32_t)__builtin_amdgcn_readfirstlane(
      (int)(group * kWaves + (threadIdx.x >> 6)));
  if (slot >= p.runs.tokens * p.runs.top_k) return;
  const uint32_t t = slot / p.runs.top_k, bytes = p.chunks * 16;
  const uint32_t r = (uint32_t)p.runs.dest[slot];
  if (r >= p.runs.rows) {
    if (p.dw && lane == 0) p.dw[slot] = 0.0f;
    return;
  }
  const float w = p.weight ? p.weight[slot] : 1.0f;
  const RowBuffer x = row_buffer(p.x, (uint64_t)t * bytes, bytes);
  const RowBuffer y = row_buffer(p.y, p.dw ? (uint64_t)r * bytes : 0, p.dw ? bytes : 0);
  float dot = 0.0f;
  u32x4 xn = buffer_load16<0>(x, lane * 16), yn = buffer_load16(y, lane * 16);
  for (uint32_t c = lane; c - lane < p.chunks; c += 64) {
    float d[8], f[8], v[8];
    unpack8(xn, d);
    unpack8(yn, f);
    xn = buffer_load16<0>(x, (c + 64) * 16);
    yn = buffer_load16(y, (c + 64) * 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) dot = __builtin_fmaf(d[i], f[i], dot);
    if (c >= p.chunks) continue;                        // a group's lanes leave together
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = w * d[i];
    if (p.dy)
      store_stream(reinterpret_cast<u32x4*>(p.dy) + (uint64_t)r * p.chunks + c, pack8_bf16(v));
    if (p.cast.q) {
      const ChunkScale s = chunk_scale<kFmt>(p.cast, c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * s.inv;
      put_codes<kFmt>(p.cast, r, p.chunks, c, v);
      put_scale(p.cast, r, s);
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
  // Four tokens of one or two slots where there is more than the card holds at
  // once, 8192 waves, twice over (16384 x 1 x 2048: 41 to 44 us with one token a
  // wave, 32 to 34 with four; 8399 x 2 x 1408, a quarter of the slots with rows:
  // 17.6 and 13.1; two tokens of four slots, 8192 x 4 x 2048: 33.4 and 33.8).
  const bool four = p.top_k <= 2 && (uint64_t)p.tokens * segs >= 2 * 8192;
  const uint32_t tokens = four ? 4 : 1;
  const uint64_t items = ((uint64_t)p.tokens + tokens - 1) / tokens * segs;
  const uint64_t groups = (items + kWaves - 1) / kWaves;
  if (groups >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  return launch_groups(four ? combine_kernel<4> : combine_kernel<1>, groups, kThreads, stream, p,
                       segs);
}

hipError_t launch_combine_backward(const DispatchCast& p, hipStream_t stream) {
  const uint64_t groups = ((uint64_t)p.runs.tokens * p.runs.top_k + kWaves - 1) / kWaves;
  const uint64_t all = groups + (p.cast.q || p.dy ? pad_groups(p.runs) : 0);
  if (all >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  auto kernel = p.cast.fmt == kE4M3   ? combine_backward_kernel<kE4M3>
                : p.cast.fmt == kE5M2 ? combine_backward_kernel<kE5M2>
                : p.cast.fmt == kE2M1 ? combine_backward_kernel<kE2M1>
                                      : combine_backward_kernel<kE5M6>;
  return launch_groups(kernel, all, kThreads, stream, p, (uint32_t)groups);
}

}  // namespace qcast
