// norm.hip -- the norms around a block, its gate and the scaled residual,
// fused with the per-token cast of the next block's input.
//
// For a row with the block's output y, the residual stream h, n = cols:
//   r1 = 1 / sqrt(mean(y^2) + eps), a = y * r1          (only with w_post)
//   t  = a * (w_post + offset) * gate
//   h' = alpha * h + t
//   r2 = 1 / sqrt(mean(h'^2) + eps)
//   x  = h' * r2 * (w_pre + offset)
// and x is cast per token (qcast_device.h), any format and scale layout.
// Everything is fp32 in registers. h' is rounded once, to the bf16 it is
// stored in; r2, x and the checkpoint of h' come from the unrounded sum, so
// no later value depends on which way that rounding went.
//
// What it must move: y and h read, h' and the codes written (7 bytes per
// element with 8-bit codes, 9 with both 8-bit checkpoints), so it is bound by
// HBM bandwidth, or by the launch for a few rows.
//
// gfx950 design. One workgroup per row: a lane holds kC chunks of 8 columns
// in registers from the one load to the last store, so the row crosses HBM
// once although it is reduced twice. Each sum is a wave butterfly and one
// LDS exchange (the two use separate words, one barrier each).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

constexpr int kMaxWaves = 16;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float* part) {
  v = wave_sum(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = part[0];
  for (int i = 1; i < waves; ++i) s += part[i];
  return s;
}

template <int kC>
__global__ __launch_bounds__(1024) void norm_kernel(NormForward p) {
  __shared__ float part[2][kMaxWaves];
  const uint32_t row = blockIdx.x;
  const uint32_t chunks = p.chunks;
  const u32x4* hr = reinterpret_cast<const u32x4*>(p.h) + (int64_t)row * chunks;
  const u32x4* yr = reinterpret_cast<const u32x4*>(p.y) + (int64_t)row * chunks;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 hraw[kC], yraw[kC], wq[kC], wp[kC], gt[kC];
  float hv[kC][8];
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t jc = threadIdx.x + k * blockDim.x;
    const bool valid = jc < chunks;
    yraw[k] = (valid && p.y) ? load_stream(yr + jc) : zero;
    hraw[k] = valid ? load_stream(hr + jc) : zero;
    wp[k] = (valid && p.w_post) ? reinterpret_cast<const u32x4*>(p.w_post)[jc] : zero;
    gt[k] = zero;
    if (valid && p.gate_kind == kGateChannel)
      gt[k] = reinterpret_cast<const u32x4*>(p.gate)[jc];
    else if (valid && p.gate_kind == kGateFull)
      gt[k] = load_stream(reinterpret_cast<const u32x4*>(p.gate) + (int64_t)row * chunks + jc);
    wq[k] = valid ? reinterpret_cast<const u32x4*>(p.w_pre)[jc] : zero;
  }
  const float row_gate =
      p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.0f;

#pragma unroll
  for (int k = 0; k < kC; ++k) unpack8(hraw[k], hv[k]);
  if (p.y) {
    float r1 = 1.0f;
    if (p.w_post) {
      float ss = 0.0f;
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        float v[8];
        unpack8(yraw[k], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
      }
      ss = block_sum(ss, part[0]);
      r1 = 1.0f / sqrtf(ss / p.n + p.eps);
      if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = r1;
    }
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      float y[8], w[8], g[8];
      unpack8(yraw[k], y);
      unpack8(wp[k], w);
      unpack8(gt[k], g);
      if (p.y_ckpt.q && jc < chunks) checkpoint_chunk(p.y_ckpt, row, jc, chunks, y);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float t = y[i];
        if (p.w_post) t = t * r1 * (w[i] + p.offset);
        if (p.gate_kind == kGateChannel || p.gate_kind == kGateFull) t = t * g[i];
        t = t * row_gate;
        hv[k][i] = p.alpha * hv[k][i] + t;
      }
      if (jc < chunks)
        store_stream(reinterpret_cast<u32x4*>(p.h_out) + (int64_t)row * chunks + jc,
                     pack8_bf16(hv[k]));
    }
  }

  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < kC; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(hv[k][i], hv[k][i], ss);
  }
  ss = block_sum(ss, part[1]);
  const float r2 = 1.0f / sqrtf(ss / p.n + p.eps);
  if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[row] = r2;
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t jc = threadIdx.x + k * blockDim.x;
    if (jc < chunks) {
      float v[8], w[8];
      unpack8(wq[k], w);
      if (p.h_ckpt.q) checkpoint_chunk(p.h_ckpt, row, jc, chunks, hv[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = hv[k][i] * r2 * (w[i] + p.offset);
      if (p.x_out)
        store_stream(reinterpret_cast<u32x4*>(p.x_out) + (int64_t)row * chunks + jc,
                     pack8_bf16(v));
      if (p.cast.q) cast_chunk(p.cast, row, jc, chunks, v);
    }
  }
}

}  // namespace

hipError_t launch_norm(const NormForward& p, int64_t rows, hipStream_t stream) {
  if (rows == 0 || p.chunks == 0) return hipSuccess;
  if (rows >= (int64_t(1) << 31) || p.chunks > kNormMaxChunks) return hipErrorInvalidValue;
  const int kc = p.chunks > 2048 ? 4 : p.chunks > 256 ? 2 : 1;
  const unsigned threads = (unsigned)(((p.chunks + kc - 1) / kc + 63) / 64 * 64);
  auto kernel = kc == 1 ? norm_kernel<1> : kc == 2 ? norm_kernel<2> : norm_kernel<4>;
  launch_kernel(kernel, dim3((unsigned)rows), dim3(threads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace qcast
