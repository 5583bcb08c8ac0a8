// norm_backward.hip -- gradient of the norms around a block (norm.hip), from
// bf16 activations or from their 8-bit checkpoints, fused with the per-token
// cast of the block's output gradient.
//
// With xh = h' * r2, a = y * r1 (r1 = 1 and no weight without a post-norm),
// wq = w_pre + offset, wp = w_post + offset, dx the gradient of x and dh' the
// gradient that reaches h' along the residual stream:
//   g  = dx * wq
//   dH = dh' + r2 * (g - xh * mean(g * xh))
//   dh = bf16(alpha * dH)
//   dz = dH * gate,  da = dz * wp
//   dy = r1 * (da - a * mean(da * a))
//   dw_pre = sum_rows dx * xh,  dw_post = sum_rows dz * a
//   dgate  = dH * a * wp, summed over what the gate was broadcast along
// and dy is cast per token. The rounding of h' to bf16 and of the checkpoints
// to 8 bits have derivative one.
//
// One reduction round per row: da depends on mean(g * xh), but linearly, so
// with b = dh' + r2 * g the sums S1 = sum g * xh, S2 = sum b * c and
// S3 = sum xh * c, c = gate * wp * a, are taken together and
//   sum da * a = S2 - r2 * (S1 / n) * S3.
//
// gfx950 design. Workgroups walk the rows with a stride, so a lane meets the
// same columns in every row and holds the sums of both weights' gradients and
// of a channel gate's in fp32 registers; each workgroup writes its sums to
// the workspace once and a second kernel adds them up in a fixed order (no
// atomics: the result does not depend on which workgroup ends first).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kJoinRows = 16;      // waves of the joining workgroup

// The lane's raw data of one chunk of one row.
template <bool kSaved8>
struct Chunk {
  u32x4 dx, dh, gate;
  u32x4 hs, ys;          // kSaved8: the codes in the low half
  float hsf, ysf;
};

template <bool kSaved8>
__device__ __forceinline__ Chunk<kSaved8> load_chunk(const NormBackward& p, uint32_t row,
                                                     uint32_t jc, bool valid) {
  const int64_t at = (int64_t)row * p.chunks + jc;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  Chunk<kSaved8> c;
  c.dx = valid ? load_stream(reinterpret_cast<const u32x4*>(p.dx) + at) : zero;
  c.dh = (valid && p.dh_in) ? load_stream(reinterpret_cast<const u32x4*>(p.dh_in) + at) : zero;
  c.gate = (valid && p.gate_kind == kGateFull)
               ? load_stream(reinterpret_cast<const u32x4*>(p.gate) + at)
               : zero;
  c.hs = zero;
  c.ys = zero;
  c.hsf = c.ysf = 1.0f;
  if constexpr (kSaved8) {
    if (valid) {
      const u32x2 h = load_stream(static_cast<const u32x2*>(p.saved_h) + at);
      c.hs.x = h.x;
      c.hs.y = h.y;
      const int64_t s = (int64_t)row * (p.chunks / 16) + jc / 16;
      c.hsf = p.saved_h_sf[s];
      if (p.saved_y) {
        const u32x2 y = load_stream(static_cast<const u32x2*>(p.saved_y) + at);
        c.ys.x = y.x;
        c.ys.y = y.y;
        c.ysf = p.saved_y_sf[s];
      }
    }
  } else {
    if (valid) {
      c.hs = load_stream(static_cast<const u32x4*>(p.saved_h) + at);
      if (p.saved_y) c.ys = load_stream(static_cast<const u32x4*>(p.saved_y) + at);
    }
  }
  return c;
}

template <bool kSaved8>
__device__ __forceinline__ void saved_values(const u32x4& raw, float sf, int fmt, float v[8]) {
  if constexpr (kSaved8) {
    const u32x2 w = {raw.x, raw.y};
    if (fmt == kE4M3) decode8<kE4M3>(w, sf, v);
    else decode8<kE5M2>(w, sf, v);
  } else {
    unpack8(raw, v);
  }
}

template <int kC, bool kSaved8>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBackward p, uint32_t rows) {
  __shared__ float part[2][kMaxWaves][3];
  const uint32_t chunks = p.chunks;
  const int waves = blockDim.x >> 6;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  u32x4 wq[kC], wp[kC], gc[kC];
  float s_pre[kC][8], s_post[kC][8], s_gate[kC][8];
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t jc = threadIdx.x + k * blockDim.x;
    const bool valid = jc < chunks;
    wq[k] = valid ? reinterpret_cast<const u32x4*>(p.w_pre)[jc] : zero;
    wp[k] = (valid && p.w_post) ? reinterpret_cast<const u32x4*>(p.w_post)[jc] : zero;
    gc[k] = (valid && p.gate_kind == kGateChannel) ? reinterpret_cast<const u32x4*>(p.gate)[jc]
                                                   : zero;
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[k][i] = s_post[k][i] = s_gate[k][i] = 0.0f;
  }
  const bool has_gate_vec = p.gate_kind == kGateChannel || p.gate_kind == kGateFull;
  int parity = 0;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    Chunk<kSaved8> c[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      c[k] = load_chunk<kSaved8>(p, row, jc, jc < chunks);
    }
    const float r2 = p.rstd_pre[row];
    const float r1 = p.rstd_post ? p.rstd_post[row] : 1.0f;
    const float row_gate =
        p.gate_kind == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.0f;
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      float dx[8], dh[8], xh[8], a[8], q[8], w[8], g[8];
      unpack8(c[k].dx, dx);
      unpack8(c[k].dh, dh);
      saved_values<kSaved8>(c[k].hs, c[k].hsf, p.saved_fmt, xh);
      saved_values<kSaved8>(c[k].ys, c[k].ysf, p.saved_fmt, a);
      unpack8(wq[k], q);
      unpack8(wp[k], w);
      unpack8(p.gate_kind == kGateFull ? c[k].gate : gc[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = xh[i] * r2;
        const float gx = dx[i] * (q[i] + p.offset);
        s1 = __builtin_fmaf(gx, x, s1);
        s_pre[k][i] = __builtin_fmaf(dx[i], x, s_pre[k][i]);
        if (p.saved_y) {
          float cc = a[i] * r1;
          if (p.w_post) cc = cc * (w[i] + p.offset);
          if (has_gate_vec) cc = cc * g[i];
          s2 = __builtin_fmaf(__builtin_fmaf(r2, gx, dh[i]), cc, s2);
          s3 = __builtin_fmaf(x, cc, s3);
        }
      }
    }
    s1 = wave_sum(s1);
    if (p.saved_y) {
      s2 = wave_sum(s2);
      s3 = wave_sum(s3);
    }
    if (waves > 1) {
      if ((threadIdx.x & 63) == 0) {
        float* o = part[parity][threadIdx.x >> 6];
        o[0] = s1;
        o[1] = s2;
        o[2] = s3;
      }
      __syncthreads();
      s1 = s2 = s3 = 0.0f;
      for (int i = 0; i < waves; ++i) {
        s1 += part[parity][i][0];
        s2 += part[parity][i][1];
        s3 += part[parity][i][2];
      }
    }
    const float m1 = s1 / p.n;
    const float along = s2 - r2 * m1 * s3;      // sum dH * c, without a token gate
    if (p.gate_kind == kGateToken && p.dgate && threadIdx.x == 0)
      static_cast<float*>(p.dgate)[row] = along;
    const float m2 = p.w_post ? along * row_gate / p.n : 0.0f;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      float dx[8], dh[8], xh[8], a[8], q[8], w[8], g[8], dgate[8], dy[8];
      unpack8(c[k].dx, dx);
      unpack8(c[k].dh, dh);
      saved_values<kSaved8>(c[k].hs, c[k].hsf, p.saved_fmt, xh);
      saved_values<kSaved8>(c[k].ys, c[k].ysf, p.saved_fmt, a);
      unpack8(wq[k], q);
      unpack8(wp[k], w);
      unpack8(p.gate_kind == kGateFull ? c[k].gate : gc[k], g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gx = dx[i] * (q[i] + p.offset);
        const float d = __builtin_fmaf(r2, gx - xh[i] * r2 * m1, dh[i]);
        dh[i] = p.alpha * d;
        const float aa = a[i] * r1;
        const float wi = p.w_post ? w[i] + p.offset : 1.0f;
        dgate[i] = d * aa * wi;
        const float dz = (has_gate_vec ? d * g[i] : d) * row_gate;
        s_post[k][i] = __builtin_fmaf(dz, aa, s_post[k][i]);
        if (p.gate_kind == kGateChannel) s_gate[k][i] += dgate[i];
        dy[i] = p.w_post ? r1 * (dz * wi - aa * m2) : dz;
      }
      if (jc < chunks) {
        const int64_t at = (int64_t)row * chunks + jc;
        store_stream(reinterpret_cast<u32x4*>(p.dh_out) + at, pack8_bf16(dh));
        if (p.saved_y) {
          if (p.gate_kind == kGateFull && p.dgate)
            store_stream(static_cast<u32x4*>(p.dgate) + at, pack8_bf16(dgate));
          if (p.dy_out) store_stream(reinterpret_cast<u32x4*>(p.dy_out) + at, pack8_bf16(dy));
          if (p.cast.q) cast_chunk(p.cast, row, jc, chunks, dy);
        }
      }
    }
  }
  // this workgroup's column sums: [workgroup][vector][column]
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t jc = threadIdx.x + k * blockDim.x;
    if (jc < chunks) {
#pragma unroll
      for (int v = 0; v < 3; ++v) {
        float* const to = p.sums[v];
        if (!to) continue;
        float* o = gridDim.x == 1 ? to + 8 * jc
                                  : p.ws + ((int64_t)blockIdx.x * 3 + v) * 8 * chunks + 8 * jc;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = v == 0 ? s_pre[k][i] : v == 1 ? s_post[k][i] : s_gate[k][i];
      }
    }
  }
}

// out[v][col] = sum over the `parts` workgroups of ws[part][v][col], in a
// fixed order: wave w of a workgroup adds parts w, w + 16, ..., then the 16
// partial sums are added in order.
__global__ __launch_bounds__(64 * kJoinRows) void norm_backward_join_kernel(
    const float* __restrict__ ws, uint32_t parts, uint32_t cols, NormSums out) {
  __shared__ float part[kJoinRows][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const uint32_t col = blockIdx.x * 64 + lane;
  const int v = blockIdx.y;
  float* const to = out.p[v];
  if (!to) return;                       // uniform over the workgroup
  float s = 0.0f;
  if (col < cols)
    for (uint32_t i = wave; i < parts; i += kJoinRows) s += ws[((int64_t)i * 3 + v) * cols + col];
  part[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && col < cols) {
    float t = part[0][lane];
    for (int i = 1; i < kJoinRows; ++i) t += part[i][lane];
    to[col] = t;
  }
}

}  // namespace

hipError_t launch_norm_backward(const NormBackward& p, int64_t rows, hipStream_t stream) {
  if (p.chunks == 0) return hipSuccess;
  const uint32_t cols = p.chunks * 8;
  const NormSums out{{p.sums[0], p.sums[1], p.sums[2]}};
  const bool any_sum = out.p[0] || out.p[1] || out.p[2];
  if (rows == 0) {                       // sums over no rows: zeros
    if (!any_sum) return hipSuccess;
    launch_kernel(norm_backward_join_kernel, dim3((cols + 63) / 64, 3), dim3(64 * kJoinRows), 0,
                  stream, (const float*)nullptr, 0u, cols, out);
    return hipGetLastError();
  }
  if (rows >= (int64_t(1) << 31) || p.chunks > kNormMaxChunks) return hipErrorInvalidValue;
  const int kc = p.chunks > 2048 ? 4 : p.chunks > 1024 ? 2 : 1;
  const unsigned threads = (unsigned)(((p.chunks + kc - 1) / kc + 63) / 64 * 64);
  const unsigned grid = (unsigned)(rows < kNormParts ? rows : kNormParts);
  auto kernel = p.saved_fmt ? (kc == 1   ? norm_backward_kernel<1, true>
                               : kc == 2 ? norm_backward_kernel<2, true>
                                         : norm_backward_kernel<4, true>)
                            : (kc == 1   ? norm_backward_kernel<1, false>
                               : kc == 2 ? norm_backward_kernel<2, false>
                                         : norm_backward_kernel<4, false>);
  launch_kernel(kernel, dim3(grid), dim3(threads), 0, stream, p, (uint32_t)rows);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || grid == 1 || !any_sum) return err;
  launch_kernel(norm_backward_join_kernel, dim3((cols + 63) / 64, 3), dim3(64 * kJoinRows), 0,
                stream, (const float*)p.ws, (uint32_t)grid, cols, out);
  return hipGetLastError();
}

}  // namespace qcast
