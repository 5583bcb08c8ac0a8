// matvec.hip -- products of a few rows with E2M1 weights and group scales.
//
// A wave forms one output value: a lane takes 32 weights at a time (16 bytes,
// inside one scale group), sums their fp32 products with x and adds the sum
// times the scales.
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

constexpr uint32_t kWaves = kThreads / 64;

template <int kX>
__device__ __forceinline__ float dot32(const Matvec& p, const u32x4& codes, uint32_t xr,
                                       uint32_t j) {
  float s = 0.0f;
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    float x[8];
    const uint64_t at = (uint64_t)xr * p.k + j * 32 + b * 8;
    if constexpr (kX == 0) {
      unpack8(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) + at), x);
    } else {
      decode8<kX>(*reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.x) + at), 1.0f, x);
    }
    const f32x2 w0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[b], 1.0f, 0);
    const f32x2 w1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[b], 1.0f, 1);
    const f32x2 w2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[b], 1.0f, 2);
    const f32x2 w3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes[b], 1.0f, 3);
    s = __builtin_fmaf(w0.x, x[0], s);
    s = __builtin_fmaf(w0.y, x[1], s);
    s = __builtin_fmaf(w1.x, x[2], s);
    s = __builtin_fmaf(w1.y, x[3], s);
    s = __builtin_fmaf(w2.x, x[4], s);
    s = __builtin_fmaf(w2.y, x[5], s);
    s = __builtin_fmaf(w3.x, x[6], s);
    s = __builtin_fmaf(w3.y, x[7], s);
  }
  return s;
}

template <int kX>
__global__ __launch_bounds__(kThreads) void matvec_kernel(Matvec p) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)blockIdx.x * kWaves + (threadIdx.x >> 6);
  const uint32_t r = (uint32_t)(item / p.n), i = (uint32_t)(item % p.n);
  if (r >= p.rows) return;
  int64_t e = 0;
  if (p.ids) e = p.wide ? static_cast<const int64_t*>(p.ids)[r] : static_cast<const int32_t*>(p.ids)[r];
  float acc = 0.0f;
  if (e >= 0 && e < p.experts) {
    const uint32_t xr = r / (p.rows / p.x_rows);
    const uint64_t row = (uint64_t)e * p.n + i;
    const uint32_t blocks = p.k / 32, wg = blocks >> p.w_shift;
    const u32x4* w = reinterpret_cast<const u32x4*>(p.w) + row * blocks;
    for (uint32_t j = lane; j < blocks; j += 64) {
      const uint64_t g = row * wg + (j >> p.w_shift);
      float s = p.packed
                    ? __uint_as_float((uint32_t)static_cast<const uint8_t*>(p.w_sf)[g] << 23)
                    : static_cast<const float*>(p.w_sf)[g];
      if constexpr (kX != 0)
        s = s * p.x_sf[(uint64_t)xr * (blocks >> p.x_shift) + (j >> p.x_shift)];
      acc = __builtin_fmaf(dot32<kX>(p, w[j], xr, j), s, acc);
    }
  }
  acc = wave_sum(acc);
  if (lane == 0) {
    const uint64_t at = (uint64_t)r * p.n + i;
    if (p.out_bf16) static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16(acc, 0.0f);
    else static_cast<float*>(p.out)[at] = acc;
  }
}

}  // namespace

bool matvec_fits(int64_t rows, int64_t n) { return n == 0 || rows < (int64_t(1) << 33) / n; }

hipError_t launch_matvec(const Matvec& p, hipStream_t stream, const LaunchCaps&) {
  const uint64_t groups = ((uint64_t)p.rows * p.n + kWaves - 1) / kWaves;
  if (groups >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  if (groups == 0) return hipSuccess;
  auto kernel = p.x_fmt == 0 ? matvec_kernel<0> : p.x_fmt == kE4M3 ? matvec_kernel<kE4M3>
                                                                   : matvec_kernel<kE5M2>;
  launch_kernel(kernel, dim3((uint32_t)groups), dim3(kThreads), 0, stream, p);
  return hipGetLastError();
}

}  // namespace qcast
