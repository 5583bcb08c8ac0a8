// qcast_row.h -- device helpers of the kernels that hold a whole row, or a
// 128 x 128 tile, of fp32 values in registers before they cast it: wave and
// workgroup sums, 8-bit decoding, and the per-token cast of an 8-column chunk
// with the group size and the format chosen at run time.
//
// Decoding and encoding are the conversions of qcast_device.h; a decoded
// value is the fp32 product code * sf, as cast_back forms it (in the norm
// backward code * (sf * r), r the row's factor 1 / sqrt(...): one rounding
// placed otherwise).
#pragma once

#include "qcast_device.h"

namespace qcast {

// A row in memory as a buffer of `bytes` bytes (base and bytes the same in
// every lane): a lane past its end loads zeros, without a branch around the
// load. The compiler then knows how many operations follow one, and a wait for
// a row that was asked for earlier is not a wait for everything.
using RowBuffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ RowBuffer row_buffer(const void* base, uint64_t at, uint32_t bytes) {
  constexpr int kRawDwords = 0x00027000;       // no swizzle, no stride, 32-bit data
  return __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(static_cast<const uint8_t*>(base)) + at, 0, bytes, kRawDwords);
}
constexpr int kNonTemporal = 2;
template <int kPolicy = kNonTemporal>
__device__ __forceinline__ u32x4 buffer_load16(RowBuffer b, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, kPolicy);
}

// Orders the wave's own LDS accesses: what one lane wrote, another reads next.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Sums over the wave64: every lane ends with the same bits (each step adds a
// pair of lanes' values, and fp32 addition commutes).
template <int kCtrl>
__device__ __forceinline__ float add_dpp(float v) {
  return v + __uint_as_float(dpp<kCtrl>(__float_as_uint(v)));
}
// Sum over aligned runs of 16 lanes.
__device__ __forceinline__ float row16_sum(float v) {
  v = add_dpp<kDppXor1>(v);
  v = add_dpp<kDppXor2>(v);
  v = add_dpp<kDppHalfMirror>(v);
  return add_dpp<kDppMirror>(v);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  const uint32_t b = __float_as_uint(v);
  const auto r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  v = __uint_as_float((uint32_t)r[0]) + __uint_as_float((uint32_t)r[1]);
  const uint32_t c = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  return __uint_as_float((uint32_t)s[0]) + __uint_as_float((uint32_t)s[1]);
}

// Sums of three values over the workgroup (at most 16 waves), the same bits
// in every thread: `part` holds one row of 4 words per wave. One barrier;
// every lane then reads one wave's row (one LDS trip, however many waves) and
// the rows are added across the 16 lanes.
__device__ __forceinline__ void block_sum3(float& a, float& b, float& c, float (*part)[4],
                                           int waves) {
  a = wave_sum(a);
  b = wave_sum(b);
  c = wave_sum(c);
  if (waves == 1) return;
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  if ((threadIdx.x & 63) == 0)
    *reinterpret_cast<f32x4*>(part[threadIdx.x >> 6]) = f32x4{a, b, c, 0.0f};
  __syncthreads();
  const int i = threadIdx.x & 15;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (i < waves) v = *reinterpret_cast<const f32x4*>(part[i]);
  a = row16_sum(v.x);
  b = row16_sum(v.y);
  c = row16_sum(v.z);
}

// Abs-maxima of 8 and of 4 values. Starting from zero, every step is one
// v_max3_f32 with its operands' signs dropped; a first pair by itself costs
// three instructions where the compiler cannot see that its values came from
// arithmetic.
__device__ __forceinline__ float absmax8_of(const float v[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; i += 2) m = fmaxf(fmaxf(m, fabsf(v[i])), fabsf(v[i + 1]));
  return m;
}

__device__ __forceinline__ float absmax4(float a, float b, float c, float d) {
  return fmaxf(fmaxf(fmaxf(fmaxf(0.0f, fabsf(a)), fabsf(b)), fabsf(c)), fabsf(d));
}

// Abs-max over the aligned run of 2^shift lanes (4, 8 or 16; shift is the
// same in every lane).
__device__ __forceinline__ float run_max(float m, int shift) {
  uint32_t b = __float_as_uint(m);
  b = umax(b, dpp<kDppXor1>(b));
  b = umax(b, dpp<kDppXor2>(b));
  if (shift >= 3) b = umax(b, dpp<kDppHalfMirror>(b));
  if (shift >= 4) b = umax(b, dpp<kDppMirror>(b));
  return __uint_as_float(b);
}

// Four 8-bit codes of a word -> four fp32 (exact).
typedef float f32x2 __attribute__((ext_vector_type(2)));
template <int kFmt>
__device__ __forceinline__ void decode4(uint32_t w, float v[4]) {
  static_assert(kFmt == kE4M3 || kFmt == kE5M2, "8-bit formats only");
  f32x2 lo, hi;
  if constexpr (kFmt == kE4M3) {
    lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
  }
  v[0] = lo.x;
  v[1] = lo.y;
  v[2] = hi.x;
  v[3] = hi.y;
}
template <int kFmt>
__device__ __forceinline__ void decode8(const u32x2& w, float sf, float v[8]) {
  decode4<kFmt>(w.x, v);
  decode4<kFmt>(w.y, v + 4);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * sf;
}

// Two fp32 -> two bf16 (nearest even) in one dword (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ u32x4 pack8_bf16(const float v[8]) {
  return u32x4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
               pack_bf16(v[6], v[7])};
}

// Store the scale of group kr of row r, held by the 2^shift lanes of the
// group (store_row_group_scale with the run length at run time).
__device__ __forceinline__ void store_run_scale(void* sf, uint32_t r, uint32_t kr, const Scale& s,
                                                const SfLayout& lay, int shift) {
  const int lane = threadIdx.x & 63;
  const bool col = (lay.flags & kSfColMajor) != 0;
  if (lay.flags & kSfPacked) {
    const int n = 1 << shift;
    const uint32_t e = __float_as_uint(s.sf) >> 23;
    const uint32_t w = e | ((uint32_t)__shfl((int)e, lane + n) << 8) |
                       ((uint32_t)__shfl((int)e, lane + 2 * n) << 16) |
                       ((uint32_t)__shfl((int)e, lane + 3 * n) << 24);
    if ((lane & (4 * n - 1)) == 0) {
      const uint32_t idx = col ? (kr / 4) * lay.rows_pad + r : r * (lay.gpr / 4) + kr / 4;
      static_cast<uint32_t*>(sf)[idx] = w;
    }
  } else if ((lane & ((1 << shift) - 1)) == 0) {
    float* to = static_cast<float*>(sf) + (col ? r : (uint64_t)r * lay.gpr);
    to[col ? kr * lay.rows_pad : kr] = s.sf;
  }
}

// Codes of chunk first + jc; `first`, the same in every lane, goes into a
// scalar base.
template <int kFmt, typename I>
__device__ __forceinline__ void encode_chunk(const RowCast& rc, uint64_t first, I jc,
                                             const float v[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
  store_chunk8<kFmt>(rc.q + first * code_bytes<kFmt>(8), jc, y);
}
// Codes of a chunk in the cast's format, with the inverse scale known.
template <typename I>
__device__ __forceinline__ void encode_chunk_any(const RowCast& rc, uint64_t first, I jc,
                                                 const float v[8], float inv) {
  switch (rc.fmt) {
    case kE4M3: encode_chunk<kE4M3>(rc, first, jc, v, inv); break;
    case kE5M2: encode_chunk<kE5M2>(rc, first, jc, v, inv); break;
    case kE2M1: encode_chunk<kE2M1>(rc, first, jc, v, inv); break;
    default: encode_chunk<kE5M6>(rc, first, jc, v, inv); break;
  }
}

// group_scale with the format at run time, and possibly another one in every
// lane: its constants are values (the same sequence, so the same bits).
struct ScaleRule {
  float floor, max, recip, lo, hi;
};
__device__ __forceinline__ ScaleRule scale_rule(int fmt, float floor) {
  ScaleRule r;
  r.floor = floor;
  r.max = fmt == kE4M3 ? kE4M3Max : fmt == kE5M2 ? kE5M2Max : fmt == kE2M1 ? kE2M1Max : kE5M6Max;
  r.recip = fmt == kE4M3   ? 1.0f / kE4M3Max
            : fmt == kE5M2 ? 1.0f / kE5M2Max
            : fmt == kE2M1 ? 1.0f / kE2M1Max
                           : 1.0f / kE5M6Max;
  r.lo = r.max * 0x1.0p-126f;
  r.hi = fmt == kE2M1 ? kE2M1Max * 0x1.0p124f : __builtin_huge_valf();
  return r;
}
__device__ __forceinline__ Scale scale_by(const ScaleRule& r, float amax) {
  const float a = amax < r.floor ? r.floor : amax;
  Scale s;
  if (a >= r.lo && a < r.hi) {
    const float q0 = a * r.recip;
    s.sf = __builtin_fmaf(__builtin_fmaf(-q0, r.max, a), r.recip, q0);
    const float y0 = __builtin_amdgcn_rcpf(s.sf);
    s.inv = __builtin_fmaf(__builtin_fmaf(-s.sf, y0, 1.0f), y0, y0);
  } else {
    s.sf = a / r.max;
    s.inv = 1.0f / s.sf;
  }
  return s;
}

// Cast chunk jc (columns 8 jc .. 8 jc + 7) of row `row` (of `chunks` chunks).
// The lanes of a scale group call this together, lane = jc mod 64.
__device__ __forceinline__ void cast_chunk(const RowCast& rc, uint32_t row, uint32_t jc,
                                           uint32_t chunks, const float v[8]) {
  Scale s = scale_by(scale_rule(rc.fmt, rc.floor), run_max(absmax8_of(v), rc.shift));
  if (rc.lay.flags & kSfRound) s = round_scale_pow2(s);
  encode_chunk_any(rc, 0, (int64_t)row * chunks + jc, v, s.inv);
  store_run_scale(rc.sf, row, jc >> rc.shift, s, rc.lay, rc.shift);
}

// 1 / sqrt(v) for normal v > 0: the hardware's root (1 ulp) and one Newton
// step on its residual. 0 gives infinity and infinity 0, as the quotient does.
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float e = __builtin_fmaf(-v * r, r, 1.0f);
  const float c = __builtin_fmaf(0.5f * r, e, r);
  return (v > 0.0f && v < __builtin_huge_valf()) ? c : r;
}

// Sum over the workgroup (at most 16 waves), the same bits in every thread.
__device__ __forceinline__ float block_sum(float v, float* part, int waves) {
  v = wave_sum(v);
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  const int i = threadIdx.x & 15;
  return row16_sum(i < waves ? part[i] : 0.0f);
}

}  // namespace qcast
