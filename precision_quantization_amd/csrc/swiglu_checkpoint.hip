// swiglu_checkpoint.hip -- SwiGLU forward fused with the per-token cast of its
// value and with the 8-bit per-token cast of its input (the checkpoint that
// the backward pass reads in place of h).
//
// v = silu(g) * u * w as in swiglu.hip, in fp32 from h itself; the checkpoint
// is the per-token cast of the rows (gate | up) of h. Separate calls read h
// twice (4 bytes per gate and up pair more).
//
// What it must move per pair: 4 bytes of h, 1 of codes of v (8-bit formats),
// 2 of checkpoint, and 3 scales per group: bound by HBM bandwidth. 8192 x
// 2048: 20 us, 5.9 TB/s.
//
// gfx950 design. A lane owns 8 consecutive columns j of one row: the gate and
// up chunks are one 16-byte load each and serve all three casts, whose
// abs-maxima share one reduction pattern over the group's lanes; the maxima
// of the two input chunks are taken on packed 16-bit magnitudes.
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Chunk-to-row division: (c * magic) >> 40 is exact for c < 2^24 and chunks
// per row < 2^16.
constexpr int64_t kMaxChunksPerLaunch = int64_t(1) << 24;
constexpr int64_t kMaxChunksPerRow = int64_t(1) << 16;

// Abs-max over the group's lanes of 8 packed bf16.
template <int kLanes>
__device__ __forceinline__ float packed_group_max(const u32x4& r) {
  uint32_t m = pk_umax16(pk_umax16(r.x & 0x7fff7fffu, r.y & 0x7fff7fffu),
                         pk_umax16(r.z & 0x7fff7fffu, r.w & 0x7fff7fffu));
  m = pk_umax16(m, dpp<kDppXor1>(m));
  m = pk_umax16(m, dpp<kDppXor2>(m));
  if (kLanes >= 8) m = pk_umax16(m, dpp<kDppHalfMirror>(m));
  if (kLanes >= 16) m = pk_umax16(m, dpp<kDppMirror>(m));
  return fmaxf(bf16_lo(m), bf16_hi(m));
}

template <int kCkpt, int kLanes>
__device__ __forceinline__ void checkpoint8(const u32x4& raw, float floor, uint8_t* q, uint32_t c,
                                            float* sf) {
  const Scale s = group_scale<kCkpt>(packed_group_max<kLanes>(raw), floor);
  float v[8];
  unpack8(raw, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * s.inv;
  store_chunk8<kCkpt>(q, c, v);
  if ((threadIdx.x & (kLanes - 1)) == 0) *sf = s.sf;
}

template <int kLanes, int kFmt, int kCkpt>
__global__ __launch_bounds__(kThreads) void swiglu_checkpoint_kernel(
    const uint16_t* __restrict__ h, const float* __restrict__ w, uint32_t nchunks,
    uint32_t chunks_per_row, uint64_t row_magic, float floor, float ckpt_floor, float clamp,
    uint32_t row0, SfLayout lay, uint8_t* __restrict__ q, void* __restrict__ sf,
    uint8_t* __restrict__ ckpt, float* __restrict__ ckpt_sf) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= nchunks) return;       // a group's lanes leave together
  const uint32_t row = (uint32_t)(((uint64_t)c * row_magic) >> 40);
  const uint32_t jc = c - row * chunks_per_row;
  const uint32_t hc = row * 2 * chunks_per_row + jc;
  const u32x4* src = reinterpret_cast<const u32x4*>(h) + hc;
  // plain loads: h was just written by a product, and what of it is in the
  // Infinity Cache is read from there (20.2 against 22.0 us, 8192 x 2048)
  const u32x4 graw = src[0];
  const u32x4 uraw = src[chunks_per_row];
  const float wr = w ? w[row] : 1.0f;

  float* crow = ckpt_sf + hc / kLanes;
  checkpoint8<kCkpt, kLanes>(graw, ckpt_floor, ckpt, hc, crow);
  checkpoint8<kCkpt, kLanes>(uraw, ckpt_floor, ckpt, hc + chunks_per_row,
                             crow + chunks_per_row / kLanes);
  float g[8], u[8], v[8];
  unpack8(graw, g);
  unpack8(uraw, u);
  if (clamp > 0.0f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) clamp_gate_up(g[i], u[i], clamp);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float e = __builtin_amdgcn_exp2f(-g[i] * kLog2e);
    v[i] = g[i] * __builtin_amdgcn_rcpf(1.0f + e) * u[i];
    if (w) v[i] = v[i] * wr;
  }
  Scale s = group_scale<kFmt>(lane_group_max<kLanes>(absmax8(v)), floor);
  if (lay.flags & kSfRound) s = round_scale_pow2(s);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] * s.inv;
  store_chunk8<kFmt>(q, c, v);
  store_row_group_scale<kLanes>(sf, row0 + row, jc / kLanes, s, lay);
}

template <int kLanes, int kFmt>
hipError_t launch(const uint16_t* h, const float* w, int64_t rows, int64_t cols, float clamp,
                  const RowCast& cast, const RowCast& ckpt, hipStream_t stream) {
  const int64_t cpr = cols / 8;
  const uint64_t magic = ((uint64_t(1) << 40) + (uint64_t)cpr - 1) / (uint64_t)cpr;
  const int64_t slab_rows = kMaxChunksPerLaunch / cpr;
  auto kernel = ckpt.fmt == kE4M3 ? swiglu_checkpoint_kernel<kLanes, kFmt, kE4M3>
                                  : swiglu_checkpoint_kernel<kLanes, kFmt, kE5M2>;
  for (int64_t r0 = 0; r0 < rows; r0 += slab_rows) {
    const int64_t nr = rows - r0 < slab_rows ? rows - r0 : slab_rows;
    const uint32_t nchunks = (uint32_t)(nr * cpr);
    launch_kernel(kernel, dim3((nchunks + kThreads - 1) / kThreads), dim3(kThreads), 0, stream,
                  h + r0 * 2 * cols, w ? w + r0 : nullptr, nchunks, (uint32_t)cpr, magic,
                  cast.floor, ckpt.floor, clamp, (uint32_t)r0, cast.lay,
                  cast.q + code_bytes<kFmt>(r0 * cols), cast.sf, ckpt.q + r0 * 2 * cols,
                  static_cast<float*>(ckpt.sf) + r0 * 2 * cpr / kLanes);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

template <int kFmt>
hipError_t launch_g(const uint16_t* h, const float* w, int64_t rows, int64_t cols, int group,
                    float clamp, const RowCast& cast, const RowCast& ckpt, hipStream_t stream) {
  switch (group) {
    case 32: return launch<4, kFmt>(h, w, rows, cols, clamp, cast, ckpt, stream);
    case 64: return launch<8, kFmt>(h, w, rows, cols, clamp, cast, ckpt, stream);
    case 128: return launch<16, kFmt>(h, w, rows, cols, clamp, cast, ckpt, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_swiglu_checkpoint(const void* h, int64_t rows, int64_t cols, const float* w,
                                    int group, float swiglu_clamp, const RowCast& cast,
                                    const RowCast& ckpt, hipStream_t stream) {
  if (rows == 0 || cols == 0) return hipSuccess;
  if (cols / 8 >= kMaxChunksPerRow || rows >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  const uint16_t* hp = static_cast<const uint16_t*>(h);
  switch (cast.fmt) {
    case kE4M3: return launch_g<kE4M3>(hp, w, rows, cols, group, swiglu_clamp, cast, ckpt, stream);
    case kE5M2: return launch_g<kE5M2>(hp, w, rows, cols, group, swiglu_clamp, cast, ckpt, stream);
    case kE2M1: return launch_g<kE2M1>(hp, w, rows, cols, group, swiglu_clamp, cast, ckpt, stream);
    case kE5M6: return launch_g<kE5M6>(hp, w, rows, cols, group, swiglu_clamp, cast, ckpt, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qcast
