// swiglu_backward_checkpoint.hip -- SwiGLU backward from the 8-bit checkpoint
// of its input, with every operand of the products that follow in one pass.
//
// With g, u = code * sf (fp32, clamped as in swiglu_backward.hip):
//   s = 1 / (1 + exp(-g)), silu = g * s, silu' = s + silu * (1 - s)
//   dg = (dv * w) * u * silu',  du = (dv * w) * silu,  v = silu * u * w
//   dw[r] = sum_j dv * silu * u
// The rows [dg | du] are cast per token (groups of 128 channels); [dg | du]
// and v are cast along the tokens (groups of 128) and written transposed.
//
// What it must move per pair: 2 bytes of checkpoint and 2 of dv in, 2 of
// per-token codes and 3 of transposed codes out. Per pair it also issues
// about 45 vector instructions (an exponential, a reciprocal, five encodings
// with their scalings and maxima), which take about as long as the bytes.
//
// gfx950 design. A workgroup of 512 owns 128 tokens x 128 channels of both
// halves, so both directions' groups are whole inside it and each value is
// formed once. A lane holds 8 channels of 4 consecutive tokens: 16 lanes are
// one token's group (a DPP reduction), and 4 tokens of a channel are one
// dword of the transposed codes.
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"
#include "qcast_tile.h"

namespace qcast {
namespace {

constexpr int kBlock = 512;
constexpr int kWaves = kBlock / 64;
constexpr float kLog2e = 1.4426950408889634f;

// Column maxima of the lane's 4 tokens over the wave's 4 lanes that hold the
// same 8 channels (lanes i, i ^ 16, i ^ 32), written by the first of them.
__device__ __forceinline__ void column_max(const float (&v)[4][8], float* out) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float m = fmaxf(fmaxf(fabsf(v[0][j]), fabsf(v[1][j])),
                          fmaxf(fabsf(v[2][j]), fabsf(v[3][j])));
    const uint32_t b = max_xor32(max_xor16(__float_as_uint(m)));
    if ((threadIdx.x & 63) < 16) out[j] = __uint_as_float(b);
  }
}

template <int kFmt>
__device__ __forceinline__ void put_codes(const float (&v)[4][8], const float* inv, uint32_t c0,
                                          uint32_t quad, uint32_t* tile) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = inv[j];
    tile[swizzled(c0 + j, quad)] =
        fp8x4<kFmt>(v[0][j] * s, v[1][j] * s, v[2][j] * s, v[3][j] * s);
  }
}

// Per-token cast of one half's 8 channels of one token.
template <int kFmt>
__device__ __forceinline__ void row_cast(const SwigluTile& p, const float (&v)[8], uint32_t t,
                                         uint32_t group, uint64_t at, bool valid) {
  Scale s = group_scale<kFmt>(lane_group_max<16>(absmax8(v)), p.floor);
  if (p.lay.flags & kSfRound) s = round_scale_pow2(s);
  if (!valid) return;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = v[j] * s.inv;
  u32x2 o;
  o.x = fp8x4<kFmt>(y[0], y[1], y[2], y[3]);
  o.y = fp8x4<kFmt>(y[4], y[5], y[6], y[7]);
  store_stream(reinterpret_cast<u32x2*>(p.q + at), o);
  if ((threadIdx.x & 15) == 0) store_lone_scale(p.sf, t, group, s, p.lay);
}

template <int kIn, int kFmt>
__global__ __launch_bounds__(kBlock, 4) void swiglu_backward_tile_kernel(SwigluTile p,
                                                                          TileWalk tw) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[3][kTile * 32];
  __shared__ float amax_s[kWaves][3 * kTile];
  __shared__ float inv_s[3 * kTile];
  const uint32_t tau = (blockIdx.x % kTileXcds) * tw.per_xcd + blockIdx.x / kTileXcds;
  if (tau >= tw.ntiles) return;
  const uint32_t ct = tau / tw.ntg, gt = tau - ct * tw.ntg;
  const uint32_t c0 = ct * kTile, t0 = gt * kTile;
  const uint32_t ch = threadIdx.x & 15;          // 8-channel chunk
  const uint32_t quad = threadIdx.x >> 4;        // 4 tokens
  const uint32_t cols = p.cols;
  const uint32_t gpr = cols / 64;                // checkpoint groups per row

  u32x2 graw[4], uraw[4];
  u32x4 draw[4];
  float gsf[4], usf[4], wr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = t0 + quad * 4 + i;
    graw[i] = uraw[i] = u32x2{0u, 0u};
    draw[i] = u32x4{0u, 0u, 0u, 0u};
    gsf[i] = usf[i] = 0.0f;
    wr[i] = 1.0f;
    if (t < p.rows) {
      const uint64_t at = (uint64_t)t * 2 * cols + c0 + ch * 8;
      graw[i] = load_stream(reinterpret_cast<const u32x2*>(p.ckpt + at));
      uraw[i] = load_stream(reinterpret_cast<const u32x2*>(p.ckpt + at + cols));
      draw[i] = load_stream(reinterpret_cast<const u32x4*>(p.dv + (uint64_t)t * cols + c0 + ch * 8));
      gsf[i] = p.ckpt_sf[(uint64_t)t * gpr + ct];
      usf[i] = p.ckpt_sf[(uint64_t)t * gpr + gpr / 2 + ct];
      if (p.w) wr[i] = p.w[t];
    }
  }
  float dg[4][8], du[4][8], v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = t0 + quad * 4 + i;
    float g[8], u[8], d[8];
    decode8<kIn>(graw[i], gsf[i], g);
    decode8<kIn>(uraw[i], usf[i], u);
    unpack8(draw[i], d);
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      bool g_pass = true, u_pass = true;
      if (p.clamp > 0.0f) {
        g_pass = !(g[j] > p.clamp);
        u_pass = !(u[j] > p.clamp) && !(u[j] < -p.clamp);
        g[j] = g_pass ? g[j] : p.clamp;
        u[j] = u[j] > p.clamp ? p.clamp : (u[j] < -p.clamp ? -p.clamp : u[j]);
      }
      const float e = __builtin_amdgcn_exp2f(-g[j] * kLog2e);
      const float s = __builtin_amdgcn_rcpf(1.0f + e);
      const float silu = g[j] * s;
      const float dsilu = s + silu * (1.0f - s);
      const float x = silu * u[j];
      dot = __builtin_fmaf(d[j], x, dot);
      const float dvw = d[j] * wr[i];
      v[i][j] = x * wr[i];
      dg[i][j] = g_pass ? dvw * u[j] * dsilu : 0.0f;
      du[i][j] = u_pass ? dvw * silu : 0.0f;
    }
    if (p.dw) {
      dot = row16_sum(dot);
      if (ch == 0 && t < p.rows) {
        if (tw.nct == 1) p.dw[t] = dot;
        else p.ws[(uint64_t)ct * p.rows + t] = dot;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = t0 + quad * 4 + i;
    const uint64_t at = (uint64_t)t * 2 * cols + c0 + ch * 8;
    row_cast<kFmt>(p, dg[i], t, ct, at, t < p.rows);
    row_cast<kFmt>(p, du[i], t, tw.nct + ct, at + cols, t < p.rows);
  }
  if (!p.dh.qT && !p.v.qT) return;               // uniform over the grid
  float* am = amax_s[threadIdx.x >> 6] + ch * 8;
  column_max(dg, am);
  column_max(du, am + kTile);
  column_max(v, am + 2 * kTile);
  __syncthreads();
  if (threadIdx.x < 3 * kTile) {
    const uint32_t k = threadIdx.x / kTile, c = threadIdx.x % kTile;
    float m = amax_s[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) m = fmaxf(m, amax_s[i][threadIdx.x]);
    const TileCast& out = k == 2 ? p.v : p.dh;
    if (out.qT)
      inv_s[threadIdx.x] = channel_scale<kFmt>(out, c0 + c + (k == 1 ? cols : 0), gt, m, p.floor);
  }
  __syncthreads();
  const uint32_t rows_T = tw.ntg * kTile;
  if (p.dh.qT) {
    put_codes<kFmt>(dg, inv_s + ch * 8, ch * 8, quad, tile[0]);
    put_codes<kFmt>(du, inv_s + kTile + ch * 8, ch * 8, quad, tile[1]);
  }
  if (p.v.qT) put_codes<kFmt>(v, inv_s + 2 * kTile + ch * 8, ch * 8, quad, tile[2]);
  __syncthreads();
  if (p.dh.qT) {
    store_tile_rows<kBlock>(tile[0], p.dh.qT, c0, kTile, gt, rows_T);
    store_tile_rows<kBlock>(tile[1], p.dh.qT, c0 + cols, kTile, gt, rows_T);
  }
  if (p.v.qT) store_tile_rows<kBlock>(tile[2], p.v.qT, c0, kTile, gt, rows_T);
}

// dw[r] = sum over the channel tiles of their partial sums, in tile order.
__global__ __launch_bounds__(kThreads) void row_weight_join_kernel(const float* __restrict__ ws,
                                                                   uint32_t rows, uint32_t nct,
                                                                   float* __restrict__ dw) {
  const uint32_t r = blockIdx.x * kThreads + threadIdx.x;
  if (r >= rows) return;
  float s = ws[r];
  for (uint32_t i = 1; i < nct; ++i) s += ws[(uint64_t)i * rows + r];
  dw[r] = s;
}

}  // namespace

hipError_t launch_swiglu_backward_checkpoint(const SwigluTile& p, int ckpt_fmt, int fmt,
                                             hipStream_t stream) {
  const TileWalk tw = make_tile_walk(p.rows, p.cols);
  if (tw.ntiles == 0) return hipSuccess;
  auto kernel = ckpt_fmt == kE4M3 ? (fmt == kE4M3 ? swiglu_backward_tile_kernel<kE4M3, kE4M3>
                                                  : swiglu_backward_tile_kernel<kE4M3, kE5M2>)
                                  : (fmt == kE4M3 ? swiglu_backward_tile_kernel<kE5M2, kE4M3>
                                                  : swiglu_backward_tile_kernel<kE5M2, kE5M2>);
  launch_kernel(kernel, dim3(tw.per_xcd * kTileXcds), dim3(kBlock), 0, stream, p, tw);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.dw || tw.nct == 1) return err;
  launch_kernel(row_weight_join_kernel, dim3((p.rows + kThreads - 1) / kThreads), dim3(kThreads),
                0, stream, (const float*)p.ws, p.rows, tw.nct, p.dw);
  return hipGetLastError();
}

}  // namespace qcast
