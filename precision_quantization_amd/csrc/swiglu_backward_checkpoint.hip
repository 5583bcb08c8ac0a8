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
// about 42 vector instructions (an exponential, a reciprocal, five encodings
// with their scalings and maxima): 22 us of the vector units' time for 8192 x
// 2048, beside 25 us of a copy's for the bytes. Measured 31 to 32 us (29
// without dw's second launch) with the inputs in the Infinity Cache; 39.7 with
// none there, and 39.6 with dv just used and the checkpoint long unused, as in
// a training step.
//
// gfx950 design. A workgroup of 512 owns 128 tokens x 128 channels of both
// halves, so both directions' groups are whole inside it and each value is
// formed once. A lane holds 8 channels of 4 consecutive tokens: 16 lanes are
// one token's group, and 4 tokens of a channel are one dword of the
// transposed codes. The 8 rows (4 tokens, two halves) of 16 lanes are reduced
// as one butterfly that leaves one row per lane, which forms that row's scale
// and hands it back by row broadcast: one scale computation per lane instead
// of 8. dw is summed over a tile's channels here and over the tiles by a
// second kernel in tile order. (Measured and left: one workgroup per compute
// unit that walks tiles with the next one's loads in flight, 34 us; the last
// tile of a token group joining the sums behind device-scope fences, 75 us.)
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"
#include "qcast_tile.h"

namespace qcast {
namespace {

// channel tiles per strip: 32.1 us against 35.6 with 1, 33.0 with 2, 32.5 with 8
constexpr uint32_t kStrip = 4;

constexpr int kBlock = 512;
constexpr int kWaves = kBlock / 64;
constexpr float kLog2e = 1.4426950408889634f;

// Column maxima of the lane's 4 tokens and 8 channels over the wave's 4 lanes
// that hold the same channels (lane bits 4 and 5), as a butterfly whose
// exchanges each carry two channels: afterwards a lane holds channels
// 4 * bit 4 + 2 * bit 5 + {0, 1} of its chunk (6 swaps and 6 maxima instead
// of 16 and 16).
__device__ __forceinline__ void column_max(const float (&v)[4][8], float* out) {
  uint32_t m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    m[j] = __float_as_uint(absmax4(v[0][j], v[1][j], v[2][j], v[3][j]));
  uint32_t n[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const auto r = __builtin_amdgcn_permlane16_swap(m[j], m[j + 4], false, false);
    n[j] = umax((uint32_t)r[0], (uint32_t)r[1]);
  }
  float o[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto r = __builtin_amdgcn_permlane32_swap(n[j], n[j + 2], false, false);
    o[j] = __uint_as_float(umax((uint32_t)r[0], (uint32_t)r[1]));
  }
  const uint32_t l = threadIdx.x;
  float* to = out + ((l >> 4) & 1) * 4 + ((l >> 5) & 1) * 2;
  to[0] = o[0];
  to[1] = o[1];
}

// The abs-maxima of 8 (half, token) rows over their 16 lanes, m[4 * half +
// token] the lane's own, as a butterfly that halves the rows a lane follows:
// lane l ends with the maximum of half l >> 3, token (l >> 1) & 3.
__device__ __forceinline__ float row_max8(const uint32_t (&m)[8]) {
  const uint32_t l = threadIdx.x;
  uint32_t n[4], o[2];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t a = umax(m[k], dpp<kDppRor8>(m[k]));
    const uint32_t b = umax(m[k + 4], dpp<kDppRor8>(m[k + 4]));
    n[k] = (l & 8) ? b : a;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {      // lanes i and 7 - i: bit 2 differs
    const uint32_t a = umax(n[k], dpp<kDppHalfMirror>(n[k]));
    const uint32_t b = umax(n[k + 2], dpp<kDppHalfMirror>(n[k + 2]));
    o[k] = (l & 4) ? b : a;
  }
  const uint32_t a = umax(o[0], dpp<kDppXor2>(o[0]));
  const uint32_t b = umax(o[1], dpp<kDppXor2>(o[1]));
  const uint32_t r = (l & 2) ? b : a;
  return __uint_as_float(umax(r, dpp<kDppXor1>(r)));
}
// The value that lane 8 * half + 2 * token of the row of 16 lanes holds.
template <int kHalf, int kToken>
__device__ __forceinline__ float from_row(float v) {
  constexpr int kNewBcast0 = 0x150;
  return __uint_as_float(dpp<kNewBcast0 + 8 * kHalf + 2 * kToken>(__float_as_uint(v)));
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

template <int kFmt>
__device__ __forceinline__ void row_codes(const float (&v)[8], float inv, uint8_t* q) {
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = v[j] * inv;
  u32x2 o;
  o.x = fp8x4<kFmt>(y[0], y[1], y[2], y[3]);
  o.y = fp8x4<kFmt>(y[4], y[5], y[6], y[7]);
  store_stream(reinterpret_cast<u32x2*>(q), o);
}

// The per-token codes of the lane's 4 tokens, both halves. q: the address of
// the lane's gate chunk of its first token; left: tokens that exist.
template <int kFmt, int kToken>
__device__ __forceinline__ void token_codes(const float (&dg)[4][8], const float (&du)[4][8],
                                            float inv, uint8_t* q, uint32_t cols, int left) {
  const float ig = from_row<0, kToken>(inv), iu = from_row<1, kToken>(inv);
  if (kToken < left) {
    row_codes<kFmt>(dg[kToken], ig, q + (uint64_t)kToken * 2 * cols);
    row_codes<kFmt>(du[kToken], iu, q + (uint64_t)kToken * 2 * cols + cols);
  }
}

// kLayout: scale options other than plain fp32. kT: transposed codes are
// wanted too.
template <int kIn, int kFmt, bool kClamp, bool kLayout, bool kT>
__global__ __launch_bounds__(kBlock, 4) void swiglu_backward_tile_kernel(SwigluTile p,
                                                                          TileWalk tw) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[3][kTileDw];
  __shared__ float amax_s[kWaves][3 * kTile];
  __shared__ float inv_s[3 * kTile];
  const uint32_t tau = (blockIdx.x % kTileXcds) * tw.per_xcd + blockIdx.x / kTileXcds;
  if (tau >= tw.ntiles) return;
  const TilePos tp = tile_pos(tau, tw);
  const uint32_t ct = tp.ct, gt = tp.gt;
  const uint32_t c0 = ct * kTile, t0 = gt * kTile;
  const uint32_t ch = threadIdx.x & 15;          // 8-channel chunk
  const uint32_t quad = threadIdx.x >> 4;        // 4 tokens
  const uint32_t cols = p.cols;
  const uint32_t gpr = cols / 64;                // groups of a row [dg | du]
  const uint32_t cpr = (2 * cols) >> (p.ckpt_shift + 3);   // checkpoint groups of a row

  u32x2 graw[4], uraw[4];
  u32x4 draw[4];
  float gsf[4], usf[4], wr[4];
  const uint32_t tq = t0 + quad * 4;
  const int left = (int)(p.rows - tq);           // of the lane's tokens, those that exist
  const uint8_t* cp = p.ckpt + (uint64_t)tq * 2 * cols + c0 + ch * 8;
  const uint16_t* dp = p.dv + (uint64_t)tq * cols + c0 + ch * 8;
  // the lane's 8 channels lie in one group of 32, 64 or 128
  const float* sp = p.ckpt_sf + (uint64_t)tq * cpr + (ct << (4 - p.ckpt_shift)) +
                    (ch >> p.ckpt_shift);
  // plain loads: 32 us where the inputs are in the Infinity Cache (a gradient
  // that the product before has just written) against 41 with streaming
  // loads, and no slower from HBM (40.6 against 41.3; 8192 x 2048)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    graw[i] = uraw[i] = u32x2{0u, 0u};
    draw[i] = u32x4{0u, 0u, 0u, 0u};
    gsf[i] = usf[i] = 0.0f;
    wr[i] = 1.0f;
    if (i < left) {
      graw[i] = *reinterpret_cast<const u32x2*>(cp + i * 2 * cols);
      uraw[i] = *reinterpret_cast<const u32x2*>(cp + i * 2 * cols + cols);
      draw[i] = *reinterpret_cast<const u32x4*>(dp + i * cols);
      gsf[i] = sp[i * cpr];
      usf[i] = sp[i * cpr + cpr / 2];
      if (p.w) wr[i] = p.w[tq + i];
    }
  }
  float dg[4][8], du[4][8], v[4][8];
  float dot[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float g[4], u[4], d[4];
      decode4<kIn>(k ? graw[i].y : graw[i].x, g);
      decode4<kIn>(k ? uraw[i].y : uraw[i].x, u);
      const uint32_t d01 = k ? draw[i].z : draw[i].x, d23 = k ? draw[i].w : draw[i].y;
      d[0] = bf16_lo(d01);
      d[1] = bf16_hi(d01);
      d[2] = bf16_lo(d23);
      d[3] = bf16_hi(d23);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[j] = g[j] * gsf[i];
        u[j] = u[j] * usf[i];
        bool g_pass = true, u_pass = true;
        if (kClamp) {
          g_pass = !(g[j] > p.clamp);
          u_pass = !(u[j] > p.clamp) && !(u[j] < -p.clamp);
          g[j] = g_pass ? g[j] : p.clamp;
          u[j] = u[j] > p.clamp ? p.clamp : (u[j] < -p.clamp ? -p.clamp : u[j]);
        }
        const float e = __builtin_amdgcn_exp2f(-g[j] * kLog2e);
        const float s = __builtin_amdgcn_rcpf(1.0f + e);
        const float silu = g[j] * s;
        const float dsilu = __builtin_fmaf(silu, 1.0f - s, s);
        const float x = silu * u[j];
        dot[i] = __builtin_fmaf(d[j], x, dot[i]);
        const float dvw = d[j] * wr[i];
        if (kT) {
          v[i][4 * k + j] = x * wr[i];
          // formed here: the compiler would sink it to its use, and its
          // factors would stay live until there
          asm volatile("" : "+v"(v[i][4 * k + j]));
        }
        dg[i][4 * k + j] = g_pass ? dvw * u[j] * dsilu : 0.0f;
        du[i][4 * k + j] = u_pass ? dvw * silu : 0.0f;
      }
      asm volatile("" : "+v"(dot[i]));
      // four pairs at a time: interleaved, the lane's 32 need more registers
      // than two workgroups on a CU leave it
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  {
    // per-token casts: each lane forms the scale of one of the 8 rows
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = __float_as_uint(absmax8_of(dg[i]));
      m[4 + i] = __float_as_uint(absmax8_of(du[i]));
    }
    Scale s = group_scale<kFmt>(row_max8(m), p.floor);
    if (kLayout && (p.lay.flags & kSfRound)) s = round_scale_pow2(s);
    const uint32_t t = tq + ((ch >> 1) & 3);
    const uint32_t group = (ch >> 3) * tw.nct + ct;
    if (!(ch & 1) && t < p.rows) {
      if (kLayout) store_lone_scale(p.sf, t, group, s, p.lay);
      else static_cast<float*>(p.sf)[(uint64_t)t * gpr + group] = s.sf;
    }
    uint8_t* q = p.q + (uint64_t)tq * 2 * cols + c0 + ch * 8;
    token_codes<kFmt, 0>(dg, du, s.inv, q, cols, left);
    token_codes<kFmt, 1>(dg, du, s.inv, q, cols, left);
    token_codes<kFmt, 2>(dg, du, s.inv, q, cols, left);
    token_codes<kFmt, 3>(dg, du, s.inv, q, cols, left);
  }
  {
    float* to = tw.nct == 1 ? p.dw : p.ws + (uint64_t)ct * p.rows;
#pragma unroll
    for (int i = 0; i < 4; ++i) dot[i] = row16_sum(dot[i]);
    const float mine = (ch & 2) ? ((ch & 1) ? dot[3] : dot[2]) : ((ch & 1) ? dot[1] : dot[0]);
    if (p.dw && ch < 4 && (int)ch < left) to[tq + ch] = mine;
  }
  if constexpr (!kT) return;
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
    if (k == 2 ? p.v.qT : p.dh.qT)
      inv_s[threadIdx.x] = channel_scale<kFmt, kLayout>(k == 2 ? p.v.sf : p.dh.sf,
                                                        k == 2 ? p.v.lay : p.dh.lay,
                                                        c0 + c + (k == 1 ? cols : 0), gt, m,
                                                        p.floor);
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
    store_tile_rows<kBlock, true>(tile[0], p.dh.qT, c0, kTile, gt, rows_T);
    store_tile_rows<kBlock, true>(tile[1], p.dh.qT, c0 + cols, kTile, gt, rows_T);
  }
  if (p.v.qT) store_tile_rows<kBlock, true>(tile[2], p.v.qT, c0, kTile, gt, rows_T);
}

constexpr uint32_t kJoin = 16;

// dw[r] = sum over the channel tiles of their partial sums, in tile order.
__global__ __launch_bounds__(64) void row_weight_join_kernel(const float* __restrict__ ws,
                                                                   uint32_t rows, uint32_t nct,
                                                                   float* __restrict__ dw) {
  const uint32_t r = blockIdx.x * 64 + threadIdx.x;
  if (r >= rows) return;
  float s = 0.0f;
  for (uint32_t i0 = 0; i0 < nct; i0 += kJoin) {
    float v[kJoin];                       // all loads in flight before the first sum
#pragma unroll
    for (uint32_t i = 0; i < kJoin; ++i)
      v[i] = i0 + i < nct ? ws[(uint64_t)(i0 + i) * rows + r] : 0.0f;
#pragma unroll
    for (uint32_t i = 0; i < kJoin; ++i) s += v[i];
  }
  dw[r] = s;
}

template <int kIn, int kFmt, bool kClamp>
auto pick_form(const SwigluTile& p) {
  const bool t = p.dh.qT || p.v.qT;
  return p.lay.flags ? (t ? swiglu_backward_tile_kernel<kIn, kFmt, kClamp, true, true>
                          : swiglu_backward_tile_kernel<kIn, kFmt, kClamp, true, false>)
                     : (t ? swiglu_backward_tile_kernel<kIn, kFmt, kClamp, false, true>
                          : swiglu_backward_tile_kernel<kIn, kFmt, kClamp, false, false>);
}
template <int kIn, int kFmt>
auto pick(const SwigluTile& p) {
  return p.clamp > 0.0f ? pick_form<kIn, kFmt, true>(p) : pick_form<kIn, kFmt, false>(p);
}

}  // namespace

hipError_t launch_swiglu_backward_checkpoint(const SwigluTile& p, int ckpt_fmt, int fmt,
                                             hipStream_t stream) {
  const TileWalk tw = make_tile_walk(p.rows, p.cols, kStrip);
  if (tw.ntiles == 0) return hipSuccess;
  auto kernel = ckpt_fmt == kE4M3
                    ? (fmt == kE4M3 ? pick<kE4M3, kE4M3>(p) : pick<kE4M3, kE5M2>(p))
                    : (fmt == kE4M3 ? pick<kE5M2, kE4M3>(p) : pick<kE5M2, kE5M2>(p));
  launch_kernel(kernel, dim3(tw.per_xcd * kTileXcds), dim3(kBlock), 0, stream, p, tw);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || !p.dw || tw.nct == 1) return err;
  launch_kernel(row_weight_join_kernel, dim3((p.rows + 63) / 64), dim3(64), 0, stream,
                (const float*)p.ws, p.rows, tw.nct, p.dw);
  return hipGetLastError();
}

}  // namespace qcast
