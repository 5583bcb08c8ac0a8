// recast.hip -- stored per-token 8-bit codes cast again along the tokens and
// written transposed (the operand of a weight gradient from an activation
// that the forward pass kept in 8 bits).
//
// x[t][c] = decode(code) * sf[t][c / in_group] in fp32; then the per-channel
// cast over 128 tokens written transposed (per_channel_t.hip), with the last
// token group filled up with zeros. Going through cast_back and the bf16
// transposed cast moves 6 bytes per element and rounds to bf16 on the way;
// this moves 2.
//
// gfx950 design. A workgroup owns 128 tokens x 128 channels. A lane loads 16
// consecutive channels (16 bytes) of 4 consecutive tokens and keeps the
// codes, not the values: they are decoded once for the maxima and again for
// the codes, which costs one conversion per two values and saves 64
// registers. 8 lanes cover a token's 128 channels. Bound by HBM traffic in
// 128-byte pieces on both sides: 44 us for 16384 x 7168, 5.5 TB/s (a copy of
// as many bytes 39; twice the tokens per tile, 256-byte pieces out, 3 us more).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"
#include "qcast_tile.h"

namespace qcast {
namespace {

// The fp32 value of code j (0..15) of a token's 16 codes.
template <int kIn>
__device__ __forceinline__ void decode_word(uint32_t w, float sf, float v[4]) {
  decode4<kIn>(w, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = v[i] * sf;
}

// kLayout: scale options other than plain fp32. kWide: input groups of 128,
// one scale per token of the tile.
template <int kIn, int kFmt, bool kLayout, bool kWide>
__global__ __launch_bounds__(kThreads) void recast_kernel(RecastTile p, TileWalk tw) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[kTileDw];
  __shared__ float amax_s[kThreads / 64][kTile];
  __shared__ float inv_s[kTile];
  const uint32_t tau = (blockIdx.x % kTileXcds) * tw.per_xcd + blockIdx.x / kTileXcds;
  if (tau >= tw.ntiles) return;
  const TilePos tp = tile_pos(tau, tw);
  const uint32_t ct = tp.ct, gt = tp.gt;
  const uint32_t c0 = ct * kTile, t0 = gt * kTile;
  const uint32_t nc = p.cols - c0 < kTile ? p.cols - c0 : kTile;
  const uint32_t ch = threadIdx.x & 7;           // 16-channel chunk
  const uint32_t quad = threadIdx.x >> 3;        // 4 tokens
  const bool valid_ch = ch * 16 < nc;
  const uint32_t gpr = p.cols >> (p.shift + 3);
  u32x4 raw[4];
  float sf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t t = t0 + quad * 4 + i;
    raw[i] = u32x4{0u, 0u, 0u, 0u};
    sf[i] = 0.0f;
    if (valid_ch && t < p.rows) {
      const uint64_t at = (uint64_t)t * p.cols + c0 + ch * 16;
      raw[i] = load_stream(reinterpret_cast<const u32x4*>(p.q + at));
      // 16 channels lie in one group: groups of 32, 64 and 128 are whole chunks
      if (!kWide) sf[i] = p.sf[(uint64_t)t * gpr + ((c0 + ch * 16) >> (p.shift + 3))];
    }
  }
  if constexpr (kWide) {
    const uint32_t tw0 = t0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 32;
    token_scales<4, 8>(p.sf + ct, gpr, tw0, p.rows, sf);
  }
  // Column maxima of the lane's 4 tokens, then over the 8 lanes of the wave
  // that hold the same 16 channels (lane bits 3, 4, 5), as a butterfly whose
  // exchanges carry two channels each: a lane ends with two of the 16.
  uint32_t m[16];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    float t[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) decode_word<kIn>(raw[i][w], sf[i], t[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      m[4 * w + j] = __float_as_uint(absmax4(t[0][j], t[1][j], t[2][j], t[3][j]));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {        // bit 4: upper 8 channels
    const auto r = __builtin_amdgcn_permlane16_swap(m[j], m[j + 8], false, false);
    m[j] = umax((uint32_t)r[0], (uint32_t)r[1]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {        // bit 5: upper 4 of those
    const auto r = __builtin_amdgcn_permlane32_swap(m[j], m[j + 4], false, false);
    m[j] = umax((uint32_t)r[0], (uint32_t)r[1]);
  }
  const bool odd = (threadIdx.x & 8) != 0;   // bit 3: upper 2 of those
  const uint32_t c2 = ch * 16 + ((threadIdx.x >> 4) & 1) * 8 + ((threadIdx.x >> 5) & 1) * 4 +
                      (odd ? 2 : 0);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint32_t keep = odd ? m[j + 2] : m[j], send = odd ? m[j] : m[j + 2];
    amax_s[threadIdx.x >> 6][c2 + j] = __uint_as_float(umax(keep, dpp<kDppRor8>(send)));
  }
  __syncthreads();
  if (threadIdx.x < kTile) {
    const uint32_t c = threadIdx.x;
    float m = amax_s[0][c];
#pragma unroll
    for (int i = 1; i < kThreads / 64; ++i) m = fmaxf(m, amax_s[i][c]);
    if (c < nc) inv_s[c] = channel_scale<kFmt, kLayout>(p.out.sf, p.out.lay, c0 + c, gt, m, p.floor);
  }
  __syncthreads();
  if (valid_ch) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      float v[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) decode_word<kIn>(raw[i][w], sf[i], v[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t c = ch * 16 + 4 * w + j;
        const float inv = inv_s[c];
        tile[swizzled(c, quad)] =
            fp8x4<kFmt>(v[0][j] * inv, v[1][j] * inv, v[2][j] * inv, v[3][j] * inv);
      }
    }
  }
  __syncthreads();
  // plain stores: 50.3 against 52.8 us with streaming ones (16384 x 7168); the
  // tiles of neighbouring token groups write the other parts of these rows
  store_tile_rows<kThreads, false>(tile, p.out.qT, c0, nc, gt, tw.ntg * kTile);
}

template <int kIn, int kFmt>
auto pick(const RecastTile& p) {
  const bool layout = p.out.lay.flags != 0, wide = p.shift == 4;
  return layout ? (wide ? recast_kernel<kIn, kFmt, true, true> : recast_kernel<kIn, kFmt, true, false>)
                : (wide ? recast_kernel<kIn, kFmt, false, true>
                        : recast_kernel<kIn, kFmt, false, false>);
}

}  // namespace

bool tile_fits(int64_t rows, int64_t cols, int64_t stride) {
  const int64_t lim = int64_t(1) << 31;
  if (rows < 0 || rows >= lim || stride >= lim) return false;
  const int64_t ntg = (rows + kTile - 1) / kTile;
  const int64_t nct = (cols + kTile - 1) / kTile;
  return (nct == 0 || ntg < (lim - 16) / nct) && (int64_t)kTile * stride < lim &&
         (int64_t)kTile * kTile * ntg < lim;
}

hipError_t launch_recast(const RecastTile& p, int in_fmt, int fmt, hipStream_t stream) {
  // Channel tiles per strip: an XCD's share of them, 2 to 8, so that the tiles
  // that read one token's scales run together on one L2 (56 tiles: 46.4 us with
  // 7, 47.9 with 2).
  const uint32_t share = ((p.cols + kTile - 1) / kTile + kTileXcds - 1) / kTileXcds;
  const TileWalk tw = make_tile_walk(p.rows, p.cols, share < 2 ? 2 : share > 8 ? 8 : share);
  if (tw.ntiles == 0) return hipSuccess;
  auto kernel = in_fmt == kE4M3 ? (fmt == kE4M3 ? pick<kE4M3, kE4M3>(p) : pick<kE4M3, kE5M2>(p))
                                : (fmt == kE4M3 ? pick<kE5M2, kE4M3>(p) : pick<kE5M2, kE5M2>(p));
  launch_kernel(kernel, dim3(tw.per_xcd * kTileXcds), dim3(kThreads), 0, stream, p, tw);
  return hipGetLastError();
}

}  // namespace qcast
