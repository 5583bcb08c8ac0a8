// qcast_tile.h -- what the kernels on tiles of 128 tokens x 128 channels
// share: the walk over the tiles, the LDS tile in which 8-bit codes are
// transposed, and the scales of the 128 channels.
//
// Codes wait in LDS as rows of 128 tokens (32 dwords) per channel, a dword
// holding 4 consecutive tokens. Rows are 36 dwords apart and the dword index
// is XOR-swizzled in whole 16-byte groups by the channel: 16 lanes writing
// channels 8 (or 16) apart and the same tokens then fall on distinct banks
// (36 * 8 is 32 mod 64, so every other such lane takes the other half), and a
// 16-byte run of tokens stays contiguous and aligned for the read-back.
#pragma once

#include "qcast_device.h"
#include "qcast_kernels.h"

namespace qcast {

constexpr uint32_t kTile = 128;              // tokens and channels of a tile
constexpr uint32_t kTileXcds = 8;

// Tile walk: each XCD takes a contiguous range of tiles, in strips of `strip`
// channel tiles: token group outer, channel tile inner.
struct TileWalk {
  uint32_t ntg, nct, ntiles, per_xcd, strip;
  FastDiv strip_div;       // by strip * ntg
};
struct TilePos {
  uint32_t ct, gt;
};
inline TileWalk make_tile_walk(int64_t rows, int64_t cols, uint32_t strip) {
  TileWalk w;
  w.ntg = (uint32_t)((rows + kTile - 1) / kTile);
  w.nct = (uint32_t)((cols + kTile - 1) / kTile);
  w.ntiles = w.ntg * w.nct;
  w.per_xcd = (w.ntiles + kTileXcds - 1) / kTileXcds;
  w.strip = strip;
  w.strip_div = make_fast_div(w.ntg * strip ? w.ntg * strip : 1);
  return w;
}
__device__ __forceinline__ TilePos tile_pos(uint32_t tau, const TileWalk& w) {
  const uint32_t s = fast_div(tau, w.strip_div);
  const uint32_t rem = tau - s * w.strip * w.ntg;
  const uint32_t width = w.nct - s * w.strip < w.strip ? w.nct - s * w.strip : w.strip;
  TilePos p;
  p.gt = rem / width;
  p.ct = s * w.strip + (rem - p.gt * width);
  return p;
}

constexpr uint32_t kTileRowDw = 36;
constexpr uint32_t kTileDw = kTile * kTileRowDw;
__device__ __forceinline__ uint32_t swizzled(uint32_t channel, uint32_t dword) {
  return channel * kTileRowDw + (dword ^ (4 * ((channel >> 4) & 7)));
}

// The lane's scales of its kTokens consecutive tokens (lane / kLanes of the
// wave's 64 / kLanes such runs, the wave's first token t0; sf[t * stride] the
// scale of token t), 0 for tokens past `rows`. They come through scalar loads,
// one per token of the wave, and a select: as vector loads their cache lines,
// one per token for 4 bytes, take as many requests as the tokens' codes
// themselves (recast of 16384 x 7168: 50.3 us, 44.2 this way, 41.8 with no
// scales to load; with the index clamped instead of the branch 47). For two
// scales per token beside four times the bytes, as in the SwiGLU backward,
// the vector loads are faster (32.5 against 35.9 us).
template <int kTokens, int kLanes>
__device__ __forceinline__ void token_scales(const float* __restrict__ sf, uint32_t stride,
                                             uint32_t t0, uint32_t rows, float out[kTokens]) {
  constexpr uint32_t kRuns = 64 / kLanes;
  const uint32_t run = (threadIdx.x & 63) / kLanes;
#pragma unroll
  for (uint32_t i = 0; i < kTokens; ++i) {
    float v = 0.0f;
#pragma unroll
    for (uint32_t r = 0; r < kRuns; ++r) {
      const uint32_t t = t0 + r * kTokens + i;
      const float s = t < rows ? sf[(uint64_t)t * stride] : 0.0f;
      v = run == r ? s : v;
    }
    out[i] = t0 + run * kTokens + i < rows ? v : 0.0f;
  }
}

// The scale of one channel over the tile's tokens, formed and stored by one
// lane; returns what its values are multiplied by.
template <int kFmt, bool kLayout>
__device__ __forceinline__ float channel_scale(void* sf, const SfLayout& lay, uint32_t channel,
                                               uint32_t group, float amax, float floor) {
  Scale s = group_scale<kFmt>(amax, floor);
  if (kLayout) {
    if (lay.flags & kSfRound) s = round_scale_pow2(s);
    store_lone_scale(sf, channel, group, s, lay);
  } else {
    static_cast<float*>(sf)[(uint64_t)channel * lay.gpr + group] = s.sf;
  }
  return s.inv;
}

// Store the LDS tile's channel rows [c0, c0 + nc) of token group gt, 16
// tokens per lane. rows_T: codes per channel row. kN threads call this.
// kStream: past the caches; else with plain stores.
template <int kN, bool kStream>
__device__ __forceinline__ void store_tile_rows(const uint32_t* tile, uint8_t* qT, uint32_t c0,
                                                uint32_t nc, uint32_t gt, uint32_t rows_T) {
  uint8_t* out = qT + (uint64_t)c0 * rows_T + gt * kTile;
#pragma unroll
  for (uint32_t r = 0; r < kTile * 8 / kN; ++r) {
    const uint32_t idx = threadIdx.x + r * kN;
    const uint32_t c = idx / 8, v = idx % 8;
    if (c < nc) {
      const u32x4 val = *reinterpret_cast<const u32x4*>(tile + swizzled(c, 4 * v));
      u32x4* to = reinterpret_cast<u32x4*>(out + c * rows_T + 16 * v);
      if (kStream) store_stream(to, val);
      else *to = val;
    }
  }
}

}  // namespace qcast
