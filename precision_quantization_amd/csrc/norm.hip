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
// HBM bandwidth, or by the launch for a few rows. 4096 x 7168 with a channel
// gate and both checkpoints: 48 us, 5.5 TB/s (a copy of as many bytes: 42.5;
// with the barriers, the loads or the stores taken out 46, 44 or 47: its vector
// instructions are the most of it); without checkpoints 37; one row 3.6; with
// two chunks a lane 1024 x 16384 28 (a copy: 25).
//
// gfx950 design. A workgroup holds a row in registers from the load to the
// last store (a lane kC chunks of 8 columns), so the row crosses HBM once
// although it is reduced twice; each sum is a wave butterfly and one LDS trip.
// It walks the rows with a stride of the grid, which leaves the columns'
// factors in registers and lets the next two rows be loaded while this one is
// worked on. Rows are read as buffers, so no branch stands around a load, and
// the next row is waited for ahead of this row's stores: operations complete
// in order, so a wait after the stores is a wait for them too (one row ahead
// with branches 53 us, two rows 50, as buffers 49). The up to three casts of a
// chunk (x and the two checkpoints)
// need three scales: lane j of a quad forms the j-th and the quad exchanges
// them, so a lane runs the scale's 30 instructions once.
#include <type_traits>

#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

// Waves resident on a compute unit that the grid is sized for. One workgroup
// of 14 waves per compute unit with rows on their way beats two that share it
// (measured with one row ahead, 4096 x 7168: 53 us against 56; without
// checkpoints, where two fit in the registers, 44 against 46).
constexpr unsigned kResidentWaves = 16;
constexpr int kMaxUnits = 4096;
// Inputs of up to this many bytes are all read with plain loads: what of them
// the 256 MB Infinity Cache still holds comes from there. Of larger ones, which
// would push each other out, only y is, which the block has just written. What
// the cache holds is not known here, so the rule goes by size. Plain against
// streaming loads of h, in us: 8192 x 2048 (67 MB) with y and h just used 25.9
// against 28.9, h alone 29.0 against 31.0, y alone 28.9 against 28.3, neither
// 31.0 against 31.8; 16384 x 512 (34 MB) 13.5 against 15.4, 13.5 against 16.5,
// 14.4 against 14.3, 18.2 against 17.6. It loses most with a cold elementwise
// gate (16384 x 512, y just used: 20.2 against 17.7), and past the bound
// (4096 x 7168, 117 MB, inputs long unused: 50 against 49).
constexpr int64_t kCachedBytes = int64_t(96) << 20;
constexpr int kMaxWaves = 16;

// The value lane j of the quad holds.
template <int kJ>
__device__ __forceinline__ float from_quad(float v) {
  return __uint_as_float(dpp<kJ * 0x55>(__float_as_uint(v)));
}

struct RowChunk {
  u32x4 y, h, gate;
};
// The chunk at byte `at` of a row; zeros past the row's end, and where there
// is no such row. `row` is the same in every lane.
template <int kGate, bool kY, bool kCached>
__device__ __forceinline__ void load_row_chunk(RowChunk& c, const NormForward& p, uint32_t row,
                                               uint32_t rows, uint32_t at) {
  const uint32_t bytes = row < rows ? p.chunks * 16 : 0;
  const uint64_t start = (uint64_t)(row < rows ? row : 0) * p.chunks * 16;
  constexpr int kPolicy = kCached ? 0 : kNonTemporal;
  if (kY) c.y = buffer_load16<0>(row_buffer(p.y, start, bytes), at);
  c.h = buffer_load16<kPolicy>(row_buffer(p.h, start, bytes), at);
  if (kGate == kGateFull) c.gate = buffer_load16<kPolicy>(row_buffer(p.gate, start, bytes), at);
}
// Waits for a chunk's loads here.
template <int kGate, bool kY>
__device__ __forceinline__ void arrive(RowChunk& c) {
  asm volatile("" : "+v"(c.h));
  if constexpr (kY) asm volatile("" : "+v"(c.y));
  if constexpr (kGate == kGateFull) asm volatile("" : "+v"(c.gate));
}

// kGate: kGateFull, kGateToken, or kGateNone for both other kinds (a channel
// gate is one of the column factors). kY: there is a block output. kCkpt: the
// checkpoints' format, 0 for none.
template <int kC, int kGate, bool kY, int kCkpt, bool kCached>
__global__ __launch_bounds__(1024) void norm_kernel(NormForward p, uint32_t rows) {
  constexpr bool kAhead = kC == 1;
  __shared__ float part[4][kMaxWaves];
  const uint32_t chunks = p.chunks;
  const uint32_t lane_at = threadIdx.x * 16, chunk_step = blockDim.x * 16;
  float c[kC][8], q[kC][8];
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t at = lane_at + k * chunk_step;
    // without w_post, or a channel gate, an empty buffer: zeros
    const bool channel = p.gate_kind == kGateChannel;
    const u32x4 wq = buffer_load16<0>(row_buffer(p.w_pre, 0, chunks * 16), at);
    const u32x4 wp = buffer_load16<0>(row_buffer(p.w_post, 0, p.w_post ? chunks * 16 : 0), at);
    const u32x4 wg = buffer_load16<0>(row_buffer(p.gate, 0, channel ? chunks * 16 : 0), at);
    float g[8];
    unpack8(wq, q[k]);
    unpack8(wp, c[k]);
    unpack8(wg, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[k][i] = q[k][i] + p.offset;
      c[k][i] = p.w_post ? c[k][i] + p.offset : 1.0f;
      if (channel) c[k][i] = c[k][i] * g[i];
    }
  }
  // lane j of a quad: the scale of x (0), of y's checkpoint (1), of h's (2)
  const int j = threadIdx.x & 3;
  const ScaleRule rule = (kCkpt && j) ? scale_rule(kCkpt, p.h_ckpt.floor)
                                      : scale_rule(p.cast.fmt, p.cast.floor);
  const int waves = blockDim.x >> 6;
  RowChunk first[kC], second[kC];
  const uint32_t step = gridDim.x;
  if (kAhead) {
    load_row_chunk<kGate, kY, kCached>(first[0], p, blockIdx.x, rows, lane_at);
    load_row_chunk<kGate, kY, kCached>(second[0], p, blockIdx.x + step, rows, lane_at);
  }
  // The row whose chunks `mine` holds; `other` holds the one after it.
  // buf alternates, so that a row's words in `part` outlive their last reader.
  const auto work = [&](RowChunk(&mine)[kC], RowChunk(&other)[kC], uint32_t row,
                        int buf) __attribute__((always_inline)) {
    const float row_gate = kGate == kGateToken ? static_cast<const float*>(p.gate)[row] : 1.0f;
    float hv[kC][8], y[kC][8], full[kGate == kGateFull ? kC : 1][8];
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      if (!kAhead)
        load_row_chunk<kGate, kY, kCached>(mine[k], p, row, rows, lane_at + k * chunk_step);
      unpack8(mine[k].h, hv[k]);
      if (kY) unpack8(mine[k].y, y[k]);
      if (kGate == kGateFull) unpack8(mine[k].gate, full[k]);
    }
    if (kAhead) load_row_chunk<kGate, kY, kCached>(mine[0], p, row + 2 * step, rows, lane_at);
    if constexpr (kY) {
      float r1 = 1.0f;
      if (p.w_post) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < kC; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(y[k][i], y[k][i], ss);
        ss = block_sum(ss, part[buf], waves);
        r1 = inv_sqrt(__builtin_fmaf(ss, p.inv_n, p.eps));
        if (p.rstd_post && threadIdx.x == 0) p.rstd_post[row] = r1;
      }
      if (kGate == kGateToken) r1 = r1 * row_gate;
      if (kAhead && p.alpha != 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) hv[0][i] = p.alpha * hv[0][i];
      }
#pragma unroll
      for (int k = 0; k < kC; ++k) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = y[k][i] * r1;
          if constexpr (kAhead) {
            hv[k][i] = kGate == kGateFull ? __builtin_fmaf(a * c[k][i], full[k][i], hv[k][i])
                                          : __builtin_fmaf(a, c[k][i], hv[k][i]);
          } else {
            const float t = kGate == kGateFull ? a * c[k][i] * full[k][i] : a * c[k][i];
            hv[k][i] = __builtin_fmaf(p.alpha, hv[k][i], t);
          }
        }
      }
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < kC; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = __builtin_fmaf(hv[k][i], hv[k][i], ss);
    ss = block_sum(ss, part[buf + 1], waves);
    const float r2 = inv_sqrt(__builtin_fmaf(ss, p.inv_n, p.eps));
    if (p.rstd_pre && threadIdx.x == 0) p.rstd_pre[row] = r2;
    if (kAhead) arrive<kGate, kY>(other[0]);
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      // The chunk: the row's first one in a scalar base and an index into the
      // row, or (two chunks a lane, where these offsets would take registers
      // for the whole loop) one index.
      const uint64_t first_chunk = (uint64_t)row * chunks;
      const uint64_t at = kAhead ? first_chunk : 0;
      using Index = std::conditional_t<kAhead, uint32_t, uint64_t>;
      const Index ix = kAhead ? jc : (Index)(first_chunk + jc);
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = hv[k][i] * r2 * q[k][i];
      if (jc >= chunks) continue;      // the lanes of a scale group leave together
      if (kY) store_stream(reinterpret_cast<u32x4*>(p.h_out) + at + ix, pack8_bf16(hv[k]));
      if (p.x_out) store_stream(reinterpret_cast<u32x4*>(p.x_out) + at + ix, pack8_bf16(x));
      float amax = run_max(absmax8_of(x), p.cast.shift);
      if (kCkpt) {
        const float ha = lane_group_max<16>(absmax8_of(hv[k]));
        amax = j == 2 ? ha : amax;
        if (kY) {
          const float ya = lane_group_max<16>(absmax8_of(y[k]));
          amax = j == 1 ? ya : amax;
        }
      }
      Scale s = scale_by(rule, amax);
      if ((p.cast.lay.flags & kSfRound) && !(kCkpt && j)) s = round_scale_pow2(s);
      if (p.cast.q) {
        encode_chunk_any(p.cast, at, ix, x, kCkpt ? from_quad<0>(s.inv) : s.inv);
        store_run_scale(p.cast.sf, row, jc >> p.cast.shift, s, p.cast.lay, p.cast.shift);
      }
      if constexpr (kCkpt != 0) {
        const uint64_t sat = (uint64_t)row * (chunks / 16) + jc / 16;
        const int l = threadIdx.x & 15;
        if (p.h_ckpt.q) {
          encode_chunk<kCkpt>(p.h_ckpt, at, ix, hv[k], from_quad<2>(s.inv));
          if (l == 2) static_cast<float*>(p.h_ckpt.sf)[sat] = s.sf;
        }
        if (kY && p.y_ckpt.q) {
          encode_chunk<kCkpt>(p.y_ckpt, at, ix, y[k], from_quad<1>(s.inv));
          if (l == 1) static_cast<float*>(p.y_ckpt.sf)[sat] = s.sf;
        }
      }
    }
  };
  uint32_t row = blockIdx.x;
  if constexpr (kAhead) {
    while (true) {
      work(first, second, row, 0);
      row = __builtin_amdgcn_readfirstlane(row + step);
      if (row >= rows) break;
      work(second, first, row, 2);
      row = __builtin_amdgcn_readfirstlane(row + step);
      if (row >= rows) break;
    }
  } else {
    int buf = 0;
    for (; row < rows; row = __builtin_amdgcn_readfirstlane(row + step), buf ^= 2)
      work(first, first, row, buf);
  }
}

template <int kC, bool kCached, int kGate, bool kY>
auto pick_ckpt(const NormForward& p) {
  const int f = (p.h_ckpt.q || p.y_ckpt.q) ? p.h_ckpt.fmt : 0;
  return f == 0       ? norm_kernel<kC, kGate, kY, 0, kCached>
         : f == kE4M3 ? norm_kernel<kC, kGate, kY, kE4M3, kCached>
                      : norm_kernel<kC, kGate, kY, kE5M2, kCached>;
}
template <int kC, bool kCached>
auto pick(const NormForward& p) {
  return !p.y                        ? pick_ckpt<kC, kCached, kGateNone, false>(p)
         : p.gate_kind == kGateFull  ? pick_ckpt<kC, kCached, kGateFull, true>(p)
         : p.gate_kind == kGateToken ? pick_ckpt<kC, kCached, kGateToken, true>(p)
                                     : pick_ckpt<kC, kCached, kGateNone, true>(p);
}

}  // namespace

hipError_t launch_norm(const NormForward& p, int64_t rows, hipStream_t stream,
                       const LaunchCaps& caps) {
  if (rows == 0 || p.chunks == 0) return hipSuccess;
  if (rows >= (int64_t(1) << 31) || p.chunks > kNormMaxChunks) return hipErrorInvalidValue;
  const int inputs = 1 + (p.y != nullptr) + (p.gate_kind == kGateFull);
  const bool cached = rows * p.chunks * 16 * inputs <= kCachedBytes;
  const int kc = p.chunks > 1024 ? 2 : 1;
  const unsigned threads = (unsigned)(((p.chunks + kc - 1) / kc + 63) / 64 * 64);
  const unsigned waves = threads / 64;
  // whatever the override says, row + 2 * grid stays within 32 bits
  const int64_t cus = caps.num_cus < kMaxUnits ? caps.num_cus : kMaxUnits;
  const int64_t resident = cus * (waves < kResidentWaves ? kResidentWaves / waves : 1);
  const unsigned grid = (unsigned)(rows < resident ? rows : resident);
  auto kernel = kc == 1 ? (cached ? pick<1, true>(p) : pick<1, false>(p))
                        : (cached ? pick<2, true>(p) : pick<2, false>(p));
  launch_kernel(kernel, dim3(grid), dim3(threads), 0, stream, p, (uint32_t)rows);
  return hipGetLastError();
}

}  // namespace qcast
