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
// with b = dh' + r2 * g (then dH = b - r2 * mean(g * xh) * xh) the sums
// S1 = sum g * xh, S2 = sum b * c and S3 = sum xh * c, c = gate * wp * a, are
// taken together and
//   sum da * a = S2 - r2 * (S1 / n) * S3.
//
// gfx950 design. Workgroups walk the rows with a stride, so a lane meets the
// same columns in every row and holds the column sums in fp32 registers; each
// workgroup writes its sums to the workspace once and a second kernel adds
// them up in a fixed order (no atomics, and a grid that follows from the
// sizes alone: the result depends on nothing else). A channel gate and w_post
// are the same in every row, so their gradients are one sum T = sum d * a:
// dw_post = gate * T, dgate = wp * T. With one chunk of 8 columns per lane
// (rows of up to 8192) the next row is loaded while the current one is
// worked on, and the values of the first half are kept for the second; longer
// rows (up to 16384) keep the packed inputs, form the values again, and hold
// the column sums in LDS (128 KB, each lane its own words). With a block output
// 13 to 30 registers of a lane spill.
//
// What it must move: dx, dh', both saved tensors, dh and the codes of dy (9
// bytes per element from 8-bit checkpoints, 11 from bf16), plus 8 bytes per
// column and workgroup of partial sums. 4096 x 7168, channel gate, from
// checkpoints: 54 us, of which the join takes 5 (a copy of 264 MB: 42). Past
// 8192 columns, without a row ahead: 1024 x 16384 58 us (a copy: 25).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kMaxWaves = 16;
constexpr int kJoinWaves = 16;     // waves of the joining workgroup
constexpr int kJoinAhead = 8;      // parts a lane loads at once

// The lane's raw data of one chunk of one row: bf16 octets, or 8-bit codes in
// the low two words with their scales.
// r1, r2 and a token gate of its row travel with it, so that nothing loaded
// later has to be waited for before the row can be worked on.
struct Chunk {
  u32x4 dx, dh, gate, hs, ys;
  float hsf, ysf, r1, r2, row_gate;
};

template <int kSaved, int kGate, bool kY>
__device__ __forceinline__ Chunk load_chunk(const NormBackward& p, uint32_t row, uint32_t jc,
                                            bool valid) {
  const int64_t at = (int64_t)row * p.chunks + jc;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  Chunk c;
  c.dx = c.dh = c.gate = c.hs = c.ys = zero;
  c.hsf = c.ysf = c.r1 = c.row_gate = 1.0f;
  c.r2 = p.rstd_pre[row];
  if (kY && p.rstd_post) c.r1 = p.rstd_post[row];
  if (kGate == kGateToken) c.row_gate = static_cast<const float*>(p.gate)[row];
  if (!valid) return c;
  // The gradients were written by the calls before this one, the saved tensors
  // long before: plain loads for the first alone, so that what the Infinity
  // Cache holds of them is read there and stays (bf16, 8192 x 2048 41 us
  // against 47, 4096 x 7168 with the gradients just written 58 against 65).
  c.dx = reinterpret_cast<const u32x4*>(p.dx)[at];
  if (p.dh_in) c.dh = reinterpret_cast<const u32x4*>(p.dh_in)[at];
  if (kGate == kGateFull) c.gate = load_stream(reinterpret_cast<const u32x4*>(p.gate) + at);
  if constexpr (kSaved != 0) {
    const int64_t s = (int64_t)row * (p.chunks / 16) + jc / 16;
    const u32x2 h = load_stream(static_cast<const u32x2*>(p.saved_h) + at);
    c.hs.x = h.x;
    c.hs.y = h.y;
    c.hsf = p.saved_h_sf[s];
    if (kY) {
      const u32x2 y = load_stream(static_cast<const u32x2*>(p.saved_y) + at);
      c.ys.x = y.x;
      c.ys.y = y.y;
      c.ysf = p.saved_y_sf[s];
    }
  } else {
    c.hs = load_stream(static_cast<const u32x4*>(p.saved_h) + at);
    if (kY) c.ys = load_stream(static_cast<const u32x4*>(p.saved_y) + at);
  }
  return c;
}

// Waits for the loads of a chunk here. Memory operations complete in order, so
// a wait after the current row's stores would be a wait for those stores too.
template <int kSaved, int kGate, bool kY>
__device__ __forceinline__ void arrive(Chunk& c) {
  asm volatile("" : "+v"(c.dx), "+v"(c.dh), "+v"(c.r2));
  if constexpr (kSaved != 0) {
    asm volatile("" : "+v"(c.hs.x), "+v"(c.hs.y), "+v"(c.hsf));
    if constexpr (kY) asm volatile("" : "+v"(c.ys.x), "+v"(c.ys.y), "+v"(c.ysf));
  } else {
    asm volatile("" : "+v"(c.hs));
    if constexpr (kY) asm volatile("" : "+v"(c.ys));
  }
  if constexpr (kY) asm volatile("" : "+v"(c.r1));
  if constexpr (kGate == kGateToken) asm volatile("" : "+v"(c.row_gate));
}

template <int kSaved>
__device__ __forceinline__ void saved_values(const u32x4& raw, float sf, float v[8]) {
  if constexpr (kSaved != 0) {
    decode8<kSaved>(u32x2{raw.x, raw.y}, sf, v);
  } else {
    unpack8(raw, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * sf;
  }
}

// The factors of a chunk's columns: q = w_pre + offset, and c = wp (times a
// channel gate; 1 without w_post).
__device__ __forceinline__ void column_factors(const NormBackward& p, uint32_t jc, float q[8],
                                               float c[8]) {
  // past the row, without w_post or a channel gate: zeros of an empty buffer
  const bool channel = p.gate_kind == kGateChannel;
  const uint32_t n = p.chunks * 16;
  const u32x4 wq = buffer_load16<0>(row_buffer(p.w_pre, 0, n), jc * 16);
  const u32x4 wp = buffer_load16<0>(row_buffer(p.w_post, 0, p.w_post ? n : 0), jc * 16);
  const u32x4 wg = buffer_load16<0>(row_buffer(p.gate, 0, channel ? n : 0), jc * 16);
  float g[8];
  unpack8(wq, q);
  unpack8(wp, c);
  unpack8(wg, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    q[i] = q[i] + p.offset;
    c[i] = p.w_post ? c[i] + p.offset : 1.0f;
    if (channel) c[i] = c[i] * g[i];
  }
}

// The fp32 values of a chunk that both halves of a row's work use.
struct Values {
  float x[8], a[8], b[8], c[8];      // xh, a, dh' + r2 * dx * q, gate * wp
};

template <int kSaved, int kGate, bool kY>
__device__ __forceinline__ Values chunk_values(const Chunk& ch, const float q[8],
                                               const float c[8], float dx[8],
                                               float gx[8]) {
  Values v;
  unpack8(ch.dx, dx);
  unpack8(ch.dh, v.b);
  // code * sf * r in one product: code * (sf * r)
  saved_values<kSaved>(ch.hs, kSaved ? ch.hsf * ch.r2 : ch.r2, v.x);
  if (kY) saved_values<kSaved>(ch.ys, kSaved ? ch.ysf * ch.r1 : ch.r1, v.a);
  float g[8];
  if (kGate == kGateFull) unpack8(ch.gate, g);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    gx[i] = dx[i] * q[i];
    v.b[i] = __builtin_fmaf(ch.r2, gx[i], v.b[i]);
    v.c[i] = kGate == kGateFull ? c[i] * g[i] : c[i];
  }
  return v;
}

// A lane's 8 column sums in two LDS rows of one f32x4 per thread.
__device__ __forceinline__ void load_sums(const f32x4* row, float v[8]) {
  const f32x4 a = row[threadIdx.x], b = row[1024 + threadIdx.x];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store_sums(f32x4* row, const float v[8]) {
  row[threadIdx.x] = f32x4{v[0], v[1], v[2], v[3]};
  row[1024 + threadIdx.x] = f32x4{v[4], v[5], v[6], v[7]};
}

// kSaved: 0 for bf16, else the format of the 8-bit checkpoints. kGate:
// kGateFull, kGateToken, or kGateNone for both other kinds (a channel gate is
// one of the column factors). kY: there is a block output.
template <int kC, int kSaved, int kGate, bool kY>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBackward p, uint32_t rows) {
  constexpr bool kKeep = kC == 1;
  __shared__ __attribute__((aligned(16))) float part[2][kMaxWaves][4];
  const uint32_t chunks = p.chunks;
  constexpr bool kFull = kGate == kGateFull;
  // the lane's column sums: registers, or (kC == 2) its own LDS words
  __shared__ __attribute__((aligned(16))) f32x4 acc[kKeep ? 1 : 4 * kC * 1024];
  float q[kC][8], c[kC][8], s_pre[8], s_post[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s_pre[i] = s_post[i] = 0.0f;
  if constexpr (kKeep) {
    column_factors(p, threadIdx.x, q[0], c[0]);
  } else {
#pragma unroll
    for (int i = 0; i < 4 * kC; ++i) acc[i * 1024 + threadIdx.x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }
  Chunk next;
  if (kKeep)
    next = load_chunk<kSaved, kGate, kY>(p, blockIdx.x, threadIdx.x, threadIdx.x < chunks);
  int parity = 0;
  const int waves = blockDim.x >> 6;
  for (uint32_t row = blockIdx.x; row < rows; row += gridDim.x, parity ^= 1) {
    Chunk ch[kC];
    if constexpr (kKeep) {
      ch[0] = next;
      if (row + gridDim.x < rows)
        next = load_chunk<kSaved, kGate, kY>(p, row + gridDim.x, threadIdx.x,
                                             threadIdx.x < chunks);
    } else {
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        const uint32_t jc = threadIdx.x + k * blockDim.x;
        ch[k] = load_chunk<kSaved, kGate, kY>(p, row, jc, jc < chunks);
      }
    }
    const float r1 = ch[0].r1, r2 = ch[0].r2, row_gate = ch[0].row_gate;
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
    Values kept;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      if (!kKeep) column_factors(p, jc, q[k], c[k]);
      float dx[8], gx[8];
      const Values v = chunk_values<kSaved, kGate, kY>(ch[k], q[k], c[k], dx, gx);
      if constexpr (!kKeep) load_sums(acc + 4 * k * 1024, s_pre);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        s1 = __builtin_fmaf(gx[i], v.x[i], s1);
        s_pre[i] = __builtin_fmaf(dx[i], v.x[i], s_pre[i]);
        if (kY) {
          const float cc = v.a[i] * v.c[i];
          s2 = __builtin_fmaf(v.b[i], cc, s2);
          s3 = __builtin_fmaf(v.x[i], cc, s3);
        }
      }
      if constexpr (kKeep) kept = v;
      else store_sums(acc + 4 * k * 1024, s_pre);
    }
    block_sum3(s1, s2, s3, part[parity], waves);
    const float m1 = s1 * p.inv_n;
    const float r2m1 = r2 * m1;
    const float along = s2 - r2m1 * s3;      // sum dH * a * c, without a token gate
    if (kY && kGate == kGateToken && p.dgate && threadIdx.x == 0)
      static_cast<float*>(p.dgate)[row] = along;
    const float m2 = (kY && p.w_post) ? along * row_gate * p.inv_n : 0.0f;
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      const uint32_t jc = threadIdx.x + k * blockDim.x;
      Values v;
      if constexpr (kKeep) {
        v = kept;
      } else {
        float dx[8], gx[8];
        column_factors(p, jc, q[k], c[k]);
        v = chunk_values<kSaved, kGate, kY>(ch[k], q[k], c[k], dx, gx);
      }
      float g[8], d[8], out[8];
      if (kFull) unpack8(ch[k].gate, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        d[i] = __builtin_fmaf(-v.x[i], r2m1, v.b[i]);
        out[i] = p.alpha * d[i];
      }
      const int64_t at = (int64_t)row * chunks + jc;
      const u32x4 dh_bits = pack8_bf16(out);
      // 4096 x 7168: 54 us against 57, 8192 x 5120 in bf16: 82 against 99 (with
      // an elementwise gate there are no registers for it: 1000 x 2048 15.4
      // against 14.3)
      if constexpr (kKeep && !kFull) arrive<kSaved, kGate, kY>(next);
      if (jc < chunks) store_stream(reinterpret_cast<u32x4*>(p.dh_out) + at, dh_bits);
      if (kY) {
        if constexpr (!kKeep) load_sums(acc + (4 * k + 2) * 1024, s_post);
        // without the column's own factors: d * a * (token or elementwise gate)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float dz = kFull ? d[i] * g[i] : kGate == kGateToken ? d[i] * row_gate : d[i];
          s_post[i] = __builtin_fmaf(dz, v.a[i], s_post[i]);
          out[i] = dz * (kFull ? c[k][i] : v.c[i]);
          if (p.w_post) out[i] = r1 * __builtin_fmaf(-v.a[i], m2, out[i]);
        }
        if constexpr (!kKeep) store_sums(acc + (4 * k + 2) * 1024, s_post);
        if (jc < chunks) {
          if (kFull && p.dgate) {
            float dg[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) dg[i] = d[i] * v.a[i] * c[k][i];
            store_stream(static_cast<u32x4*>(p.dgate) + at, pack8_bf16(dg));
          }
          if (p.dy_out) store_stream(reinterpret_cast<u32x4*>(p.dy_out) + at, pack8_bf16(out));
          if (p.cast.q) cast_chunk(p.cast, row, jc, chunks, out);
        }
      }
    }
  }
  // this workgroup's column sums: [workgroup][2][column]
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    const uint32_t jc = threadIdx.x + k * blockDim.x;
    if (jc < chunks) {
      if constexpr (!kKeep) {
        load_sums(acc + 4 * k * 1024, s_pre);
        load_sums(acc + (4 * k + 2) * 1024, s_post);
      }
      float* o = p.ws + (int64_t)blockIdx.x * 2 * 8 * chunks + 8 * jc;
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<f32x4*>(o + i) =
            f32x4{s_pre[i], s_pre[i + 1], s_pre[i + 2], s_pre[i + 3]};
        if (kY)
          *reinterpret_cast<f32x4*>(o + 8 * chunks + i) =
              f32x4{s_post[i], s_post[i + 1], s_post[i + 2], s_post[i + 3]};
      }
    }
  }
}

// The column gradients from the sums of `parts` workgroups, added in a fixed
// order: wave w of a workgroup adds parts w, w + 16, ..., then the 16 partial
// sums are added in order. blockIdx.y 0: dw_pre; 1: T, which gives dw_post
// (times a channel gate) and a channel gate's gradient (times wp).
__global__ __launch_bounds__(64 * kJoinWaves) void norm_backward_join_kernel(NormBackward p,
                                                                           uint32_t parts) {
  __shared__ float part[kJoinWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const uint32_t cols = p.chunks * 8;
  const uint32_t col = blockIdx.x * 64 + lane;
  const float* ws = p.ws + (int64_t)blockIdx.y * cols + col;
  float s = 0.0f;
  if (col < cols) {
    for (uint32_t i0 = wave; i0 < parts; i0 += kJoinWaves * kJoinAhead) {
      float v[kJoinAhead];                // all loads in flight before the first sum
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) {
        const uint32_t j = i0 + i * kJoinWaves;
        v[i] = j < parts ? ws[(int64_t)j * 2 * cols] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < kJoinAhead; ++i) s += v[i];
    }
  }
  part[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= cols) return;
  float t = part[0][lane];
  for (int i = 1; i < kJoinWaves; ++i) t += part[i][lane];
  if (blockIdx.y == 0) {
    if (p.sums[0]) p.sums[0][col] = t;
    return;
  }
  const bool channel = p.gate_kind == kGateChannel;
  if (p.sums[1])
    p.sums[1][col] =
        channel ? t * bf16_lo(static_cast<const uint16_t*>(p.gate)[col]) : t;
  if (p.sums[2]) p.sums[2][col] = p.w_post ? t * (bf16_lo(p.w_post[col]) + p.offset) : t;
}

template <int kC, int kSaved>
auto pick(const NormBackward& p) {
  return !p.saved_y                    ? norm_backward_kernel<kC, kSaved, kGateNone, false>
         : p.gate_kind == kGateFull  ? norm_backward_kernel<kC, kSaved, kGateFull, true>
         : p.gate_kind == kGateToken ? norm_backward_kernel<kC, kSaved, kGateToken, true>
                                     : norm_backward_kernel<kC, kSaved, kGateNone, true>;
}
template <int kC>
auto pick_saved(const NormBackward& p) {
  return p.saved_fmt == 0       ? pick<kC, 0>(p)
         : p.saved_fmt == kE4M3 ? pick<kC, kE4M3>(p)
                                : pick<kC, kE5M2>(p);
}

}  // namespace

hipError_t launch_norm_backward(const NormBackward& p, int64_t rows, uint32_t parts,
                                hipStream_t stream) {
  if (p.chunks == 0) return hipSuccess;
  if (rows >= (int64_t(1) << 31) || p.chunks > kNormMaxChunks) return hipErrorInvalidValue;
  if (parts) {
    const int kc = p.chunks > 1024 ? 2 : 1;
    const unsigned threads = (unsigned)(((p.chunks + kc - 1) / kc + 63) / 64 * 64);
    auto kernel = kc == 1 ? pick_saved<1>(p) : pick_saved<2>(p);
    launch_kernel(kernel, dim3(parts), dim3(threads), 0, stream, p, (uint32_t)rows);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  // with no rows, the sums over them: zeros
  if (!p.sums[0] && !p.sums[1] && !p.sums[2]) return hipSuccess;
  launch_kernel(norm_backward_join_kernel,
                dim3((p.chunks * 8 + 63) / 64, p.sums[1] || p.sums[2] ? 2 : 1),
                dim3(64 * kJoinWaves), 0, stream, p, parts);
  return hipGetLastError();
}

}  // namespace qcast
