// qcast_kernels.h -- launchers of the gfx950 cast kernels (internal to the
// library; the C ABI in qcast_abi.hip validates arguments before calling).
#pragma once

#include <hip/hip_ext.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qcast_device.h"

namespace qcast {

// Start and stop events for the next kernel launched by the calling thread
// (qcast_bench_time_next); both null when none were asked for. Taking them
// clears them.
struct LaunchTiming {
  hipEvent_t start;
  hipEvent_t stop;
};
LaunchTiming take_launch_timing();

// Every kernel of the library is launched through here: with timing events
// pending, hipExtLaunchKernel records them from the dispatch itself (the
// kernel's own start and end, with no marker packets around it).
template <typename... KArgs, typename... Args>
inline void launch_kernel(void (*kernel)(KArgs...), dim3 grid, dim3 block, uint32_t shmem,
                          hipStream_t stream, Args... args) {
  const LaunchTiming t = take_launch_timing();
  hipExtLaunchKernelGGL(kernel, grid, block, shmem, stream, t.start, t.stop, 0u, args...);
}

// A grid has fewer than 2^32 threads: more workgroups than that take several
// launches, launch(first workgroup's number, workgroups). Whole ones are a
// multiple of the 8 XCDs long.
template <typename F>
inline hipError_t each_launch(uint64_t groups, uint32_t threads, F&& launch) {
  const uint64_t most = ((uint64_t(1) << 32) / threads - 1) / 8 * 8;
  for (uint64_t first = 0; first < groups; first += most) {
    launch((uint32_t)first, (uint32_t)(groups - first < most ? groups - first : most));
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

// The same for a kernel whose last argument is the first workgroup's number.
template <typename... KArgs, typename... Args>
inline hipError_t launch_groups(void (*kernel)(KArgs...), uint64_t groups, uint32_t threads,
                                hipStream_t stream, const Args&... args) {
  return each_launch(groups, threads, [&](uint32_t first, uint32_t n) {
    launch_kernel(kernel, dim3(n), dim3(threads), 0, stream, args..., first);
  });
}

// Whether a shape fits the kernels' 32-bit tile counts and in-tile offsets
// (checked by the C ABI before any HIP call; the launchers check again).
bool per_block_fits(int64_t rows, int64_t cols);
bool per_channel_t_fits(int64_t rows, int64_t cols, int64_t row_stride, int fmt);
bool per_channel_fits(int64_t rows, int64_t cols);
bool cast_back_fits(int64_t rows, int64_t cols);

// Launch shape knobs shared by the launchers.
struct LaunchCaps {
  int num_cus;          // compute units on the device (or the override)
};

// The scale-factor layout of a per-token cast of [rows, cols] with `group`.
inline SfLayout make_sf_layout(int64_t rows, int64_t cols, int group, uint32_t flags) {
  SfLayout lay;
  lay.flags = (flags & kSfPacked) ? (flags | kSfRound) : flags;
  lay.gpr = (uint32_t)(cols / group);
  lay.rows_pad = (uint32_t)((rows + 3) / 4 * 4);
  lay.inv_gpr = lay.gpr ? 1.0 / (double)lay.gpr : 0.0;
  return lay;
}

// x [rows, cols] bf16 -> per-token codes + scales in the layout sf_flags
// (kSf* bits); group in {32, 64, 128}; fmt kE4M3, kE5M2 or kE2M1. Requires
// cols % group == 0, and (cols / group) % 4 == 0 for kSfPacked.
hipError_t launch_per_token(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                            float floor, uint32_t sf_flags, void* q, void* sf,
                            hipStream_t stream, const LaunchCaps& caps);

// h [rows, 2*cols] bf16 (gate | up), w [rows] fp32 or null -> 8-bit codes
// (kE4M3 / kE5M2) + scales of silu(gate) * up * w; group in {32, 64, 128};
// cols % group == 0. swiglu_clamp > 0 clamps gate and up first and adds the
// number of changed values to *clamp_count (when not null), through the
// zeroed count workspace count_ws (kCountSlots slots, left zeroed) when that
// is not null, else with one atomic per workgroup of a capped grid.
hipError_t launch_swiglu_per_token(const void* h, int64_t rows, int64_t cols, const float* w,
                                   int fmt, int group, float floor, uint32_t sf_flags,
                                   float swiglu_clamp, unsigned long long* clamp_count,
                                   unsigned long long* count_ws, void* q, void* sf,
                                   hipStream_t stream, const LaunchCaps& caps);

// SwiGLU backward: h [rows, 2*cols] bf16, dv [rows, cols] bf16, w or null
// -> codes of the rows [dgate | dup] (2*cols columns each) + scales in the
// per-token layout sf_flags of those rows; (cols / group) % 4 == 0 for
// kSfPacked.
hipError_t launch_swiglu_backward(const void* h, const void* dv, int64_t rows, int64_t cols,
                                  const float* w, int fmt, int group, float floor,
                                  uint32_t sf_flags, float swiglu_clamp, void* q, void* sf,
                                  hipStream_t stream, const LaunchCaps& caps);

// x [rows, cols] bf16 -> codes + one scale per 128 x 128 block (rounded up
// to a power of two when sf_flags has kSfRound; no other option).
hipError_t launch_per_block(const void* x, int64_t rows, int64_t cols, int fmt, float floor,
                            uint32_t sf_flags, void* q, float* sf, hipStream_t stream,
                            const LaunchCaps& caps);

// x [rows (tokens), cols (channels)] bf16 -> qT [cols, rows] codes + scales
// in the per-token layout sf_flags of x^T (rows = the cols channels, groups
// = the rows/128 token groups); rows % 128 == 0, cols % 8 == 0, and
// (rows / 128) % 4 == 0 for kSfPacked.
hipError_t launch_per_channel_T(const void* x, int64_t rows, int64_t cols, int fmt, float floor,
                                uint32_t sf_flags, void* qT, void* sf, hipStream_t stream,
                                const LaunchCaps& caps);

// The memory traffic of launch_per_channel_T alone (same grid, loads and
// qT stores; meaningless bytes, no scales), for measurement.
hipError_t launch_per_channel_T_traffic(const void* x, int64_t rows, int64_t cols, void* qT,
                                        hipStream_t stream);

// SwiGLU of h [rows, 2*cols] (clamped when swiglu_clamp > 0, changed values
// added to *clamp_count when not null, through count_ws as above), then the
// per-channel cast written transposed: qT [cols, rows], scales as
// launch_per_channel_T writes them.
hipError_t launch_swiglu_per_channel_T(const void* h, int64_t rows, int64_t cols, const float* w,
                                       int fmt, float floor, uint32_t sf_flags,
                                       float swiglu_clamp, unsigned long long* clamp_count,
                                       unsigned long long* count_ws, void* qT, void* sf,
                                       hipStream_t stream, const LaunchCaps& caps);

// x [rows (tokens), cols (channels)] bf16 -> q [rows, cols] 8-bit codes in the
// input layout + sf [rows/128, cols] (rounded up to powers of two with
// kSfRound, the one option); rows % 128 == 0, cols % 8 == 0.
hipError_t launch_per_channel(const void* x, int64_t rows, int64_t cols, int fmt, float floor,
                              uint32_t sf_flags, void* q, float* sf, hipStream_t stream,
                              const LaunchCaps& caps);

// q per-token codes [rows, cols] (or [rows, cols/2] E2M1) + sf [rows, cols/group]
// -> out [rows, cols] bf16 (out_bf16) or fp32: decode(q) * sf.
hipError_t launch_cast_back(const void* q, const float* sf, int64_t rows, int64_t cols, int fmt,
                            int group, bool out_bf16, void* out, hipStream_t stream,
                            const LaunchCaps& caps);

// A per-token cast whose format and group are fixed for a launch.
struct RowCast {
  uint8_t* q;      // codes; null: nothing is cast
  void* sf;        // scales in the layout lay
  SfLayout lay;
  float floor;
  int fmt;         // Fmt
  int shift;       // log2 of the lanes of a group (group = 8 << shift)
};
inline RowCast make_row_cast(int64_t rows, int64_t cols, int fmt, int group, float floor,
                             uint32_t sf_flags, void* q, void* sf) {
  return RowCast{static_cast<uint8_t*>(q), sf, make_sf_layout(rows, cols, group, sf_flags), floor,
                 fmt, group == 32 ? 2 : group == 64 ? 3 : 4};
}

// As launch_swiglu_per_token (without a counter), and the per-token codes of
// h itself in ckpt (8-bit format, same group, row-major scales).
hipError_t launch_swiglu_checkpoint(const void* h, int64_t rows, int64_t cols, const float* w,
                                    int group, float swiglu_clamp, const RowCast& cast,
                                    const RowCast& ckpt, hipStream_t stream);

// What the tile kernels (128 tokens x 128 channels) are called with: one
// transposed cast of 128-token groups, rows padded to whole groups.
struct TileCast {
  uint8_t* qT;     // [channels][rows_T] 8-bit codes; null: not written
  void* sf;
  SfLayout lay;    // rows = channels, groups = rows_T / 128
};
struct SwigluTile {
  const uint8_t* ckpt;       // [rows, 2*cols] codes of (gate | up)
  const float* ckpt_sf;      // [rows, 2*cols / (8 << ckpt_shift)]
  const uint16_t* dv;        // [rows, cols] bf16
  const float* w;            // [rows] or null
  uint8_t* q;                // [rows, 2*cols] codes of [dg | du]
  void* sf;
  SfLayout lay;              // of the rows [dg | du]
  TileCast dh, v;            // transposed [dg | du] and v
  float* dw;                 // [rows] or null
  float* ws;                 // [cols/128][rows] partial sums of dw
  float floor;
  float clamp;               // 0: none
  int ckpt_shift;            // log2(ckpt_group / 8)
  uint32_t rows, cols;
};
hipError_t launch_swiglu_backward_checkpoint(const SwigluTile& p, int ckpt_fmt, int fmt,
                                             hipStream_t stream);

struct RecastTile {
  const uint8_t* q;          // [rows, cols] codes
  const float* sf;           // [rows, cols / (8 << shift)]
  TileCast out;
  float floor;
  int shift;                 // log2(in_group / 8)
  uint32_t rows, cols;
};
hipError_t launch_recast(const RecastTile& p, int in_fmt, int fmt, hipStream_t stream);

// Whether the tile kernels' 32-bit tile counts and in-tile offsets hold for
// rows x cols values read from rows of `stride` elements.
bool tile_fits(int64_t rows, int64_t cols, int64_t stride);

// The norms around a block (norm.hip, norm_backward.hip).
enum GateKind : int { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };
constexpr uint32_t kNormMaxChunks = 2048;      // 16384 columns: 1024 threads x 2 chunks of 8

struct NormForward {
  const uint16_t* y;         // or null
  const uint16_t* h;
  const uint16_t* w_post;    // or null
  const uint16_t* w_pre;
  const void* gate;          // by gate_kind
  uint16_t* h_out;
  uint16_t* x_out;           // or null
  float* rstd_post;          // or null
  float* rstd_pre;           // or null
  RowCast cast, y_ckpt, h_ckpt;
  int gate_kind;
  float alpha, offset, eps;
  float inv_n;               // 1 / cols
  uint32_t chunks;           // cols / 8
};
hipError_t launch_norm(const NormForward& p, int64_t rows, hipStream_t stream,
                       const LaunchCaps& caps);

struct NormBackward {
  const uint16_t* dx;
  const uint16_t* dh_in;     // or null
  const void* saved_h;       // bf16, or 8-bit codes with scales
  const float* saved_h_sf;
  const void* saved_y;       // or null
  const float* saved_y_sf;
  const float* rstd_pre;
  const float* rstd_post;    // null without w_post
  const uint16_t* w_post;    // or null
  const uint16_t* w_pre;
  const void* gate;
  uint16_t* dh_out;
  uint16_t* dy_out;          // or null
  float* sums[3];            // dw_pre, dw_post, dgate of a channel gate; each may be null
  void* dgate;               // of a token or full gate, or null
  float* ws;                 // [parts][2][cols]
  RowCast cast;
  int saved_fmt;             // 0: bf16
  int gate_kind;
  float alpha, offset;
  float inv_n;               // 1 / cols
  uint32_t chunks;
};
// parts: workgroups that walk the rows (at most rows)
hipError_t launch_norm_backward(const NormBackward& p, int64_t rows, uint32_t parts,
                                hipStream_t stream);

// A mixture-of-experts layer's rows (expert_sort.hip, dispatch.hip, combine.hip).
struct ExpertSort {
  const void* ids;           // int32, or int64 when wide
  const float* weight;       // or null, with row_weight
  int32_t* dest;
  int32_t* source;
  int32_t* offsets;
  int32_t* counts;
  float* row_weight;
  int32_t* ws;               // [parts][experts], null for one part
  int64_t first;
  uint32_t slots, rows, experts, align;
  uint32_t part;             // slots of a workgroup
  bool wide;
};
hipError_t launch_expert_sort(const ExpertSort& p, hipStream_t stream);

// Where a token's slots go, and what of the output is padding.
struct ExpertRuns {
  const int32_t* dest;       // [tokens][top_k]
  const int32_t* offsets;    // [experts + 1] or null: no padding
  const int32_t* counts;     // [experts]
  uint32_t tokens, top_k, experts, align, rows;
};

struct DispatchCodes {
  ExpertRuns runs;
  const u32x4* in;
  u32x4* out;
  const uint32_t* sf_in;     // or null
  uint32_t* sf_out;
  uint32_t chunks;           // 16-byte chunks of a row
  uint32_t words;            // scale words of a row
  uint32_t pad_in, pad_out;  // rows of a column-major layout; 0: row-major
};
hipError_t launch_dispatch_codes(const DispatchCodes& p, hipStream_t stream);

// Rows of fp32 weight * x cast per token at their places.
struct DispatchCast {
  ExpertRuns runs;
  const uint16_t* x;         // [tokens, cols]
  const float* weight;       // [tokens, top_k] or null
  const uint16_t* y;         // [rows, cols]; null without dw
  uint16_t* dy;              // [rows, cols] bf16 or null
  float* dw;                 // [tokens, top_k] or null
  RowCast cast;              // q may be null
  uint32_t chunks;           // cols / 8
};
hipError_t launch_dispatch_cast(const DispatchCast& p, hipStream_t stream);
hipError_t launch_combine_backward(const DispatchCast& p, hipStream_t stream);

struct Combine {
  const uint16_t* y;
  const int32_t* dest;       // or null: slot s is row s
  const float* weight;       // or null
  const uint16_t* base;      // or null
  uint16_t* out;
  uint32_t rows, tokens, top_k, chunks;
};
hipError_t launch_combine(const Combine& p, hipStream_t stream);

// out[r][i] = sum_j x[r / per][j] * W[ids[r]][i][j] (matvec.hip).
struct Matvec {
  const void* x;             // bf16, or codes in x_fmt
  const float* x_sf;
  const uint8_t* w;
  const void* w_sf;          // fp32, or packed words
  const void* ids;           // or null
  void* out;
  int64_t experts;
  int x_fmt, x_shift, w_shift;   // groups of 32 << shift
  bool packed, wide, out_bf16;
  uint32_t rows, x_rows, n, k;
};
bool matvec_fits(int64_t rows, int64_t n, int64_t experts, bool ids);
hipError_t launch_matvec(const Matvec& p, hipStream_t stream);

}  // namespace qcast
