// matvec.hip -- products of a few rows with E2M1 weights and group scales.
//
// out[r][i] = sum_g sf[i][g] * (sum_{j in g} code[i][j] * x[r][j]), the inner
// sum over one scale group in the matrix cores (an E2M1 value and an 8-bit
// code are bf16 values: nothing is rounded on the way in), the outer one in
// fp32. A weight is read once for the rows of a pass that share it (up to 16,
// launch_matvec): bound by HBM reads of the weights.
//
// gfx950 design. v_mfma_f32_16x16x32_bf16 with x as A (16 rows) and the
// weights as B (16 columns, which are 16 rows of w): of one step's 32 k, lane
// (n = lane % 16, c = lane / 16) holds k = 8 c .. 8 c + 7 of both. A unit is
// 256 k of the 16 rows: two loads of 8 rows x 128 bytes, a lane 16 bytes (32
// codes) of each. Whole 128-byte lines in one instruction: with 16 rows x 64
// bytes an instruction a bare read of 7168 x 18432 codes takes 15.1 us, so
// 11.3. to_steps() then changes three lane bits with three bits of the
// register's number. Row m of x sits at A's row 4 (m % 4) + m / 4, so that 4 kI
// rows lie in the first kI of a lane's four results.
//
// A wave has a column tile and a share of its k, and asks for two turns of
// weights and scales ahead; scales go through a piece of LDS that is the
// wave's own (a lane that loaded its own row's scale of every step asked for
// each of them four times: 3 us more on that weight). The waves that share a
// tile take its turns in turn and add their sums in a fixed order. x is in LDS
// for the whole workgroup: all of it, or stages of it. Many rows without experts
// bring theirs with the weights instead, through the wave's own LDS, so that no
// wave waits for another. One row of 7168 x 18432 in groups of 32: 19 us (82.6
// MB, 4.3 TB/s); 8 experts' 4096 x 7168 in groups of 128: 26 us (4.8 TB/s); 16
// tokens to 8 of 32 experts of 7168 x 2048, groups of 32: 54 to 60 us (28 experts
// hit, 217 MB, 3.6 to 4.0 TB/s). Every variant spills 43 to 84 scalar registers, a
// third of them, all with 8-bit x, up to 22 vector registers a lane.
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"
#include "qcast_stages.h"

#include <cmath>

namespace qcast {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kUnit = 256;            // k of a unit: 128 bytes of a row of w
constexpr uint32_t kXRow = kUnit * 2 + 16; // a unit's row of x in LDS: 4 banks apart

struct MatvecLaunch {
  Matvec p;
  uint32_t first;        // the first workgroup's number
  uint32_t tiles;        // workgroups along n; with several passes a multiple of 8
  uint32_t n_waves;      // column tiles of a workgroup
  uint32_t k_waves;      // waves that share a column tile
  uint32_t n_loop;       // column tiles that a wave takes one after the other
  uint32_t pass;         // rows that are taken at once
  uint32_t passes;       // workgroups that share the passes of a slot's tiles
  bool few;              // no more than two column tiles for each compute unit
  uint32_t x_lds;        // bytes of LDS for x
  uint32_t slots;        // 0: no ids
  bool by_row;           // a slot is a row (the first of its expert), else an expert
};

// From the chunks that the lanes loaded, w[0] of row lane % 8 and w[1] of the
// row 8 further, chunk lane / 8 each, to the steps' operands: register j holds
// chunk j, dword lane / 16, of row lane % 16. Three lane bits change places with
// three bits of the register's number: the chunk's upper two with the dword's
// (v_permlane32_swap, v_permlane16_swap), its lowest with the row's highest.
__device__ __forceinline__ void to_steps(const u32x4 (&w)[2], uint32_t (&r)[8]) {
  uint32_t x[2][4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    x[h][0] = w[h].x;
    x[h][1] = w[h].y;
    x[h][2] = w[h].z;
    x[h][3] = w[h].w;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto v = __builtin_amdgcn_permlane32_swap(x[h][i], x[h][i + 2], false, false);
      x[h][i] = (uint32_t)v[0];
      x[h][i + 2] = (uint32_t)v[1];
    }
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const auto v = __builtin_amdgcn_permlane16_swap(x[h][i], x[h][i + 1], false, false);
      x[h][i] = (uint32_t)v[0];
      x[h][i + 1] = (uint32_t)v[1];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // lanes 8..15 of a row of 16 take the other's register from 8 lanes away
    r[2 * i] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[0][i], (int)x[1][i], kDppRor8, 0xF,
                                                     0xC, false);
    r[2 * i + 1] = (uint32_t)__builtin_amdgcn_update_dpp((int)x[1][i], (int)x[0][i], kDppRor8,
                                                         0xF, 0x3, false);
  }
}

// Eight E2M1 codes -> eight bf16 (exact).
__device__ __forceinline__ bf16x8 e2m1_bf16(uint32_t w) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// A barrier for LDS alone: loads in flight stay so.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// How x comes: bf16; 8-bit codes with scales of 32 or 64 k (every step of 32 k
// is scaled); or with scales of 128 k (every block of 128 k is).
enum XKind : int { kXPlain = 0, kXStep = 1, kXBlock = 2 };

// A variant: the weights' scale groups (32 << kShift k, fp32 or packed), how x
// comes, how many of its rows a pass takes at most (4 or 16), and where it is:
// all of it in LDS for the workgroup, stages of it there, or with the weights,
// through each wave's own LDS.
enum XPlace : int { kWhole = 0, kStages = 1, kWithW = 2 };
template <int kShift, bool kPacked, int kX, int kR, int kAt>
struct Variant {
  static constexpr bool kOwn = kAt == kWithW;
  static constexpr int kI = kR / 4;                    // results of a lane's four that hold rows
  static constexpr int kUnits = kR == 4 ? 2 : 1;       // units of a turn
  static constexpr int kAhead = kOwn && kX == kXStep ? 1 : 2;    // turns in flight
  static constexpr int kTiles = kOwn ? 2 : 1;          // tiles of 16 columns that share x
  static constexpr int kWaves = kOwn ? 8 : 16;         // most waves of a workgroup
  static constexpr uint32_t kCols = 16 * kTiles;
  static constexpr int kGroups = kUnits * 8 >> kShift; // of a row of w, in a turn
  static constexpr int kPer = kGroups >= 4 ? kGroups / 4 : 1;   // of them, one lane's
  static constexpr int kSteps = kX == kXPlain ? 0 : kX == kXStep ? 8 : 2;  // scales of a unit of x
  static constexpr uint32_t kXUnit = kUnit * 2 + kSteps * 4;   // bytes of a unit of a row of x
  static constexpr uint32_t kSfRow = kGroups * 4 + 16; // a row's scales in LDS
  // a wave's LDS: its scales of w, its x, and its sums of two tiles
  static constexpr uint32_t kXAt = 16 * kTiles * kSfRow;
  static constexpr uint32_t kSums = kXAt + (kOwn ? kR * kXRow : 0);
  static constexpr uint32_t kLds = kSums + 2 * kTiles * kI * 256;

  // What a lane has in flight for one turn.
  struct Turn {
    u32x4 w[kUnits][kTiles][2];          // of rows lane % 8 and 8 more: chunk lane / 8
    uint32_t sf[kTiles][kPer];           // of row lane / 4, as stored (packed: a byte each)
    // its own x: rows lane / 16 + 4 i, and the scales of the rows of its results
    u32x4 x[!kOwn ? 1 : kX == kXPlain ? 2 * kI : kI];
    float xs[kI][kOwn && kX != kXPlain ? kSteps : 1];
  };
};

// Where a wave reads. The rows of a column tile are buffers: an offset past
// their end (a row past n, a unit past the last whole one) loads zeros, so that
// the loads ahead need no branch and the compiler waits for no more than it
// must.
constexpr uint32_t kPastEnd = 0x80000000u;
struct Places {
  RowBuffer w, sf;
  uint32_t w_at, w_half, sf_at, sf_tile;
  uint32_t end;                          // whole units
};
// Where its own x is.
template <int kI>
struct OwnRows {
  const uint8_t* x[kI];
  const float* s[kI];
};

template <typename V, int kShift, bool kPacked>
__device__ __forceinline__ void load_turn(typename V::Turn& t, const Places& r,
                                            uint32_t unit) {
#pragma unroll
  for (int p = 0; p < V::kUnits; ++p) {
    const uint32_t at = r.w_at + (unit + p < r.end ? (unit + p) * (kUnit / 2) : kPastEnd);
#pragma unroll
    for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        t.w[p][t2][h] = __builtin_amdgcn_raw_buffer_load_b128(
            r.w, at + (2 * t2 + h) * r.w_half, 0, kNonTemporal);
  }
  constexpr int kSize = kPacked ? 1 : 4;
#pragma unroll
  for (int t2 = 0; t2 < V::kTiles; ++t2) {
    const uint32_t at = r.sf_at + t2 * r.sf_tile +
                        (unit < r.end ? unit * (8 >> kShift) * kSize : kPastEnd);
    if constexpr (V::kPer * kSize == 16) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r.sf, at, 0, 0);
      t.sf[t2][0] = v.x;
      t.sf[t2][1] = v.y;
      t.sf[t2][2] = v.z;
      t.sf[t2][3] = v.w;
    } else if constexpr (V::kPer * kSize == 8) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r.sf, at, 0, 0);
      t.sf[t2][0] = v.x;
      t.sf[t2][1] = v.y;
    } else if constexpr (V::kPer * kSize == 4) {
      t.sf[t2][0] = __builtin_amdgcn_raw_buffer_load_b32(r.sf, at, 0, 0);
    } else if constexpr (V::kPer * kSize == 2) {
      t.sf[t2][0] = __builtin_amdgcn_raw_buffer_load_b16(r.sf, at, 0, 0);
    } else {
      t.sf[t2][0] = __builtin_amdgcn_raw_buffer_load_b8(r.sf, at, 0, 0);
    }
  }
}

// The unit that k ends in, as the first unit of a turn: zeros past k.
template <typename V, int kShift, bool kPacked>
__device__ __forceinline__ void load_tail(typename V::Turn& t, const Places& r,
                                            uint32_t k) {
  const uint32_t lane = threadIdx.x & 63;
  const uint32_t unit = k / kUnit, k0 = unit * kUnit;
#pragma unroll
  for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      t.w[0][t2][h] = __builtin_amdgcn_raw_buffer_load_b128(
          r.w, k0 + (lane >> 3) * 32 < k
                   ? r.w_at + unit * (kUnit / 2) + (2 * t2 + h) * r.w_half : kPastEnd, 0, 0);
  constexpr int kSize = kPacked ? 1 : 4;
  constexpr int kParts = V::kGroups / V::kPer;         // lanes that have a row's groups
#pragma unroll
  for (int t2 = 0; t2 < V::kTiles; ++t2) {
    uint32_t word = 0;
#pragma unroll
    for (int g = 0; g < V::kPer; ++g) {
      const uint32_t j = (lane & (kParts - 1)) * V::kPer + g;    // the group, in the turn
      const bool in = j < (8 >> kShift) && k0 + (j << kShift) * 32 < k;
      const uint32_t at =
          in ? r.sf_at + t2 * r.sf_tile + (unit * (8 >> kShift) + g) * kSize : kPastEnd;
      if constexpr (kPacked)
        word |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(r.sf, at, 0, 0) << (8 * g);
      else
        t.sf[t2][g] = __builtin_amdgcn_raw_buffer_load_b32(r.sf, at, 0, 0);
    }
    if constexpr (kPacked) t.sf[t2][0] = word;
  }
}

// Eight 8-bit codes -> eight bf16 (exact).
__device__ __forceinline__ u32x4 codes_bf16(uint32_t a, uint32_t b, int fmt) {
  float v[8];
  if (fmt == kE4M3) {
    decode4<kE4M3>(a, v);
    decode4<kE4M3>(b, v + 4);
  } else {
    decode4<kE5M2>(a, v);
    decode4<kE5M2>(b, v + 4);
  }
  return pack8_bf16(v);
}

// A turn's own x (one unit). One past the last whole unit reads the rows' first
// bytes, and is not used.
template <typename V, int kX>
__device__ __forceinline__ void load_own_x(typename V::Turn& t, const OwnRows<V::kI>& r,
                                           uint32_t unit, uint32_t full, uint32_t shift) {
  const uint32_t lane = threadIdx.x & 15;
  const bool in = unit < full;
  const uint32_t at = in ? unit * (kX == kXPlain ? kUnit * 2 : kUnit) + lane * 16 : 0;
#pragma unroll
  for (int i = 0; i < V::kI; ++i) {
    if constexpr (kX == kXPlain) {
      t.x[2 * i] = *reinterpret_cast<const u32x4*>(r.x[i] + at);
      t.x[2 * i + 1] = *reinterpret_cast<const u32x4*>(r.x[i] + at + (in ? 256 : 0));
    } else {
      t.x[i] = *reinterpret_cast<const u32x4*>(r.x[i] + at);
#pragma unroll
      for (int g = 0; g < V::kSteps; ++g) {
        // scales of 128 k, or of 32 << shift k
        const uint32_t j = kX == kXBlock ? unit * 2 + g : (unit * 8 + g) >> shift;
        t.xs[i][g] = r.s[i][in ? j : 0];
      }
    }
  }
}

// The same of the unit that k ends in: zeros past k.
template <typename V, int kX>
__device__ __forceinline__ void load_own_tail(typename V::Turn& t, const OwnRows<V::kI>& r,
                                              uint32_t k, uint32_t shift) {
  const uint32_t lane = threadIdx.x & 15, k0 = k / kUnit * kUnit;
#pragma unroll
  for (int i = 0; i < V::kI; ++i) {
    if constexpr (kX == kXPlain) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t at = k0 + h * 128 + lane * 8;
        t.x[2 * i + h] = u32x4{0, 0, 0, 0};
        if (at < k) t.x[2 * i + h] = *reinterpret_cast<const u32x4*>(r.x[i] + at * 2);
      }
    } else {
      t.x[i] = u32x4{0, 0, 0, 0};
      if (k0 + lane * 16 < k) t.x[i] = *reinterpret_cast<const u32x4*>(r.x[i] + k0 + lane * 16);
#pragma unroll
      for (int g = 0; g < V::kSteps; ++g) {
        const uint32_t at = k0 + g * (kX == kXBlock ? 128 : 32);
        t.xs[i][g] = at < k ? r.s[i][at / 32 >> (kX == kXBlock ? 2 : shift)] : 0.0f;
      }
    }
  }
}

// The fp32 of a UE8M0 byte: 2^(b - 127), subnormal for 0, and NaN for 255. The
// conversions' scale is the exponent field of an fp32, read so: one times it.
__device__ __forceinline__ uint32_t e8m0(uint32_t b) {
  constexpr int kOne = 0x38;             // E4M3
  return __float_as_uint(
      __builtin_amdgcn_cvt_scalef32_f32_fp8(kOne, __uint_as_float(b << 23), 0));
}

// The turn's scales of w to the wave's LDS, as fp32.
template <typename V, bool kPacked>
__device__ __forceinline__ void store_scales(const typename V::Turn& t, uint8_t* mine) {
  const uint32_t lane = threadIdx.x & 63;
  constexpr int kParts = V::kGroups / V::kPer;
#pragma unroll
  for (int t2 = 0; t2 < V::kTiles; ++t2) {
    uint8_t* to =
        mine + (t2 * 16 + (lane >> 2)) * V::kSfRow + (lane & (kParts - 1)) * V::kPer * 4;
    uint32_t f[V::kPer];
#pragma unroll
    for (int g = 0; g < V::kPer; ++g)
      f[g] = kPacked ? e8m0(t.sf[t2][0] >> (8 * g) & 0xffu) : t.sf[t2][g];
    if constexpr (V::kPer == 4) *reinterpret_cast<u32x4*>(to) = u32x4{f[0], f[1], f[2], f[3]};
    else if constexpr (V::kPer == 2) *reinterpret_cast<u32x2*>(to) = u32x2{f[0], f[1]};
    else *reinterpret_cast<uint32_t*>(to) = f[0];
  }
}

// The turn's own x to the wave's LDS, as bf16.
template <typename V, int kX>
__device__ __forceinline__ void store_own_x(const typename V::Turn& t, uint8_t* mine, int fmt) {
  const uint32_t lane = threadIdx.x & 63;
  uint8_t* to = mine + V::kXAt + (lane >> 4) * kXRow + (lane & 15) * (kX == kXPlain ? 16 : 32);
#pragma unroll
  for (int i = 0; i < V::kI; ++i) {
    if constexpr (kX == kXPlain) {
      *reinterpret_cast<u32x4*>(to + i * 4 * kXRow) = t.x[2 * i];
      *reinterpret_cast<u32x4*>(to + i * 4 * kXRow + 256) = t.x[2 * i + 1];
    } else {
      *reinterpret_cast<u32x4*>(to + i * 4 * kXRow) = codes_bf16(t.x[i].x, t.x[i].y, fmt);
      *reinterpret_cast<u32x4*>(to + i * 4 * kXRow + 16) = codes_bf16(t.x[i].z, t.x[i].w, fmt);
    }
  }
}

// Units [u0, u0 + units) of x of the pass's cnt rows (row m in lane m of list),
// as bf16, rows of `stride` bytes, zeros past k; and their scales, V::kSteps of
// a unit, to rows of s_stride. Four loads in flight.
template <typename V, int kX>
__device__ __forceinline__ void stage_x(const Matvec& p, uint8_t* lds, float* scales,
                                        uint32_t list, uint32_t cnt, uint32_t per, uint32_t u0,
                                        uint32_t units, uint32_t stride, uint32_t s_stride) {
  const uint32_t chunks = units * (kUnit / 8), all = cnt * chunks;
  constexpr int kBatch = 4;
  for (uint32_t i0 = threadIdx.x; i0 - (threadIdx.x & 63) < all; i0 += kBatch * blockDim.x) {
    u32x4 v[kBatch];
    float sx[kBatch];
    uint32_t m[kBatch], j[kBatch];
#pragma unroll
    for (int a = 0; a < kBatch; ++a) {
      const uint32_t i = i0 + a * blockDim.x;
      m[a] = i < all ? i / chunks : 0;
      j[a] = i - m[a] * chunks;
      const uint64_t x_row = (uint32_t)__shfl((int)list, (int)m[a]) / per;
      const uint32_t at = u0 * kUnit + j[a] * 8;
      v[a] = u32x4{0, 0, 0, 0};
      sx[a] = 0.0f;
      if (i < all && at < p.k) {
        if constexpr (kX == kXPlain) {
          v[a] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) +
                                                 x_row * p.k + at);
        } else {
          const u32x2 q = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.x) +
                                                          x_row * p.k + at);
          v[a].x = q.x;
          v[a].y = q.y;
          sx[a] = p.x_sf[x_row * (p.k / 32 >> p.x_shift) + (at / 32 >> p.x_shift)];
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kBatch; ++a) {
      if (i0 + a * blockDim.x < all) {
        if constexpr (kX != kXPlain) {
          constexpr uint32_t kOf = kUnit / 8 / V::kSteps;      // chunks of a scale
          v[a] = codes_bf16(v[a].x, v[a].y, p.x_fmt);
          if (j[a] % kOf == 0) scales[m[a] * s_stride + j[a] / kOf] = sx[a];
        }
        *reinterpret_cast<u32x4*>(lds + m[a] * stride + j[a] * 16) = v[a];
      }
    }
  }
}

template <int kShift, bool kPacked, int kX, int kR, int kAt>
__global__ __launch_bounds__((kAt == kWithW ? 512 : 1024)) void matvec_kernel(MatvecLaunch l) {
  using V = Variant<kShift, kPacked, kX, kR, kAt>;
  constexpr bool kOwn = V::kOwn;
  constexpr int kI = V::kI;
  const Matvec& p = l.p;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];    // the waves', then x
  const uint32_t lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t wn = wave / l.k_waves, wk = wave - wn * l.k_waves;
  // the passes of the same tiles are 8 workgroups apart: on one XCD, whose L2
  // they find the weights in
  const uint32_t group = blockIdx.x + l.first, slot = group / (l.tiles * l.passes);
  const uint32_t b = group - slot * (l.tiles * l.passes);
  const uint32_t b8 = b / 8, pass0 = b8 % l.passes;
  const uint32_t tile0 = ((b8 / l.passes * 8 + b % 8) * l.n_waves + wn) * l.n_loop;

  auto id_of = [&](uint32_t r) {
    const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[r]
                              : (int64_t)static_cast<const int32_t*>(p.ids)[r];
    return (uint64_t)id < (uint64_t)p.experts ? (int32_t)id : -1;
  };
  int32_t expert = 0;
  if (l.slots) expert = l.by_row ? id_of(slot) : slot < p.experts ? (int32_t)slot : -1;
  expert = __builtin_amdgcn_readfirstlane(expert);
  const bool none = expert < 0;                // the slot of rows that have no expert

  const uint32_t w_row = p.k / 2, sf_row = (p.k / (32 << kShift)) * (kPacked ? 1 : 4);
  Places at;
  at.w_at = (lane & 7) * w_row + (lane >> 3) * 16;
  at.w_half = 8 * w_row;
  at.sf_tile = 16 * sf_row;
  constexpr int kParts = V::kGroups / V::kPer;
  at.sf_at = (lane >> 2) * sf_row + (lane & (kParts - 1)) * V::kPer * (kPacked ? 1 : 4);
  at.end = none ? 0 : p.k / kUnit;
  auto to_tile = [&](Places& to, uint32_t tile) {
    const uint32_t held =
        tile * V::kCols >= p.n ? 0 : p.n - tile * V::kCols < V::kCols ? p.n - tile * V::kCols : V::kCols;
    const uint64_t row0 = held && !none ? (uint64_t)expert * p.n + tile * V::kCols : 0;
    to.w = row_buffer(p.w, row0 * w_row, held * w_row);
    to.sf = row_buffer(p.w_sf, row0 * sf_row, held * sf_row);
  };
  // this wave's turns of a tile (wk, wk + k_waves, ...), and in all its tiles;
  // with stages there is one tile
  const uint32_t full = at.end;
  const uint32_t all_turns = (full + V::kUnits - 1) / V::kUnits;
  const uint32_t turns = wk < all_turns ? (all_turns - wk - 1) / l.k_waves + 1 : 0;
  const uint32_t items = turns * l.n_loop;
  const bool ends = !none && p.k % kUnit != 0 && wk == l.k_waves - 1;
  const uint32_t per = p.rows / p.x_rows;     // rows of a row of x, with ids or without
  uint8_t* const mine = lds + wave * V::kLds;
  uint8_t* const x_lds = lds + l.n_waves * l.k_waves * V::kLds;
  const uint8_t* const sa = mine + n * V::kSfRow;
  // A's row n is row m; rows that there are not give results that nobody reads
  const uint32_t m_of_lane = (n >> 2) + 4 * ((n & 3) % kI);

  // the ring; the next turn that it asks for is `ahead` of tile `ahead_tile`
  typename V::Turn ring[V::kAhead];
  OwnRows<kI> own;
  uint32_t ahead = wk, ahead_tile = tile0;
  auto next = [&]() {
    ahead += l.k_waves;
    if (ahead >= all_turns) {
      ahead = wk;
      ++ahead_tile;
      to_tile(at, ahead_tile < tile0 + l.n_loop ? ahead_tile : 0x7ffffffu);
    }
  };
  auto begin = [&]() {
    ahead = wk;
    ahead_tile = tile0;
    to_tile(at, tile0);
#pragma unroll
    for (int a = 0; a < V::kAhead; ++a) {
      load_turn<V, kShift, kPacked>(ring[a], at, ahead * V::kUnits);
      if constexpr (kOwn) load_own_x<V, kX>(ring[a], own, ahead * V::kUnits, full, p.x_shift);
      next();
    }
  };
  // without its own x the first weights are asked for before it is known whose
  // rows they meet
  if (!kOwn && items && pass0 == 0) begin();
  uint32_t from = 0, before = 0;               // ids that are read, their rows of this expert
  for (uint32_t first = pass0 * l.pass;; first += l.passes * l.pass) {
    // the rows of this pass: those with the slot's expert, l.pass at a time; lane
    // m holds the m-th. The next pass goes on with the last 64 ids of this one.
    uint32_t cnt = 0, list = 0;
    if (l.slots) {
      uint32_t seen = before;
      bool leads = true;
      for (uint32_t r0 = from; r0 < p.rows && seen < first + l.pass; r0 += 64) {
        from = r0;
        before = seen;
        const uint32_t r = r0 + lane;
        bool same = false;
        if (r < p.rows) same = none && l.by_row ? r == slot : id_of(r) == expert;
        const uint64_t set = __builtin_amdgcn_ballot_w64(same);
        if (l.by_row && seen == 0 && set != 0)
          leads = r0 + (uint32_t)__builtin_ctzll(set) == slot;
        const uint32_t rank =
            seen + (uint32_t)__builtin_popcountll(set & ((1ull << lane) - 1)) - first;
        const uint32_t had = seen - first;     // below zero before the pass begins
        seen += (uint32_t)__builtin_popcountll(set);
        const uint32_t to = same && rank < l.pass ? rank : 63;
        const uint32_t got = (uint32_t)__builtin_amdgcn_ds_permute((int)(to * 4), (int)r);
        if (lane < l.pass && (int32_t)(lane - had) >= 0 && (int32_t)(seen - first - lane) > 0)
          list = got;
      }
      if (!leads) return;                      // an earlier row's slot has this expert
      if (seen <= first) return;
      cnt = seen - first < l.pass ? seen - first : l.pass;
    } else {
      if (p.rows <= first) return;
      cnt = p.rows - first < l.pass ? p.rows - first : l.pass;
      list = first + lane;
    }
    uint32_t row[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i)
      row[i] = (uint32_t)__shfl((int)list, c + 4 * i < cnt ? (int)(c + 4 * i) : 0);

    if constexpr (kOwn) {
#pragma unroll
      for (int i = 0; i < kI; ++i) {
        const uint64_t x_row = row[i] / per;
        own.x[i] = static_cast<const uint8_t*>(p.x) + x_row * p.k * (kX == kXPlain ? 2 : 1);
        own.s[i] = p.x_sf + (kX == kXPlain ? 0 : x_row * (p.k / 32 >> p.x_shift));
      }
    }

    // x in LDS: all of it, or stages of as many units as fit, in whole rounds of
    // the waves' rings (the launch sees to it that one fits)
    const uint32_t units = none ? 0 : (p.k + kUnit - 1) / kUnit;
    uint32_t stage = units;
    if constexpr (kAt == kStages)
      stage = stage_units(l.x_lds, cnt, V::kXUnit, l.k_waves * V::kUnits * V::kAhead, units);
    const uint32_t stride = kOwn ? kXRow : stage * (kUnit * 2) + 16, s_stride = stage * V::kSteps;
    float* const scales = reinterpret_cast<float*>(x_lds + cnt * stride);
    const uint8_t* const xa = (kOwn ? mine + V::kXAt : x_lds) +
                              (kOwn || m_of_lane < cnt ? m_of_lane : 0) * stride + c * 16;
    const float* xs[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i) xs[i] = scales + (c + 4 * i < cnt ? c + 4 * i : 0) * s_stride;
    uint32_t u0 = 0;                           // the first unit there now

    float acc[V::kTiles][kI];
#pragma unroll
    for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
      for (int i = 0; i < kI; ++i) acc[t2][i] = 0.0f;
    // the units of a turn, `unit` on, that lie before `end`
    auto add_turn = [&](const typename V::Turn& t, uint32_t unit, uint32_t end) {
      store_scales<V, kPacked>(t, mine);
      if constexpr (kOwn) store_own_x<V, kX>(t, mine, p.x_fmt);
      wave_order();
#pragma unroll
      for (int u = 0; u < V::kUnits; ++u) {
        if (u > 0 && unit + u >= end) break;
        constexpr int kOfUnit = 8 >> kShift;
        const uint32_t here = unit + u - (kAt == kStages ? u0 : 0);
        uint32_t r[V::kTiles][8];
#pragma unroll
        for (int t2 = 0; t2 < V::kTiles; ++t2) to_steps(t.w[u][t2], r[t2]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bf16x8 a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                                  xa + (kOwn ? 0 : here * (kUnit * 2)) +
                                                  h * 256 + j * 64));
          constexpr int kHalf = kX == kXStep ? 4 : 1;
          float f_x[kI][kHalf];
          if constexpr (kX != kXPlain) {
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
              for (int g = 0; g < kHalf; ++g)
                f_x[i][g] = kOwn ? t.xs[i][kOwn ? h * kHalf + g : 0]
                                 : xs[i][here * V::kSteps + h * kHalf + g];
          }
          float s[V::kTiles][4 >> kShift];
#pragma unroll
          for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
            for (int g = 0; g < (4 >> kShift); ++g)
              s[t2][g] = reinterpret_cast<const float*>(sa + t2 * 16 * V::kSfRow)[
                  u * kOfUnit + h * (4 >> kShift) + g];
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int t2 = 0; t2 < V::kTiles; ++t2) {
            f32x4 d;
            float block[kI];
#pragma unroll
            for (int i = 0; i < kI; ++i) block[i] = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              constexpr int kSteps = kX == kXStep ? 1 : 1 << kShift;     // between scalings
              d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  a[j], e2m1_bf16(r[t2][h * 4 + j]), j % kSteps == 0 ? f32x4{0, 0, 0, 0} : d, 0,
                  0, 0);
              if (j % kSteps == kSteps - 1) {
                const float f = s[t2][j >> kShift];
#pragma unroll
                for (int i = 0; i < kI; ++i) {
                  if constexpr (kX == kXPlain) {
                    acc[t2][i] = __builtin_fmaf(d[i], f, acc[t2][i]);
                  } else if constexpr (kX == kXStep) {
                    acc[t2][i] = __builtin_fmaf(d[i], f * f_x[i][j], acc[t2][i]);
                  } else {
                    block[i] = __builtin_fmaf(d[i], f, block[i]);
                    if (j == 3) acc[t2][i] = __builtin_fmaf(block[i], f_x[i][0], acc[t2][i]);
                  }
                }
              }
            }
          }
        }
      }
      wave_order();
    };
    // a tile's sums: what is left of k, the other waves' sums in their order, and
    // the output. One barrier: the next tile's sums go to the other half.
    uint32_t tile = tile0;
    auto flush = [&]() {
      if (ends) {
        Places last = at;
        to_tile(last, tile);
        typename V::Turn t;
        load_tail<V, kShift, kPacked>(t, last, p.k);
        if constexpr (kOwn) load_own_tail<V, kX>(t, own, p.k, p.x_shift);
        add_turn(t, full, full + 1);
      }
      const uint32_t half = (tile - tile0) & 1;
      if (l.k_waves > 1) {
        if (wk) {
#pragma unroll
          for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
            for (int i = 0; i < kI; ++i)
              reinterpret_cast<float*>(mine + V::kSums)[((half * V::kTiles + t2) * kI + i) * 64 +
                                                        lane] = acc[t2][i];
        }
        lds_barrier();
      }
      if (wk == 0) {
        for (uint32_t k = 1; k < l.k_waves; ++k) {
#pragma unroll
          for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
            for (int i = 0; i < kI; ++i)
              acc[t2][i] = acc[t2][i] +
                           reinterpret_cast<const float*>(mine + k * V::kLds + V::kSums)[
                               ((half * V::kTiles + t2) * kI + i) * 64 + lane];
        }
#pragma unroll
        for (int t2 = 0; t2 < V::kTiles; ++t2) {
          const uint32_t col = tile * V::kCols + t2 * 16 + n;
#pragma unroll
          for (int i = 0; i < kI; ++i) {
            if (col < p.n && c + 4 * i < cnt) {
              const uint64_t to = (uint64_t)row[i] * p.n + col;
              if (p.out_bf16)
                static_cast<uint16_t*>(p.out)[to] = (uint16_t)pack_bf16(acc[t2][i], 0.0f);
              else
                static_cast<float*>(p.out)[to] = acc[t2][i];
            }
          }
        }
      }
#pragma unroll
      for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
        for (int i = 0; i < kI; ++i) acc[t2][i] = 0.0f;
      ++tile;
    };
    if (items && (kOwn || first)) begin();
    // a turn, and the one that takes its place in the ring; places are fixed, so
    // that nothing waits for a load but its use
    uint32_t turn = wk;
    auto refill = [&](typename V::Turn& t) {
      load_turn<V, kShift, kPacked>(t, at, ahead * V::kUnits);
      if constexpr (kOwn) load_own_x<V, kX>(t, own, ahead * V::kUnits, full, p.x_shift);
      next();
    };
    if constexpr (kAt == kStages) {
      for (uint32_t held = 0; u0 < units; u0 += held) {
        held = units - u0 < stage ? units - u0 : stage;
        if (u0) lds_barrier();                 // the last units have been read
        stage_x<V, kX>(p, x_lds, scales, list, cnt, per, u0, held, stride, s_stride);
        lds_barrier();
        const uint32_t end = u0 + held < units ? (u0 + held) / V::kUnits : all_turns;
        while (turn < end) {
#pragma unroll
          for (int a = 0; a < V::kAhead; ++a) {
            if (turn < end) {
              add_turn(ring[a], turn * V::kUnits, full);
              turn += l.k_waves;
            }
            refill(ring[a]);
          }
        }
      }
      u0 = units ? (units - 1) / stage * stage : 0;        // the last stage is still there
      flush();
    } else {
      if constexpr (kAt == kWhole) {
        if (units) stage_x<V, kX>(p, x_lds, scales, list, cnt, per, 0, units, stride, s_stride);
        lds_barrier();
      }
      for (uint32_t q = 0; q < items; q += V::kAhead) {
#pragma unroll
        for (int a = 0; a < V::kAhead; ++a) {
          if (q + a < items) {
            add_turn(ring[a], turn * V::kUnits, full);
            turn += l.k_waves;
            if (turn >= all_turns) {
              flush();
              turn = wk;
            }
          }
          refill(ring[a]);
        }
      }
      if (!items)
        for (uint32_t t = 0; t < l.n_loop; ++t) flush();
    }
    __syncthreads();                           // LDS has been read
  }
}

// The launch shapes, and with them the order of the sums, are those of a whole
// card, whatever the partition or qcast_set_num_cus.
constexpr uint32_t kCus = 256;

// LDS for the whole of x at most, and for a stage of it; with few tiles, for
// either: more waves can share one then (44 rows to 2 of 4 experts of 3697 x
// 14592: 42 us, 51 with stages of 48 KB).
constexpr uint32_t kWholeBytes = 72 * 1024, kStageBytes = 48 * 1024, kFewBytes = 112 * 1024;

// Experts that the rows hit, were the choice even and a row of x's all different.
double live_experts(const Matvec& p) {
  if (p.experts == 0 || p.x_rows == 0) return 0;
  const double per = (double)(p.rows / p.x_rows) / p.experts;
  return p.experts * (1 - std::pow(per < 1 ? 1 - per : 0, (double)p.x_rows));
}

// LDS that all of x of a pass takes; `steps` scales of a unit.
uint64_t x_bytes(const MatvecLaunch& l, uint32_t steps) {
  const uint32_t units = (l.p.k + kUnit - 1) / kUnit;
  return (uint64_t)l.pass * (units * (kUnit * 2 + steps * 4) + 16);
}

template <int kShift, bool kPacked, int kX, int kR, int kAt>
hipError_t launch_variant(MatvecLaunch l, hipStream_t stream) {
  using V = Variant<kShift, kPacked, kX, kR, kAt>;
  const uint32_t units = (l.p.k + kUnit - 1) / kUnit;
  const uint32_t tiles = (l.p.n + V::kCols - 1) / V::kCols;
  const uint32_t slots = l.slots ? l.slots : 1;
  const uint64_t work = (uint64_t)tiles * slots * l.passes;
  // x and 8 waves take more than half of LDS: a compute unit has one workgroup
  const uint64_t whole = x_bytes(l, V::kSteps);
  l.x_lds = kAt == kWithW ? 0 : kAt == kWhole ? (uint32_t)whole : l.few ? kFewBytes : kStageBytes;
  const bool alone = kAt != kWithW && l.x_lds + 8 * V::kLds > 80 * 1024;
  // Waves that share a tile: until there are 6 waves for each of 256 compute
  // units, of four units of k or more (one row of 7168 x 18432: 45 us with two,
  // 18 with four, 18.5 with eight). Two at least, in stages (8 tokens to 8 of 32
  // experts of 4096 x 7168: 80 us, 82 with one, 99 with four) but for the
  // largest calls (64 tokens to 8 of 256: 520 with one, 634 with two); with up
  // to four rows of 4096 k or more (32 to 8 of 256 of 2048 x 7168: 210, 224 with
  // one; but 4 to 8 of 32 of 7168 x 2048, 43 with one and 49 with two); and in a
  // workgroup alone on its compute unit (16 to 8 of 32 of 7168 x 2048: 53, 56).
  const bool two = kAt == kStages ? work < kCus * 64
                   : kAt == kWithW ? false
                   : kR == 4       ? units >= 16
                                   : alone && units >= 8;
  l.k_waves = two ? 2 : 1;
  while (l.k_waves < V::kWaves && l.k_waves * 4 <= units && work * l.k_waves < kCus * 6)
    l.k_waves *= 2;
  if constexpr (kAt == kStages) {
    // A stage holds one round of the rings at least (16 rows of one wave's two
    // units, with 8 scales each, take 17 KB). One of no units would never end.
    constexpr uint32_t kOfWave = V::kUnits * V::kAhead;
    static_assert(stage_units(kStageBytes, kR, V::kXUnit, kOfWave, ~0u) > 0, "a wave's round");
    l.k_waves = stage_waves(l.x_lds, l.pass, V::kXUnit, kOfWave, l.k_waves);
    if (units && stage_units(l.x_lds, l.pass, V::kXUnit, l.k_waves * kOfWave, units) == 0)
      return hipErrorInvalidValue;
  }
  // Workgroups of up to 8 waves (16 if alone), and how many column tiles a wave
  // takes one after the other with x where it is: the least time of the compute
  // unit with the most workgroups, in times of a unit of k of a tile (0.1 us).
  // Their work adds up; starts (5 us: ids, x, the first weights) are waited for
  // once for all that are there together. 16 tokens to 8 of 32 experts of 7168 x
  // 2048: 87 us with one tile, 74 with two, 64 with four, 53 with seven, 60 with
  // eight; a token's 4 of 9216 x 7168: 39 with 2 x 4 waves and two tiles, 30 with
  // 2 x 2 and one. With passes of four two tiles at most: more make an expert
  // with many rows a long tail (32 tokens to 8 of 256: 210 with two, 259 with four).
  uint32_t most = (alone ? 16 : kAt == kWithW ? 4 : 8) / l.k_waves;
  while (most > 1 && most > tiles) most /= 2;
  if (most == 0) most = 1;
  const uint32_t loops = kAt != kWhole ? 1 : kR == 4 ? 2 : 8;
  const double live = l.slots ? live_experts(l.p) : l.passes;
  constexpr double kStart = 53;
  double least = 1e300;
  for (uint32_t n = most; n == most || (n > 0 && n * l.k_waves >= 4); n /= 2) {
    const uint32_t waves = n * l.k_waves, room = 160 * 1024 / (l.x_lds + waves * V::kLds);
    const uint32_t together = waves >= 16 || room < 2 ? 1 : room < 16 / waves ? room : 16 / waves;
    for (uint32_t loop = 1; loop <= loops; ++loop) {
      const double groups = (double)((tiles + n * loop - 1) / (n * loop)) * live;
      const double each = std::ceil(groups / kCus);
      const double cost = each * n * loop * units * V::kTiles + std::ceil(each / together) * kStart;
      if (cost < least) least = cost, l.n_waves = n, l.n_loop = loop;
    }
  }
  l.tiles = (tiles + l.n_waves * l.n_loop - 1) / (l.n_waves * l.n_loop);
  if (l.passes > 1) l.tiles = (l.tiles + 7) / 8 * 8;
  const uint64_t groups = (uint64_t)l.tiles * slots * l.passes;
  const uint32_t waves = l.n_waves * l.k_waves;
  if (groups >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  static_assert(16 * Variant<0, false, kXStep, 16, kWhole>::kLds + kFewBytes <= 160 * 1024 &&
                    8 * Variant<0, false, kXStep, 16, kWithW>::kLds <= 160 * 1024,
                "LDS");
  return each_launch(groups, waves * 64, [&](uint32_t first, uint32_t n) {
    l.first = first;
    launch_kernel(matvec_kernel<kShift, kPacked, kX, kR, kAt>, dim3(n), dim3(waves * 64),
                  waves * V::kLds + l.x_lds, stream, l);
  });
}

// Where x is. Whole up to 72 KB (5 rows of 16384 x 5120: 14 us, 19 with the
// weights; 16 tokens to 8 of 32 experts of 7168 x 2048: 54 to 60, 82 to 90 in
// stages). Past
// that the rows of an expert come in stages (8 tokens to 8 of 32 experts of
// 4096 x 7168: 80 us, 109 with the weights), and so do up to four rows without
// experts; more of those, whose workgroups would each stage all of x for few
// tiles, with the weights (16 rows of 7168 x 18432: 28 us, 37 in stages).
template <int kShift, bool kPacked, int kX>
hipError_t launch_rows(const MatvecLaunch& l, hipStream_t stream) {
  const bool whole = x_bytes(l, Variant<kShift, kPacked, kX, 16, kWhole>::kSteps) <=
                     (l.few ? kFewBytes : kWholeBytes);
  if (l.pass <= 4)
    return whole ? launch_variant<kShift, kPacked, kX, 4, kWhole>(l, stream)
                 : launch_variant<kShift, kPacked, kX, 4, kStages>(l, stream);
  return whole     ? launch_variant<kShift, kPacked, kX, 16, kWhole>(l, stream)
         : l.slots ? launch_variant<kShift, kPacked, kX, 16, kStages>(l, stream)
                   : launch_variant<kShift, kPacked, kX, 16, kWithW>(l, stream);
}

template <int kShift, bool kPacked>
hipError_t launch_x(const MatvecLaunch& l, hipStream_t stream) {
  return !l.p.x_fmt         ? launch_rows<kShift, kPacked, kXPlain>(l, stream)
         : l.p.x_shift == 2 ? launch_rows<kShift, kPacked, kXBlock>(l, stream)
                            : launch_rows<kShift, kPacked, kXStep>(l, stream);
}

template <int kShift>
hipError_t launch_s(const MatvecLaunch& l, hipStream_t stream) {
  return l.p.packed ? launch_x<kShift, true>(l, stream) : launch_x<kShift, false>(l, stream);
}

int64_t slots_of(int64_t rows, int64_t experts, bool ids) {
  return !ids ? 0 : rows <= experts ? rows : experts + 1;
}

}  // namespace

bool matvec_fits(int64_t rows, int64_t n, int64_t experts, bool ids) {
  const int64_t slots = slots_of(rows, experts, ids);
  return (slots == 0 || (n + 15) / 16 < (int64_t(1) << 31) / slots) &&
         (n == 0 || rows < (int64_t(1) << 40) / n);
}

// Shapes follow from the sizes alone, and so does the order of the sums.
hipError_t launch_matvec(const Matvec& p, hipStream_t stream) {
  if (p.rows == 0 || p.n == 0) return hipSuccess;
  MatvecLaunch l{};
  l.p = p;
  l.slots = (uint32_t)slots_of(p.rows, p.experts, p.ids != nullptr);
  l.by_row = l.slots == p.rows && (int64_t)p.rows <= p.experts;
  // Rows that one reading of a weight serves: all of them up to 16; of an expert
  // one with one row of x (a token's experts are different ones), four up to a row
  // for each expert (8 rows to 32 experts of 7168 x 2048: 17 us, 28 with passes of
  // one; 2 tokens to 8 of 32 of 4096 x 7168: 42 us, 45 with 16; 4 to 8 of 32 of
  // 7168 x 2048 with e4m3: 43 and 48; 32 to 8 of 256: 210 and 207).
  uint32_t rows = p.rows;
  if (p.ids) rows = p.rows > p.experts ? 16 : p.x_rows == 1 ? 1 : 4;
  l.pass = p.rows < rows ? p.rows : rows < 16 ? rows : 16;
  // Without experts up to 8 passes at the same time (64 rows of 7168 x 7168: 47 us
  // one after the other, 33; 50 rows of 120 x 5888: 35 and 11). How many an
  // expert has is not known here, and workgroups that find no rows cost more than
  // they save (32 tokens to 2 of 8 experts of 14336 x 4096: 68 us, 73 with three).
  const uint32_t passes = p.ids ? 1 : (p.rows + l.pass - 1) / l.pass;
  l.passes = passes < 8 ? passes : 8;
  const uint64_t tiles = ((uint64_t)p.n + 15) / 16 * (l.slots ? l.slots : 1);
  if ((tiles + 8 * (uint64_t)l.slots + 8) * l.passes >= uint64_t(1) << 31) l.passes = 1;
  const double here = p.ids ? (p.n + 15) / 16 * live_experts(p) : (double)tiles * l.passes;
  l.few = here <= 2 * kCus;
  switch (p.w_shift) {
    case 0: return launch_s<0>(l, stream);
    case 1: return launch_s<1>(l, stream);
    case 2: return launch_s<2>(l, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qcast
