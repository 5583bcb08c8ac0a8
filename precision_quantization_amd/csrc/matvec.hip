// matvec.hip -- products of a few rows with E2M1 weights and group scales.
//
// out[r][i] = sum_g sf[i][g] * (sum_{j in g} code[i][j] * x[r][j]), the inner
// sum over one scale group in the matrix cores (an E2M1 value and an 8-bit
// code are bf16 values: nothing is rounded on the way in), the outer one in
// fp32. A weight is read once for up to 16 rows that share it: bound by HBM
// reads of the weights.
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
// each of them four times: 3 us more on that weight). x is in LDS for the whole
// workgroup, which then takes several column tiles, or, where it does not fit,
// comes with the weights through the wave's own LDS, so that no wave waits for
// another until those that share a tile add their sums, in a fixed order. Row 1
// of 7168 x 18432 in groups of 32: 18.9 us (82.6 MB, 4.4 TB/s); 8 experts'
// 4096 x 7168 in groups of 128: 26 us (4.8 TB/s).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kUnit = 256;            // k of a unit: 128 bytes of a row of w
constexpr uint32_t kXRow = kUnit * 2 + 16; // a unit's row of x in LDS: 4 banks apart

struct MatvecLaunch {
  Matvec p;
  uint32_t tiles;        // workgroups along n
  uint32_t n_waves;      // column tiles of a workgroup
  uint32_t k_waves;      // waves that share a column tile
  uint32_t n_loop;       // column tiles that a wave takes one after the other
  uint32_t pass;         // rows that are taken at once
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
// comes, how many of its rows a pass takes at most (4 or 16), and whether all of
// x is in LDS, for all waves, or comes with the weights, to each wave's own LDS.
template <int kShift, bool kPacked, int kX, int kR, bool kAll>
struct Variant {
  static constexpr int kI = kR / 4;                    // results of a lane's four that hold rows
  static constexpr int kUnits = kAll && kR == 4 ? 2 : 1;   // units of a turn
  static constexpr int kAhead = !kAll && kX == kXStep ? 1 : 2;   // turns in flight
  static constexpr int kWaves = kAll || kR == 4 ? 16 : 8;        // most waves of a workgroup
  static constexpr int kTiles = kAll || kR == 4 ? 1 : 2;         // tiles of 16 columns that share x
  static constexpr uint32_t kCols = 16 * kTiles;
  static constexpr int kGroups = kUnits * 8 >> kShift; // of a row of w, in a turn
  static constexpr int kPer = kGroups >= 4 ? kGroups / 4 : 1;   // of them, one lane's
  static constexpr int kXLoads = kAll ? 1 : kX == kXPlain ? 2 * kI : kI;
  static constexpr int kXScales = kX == kXPlain || kAll ? 1 : kX == kXBlock ? 2 : 8;   // of a unit
  static constexpr int kSteps = kX == kXStep ? 8 : 2;  // scales of a unit of a row of x in LDS
  static constexpr uint32_t kSfRow = kGroups * 4 + 16; // a row's scales of w in LDS
  static constexpr uint32_t kXBytes = kAll ? 0 : kR * kXRow;
  // a wave's LDS: its x, scales of w, and its sums of two tiles
  static constexpr uint32_t kSums = kXBytes + 16 * kTiles * kSfRow;
  static constexpr uint32_t kLds = kSums + 2 * kTiles * kI * 256;

  // What a lane has in flight for one turn.
  struct Turn {
    u32x4 w[kUnits][kTiles][2];          // of rows lane % 8 and 8 more: chunk lane / 8
    uint32_t sf[kTiles][kPer];           // of row lane / 4, as stored (packed: a byte each)
    u32x4 x[kXLoads];
    float xs[kUnits][kI][kXScales];      // of the rows of the lane's results
  };
};

// Where a wave reads. The 16 rows of a column tile are buffers: an offset past
// their end (a row past n, a unit past the wave's last) loads zeros, so that
// the loads ahead need no branch and the compiler waits for no more than it
// must. Units past the last read x's first bytes, and are not used.
constexpr uint32_t kPastEnd = 0x80000000u;
template <int kI>
struct Places {
  RowBuffer w, sf;
  uint32_t w_at, w_half, sf_at, sf_tile;
  const uint8_t* x[kI];
  const float* xs[kI];
  uint32_t end;                          // of the wave's whole units
};

template <typename V, int kShift, bool kPacked, int kX>
__device__ __forceinline__ void load_turn_w(typename V::Turn& t, const Places<V::kI>& r,
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

template <typename V, int kX>
__device__ __forceinline__ void load_turn_x(typename V::Turn& t, const Places<V::kI>& r,
                                            uint32_t unit, uint32_t shift) {
  const uint32_t lane = threadIdx.x & 63;
  constexpr uint32_t kRowBytes = kX == kXPlain ? kUnit * 2 : kUnit;
  const bool in = unit < r.end;
  const uint32_t at = in ? unit * kRowBytes + (lane & 15) * 16 : 0;
#pragma unroll
  for (int i = 0; i < V::kI; ++i) {
    if constexpr (kX == kXPlain) {
      t.x[2 * i] = *reinterpret_cast<const u32x4*>(r.x[i] + at);
      t.x[2 * i + 1] = *reinterpret_cast<const u32x4*>(r.x[i] + at + (in ? 256 : 0));
    } else {
      t.x[i] = *reinterpret_cast<const u32x4*>(r.x[i] + at);
    }
  }
  if constexpr (kX != kXPlain) {
#pragma unroll
    for (int p = 0; p < V::kUnits; ++p)
#pragma unroll
      for (int i = 0; i < V::kI; ++i)
#pragma unroll
        for (int g = 0; g < V::kXScales; ++g) {
          // scales of 128 k, or of 32 << shift k
          const uint32_t u = unit + p;
          const uint32_t j = kX == kXBlock ? u * 2 + g : (u * 8 + g) >> shift;
          t.xs[p][i][g] = r.xs[i][u < r.end ? j : 0];
        }
  }
}

// The unit that k ends in, as the first unit of a turn: zeros past k.
template <typename V, int kShift, bool kPacked, int kX>
__device__ __forceinline__ void load_tail_w(typename V::Turn& t, const Places<V::kI>& r,
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

template <typename V, int kX>
__device__ __forceinline__ void load_tail_x(typename V::Turn& t, const Places<V::kI>& r,
                                            uint32_t k, uint32_t shift) {
  const uint32_t lane = threadIdx.x & 63, k0 = k / kUnit * kUnit;
  // 8 (or, of codes, 16) k a lane
#pragma unroll
  for (int q = 0; q < V::kXLoads; ++q) {
    constexpr bool kBf16 = kX == kXPlain;
    const int i = kBf16 ? q / 2 : q;
    const uint32_t at = kBf16 ? (q % 2) * 128 + (lane & 15) * 8 : (lane & 15) * 16;
    t.x[q] = u32x4{0, 0, 0, 0};
    if (k0 + at < k)
      t.x[q] = *reinterpret_cast<const u32x4*>(r.x[i] + (k0 + at) * (kBf16 ? 2 : 1));
  }
  if constexpr (kX != kXPlain) {
#pragma unroll
    for (int i = 0; i < V::kI; ++i)
#pragma unroll
      for (int g = 0; g < V::kXScales; ++g) {
        const uint32_t at = k0 + g * (kX == kXBlock ? 128 : 32);
        t.xs[0][i][g] = at < k ? r.xs[i][at / 32 >> (kX == kXBlock ? 2 : shift)] : 0.0f;
      }
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

// The turn's x (as bf16) and scales (as fp32) to the wave's LDS.
template <typename V, bool kPacked, int kX, bool kAll>
__device__ __forceinline__ void store_turn(const typename V::Turn& t, uint8_t* mine, int fmt) {
  const uint32_t lane = threadIdx.x & 63;
  if constexpr (!kAll) {
    uint8_t* to = mine + (lane >> 4) * kXRow + (lane & 15) * (kX == kXPlain ? 16 : 32);
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
  constexpr int kParts = V::kGroups / V::kPer;
#pragma unroll
  for (int t2 = 0; t2 < V::kTiles; ++t2) {
    uint8_t* to = mine + V::kXBytes + (t2 * 16 + (lane >> 2)) * V::kSfRow +
                  (lane & (kParts - 1)) * V::kPer * 4;
    uint32_t f[V::kPer];
#pragma unroll
    for (int g = 0; g < V::kPer; ++g)
      f[g] = kPacked ? (t.sf[t2][0] >> (8 * g) & 0xffu) << 23 : t.sf[t2][g];
    if constexpr (V::kPer == 4) *reinterpret_cast<u32x4*>(to) = u32x4{f[0], f[1], f[2], f[3]};
    else if constexpr (V::kPer == 2) *reinterpret_cast<u32x2*>(to) = u32x2{f[0], f[1]};
    else *reinterpret_cast<uint32_t*>(to) = f[0];
  }
}

// All of x of the pass's cnt rows (row m in lane m of list), as bf16, rows of
// `stride` bytes, zeros to the end of the last unit; and their scales, V::kSteps
// of a unit, to `scales`. Four loads in flight.
template <typename V, int kX>
__device__ __forceinline__ void stage_x(const Matvec& p, uint8_t* lds, float* scales,
                                        uint32_t list, uint32_t cnt, uint32_t per,
                                        uint32_t units, uint32_t stride) {
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
      v[a] = u32x4{0, 0, 0, 0};
      sx[a] = 0.0f;
      if (i < all && j[a] * 8 < p.k) {
        if constexpr (kX == kXPlain) {
          v[a] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.x) +
                                                 x_row * p.k + j[a] * 8);
        } else {
          const u32x2 q = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(p.x) +
                                                          x_row * p.k + j[a] * 8);
          v[a].x = q.x;
          v[a].y = q.y;
          sx[a] = p.x_sf[x_row * (p.k / 32 >> p.x_shift) + (j[a] / 4 >> p.x_shift)];
        }
      }
    }
#pragma unroll
    for (int a = 0; a < kBatch; ++a) {
      if (i0 + a * blockDim.x < all) {
        uint8_t* row = lds + m[a] * stride;
        if constexpr (kX != kXPlain) {
          constexpr uint32_t kOf = kUnit / 8 / V::kSteps;      // chunks of a scale
          v[a] = codes_bf16(v[a].x, v[a].y, p.x_fmt);
          if (j[a] % kOf == 0) scales[m[a] * units * V::kSteps + j[a] / kOf] = sx[a];
        }
        *reinterpret_cast<u32x4*>(row + j[a] * 16) = v[a];
      }
    }
  }
}

template <int kShift, bool kPacked, int kX, int kR, bool kAll>
__global__ __launch_bounds__((Variant<kShift, kPacked, kX, kR, kAll>::kWaves * 64)) void
matvec_kernel(MatvecLaunch l) {
  using V = Variant<kShift, kPacked, kX, kR, kAll>;
  constexpr int kI = V::kI;
  const Matvec& p = l.p;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];    // the waves', then all of x
  const uint32_t lane = threadIdx.x & 63, n = lane & 15, c = lane >> 4;
  const uint32_t wave = (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const uint32_t wn = wave / l.k_waves, wk = wave - wn * l.k_waves;
  const uint32_t slot = blockIdx.x / l.tiles;
  const uint32_t tile0 = ((blockIdx.x - slot * l.tiles) * l.n_waves + wn) * l.n_loop;

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
  Places<kI> at;
  at.w_at = (lane & 7) * w_row + (lane >> 3) * 16;
  at.w_half = 8 * w_row;
  at.sf_tile = 16 * sf_row;
  constexpr int kParts = V::kGroups / V::kPer;
  at.sf_at = (lane >> 2) * sf_row + (lane & (kParts - 1)) * V::kPer * (kPacked ? 1 : 4);
  auto to_tile = [&](uint32_t tile) {
    const uint32_t held =
        tile * V::kCols >= p.n ? 0 : p.n - tile * V::kCols < V::kCols ? p.n - tile * V::kCols : V::kCols;
    const uint64_t row0 = held && !none ? (uint64_t)expert * p.n + tile * V::kCols : 0;
    at.w = row_buffer(p.w, row0 * w_row, held * w_row);
    at.sf = row_buffer(p.w_sf, row0 * sf_row, held * sf_row);
  };
  // this wave's whole units of a tile, [begin, end), and its turns in all tiles
  const uint32_t full = none ? 0 : p.k / kUnit;
  const uint32_t begin = full * wk / l.k_waves;
  at.end = full * (wk + 1) / l.k_waves;
  const bool ends = !none && p.k % kUnit != 0 && wk == l.k_waves - 1;
  const uint32_t turns = (at.end - begin + V::kUnits - 1) / V::kUnits;
  const uint32_t items = turns * l.n_loop;
  const uint32_t per = l.slots ? p.rows / p.x_rows : 1;
  uint8_t* const mine = lds + wave * V::kLds;
  uint8_t* const x_all = lds + l.n_waves * l.k_waves * V::kLds;
  // A's row n is row m; rows that there are not give results that nobody reads
  const uint32_t m_of_lane = (n >> 2) + 4 * ((n & 3) % kI);
  const uint32_t all_units = (p.k + kUnit - 1) / kUnit;
  const uint32_t x_stride = kAll ? all_units * (kUnit * 2) + 16 : kXRow;
  float* const x_scales = reinterpret_cast<float*>(x_all + l.pass * x_stride);
  const uint8_t* const sa = mine + V::kXBytes + n * V::kSfRow;

  // the ring; the next turn starts at unit `ahead` of tile `ahead_tile`
  typename V::Turn ring[V::kAhead];
  uint32_t ahead = begin, ahead_tile = tile0;
  auto next = [&]() {
    ahead += V::kUnits;
    if (ahead >= at.end) {
      ahead = begin;
      ++ahead_tile;
      to_tile(ahead_tile < tile0 + l.n_loop ? ahead_tile : 0xfffffffu);
    }
  };
  // the first turn's weights are asked for before it is known whose rows they meet
  to_tile(tile0);
  if (items) load_turn_w<V, kShift, kPacked, kX>(ring[0], at, ahead);
  for (uint32_t first = 0;; first += l.pass) {
    // the rows of this pass: those with the slot's expert, l.pass at a time; lane
    // m holds the m-th
    uint32_t cnt = 0, list = 0;
    if (l.slots) {
      uint32_t seen = 0;
      bool leads = true;
      for (uint32_t r0 = 0; r0 < p.rows; r0 += 64) {
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
    for (int i = 0; i < kI; ++i) {
      const uint32_t m = c + 4 * i;
      row[i] = (uint32_t)__shfl((int)list, m < cnt ? (int)m : 0);
      const uint64_t x_row = row[i] / per;
      at.x[i] = static_cast<const uint8_t*>(p.x) + x_row * p.k * (kX == kXPlain ? 2 : 1);
      at.xs[i] = p.x_sf + (kX == kXPlain ? 0 : x_row * (p.k / 32 >> p.x_shift));
    }

    if constexpr (kAll) {
      if (!none) stage_x<V, kX>(p, x_all, x_scales, list, cnt, per, all_units, x_stride);
      lds_barrier();
    }
    const uint8_t* const xa =
        (kAll ? x_all : mine) + (kAll && m_of_lane >= cnt ? 0 : m_of_lane) * x_stride + c * 16;
    const float* xs[kI];
#pragma unroll
    for (int i = 0; i < kI; ++i)
      xs[i] = x_scales + (c + 4 * i < cnt ? c + 4 * i : 0) * all_units * V::kSteps;

    float acc[V::kTiles][kI];
#pragma unroll
    for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
      for (int i = 0; i < kI; ++i) acc[t2][i] = 0.0f;
    auto add_turn = [&](const typename V::Turn& t, uint32_t unit, uint32_t held) {
      store_turn<V, kPacked, kX, kAll>(t, mine, p.x_fmt);
      wave_order();
#pragma unroll
      for (int u = 0; u < V::kUnits; ++u) {
        if (u > 0 && u >= (int)held) break;
        constexpr int kOfUnit = 8 >> kShift;
        uint32_t r[V::kTiles][8];
#pragma unroll
        for (int t2 = 0; t2 < V::kTiles; ++t2) to_steps(t.w[u][t2], r[t2]);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bf16x8 a[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            a[j] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(
                                                  xa + (kAll ? (unit + u) * (kUnit * 2) : 0) +
                                                  h * 256 + j * 64));
          float f_x[kI][kX == kXStep ? 4 : 1];
          if constexpr (kX != kXPlain) {
            constexpr int kHalf = kX == kXStep ? 4 : 1;
#pragma unroll
            for (int i = 0; i < kI; ++i)
#pragma unroll
              for (int g = 0; g < kHalf; ++g)
                f_x[i][g] = kAll ? xs[i][(unit + u) * V::kSteps + h * kHalf + g]
                                 : t.xs[u][i][kAll ? 0 : h * kHalf + g];
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
        Places<kI> last = at;
        const uint32_t held =
            tile * V::kCols >= p.n ? 0 : p.n - tile * V::kCols < V::kCols ? p.n - tile * V::kCols : V::kCols;
        const uint64_t row0 = held ? (uint64_t)expert * p.n + tile * V::kCols : 0;
        last.w = row_buffer(p.w, row0 * w_row, held * w_row);
        last.sf = row_buffer(p.w_sf, row0 * sf_row, held * sf_row);
        typename V::Turn t;
        load_tail_w<V, kShift, kPacked, kX>(t, last, p.k);
        if constexpr (!kAll) load_tail_x<V, kX>(t, last, p.k, p.x_shift);
        add_turn(t, full, 1);
      }
      const uint32_t half = (tile - tile0) & 1;
      if (l.k_waves > 1) {
        if (wk) {
#pragma unroll
          for (int t2 = 0; t2 < V::kTiles; ++t2)
#pragma unroll
            for (int i = 0; i < kI; ++i) reinterpret_cast<float*>(mine + V::kSums)[((half * V::kTiles + t2) * kI + i) * 64 + lane] =
                  acc[t2][i];
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
    if (items) {
      if (first) {
        ahead = begin;
        ahead_tile = tile0;
        to_tile(tile0);
        load_turn_w<V, kShift, kPacked, kX>(ring[0], at, ahead);
      }
      if constexpr (!kAll) load_turn_x<V, kX>(ring[0], at, ahead, p.x_shift);
      next();
#pragma unroll
      for (int a = 1; a < V::kAhead; ++a) {
        load_turn_w<V, kShift, kPacked, kX>(ring[a], at, ahead);
        if constexpr (!kAll) load_turn_x<V, kX>(ring[a], at, ahead, p.x_shift);
        next();
      }
      // places in the ring are fixed, so that nothing waits for a load but its use
      uint32_t unit = begin;
      for (uint32_t q = 0; q < items; q += V::kAhead) {
#pragma unroll
        for (int a = 0; a < V::kAhead; ++a) {
          if (q + a < items) {
            add_turn(ring[a], unit, at.end - unit);
            unit += V::kUnits;
            if (unit >= at.end) {
              flush();
              unit = begin;
            }
          }
          load_turn_w<V, kShift, kPacked, kX>(ring[a], at, ahead);
          if constexpr (!kAll) load_turn_x<V, kX>(ring[a], at, ahead, p.x_shift);
          next();
        }
      }
    } else {
      for (uint32_t t = 0; t < l.n_loop; ++t) flush();
    }
    if (kAll || l.k_waves > 1) __syncthreads();          // LDS has been read
  }
}

template <int kShift, bool kPacked, int kX, int kR, bool kAll>
hipError_t launch_variant(const MatvecLaunch& l, uint32_t x_lds, uint32_t groups,
                          hipStream_t stream) {
  const uint32_t waves = l.n_waves * l.k_waves;
  launch_kernel(matvec_kernel<kShift, kPacked, kX, kR, kAll>, dim3(groups), dim3(waves * 64),
                waves * Variant<kShift, kPacked, kX, kR, kAll>::kLds + x_lds, stream, l);
  return hipGetLastError();
}

template <int kShift, bool kPacked, int kX>
hipError_t launch_rows(const MatvecLaunch& l, bool all, uint32_t lds, uint32_t groups,
                       hipStream_t stream) {
  if (l.pass <= 4)
    return all ? launch_variant<kShift, kPacked, kX, 4, true>(l, lds, groups, stream)
               : launch_variant<kShift, kPacked, kX, 4, false>(l, 0, groups, stream);
  return all ? launch_variant<kShift, kPacked, kX, 16, true>(l, lds, groups, stream)
             : launch_variant<kShift, kPacked, kX, 16, false>(l, 0, groups, stream);
}

template <int kShift, bool kPacked>
hipError_t launch_x(const MatvecLaunch& l, bool all, uint32_t lds, uint32_t groups,
                    hipStream_t stream) {
  return !l.p.x_fmt          ? launch_rows<kShift, kPacked, kXPlain>(l, all, lds, groups, stream)
         : l.p.x_shift == 2  ? launch_rows<kShift, kPacked, kXBlock>(l, all, lds, groups, stream)
                             : launch_rows<kShift, kPacked, kXStep>(l, all, lds, groups, stream);
}

template <int kShift>
hipError_t launch_s(const MatvecLaunch& l, bool all, uint32_t lds, uint32_t groups,
                    hipStream_t stream) {
  return l.p.packed ? launch_x<kShift, true>(l, all, lds, groups, stream)
                    : launch_x<kShift, false>(l, all, lds, groups, stream);
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
  const uint32_t units = (p.k + kUnit - 1) / kUnit;
  // rows that one reading of a weight serves
  uint32_t rows = p.rows;
  if (p.ids) {
    const uint32_t even = (uint32_t)((p.rows + p.experts - 1) / (p.experts ? p.experts : 1));
    rows = p.rows < 2 * even + 2 ? p.rows : 2 * even + 2;
    if ((int64_t)p.rows * p.rows <= 4 * p.experts) rows = 1;
  }
  l.pass = rows < 16 ? rows : 16;
  // All of x in LDS where it fits beside the waves' own: 16 tokens to 8 of 32
  // experts' 7168 x 2048 take 63 us so and 81 otherwise; one row of 18432, 18.9
  // and 19.8.
  constexpr uint32_t kXLds = 96 * 1024;
  const uint32_t row_lds = units * (kUnit * 2 + (!p.x_fmt ? 0 : p.x_shift == 2 ? 8 : 32)) + 16;
  const bool all = (uint64_t)l.pass * row_lds <= kXLds;
  const uint32_t lds = all ? l.pass * row_lds : 0;
  const uint32_t most = all || l.pass <= 4 ? 16 : 8;
  const uint32_t cols = all || l.pass <= 4 ? 16 : 32;
  const uint32_t tiles = (p.n + cols - 1) / cols;
  const uint64_t work = (uint64_t)tiles * (l.slots ? l.slots : 1);
  // Waves that share a tile: until there are 6 waves for each of 256 compute
  // units, of four units of k or more (7168 x 18432: 48 us with one, 19 with four,
  // 24 with 16). Workgroups of 8 waves; tiles one after the other past 24 waves
  // for each (the 32 experts: 62 us with one, 58 with two, 72 with four).
  constexpr uint32_t kCus = 256;
  l.k_waves = 1;
  while (l.k_waves < most && l.k_waves * 4 <= units && work * l.k_waves < kCus * 6)
    l.k_waves *= 2;
  l.n_waves = l.k_waves < 8 ? 8 / l.k_waves : 1;
  while (l.n_waves > 1 && l.n_waves > tiles) l.n_waves /= 2;
  const uint64_t loops = work * l.k_waves / (kCus * 24);
  l.n_loop = loops < 1 ? 1 : loops > 8 ? 8 : (uint32_t)loops;
  l.tiles = (tiles + l.n_waves * l.n_loop - 1) / (l.n_waves * l.n_loop);
  const uint64_t groups = (uint64_t)l.tiles * (l.slots ? l.slots : 1);
  if (groups >= (uint64_t(1) << 31)) return hipErrorInvalidValue;
  switch (p.w_shift) {
    case 0: return launch_s<0>(l, all, lds, (uint32_t)groups, stream);
    case 1: return launch_s<1>(l, all, lds, (uint32_t)groups, stream);
    case 2: return launch_s<2>(l, all, lds, (uint32_t)groups, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace qcast
