// expert_sort.hip -- the slots (token, k) of a batch sorted by expert: a
// counting sort, stable, so that the result does not depend on timing.
//
// counts[e] = slots of expert e, offsets[e+1] = offsets[e] + counts[e] rounded
// up to `align`, and the row of a slot = offsets[e] + the number of earlier
// slots of e. A wave takes 64 slots at a time; which of its lanes hold the
// same expert comes from one ballot per bit of the expert's number, so no
// atomic decides an order: a lane's rank is the count of lower lanes with its
// expert, and one lane per expert adds the whole count to the wave's own
// column of counts in LDS.
//
// It moves 12 to 24 bytes a slot, 3.4 MB with the rows' padding for 16384 x 8
// slots with weights: bound by launches and by the chain of loads, LDS and cache
// trips (10.3 us; 8 x 8 slots 5.3).
#include "qcast_device.h"
#include "qcast_kernels.h"
#include "qcast_row.h"

namespace qcast {
namespace {

constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / 64;

// The expert of a slot, counted from `first`; `experts` where it is not here.
__device__ __forceinline__ uint32_t expert_of(const ExpertSort& p, uint32_t slot) {
  const int64_t id = p.wide ? static_cast<const int64_t*>(p.ids)[slot]
                            : (int64_t)static_cast<const int32_t*>(p.ids)[slot];
  const uint64_t e = (uint64_t)id - (uint64_t)p.first;
  return e < p.experts ? (uint32_t)e : p.experts;
}

// Lanes of the wave with this lane's expert (of a lane that has one).
__device__ __forceinline__ uint64_t same_expert(uint32_t e, uint32_t experts) {
  uint64_t same = __builtin_amdgcn_ballot_w64(e < experts);
  for (uint32_t b = 1; b < experts; b <<= 1) {
    const uint64_t set = __builtin_amdgcn_ballot_w64((e & b) != 0);
    same &= (e & b) ? set : ~set;
  }
  return same;
}

// The slots of a wave: [begin, end) of the part.
__device__ __forceinline__ void wave_slots(const ExpertSort& p, uint32_t part, uint32_t& begin,
                                           uint32_t& end) {
  const uint32_t wave = threadIdx.x >> 6;
  const uint32_t p0 = part * p.part;
  const uint32_t p1 = p.slots - p0 < p.part ? p.slots : p0 + p.part;
  const uint32_t per = ((p1 - p0 + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  begin = p1 - p0 < wave * per ? p1 : p0 + wave * per;
  end = p1 - begin < per ? p1 : begin + per;
}

// Experts of a wave's slots, 64 at a time: the first kHeld times in registers
// (each is waited for before the next is asked for, as every load has a branch of
// its bounds and of the ids' width); the rest (parts of more than 4096 slots) read
// again.
constexpr int kHeld = 4;
struct Slots {
  uint32_t e[kHeld];
  __device__ __forceinline__ void load(const ExpertSort& p, uint32_t begin, uint32_t end) {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t s = begin + i * 64 + lane;
      e[i] = s < end ? expert_of(p, s) : p.experts;
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(const ExpertSort& p, uint32_t begin, uint32_t end,
                                       F&& f) const {
    const uint32_t lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (begin + i * 64 < end) f(begin + i * 64 + lane, e[i]);
    for (uint32_t s = begin + kHeld * 64; s < end; s += 64)
      f(s + lane, s + lane < end ? expert_of(p, s + lane) : p.experts);
  }
};

// The counts of one part (a workgroup's slots). kExperts: room in LDS.
template <uint32_t kExperts>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(ExpertSort p) {
  __shared__ uint32_t counts[kExperts];
  uint32_t begin, end;
  wave_slots(p, blockIdx.x, begin, end);
  Slots slots;
  slots.load(p, begin, end);
  for (uint32_t i = threadIdx.x; i < kExperts; i += kSortThreads) counts[i] = 0;
  __syncthreads();
  slots.each(p, begin, end, [&](uint32_t, uint32_t e) {
    if (e < p.experts) atomicAdd(&counts[e], 1u);      // whole numbers: in any order the same
  });
  __syncthreads();
  if (threadIdx.x < p.experts)
    p.ws[blockIdx.x * p.experts + threadIdx.x] = (int32_t)counts[threadIdx.x];
}

// Rows without a slot.
__device__ __forceinline__ void no_slot(const ExpertSort& p, uint32_t row) {
  p.source[row] = -1;
  if (p.row_weight) p.row_weight[row] = 0.0f;
}

template <uint32_t kExperts>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(ExpertSort p) {
  constexpr uint32_t kQ = kSortThreads / kExperts;     // threads of an expert
  constexpr uint32_t kQWaves = kSortWaves / kQ;
  __shared__ uint32_t columns[kSortWaves][kExperts];   // a wave's slots of each expert
  __shared__ uint32_t sums[3][kQ][kExperts];           // of parts in all, of parts before, of waves
  __shared__ uint32_t start[kExperts + 1], held[kExperts], wave_sums[kSortWaves];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const uint32_t e = threadIdx.x % kExperts, q = threadIdx.x / kExperts;
  const bool mine = e < p.experts;
  uint32_t begin = 0, end = 0;
  // with one part every workgroup counts it, the first has its slots, and all
  // share the rows without one
  const uint32_t part = p.ws ? blockIdx.x : 0;
  if (p.slots) wave_slots(p, part, begin, end);
  Slots slots;
  slots.load(p, begin, end);
  // thread (e, q): the slots of expert e in a kQ-th of the parts
  uint32_t total = 0, before = 0;
  if (p.ws && mine) {
    const uint32_t b1 = gridDim.x * (q + 1) / kQ;
    uint32_t b = gridDim.x * q / kQ;
    for (; b + 8 <= b1; b += 8) {
      uint32_t n[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) n[i] = (uint32_t)p.ws[(b + i) * p.experts + e];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        total += n[i];
        before += b + i < blockIdx.x ? n[i] : 0;
      }
    }
    for (; b < b1; ++b) {
      const uint32_t n = (uint32_t)p.ws[b * p.experts + e];
      total += n;
      before += b < blockIdx.x ? n : 0;
    }
  }
  for (uint32_t i = threadIdx.x; i < kSortWaves * kExperts; i += kSortThreads)
    (&columns[0][0])[i] = 0;
  __syncthreads();
  uint32_t* column = columns[wave];
  slots.each(p, begin, end, [&](uint32_t, uint32_t x) {
    if (x < p.experts) atomicAdd(&column[x], 1u);
  });
  __syncthreads();
  uint32_t in_waves = 0;
#pragma unroll
  for (uint32_t w = 0; w < kQWaves; ++w) in_waves += columns[q * kQWaves + w][e];
  sums[0][q][e] = total;
  sums[1][q][e] = before;
  sums[2][q][e] = in_waves;
  __syncthreads();
  total = before = 0;
#pragma unroll
  for (uint32_t i = 0; i < kQ; ++i) {
    const uint32_t n = sums[2][i][e];
    total += p.ws ? sums[0][i][e] : n;
    before += sums[1][i][e] + (i < q ? n : 0);
  }
  // the slots of expert e before each of these waves
#pragma unroll
  for (uint32_t w = 0; w < kQWaves; ++w) {
    const uint32_t n = columns[q * kQWaves + w][e];
    columns[q * kQWaves + w][e] = before;
    before += n;
  }
  // offsets: the sum of the runs before e, within the wave and over the waves
  const uint32_t run = mine && q == 0 ? (total + p.align - 1) & ~(p.align - 1) : 0;
  uint32_t upto = run;
#pragma unroll
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const uint32_t v = (uint32_t)__shfl_up((int)upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) wave_sums[wave] = upto;
  __syncthreads();
  if (mine && q == 0) {
    uint32_t base = 0;
    for (uint32_t w = 0; w < wave; ++w) base += wave_sums[w];
    upto += base;
    start[e] = upto - run;
    held[e] = total;
    if (e == p.experts - 1) start[p.experts] = upto;
    if (blockIdx.x == 0) {
      p.counts[e] = (int32_t)total;
      p.offsets[e] = (int32_t)(upto - run);
      if (e == p.experts - 1) p.offsets[p.experts] = (int32_t)upto;
    }
  }
  __syncthreads();
  if (part == blockIdx.x) slots.each(p, begin, end, [&](uint32_t slot, uint32_t x) {
    const uint64_t same = same_expert(x, p.experts);
    const uint64_t lower = same & ((1ull << lane) - 1);
    if (x < p.experts) {
      const uint32_t at = column[x];
      const uint32_t row = start[x] + at + (uint32_t)__builtin_popcountll(lower);
      if (lower == 0) column[x] = at + (uint32_t)__builtin_popcountll(same);
      p.dest[slot] = (int32_t)row;
      p.source[row] = (int32_t)slot;
      if (p.row_weight) p.row_weight[row] = p.weight[slot];
    } else if (slot < end) {
      p.dest[slot] = -1;
    }
    wave_order();
  });
  // padding rows, a wave for an expert, and the rows behind the last run
  for (uint32_t x = blockIdx.x * kSortWaves + wave; x < p.experts; x += gridDim.x * kSortWaves)
    for (uint32_t r = start[x] + held[x] + lane; r < start[x + 1]; r += 64) no_slot(p, r);
  for (uint32_t r = start[p.experts] + blockIdx.x * kSortThreads + threadIdx.x; r < p.rows;
       r += gridDim.x * kSortThreads)
    no_slot(p, r);
}

template <uint32_t kExperts>
hipError_t launch(const ExpertSort& p, uint32_t parts, hipStream_t stream) {
  if (parts > 1) {
    launch_kernel(sort_count_kernel<kExperts>, dim3(parts), dim3(kSortThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  // rows without a slot: a workgroup for 4096 rows, up to 16 (512 x 8 slots of 256
  // experts in runs of 128, 36608 rows: 11.7 us with one workgroup, 8.4 with nine)
  const uint32_t fill = p.rows / 4096 < 16 ? p.rows / 4096 + 1 : 16;
  launch_kernel(sort_place_kernel<kExperts>, dim3(parts > 1 ? parts : fill), dim3(kSortThreads),
                0, stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_expert_sort(const ExpertSort& p, hipStream_t stream) {
  const uint32_t parts = p.slots > p.part ? (p.slots + p.part - 1) / p.part : 1;
  if (parts > 1 && !p.ws) return hipErrorInvalidValue;
  ExpertSort q = p;
  if (parts == 1) q.ws = nullptr;
  if (p.experts <= 256) return launch<256>(q, parts, stream);
  if (p.experts <= 1024) return launch<1024>(q, parts, stream);
  return hipErrorInvalidValue;
}

}  // namespace qcast
