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
// What it must move is about a megabyte at most: bound by launches and by the
// chain of LDS and cache trips.
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

// Count the slots [begin, end) of this wave into its column of `column`.
__device__ __forceinline__ void count_wave(const ExpertSort& p, uint32_t begin, uint32_t end,
                                           uint32_t* column) {
  const uint32_t lane = threadIdx.x & 63;
  for (uint32_t s = begin; s < end; s += 64) {
    const uint32_t e = s + lane < end ? expert_of(p, s + lane) : p.experts;
    const uint64_t same = same_expert(e, p.experts);
    if (e < p.experts && (same & ((1ull << lane) - 1)) == 0)
      column[e] += (uint32_t)__builtin_popcountll(same);
    wave_order();
  }
}

__device__ __forceinline__ void wave_slots(const ExpertSort& p, uint32_t& begin, uint32_t& end) {
  const uint32_t wave = threadIdx.x >> 6;
  const uint32_t p0 = blockIdx.x * p.part;                     // < slots
  const uint32_t p1 = p.slots - p0 < p.part ? p.slots : p0 + p.part;
  const uint32_t per = ((p1 - p0 + kSortWaves - 1) / kSortWaves + 63) / 64 * 64;
  begin = p1 - p0 < wave * per ? p1 : p0 + wave * per;
  end = p1 - begin < per ? p1 : begin + per;
}

// The counts of one part (a workgroup's slots). kExperts: room in LDS.
template <uint32_t kExperts>
__global__ __launch_bounds__(kSortThreads) void sort_count_kernel(ExpertSort p) {
  __shared__ uint32_t columns[kSortWaves][kExperts];
  for (uint32_t i = threadIdx.x; i < kSortWaves * kExperts; i += kSortThreads)
    (&columns[0][0])[i] = 0;
  __syncthreads();
  uint32_t begin, end;
  wave_slots(p, begin, end);
  count_wave(p, begin, end, columns[threadIdx.x >> 6]);
  __syncthreads();
  if (threadIdx.x < p.experts) {
    uint32_t n = 0;
    for (uint32_t w = 0; w < kSortWaves; ++w) n += columns[w][threadIdx.x];
    p.ws[blockIdx.x * p.experts + threadIdx.x] = (int32_t)n;
  }
}

// Rows without a slot.
__device__ __forceinline__ void no_slot(const ExpertSort& p, uint32_t row) {
  p.source[row] = -1;
  if (p.row_weight) p.row_weight[row] = 0.0f;
}

template <uint32_t kExperts>
__global__ __launch_bounds__(kSortThreads) void sort_place_kernel(ExpertSort p) {
  __shared__ uint32_t columns[kSortWaves][kExperts];
  __shared__ uint32_t start[kExperts + 1];
  __shared__ uint32_t sums[kSortWaves];
  const uint32_t wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (uint32_t i = threadIdx.x; i < kSortWaves * kExperts; i += kSortThreads)
    (&columns[0][0])[i] = 0;
  __syncthreads();
  uint32_t begin = 0, end = 0;
  if (p.slots) wave_slots(p, begin, end);
  uint32_t* column = columns[wave];
  count_wave(p, begin, end, column);
  __syncthreads();

  // thread e: the slots of expert e before each wave, and in all
  uint32_t total = 0, run = 0;
  if (threadIdx.x < p.experts) {
    uint32_t before = 0;
    if (p.ws) {
      for (uint32_t b = 0; b < gridDim.x; ++b) {
        const uint32_t n = (uint32_t)p.ws[b * p.experts + threadIdx.x];
        total += n;
        before += b < blockIdx.x ? n : 0;
      }
    }
    for (uint32_t w = 0; w < kSortWaves; ++w) {
      const uint32_t n = columns[w][threadIdx.x];
      columns[w][threadIdx.x] = before;
      before += n;
    }
    if (!p.ws) total = before;
    run = (total + p.align - 1) & ~(p.align - 1);
  }
  // offsets: the sum of the runs before e, within the wave and over the waves
  uint32_t upto = run;
  for (uint32_t d = 1; d < 64; d <<= 1) {
    const uint32_t v = (uint32_t)__shfl_up((int)upto, d);
    if (lane >= d) upto += v;
  }
  if (lane == 63) sums[wave] = upto;
  __syncthreads();
  uint32_t base = 0;
  for (uint32_t w = 0; w < wave; ++w) base += sums[w];
  if (threadIdx.x < p.experts) {
    start[threadIdx.x] = base + upto - run;
    if (threadIdx.x == p.experts - 1) start[p.experts] = base + upto;
    if (blockIdx.x == 0) {
      p.counts[threadIdx.x] = (int32_t)total;
      p.offsets[threadIdx.x] = (int32_t)(base + upto - run);
      if (threadIdx.x == p.experts - 1) p.offsets[p.experts] = (int32_t)(base + upto);
    }
    // padding rows, the experts dealt to the workgroups
    if (threadIdx.x % gridDim.x == blockIdx.x)
      for (uint32_t r = base + upto - run + total; r < base + upto; ++r) no_slot(p, r);
  }
  __syncthreads();
  for (uint32_t r = start[p.experts] + blockIdx.x * kSortThreads + threadIdx.x; r < p.rows;
       r += gridDim.x * kSortThreads)
    no_slot(p, r);

  for (uint32_t s = begin; s < end; s += 64) {
    const uint32_t slot = s + lane;
    const uint32_t e = slot < end ? expert_of(p, slot) : p.experts;
    const uint64_t same = same_expert(e, p.experts);
    const uint64_t lower = same & ((1ull << lane) - 1);
    if (e < p.experts) {
      const uint32_t at = column[e];
      const uint32_t row = start[e] + at + (uint32_t)__builtin_popcountll(lower);
      if (lower == 0) column[e] = at + (uint32_t)__builtin_popcountll(same);
      p.dest[slot] = (int32_t)row;
      p.source[row] = (int32_t)slot;
      if (p.row_weight) p.row_weight[row] = p.weight[slot];
    } else if (slot < end) {
      p.dest[slot] = -1;
    }
    wave_order();
  }
}

template <uint32_t kExperts>
hipError_t launch(const ExpertSort& p, uint32_t parts, hipStream_t stream) {
  if (parts > 1) {
    launch_kernel(sort_count_kernel<kExperts>, dim3(parts), dim3(kSortThreads), 0, stream, p);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  launch_kernel(sort_place_kernel<kExperts>, dim3(parts), dim3(kSortThreads), 0, stream, p);
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
