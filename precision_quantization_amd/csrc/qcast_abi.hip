// qcast_abi.hip -- the C ABI declared in include/qcast.h: argument checks,
// the format floors, the compute-unit count, and dispatch to the launchers.
//
// Floors ("DeepSeek开源TileKernels：用Python写的GPU算子逼近硬件性能上限", §3.1):
// 1e-4 for E4M3 and the E2M1 maximum times 2^-126 for E2M1, unless the caller
// passes its own clamp_min > 0; E5M2 and E5M6, for which the page names
// none, take the E4M3 floor.
#include <atomic>
#include <mutex>

#include "qcast.h"
#include "qcast_device.h"
#include "qcast_kernels.h"

// The clamp-count slots of qcast_swiglu_per_token_noalloc: a file-scope
// device array (one copy per GPU, held until the process ends), used in
// place of a caller's count workspace. Host code never passes its name to a
// kernel (on the host it is only a stand-in for the symbol); it uses the
// device address that hipGetSymbolAddress returns for the current device.
static __device__ __align__(256) unsigned long long scratch[QCAST_NOALLOC_SCRATCH_BYTES / 8];

namespace {

static_assert(qcast::kCountSlots * qcast::kSlotWords * sizeof(uint64_t) == QCAST_COUNT_WS_BYTES,
              "count workspace size");

constexpr int kMaxDevices = 64;
std::atomic<int> g_cu_count[kMaxDevices];   // 0 = not queried yet
std::atomic<int> g_cu_override{0};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

float default_floor(int fmt) {
  if (fmt == QCAST_FMT_E2M1) return 6.0f * 0x1.0p-126f;   // E2M1 maximum times 2^-126
  return 1e-4f;   // E4M3; E5M2 and E5M6 take the same floor
}

bool any_fmt(int fmt) {
  return fmt == QCAST_FMT_E4M3 || fmt == QCAST_FMT_E2M1 || fmt == QCAST_FMT_E5M2 ||
         fmt == QCAST_FMT_E5M6;
}

float floor_for(int fmt, float clamp_min) {
  return clamp_min > 0.0f ? clamp_min : default_floor(fmt);
}

// A caller's floor must be a number below +inf: NaN would silently select the
// default, and +inf would make every scale infinite (and, rounded to a power
// of two, wrap its inverse's exponent).
bool clamp_min_ok(float c) { return c == c && c <= 3.4028235e38f; }

int caps_for_current_device(qcast::LaunchCaps* caps) {
  const int override_n = g_cu_override.load(std::memory_order_relaxed);
  if (override_n > 0) {
    caps->num_cus = override_n;
    return QCAST_OK;
  }
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return QCAST_ERR_DEVICE;
  if (dev < kMaxDevices) {
    int n = g_cu_count[dev].load(std::memory_order_relaxed);
    if (n <= 0) {
      if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess ||
          n <= 0)
        return QCAST_ERR_DEVICE;
      g_cu_count[dev].store(n, std::memory_order_relaxed);
    }
    caps->num_cus = n;
    return QCAST_OK;
  }
  int n = 0;
  if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0)
    return QCAST_ERR_DEVICE;
  caps->num_cus = n;
  return QCAST_OK;
}

int finish(hipError_t err) { return err == hipSuccess ? QCAST_OK : QCAST_ERR_LAUNCH; }

// Device address of `scratch` on the current device, looked up once per
// device (with that device current) and kept.
std::atomic<void*> g_scratch_ptr[kMaxDevices];
std::mutex g_scratch_mu;

int scratch_for_current_device(unsigned long long** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return QCAST_ERR_DEVICE;
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (!p) {
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    p = g_scratch_ptr[dev].load(std::memory_order_relaxed);
    if (!p) {
      if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p)
        return QCAST_ERR_DEVICE;
      g_scratch_ptr[dev].store(p, std::memory_order_release);
    }
  }
  *out = static_cast<unsigned long long*>(p);
  return QCAST_OK;
}

// Zeroes n 64-bit words (a fill kernel, not a memset: a caller may capture
// the call in a graph).
__global__ __launch_bounds__(qcast::kThreads) void zero_words(unsigned long long* p, int n) {
  for (int i = threadIdx.x; i < n; i += qcast::kThreads) p[i] = 0ull;
}

// A clamp bound of +inf clamps nothing; so does any bound <= 0.
float clamp_value(float c) { return (c > 0.0f && c <= 3.4028235e38f) ? c : 0.0f; }

bool per_token_group_ok(int group) { return group == 32 || group == 64 || group == 128; }

bool sf_flags_ok(int flags) {
  return (flags & ~(QCAST_SF_ROUND_POW2 | QCAST_SF_COL_MAJOR | QCAST_SF_PACKED_UE8M0)) == 0;
}

// Group indices are 32-bit in the scale store; packed words need whole
// quadruples of groups in every row.
bool sf_shape_ok(int64_t rows, int64_t cols, int group, int flags) {
  if (cols > 0 && rows > ((int64_t(1) << 31) - 1) / (cols / group > 0 ? cols / group : 1))
    return false;
  if ((flags & QCAST_SF_PACKED_UE8M0) && (cols / group) % 4 != 0) return false;
  return true;
}

// Element counts beyond 2^62 would overflow the kernels' int64 offsets.
bool too_big(int64_t rows, int64_t cols) {
  return cols > 0 && rows > (int64_t(1) << 62) / cols;
}

// Argument checks of the per-token SwiGLU casts, before any HIP call;
// *empty when the call casts nothing (and launches nothing).
int check_swiglu_ex(const void* h, int64_t rows, int64_t cols, const float* row_weight, int fmt,
                    int group, float clamp_min, int sf_flags, float swiglu_clamp, const void* q,
                    const void* sf, const uint64_t* clamp_count, const void* count_ws,
                    bool* empty) {
  *empty = false;
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(group)) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % group != 0 || cols / 8 >= (int64_t(1) << 16) ||
      too_big(rows, 2 * cols) || !sf_shape_ok(rows, cols, group, sf_flags))
    return QCAST_ERR_SHAPE;
  if (swiglu_clamp != swiglu_clamp) return QCAST_ERR_VALUE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) {
    *empty = true;
    return QCAST_OK;
  }
  if (!h || !q || !sf) return QCAST_ERR_NULL;
  if (!aligned(h, 16) || !aligned(q, 16) || !aligned(sf, 4) ||
      (row_weight && !aligned(row_weight, 4)) || (clamp_count && !aligned(clamp_count, 8)) ||
      (count_ws && !aligned(count_ws, 128)))
    return QCAST_ERR_ALIGN;
  return QCAST_OK;
}

bool fp8_fmt(int fmt) { return fmt == QCAST_FMT_E4M3 || fmt == QCAST_FMT_E5M2; }

bool finite_value(float v) { return v == v && v >= -3.4028235e38f && v <= 3.4028235e38f; }

// QCAST_OK where there is a device to launch on.
int device_ok() {
  qcast::LaunchCaps caps;
  return caps_for_current_device(&caps);
}

static_assert(QCAST_NORM_MAX_COLS == 8 * qcast::kNormMaxChunks, "longest row of the norms");

// The scalar arguments of the norm entry points; `saved_fmt` is the format
// of 8-bit checkpoints, 0 for none.
int check_norm(int64_t rows, int64_t cols, int fmt, int group, float clamp_min, int sf_flags,
               int gate_kind, float residual_scale, float weight_offset, int saved_fmt) {
  if (!any_fmt(fmt) || (saved_fmt != 0 && !fp8_fmt(saved_fmt))) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(group)) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % group != 0 || cols > QCAST_NORM_MAX_COLS ||
      rows >= (int64_t(1) << 31) || (saved_fmt != 0 && cols % 128 != 0) ||
      !sf_shape_ok(rows, cols, group, sf_flags))
    return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min) || !finite_value(residual_scale) || !finite_value(weight_offset) ||
      gate_kind < QCAST_GATE_NONE || gate_kind > QCAST_GATE_FULL)
    return QCAST_ERR_VALUE;
  return QCAST_OK;
}

}  // namespace

extern "C" {

int qcast_abi_version(void) { return QCAST_ABI_VERSION; }

const char* qcast_status_str(int status) {
  switch (status) {
    case QCAST_OK: return "ok";
    case QCAST_ERR_NULL: return "a required pointer is NULL";
    case QCAST_ERR_SHAPE:
      return "unsupported shape (negative, not divisible as required, or past the 32-bit "
             "indexing limits)";
    case QCAST_ERR_ALIGN: return "pointer not aligned as required";
    case QCAST_ERR_FORMAT: return "format not supported by this entry point";
    case QCAST_ERR_GROUP: return "group or block size not supported";
    case QCAST_ERR_LAUNCH: return "kernel launch failed";
    case QCAST_ERR_DEVICE: return "no usable HIP device";
    case QCAST_ERR_VALUE: return "a scalar argument is out of range";
  }
  return "unknown status";
}

void qcast_set_num_cus(int n) { g_cu_override.store(n > 0 ? n : 0, std::memory_order_relaxed); }

int qcast_per_token_sf(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                       float clamp_min, int sf_flags, void* q, void* sf, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(group)) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % group != 0 || too_big(rows, cols) ||
      !sf_shape_ok(rows, cols, group, sf_flags))
    return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!x || !q || !sf) return QCAST_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_per_token(x, rows, cols, fmt, group, floor_for(fmt, clamp_min),
                                        (uint32_t)sf_flags, q, sf,
                                        static_cast<hipStream_t>(stream), caps));
}

int qcast_per_token(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                    float clamp_min, void* q, float* sf, void* stream) {
  return qcast_per_token_sf(x, rows, cols, fmt, group, clamp_min, 0, q, sf, stream);
}

int qcast_e2m1(const void* x, int64_t rows, int64_t cols, int group, float clamp_min,
               uint8_t* q_packed, float* sf, void* stream) {
  return qcast_per_token(x, rows, cols, QCAST_FMT_E2M1, group, clamp_min, q_packed, sf, stream);
}

int qcast_swiglu_per_token_ex(const void* h, int64_t rows, int64_t cols,
                              const float* row_weight, int fmt, int group, float clamp_min,
                              int sf_flags, float swiglu_clamp, void* q, void* sf,
                              uint64_t* clamp_count, void* count_ws, void* stream) {
  bool empty = false;
  int rc = check_swiglu_ex(h, rows, cols, row_weight, fmt, group, clamp_min, sf_flags,
                           swiglu_clamp, q, sf, clamp_count, count_ws, &empty);
  if (rc != QCAST_OK || empty) return rc;
  qcast::LaunchCaps caps;
  if ((rc = caps_for_current_device(&caps)) != QCAST_OK) return rc;
  return finish(qcast::launch_swiglu_per_token(
      h, rows, cols, row_weight, fmt, group, floor_for(fmt, clamp_min), (uint32_t)sf_flags,
      clamp_value(swiglu_clamp), reinterpret_cast<unsigned long long*>(clamp_count),
      static_cast<unsigned long long*>(count_ws), q, sf, static_cast<hipStream_t>(stream), caps));
}

int qcast_swiglu_per_token_noalloc(const void* h, int64_t rows, int64_t cols,
                                   const float* row_weight, int fmt, int group, float clamp_min,
                                   int sf_flags, float swiglu_clamp, void* q, void* sf,
                                   uint64_t* clamp_count, void* stream) {
  static_assert(sizeof(scratch) == QCAST_NOALLOC_SCRATCH_BYTES, "scratch size");
  bool empty = false;
  int rc = check_swiglu_ex(h, rows, cols, row_weight, fmt, group, clamp_min, sf_flags,
                           swiglu_clamp, q, sf, clamp_count, nullptr, &empty);
  if (rc != QCAST_OK || empty) return rc;
  // The count slots are reused by every slab of rows, so every shape needs
  // QCAST_COUNT_WS_BYTES of scratch, no more; a library built with a
  // smaller array refuses the counting call.
  const bool counting = clamp_count && clamp_value(swiglu_clamp) > 0.0f;
  if (counting && sizeof(scratch) < QCAST_COUNT_WS_BYTES) return QCAST_ERR_SHAPE;
  qcast::LaunchCaps caps;
  if ((rc = caps_for_current_device(&caps)) != QCAST_OK) return rc;
  unsigned long long* slots = nullptr;
  if (counting) {
    if ((rc = scratch_for_current_device(&slots)) != QCAST_OK) return rc;
    // The array keeps what the last call on this GPU left in it: clear the
    // slots on the stream, ahead of the cast.
    hipLaunchKernelGGL(zero_words, dim3(1), dim3(qcast::kThreads), 0,
                       static_cast<hipStream_t>(stream), slots,
                       (int)(QCAST_COUNT_WS_BYTES / sizeof(unsigned long long)));
    if (hipGetLastError() != hipSuccess) return QCAST_ERR_LAUNCH;
  }
  return finish(qcast::launch_swiglu_per_token(
      h, rows, cols, row_weight, fmt, group, floor_for(fmt, clamp_min), (uint32_t)sf_flags,
      clamp_value(swiglu_clamp), reinterpret_cast<unsigned long long*>(clamp_count), slots, q,
      sf, static_cast<hipStream_t>(stream), caps));
}

int qcast_swiglu_per_token_sf(const void* h, int64_t rows, int64_t cols,
                              const float* row_weight, int fmt, int group, float clamp_min,
                              int sf_flags, void* q, void* sf, void* stream) {
  return qcast_swiglu_per_token_ex(h, rows, cols, row_weight, fmt, group, clamp_min, sf_flags,
                                   0.0f, q, sf, nullptr, nullptr, stream);
}

int qcast_swiglu_backward_per_token_sf(const void* h, const void* dv, int64_t rows,
                                       int64_t cols, const float* row_weight, int fmt, int group,
                                       float clamp_min, int sf_flags, float swiglu_clamp, void* q,
                                       void* sf, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(group)) return QCAST_ERR_GROUP;
  // The scales are those of rows of 2 * cols values; a packed word never
  // straddles the dg and du halves.
  if (rows < 0 || cols < 0 || cols % group != 0 || cols / 8 >= (int64_t(1) << 16) ||
      too_big(rows, 2 * cols) || !sf_shape_ok(rows, 2 * cols, group, sf_flags) ||
      ((sf_flags & QCAST_SF_PACKED_UE8M0) && (cols / group) % 4 != 0))
    return QCAST_ERR_SHAPE;
  if (swiglu_clamp != swiglu_clamp) return QCAST_ERR_VALUE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!h || !dv || !q || !sf) return QCAST_ERR_NULL;
  if (!aligned(h, 16) || !aligned(dv, 16) || !aligned(q, 16) || !aligned(sf, 4) ||
      (row_weight && !aligned(row_weight, 4)))
    return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_swiglu_backward(
      h, dv, rows, cols, row_weight, fmt, group, floor_for(fmt, clamp_min), (uint32_t)sf_flags,
      clamp_value(swiglu_clamp), q, sf, static_cast<hipStream_t>(stream), caps));
}

int qcast_swiglu_backward_per_token(const void* h, const void* dv, int64_t rows, int64_t cols,
                                    const float* row_weight, int fmt, int group, float clamp_min,
                                    float swiglu_clamp, void* q, float* sf, void* stream) {
  return qcast_swiglu_backward_per_token_sf(h, dv, rows, cols, row_weight, fmt, group, clamp_min,
                                            0, swiglu_clamp, q, sf, stream);
}

int qcast_swiglu_per_channel_T_sf(const void* h, int64_t rows, int64_t cols,
                                  const float* row_weight, int fmt, int group, float clamp_min,
                                  int sf_flags, float swiglu_clamp, void* qT, void* sf,
                                  uint64_t* clamp_count, void* count_ws, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (group != 128) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || rows % group != 0 || cols % 8 != 0 || too_big(rows, 2 * cols) ||
      !qcast::per_channel_t_fits(rows, cols, 2 * cols, fmt) ||
      ((sf_flags & QCAST_SF_PACKED_UE8M0) && (rows / group) % 4 != 0))
    return QCAST_ERR_SHAPE;
  if (swiglu_clamp != swiglu_clamp) return QCAST_ERR_VALUE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!h || !qT || !sf) return QCAST_ERR_NULL;
  if (!aligned(h, 16) || !aligned(qT, 16) || !aligned(sf, 4) ||
      (row_weight && !aligned(row_weight, 4)) || (clamp_count && !aligned(clamp_count, 8)) ||
      (count_ws && !aligned(count_ws, 128)))
    return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_swiglu_per_channel_T(
      h, rows, cols, row_weight, fmt, floor_for(fmt, clamp_min), (uint32_t)sf_flags,
      clamp_value(swiglu_clamp), reinterpret_cast<unsigned long long*>(clamp_count),
      static_cast<unsigned long long*>(count_ws), qT, sf, static_cast<hipStream_t>(stream),
      caps));
}

int qcast_swiglu_per_channel_T(const void* h, int64_t rows, int64_t cols, const float* row_weight,
                               int fmt, int group, float clamp_min, float swiglu_clamp, void* qT,
                               float* sf, uint64_t* clamp_count, void* count_ws,
                               void* stream) {
  return qcast_swiglu_per_channel_T_sf(h, rows, cols, row_weight, fmt, group, clamp_min, 0,
                                       swiglu_clamp, qT, sf, clamp_count, count_ws, stream);
}

int qcast_swiglu_per_token(const void* h, int64_t rows, int64_t cols, const float* row_weight,
                           int fmt, int group, float clamp_min, void* q, float* sf,
                           void* stream) {
  return qcast_swiglu_per_token_sf(h, rows, cols, row_weight, fmt, group, clamp_min, 0, q, sf,
                                   stream);
}

int qcast_per_block_sf(const void* x, int64_t rows, int64_t cols, int fmt, int block,
                       float clamp_min, int sf_flags, void* q, float* sf, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (sf_flags & ~QCAST_SF_ROUND_POW2) return QCAST_ERR_FORMAT;
  if (block != 128) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || rows % block != 0 || cols % block != 0 || too_big(rows, cols) ||
      !qcast::per_block_fits(rows, cols))
    return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!x || !q || !sf) return QCAST_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_per_block(x, rows, cols, fmt, floor_for(fmt, clamp_min),
                                        (uint32_t)sf_flags, q, sf,
                                        static_cast<hipStream_t>(stream), caps));
}

int qcast_per_block(const void* x, int64_t rows, int64_t cols, int fmt, int block,
                    float clamp_min, void* q, float* sf, void* stream) {
  return qcast_per_block_sf(x, rows, cols, fmt, block, clamp_min, 0, q, sf, stream);
}

int qcast_per_channel_T_sf(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                           float clamp_min, int sf_flags, void* qT, void* sf, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (group != 128) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || rows % group != 0 || cols % 8 != 0 || too_big(rows, cols) ||
      !qcast::per_channel_t_fits(rows, cols, cols, fmt) ||
      ((sf_flags & QCAST_SF_PACKED_UE8M0) && (rows / group) % 4 != 0))
    return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!x || !qT || !sf) return QCAST_ERR_NULL;
  if (!aligned(x, 16) || !aligned(qT, 16) || !aligned(sf, 4)) return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_per_channel_T(x, rows, cols, fmt, floor_for(fmt, clamp_min),
                                            (uint32_t)sf_flags, qT, sf,
                                            static_cast<hipStream_t>(stream), caps));
}

int qcast_per_channel_T(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                        float clamp_min, void* qT, float* sf, void* stream) {
  return qcast_per_channel_T_sf(x, rows, cols, fmt, group, clamp_min, 0, qT, sf, stream);
}

int qcast_per_channel_sf(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                         float clamp_min, int sf_flags, void* q, float* sf, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (sf_flags & ~QCAST_SF_ROUND_POW2) return QCAST_ERR_FORMAT;
  if (group != 128) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || rows % group != 0 || cols % 8 != 0 || too_big(rows, cols) ||
      !qcast::per_channel_fits(rows, cols))
    return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!x || !q || !sf) return QCAST_ERR_NULL;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(sf, 4)) return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_per_channel(x, rows, cols, fmt, floor_for(fmt, clamp_min),
                                          (uint32_t)sf_flags, q, sf,
                                          static_cast<hipStream_t>(stream), caps));
}

int qcast_per_channel(const void* x, int64_t rows, int64_t cols, int fmt, int group,
                      float clamp_min, void* q, float* sf, void* stream) {
  return qcast_per_channel_sf(x, rows, cols, fmt, group, clamp_min, 0, q, sf, stream);
}

int qcast_cast_back(const void* q, const float* sf, int64_t rows, int64_t cols, int fmt,
                    int group, int out_dtype, void* out, void* stream) {
  if (!any_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (out_dtype != QCAST_OUT_BF16 && out_dtype != QCAST_OUT_F32) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(group)) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % group != 0 || too_big(rows, cols) ||
      !qcast::cast_back_fits(rows, cols))
    return QCAST_ERR_SHAPE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!q || !sf || !out) return QCAST_ERR_NULL;
  if (!aligned(q, 16) || !aligned(sf, 4) || !aligned(out, 16)) return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  const int rc = caps_for_current_device(&caps);
  if (rc != QCAST_OK) return rc;
  return finish(qcast::launch_cast_back(q, sf, rows, cols, fmt, group, out_dtype == QCAST_OUT_BF16,
                                        out, static_cast<hipStream_t>(stream), caps));
}

int qcast_swiglu_checkpoint(const void* h, int64_t rows, int64_t cols, const float* row_weight,
                            int fmt, int group, float clamp_min, int sf_flags, float swiglu_clamp,
                            void* q, void* sf, int ckpt_fmt, void* ckpt, float* ckpt_sf,
                            void* stream) {
  bool empty;
  const int rc = check_swiglu_ex(h, rows, cols, row_weight, fmt, group, clamp_min, sf_flags,
                                 swiglu_clamp, q, sf, nullptr, nullptr, &empty);
  if (!fp8_fmt(ckpt_fmt)) return QCAST_ERR_FORMAT;
  if (rc != QCAST_OK) return rc;
  if (!sf_shape_ok(rows, 2 * cols, group, 0)) return QCAST_ERR_SHAPE;
  if (empty) return QCAST_OK;
  if (!ckpt || !ckpt_sf) return QCAST_ERR_NULL;
  if (!aligned(ckpt, 16) || !aligned(ckpt_sf, 4)) return QCAST_ERR_ALIGN;
  if (const int drc = device_ok()) return drc;
  return finish(qcast::launch_swiglu_checkpoint(
      h, rows, cols, row_weight, group, clamp_value(swiglu_clamp),
      qcast::make_row_cast(rows, cols, fmt, group, floor_for(fmt, clamp_min), (uint32_t)sf_flags,
                           q, sf),
      qcast::make_row_cast(rows, 2 * cols, ckpt_fmt, group, default_floor(ckpt_fmt), 0, ckpt,
                           ckpt_sf),
      static_cast<hipStream_t>(stream)));
}

int qcast_swiglu_backward_checkpoint(const void* ckpt, const float* ckpt_sf, const void* dv,
                                     int64_t rows, int64_t cols, const float* row_weight,
                                     int ckpt_fmt, int fmt, int group, float clamp_min,
                                     int sf_flags, float swiglu_clamp, void* q, void* sf,
                                     void* dhT, void* dhT_sf, void* vT, void* vT_sf, float* dw,
                                     void* ws, void* stream) {
  return qcast_swiglu_backward_checkpoint_ex(ckpt, ckpt_sf, dv, rows, cols, row_weight, ckpt_fmt,
                                             128, fmt, group, clamp_min, sf_flags, swiglu_clamp,
                                             q, sf, dhT, dhT_sf, vT, vT_sf, dw, ws, stream);
}

int qcast_swiglu_backward_checkpoint_ex(const void* ckpt, const float* ckpt_sf, const void* dv,
                                        int64_t rows, int64_t cols, const float* row_weight,
                                        int ckpt_fmt, int ckpt_group, int fmt, int group,
                                        float clamp_min, int sf_flags, float swiglu_clamp,
                                        void* q, void* sf, void* dhT, void* dhT_sf, void* vT,
                                        void* vT_sf, float* dw, void* ws, void* stream) {
  if (!fp8_fmt(fmt) || !fp8_fmt(ckpt_fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (group != 128 || !per_token_group_ok(ckpt_group)) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % 128 != 0 || too_big(rows, 2 * cols) ||
      !qcast::tile_fits(rows, cols, 2 * cols))
    return QCAST_ERR_SHAPE;
  const int64_t rows_T = (rows + 127) / 128 * 128;
  if (sf_flags & QCAST_SF_PACKED_UE8M0) {
    if ((cols / 128) % 4 != 0 || ((dhT || vT) && (rows_T / 128) % 4 != 0)) return QCAST_ERR_SHAPE;
  }
  if (swiglu_clamp != swiglu_clamp) return QCAST_ERR_VALUE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) {
    if (rows == 0 || !dw) return QCAST_OK;
    return QCAST_ERR_SHAPE;                       // dw over no columns
  }
  if (!ckpt || !ckpt_sf || !dv || !q || !sf || (dhT != nullptr) != (dhT_sf != nullptr) ||
      (vT != nullptr) != (vT_sf != nullptr) || (dw && cols > 128 && !ws))
    return QCAST_ERR_NULL;
  if (!aligned(ckpt, 16) || !aligned(ckpt_sf, 4) || !aligned(dv, 16) || !aligned(q, 16) ||
      !aligned(sf, 4) || !aligned(row_weight, 4) || !aligned(dhT, 16) || !aligned(dhT_sf, 4) ||
      !aligned(vT, 16) || !aligned(vT_sf, 4) || !aligned(dw, 4) || !aligned(ws, 16))
    return QCAST_ERR_ALIGN;
  if (const int drc = device_ok()) return drc;
  qcast::SwigluTile p{};
  p.ckpt = static_cast<const uint8_t*>(ckpt);
  p.ckpt_sf = ckpt_sf;
  p.dv = static_cast<const uint16_t*>(dv);
  p.w = row_weight;
  p.q = static_cast<uint8_t*>(q);
  p.sf = sf;
  p.lay = qcast::make_sf_layout(rows, 2 * cols, 128, (uint32_t)sf_flags);
  p.dh = qcast::TileCast{static_cast<uint8_t*>(dhT), dhT_sf,
                         qcast::make_sf_layout(2 * cols, rows_T, 128, (uint32_t)sf_flags)};
  p.v = qcast::TileCast{static_cast<uint8_t*>(vT), vT_sf,
                        qcast::make_sf_layout(cols, rows_T, 128, (uint32_t)sf_flags)};
  p.dw = dw;
  p.ws = static_cast<float*>(ws);
  p.floor = floor_for(fmt, clamp_min);
  p.clamp = clamp_value(swiglu_clamp);
  p.ckpt_shift = ckpt_group == 32 ? 2 : ckpt_group == 64 ? 3 : 4;
  p.rows = (uint32_t)rows;
  p.cols = (uint32_t)cols;
  return finish(qcast::launch_swiglu_backward_checkpoint(p, ckpt_fmt, fmt,
                                                         static_cast<hipStream_t>(stream)));
}

int qcast_recast_per_channel_T(const void* q_in, const float* sf_in, int64_t rows, int64_t cols,
                               int in_fmt, int in_group, int fmt, int group, float clamp_min,
                               int sf_flags, void* qT, void* sf, void* stream) {
  if (!fp8_fmt(in_fmt) || !fp8_fmt(fmt)) return QCAST_ERR_FORMAT;
  if (!sf_flags_ok(sf_flags)) return QCAST_ERR_FORMAT;
  if (!per_token_group_ok(in_group) || group != 128) return QCAST_ERR_GROUP;
  if (rows < 0 || cols < 0 || cols % in_group != 0 || too_big(rows, cols) ||
      !qcast::tile_fits(rows, cols, cols))
    return QCAST_ERR_SHAPE;
  const int64_t rows_T = (rows + 127) / 128 * 128;
  if ((sf_flags & QCAST_SF_PACKED_UE8M0) && (rows_T / 128) % 4 != 0) return QCAST_ERR_SHAPE;
  if (!clamp_min_ok(clamp_min)) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!q_in || !sf_in || !qT || !sf) return QCAST_ERR_NULL;
  if (!aligned(q_in, 16) || !aligned(sf_in, 4) || !aligned(qT, 16) || !aligned(sf, 4))
    return QCAST_ERR_ALIGN;
  if (const int drc = device_ok()) return drc;
  qcast::RecastTile p{};
  p.q = static_cast<const uint8_t*>(q_in);
  p.sf = sf_in;
  p.out = qcast::TileCast{static_cast<uint8_t*>(qT), sf,
                          qcast::make_sf_layout(cols, rows_T, 128, (uint32_t)sf_flags)};
  p.floor = floor_for(fmt, clamp_min);
  p.shift = in_group == 32 ? 2 : in_group == 64 ? 3 : 4;
  p.rows = (uint32_t)rows;
  p.cols = (uint32_t)cols;
  return finish(qcast::launch_recast(p, in_fmt, fmt, static_cast<hipStream_t>(stream)));
}

int qcast_norm_per_token(const void* y, const void* h, int64_t rows, int64_t cols,
                         const void* w_post, const void* w_pre, const void* gate, int gate_kind,
                         float residual_scale, float weight_offset, float eps, int fmt, int group,
                         float clamp_min, int sf_flags, void* h_out, void* q, void* sf,
                         void* x_out, float* rstd_post, float* rstd_pre, int ckpt_fmt,
                         void* y_ckpt, float* y_ckpt_sf, void* h_ckpt, float* h_ckpt_sf,
                         void* stream) {
  const bool ckpt = y_ckpt || y_ckpt_sf || h_ckpt || h_ckpt_sf;
  if (ckpt && !fp8_fmt(ckpt_fmt)) return QCAST_ERR_FORMAT;
  int rc = check_norm(rows, cols, fmt, group, clamp_min, sf_flags, gate_kind, residual_scale,
                      weight_offset, ckpt ? ckpt_fmt : 0);
  if (rc != QCAST_OK) return rc;
  if (!(eps >= 0.0f) || !finite_value(eps)) return QCAST_ERR_VALUE;
  if (!y && residual_scale != 1.0f) return QCAST_ERR_VALUE;
  if (rows == 0 || cols == 0) return QCAST_OK;
  if (!h || !w_pre || (q != nullptr) != (sf != nullptr) || (!q && !x_out) ||
      (gate != nullptr) != (gate_kind != QCAST_GATE_NONE) || (y != nullptr) != (h_out != nullptr) ||
      (!y && (w_post || gate || y_ckpt)) || (!w_post && rstd_post) ||
      (y_ckpt != nullptr) != (y_ckpt_sf != nullptr) ||
      (h_ckpt != nullptr) != (h_ckpt_sf != nullptr))
    return QCAST_ERR_NULL;
  if (!aligned(y, 16) || !aligned(h, 16) || !aligned(w_post, 16) || !aligned(w_pre, 16) ||
      !aligned(gate, gate_kind == QCAST_GATE_TOKEN ? 4 : 16) || !aligned(h_out, 16) ||
      !aligned(q, 16) || !aligned(sf, 4) || !aligned(x_out, 16) || !aligned(rstd_post, 4) ||
      !aligned(rstd_pre, 4) || !aligned(y_ckpt, 16) || !aligned(y_ckpt_sf, 4) ||
      !aligned(h_ckpt, 16) || !aligned(h_ckpt_sf, 4))
    return QCAST_ERR_ALIGN;
  qcast::LaunchCaps caps;
  if (const int crc = caps_for_current_device(&caps)) return crc;
  qcast::NormForward p{};
  p.y = static_cast<const uint16_t*>(y);
  p.h = static_cast<const uint16_t*>(h);
  p.w_post = static_cast<const uint16_t*>(w_post);
  p.w_pre = static_cast<const uint16_t*>(w_pre);
  p.gate = gate;
  p.h_out = static_cast<uint16_t*>(h_out);
  p.x_out = static_cast<uint16_t*>(x_out);
  p.rstd_post = rstd_post;
  p.rstd_pre = rstd_pre;
  p.cast = qcast::make_row_cast(rows, cols, fmt, group, floor_for(fmt, clamp_min),
                                (uint32_t)sf_flags, q, sf);
  p.y_ckpt = qcast::make_row_cast(rows, cols, ckpt_fmt, 128, default_floor(ckpt_fmt), 0, y_ckpt,
                                  y_ckpt_sf);
  p.h_ckpt = qcast::make_row_cast(rows, cols, ckpt_fmt, 128, default_floor(ckpt_fmt), 0, h_ckpt,
                                  h_ckpt_sf);
  p.gate_kind = gate_kind;
  p.alpha = residual_scale;
  p.offset = weight_offset;
  p.eps = eps;
  p.inv_n = 1.0f / (float)cols;
  p.chunks = (uint32_t)(cols / 8);
  return finish(qcast::launch_norm(p, rows, static_cast<hipStream_t>(stream), caps));
}

int qcast_norm_backward_per_token(const void* dx, const void* dh_in, int64_t rows, int64_t cols,
                                  int saved_fmt, const void* saved_h, const float* saved_h_sf,
                                  const void* saved_y, const float* saved_y_sf,
                                  const float* rstd_post, const float* rstd_pre,
                                  const void* w_post, const void* w_pre, const void* gate,
                                  int gate_kind, float residual_scale, float weight_offset,
                                  int fmt, int group, float clamp_min, int sf_flags,
                                  void* dh_out, void* q, void* sf, void* dy_out, float* dw_post,
                                  float* dw_pre, void* dgate, void* ws, void* stream) {
  const int rc = check_norm(rows, cols, fmt, group, clamp_min, sf_flags, gate_kind,
                            residual_scale, weight_offset, saved_fmt);
  if (rc != QCAST_OK) return rc;
  if (cols == 0)                                  // a token gate's sums over no columns
    return rows > 0 && gate_kind == QCAST_GATE_TOKEN && dgate ? QCAST_ERR_SHAPE : QCAST_OK;
  const bool saved8 = saved_fmt != 0;
  if (rows > 0) {
    if (!dx || !saved_h || !rstd_pre || !w_pre || !dh_out || (saved8 && !saved_h_sf) ||
        (!saved8 && (saved_h_sf || saved_y_sf)) || (saved8 && (saved_y != nullptr) !=
        (saved_y_sf != nullptr)) || (rstd_post != nullptr) != (w_post != nullptr) ||
        (gate != nullptr) != (gate_kind != QCAST_GATE_NONE) ||
        (q != nullptr) != (sf != nullptr) || (saved_y && !q && !dy_out) ||
        (!saved_y && (w_post || gate || q || dy_out)) || !ws)
      return QCAST_ERR_NULL;
  }
  // these read the channel gate and w_post even where there are no rows
  if ((dw_post && !w_post) || (dgate && !gate) || (gate_kind == QCAST_GATE_CHANNEL && !gate))
    return QCAST_ERR_NULL;
  const int gate_align = gate_kind == QCAST_GATE_TOKEN ? 4 : 16;
  if (!aligned(dx, 16) || !aligned(dh_in, 16) || !aligned(saved_h, 16) ||
      !aligned(saved_h_sf, 4) || !aligned(saved_y, 16) || !aligned(saved_y_sf, 4) ||
      !aligned(rstd_post, 4) || !aligned(rstd_pre, 4) || !aligned(w_post, 16) ||
      !aligned(w_pre, 16) || !aligned(gate, gate_align) || !aligned(dh_out, 16) ||
      !aligned(q, 16) || !aligned(sf, 4) || !aligned(dy_out, 16) || !aligned(dw_post, 16) ||
      !aligned(dw_pre, 16) || !aligned(dgate, gate_align) || !aligned(ws, 16))
    return QCAST_ERR_ALIGN;
  const bool channel = gate_kind == QCAST_GATE_CHANNEL;
  if (rows == 0 && !dw_pre && !dw_post && !(channel && dgate)) return QCAST_OK;
  if (const int drc = device_ok()) return drc;
  qcast::NormBackward p{};
  p.dx = static_cast<const uint16_t*>(dx);
  p.dh_in = static_cast<const uint16_t*>(dh_in);
  p.saved_h = saved_h;
  p.saved_h_sf = saved_h_sf;
  p.saved_y = saved_y;
  p.saved_y_sf = saved_y_sf;
  p.rstd_pre = rstd_pre;
  p.rstd_post = rstd_post;
  p.w_post = static_cast<const uint16_t*>(w_post);
  p.w_pre = static_cast<const uint16_t*>(w_pre);
  p.gate = gate;
  p.dh_out = static_cast<uint16_t*>(dh_out);
  p.dy_out = static_cast<uint16_t*>(dy_out);
  p.sums[0] = dw_pre;
  p.sums[1] = dw_post;
  p.sums[2] = channel ? static_cast<float*>(dgate) : nullptr;
  p.dgate = dgate;
  p.ws = static_cast<float*>(ws);
  p.cast = qcast::make_row_cast(rows, cols, fmt, group, floor_for(fmt, clamp_min),
                                (uint32_t)sf_flags, q, sf);
  p.saved_fmt = saved_fmt;
  p.gate_kind = gate_kind;
  p.alpha = residual_scale;
  p.offset = weight_offset;
  p.inv_n = 1.0f / (float)cols;
  p.chunks = (uint32_t)(cols / 8);
  return finish(qcast::launch_norm_backward(p, rows, (uint32_t)qcast_norm_ws_rows(rows, cols),
                                            static_cast<hipStream_t>(stream)));
}

}  // extern "C"
