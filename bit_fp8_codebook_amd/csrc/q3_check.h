// Host-side checks and layout arithmetic shared by the C ABI's entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstring>

#include "../../include/q3.h"
#include "q3_internal.h"

namespace q3::check {

inline constexpr int64_t kGroup = 32;
inline constexpr int64_t kMaxPlaneBytes = (int64_t(1) << 31) - (int64_t(1) << 24);   // per plane, and for x

inline int64_t padded_groups(int64_t k) { return (k / kGroup + 3) / 4 * 4; }
inline int64_t tiles_of(int64_t n) { return (n + 15) / 16; }
inline int64_t code_plane_bytes(int64_t n, int64_t k) { return tiles_of(n) * 192 * padded_groups(k); }
inline int64_t scale_plane_bytes(int64_t n, int64_t k) { return tiles_of(n) * 16 * padded_groups(k); }
inline int64_t code_plane_bytes2(int64_t n, int64_t k) { return tiles_of(n) * 128 * padded_groups(k); }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline q3_status check_shape(int64_t n, int64_t k) {
  if (n < 0) return Q3_ERR_INVALID_ARG;
  if (k <= 0 || k % kGroup != 0 || k > (int64_t(1) << 30)) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (n > (int64_t(1) << 31)) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

// Packed planes of one matrix: pointers present, aligned, addressable.
inline q3_status check_planes(int64_t n, int64_t k, const void* code, const void* scale, const void* cb) {
  q3_status st = check_shape(n, k);
  if (st != Q3_OK) return st;
  if (n > 0 && (!code || !scale || !cb)) return Q3_ERR_INVALID_ARG;
  if (!aligned(code, 16) || !aligned(scale, 4) || !aligned(cb, 8)) return Q3_ERR_MISALIGNED;
  // The kernels address each plane through a 32-bit buffer resource.
  if (code_plane_bytes(n, k) > kMaxPlaneBytes || n * 8 > kMaxPlaneBytes) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

// The two-bit draft head's planes: 4-byte codebook rows.
inline q3_status check_planes2(int64_t n, int64_t k, const void* code, const void* scale, const void* cb) {
  q3_status st = check_shape(n, k);
  if (st != Q3_OK) return st;
  if (n > 0 && (!code || !scale || !cb)) return Q3_ERR_INVALID_ARG;
  if (!aligned(code, 16) || !aligned(scale, 4) || !aligned(cb, 4)) return Q3_ERR_MISALIGNED;
  if (code_plane_bytes2(n, k) > kMaxPlaneBytes || n * 4 > kMaxPlaneBytes) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

inline q3_status check_mxfp8(const q3_mxfp8_matrix* h) {
  if (!h) return Q3_ERR_INVALID_ARG;
  q3_status st = check_shape(h->n, h->k);
  if (st != Q3_OK) return st;
  if (h->n < 1 || !h->elements || !h->scales) return Q3_ERR_INVALID_ARG;
  if (h->ld_elements < h->k || h->ld_scales < h->k / kGroup) return Q3_ERR_INVALID_ARG;
  if (h->ld_elements % 16 || !aligned(h->elements, 16)) return Q3_ERR_MISALIGNED;
  if (h->n * h->ld_elements > kMaxPlaneBytes || h->n * h->ld_scales > kMaxPlaneBytes) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

inline q3_status check_matrix(const q3_matrix* w) {
  if (!w) return Q3_ERR_INVALID_ARG;
  return check_planes(w->n, w->k, w->code_plane, w->scale_plane, w->codebook);
}

inline q3_status check_tokens(int64_t k, int64_t n, const uint16_t* x, int64_t m, int64_t ldx, const float* y,
                       int64_t ldy, int64_t m_max) {
  if (m < 1 || m > m_max) return Q3_ERR_UNSUPPORTED_SHAPE;
  if (!x || (!y && n > 0)) return Q3_ERR_INVALID_ARG;
  if (ldx < k || ldy < n) return Q3_ERR_INVALID_ARG;
  if (ldx % 8 || !aligned(x, 16) || !aligned(y, 4)) return Q3_ERR_MISALIGNED;
  if ((m - 1) * ldx * 2 + k * 2 > kMaxPlaneBytes) return Q3_ERR_UNSUPPORTED_SHAPE;
  return Q3_OK;
}

// gfx950 check, once per device (the only global state of the library).
inline std::atomic<int> g_device_ok[64];

inline q3_status check_device() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return Q3_ERR_HIP;
  if (dev < 0 || dev >= 64) return Q3_ERR_UNSUPPORTED_DEVICE;
  int state = g_device_ok[dev].load(std::memory_order_acquire);
  if (state == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return Q3_ERR_HIP;
    state = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    g_device_ok[dev].store(state, std::memory_order_release);
  }
  return state == 1 ? Q3_OK : Q3_ERR_UNSUPPORTED_DEVICE;
}

inline q3_status from_hip(hipError_t e) { return e == hipSuccess ? Q3_OK : Q3_ERR_HIP; }

inline q3::PlaneView view_of(const q3_matrix* w) {
  q3::PlaneView v;
  v.code = static_cast<const uint8_t*>(w->code_plane);
  v.scale = static_cast<const uint8_t*>(w->scale_plane);
  v.cb = static_cast<const uint8_t*>(w->codebook);
  v.n = w->n;
  v.groups = static_cast<int32_t>(w->k / kGroup);
  return v;
}

}  // namespace q3::check
