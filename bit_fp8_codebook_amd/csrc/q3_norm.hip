// Residual norms: the end of one block and the start of the next.
//
//   t  = post_w * y * rsqrt(mean(y^2) + eps)   (or y)
//   r' = r + scale * gate * t
//   x  = pre_w * r' * rsqrt(mean(r'^2) + eps)
//
// and the backward pass, with s, sy the two reciprocal roots, h = r' s,
// yh = y sy and a = dx pre_w:
//   G    = dr' + s (a - h mean(a h))          the gradient of r' and of r
//   dt   = scale gate G,  b = dt post_w
//   dy   = sy (b - yh mean(b yh))             (dt without a post norm)
//   dgate = scale t G, dpost_w = sum dt yh, dpre_w = sum dx h
//
// Both are bound by memory: each row is read once into registers (8 elements
// per thread up to 8192 columns, 12 or 16 above), reduced, and written once.  A
// row belongs to a group of T threads, the smallest of 64..1024 with 8 T >= n;
// up to 512 columns that is one wave, so a 256-thread block takes four rows and
// no reduction crosses a wave.  The backward pass sums its weight gradients over
// tokens in LDS, or past 12288 columns, where three rows of sums do not fit, in the
// partial rows themselves: a fixed number of groups walks the rows, each leaves one
// partial row per gradient, and a second launch adds those in group order (no
// atomics, so the same call gives the same bits).  All statistics and sums are fp32.
// Measured: 8192 x 8192 fp32 forward 213 us (5.7 TB/s), backward 379 + 5 us (5.3
// TB/s); 2047 x 5120 bf16 backward 41 + 6 us, of which the partial rows are a
// quarter of the bytes; 1 x 4096 forward 2.8 us.  4096 rows backward, fp32: 12288
// columns 192 us (5.8 TB/s), 12292 454, 16384 522 (2.8 TB/s: the sums move with
// every row).
#include <type_traits>

#include "q3_device.h"
#include "../../include/q3_block.h"
#include "q3_internal.h"

namespace q3 {
namespace {

constexpr int kMaxGroups = 262144;  // threads of the backward pass over all groups

template <int T>
constexpr int rows_per_block() { return T == 64 ? 4 : 1; }
template <int T>
constexpr int block_threads() { return T == 64 ? 256 : T; }

__device__ __forceinline__ uint32_t bf16_bits(float a, float b) {
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

// A row as a buffer resource: columns past n and every column of a null row
// read as zero and are not stored, with no
// branch and one register of address per thread.  The base is wave-uniform.
template <typename E>
__device__ __forceinline__ rsrc_t row_of(const E* base, int64_t row, int64_t ld, int n) {
  return make_rsrc(base ? base + row * ld : nullptr, base ? (uint32_t)n * sizeof(E) : 0u);
}

// A thread's EL elements of a row, V (1 or 4) consecutive ones at a time, as
// they were loaded (bf16 vectors stay packed until they are used).
template <int V, int EL, typename E>
struct Loaded {
  static constexpr bool kPacked = V == 4 && sizeof(E) == 2;
  uint32_t w[kPacked ? EL / 2 : EL];
  __device__ __forceinline__ float at(int e) const {
    if constexpr (kPacked) return __builtin_bit_cast(float, e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16);
    else if constexpr (sizeof(E) == 2) return __builtin_bit_cast(float, w[e] << 16);
    else return __builtin_bit_cast(float, w[e]);
  }
};
template <int T, int V, int EL, typename E>
__device__ __forceinline__ void fetch(rsrc_t row, int t, Loaded<V, EL, E>& o) {
  const uint32_t at = (uint32_t)(t * V) * sizeof(E);
#pragma unroll
  for (int c = 0; c < EL / V; ++c) {
    const uint32_t off = at + (uint32_t)(c * T * V) * sizeof(E);
    if constexpr (V == 4 && sizeof(E) == 4) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(row, off, 0, 0);
#pragma unroll
      for (int e = 0; e < 4; ++e) o.w[4 * c + e] = v[e];
    } else if constexpr (V == 4) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(row, off, 0, 0);
      o.w[2 * c] = v.x;
      o.w[2 * c + 1] = v.y;
    } else if constexpr (sizeof(E) == 4) {
      o.w[c] = __builtin_amdgcn_raw_buffer_load_b32(row, off, 0, 0);
    } else {
      o.w[c] = __builtin_amdgcn_raw_buffer_load_b16(row, off, 0, 0);
    }
  }
}
template <int T, int V, int EL, typename E>
__device__ __forceinline__ void store_row(rsrc_t row, int t, const float (&v)[EL], E) {
  const uint32_t at = (uint32_t)(t * V) * sizeof(E);
#pragma unroll
  for (int c = 0; c < EL / V; ++c) {
    const uint32_t off = at + (uint32_t)(c * T * V) * sizeof(E);
    const float* p = v + c * V;
    if constexpr (V == 4 && sizeof(E) == 4) {
      u32x4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __builtin_bit_cast(uint32_t, p[e]);
      __builtin_amdgcn_raw_buffer_store_b128(u, row, off, 0, 0);
    } else if constexpr (V == 4) {
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_bits(p[0], p[1]), bf16_bits(p[2], p[3])}, row, off, 0, 0);
    } else if constexpr (sizeof(E) == 4) {
      __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, p[0]), row, off, 0, 0);
    } else {
      __builtin_amdgcn_raw_buffer_store_b16((uint16_t)bf16_bits(p[0], 0.f), row, off, 0, 0);
    }
  }
}
// A weight row; ones without one.
template <int T, int V, int EL>
__device__ __forceinline__ void weights(const float* w, int n, int t, float (&o)[EL]) {
  Loaded<V, EL, float> v;
  fetch<T>(row_of(w, 0, 0, n), t, v);
#pragma unroll
  for (int e = 0; e < EL; ++e) o[e] = w ? v.at(e) : 1.f;
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off > 0; off /= 2) v += __shfl_xor(v, off, 64);
  return v;
}

// Sums of K values over the group; every thread gets them.  `red` holds
// K * 16 floats; two calls in a row need different buffers (one barrier each).
template <int T, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* red, int t) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    if ((t & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * W + (t >> 6)] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) s += red[k * W + w];
      v[k] = s;
    }
  }
}

template <typename E, int V, int T, int EL>
__global__ __launch_bounds__(block_threads<T>()) void residual_norm_kernel(NormArgs a) {
  __shared__ float red[2][16];
  const int t = threadIdx.x % T;
  const int64_t row = (int64_t)blockIdx.x * rows_per_block<T>() + __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  if (row >= a.m) return;   // whole groups; T == 64 has no barriers
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  Loaded<V, EL, E> in;
  Loaded<V, EL, float> y, g;
  fetch<T>(row_of(a.y, row, a.ldy, n), t, y);
  fetch<T>(row_of(static_cast<const E*>(a.r), row, a.ldr, n), t, in);
  fetch<T>(row_of(a.gate, row, a.ld_gate, n), t, g);
  float w[EL], r[EL];
  weights<T, V, EL>(a.post_w, n, t, w);
  float sy = 1.f;
  if (a.post_w) {
    float q[1] = {0.f};
#pragma unroll
    for (int e = 0; e < EL; ++e) q[0] += y.at(e) * y.at(e);
    group_sum<T>(q, red[0], t);
    sy = rsqrtf(q[0] * inv_n + a.eps);
  }
#pragma unroll
  for (int e = 0; e < EL; ++e) {
    const float u = a.scale * (y.at(e) * sy * w[e]);
    r[e] = in.at(e);
    if (a.y) r[e] += a.gate ? u * g.at(e) : u;
  }
  if (a.r_out && (a.y || a.r_out != a.r))
    store_row<T, V, EL>(row_of(static_cast<E*>(a.r_out), row, a.ldr_out, n), t, r, E{});
  if (a.x) {
    float q[1] = {0.f};
    weights<T, V, EL>(a.pre_w, n, t, w);
#pragma unroll
    for (int e = 0; e < EL; ++e) q[0] += r[e] * r[e];
    group_sum<T>(q, red[1], t);
    const float s = rsqrtf(q[0] * inv_n + a.eps);
#pragma unroll
    for (int e = 0; e < EL; ++e) w[e] *= r[e] * s;
    store_row<T, V, EL>(row_of(a.x, row, a.ldx, n), t, w, uint16_t{});
  }
}

// A group's sums over its rows.  Each thread adds to its own columns only, so
// nothing is shared and no barrier is needed.  Up to 12288 columns they live in
// LDS; above, where three rows would not fit, in the group's partial rows.
template <int T, int V, int EL>
__device__ __forceinline__ void add_own(float* acc, int n, int t, const float (&v)[EL]) {
#pragma unroll
  for (int c = 0; c < EL / V; ++c) {
    const int col = (c * T + t) * V;
    if (EL == 16 && col >= n) continue;   // LDS rows are whole
    float* p = acc + col;
    if constexpr (V == 4) {
      f32x4 x = *reinterpret_cast<f32x4*>(p);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] += v[4 * c + e];
      *reinterpret_cast<f32x4*>(p) = x;
    } else {
      *p += v[c];
    }
  }
}

// All of a row's loads are issued at its start.  Two or more groups share a CU
// up to 6144 columns, so one loads while another reduces (2047 x 5120 bf16 in
// one group of 1024 threads per CU: 72 us, 2.2 TB/s); with the sums in LDS the
// rest fits 128 registers.  Loading the next row ahead into registers as well
// spills, and the spills wait for the very loads (8192 x 8192: 397 -> 576 us).
template <typename E, int V, int T, int EL>
__global__ __launch_bounds__(block_threads<T>()) __attribute__((amdgpu_waves_per_eu(4)))
void residual_norm_back_kernel(NormBackArgs a) {
  __shared__ float red[2][48];
  extern __shared__ __align__(16) float sums[];   // [groups of the block][3][T * EL]
  const int t = threadIdx.x % T;
  const int64_t group =
      (int64_t)blockIdx.x * rows_per_block<T>() + __builtin_amdgcn_readfirstlane(threadIdx.x / T);
  if (group >= a.groups) return;
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  constexpr bool kLds = EL < 16;
  constexpr bool kKeep = T * EL <= 8192;   // weights in registers; above, read again for each row
  float* part[3] = {a.part_pre, a.part_post, a.part_gate};
  float* acc[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    acc[k] = kLds ? sums + ((threadIdx.x / T) * 3 + k) * (T * EL) : part[k] + group * n;
#pragma unroll
    for (int c = 0; c < EL / V; ++c) {
      const int col = (c * T + t) * V;
      if (kLds || (part[k] && col < n)) {
#pragma unroll
        for (int e = 0; e < V; ++e) acc[k][col + e] = 0.f;
      }
    }
  }

  float pre_w[EL], post_w[EL];
  if constexpr (kKeep) {
    weights<T, V, EL>(a.pre_w, n, t, pre_w);
    weights<T, V, EL>(a.post_w, n, t, post_w);
  }
  const bool gates = a.gate != nullptr;
  struct Row {
    Loaded<V, EL, E> r, dr;
    Loaded<V, EL, float> da, y, g;
  };
  auto load = [&](int64_t row, Row& o) {
    fetch<T>(row_of(static_cast<const E*>(a.r), row, a.ldr, n), t, o.r);
    fetch<T>(row_of(a.dx, row, a.ld_dx, n), t, o.da);
    fetch<T>(row_of(a.y, row, a.ldy, n), t, o.y);
    fetch<T>(row_of(static_cast<const E*>(a.dr_out), row, a.ld_dr_out, n), t, o.dr);
    fetch<T>(row_of(a.gate, row, a.ld_gate, n), t, o.g);
  };
  for (int64_t row = group; row < a.m; row += a.groups) {
    Row cur;
    load(row, cur);
    const auto& r = cur.r;
    const auto& dr = cur.dr;
    const auto& da = cur.da;
    const auto& y = cur.y;
    const auto& g = cur.g;
    if constexpr (!kKeep) weights<T, V, EL>(a.pre_w, n, t, pre_w);
    float q[3] = {0.f, 0.f, 0.f};
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      q[0] += r.at(e) * r.at(e);
      q[1] += da.at(e) * pre_w[e] * r.at(e);
      q[2] += y.at(e) * y.at(e);
    }
    group_sum<T>(q, red[0], t);
    const float s = rsqrtf(q[0] * inv_n + a.eps), c1 = q[1] * inv_n * s;
    float grad[EL], add[EL];
#pragma unroll
    for (int e = 0; e < EL; ++e) {
      const float h = r.at(e) * s;
      add[e] = da.at(e) * h;
      grad[e] = dr.at(e) + s * (da.at(e) * pre_w[e] - h * c1);
    }
    if (a.part_pre) add_own<T, V, EL>(acc[0], n, t, add);
    store_row<T, V, EL>(row_of(static_cast<E*>(a.dr), row, a.ld_dr, n), t, grad, E{});
    if (a.y) {
      float dg[EL];
      if constexpr (!kKeep) weights<T, V, EL>(a.post_w, n, t, post_w);
      if (a.post_w) {
        const float sy = rsqrtf(q[2] * inv_n + a.eps);
        float p[1] = {0.f};
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const float yh = y.at(e) * sy, u = a.scale * grad[e], dt = gates ? u * g.at(e) : u;
          dg[e] = u * yh * post_w[e];
          add[e] = dt * yh;
          grad[e] = dt * post_w[e];   // b
          p[0] += grad[e] * yh;
        }
        group_sum<T>(p, red[1], t);
        const float c2 = p[0] * inv_n;
#pragma unroll
        for (int e = 0; e < EL; ++e) grad[e] = sy * (grad[e] - y.at(e) * sy * c2);
        if (a.part_post) add_own<T, V, EL>(acc[1], n, t, add);
      } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const float u = a.scale * grad[e];
          dg[e] = u * y.at(e);
          grad[e] = gates ? u * g.at(e) : u;
        }
      }
      if (a.dy) store_row<T, V, EL>(row_of(a.dy, row, a.ld_dy, n), t, grad, uint16_t{});
      if (a.part_gate) add_own<T, V, EL>(acc[2], n, t, dg);
      else if (a.dgate) store_row<T, V, EL>(row_of(a.dgate, row, a.ld_dgate, n), t, dg, float{});
    }
    // The next row's first reduction writes red[0], last read before this
    // row's second barrier; without a post norm that barrier is missing.
    if constexpr (T > 64) {
      if (!(a.y && a.post_w)) __syncthreads();
    }
  }
  if constexpr (kLds) {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (part[k]) {
        float v[EL];
#pragma unroll
        for (int c = 0; c < EL / V; ++c)
#pragma unroll
          for (int e = 0; e < V; ++e) v[c * V + e] = acc[k][(c * T + t) * V + e];
        store_row<T, V, EL>(row_of(part[k], group, n, n), t, v, float{});
      }
  }
}

// Column sums of the groups' partial rows: 64 columns per block, 16 waves each
// adding every 16th group in order, then the 16 sums in wave order.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* p0, const float* p1, const float* p2, float* o0,
                                                           float* o1, float* o2, int64_t groups, int n) {
  __shared__ float red[16][64];
  const float* p = blockIdx.y == 0 ? p0 : (blockIdx.y == 1 ? p1 : p2);
  float* o = blockIdx.y == 0 ? o0 : (blockIdx.y == 1 ? o1 : o2);
  if (!o) return;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int col = blockIdx.x * 64 + lane;
  float s = 0.f;
  if (col < n) {
#pragma unroll 8
    for (int64_t g = w; g < groups; g += 16) s += p[g * n + col];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && col < n) {
    float v = red[0][lane];
#pragma unroll
    for (int k = 1; k < 16; ++k) v += red[k][lane];
    o[col] = v;
  }
}

// Threads of a row's group: 8 elements each up to 8192 columns (the backward
// pass 12 between 4096 and 6144, so that two groups fit a CU), then 1024 x 16
// (the backward pass 1024 x 12 up to 12288).
int threads_for(int n, bool back) {
  int t = 64;
  while (t < 1024 && t * 8 < n) t *= 2;
  return back && t == 1024 && n <= 6144 ? 512 : t;
}

template <bool kBack, typename F>
hipError_t pick(int32_t r_type, bool vec, int n, F&& f) {
  auto by_t = [&](auto e, auto v) -> hipError_t {
    constexpr std::integral_constant<int, 8> e8{};
    if constexpr (kBack)
      if (n > 8192 && n <= 12288)
        return f(e, v, std::integral_constant<int, 1024>{}, std::integral_constant<int, 12>{});
    if (n > 8192) return f(e, v, std::integral_constant<int, 1024>{}, std::integral_constant<int, 16>{});
    switch (threads_for(n, kBack)) {
      case 64: return f(e, v, std::integral_constant<int, 64>{}, e8);
      case 128: return f(e, v, std::integral_constant<int, 128>{}, e8);
      case 256: return f(e, v, std::integral_constant<int, 256>{}, e8);
      case 512:
        if constexpr (kBack)
          if (n > 4096) return f(e, v, std::integral_constant<int, 512>{}, std::integral_constant<int, 12>{});
        return f(e, v, std::integral_constant<int, 512>{}, e8);
      default: return f(e, v, std::integral_constant<int, 1024>{}, e8);
    }
  };
  const auto v1 = std::integral_constant<int, 1>{};
  const auto v4 = std::integral_constant<int, 4>{};
  if (r_type == Q3_BF16) return vec ? by_t(uint16_t{}, v4) : by_t(uint16_t{}, v1);
  return vec ? by_t(float{}, v4) : by_t(float{}, v1);
}

}  // namespace

// A launch takes less than 2^32 threads: 2^26 - 4 rows of up to 512 columns, 2^22 - 1
// of more than 4096.  More rows go in several.
hipError_t launch_residual_norm(const NormArgs& a, int32_t r_type, bool vec, hipStream_t s) {
  return pick<false>(r_type, vec, a.n, [&](auto e, auto v, auto t, auto el) {
    using E = decltype(e);
    constexpr int T = decltype(t)::value;
    constexpr int64_t most = 0xFFFFFFFFll / block_threads<T>() * rows_per_block<T>();
    for (int64_t at = 0; at < a.m; at += most) {
      NormArgs b = a;
      b.m = a.m - at < most ? a.m - at : most;
      if (b.y) b.y += at * a.ldy;
      if (b.gate) b.gate += at * a.ld_gate;
      b.r = static_cast<const E*>(a.r) + at * a.ldr;
      if (b.r_out) b.r_out = static_cast<E*>(a.r_out) + at * a.ldr_out;
      if (b.x) b.x += at * a.ldx;
      const unsigned blocks = (unsigned)((b.m + rows_per_block<T>() - 1) / rows_per_block<T>());
      hipLaunchKernelGGL((residual_norm_kernel<E, decltype(v)::value, T, decltype(el)::value>), dim3(blocks),
                         dim3(block_threads<T>()), 0, s, b);
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  });
}

// Row groups of the backward pass: all the rows, up to 256 K threads.
int64_t norm_back_groups(int64_t m, int n) {
  const int64_t most = kMaxGroups / threads_for(n, true);
  return m < most ? m : most;
}

hipError_t launch_residual_norm_back(const NormBackArgs& a, int32_t r_type, bool vec, float* dpre, float* dpost,
                                     float* dgate_row, hipStream_t s) {
  const hipError_t err = pick<true>(r_type, vec, a.n, [&](auto e, auto v, auto t, auto el) {
    constexpr int T = decltype(t)::value;
    const unsigned blocks = (unsigned)((a.groups + rows_per_block<T>() - 1) / rows_per_block<T>());
    constexpr int V = decltype(v)::value, EL = decltype(el)::value;
    constexpr size_t shm = EL < 16 ? (size_t)rows_per_block<T>() * 3 * T * EL * 4 : 0;
    static LdsAllowance seen;
    const hipError_t ok =
        allow_dynamic_lds(reinterpret_cast<const void*>(residual_norm_back_kernel<decltype(e), V, T, EL>), shm, seen);
    if (ok != hipSuccess) return ok;
    hipLaunchKernelGGL((residual_norm_back_kernel<decltype(e), V, T, EL>), dim3(blocks), dim3(block_threads<T>()), shm,
                       s, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || !(dpre || dpost || dgate_row)) return err;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((a.n + 63) / 64), 3), dim3(1024), 0, s, a.part_pre,
                     a.part_post, a.part_gate, dpre, dpost, dgate_row, a.groups, a.n);
  return hipGetLastError();
}

}  // namespace q3
