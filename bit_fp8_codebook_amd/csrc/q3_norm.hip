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
// per thread up to 8192 columns, 16 above), reduced, and written once.  A row
// belongs to a group of T threads, the smallest of 64..1024 with 8 T >= n; up
// to 512 columns that is one wave, so a 256-thread block takes four rows and no reduction crosses a
// wave.  The backward pass sums its weight gradients over tokens in registers:
// a fixed number of groups walks the rows, each leaves one partial row per
// gradient, and a second launch adds those in group order (no atomics, so the
// same call gives the same bits).  All statistics and sums are fp32.
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

// V consecutive elements of a row (V = 1 or 4, aligned to V elements).
template <int V, typename E>
__device__ __forceinline__ void load_v(const E* p, float* out) {
  if constexpr (V == 4 && sizeof(E) == 4) {
    const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = v[e];
  } else if constexpr (V == 4) {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      out[2 * e] = __builtin_bit_cast(float, v[e] << 16);
      out[2 * e + 1] = __builtin_bit_cast(float, v[e] & 0xFFFF0000u);
    }
  } else if constexpr (sizeof(E) == 4) {
    out[0] = *p;
  } else {
    out[0] = __builtin_bit_cast(float, (uint32_t)*p << 16);
  }
}
__device__ __forceinline__ uint32_t bf16_bits(float a, float b) {
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
template <int V, typename E>
__device__ __forceinline__ void store_v(E* p, const float* v) {
  if constexpr (V == 4 && sizeof(E) == 4) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
  } else if constexpr (V == 4) {
    *reinterpret_cast<u32x2*>(p) = u32x2{bf16_bits(v[0], v[1]), bf16_bits(v[2], v[3])};
  } else if constexpr (sizeof(E) == 4) {
    *p = v[0];
  } else {
    *p = (uint16_t)bf16_bits(v[0], 0.f);
  }
}

// The group's part of a row (a null row reads as `fill`; columns past n as 0).
template <int T, int V, int EL, typename E>
__device__ __forceinline__ void load_row(const E* row, int n, int t, float fill, float (&v)[EL]) {
#pragma unroll
  for (int c = 0; c < EL / V; ++c) {
    const int col = (c * T + t) * V;
    if (col < n && row) {
      load_v<V>(row + col, v + c * V);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) v[c * V + e] = col < n ? fill : 0.f;
    }
  }
}
template <int T, int V, int EL, typename E>
__device__ __forceinline__ void store_row(E* row, int n, int t, const float (&v)[EL]) {
#pragma unroll
  for (int c = 0; c < EL / V; ++c) {
    const int col = (c * T + t) * V;
    if (col < n) store_v<V>(row + col, v + c * V);
  }
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
  const int64_t row = (int64_t)blockIdx.x * rows_per_block<T>() + threadIdx.x / T;
  if (row >= a.m) return;   // whole groups; T == 64 has no barriers
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  float r[EL];
  load_row<T, V, EL>(static_cast<const E*>(a.r) + row * a.ldr, n, t, 0.f, r);
  if (a.y) {
    float y[EL], g[EL];
    load_row<T, V, EL>(a.y + row * a.ldy, n, t, 0.f, y);
    load_row<T, V, EL>(a.gate ? a.gate + row * a.ld_gate : nullptr, n, t, 1.f, g);
    if (a.post_w) {
      float w[EL], q[1] = {0.f};
      load_row<T, V, EL>(a.post_w, n, t, 0.f, w);
#pragma unroll
      for (int e = 0; e < EL; ++e) q[0] += y[e] * y[e];
      group_sum<T>(q, red[0], t);
      const float sy = rsqrtf(q[0] * inv_n + a.eps);
#pragma unroll
      for (int e = 0; e < EL; ++e) y[e] = y[e] * sy * w[e];
    }
#pragma unroll
    for (int e = 0; e < EL; ++e) r[e] += a.scale * g[e] * y[e];
    store_row<T, V, EL>(static_cast<E*>(a.r_out) + row * a.ldr_out, n, t, r);
  } else if (a.r_out && a.r_out != a.r) {
    store_row<T, V, EL>(static_cast<E*>(a.r_out) + row * a.ldr_out, n, t, r);
  }
  if (a.x) {
    float w[EL], q[1] = {0.f};
    load_row<T, V, EL>(a.pre_w, n, t, 1.f, w);
#pragma unroll
    for (int e = 0; e < EL; ++e) q[0] += r[e] * r[e];
    group_sum<T>(q, red[1], t);
    const float s = rsqrtf(q[0] * inv_n + a.eps);
#pragma unroll
    for (int e = 0; e < EL; ++e) w[e] *= r[e] * s;
    store_row<T, V, EL>(a.x + row * a.ldx, n, t, w);
  }
}

template <typename E, int V, int T, int EL>
__global__ __launch_bounds__(block_threads<T>()) void residual_norm_back_kernel(NormBackArgs a) {
  __shared__ float red[2][48];
  const int t = threadIdx.x % T;
  const int64_t group = (int64_t)blockIdx.x * rows_per_block<T>() + threadIdx.x / T;
  if (group >= a.groups) return;
  const int n = a.n;
  const float inv_n = 1.0f / (float)n;
  float acc_pre[EL], acc_post[EL], acc_gate[EL];
#pragma unroll
  for (int e = 0; e < EL; ++e) acc_pre[e] = acc_post[e] = acc_gate[e] = 0.f;

  for (int64_t row = group; row < a.m; row += a.groups) {
    float r[EL], da[EL], dr[EL], y[EL], q[3] = {0.f, 0.f, 0.f};
    load_row<T, V, EL>(static_cast<const E*>(a.r) + row * a.ldr, n, t, 0.f, r);
    load_row<T, V, EL>(a.dx ? a.dx + row * a.ld_dx : nullptr, n, t, 0.f, da);
    load_row<T, V, EL>(a.y ? a.y + row * a.ldy : nullptr, n, t, 0.f, y);
    load_row<T, V, EL>(a.dr_out ? static_cast<const E*>(a.dr_out) + row * a.ld_dr_out : nullptr, n, t, 0.f, dr);
    {
      float w[EL];
      load_row<T, V, EL>(a.pre_w, n, t, 1.f, w);
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        q[0] += r[e] * r[e];
        q[1] += da[e] * w[e] * r[e];
        q[2] += y[e] * y[e];
      }
      group_sum<T>(q, red[0], t);
      const float s = rsqrtf(q[0] * inv_n + a.eps), c1 = q[1] * inv_n * s;
#pragma unroll
      for (int e = 0; e < EL; ++e) {
        const float h = r[e] * s;
        acc_pre[e] += da[e] * h;
        dr[e] += s * (da[e] * w[e] - h * c1);
      }
    }
    store_row<T, V, EL>(static_cast<E*>(a.dr) + row * a.ld_dr, n, t, dr);
    if (a.y) {
      float g[EL];
      load_row<T, V, EL>(a.gate ? a.gate + row * a.ld_gate : nullptr, n, t, 1.f, g);
      if (a.post_w) {
        const float sy = rsqrtf(q[2] * inv_n + a.eps);
        float w[EL], p[1] = {0.f};
        load_row<T, V, EL>(a.post_w, n, t, 0.f, w);
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const float yh = y[e] * sy, u = a.scale * dr[e], dt = u * g[e];
          const float dg = u * yh * w[e];
          acc_post[e] += dt * yh;
          y[e] = yh;
          dr[e] = dt * w[e];   // b
          g[e] = dg;
          p[0] += dr[e] * yh;
        }
        group_sum<T>(p, red[1], t);
        const float c2 = p[0] * inv_n;
#pragma unroll
        for (int e = 0; e < EL; ++e) dr[e] = sy * (dr[e] - y[e] * c2);
      } else {
#pragma unroll
        for (int e = 0; e < EL; ++e) {
          const float u = a.scale * dr[e];
          dr[e] = u * g[e];
          g[e] = u * y[e];
        }
      }
      if (a.dy) store_row<T, V, EL>(a.dy + row * a.ld_dy, n, t, dr);
      if (a.dgate) {
        if (a.ld_gate) {
          store_row<T, V, EL>(a.dgate + row * a.ld_dgate, n, t, g);
        } else {
#pragma unroll
          for (int e = 0; e < EL; ++e) acc_gate[e] += g[e];
        }
      }
    }
    // The next row's first reduction writes red[0], last read before this
    // row's second barrier; without a post norm that barrier is missing.
    if constexpr (T > 64) {
      if (!(a.y && a.post_w)) __syncthreads();
    }
  }
  const int64_t at = group * n;
  if (a.part_pre) store_row<T, V, EL>(a.part_pre + at, n, t, acc_pre);
  if (a.part_post) store_row<T, V, EL>(a.part_post + at, n, t, acc_post);
  if (a.part_gate) store_row<T, V, EL>(a.part_gate + at, n, t, acc_gate);
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
// pass keeps five rows and three sums of them in registers), then 1024 x 16.
int threads_for(int n) {
  int t = 64;
  while (t < 1024 && t * 8 < n) t *= 2;
  return t;
}

template <typename F>
hipError_t pick(int32_t r_type, bool vec, int n, F&& f) {
  auto by_t = [&](auto e, auto v) -> hipError_t {
    constexpr std::integral_constant<int, 8> e8{};
    if (n > 8192) return f(e, v, std::integral_constant<int, 1024>{}, std::integral_constant<int, 16>{});
    switch (threads_for(n)) {
      case 64: return f(e, v, std::integral_constant<int, 64>{}, e8);
      case 128: return f(e, v, std::integral_constant<int, 128>{}, e8);
      case 256: return f(e, v, std::integral_constant<int, 256>{}, e8);
      case 512: return f(e, v, std::integral_constant<int, 512>{}, e8);
      default: return f(e, v, std::integral_constant<int, 1024>{}, e8);
    }
  };
  const auto v1 = std::integral_constant<int, 1>{};
  const auto v4 = std::integral_constant<int, 4>{};
  if (r_type == Q3_BF16) return vec ? by_t(uint16_t{}, v4) : by_t(uint16_t{}, v1);
  return vec ? by_t(float{}, v4) : by_t(float{}, v1);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, int32_t r_type, bool vec, hipStream_t s) {
  return pick(r_type, vec, a.n, [&](auto e, auto v, auto t, auto el) {
    constexpr int T = decltype(t)::value;
    const unsigned blocks = (unsigned)((a.m + rows_per_block<T>() - 1) / rows_per_block<T>());
    hipLaunchKernelGGL((residual_norm_kernel<decltype(e), decltype(v)::value, T, decltype(el)::value>), dim3(blocks),
                       dim3(block_threads<T>()), 0, s, a);
    return hipGetLastError();
  });
}

// Row groups of the backward pass: all the rows, up to 256 K threads.
int64_t norm_back_groups(int64_t m, int n) {
  const int64_t most = kMaxGroups / threads_for(n);
  return m < most ? m : most;
}

hipError_t launch_residual_norm_back(const NormBackArgs& a, int32_t r_type, bool vec, float* dpre, float* dpost,
                                     float* dgate_row, hipStream_t s) {
  const hipError_t err = pick(r_type, vec, a.n, [&](auto e, auto v, auto t, auto el) {
    constexpr int T = decltype(t)::value;
    const unsigned blocks = (unsigned)((a.groups + rows_per_block<T>() - 1) / rows_per_block<T>());
    hipLaunchKernelGGL((residual_norm_back_kernel<decltype(e), decltype(v)::value, T, decltype(el)::value>), dim3(blocks),
                       dim3(block_threads<T>()), 0, s, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || !(dpre || dpost || dgate_row)) return err;
  hipLaunchKernelGGL(norm_reduce_kernel, dim3((unsigned)((a.n + 63) / 64), 3), dim3(1024), 0, s, a.part_pre,
                     a.part_post, a.part_gate, dpre, dpost, dgate_row, a.groups, a.n);
  return hipGetLastError();
}

}  // namespace q3
