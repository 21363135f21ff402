// Head norms and the rotation by position, between the qkv product and attention.
//
// For each query and key head of a token (d values, of which r are rotated):
//   h = x s, s = rsqrt(mean(x^2) + eps);  n = h w          (w NULL: n = x)
//   o_a = n_a cos - n_b sin,  o_b = n_b cos + n_a sin      (a, b a pair, angle position * freq)
// and the backward pass, with do the gradient of o:
//   dn_a = do_a cos + do_b sin,  dn_b = do_b cos - do_a sin
//   dw = sum dn h,  a = dn w,  dx = s (a - h mean(a h))
//
// Both are bound by memory: 4 bytes in and 2 out per value (backward 4 and 2 or
// 4 in, 2 out).  A token is a block of 256 threads; a head belongs to a group of L
// lanes with 8 values each (L the power of two with 8 L >= d), so the mean is a
// few lane exchanges and loads and stores are 32 and 16 bytes a lane.  The
// token's angles are formed once by the block: position * freq in 64 bits,
// reduced there to [-pi, pi], where a 32-bit sine is good to 2^-22 whatever the
// position.
#include <type_traits>

#include "q3_device.h"
#include "../../include/q3_block.h"
#include "q3_internal.h"
#include "q3_paged.h"

namespace q3 {
namespace {

constexpr int kThreads = 256;

// Values of the token's angles; [0] cosines, [1] sines.
typedef float Turn[2][128];

__device__ __forceinline__ void angle_of(double position, float freq, float& c, float& s) {
  constexpr double kTurns = 0.15915494309189535;              // 1 / (2 pi)
  constexpr double kHigh = 6.283185307179586, kLow = 2.4492935982947064e-16;   // 2 pi
  double a = position * (double)freq;
  const double k = rint(a * kTurns);
  a = fma(-k, kLow, fma(-k, kHigh, a));
  sincosf((float)a, &s, &c);
}

struct Vec8 {
  float v[8];
};
__device__ __forceinline__ Vec8 load8(const float* p) {
  const f32x4 a = reinterpret_cast<const f32x4*>(p)[0], b = reinterpret_cast<const f32x4*>(p)[1];
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ Vec8 load8(const uint16_t* p) {
  const u32x4 u = *reinterpret_cast<const u32x4*>(p);
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o.v[2 * i] = __builtin_bit_cast(float, u[i] << 16);
    o.v[2 * i + 1] = __builtin_bit_cast(float, u[i] & 0xFFFF0000u);
  }
  return o;
}
__device__ __forceinline__ void store8(uint16_t* p, const Vec8& x) {
  u32x4 u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bf16x2 b = {static_cast<__bf16>(x.v[2 * i]), static_cast<__bf16>(x.v[2 * i + 1])};
    u[i] = __builtin_bit_cast(uint32_t, b);
  }
  *reinterpret_cast<u32x4*>(p) = u;
}
// A weight's eight values at e (4-byte aligned); ones without one.
__device__ __forceinline__ Vec8 weight8(const float* w, int e, bool live) {
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = w && live ? w[e + i] : 1.f;
  return o;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = 1; off < L; off *= 2) v += __shfl_xor(v, off, 64);
  return v;
}

// The rotation of a lane's eight values, those from e = 8 (lane % L) on; sign -1
// turns back.  `swap` is the wave's own 512 floats of LDS.  Every lane of the
// wave comes here.
template <int L>
__device__ __forceinline__ void rotate(Vec8& x, int rot, bool interleaved, const Turn& turn, float sign, float* swap,
                                       int lane) {
  const int e = 8 * (lane % L);
  if (interleaved) {
    if (e >= rot) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e + 2 * i < rot) {   // rot is even
        const float c = turn[0][e / 2 + i], s = sign * turn[1][e / 2 + i];
        const float a = x.v[2 * i], b = x.v[2 * i + 1];
        x.v[2 * i] = a * c - b * s;
        x.v[2 * i + 1] = b * c + a * s;
      }
    }
    return;
  }
  // Halves: value j goes with j + rot/2, which stands in another lane.
  const int half = rot / 2;
  if (rot == 0) return;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int i = 0; i < 8; ++i) swap[lane * 8 + i] = x.v[i];
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  const float* head = swap + (lane / L) * (8 * L);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = e + i;
    if (j < rot) {
      const bool low = j < half;
      const int at = low ? j : j - half;
      const float other = head[low ? j + half : at];
      const float c = turn[0][at], s = low ? -sign * turn[1][at] : sign * turn[1][at];
      x.v[i] = x.v[i] * c + other * s;
    }
  }
}

// One token per block (blockIdx.x); blockIdx.y takes every gridDim.y-th run of
// 256 / L heads.
template <int L>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(RopeArgs a) {
  __shared__ __align__(16) Turn turn;
  __shared__ __align__(16) float swap[kThreads / 64][512];
  constexpr int kHeads = kThreads / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = a.first + blockIdx.x;
  const int e = 8 * (threadIdx.x % L);
  const bool live = e < a.d;
  const int heads = a.hq + 2 * a.hk;

  int64_t position = 0, page = -1;
  if (a.batch.sequences) {
    const int s = find_sequence(a.batch, (int)row, lane);
    if (s == a.batch.sequences) return;   // the whole block
    position = (int64_t)a.batch.kv_len[s] - (a.batch.q_start[s + 1] - row);
    page = find_page(a.batch, a.cache, s, position);
  }
  const int64_t inside = position & ((1 << a.cache.shift) - 1);
  if (a.positions) position = a.positions[row];
  for (int t = threadIdx.x; t < a.rot / 2; t += kThreads) angle_of((double)position, a.freq[t], turn[0][t], turn[1][t]);
  __syncthreads();

  for (int h0 = blockIdx.y * kHeads; h0 < heads; h0 += gridDim.y * kHeads) {
    const int h = h0 + threadIdx.x / L;
    const bool here = live && h < heads;
    Vec8 x = {};
    if (here) x = load8(a.qkv + row * a.ld + (int64_t)h * a.d + e);
    const bool query = h < a.hq, value = h >= a.hq + a.hk;
    const float* w = value ? nullptr : query ? a.wq : a.wk;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q += x.v[i] * x.v[i];
    const float s = rsqrtf(group_sum<L>(q) / (float)a.d + a.eps);
    Vec8 o = x;
    if (w) {
      const Vec8 g = weight8(w, e, here);
#pragma unroll
      for (int i = 0; i < 8; ++i) o.v[i] = x.v[i] * s * g.v[i];
    }
    rotate<L>(o, a.rot, a.interleaved, turn, 1.f, swap[wave], lane);
    if (!here) continue;
    if (query) {
      store8(a.q + row * a.ldq + (int64_t)h * a.d + e, o);
    } else {
      const int kh = value ? h - a.hq - a.hk : h - a.hq;
      if (value) o = x;
      if (!a.batch.sequences) {
        store8((value ? a.v + row * a.ldv : a.k + row * a.ldk) + (int64_t)kh * a.d + e, o);
      } else if (page >= 0) {
        uint16_t* to = (value ? a.cache.v : a.cache.k) + page * a.cache.page_stride;
        store8(to + (((int64_t)kh << a.cache.shift) + inside) * a.d + e, o);
      }
    }
  }
}

// Blocks walk the tokens; a thread adds up the weight gradients of its eight
// values over its heads, the block's groups are added in order at the end.
template <int L, typename E>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_back_kernel(RopeBackArgs a) {
  __shared__ __align__(16) Turn turn[2];
  __shared__ __align__(16) float swap[kThreads / 64][512];
  constexpr int kHeads = kThreads / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = 8 * (threadIdx.x % L);
  const bool live = e < a.d;
  const int heads = a.hq + 2 * a.hk;
  Vec8 sums[2] = {};
  const Vec8 wq = weight8(a.wq, e, live), wk = weight8(a.wk, e, live);
  int parity = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += a.groups, parity ^= 1) {
    // The other buffer's readers are a barrier behind.
    for (int t = threadIdx.x; t < a.rot / 2; t += kThreads)
      angle_of((double)a.positions[row], a.freq[t], turn[parity][0][t], turn[parity][1][t]);
    __syncthreads();
    for (int h0 = 0; h0 < heads; h0 += kHeads) {
      const int h = h0 + threadIdx.x / L;
      const bool here = live && h < heads;
      const bool query = h < a.hq, value = h >= a.hq + a.hk;
      Vec8 g = {};
      if (here) {
        if (query) {
          if (a.dq) g = load8(static_cast<const E*>(a.dq) + row * a.ld_dq + (int64_t)h * a.d + e);
        } else if (!value) {
          if (a.dk) g = load8(static_cast<const E*>(a.dk) + row * a.ld_dk + (int64_t)(h - a.hq) * a.d + e);
        } else if (a.dv) {
          g = load8(static_cast<const E*>(a.dv) + row * a.ld_dv + (int64_t)(h - a.hq - a.hk) * a.d + e);
        }
      }
      const bool norm = !value && (query ? a.wq : a.wk);
      Vec8 x = {};
      if (here && norm) x = load8(a.qkv + row * a.ld + (int64_t)h * a.d + e);
      Vec8 dn = g;
      rotate<L>(dn, a.rot, a.interleaved, turn[parity], -1.f, swap[wave], lane);
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q += x.v[i] * x.v[i];
      const float s = rsqrtf(group_sum<L>(q) / (float)a.d + a.eps);
      float c = 0.f;
      Vec8 b;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x.v[i] *= s;   // h
        b.v[i] = dn.v[i] * (query ? wq.v[i] : wk.v[i]);
        c += b.v[i] * x.v[i];
      }
      c = group_sum<L>(c) / (float)a.d;
      if (!here) continue;
      if (norm) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = dn.v[i] * x.v[i];
          if (query) sums[0].v[i] += p;
          else sums[1].v[i] += p;
          g.v[i] = s * (b.v[i] - x.v[i] * c);
        }
      } else if (!value) {
        g = dn;
      }
      store8(a.dqkv + row * a.ld_out + (int64_t)h * a.d + e, g);
    }
  }
  if (!a.part) return;
  __shared__ float all[2][kThreads][9];   // 9: no two lanes of a step on one bank
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) all[k][threadIdx.x][i] = sums[k].v[i];
  __syncthreads();
  for (int t = threadIdx.x; t < 2 * a.d; t += kThreads) {
    const int k = t >= a.d, j = k ? t - a.d : t;
    float v = 0.f;
    for (int g = 0; g < kHeads; ++g) v += all[k][g * L + j / 8][j % 8];
    a.part[((int64_t)blockIdx.x * 2 + k) * a.d + j] = v;
  }
}

// Column sums of the groups' rows [groups][columns]: 16 columns a block, 64
// threads each every 64th row in order, then the 64 sums in order.
__global__ __launch_bounds__(1024) void rope_reduce_kernel(const float* part, int64_t groups, int d, float* dwq,
                                                           float* dwk) {
  __shared__ float red[64][17];
  const int c = threadIdx.x & 15, r = threadIdx.x >> 4, columns = 2 * d;
  const int col = blockIdx.x * 16 + c;   // d is a multiple of 16
  float s = 0.f;
#pragma unroll 8
  for (int64_t g = r; g < groups; g += 64) s += part[g * columns + col];
  red[r][c] = s;
  __syncthreads();
  if (threadIdx.x < 16) {
    float v = 0.f;
    for (int i = 0; i < 64; ++i) v += red[i][c];
    float* o = col < d ? dwq : dwk;
    if (o) o[col < d ? col : col - d] = v;
  }
}

template <typename F>
hipError_t by_lanes(int d, F&& f) {
  if (d <= 16) return f(std::integral_constant<int, 2>{});
  if (d <= 32) return f(std::integral_constant<int, 4>{});
  if (d <= 64) return f(std::integral_constant<int, 8>{});
  if (d <= 128) return f(std::integral_constant<int, 16>{});
  return f(std::integral_constant<int, 32>{});
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& args, hipStream_t s) {
  return by_lanes(args.d, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const int runs = (args.hq + 2 * args.hk + kThreads / L - 1) / (kThreads / L);
    // Few tokens: a block per run of heads, so that one token's heads load at once.
    const unsigned split = args.m >= 1024 ? 1u : (unsigned)runs;
    RopeArgs a = args;
    constexpr int64_t most = int64_t(1) << 22;   // a launch takes less than 2^32 threads
    for (a.first = 0; a.first < a.m; a.first += most) {
      const int64_t rows = a.m - a.first < most ? a.m - a.first : most;
      hipLaunchKernelGGL(qk_norm_rope_kernel<L>, dim3((unsigned)rows, split), dim3(kThreads), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

// Blocks of the backward pass: four a CU, each leaves one row of partial sums.
int64_t rope_back_groups(int64_t m) { return m < 1024 ? m : 1024; }

hipError_t launch_qk_norm_rope_back(const RopeBackArgs& a, int32_t d_type, hipStream_t s) {
  const hipError_t err = by_lanes(a.d, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    if (d_type == Q3_BF16)
      hipLaunchKernelGGL((qk_norm_rope_back_kernel<L, uint16_t>), dim3((unsigned)a.groups), dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((qk_norm_rope_back_kernel<L, float>), dim3((unsigned)a.groups), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || !a.part) return err;
  hipLaunchKernelGGL(rope_reduce_kernel, dim3((unsigned)(2 * a.d / 16)), dim3(1024), 0, s, a.part, a.groups, a.d,
                     a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace q3
