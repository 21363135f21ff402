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
// few lane exchanges.  A lane's values are two runs of four: where halves are
// rotated, four values and their four partners, so that the rotation stays in the
// lane (a half that is no multiple of four goes through LDS instead).  The
// token's angles are formed once by the block while the first heads' loads are
// under way.
//
// Measured: 4 prompts' 6054 tokens of 32 + 2 x 8 heads of 128 39 us, 5.7 TB/s (with a
// kernel for all pairings 46, with halves through LDS and angles by the library's sine
// 70); one token 4.3 us.  Backward, 4095 tokens of 80 heads of 128: 74 us on fresh rows,
// 4.5 TB/s (83 with fp32 gradients, 5.0), 56 where a third of them is in the memory-side
// cache, and 4 for the weights' sums (a call 77, with a kernel for all pairings 92).
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

// Cosine and sine of position * freq.  The angle is taken to turns in 64 bits with
// the product's and 1 / (2 pi)'s own remainders, to its place in a quarter turn, and
// from there by the series of both up to the eleventh power (left over below
// 2^-29 at pi / 4).
__device__ __forceinline__ void angle_of(double position, float freq, float& c, float& s) {
  constexpr double kTurns = 0.15915494309189535, kRest = -9.839338337591215e-18;   // 1 / (2 pi)
  const double a = position * (double)freq, t = a * kTurns;
  const double turn = (t - rint(t)) + fma(a, kRest, fma(a, kTurns, -t));
  const double q = rint(4.0 * turn);
  const float x = (float)((turn - 0.25 * q) * 6.283185307179586), y = x * x;
  const float sn = x + x * y * (-1.f / 6 + y * (1.f / 120 + y * (-1.f / 5040 + y * (1.f / 362880 - y * (1.f / 39916800)))));
  const float cs = 1.f + y * (-0.5f + y * (1.f / 24 + y * (-1.f / 720 + y * (1.f / 40320 - y * (1.f / 3628800)))));
  const int n = (int)q;
  c = n & 1 ? sn : cs;
  s = n & 1 ? cs : sn;
  c = (n + 1) & 2 ? -c : c;
  s = n & 2 ? -s : s;
}

struct Vec8 {
  float v[8];
};
// How values pair up: with those half a rotation away, in runs of four (also where
// nothing is rotated); adjacent ones; halves that are no multiple of four.
enum Pairing { kHalves, kAdjacent, kOddHalves };
int pairing_of(int rot, int interleaved) { return interleaved ? kAdjacent : rot % 8 == 0 ? kHalves : kOddHalves; }

// Lane l's values of a head: e[0].. and e[1]...
struct Places {
  int e[2];
  bool low;    // kHalves: e[1] are the partners of e[0]; angles from e[0] on
  bool live;   // inside the head
};
template <int P>
__device__ __forceinline__ Places places(int l, int d, int rot) {
  Places p;
  p.low = P == kHalves && l < rot / 8;
  p.live = l < d / 8;
  p.e[0] = P == kAdjacent || p.low ? 4 * l : 8 * l;
  p.e[1] = P == kAdjacent ? d / 2 + 4 * l : p.low ? rot / 2 + 4 * l : 8 * l + 4;
  return p;
}
__device__ __forceinline__ Vec8 load8(const float* p, const Places& at) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p + at.e[0]), b = *reinterpret_cast<const f32x4*>(p + at.e[1]);
  return {{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ Vec8 load8(const uint16_t* p, const Places& at) {
  Vec8 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x2 u = *reinterpret_cast<const u32x2*>(p + at.e[h]);
    o.v[4 * h] = __builtin_bit_cast(float, u.x << 16);
    o.v[4 * h + 1] = __builtin_bit_cast(float, u.x & 0xFFFF0000u);
    o.v[4 * h + 2] = __builtin_bit_cast(float, u.y << 16);
    o.v[4 * h + 3] = __builtin_bit_cast(float, u.y & 0xFFFF0000u);
  }
  return o;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
template <bool kPast = false>   // past the caches
__device__ __forceinline__ void store8(uint16_t* p, const Places& at, const Vec8& x) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const u32x2 u = {pack_bf16(x.v[4 * h], x.v[4 * h + 1]), pack_bf16(x.v[4 * h + 2], x.v[4 * h + 3])};
    u32x2* to = reinterpret_cast<u32x2*>(p + at.e[h]);
    if constexpr (kPast) __builtin_nontemporal_store(u, to);
    else *to = u;
  }
}
// A weight's values (4-byte aligned); ones without one.
__device__ __forceinline__ Vec8 weight8(const float* w, const Places& at) {
  Vec8 o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = w && at.live ? w[at.e[i / 4] + i % 4] : 1.f;
  return o;
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int off = 1; off < L; off *= 2) v += __shfl_xor(v, off, 64);
  return v;
}

// The rotation of a lane's values; sign -1 turns back.  `swap` is the wave's own
// 512 floats of LDS.  Every lane of the wave comes here.
template <int L, int P>
__device__ __forceinline__ void rotate(Vec8& x, const Places& at, int rot, const Turn& turn, float sign, float* swap,
                                       int lane) {
  if constexpr (P == kAdjacent) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int j = at.e[h] + 2 * i;
        if (j < rot) {   // rot is even
          const float c = turn[0][j / 2], s = sign * turn[1][j / 2];
          const float a = x.v[4 * h + 2 * i], b = x.v[4 * h + 2 * i + 1];
          x.v[4 * h + 2 * i] = a * c - b * s;
          x.v[4 * h + 2 * i + 1] = b * c + a * s;
        }
      }
    return;
  }
  if constexpr (P == kHalves) {
    if (!at.low) return;
    const f32x4 c = *reinterpret_cast<const f32x4*>(&turn[0][at.e[0]]), s = *reinterpret_cast<const f32x4*>(&turn[1][at.e[0]]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x.v[i], b = x.v[4 + i], t = sign * s[i];
      x.v[i] = a * c[i] - b * t;
      x.v[4 + i] = b * c[i] + a * t;
    }
    return;
  }
  if constexpr (P == kOddHalves) {
    // Value j goes with j + rot/2, which stands in another lane (e[1] = e[0] + 4 here).
    const int half = rot / 2;
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
      const int j = at.e[0] + i;
      if (j < rot) {
        const bool low = j < half;
        const int k = low ? j : j - half;
        const float other = head[low ? j + half : k];
        const float c = turn[0][k], s = low ? -sign * turn[1][k] : sign * turn[1][k];
        x.v[i] = x.v[i] * c + other * s;
      }
    }
  }
}

// One token per block (blockIdx.x); blockIdx.y takes every gridDim.y-th run of
// 256 / L heads, three of them at a time.
constexpr int kAhead = 3;
template <int L, int P>
__global__ __launch_bounds__(kThreads) void qk_norm_rope_kernel(RopeArgs a) {
  __shared__ __align__(16) Turn turn;
  __shared__ __align__(16) float swap[P == kOddHalves ? kThreads / 64 : 1][512];
  constexpr int kHeads = kThreads / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = a.first + blockIdx.x;
  const Places at = places<P>(threadIdx.x % L, a.d, a.rot);
  const int heads = a.hq + 2 * a.hk, stride = gridDim.y * kHeads;
  const float* src = a.qkv + row * a.ld;
  Vec8 x[kAhead];
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int h = h0 + k * stride + threadIdx.x / L;
      x[k] = Vec8{};
      if (at.live && h < heads) x[k] = load8(src + h * a.d, at);
    }
  };
  const int first = blockIdx.y * kHeads;
  const Vec8 wq = weight8(a.wq, at), wk = weight8(a.wk, at);

  int s = 0;
  if (a.batch.sequences) {
    s = find_sequence(a.batch, (int)row, lane);
    if (s == a.batch.sequences) return;   // the whole block; its row need not be there
  }
  load(first);   // beside what the tables say of the row
  int64_t position = 0, page = -1;
  if (a.batch.sequences) {
    position = (int64_t)a.batch.kv_len[s] - (a.batch.q_start[s + 1] - row);
    page = find_page(a.batch, a.cache, s, position);
  }
  const int64_t inside = position & ((1 << a.cache.shift) - 1);
  if (a.positions) position = a.positions[row];
  for (int t = threadIdx.x; t < a.rot / 2; t += kThreads) angle_of((double)position, a.freq[t], turn[0][t], turn[1][t]);
  __syncthreads();

  for (int h0 = first; h0 < heads; h0 += kAhead * stride) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (h0 + k * stride >= heads) break;   // the whole block
      const int h = h0 + k * stride + threadIdx.x / L;
      const bool query = h < a.hq, value = h >= a.hq + a.hk;
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q += x[k].v[i] * x[k].v[i];
      const float s = rsqrtf(group_sum<L>(q) / (float)a.d + a.eps);
      Vec8 o = x[k];
      if (query ? a.wq : a.wk) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o.v[i] = x[k].v[i] * s * (query ? wq.v[i] : wk.v[i]);
      }
      rotate<L, P>(o, at, a.rot, turn, 1.f, swap[P == kOddHalves ? wave : 0], lane);
      if (!at.live || h >= heads) continue;
      if (query) {
        store8(a.q + row * a.ldq + h * a.d, at, o);
      } else {
        const int kh = value ? h - a.hq - a.hk : h - a.hq;
        if (value) o = x[k];
        if (!a.batch.sequences) {
          store8((value ? a.v + row * a.ldv : a.k + row * a.ldk) + kh * a.d, at, o);
        } else if (page >= 0) {
          uint16_t* to = (value ? a.cache.v : a.cache.k) + page * a.cache.page_stride;
          store8(to + (((int64_t)kh << a.cache.shift) + inside) * a.d, at, o);
        }
      }
    }
  }
}

// Blocks walk the tokens (blockIdx.y takes every gridDim.y-th run of heads); a thread
// adds up the weight gradients of its eight values over its heads, the block's groups are
// added in order at the end.  The gradients go past the caches, which the rows of the
// tokens on their way fill (4095 tokens of 80 heads of 128, both launches: 76 us, without 84).
template <int L, int P, typename E>
__global__ __launch_bounds__(kThreads, 4) void qk_norm_rope_back_kernel(RopeBackArgs a) {
  __shared__ __align__(16) Turn turn[2];
  __shared__ __align__(16) float swap[P == kOddHalves ? kThreads / 64 : 1][512];
  constexpr int kHeads = kThreads / L;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const Places at = places<P>(threadIdx.x % L, a.d, a.rot);
  const int heads = a.hq + 2 * a.hk;
  Vec8 sums[2] = {};
  const Vec8 wq = weight8(a.wq, at), wk = weight8(a.wk, at);
  struct Head {
    Vec8 g, x;
  };
  // A head's gradient and, where it is normed, its values.
  auto load = [&](int64_t row, int h) {
    Head o = {};
    if (!at.live || h >= heads) return o;
    const bool query = h < a.hq, value = h >= a.hq + a.hk;
    const void* d = query ? a.dq : value ? a.dv : a.dk;
    const int64_t ld = query ? a.ld_dq : value ? a.ld_dv : a.ld_dk;
    const int k = query ? h : value ? h - a.hq - a.hk : h - a.hq;
    if (d) o.g = load8(static_cast<const E*>(d) + row * ld + k * a.d, at);
    if (!value && (query ? a.wq : a.wk)) o.x = load8(a.qkv + row * a.ld + h * a.d, at);
    return o;
  };
  int parity = 0;
  const int first = blockIdx.y * kHeads, stride = gridDim.y * kHeads;
  Head next = load(blockIdx.x, first + threadIdx.x / L);
  for (int64_t row = blockIdx.x; row < a.m; row += a.groups, parity ^= 1) {
    // The other buffer's readers are a barrier behind.
    for (int t = threadIdx.x; t < a.rot / 2; t += kThreads)
      angle_of((double)a.positions[row], a.freq[t], turn[parity][0][t], turn[parity][1][t]);
    __syncthreads();
    for (int h0 = first; h0 < heads; h0 += stride) {
      const int h = h0 + threadIdx.x / L;
      const bool query = h < a.hq, value = h >= a.hq + a.hk;
      Head cur = next;
      // The next heads', or the next token's first, while these are worked on.
      const bool more = h0 + stride < heads;
      if (more || row + a.groups < a.m)
        next = load(more ? row : row + a.groups, (more ? h0 + stride : first) + threadIdx.x / L);
      const bool norm = !value && (query ? a.wq : a.wk);
      Vec8 x = cur.x, g = cur.g, dn = g;
      rotate<L, P>(dn, at, a.rot, turn[parity], -1.f, swap[P == kOddHalves ? wave : 0], lane);
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
      if (!at.live || h >= heads) continue;
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
      store8<true>(a.dqkv + row * a.ld_out + h * a.d, at, g);
    }
  }
  if (!a.part) return;
  __shared__ float all[kThreads][9];   // 9: no two lanes of a step on one bank
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) all[threadIdx.x][i] = sums[k].v[i];
    __syncthreads();
    // The group's lane and value i hold the same column in every group of the block.
    for (int t = threadIdx.x; t < 8 * L; t += kThreads) {
      const int l = t / 8, i = t % 8;
      if (l >= a.d / 8) continue;
      float v = 0.f;
      for (int g = 0; g < kHeads; ++g) v += all[g * L + l][i];
      // (An array's element at i / 4 would go through LDS, and its address through the
      // block's size, read from host memory: 14 us of a call of 70 tokens.)
      const Places of = places<P>(l, a.d, a.rot);
      const int column = (i < 4 ? of.e[0] : of.e[1]) + i % 4;
      a.part[(((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 2 + k) * a.d + column] = v;
    }
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
hipError_t by_lanes(int d, int pairing, F&& f) {
  auto with = [&](auto lanes) {
    if (pairing == kHalves) return f(lanes, std::integral_constant<int, kHalves>{});
    if (pairing == kAdjacent) return f(lanes, std::integral_constant<int, kAdjacent>{});
    return f(lanes, std::integral_constant<int, kOddHalves>{});
  };
  if (d <= 16) return with(std::integral_constant<int, 2>{});
  if (d <= 32) return with(std::integral_constant<int, 4>{});
  if (d <= 64) return with(std::integral_constant<int, 8>{});
  if (d <= 128) return with(std::integral_constant<int, 16>{});
  return with(std::integral_constant<int, 32>{});
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs& args, hipStream_t s) {
  return by_lanes(args.d, pairing_of(args.rot, args.interleaved), [&](auto lanes, auto pairing) {
    constexpr int L = decltype(lanes)::value, P = decltype(pairing)::value;
    const int runs = (args.hq + 2 * args.hk + kThreads / L - 1) / (kThreads / L);
    // Few tokens: a block per run of heads, so that one token's heads load at once (48
    // heads of 128: 64 tokens 4.4 us, without 5.1; 256 tokens 7.1 and 6.1; 1000 17.4 and 11.8).
    const unsigned split = args.m >= 128 ? 1u : (unsigned)runs;
    RopeArgs a = args;
    constexpr int64_t most = int64_t(1) << 22;   // a launch takes less than 2^32 threads
    for (a.first = 0; a.first < a.m; a.first += most) {
      const int64_t rows = a.m - a.first < most ? a.m - a.first : most;
      hipLaunchKernelGGL((qk_norm_rope_kernel<L, P>), dim3((unsigned)rows, split), dim3(kThreads), 0, s, a);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  });
}

// Blocks of the backward pass: four a CU, each leaves one row of partial sums (4095
// tokens: 75 us, with 768 blocks 85, with 2048 80).
constexpr int64_t kBackBlocks = 1024;
int64_t rope_back_rows(int64_t m) { return m > 0 ? kBackBlocks : 0; }

hipError_t launch_qk_norm_rope_back(const RopeBackArgs& args, int32_t d_type, hipStream_t s) {
  RopeBackArgs a = args;
  a.groups = a.m < kBackBlocks ? a.m : kBackBlocks;
  int64_t rows = 0;   // of partial sums
  const hipError_t err = by_lanes(a.d, pairing_of(a.rot, a.interleaved), [&](auto lanes, auto pairing) {
    constexpr int L = decltype(lanes)::value, P = decltype(pairing)::value;
    // Few tokens: their heads in runs, as in the forward pass (48 heads of 128: 70 tokens 9.0
    // us with the sums' launch, in one run 10.9; 300 tokens 14.4 and 13.4).
    const int64_t runs = (a.hq + 2 * a.hk + kThreads / L - 1) / (kThreads / L), most = a.m < 128 ? kBackBlocks / a.groups : 1;
    const dim3 grid((unsigned)a.groups, (unsigned)(runs < most ? runs : most));
    rows = (int64_t)grid.x * grid.y;
    if (d_type == Q3_BF16)
      hipLaunchKernelGGL((qk_norm_rope_back_kernel<L, P, uint16_t>), grid, dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((qk_norm_rope_back_kernel<L, P, float>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  });
  if (err != hipSuccess || !a.part) return err;
  hipLaunchKernelGGL(rope_reduce_kernel, dim3((unsigned)(2 * a.d / 16)), dim3(1024), 0, s, a.part, rows, a.d,
                     a.dwq, a.dwk);
  return hipGetLastError();
}

}  // namespace q3
