// Products of many tokens with packed 3-bit matrices, their input gradients and
// the gated feed-forward block.
//
//   y[m][n]  = sum_k x[m][k] w[n][k]          (q3_gemm)
//   dx[m][k] = sum_n dy[m][n] w[n][k]         (q3_gemm_backward)
//   h[m][i]  = act(x . w[i]) * (x . w[I + i]) (q3_glu)
//
// Few tokens are bound by the packed weights and their dequantisation, and
// q3_linear.hip's kernels read them once for up to 64 or 128 tokens.  Many are
// bound by the matrix cores, and dequantising inside the product would repeat the
// vector work for every block of tokens; so the matrix is widened once, exactly, to
// bf16 in the caller's workspace (for the gradient: transposed) and all three run
// on one kernel: C = A B^T with both operands bf16 and contiguous along the summed
// axis.
#include <type_traits>

#include "q3_act.h"
#include "q3_device.h"
#include "q3_internal.h"

namespace q3 {
namespace {

// ---- widening -----------------------------------------------------------------

// One wave per (16-row tile, 512-k step): lane l holds row l%16 and groups
// 4*(l/16)..+3, as the planes are laid out.  Two of its groups at a time go
// through LDS, so that 8 lanes store 128 consecutive bytes of a row (stored
// straight from the lanes that dequantise, 16 bytes every 256, 22016 x 4096
// took 103 us).  out [n][gp*32]; groups past G are written as zeros.
constexpr uint32_t kWidenSlot = 128 + 16;   // a lane's two groups, padded against bank conflicts
__global__ __launch_bounds__(256) void widen_kernel(PlaneView w, uint16_t* __restrict__ out, int64_t units, int steps) {
  __shared__ __align__(16) uint8_t stage[4][64 * kWidenSlot];
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (unit >= units) return;   // whole waves; the block has no barriers
  uint8_t* st = stage[threadIdx.x >> 6];
  const int i = lane & 15, kb = lane >> 4;
  const int64_t tile = unit / steps;
  const uint32_t s = (uint32_t)(unit - tile * steps);
  const uint32_t gp = (uint32_t)((w.groups + 3) & ~3);
  const uint32_t q = step_quads(s, gp);
  const int64_t row = tile * 16 + i;
  u32x4 d[3] = {};
  uint32_t sc = 0;
  u32x2 cb = {0u, 0u};
  if ((uint32_t)kb < q && row < w.n) {
    const uint8_t* c = w.code + tile * (int64_t)(192u * gp) + 3072u * s;
#pragma unroll
    for (int j = 0; j < 3; ++j) d[j] = *reinterpret_cast<const u32x4*>(c + 16u * (16u * (q * j + kb) + i));
    sc = *reinterpret_cast<const uint32_t*>(w.scale + tile * (int64_t)(16u * gp) + 256u * s + 4u * (16u * kb + i));
    cb = *reinterpret_cast<const u32x2*>(w.cb + row * 8);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int t = 2 * half + g;
      bf16x2 v[16];
      dequant_group_bf16(d[0][t], d[1][t], d[2][t], (sc >> (8 * t)) & 255u, cb.x, cb.y, v);
      const bool real = (int)(s * 16u + kb * 4u + t) < w.groups;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        u32x4 u;
#pragma unroll
        for (int f = 0; f < 4; ++f) u[f] = real ? __builtin_bit_cast(uint32_t, v[4 * e + f]) : 0u;
        *reinterpret_cast<u32x4*>(st + lane * kWidenSlot + 64 * g + 16 * e) = u;
      }
    }
    // The wave reads what its own lanes wrote.
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int slot = 8 * c + (lane >> 3), piece = lane & 7;
      const int64_t r = tile * 16 + (slot & 15);
      const uint32_t b = (uint32_t)slot >> 4;
      if (b < q && r < w.n)
        *reinterpret_cast<u32x4*>(out + r * (int64_t)(gp * 32u) + s * 512u + b * 128u + half * 64u + piece * 8u) =
            *reinterpret_cast<const u32x4*>(st + slot * kWidenSlot + 16 * piece);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
}

// Transposed: out [k][np], np = n padded to 64 with zeros.  A block takes 64
// rows (a tile per wave) and one 512-k step, a group of each quad at a time
// through LDS.
__global__ __launch_bounds__(256) void widen_t_kernel(PlaneView w, uint16_t* __restrict__ out, int64_t np) {
  constexpr int kPad = 72;   // 64 rows and 16 bytes against bank conflicts
  __shared__ uint16_t buf[128 * kPad];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = lane & 15, kb = lane >> 4;
  const uint32_t s = blockIdx.y;
  const int64_t tile = (int64_t)blockIdx.x * 4 + wave;
  const uint32_t gp = (uint32_t)((w.groups + 3) & ~3);
  const uint32_t q = step_quads(s, gp);
  const int64_t row = tile * 16 + i;
  const bool ok = (uint32_t)kb < q && row < w.n;
  u32x4 d[3] = {};
  uint32_t sc = 0;
  u32x2 cb = {0u, 0u};
  if (ok) {
    const uint8_t* c = w.code + tile * (int64_t)(192u * gp) + 3072u * s;
#pragma unroll
    for (int j = 0; j < 3; ++j) d[j] = *reinterpret_cast<const u32x4*>(c + 16u * (16u * (q * j + kb) + i));
    sc = *reinterpret_cast<const uint32_t*>(w.scale + tile * (int64_t)(16u * gp) + 256u * s + 4u * (16u * kb + i));
    cb = *reinterpret_cast<const u32x2*>(w.cb + row * 8);
  }
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    bf16x2 v[16];
    dequant_group_bf16(d[0][t], d[1][t], d[2][t], (sc >> (8 * t)) & 255u, cb.x, cb.y, v);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint32_t u = ok ? __builtin_bit_cast(uint32_t, v[e]) : 0u;
      buf[(kb * 32 + 2 * e) * kPad + wave * 16 + i] = (uint16_t)u;
      buf[(kb * 32 + 2 * e + 1) * kPad + wave * 16 + i] = (uint16_t)(u >> 16);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = c * 256 + threadIdx.x, r = at >> 3, p = at & 7;   // k row r of the 128, 8 columns
      const int64_t k = (int64_t)s * 512 + (r >> 5) * 128 + t * 32 + (r & 31);
      if (k < (int64_t)w.groups * 32)
        *reinterpret_cast<u32x4*>(out + k * np + (int64_t)blockIdx.x * 64 + 8 * p) =
            *reinterpret_cast<const u32x4*>(&buf[r * kPad + 8 * p]);
    }
    __syncthreads();
  }
}

// dy rows padded with zeros to np columns (only when n % 8 leaves a 16-byte
// piece half filled with what the caller keeps behind the row).
__global__ __launch_bounds__(256) void pad_rows_kernel(const uint16_t* __restrict__ src, int64_t ld, int64_t n,
                                                       uint16_t* __restrict__ dst, int64_t np) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c < np) dst[(int64_t)blockIdx.y * np + c] = c < n ? src[(int64_t)blockIdx.y * ld + c] : 0;
}

// ---- C = A B^T ------------------------------------------------------------------

constexpr int kMaxGemmSplits = 8;

enum Epilogue : int { kStoreF32 = 0, kGlu = 1 };

struct GemmArgs {
  const uint16_t* a;   // [m][lda], a multiple of 8 columns valid
  int64_t lda;
  const uint16_t* b;   // [rows][ldb]
  int64_t ldb;
  int64_t m, n;        // outputs (kGlu: n = I, b holds 2I rows)
  int64_t k;           // summed columns of a (k % 8 == 0); b is zero from there to the next multiple of 64
  float* c;            // split z (blockIdx.y) of the summed axis writes c + z * split_stride
  int64_t ldc;
  int64_t split_stride;
  int vec;             // c rows 16-byte aligned
  // kGlu
  uint16_t* h;
  int64_t ldh;
  float* pre;
  int64_t ld_pre;
  int act;
  int tiles_m, tiles_n;
};

// One wave's 1 KB from memory to LDS: lane l's 16 bytes at voff + soff land at
// dst + 16 l (dst is wave-uniform).
__device__ __forceinline__ void load_lds16(rsrc_t r, uint8_t* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}

// acc0 += w x0^T, acc1 += w x1^T.  In the large block (kBig) as assembly with
// the sums in accumulation registers: a wave's 256 of them are exactly that file,
// and left to the register allocator the sums move between the two files all
// through the loop.  What the compiler then does not know it need not: the
// leading s_nop covers a vector instruction that wrote an operand, a sum is next
// used 64 products later, and the last pair of a step (`last`) ends before the
// statement does (20 wait states, more than any product needs; they pass beside
// the products), so whatever follows the loop may read or move sums at once.
template <bool kBig>
__device__ __forceinline__ void mfma_pair(bf16x8 w, bf16x8 x0, bf16x8 x1, f32x4& acc0, f32x4& acc1, bool last) {
  if constexpr (kBig) {
    if (last)
      asm volatile(
          "s_nop 1\n"
          "v_mfma_f32_16x16x32_bf16 %0, %2, %3, %0\n"
          "v_mfma_f32_16x16x32_bf16 %1, %2, %4, %1\n"
          "s_nop 15\n"
          "s_nop 3\n"
          : "+a"(acc0), "+a"(acc1)
          : "v"(w), "v"(x0), "v"(x1));
    else
      asm volatile(
          "s_nop 1\n"
          "v_mfma_f32_16x16x32_bf16 %0, %2, %3, %0\n"
          "v_mfma_f32_16x16x32_bf16 %1, %2, %4, %1\n"
          : "+a"(acc0), "+a"(acc1)
          : "v"(w), "v"(x0), "v"(x1));
  } else {
    acc0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x0, acc0, 0, 0, 0);
    acc1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, x1, acc1, 0, 0, 0);
  }
}
// acc[m] += w x[m]^T, two products at a time, each pair behind beside(pair): a
// read or a load between every two products, so that the matrix core does not
// run dry while the wave issues them.
template <int TM, typename Beside>
__device__ __forceinline__ void mfma_row(bf16x8 w, const bf16x8 (&x)[TM], f32x4 (&acc)[TM], bool last,
                                         Beside&& beside) {
#pragma unroll
  for (int m = 0; m < TM; m += 2) {
    beside(m / 2);
    mfma_pair<TM == 8>(w, x[m], x[m + 1], acc[m], acc[m + 1], last && m + 2 == TM);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Block of four waves (2 x 2) on a 32 TM x 32 TN tile (tokens x weight rows), 64
// of the summed axis at a time (whole 128-byte lines: 64-byte pieces ask the L2
// twice as often, and with four buffers of 32 the L2 bound the kernel at 1.23
// PFLOP/s) through two LDS buffers filled by direct-to-LDS loads.  A step has
// two halves of 32: while the products of one half run from registers, the
// fragments of the next are read.  The second half's fragments are read early in
// the first half, so that the buffer is free and the loads of the step after
// next leave a whole step and more before they are waited for (asked for half a
// step later, a miss of the L2 held up every step).
// A buffer row is 128 bytes in 8 chunks of 16; row r keeps chunk c at position
// c ^ (r & 7) (the loads permute which chunk a lane fetches), so the 16 rows a
// fragment read touches fall on distinct banks.  Weights are the MFMA's A
// operand: a lane then holds four consecutive weight rows of one token, which
// leave in one store.
// kGlu: half of a wave's weight rows are gate rows and half the up rows of the
// same outputs, so the product is formed in registers.
template <int TM, int TN, int kEpi>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(TM * TN > 32 ? 1 : 2)))
void gemm_kernel(GemmArgs g) {
  constexpr int BM = 32 * TM, BN = 32 * TN;
  constexpr uint32_t kABytes = BM * 128, kBuf = (BM + BN) * 128;
  constexpr int kOut = kEpi == kGlu ? BN / 2 : BN;   // outputs per tile
  extern __shared__ __align__(16) uint8_t lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;

  // Tiles go to the 8 XCDs in contiguous runs (blocks are dealt round robin),
  // and inside a run in columns of up to 8 token tiles, so the blocks that
  // share an L2 share operand tiles.
  const int total = g.tiles_m * g.tiles_n;
  const int id = blockIdx.x, xcd = id & 7, per = total >> 3, rem = total & 7;
  const int t = xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
  const int gsize = 8 * g.tiles_n, grp = t / gsize, in = t - grp * gsize;
  const int gm = g.tiles_m - grp * 8 < 8 ? g.tiles_m - grp * 8 : 8;
  const int64_t m0 = (int64_t)__builtin_amdgcn_readfirstlane(grp * 8 + in % gm) * BM;   // divisions are vector work
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(in / gm) * kOut;

  // A load instruction brings 8 rows: lane l row l/8, the chunk that belongs at
  // position l%8.  Each wave loads a quarter of the token rows and a quarter
  // of the weight rows, which lie together in memory (kGlu: the gate or the
  // up rows of one wave column).
  constexpr int kLoadsA = TM, kLoadsB = TN;
  const int r8 = lane >> 3, chunk = (lane & 7) ^ r8;
  const uint32_t lda2 = (uint32_t)g.lda * 2u, ldb2 = (uint32_t)g.ldb * 2u;
  const int64_t rows_a = g.m - m0 < BM ? g.m - m0 : BM;
  const rsrc_t ra = make_rsrc(g.a + m0 * g.lda, (uint32_t)(((rows_a - 1) * g.lda + g.k) * 2));
  const int64_t b0 = kEpi == kGlu ? n0 + (wave >> 1) * (8 * TN) : n0 + wave * (8 * TN);
  const int64_t rows_b = g.n - b0;   // weight rows from b0 on (may be negative)
  const rsrc_t rb = make_rsrc(g.b + (b0 + (kEpi == kGlu && (wave & 1) ? g.n : 0)) * g.ldb, (uint32_t)(8 * TN) * ldb2);
  uint32_t va[kLoadsA], vb[kLoadsB];
#pragma unroll
  for (int q = 0; q < kLoadsA; ++q)
    va[q] = 8 * (wave * kLoadsA + q) + r8 < rows_a ? (uint32_t)r8 * lda2 + 16u * chunk : kOob;
#pragma unroll
  for (int q = 0; q < kLoadsB; ++q) vb[q] = 8 * q + r8 < rows_b ? (uint32_t)r8 * ldb2 + 16u * chunk : kOob;

  const int64_t all = (g.k + 63) / 64;
  const int s0 = (int)(all * blockIdx.y / gridDim.y), s1 = (int)(all * (blockIdx.y + 1) / gridDim.y);
  // Load q of step s into the buffer of its parity.  Steps past the last load the
  // last one again (never used), so every step has the same number in flight.
  auto load = [&](int s, int q) {
    uint8_t* buf = lds + (s & 1) * kBuf;
    const int at = s < s1 ? s : s1 - 1;
    if (q < kLoadsA) {
      // Chunks past k (only in the last step) arrive as zeros, as all loads out
      // of range do: b's zeros there would make NaN of anything infinite.
      const uint32_t v = 64 * (int64_t)at + 8 * chunk < g.k ? va[q] : kOob;
      const uint32_t row = (uint32_t)(wave * kLoadsA + q) * 8u;
      load_lds16(ra, buf + row * 128u, v, row * lda2 + 128u * (uint32_t)at);
    } else {
      const int p = q - kLoadsA;
      const uint32_t row = (uint32_t)(wave * kLoadsB + p) * 8u;
      load_lds16(rb, buf + kABytes + row * 128u, vb[p], (uint32_t)(8 * p) * ldb2 + 128u * (uint32_t)at);
    }
  };

  f32x4 acc[TN][TM];
#pragma unroll
  for (int n = 0; n < TN; ++n)
#pragma unroll
    for (int m = 0; m < TM; ++m) acc[n][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  // Fragment address: row lane%16 of a 16-row tile, chunk 4 half + lane/16, swizzled.
  const uint32_t frag = (uint32_t)(lane & 15) * 128u + (((uint32_t)lane >> 4) ^ ((uint32_t)lane & 7u)) * 16u;
  const uint32_t fa = (uint32_t)(wm * TM) * 2048u + frag;
  const uint32_t fb = kABytes + (uint32_t)(wn * TN) * 2048u + frag;
  auto read_w = [&](int s, uint32_t half, int n) {
    return *reinterpret_cast<const bf16x8*>(lds + (s & 1) * kBuf + (fb ^ 64u * half) + n * 2048u);
  };
  auto read_x = [&](int s, uint32_t half, int m) {
    return *reinterpret_cast<const bf16x8*>(lds + (s & 1) * kBuf + (fa ^ 64u * half) + m * 2048u);
  };
  struct Frags {
    bf16x8 w[TN], x[TM];
  };
  constexpr int kLoads = kLoadsA + kLoadsB;
  constexpr int kEarly = TN / 4;            // rows of products beside which a half's fragments are read
  constexpr int kLoads1 = TN - kEarly;      // loads in the first half, one a row; the rest in the second
  auto meet = [&](auto wait) {
    __builtin_amdgcn_s_waitcnt(decltype(wait)::value);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr std::integral_constant<int, 0xC07F> read_done{};   // lgkmcnt(0)
  constexpr std::integral_constant<int, kLoads1 | 0x0F70> landed{};   // vmcnt(kLoads1)
  static_assert(kLoads1 < 16, "vmcnt's low field");
  Frags f0, f1;
  if (s0 < s1) {
#pragma unroll
    for (int q = 0; q < 2 * kLoads; ++q) load(s0 + q / kLoads, q % kLoads);
  }
  meet(std::integral_constant<int, (kLoads & 15) | (kLoads >> 4) << 14 | 0x0F70>{});
#pragma unroll
  for (int n = 0; n < TN; ++n) f0.w[n] = read_w(s0, 0, n);
#pragma unroll
  for (int m = 0; m < TM; ++m) f0.x[m] = read_x(s0, 0, m);
  for (int s = s0; s < s1; ++s) {
    // First half: its products; the second half's fragments beside the first
    // rows, then the first loads of step s+2 into the buffer that is free by then.
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      mfma_row<TM>(f0.w[n], f0.x, acc[n], false, [&](int pair) {
        constexpr int kReads = (TM + TN) / kEarly / (TM / 2);   // beside each pair
        if (n < kEarly) {
#pragma unroll
          for (int i = 0; i < kReads; ++i) {
            const int f = (n * (TM / 2) + pair) * kReads + i;
            if (f < TN) f1.w[f] = read_w(s, 1, f);
            else f1.x[f - TN] = read_x(s, 1, f - TN);
          }
        } else if (pair == 1) {
          load(s + 2, n - kEarly);
        }
      });
      if (n == kEarly - 1) meet(read_done);
    }
    meet(landed);   // step s+1: all but the loads just asked for
    // Second half; the next step's first fragments and the rest of the loads.
#pragma unroll
    for (int n = 0; n < TN; ++n) {
      mfma_row<TM>(f1.w[n], f1.x, acc[n], n + 1 == TN, [&](int pair) {
        constexpr int kRest = kLoads - kLoads1;
        const int q = kLoads1 + n * kRest / TN, q1 = kLoads1 + (n + 1) * kRest / TN;
        if (pair == 0) {
          f0.w[n] = read_w(s + 1, 0, n);
#pragma unroll
          for (int m = n * TM / TN; m < (n + 1) * TM / TN; ++m) f0.x[m] = read_x(s + 1, 0, m);
        } else if (pair == 1 && q < q1) {
          load(s + 2, q);
        }
        if (pair == TM / 2 - 1 && q + 1 < q1) load(s + 2, q + 1);
      });
    }
  }
  __builtin_amdgcn_s_waitcnt(0);   // no load into LDS outlives the block

  // Lane l holds weight rows 4*(l/16)..+3 of each tile for token l%16.
#pragma unroll
  for (int m = 0; m < TM; ++m) {
    const int64_t token = m0 + (wm * TM + m) * 16 + (lane & 15);
    if (token >= g.m) continue;
    if constexpr (kEpi == kGlu) {
      constexpr int kHalfT = TN / 2;
#pragma unroll
      for (int n = 0; n < kHalfT; ++n) {
        const int64_t i = n0 + wn * 8 * TN + n * 16 + 4 * (lane >> 4);
        if (i >= g.n) continue;   // n is a multiple of 32
        const f32x4 ga = acc[n][m], up = acc[n + kHalfT][m];
        float h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = act_value(g.act, ga[e]) * up[e];
        const bf16x2 h0 = {static_cast<__bf16>(h[0]), static_cast<__bf16>(h[1])};
        const bf16x2 h1 = {static_cast<__bf16>(h[2]), static_cast<__bf16>(h[3])};
        *reinterpret_cast<u32x2*>(g.h + token * g.ldh + i) =
            u32x2{__builtin_bit_cast(uint32_t, h0), __builtin_bit_cast(uint32_t, h1)};
        if (g.pre) {
          *reinterpret_cast<f32x4*>(g.pre + token * g.ld_pre + i) = ga;
          float* pu = g.pre + token * g.ld_pre + g.n + i;   // n % 32 == 0 keeps the alignment
          *reinterpret_cast<f32x4*>(pu) = up;
        }
      }
    } else {
      float* c = g.c + (int64_t)blockIdx.y * g.split_stride + token * g.ldc;
#pragma unroll
      for (int n = 0; n < TN; ++n) {
        const int64_t i = n0 + (wn * TN + n) * 16 + 4 * (lane >> 4);
        if (g.vec && i + 3 < g.n) {
          *reinterpret_cast<f32x4*>(c + i) = acc[n][m];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (i + e < g.n) c[i + e] = acc[n][m][e];
        }
      }
    }
  }
}

template <int TM, int TN, int kEpi>
hipError_t launch_gemm_one(GemmArgs g, int splits, hipStream_t s) {
  constexpr int BM = 32 * TM, BN = 32 * TN, kOut = kEpi == kGlu ? BN / 2 : BN;
  constexpr size_t shm = 2 * (BM + BN) * 128;
  static LdsAllowance seen;
  const hipError_t e =
      allow_dynamic_lds(reinterpret_cast<const void*>(gemm_kernel<TM, TN, kEpi>), shm, seen);
  if (e != hipSuccess) return e;
  const int64_t tm = (g.m + BM - 1) / BM, tn = (g.n + kOut - 1) / kOut;
  if (tm * tn > 0xFFFFFF) return hipErrorInvalidValue;   // 2^32 threads; outputs of that size fit no card
  g.tiles_m = (int)tm;
  g.tiles_n = (int)tn;
  hipLaunchKernelGGL((gemm_kernel<TM, TN, kEpi>), dim3((unsigned)(tm * tn), (unsigned)splits),
                     dim3(256), shm, s, g);
  return hipGetLastError();
}

// Partial planes added in split order, four columns per thread.
__global__ __launch_bounds__(256) void gemm_reduce_kernel(const float* __restrict__ part, int64_t stride, int splits,
                                                          int64_t m, int64_t n, float* __restrict__ y, int64_t ldy,
                                                          int vec) {
  const int64_t nq = (n + 3) / 4, e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= m * nq) return;
  const int64_t r = e / nq, c = 4 * (e - r * nq);
  const float* p = part + r * (4 * nq) + c;   // plane rows are padded to four columns
  f32x4 v[kMaxGemmSplits];
#pragma unroll
  for (int z = 0; z < kMaxGemmSplits; ++z)
    v[z] = z < splits ? *reinterpret_cast<const f32x4*>(p + z * stride) : f32x4{0.f, 0.f, 0.f, 0.f};
  f32x4 acc = v[0];
#pragma unroll
  for (int z = 1; z < kMaxGemmSplits; ++z) acc += v[z];
  float* o = y + r * ldy + c;
  if (vec && c + 3 < n) {
    *reinterpret_cast<f32x4*>(o) = acc;
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (c + q < n) o[q] = acc[q];
  }
}

// Block shape and splits of the summed axis for m tokens, n outputs (weight
// rows) and k summed.
struct GemmPlan {
  bool big;     // 256 x 256 blocks, else 128 x 128
  int splits;
};
// From 192 large blocks on they fill most of the 256 CUs, and each operand byte
// read serves twice the products; below, four times as many small ones balance
// better.  Measured, large and small (us): 160 blocks (2048 tokens x 5120 x 4096)
// 102 and 98; 192 (2048 x 6144 x 4096) 104 and 103, (2048 x 6144 x 8192) 196 and
// 221; 200 (2560 x 5120 x 5120) 126 and 151; 256 (1024 x 16384 x 4096) 130 and 155;
// 128 (2048 x 4096 x 11008) 246 and 191.
GemmPlan plan_gemm(int64_t m, int64_t n, int64_t k, bool may_split) {
  GemmPlan p{((m + 255) / 256) * ((n + 255) / 256) >= 192, 1};
  if (p.big || !may_split) return p;
  // Two 128 x 128 blocks fit a CU.  Fewer tiles leave CUs idle or with one: the
  // summed axis is split, at eight or more steps of 64 each, so that the partial
  // planes stay small next to the products.  From 224 tiles on nearly every CU
  // has one and a split only adds planes.  Measured, split and not (us), 512
  // tokens: 1024 x 4096 23 and 43, 4096 x 14336 98 and 139, 5120 x 8192 65 and 80,
  // 6144 x 8192 77 and 84, 7168 x 8192 86 and 86, 8192 x 8192 115 and 92.
  const int64_t tiles = ((m + 127) / 128) * ((n + 127) / 128), steps = (k + 63) / 64;
  int64_t s = tiles >= 224 ? 1 : 512 / (tiles > 0 ? tiles : 1);
  s = s < steps / 8 ? s : steps / 8;
  s = s < kMaxGemmSplits ? s : kMaxGemmSplits;
  p.splits = s > 1 ? (int)s : 1;
  return p;
}
int64_t plane_floats(int64_t m, int64_t n) { return m * ((n + 3) / 4 * 4); }
int64_t split_bytes(int64_t m, int64_t n, int64_t k) {
  const GemmPlan p = plan_gemm(m, n, k, true);
  return p.splits > 1 ? p.splits * plane_floats(m, n) * 4 : 0;
}

hipError_t launch_glu_gemm(const GemmArgs& g, hipStream_t s) {
  if (plan_gemm(g.m, 2 * g.n, g.k, false).big) return launch_gemm_one<8, 8, kGlu>(g, 1, s);
  return launch_gemm_one<4, 4, kGlu>(g, 1, s);
}

// part: split_bytes(m, n, k) bytes, 16-byte aligned.
hipError_t launch_f32_gemm(GemmArgs g, float* part, hipStream_t s) {
  const GemmPlan p = plan_gemm(g.m, g.n, g.k, true);
  if (p.splits == 1) {
    if (p.big) return launch_gemm_one<8, 8, kStoreF32>(g, 1, s);
    return launch_gemm_one<4, 4, kStoreF32>(g, 1, s);
  }
  float* y = g.c;
  const int64_t ldy = g.ldc;
  const int vec = g.vec;
  g.c = part;
  g.ldc = (g.n + 3) / 4 * 4;
  g.split_stride = plane_floats(g.m, g.n);
  g.vec = 1;
  const hipError_t e = launch_gemm_one<4, 4, kStoreF32>(g, p.splits, s);
  if (e != hipSuccess) return e;
  const int64_t blocks = (g.m * ((g.n + 3) / 4) + 255) / 256;
  hipLaunchKernelGGL(gemm_reduce_kernel, dim3((unsigned)blocks), dim3(256), 0, s, part, g.split_stride, p.splits, g.m,
                     g.n, y, ldy, vec);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }
int64_t padded_k(int64_t k) { return (k + 127) / 128 * 128; }
int64_t padded_n(int64_t n) { return (n + 63) / 64 * 64; }
constexpr int64_t kSmallM = 64;

// Tokens that go through the packed planes at a time, and in how many passes at
// most; more are multiplied with the widened matrix.  On whole 512-k steps a pass
// takes 128: a product's K is split until the chip is full, so passes pay in
// proportion to the matrix; a gated pass takes the same time up to 32768 rows
// (a pair of tiles per SIMD), and widening a time that grows with them.  Elsewhere
// a pass takes 64, which fills the chip on tall matrices only.  Measured, passes
// and widening (us), at K = 4096 where not said:
//   products  4096 rows, 128 tokens 22 and 26, 256 43 and 33; 4096 x 14336, 256 59
//             and 65, 300 78 and 73; 8192 x 8192, 384 87 and 96; 11008, 256 57 and
//             54; 14336, 256 59 and 64, 384 89 and 73; 28672, 384 120 and 153, 512
//             160 and 155; 100000, 384 468 and 580
//   gated     1024 x 1024, 128 tokens 15 and 18; 16384 rows, 128 39 and 64, 256 78
//             and 66; 22016, 384 118 and 144; 28672, 384 118 and 165, 512 158 and
//             160; 57344 x 8192, 384 433 and 576
//   by 64     11008, 128 34 and 46; 14336, 192 55 and 61, 256 70 and 64; 18432, 256
//             121 and 88; 28672, 384 141 and 153; 65536, 512 347 and 335
// and 128 a pass against 64: 28672, 128 40 and 47; 8192 x 8192, 128 30 and 53.
struct Passes {
  int64_t tokens, most;
};
Passes passes_of(int64_t n, int64_t k, bool glu) {
  auto clamp = [](int64_t v, int64_t hi) { return v < 1 ? 1 : (v > hi ? hi : v); };
  if (k % 512 == 0) return {128, glu ? (n >= 20000 ? 3 : 1) : clamp(n * k / 22000000, 3)};
  return {kSmallM, clamp(n / 4700, 7)};
}
bool in_passes(int64_t n, int64_t k, int64_t m, bool glu) {
  const Passes p = passes_of(n, k, glu);
  return m <= p.tokens * p.most;
}

hipError_t launch_widen(const PlaneView& w, uint16_t* out, hipStream_t s) {
  const uint32_t gp = (uint32_t)((w.groups + 3) & ~3);
  const int steps = (int)((gp + 15) / 16);
  const int64_t units = (w.n + 15) / 16 * steps;
  hipLaunchKernelGGL(widen_kernel, dim3((unsigned)((units + 3) / 4)), dim3(256), 0, s, w, out, units, steps);
  return hipGetLastError();
}

// The gradient of the gated pre-activations, four outputs per thread.
__global__ __launch_bounds__(256) void glu_back_kernel(const float* __restrict__ pre, int64_t ld_pre,
                                                       const float* __restrict__ dh, int64_t ld_dh, int act,
                                                       int64_t quads, int64_t inter, uint16_t* __restrict__ dpre,
                                                       int64_t ld_dpre) {
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= quads) return;
  const int64_t per = inter / 4, row = e / per, i = 4 * (e - row * per);
  const f32x4 ga = *reinterpret_cast<const f32x4*>(pre + row * ld_pre + i);
  const f32x4 up = *reinterpret_cast<const f32x4*>(pre + row * ld_pre + inter + i);
  const f32x4 d = *reinterpret_cast<const f32x4*>(dh + row * ld_dh + i);
  uint32_t og[2], ou[2];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float g2[2], u2[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float a, da;
      act_both(act, ga[2 * p + q], a, da);
      g2[q] = d[2 * p + q] * up[2 * p + q] * da;
      u2[q] = d[2 * p + q] * a;
    }
    const bf16x2 gb = {static_cast<__bf16>(g2[0]), static_cast<__bf16>(g2[1])};
    const bf16x2 ub = {static_cast<__bf16>(u2[0]), static_cast<__bf16>(u2[1])};
    og[p] = __builtin_bit_cast(uint32_t, gb);
    ou[p] = __builtin_bit_cast(uint32_t, ub);
  }
  *reinterpret_cast<u32x2*>(dpre + row * ld_dpre + i) = u32x2{og[0], og[1]};
  *reinterpret_cast<u32x2*>(dpre + row * ld_dpre + inter + i) = u32x2{ou[0], ou[1]};
}

}  // namespace

int64_t gemm_workspace_bytes(int64_t n, int64_t k, int64_t m) {
  if (in_passes(n, k, m, false)) {
    int64_t most = 0;
    const int64_t step = passes_of(n, k, false).tokens;
    for (int64_t c : {m < step ? m : step, m % step}) {
      if (c == 0) continue;
      const int64_t b = c > kSmallM ? gemm_mid_workspace_bytes(n, k, c) : gemm_small_m_workspace_bytes(n, k, c);
      most = most > b ? most : b;
    }
    return most;
  }
  return align256(n * padded_k(k) * 2) + align256(split_bytes(m, n, k));
}

hipError_t launch_gemm(const PlaneView& w, const uint16_t* x, int64_t m, int64_t ldx, float* y, int64_t ldy, void* ws,
                       hipStream_t s) {
  const int64_t k = (int64_t)w.groups * 32;
  if (w.n == 0) return hipSuccess;
  if (in_passes(w.n, k, m, false)) {
    const int64_t bytes = ws ? gemm_workspace_bytes(w.n, k, m) : 0, step = passes_of(w.n, k, false).tokens;
    for (int64_t i = 0; i < m; i += step) {
      const int64_t c = m - i < step ? m - i : step;
      const hipError_t e = c > kSmallM ? launch_gemm_mid(w, x + i * ldx, c, ldx, y + i * ldy, ldy, ws, s)
                                       : launch_gemm_small_m(w, x + i * ldx, c, ldx, y + i * ldy, ldy, ws, bytes, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  uint16_t* wide = static_cast<uint16_t*>(ws);
  const hipError_t e = launch_widen(w, wide, s);
  if (e != hipSuccess) return e;
  GemmArgs g{};
  g.a = x;
  g.lda = ldx;
  g.b = wide;
  g.ldb = padded_k(k);
  g.m = m;
  g.n = w.n;
  g.k = k;
  g.c = y;
  g.ldc = ldy;
  g.vec = (uintptr_t)y % 16 == 0 && ldy % 4 == 0;
  return launch_f32_gemm(g, reinterpret_cast<float*>(wide + align256(w.n * padded_k(k) * 2) / 2), s);
}

int64_t gemm_backward_workspace_bytes(int64_t n, int64_t k, int64_t m) {
  return align256(k * padded_n(n) * 2) + (n % 8 ? align256(m * padded_n(n) * 2) : 0) + align256(split_bytes(m, k, n));
}

hipError_t launch_gemm_backward(const PlaneView& w, const uint16_t* dy, int64_t m, int64_t ld_dy, float* dx,
                                int64_t ld_dx, void* ws, hipStream_t s) {
  const int64_t k = (int64_t)w.groups * 32, np = padded_n(w.n);
  uint16_t* wide = static_cast<uint16_t*>(ws);
  if (w.n > 0) {
    const int steps = (int)(((w.groups + 3) / 4 + 3) / 4);
    hipLaunchKernelGGL(widen_t_kernel, dim3((unsigned)(np / 64), (unsigned)steps), dim3(256), 0, s, w, wide, np);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  GemmArgs g{};
  g.a = dy;
  g.lda = ld_dy;
  g.k = w.n;
  uint16_t* rest = wide + align256(k * np * 2) / 2;
  if (w.n % 8) {
    uint16_t* padded = rest;
    rest += align256(m * np * 2) / 2;
    for (int64_t r = 0; r < m; r += 65535) {   // grid rows of one launch
      const int64_t rows = m - r < 65535 ? m - r : 65535;
      hipLaunchKernelGGL(pad_rows_kernel, dim3((unsigned)((np + 255) / 256), (unsigned)rows), dim3(256), 0, s,
                         dy + r * ld_dy, ld_dy, w.n, padded + r * np, np);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.a = padded;
    g.lda = np;
    g.k = (w.n + 7) / 8 * 8;
  }
  g.b = wide;
  g.ldb = np;
  g.m = m;
  g.n = k;
  g.c = dx;
  g.ldc = ld_dx;
  g.vec = (uintptr_t)dx % 16 == 0 && ld_dx % 4 == 0;
  return launch_f32_gemm(g, reinterpret_cast<float*>(rest), s);
}

int64_t glu_workspace_bytes(int64_t n_gu, int64_t k, int64_t m) {
  return in_passes(n_gu, k, m, true) ? 0 : align256(n_gu * padded_k(k) * 2);
}

hipError_t launch_glu(const PlaneView& gate_up, const uint16_t* x, int64_t m, int64_t ldx, int32_t act, uint16_t* h,
                      int64_t ldh, float* pre, int64_t ld_pre, void* ws, hipStream_t s) {
  if (gate_up.n == 0) return hipSuccess;
  const int64_t k = (int64_t)gate_up.groups * 32;
  if (in_passes(gate_up.n, k, m, true)) {
    const int64_t step = passes_of(gate_up.n, k, true).tokens;
    for (int64_t i = 0; i < m; i += step) {
      const int64_t c = m - i < step ? m - i : step;
      float* p = pre ? pre + i * ld_pre : nullptr;
      const hipError_t e =
          c > kSmallM ? launch_glu_mid(gate_up, x + i * ldx, c, ldx, act, h + i * ldh, ldh, p, ld_pre, s)
                      : launch_glu_small_m(gate_up, x + i * ldx, c, ldx, act, h + i * ldh, ldh, p, ld_pre, s);
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  uint16_t* wide = static_cast<uint16_t*>(ws);
  const hipError_t e = launch_widen(gate_up, wide, s);
  if (e != hipSuccess) return e;
  GemmArgs g{};
  g.a = x;
  g.lda = ldx;
  g.b = wide;
  g.ldb = padded_k(k);
  g.m = m;
  g.n = gate_up.n / 2;
  g.k = k;
  g.h = h;
  g.ldh = ldh;
  g.pre = pre;
  g.ld_pre = ld_pre;
  g.act = act;
  return launch_glu_gemm(g, s);
}

hipError_t launch_glu_backward(const float* pre, int64_t ld_pre, const float* dh, int64_t ld_dh, int32_t act,
                               int64_t m, int64_t inter, uint16_t* dpre, int64_t ld_dpre, hipStream_t s) {
  const int64_t quads = m * (inter / 4), blocks = (quads + 255) / 256;
  if (blocks > 0xFFFFFF) return hipErrorInvalidValue;   // 2^32 threads
  if (quads == 0) return hipSuccess;
  hipLaunchKernelGGL(glu_back_kernel, dim3((unsigned)blocks), dim3(256), 0, s, pre, ld_pre, dh, ld_dh, act, quads,
                     inter, dpre, ld_dpre);
  return hipGetLastError();
}

}  // namespace q3
