// Sampling: one token per row of logits from a given random number, under
// temperature, top-k, top-p and min-p.
//
// With w = exp((l - max l)/T) and the entries ranked by logit (ties: lower
// index), all three truncations keep a prefix of that ranking, so the kept set
// is "everything up to one entry" and no sort of the row is needed.  The
// weights are integers q = round(2^44 w): their sums are exact in 64 bits in
// any order (n <= 2^19), so chunks, atomics and scans give one result and the
// running sums the draw compares are those the total is made of.
//
// A row is cut into up to 16 chunks; five launches:
//   stats    per chunk: largest and smallest logit
//   hist     per chunk: entry counts and weights over 1024 bins of max l - l
//            (equal steps over the row's span, at most 32 T; the last bin
//            takes the rest), as running sums over the bins.  The bin is a
//            monotone function of the logit.
//   border   per row: the bins in which top-k, top-p and min-p can fall
//   collect  per chunk: the list of the entries inside those bins (a few hundred)
//   choose   per row: the list is sorted, which gives the exact cut; the kept
//            weight of each chunk follows from its running sums and the list,
//            and u times the total is found in a chunk, a wave's part of it and
//            an entry
// Short rows, and rows of which there are many, take the same five steps in one
// block and launch.  A row whose border bins hold more than kCand entries with
// weight (ties: logits that were rounded to few bits, or an outlier that widens the
// bins) is cut by bisection over the logits' 32-bit order instead, in the last step:
// some 35 passes of one block over the row, twice that with top-k and top-p
// (64 x 151936 rounded to bf16 around 10 with a deviation of 1, top-p 0.9: 2700 us,
// with top-k 5000 as well 3430; 33 x 50257 fits the list, 52).
//
// What bounds it: for few rows the chain of some twenty block-wide sums and
// minima, about 0.5 us each with their two barriers, and the launches (1 x 1000
// 15 us, 1 x 32000 27 us); for many the hist pass's 64-bit exponential for every
// entry and its second evaluation where the draw falls (64 x 151936 60 us, of
// which hist 19, choose 19; 4 copies of the sums against lanes that meet at a
// bin change nothing).  The row is read from memory once, then from cache.
#include <type_traits>

#include "q3_device.h"
#include "q3_internal.h"

namespace q3 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxChunks = 16;     // per row
constexpr int kBins = 1024;        // one per thread
constexpr int kCand = 2048;        // listed entries per row
constexpr int kNone = kBins;       // "no border": after every bin

struct RowInfo {
  uint64_t mass_lo;    // weight of the bins before lo
  uint64_t mass_bk;    // weight of the bins before bk
  uint64_t total;      // weight of the row
  float mx, c;         // the row's binning
  int lo, hi;          // the cut is in bins lo..hi (kNone: nothing is cut)
  int bk;              // the bin of rank top_k (kNone: no such bin)
  int cnt_lo, cnt_bk;  // entries in the bins before lo and before bk
  int want_bk;         // bk's entries are listed too, for the weight of the top_k entries
};

struct Ws {
  float2* stats;         // [m][chunks] (max, min)
  RowInfo* info;         // [m]
  int* listed;           // [m] entries listed (more than kCand: bisection)
  uint32_t* hist_cnt;    // [m][chunks][kBins] running sums (rows with top-k only)
  uint64_t* hist_mass;   // [m][chunks][kBins] running sums
  uint64_t* cand;        // [m][kCand] (order << 32 | index)
};

// A row's settings as they act: t > 0, k >= 1 (n when off), top-p and min-p
// with their off values.
struct Settings {
  double inv_t;
  double inv_t2;   // log2(e) / t
  float t;
  int k;
  double p, min_p;
  bool use_p, use_min;
};
__device__ __forceinline__ Settings settings(const SampleArgs& a, int row) {
  Settings s;
  float t = a.temperature ? a.temperature[row] : 1.f;
  const bool greedy = t <= 0.f;
  if (!(t > 0.f)) t = 1.f;
  s.t = t;
  s.inv_t = 1.0 / (double)t;
  s.inv_t2 = 1.4426950408889634 * s.inv_t;
  const int k = a.top_k ? a.top_k[row] : 0;
  s.k = greedy ? 1 : (k > 0 && k < a.n ? k : a.n);
  const float p = a.top_p ? a.top_p[row] : 1.f;
  s.use_p = p < 1.f && !greedy;
  s.p = p;
  const float mp = a.min_p ? a.min_p[row] : 0.f;
  s.use_min = mp > 0.f && !greedy;
  s.min_p = mp > 1.f ? 1.0 : (double)mp;
  return s;
}

// Order-preserving image of a logit; -0 counts as +0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t k) {
  return __builtin_bit_cast(float, (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// Entries that can be chosen: not NaN, not -inf, and the maximum itself when
// that is +inf.
__device__ __forceinline__ bool live(float l, float mx) { return l > -INFINITY && (mx < INFINITY || l == mx); }

// p f + c in one instruction with c in scalar registers (left to the compiler,
// each step also copies its constant into the accumulator).
__device__ __forceinline__ double fma_const(double p, double f, double c) {
  double r;
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(r) : "v"(p), "v"(f), "s"(c));
  return r;
}

// 2^44 exp((l - mx)/t), rounded to an integer: 2^x = 2^n 2^f with |f| <= 1/2 and
// 2^f by the polynomial of degree 10 through its values at the 11 Chebyshev
// nodes of [-1/2, 1/2] (error below 2^-51, exact at 0; the integers' half step
// at w = 1 is 2^-45).
__device__ __forceinline__ uint64_t weight(float l, float mx, double inv_t2) {
  const double x = l == mx ? 0.0 : ((double)l - (double)mx) * inv_t2;
  const double n = __builtin_rint(x), f = x - n;
  double p = fma_const(7.072585949269223e-09, f, 1.0208690299958306e-07);
  p = fma_const(p, f, 1.321544258792169e-06);
  p = fma_const(p, f, 1.5252657260200837e-05);
  p = fma_const(p, f, 0.0001540353044173605);
  p = fma_const(p, f, 0.0013333558230164974);
  p = fma_const(p, f, 0.009618129107606888);
  p = fma_const(p, f, 0.05550410866444772);
  p = fma_const(p, f, 0.24022650695910097);
  p = fma_const(p, f, 0.69314718055995);
  p = fma_const(p, f, 1.0);
  // Adding 2^52 leaves the rounded integer in the low bits.
  const double w = __builtin_ldexp(p, (int)n + 44) + 4503599627370496.0;
  return x > -46.0 ? __builtin_bit_cast(uint64_t, w) & 0x000FFFFFFFFFFFFFull : 0;
}

// Bins of equal steps of mx - l over the row's span, at most 32 temperatures.
struct Binning {
  float mx, c;
};
__device__ __forceinline__ Binning binning(float mx, float mn, float t) {
  const float span = fminf(mx - mn, 32.f * t);   // mx = +inf: only the maximum is live
  float c = span < INFINITY ? (float)(kBins - 1) / span : 0.f;
  if (!(c < 3e38f)) c = 3e38f;
  return {mx, c};
}
__device__ __forceinline__ int bin_of(float l, const Binning& b) {
  if (l == b.mx) return 0;
  const float t = (b.mx - l) * b.c;
  return t < (float)(kBins - 1) ? (int)t : kBins - 1;   // NaN goes to the last
}

// ---- wave-wide helpers --------------------------------------------------------
//
// Lane exchanges as operand modifiers (DPP): a step through LDS permutes takes
// some 65 cycles and the choose launch has over a hundred of them in a row.

enum Dpp : int { kQuad1032 = 0xB1, kQuad2301 = 0x4E, kQuad3210 = 0x1B, kShr1 = 0x111, kShr2 = 0x112, kShr4 = 0x114,
                 kShr8 = 0x118, kRor8 = 0x128, kHalfMirror = 0x141, kBcast15 = 0x142, kBcast31 = 0x143 };
// The value of the lane that `kCtrl` names; lanes without one, and rows outside
// kRows, get `none`.
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t none) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, kCtrl, kRows, 0xF, false);
}
template <int kCtrl, int kRows = 0xF>
__device__ __forceinline__ uint64_t dpp(uint64_t v, uint64_t none) {
  return (uint64_t)dpp<kCtrl, kRows>((uint32_t)(v >> 32), (uint32_t)(none >> 32)) << 32 |
         dpp<kCtrl, kRows>((uint32_t)v, (uint32_t)none);
}
// Folds the wave's values up to and with each lane: inside rows of 16, then over
// the rows (the last lane of a row, then of the lower half, to what follows).
// `none` is op's neutral value.
template <typename T, typename Op>
__device__ __forceinline__ T wave_fold(T v, T none, Op&& op) {
  v = op(v, dpp<kShr1>(v, none));
  v = op(v, dpp<kShr2>(v, none));
  v = op(v, dpp<kShr4>(v, none));
  v = op(v, dpp<kShr8>(v, none));
  v = op(v, dpp<kBcast15, 0xA>(v, none));
  v = op(v, dpp<kBcast31, 0xC>(v, none));
  return v;
}
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
  return wave_fold(v, (uint64_t)0, [](uint64_t x, uint64_t y) { return x + y; });
}
__device__ __forceinline__ uint32_t last_lane(uint32_t v) { return (uint32_t)__builtin_amdgcn_readlane((int)v, 63); }
__device__ __forceinline__ uint64_t last_lane(uint64_t v) {
  return (uint64_t)last_lane((uint32_t)(v >> 32)) << 32 | last_lane((uint32_t)v);
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) { return last_lane(wave_scan(v)); }
__device__ __forceinline__ int wave_min(int v) {
  return (int)last_lane(wave_fold((uint32_t)v, 0x7FFFFFFFu, [](uint32_t x, uint32_t y) {
    return (int)y < (int)x ? y : x;
  }));
}
__device__ __forceinline__ float wave_max(float v) {
  return __builtin_bit_cast(float, last_lane(wave_fold(__builtin_bit_cast(uint32_t, v), 0xFF800000u,
                                                       [](uint32_t x, uint32_t y) {
    return __builtin_bit_cast(uint32_t, fmaxf(__builtin_bit_cast(float, x), __builtin_bit_cast(float, y)));
  })));
}
// The value of lane l ^ kBit.
template <int kBit>
__device__ __forceinline__ uint32_t lane_xor(uint32_t v) {
  if constexpr (kBit == 1) return dpp<kQuad1032>(v, v);
  if constexpr (kBit == 2) return dpp<kQuad2301>(v, v);
  if constexpr (kBit == 4) {
    const uint32_t m = dpp<kHalfMirror>(v, v);   // l ^ 7, then ^ 3
    return dpp<kQuad3210>(m, m);
  }
  if constexpr (kBit == 8) return dpp<kRor8>(v, v);
  if constexpr (kBit >= 16) return (uint32_t)__shfl_xor((int)v, kBit, 64);
}
template <int kBit>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
  return (uint64_t)lane_xor<kBit>((uint32_t)(v >> 32)) << 32 | lane_xor<kBit>((uint32_t)v);
}

// ---- block-wide helpers (kThreads threads) ----------------------------------

// Inclusive prefix sum over the block; `part` holds kWaves values.  Leading
// barrier included, so `part` may be reused at once.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  v = wave_scan(v);
  __syncthreads();
  if (lane == 63) part[wave] = v;
  __syncthreads();
  uint64_t before = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) before += w < wave ? part[w] : 0;
  return v + before;
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* part) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t s = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += part[w];
  return s;
}
// The smallest value over the block.
__device__ __forceinline__ int block_min(int v, int* part) {
  v = wave_min(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  int s = part[0];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) s = part[w] < s ? part[w] : s;
  return s;
}
__device__ __forceinline__ float2 row_stats(const float2* st, int chunks) {
  float2 r = make_float2(-INFINITY, INFINITY);
  for (int c = threadIdx.x & 63; c < chunks; c += 64) {
    const float2 v = st[c];
    r.x = fmaxf(r.x, v.x);
    r.y = fminf(r.y, v.y);
  }
  r.x = wave_max(r.x);
  r.y = -wave_max(-r.y);
  return r;
}

// ---- launches -----------------------------------------------------------------

// Entries [begin, end) of a chunk.
struct Range {
  int begin, end;
};
__device__ __forceinline__ Range chunk_range(int c, int per, int n) {
  return {c * per, (c + 1) * per < n ? (c + 1) * per : n};
}

// The block's entries of a range in batches of kBatch per thread, each batch
// loaded while the one before it is used; the first one when the object is
// made.  Places past the range hold -inf.
template <int kBatch>
struct Entries {
  const float* l;
  int begin, end;
  float a[kBatch], b[kBatch];
  __device__ __forceinline__ void load(float (&v)[kBatch], int base) const {
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int i = base + q * kThreads + (int)threadIdx.x;
      const float x = l[i < end ? i : end - 1];   // ranges are not empty; no branch around the load
      v[q] = i < end ? x : -INFINITY;
    }
  }
  __device__ __forceinline__ Entries(const float* l_, Range r) : l(l_), begin(r.begin), end(r.end) { load(a, begin); }
  // f(logit, index); called once.
  template <typename F>
  __device__ __forceinline__ void each(F&& f) {
    constexpr int kStep = kBatch * kThreads;
    for (int base = begin; base < end; base += 2 * kStep) {
      load(b, base + kStep);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) f(a[q], base + q * kThreads + (int)threadIdx.x);
      if (base + kStep >= end) break;
      load(a, base + 2 * kStep);
#pragma unroll
      for (int q = 0; q < kBatch; ++q) f(b[q], base + kStep + q * kThreads + (int)threadIdx.x);
    }
  }
};

// Largest and smallest live logit of the block's range (infinities when there is none).
__device__ __forceinline__ float2 range_stats(const float* l, Range r, float2* part) {
  float mx = -INFINITY, mn = INFINITY;
  Entries<8> in(l, r);
  in.each([&](float v, int) {
    mx = fmaxf(mx, v);   // NaN leaves the other operand
    mn = v > -INFINITY ? fminf(mn, v) : mn;
  });
  mx = wave_max(mx);
  mn = -wave_max(-mn);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(mx, mn);
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) {
    mx = fmaxf(mx, part[w].x);
    mn = fminf(mn, part[w].y);
  }
  return make_float2(mx, mn);
}

// Entry counts (only top-k asks for them) and weights of a range over the bins,
// which the caller has cleared.
__device__ __forceinline__ void range_hist(Entries<4>& in, const Settings& s, const Binning& b, bool counts,
                                           uint32_t* cnt, unsigned long long* mass) {
  in.each([&](float v, int) {
    const int k = bin_of(v, b);
    const uint64_t q = weight(v, b.mx, s.inv_t2);   // 0 for masked entries
    if (counts && live(v, b.mx)) atomicAdd(&cnt[k], 1u);
    if (q) atomicAdd(&mass[k], (unsigned long long)q);
  });
}

__global__ __launch_bounds__(kThreads) void sample_stats_kernel(SampleArgs a, Ws ws, int per) {
  __shared__ float2 part[kWaves];
  const int row = blockIdx.y, c = blockIdx.x;
  const float2 st = range_stats(a.logits + (int64_t)row * a.ld, chunk_range(c, per, a.n), part);
  if (threadIdx.x == 0) {
    ws.stats[(int64_t)row * gridDim.x + c] = st;
    if (c == 0) ws.listed[row] = 0;
  }
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, Ws ws, int per) {
  __shared__ uint32_t cnt[kBins];
  __shared__ unsigned long long mass[kBins];
  __shared__ uint64_t part[kWaves];
  const int row = blockIdx.y, c = blockIdx.x, chunks = gridDim.x;
  Entries<4> in(a.logits + (int64_t)row * a.ld, chunk_range(c, per, a.n));
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const Settings s = settings(a, row);
  const Binning b = binning(st.x, st.y, s.t);
  const bool counts = s.k < a.n;
  cnt[threadIdx.x] = 0;
  mass[threadIdx.x] = 0;
  __syncthreads();
  range_hist(in, s, b, counts, cnt, mass);
  __syncthreads();
  const int64_t at = ((int64_t)row * chunks + c) * kBins + threadIdx.x;
  ws.hist_mass[at] = block_scan(mass[threadIdx.x], part);
  if (counts) ws.hist_cnt[at] = (uint32_t)block_scan(cnt[threadIdx.x], part);
}

// The bins in which the row's cut can fall, from the sums up to and with each
// bin (thread t's own mi and ci are those of bin t).
__device__ RowInfo find_border(const Settings& s, const Binning& b, bool counts, uint64_t mi, uint32_t ci,
                               const uint64_t* mass_in, const uint32_t* cnt_in, int* ipart) {
  const int t = threadIdx.x;
  const uint64_t total = mass_in[kBins - 1];
  const uint32_t entries = cnt_in[kBins - 1];
  auto first = [&](bool hit) { return block_min(hit ? t : kNone, ipart); };
  auto mass_before = [&](int k) -> uint64_t { return k > 0 ? mass_in[k - 1] : 0; };
  // The bin of the last of the top_k entries.  Where nothing from that bin on has
  // weight, top-k cuts nothing that could be chosen: the last bin takes all that is
  // 32 T below the maximum, at a low temperature most of the row, and listing it
  // would send the row to the bisection (64 x 151936 at T = 0.01, top_k = 50: 2289 us).
  int bk = (uint32_t)s.k < entries ? first(ci >= (uint32_t)s.k) : kNone;
  if (mass_before(bk) == total) bk = kNone;
  // The weight of the top_k entries lies between the sums before and after
  // that bin, and top-p's border between the bins where p times those fall.
  int lo = bk, hi = bk;
  if (s.use_p) {
    const uint64_t s_lo = bk == kNone ? total : (bk ? mass_in[bk - 1] : 0);
    const uint64_t s_hi = bk == kNone ? total : mass_in[bk];
    const int p_lo = first((double)mi >= s.p * (double)s_lo);
    const int p_hi = s_lo == s_hi ? p_lo : first((double)mi >= s.p * (double)s_hi);
    lo = min(lo, p_lo);
    hi = min(hi, p_hi);
  }
  if (s.use_min) {
    // Entries at x = (mx - l)/t = -ln min_p are the border; the bin arithmetic
    // in fp32 is good to 1e-6 of the bin's position, so 1e-5 either side holds it.
    const float dm = (float)(-log(s.min_p) * (double)s.t);
    const int m_lo = bin_of(b.mx - dm * 1.00001f, b), m_hi = bin_of(b.mx - dm * 0.99999f, b);
    // b.mx - d rounds by up to 2^-24 of max(|mx|, d); take the neighbours too.
    const float slack = 4e-7f * (fabsf(b.mx) + dm) * b.c;
    const int e_lo = max(0, min(m_lo, m_hi) - 1 - (slack < kBins ? (int)slack : kBins));
    const int e_hi = min(kBins - 1, max(m_lo, m_hi) + 1 + (slack < kBins ? (int)slack : kBins));
    // As for top-k: no border among entries without weight, and none of the last bin's listed.
    if (mass_before(e_lo) != total) {
      lo = min(lo, e_lo);
      hi = min(hi, mass_before(kBins - 1) == total ? min(e_hi, kBins - 2) : e_hi);
    }
  }
  RowInfo r;
  // Without counts only whether there are entries before matters (bin 0 holds the maximum).
  auto cnt_before = [&](int k) -> int { return k > 0 ? (counts ? (int)cnt_in[k - 1] : 1) : 0; };
  r.total = total;
  r.mx = b.mx;
  r.c = b.c;
  r.lo = lo;
  r.hi = hi;
  r.bk = bk;
  r.want_bk = s.use_p && bk != kNone && !(lo <= bk && bk <= hi);
  r.mass_lo = mass_before(lo);
  r.cnt_lo = cnt_before(lo);
  r.mass_bk = mass_before(bk);
  r.cnt_bk = cnt_before(bk);
  return r;
}

// A launch of its own: found by every collect block for itself, the sums' reads
// cost more than the launch (64x151936: 5 + 9 us against 20 in one).
__global__ __launch_bounds__(kThreads) void sample_border_kernel(SampleArgs a, Ws ws, int chunks) {
  __shared__ uint64_t mass_in[kBins];   // sums up to and with each bin
  __shared__ uint32_t cnt_in[kBins];
  __shared__ int ipart[kWaves];
  const int row = blockIdx.x, t = threadIdx.x;
  const Settings s = settings(a, row);
  const bool counts = s.k < a.n;
  uint64_t mi = 0;
  uint32_t ci = 0;
  const int64_t at = (int64_t)row * chunks * kBins + t;
#pragma unroll
  for (int c = 0; c < kMaxChunks; ++c) {   // all loads before the first use
    mi += c < chunks ? ws.hist_mass[at + (int64_t)c * kBins] : 0;
    ci += counts && c < chunks ? ws.hist_cnt[at + (int64_t)c * kBins] : 0;
  }
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const Binning b = binning(st.x, st.y, s.t);
  mass_in[t] = mi;
  cnt_in[t] = ci;
  __syncthreads();
  const RowInfo r = find_border(s, b, counts, mi, ci, mass_in, cnt_in, ipart);
  if (t == 0) ws.info[row] = r;
}

// The entries of a range inside the border's bins, in any order: larger logit
// first, then lower index is "greater is ranked earlier" with ~index below.
__device__ __forceinline__ void range_list(Entries<8>& in, const RowInfo& r, uint64_t* list, int& count) {
  const int lo = r.lo, hi = r.hi, bk = r.want_bk ? r.bk : -1;
  const Binning b{r.mx, r.c};
  in.each([&](float v, int i) {
    const int k = bin_of(v, b);
    if (((k >= lo && k <= hi) || k == bk) && live(v, b.mx)) {
      const int at = atomicAdd(&count, 1);
      if (at < kCand) list[at] = (uint64_t)order_of(v) << 32 | (uint32_t)~i;
    }
  });
}

__global__ __launch_bounds__(kThreads) void sample_collect_kernel(SampleArgs a, Ws ws, int per) {
  __shared__ uint64_t list[kCand];
  __shared__ int count, base;
  const int row = blockIdx.y, c = blockIdx.x, t = threadIdx.x;
  Entries<8> in(a.logits + (int64_t)row * a.ld, chunk_range(c, per, a.n));
  const RowInfo& r = ws.info[row];
  if (r.lo == kNone) return;   // nothing is cut
  if (t == 0) count = 0;
  __syncthreads();
  range_list(in, r, list, count);
  __syncthreads();
  // One place in the row's list per block; its order does not matter.
  if (t == 0) base = count ? atomicAdd(&ws.listed[row], count) : 0;
  __syncthreads();
  for (int i = t; i < count && base + i < kCand; i += kThreads) ws.cand[(int64_t)row * kCand + base + i] = list[i];
}

// Kept entries: order (logit, then lower index) at or before the cut, or in a
// bin before `lo` (0 where the order alone says it).
struct Cut {
  uint32_t order;
  int index;
  int lo;
};
__device__ __forceinline__ bool kept(float v, int i, const Binning& b, const Cut& c) {
  if (!live(v, b.mx)) return false;
  const uint32_t o = order_of(v);
  return o > c.order || (o == c.order && i <= c.index) || (c.lo && bin_of(v, b) < c.lo);
}

// The number of entries ordered above `o` and their weight.
__device__ void above(const float* l, int n, float mx, double inv_t2, uint32_t o, uint64_t* part, uint64_t& cnt,
                      uint64_t& mass) {
  uint64_t c = 0, w = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float v = l[i];
    if (live(v, mx) && order_of(v) > o) {
      ++c;
      w += weight(v, mx, inv_t2);
    }
  }
  cnt = block_sum(c, part);
  mass = block_sum(w, part);
}

// The cut by bisection over the 32-bit order, for rows with many equal or
// nearly equal logits at the border: the lowest order whose first entry is
// kept, then how many of its entries (equal logits, by index) are.
__device__ Cut bisect(const SampleArgs& a, const float* l, float mx, const Settings& s, uint64_t total,
                      uint64_t* part) {
  const int n = a.n;
  auto search = [&](bool with_p, double limit) {
    uint32_t bad = 0, good = order_of(mx);   // the maximum's first entry is always kept
    while (good - bad > 1) {
      const uint32_t mid = bad + (good - bad) / 2;
      uint64_t cnt, mass;
      above(l, n, mx, s.inv_t2, mid, part, cnt, mass);
      bool ok = cnt < (uint64_t)s.k;
      if (with_p) {
        ok = ok && (double)mass < limit;
        if (s.use_min) ok = ok && exp(((double)logit_of(mid) - (double)mx) * s.inv_t) >= s.min_p;
      }
      (ok ? good : bad) = mid;
    }
    return good;
  };
  // Entries of order `o` counted from below: how many of them the first `most` are, by index.
  auto nth_index = [&](uint32_t o, uint64_t most) {
    uint64_t seen = 0;
    int index = -1;
    for (int base = 0; base < n && seen < most; base += kThreads) {
      const int i = base + threadIdx.x;
      const bool is = i < n && live(l[i], mx) && order_of(l[i]) == o;
      const uint64_t run = seen + block_scan(is, part);
      const int at = block_min(is && run == most ? i : 0x7FFFFFFF, reinterpret_cast<int*>(part));
      if (at != 0x7FFFFFFF) index = at;
      __syncthreads();
      if (threadIdx.x == kThreads - 1) part[0] = run;
      __syncthreads();
      seen = part[0];
      __syncthreads();
    }
    return index >= 0 ? index : 0x7FFFFFFF;
  };
  uint64_t cnt, mass;
  double limit = (double)total;
  if (s.use_p) {
    uint64_t top = total;
    if (s.k < n) {
      const uint32_t ok = search(false, 0);
      above(l, n, mx, s.inv_t2, ok, part, cnt, mass);
      uint64_t c1, m1;
      above(l, n, mx, s.inv_t2, ok - 1, part, c1, m1);   // with the entries of order ok
      const uint64_t same = c1 - cnt, take = min((uint64_t)s.k - cnt, same);
      top = same ? mass + take * ((m1 - mass) / same) : mass;
    }
    limit = s.p * (double)top;
  }
  const uint32_t o = search(true, s.use_p ? limit : 1.0e300);
  above(l, n, mx, s.inv_t2, o, part, cnt, mass);
  uint64_t c1, m1;
  above(l, n, mx, s.inv_t2, o - 1, part, c1, m1);
  const uint64_t same = c1 - cnt;
  uint64_t take = min(same, (uint64_t)s.k - cnt);
  if (same && s.use_p) {
    // j of them are kept while mass + j w < limit; at least one overall.
    const double w = (double)((m1 - mass) / same);
    const double room = limit - (double)mass;
    uint64_t j = w > 0 ? (uint64_t)fmin(fmax(ceil(room / w), 0.0), (double)same) : same;
    if (j == 0) j = 1;
    take = min(take, j);
  }
  // An order without entries (the search stops between two logits) keeps all above it.
  return Cut{o, same ? nth_index(o, take) : 0x7FFFFFFF, 0};
}

// One exchange of the sort below: the lane keeps the larger or the smaller of
// its and lane ^ J's key.
template <int K, int J>
__device__ __forceinline__ uint64_t sort_step(uint64_t v) {
  const int lane = threadIdx.x & 63;
  const uint64_t o = lane_xor<J>(v);
  const bool larger = ((lane & J) == 0) == ((lane & K) == 0);
  v = (v > o) == larger ? v : o;
  if constexpr (J > 1) return sort_step<K, J / 2>(v);
  return v;
}
// Sorts the wave's 64 keys in descending order (bitonic, across lanes).
__device__ __forceinline__ uint64_t wave_sort_desc(uint64_t v) {
  v = sort_step<2, 1>(v);
  v = sort_step<4, 2>(v);
  v = sort_step<8, 4>(v);
  v = sort_step<16, 8>(v);
  v = sort_step<32, 16>(v);
  return sort_step<64, 32>(v);
}

// Sorts key[0..nc) in descending order, nc <= kCand, keys distinct: each wave
// sorts runs of 64, then a key's place is its place in its run plus, for every
// other run, how many keys there are larger (binary searches, independent of
// each other).
__device__ void sort_desc(uint64_t* key, int nc) {
  const int t = threadIdx.x, lane = t & 63;
  const int runs = (nc + 63) >> 6;
  uint64_t mine[kCand / kThreads];
  int place[kCand / kThreads];
#pragma unroll
  for (int e = 0; e < kCand / kThreads; ++e) {
    const int i = e * kThreads + t;
    if ((i >> 6) < runs) {
      mine[e] = wave_sort_desc(i < nc ? key[i] : 0);   // empty places last
      key[i] = mine[e];                                // kCand is a whole number of runs
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kCand / kThreads; ++e) {
    const int i = e * kThreads + t;
    if ((i >> 6) >= runs) continue;
    int at = lane;
#pragma unroll 4
    for (int r = 0; r < runs; ++r) {
      const uint64_t* run = key + 64 * r;
      int p = 0;
#pragma unroll
      for (int step = 32; step > 0; step /= 2) p += run[p + step - 1] > mine[e] ? step : 0;
      p += run[p] > mine[e];
      at += r == (i >> 6) ? 0 : p;
    }
    place[e] = at;
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kCand / kThreads; ++e) {
    const int i = e * kThreads + t;
    if ((i >> 6) < runs && mine[e]) key[place[e]] = mine[e];
  }
  __syncthreads();
}

// Among the lanes' weights, in lane order, the first whose running sum from
// `run` on exceeds `want`, or the last with weight; and the sum before it.
struct Pick {
  int at;
  bool hit;
  uint64_t run;
};
__device__ __forceinline__ Pick pick(uint64_t q, uint64_t run, double want) {
  const uint64_t sum = run + wave_scan(q);
  const uint64_t hit = __ballot(q && (double)sum > want), any = __ballot(q != 0);
  Pick p;
  p.hit = hit != 0;
  p.at = hit ? __builtin_ctzll(hit) : (any ? 63 - __builtin_clzll(any) : 0);
  const uint64_t before = sum - q;
  p.run = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(before >> 32), p.at) << 32 |
          (uint32_t)__builtin_amdgcn_readlane((int)before, p.at);
  return p;
}

// The row's token and logprob, from its border, the listed entries (key, unsorted;
// more than kCand: not used) and the weight of each chunk's entries in the bins
// before the border (mass, in LDS; all of it where nothing is cut).  A barrier
// stands between the writes of key and mass and the call.  part: kWaves + 1.
__device__ void choose(const SampleArgs& a, int row, const Settings& s, const RowInfo& r, int listed, int chunks,
                       int per, uint64_t* key, unsigned long long* mass, uint64_t* part, int* ipart) {
  static_assert(kCand == 2 * kThreads, "two listed entries per thread");
  const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
  const float mx = r.mx;
  if (!(mx > -INFINITY)) {   // nothing to choose from
    if (t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  const Binning b{mx, r.c};
  const float* l = a.logits + (int64_t)row * a.ld;
  Cut cut{0u, 0x7FFFFFFF, 0};   // nothing cut: every live entry is ordered above 0
  if (listed <= kCand) {
    if (r.lo != kNone) {
      const int nc = listed;
      sort_desc(key, nc);
      // Thread t holds places 2t and 2t+1; their rank and the weight before
      // them, among the listed entries.
      uint64_t w[2] = {0, 0}, before[2];
      int bin[2] = {kNone, kNone};
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < nc) {
          const float v = logit_of((uint32_t)(key[2 * t + e] >> 32));
          w[e] = weight(v, mx, s.inv_t2);
          bin[e] = bin_of(v, b);
        }
      before[0] = block_scan(w[0] + w[1], part) - w[0] - w[1];
      before[1] = before[0] + w[0];
      // Entries of bins lo..hi come before those of a separate bin bk.
      uint64_t top = r.total;
      if (s.use_p && r.bk != kNone) {
        const int64_t inside =
            r.want_bk ? (int64_t)block_sum((uint64_t)(bin[0] <= r.hi) + (uint64_t)(bin[1] <= r.hi), part) : 0;
        const int64_t base = r.want_bk ? (int64_t)r.cnt_bk - inside : (int64_t)r.cnt_lo;
        uint64_t in_k = 0;   // weight of bin bk's entries among the top_k
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (bin[e] == r.bk && base + 2 * t + e < s.k) in_k += w[e];
        top = r.mass_bk + block_sum(in_k, part);
      }
      const double limit = s.p * (double)top;
      int last = -1;   // the last kept place
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < nc && bin[e] <= r.hi) {
          const int64_t rank = (int64_t)r.cnt_lo + 2 * t + e;
          const uint64_t k = key[2 * t + e];
          bool ok = rank < s.k;
          if (s.use_p) ok = ok && (rank == 0 || (double)(r.mass_lo + before[e]) < limit);
          if (s.use_min) {
            const float v = logit_of((uint32_t)(k >> 32));
            ok = ok && (v == mx || exp(((double)v - (double)mx) * s.inv_t) >= s.min_p);
          }
          if (ok) {
            atomicAdd(&mass[~(uint32_t)k / (uint32_t)per], (unsigned long long)w[e]);
            last = 2 * t + e;
          }
        }
      last = -block_min(-last, ipart);
      if (last >= 0) {
        cut.order = (uint32_t)(key[last] >> 32);
        cut.index = (int)~(uint32_t)key[last];
      } else {   // none of the listed: the bins before lo
        cut = Cut{0xFFFFFFFFu, -1, r.lo};
      }
    }
  } else {
    cut = bisect(a, l, mx, s, r.total, part);
    for (int c = 0; c < chunks; ++c) {
      uint64_t q = 0;
      Entries<4> in(l, chunk_range(c, per, a.n));
      in.each([&](float v, int i) { q += kept(v, i, b, cut) ? weight(v, mx, s.inv_t2) : 0; });
      q = block_sum(q, part);
      if (t == 0) mass[c] = q;
    }
  }
  __syncthreads();
  float u = a.u[row];
  if (!(u > 0.f)) u = 0.f;
  // The chunk, then the wave's part of it, then the entry whose running sum
  // exceeds u times the total; for u >= 1 the last one with weight.  Every wave
  // finds them for itself where the values fit its lanes.
  const uint64_t total = wave_sum(lane < chunks ? (uint64_t)mass[lane] : 0);
  const double want = (double)u * (double)total;
  const Pick pc = pick(lane < chunks ? (uint64_t)mass[lane] : 0, 0, want);
  const bool over = !pc.hit;
  const Range rc = chunk_range(pc.at, per, a.n);
  const int part_len = ((rc.end - rc.begin + kWaves - 1) / kWaves + 63) & ~63;
  {
    constexpr int kBatch = 10;   // loads ahead of their use
    uint64_t q = 0;
    const int i1 = min(rc.end, rc.begin + (wave + 1) * part_len);
    for (int i = rc.begin + wave * part_len + lane; i < i1; i += 64 * kBatch) {
      float v[kBatch];
#pragma unroll
      for (int e = 0; e < kBatch; ++e) v[e] = i + 64 * e < i1 ? l[i + 64 * e] : -INFINITY;
#pragma unroll
      for (int e = 0; e < kBatch; ++e)
        if (kept(v[e], i + 64 * e, b, cut)) q += weight(v[e], mx, s.inv_t2);
    }
    q = wave_sum(q);
    __syncthreads();
    if (lane == 0) part[wave] = q;
    __syncthreads();
  }
  const Pick pw = pick(lane < kWaves ? part[lane] : 0, pc.run, over ? INFINITY : want);
  const int i0 = rc.begin + pw.at * part_len, i1 = min(rc.end, i0 + part_len);
  int token = -1;
  constexpr int kEach = 4;   // neighbouring entries per thread
  // kBlock: over the block's threads, else by each wave over its lanes.
  auto draw = [&](auto block) {
    constexpr bool kBlock = decltype(block)::value;
    constexpr int kWide = kBlock ? kThreads : 64;
    const int id = kBlock ? t : lane;
    uint64_t run = pw.run;
    for (int base = i0; base < i1; base += kEach * kWide) {
      const int first = base + kEach * id;
      float v[kEach];
      uint64_t q[kEach], own = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e) v[e] = first + e < i1 ? l[first + e] : -INFINITY;
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        q[e] = kept(v[e], first + e, b, cut) ? weight(v[e], mx, s.inv_t2) : 0;
        own += q[e];
      }
      uint64_t sum = run + (kBlock ? block_scan(own, part) : wave_scan(own));
      if constexpr (kBlock) {
        if (t == kThreads - 1) part[kWaves] = sum;   // read behind the barriers below
      } else {
        run = last_lane(sum);
      }
      sum -= own;
      int hit = 0x7FFFFFFF, far = -1;   // the first whose running sum exceeds it, the last with weight
#pragma unroll
      for (int e = 0; e < kEach; ++e) {
        sum += q[e];
        if (q[e] && !over && hit == 0x7FFFFFFF && (double)sum > want) hit = first + e;
        if (q[e]) far = first + e;
      }
      hit = kBlock ? block_min(hit, ipart) : wave_min(hit);
      if (hit != 0x7FFFFFFF) {
        token = hit;
        break;
      }
      far = kBlock ? -block_min(-far, ipart) : -wave_min(-far);
      token = far >= 0 ? far : token;
      if constexpr (kBlock) run = part[kWaves];
    }
  };
  if (part_len <= 2 * kEach * 64) draw(std::false_type{});
  else draw(std::true_type{});
  if (t == 0) {
    a.tokens[row] = token;
    if (a.logprobs && token < 0) {   // only if the logits changed under the call
      a.logprobs[row] = -INFINITY;
    } else if (a.logprobs) {
      const float v = l[token];
      a.logprobs[row] =
          (float)((v == mx ? 0.0 : ((double)v - (double)mx) * s.inv_t) - log((double)total * 0x1p-44));
    }
  }
}

__global__ __launch_bounds__(kThreads) void sample_choose_kernel(SampleArgs a, Ws ws, int chunks, int per) {
  __shared__ uint64_t part[kWaves + 1];
  __shared__ int ipart[kWaves];
  __shared__ unsigned long long mass[kMaxChunks];
  __shared__ uint64_t key[kCand];
  const int row = blockIdx.x, t = threadIdx.x;
  const RowInfo r = ws.info[row];
  const int listed = r.lo == kNone ? 0 : ws.listed[row];
  if (t < chunks) mass[t] = r.lo ? ws.hist_mass[((int64_t)row * chunks + t) * kBins + r.lo - 1] : 0;
  for (int i = t; i < listed && i < kCand; i += kThreads) key[i] = ws.cand[(int64_t)row * kCand + i];
  __syncthreads();
  choose(a, row, settings(a, row), r, listed, chunks, per, key, mass, part, ipart);
}

// All five steps in one block and one launch, the sums and the list in LDS and
// the row read again from the L2.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
  __shared__ uint64_t mass[kBins];
  __shared__ uint32_t cnt[kBins];
  __shared__ uint64_t key[kCand];
  __shared__ uint64_t part[kWaves + 1];
  __shared__ float2 fpart[kWaves];
  __shared__ int ipart[kWaves];
  __shared__ unsigned long long whole;
  __shared__ int count;
  const int row = blockIdx.x, t = threadIdx.x;
  const float* l = a.logits + (int64_t)row * a.ld;
  const Range all{0, a.n};
  const Settings s = settings(a, row);
  const bool counts = s.k < a.n;
  cnt[t] = 0;
  mass[t] = 0;
  if (t == 0) count = 0;
  const float2 st = range_stats(l, all, fpart);   // its barrier covers the clearing
  const Binning b = binning(st.x, st.y, s.t);
  {
    Entries<4> in(l, all);
    range_hist(in, s, b, counts, cnt, reinterpret_cast<unsigned long long*>(mass));
  }
  __syncthreads();
  const uint64_t mi = block_scan(mass[t], part);
  const uint32_t ci = counts ? (uint32_t)block_scan(cnt[t], part) : 0;
  mass[t] = mi;
  cnt[t] = ci;
  __syncthreads();
  const RowInfo r = find_border(s, b, counts, mi, ci, mass, cnt, ipart);
  if (r.lo != kNone) {
    Entries<8> in(l, all);
    range_list(in, r, key, count);
  }
  if (t == 0) whole = r.mass_lo;   // all of the row's where nothing is cut
  __syncthreads();
  choose(a, row, s, r, count, 1, a.n, key, &whole, part, ipart);
}

// Chunks for about 512 blocks over all rows (two per CU; 1024: 64x151936 69 ->
// 73 us), at most 16 per row: the border launch adds them up.
struct Plan {
  int per, chunks;
};
// One block and launch for a row that is short, or not too long where there is a
// row for every CU.  Measured, one launch against five (us): 1 x 4000 16 and 24, 1 x
// 16000 25 and 27, 1 x 32000 37 and 27; 64 x 8000 23 and 38, 64 x 50257 62 and 42;
// 256 x 16000 31 and 41, 256 x 50257 68 and 74, 256 x 151936 184 and 166.
constexpr int64_t kShortRow = 20480, kBlockRow = 65536, kManyRows = 256;
Plan plan(int64_t m, int64_t n) {
  if (n <= kShortRow || (n <= kBlockRow && m >= kManyRows)) return {(int)n, 1};
  const int64_t tiles = (n + kThreads - 1) / kThreads;
  int64_t want = (512 + m - 1) / m;
  want = want < kMaxChunks ? want : kMaxChunks;
  Plan p;
  p.per = (int)((tiles + want - 1) / want) * kThreads;
  p.chunks = (int)((n + p.per - 1) / p.per);
  return p;
}
int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

int64_t sample_workspace_bytes(int64_t m, int64_t n) {
  const Plan p = plan(m, n);
  if (p.chunks == 1) return 256;   // nothing is kept between launches
  return align256(m * p.chunks * (int64_t)sizeof(float2)) + align256(m * (int64_t)sizeof(RowInfo)) + align256(m * 4) +
         align256(m * p.chunks * kBins * 4) + align256(m * p.chunks * kBins * 8) + align256(m * kCand * 8);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t s) {
  const Plan p = plan(a.m, a.n);
  if (p.chunks == 1) {
    hipLaunchKernelGGL(sample_row_kernel, dim3((unsigned)a.m), dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  uint8_t* at = static_cast<uint8_t*>(workspace);
  auto take = [&](int64_t bytes) {
    uint8_t* r = at;
    at += align256(bytes);
    return r;
  };
  const int64_t m = a.m;
  Ws ws;
  ws.stats = reinterpret_cast<float2*>(take(m * p.chunks * (int64_t)sizeof(float2)));
  ws.info = reinterpret_cast<RowInfo*>(take(m * (int64_t)sizeof(RowInfo)));
  ws.listed = reinterpret_cast<int*>(take(m * 4));
  ws.hist_cnt = reinterpret_cast<uint32_t*>(take(m * p.chunks * kBins * 4));
  ws.hist_mass = reinterpret_cast<uint64_t*>(take(m * p.chunks * kBins * 8));
  ws.cand = reinterpret_cast<uint64_t*>(take(m * kCand * 8));
  const dim3 grid((unsigned)p.chunks, (unsigned)a.m), rows((unsigned)a.m), block(kThreads);
  hipLaunchKernelGGL(sample_stats_kernel, grid, block, 0, s, a, ws, p.per);
  hipLaunchKernelGGL(sample_hist_kernel, grid, block, 0, s, a, ws, p.per);
  hipLaunchKernelGGL(sample_border_kernel, rows, block, 0, s, a, ws, p.chunks);
  hipLaunchKernelGGL(sample_collect_kernel, grid, block, 0, s, a, ws, p.per);
  hipLaunchKernelGGL(sample_choose_kernel, rows, block, 0, s, a, ws, p.chunks, p.per);
  return hipGetLastError();
}

}  // namespace q3
