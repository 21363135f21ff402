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
// A row is cut into tiles of 1024 entries and chunks of whole tiles; five
// launches:
//   stats    per chunk: largest and smallest logit
//   hist     per chunk: entry counts and weights over 1024 bins of max l - l
//            (equal steps over the row's span, at most 32 T; the last bin
//            takes the rest).  The bin is a monotone function of the logit.
//   border   per row: the bins in which top-k, top-p and min-p can fall, from
//            the row's bin sums
//   collect  per chunk: the weight of each tile's entries in bins before those,
//            and the list of entries inside them (a few hundred)
//   choose   per row: the listed entries are ranked against each other, which
//            gives the exact cut; the tile sums are completed and searched for
//            u times their total, and the token is found inside its tile
// A row whose border bins hold more than kCand entries (large ties) is cut by
// bisection over the logits' 32-bit order instead, in the last launch.
//
// What bounds it: the row is read from memory once and twice more from cache,
// and two of the three passes evaluate an exponential per entry in 64 bits.
#include "q3_device.h"
#include "q3_internal.h"

namespace q3 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kTile = 1024;        // entries per tile (one per thread)
constexpr int kMaxTiles = 512;     // n <= 2^19
constexpr int kBins = 1024;        // one per thread
constexpr int kCand = 2048;        // listed entries per row
constexpr int kNone = kBins;       // "no border": after every bin
constexpr double kOne = 17592186044416.0;   // 2^44, the weight of the largest entry

struct RowInfo {
  uint64_t mass_lo;    // weight of the bins before lo
  uint64_t mass_bk;    // weight of the bins before bk
  uint64_t total;      // weight of the row
  int lo, hi;          // the cut is in bins lo..hi (kNone: nothing is cut)
  int bk;              // the bin of rank top_k (kNone: no such bin)
  int cnt_lo, cnt_bk;  // entries in the bins before lo and before bk
  int want_bk;         // bk's entries are listed too, for the weight of the top_k entries
  int slow;            // the lists do not fit: bisection
  int listed;          // entries listed so far
};

struct Ws {
  float2* stats;         // [m][chunks] (max, min)
  RowInfo* info;         // [m]
  uint32_t* hist_cnt;    // [m][chunks][kBins]
  uint64_t* hist_mass;   // [m][chunks][kBins]
  uint64_t* tile_mass;   // [m][tiles]
  uint64_t* cand;        // [m][kCand] (order << 32 | index)
};

// A row's settings as they act: t > 0, k >= 1 (n when off), top-p and min-p
// with their off values.
struct Settings {
  double inv_t;
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

// 2^44 exp((l - mx)/t), rounded to an integer.
__device__ __forceinline__ uint64_t weight(float l, float mx, double inv_t) {
  const double x = l == mx ? 0.0 : ((double)l - (double)mx) * inv_t;
  // Adding 2^52 leaves the rounded integer in the low bits.
  const double w = exp(x) * kOne + 4503599627370496.0;
  return __builtin_bit_cast(uint64_t, w) & 0x000FFFFFFFFFFFFFull;
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

// ---- block-wide helpers (kThreads threads) ----------------------------------

template <typename T>
__device__ __forceinline__ T wave_up(T v, int off) {
  return __shfl_up(v, off, 64);
}
__device__ __forceinline__ uint64_t wave_up64(uint64_t v, int off) {
  return (uint64_t)__shfl_up((unsigned long long)v, off, 64);
}

// Inclusive prefix sum over the block; `part` holds kWaves values.  Leading
// barrier included, so `part` may be reused at once.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* part) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const uint64_t o = wave_up64(v, off);
    if (lane >= off) v += o;
  }
  __syncthreads();
  if (lane == 63) part[wave] = v;
  __syncthreads();
  uint64_t before = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) before += w < wave ? part[w] : 0;
  return v + before;
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, uint64_t* part) {
#pragma unroll
  for (int off = 32; off > 0; off /= 2) v += (uint64_t)__shfl_xor((unsigned long long)v, off, 64);
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
#pragma unroll
  for (int off = 32; off > 0; off /= 2) {
    const int o = __shfl_xor(v, off, 64);
    v = o < v ? o : v;
  }
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
#pragma unroll
  for (int off = 32; off > 0; off /= 2) {
    r.x = fmaxf(r.x, __shfl_xor(r.x, off, 64));
    r.y = fminf(r.y, __shfl_xor(r.y, off, 64));
  }
  return r;
}

// ---- launches -----------------------------------------------------------------

__global__ __launch_bounds__(kThreads) void sample_stats_kernel(SampleArgs a, Ws ws, int tiles_per_chunk) {
  __shared__ float2 part[kWaves];
  const int row = blockIdx.y, c = blockIdx.x;
  const float* l = a.logits + (int64_t)row * a.ld;
  const int i0 = c * tiles_per_chunk * kTile;
  const int i1 = min(a.n, i0 + tiles_per_chunk * kTile);
  float mx = -INFINITY, mn = INFINITY;
#pragma unroll 4
  for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const float v = l[i];
    mx = fmaxf(mx, v);   // NaN leaves the other operand
    mn = v > -INFINITY ? fminf(mn, v) : mn;
  }
#pragma unroll
  for (int off = 32; off > 0; off /= 2) {
    mx = fmaxf(mx, __shfl_xor(mx, off, 64));
    mn = fminf(mn, __shfl_xor(mn, off, 64));
  }
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(mx, mn);
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) {
      mx = fmaxf(mx, part[w].x);
      mn = fminf(mn, part[w].y);
    }
    ws.stats[(int64_t)row * gridDim.x + c] = make_float2(mx, mn);
  }
}

__global__ __launch_bounds__(kThreads) void sample_hist_kernel(SampleArgs a, Ws ws, int tiles_per_chunk) {
  __shared__ uint32_t cnt[kBins];
  __shared__ unsigned long long mass[kBins];
  const int row = blockIdx.y, c = blockIdx.x, chunks = gridDim.x;
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const Settings s = settings(a, row);
  const Binning b = binning(st.x, st.y, s.t);
  cnt[threadIdx.x] = 0;
  mass[threadIdx.x] = 0;
  __syncthreads();
  const float* l = a.logits + (int64_t)row * a.ld;
  const int i0 = c * tiles_per_chunk * kTile;
  const int i1 = min(a.n, i0 + tiles_per_chunk * kTile);
#pragma unroll 4
  for (int i = i0 + threadIdx.x; i < i1; i += kThreads) {
    const float v = l[i];
    if (!live(v, st.x)) continue;
    const int k = bin_of(v, b);
    atomicAdd(&cnt[k], 1u);
    atomicAdd(&mass[k], (unsigned long long)weight(v, st.x, s.inv_t));
  }
  __syncthreads();
  const int64_t at = ((int64_t)row * chunks + c) * kBins + threadIdx.x;
  ws.hist_cnt[at] = cnt[threadIdx.x];
  ws.hist_mass[at] = mass[threadIdx.x];
}

__global__ __launch_bounds__(kThreads) void sample_border_kernel(SampleArgs a, Ws ws, int chunks) {
  __shared__ uint64_t part[kWaves];
  __shared__ int ipart[kWaves];
  __shared__ uint64_t mass_in[kBins];   // inclusive sums
  __shared__ uint32_t cnt_in[kBins];
  const int row = blockIdx.x, t = threadIdx.x;
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const Settings s = settings(a, row);
  const Binning b = binning(st.x, st.y, s.t);
  uint64_t mass = 0, cnt = 0;
  for (int c = 0; c < chunks; ++c) {
    const int64_t at = ((int64_t)row * chunks + c) * kBins + t;
    cnt += ws.hist_cnt[at];
    mass += ws.hist_mass[at];
  }
  const uint64_t mi = block_scan(mass, part), ci = block_scan(cnt, part);
  mass_in[t] = mi;
  cnt_in[t] = (uint32_t)ci;
  __syncthreads();
  const uint64_t total = mass_in[kBins - 1], entries = cnt_in[kBins - 1];
  auto first = [&](bool hit) { return block_min(hit ? t : kNone, ipart); };
  // The bin of the last of the top_k entries.
  const int bk = (uint64_t)s.k < entries ? first(ci >= (uint64_t)s.k) : kNone;
  // The weight of the top_k entries lies between the sums before and after
  // that bin, and top-p's border between the bins where p times those fall.
  int lo = bk, hi = bk;
  if (s.use_p) {
    const uint64_t s_lo = bk == kNone ? total : (bk ? mass_in[bk - 1] : 0);
    const uint64_t s_hi = bk == kNone ? total : mass_in[bk];
    const int p_lo = first((double)mi >= s.p * (double)s_lo), p_hi = first((double)mi >= s.p * (double)s_hi);
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
    lo = min(lo, e_lo);
    hi = min(hi, e_hi);
  }
  const int want_bk = s.use_p && bk != kNone && !(lo <= bk && bk <= hi);
  if (t == 0) {
    RowInfo r;
    auto mass_before = [&](int k) -> uint64_t { return k > 0 ? mass_in[k - 1] : 0; };
    auto cnt_before = [&](int k) -> uint32_t { return k > 0 ? cnt_in[k - 1] : 0; };
    r.total = total;
    r.lo = lo;
    r.hi = hi;
    r.bk = bk;
    r.want_bk = want_bk;
    r.mass_lo = mass_before(lo);
    r.cnt_lo = (int)cnt_before(lo);
    r.mass_bk = mass_before(bk);
    r.cnt_bk = (int)cnt_before(bk);
    uint32_t listed = lo == kNone ? 0 : cnt_in[min(hi, kBins - 1)] - cnt_before(lo);
    if (want_bk) listed += cnt_in[bk] - cnt_before(bk);
    r.slow = listed > (uint32_t)kCand;
    r.listed = 0;
    ws.info[row] = r;
  }
}

__global__ __launch_bounds__(kThreads) void sample_collect_kernel(SampleArgs a, Ws ws, int tiles_per_chunk, int tiles) {
  __shared__ uint64_t part[kWaves];
  __shared__ RowInfo r;
  const int row = blockIdx.y, c = blockIdx.x, chunks = gridDim.x, t = threadIdx.x;
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const Settings s = settings(a, row);
  const Binning b = binning(st.x, st.y, s.t);
  if (t == 0) r = ws.info[row];
  __syncthreads();
  if (r.slow) return;   // the whole block: r is shared
  const float* l = a.logits + (int64_t)row * a.ld;
  const int t0 = c * tiles_per_chunk, t1 = min(tiles, t0 + tiles_per_chunk);
  for (int tile = t0; tile < t1; ++tile) {
    const int i = tile * kTile + t;
    const float v = i < a.n ? l[i] : -INFINITY;
    uint64_t q = 0;
    if (live(v, st.x)) {
      const int k = bin_of(v, b);
      if (k < r.lo) {
        q = weight(v, st.x, s.inv_t);
      } else if (k <= r.hi || (r.want_bk && k == r.bk)) {
        const int at = atomicAdd(&ws.info[row].listed, 1);
        if (at < kCand) ws.cand[(int64_t)row * kCand + at] = (uint64_t)order_of(v) << 32 | (uint32_t)i;
      }
    }
    const uint64_t sum = block_sum(q, part);
    if (t == 0) ws.tile_mass[(int64_t)row * tiles + tile] = sum;
  }
}

// Kept entries: order (logit, then lower index) at or before the cut, or in a
// bin before `lo`.
struct Cut {
  uint32_t order;
  int index;
  int lo;
};
__device__ __forceinline__ bool kept(float v, int i, float mx, const Binning& b, const Cut& c) {
  if (!live(v, mx)) return false;
  if (bin_of(v, b) < c.lo) return true;
  const uint32_t o = order_of(v);
  return o > c.order || (o == c.order && i <= c.index);
}

// The number of entries ordered above `o` and their weight.
__device__ void above(const float* l, int n, float mx, double inv_t, uint32_t o, uint64_t* part, uint64_t& cnt,
                      uint64_t& mass) {
  uint64_t c = 0, w = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const float v = l[i];
    if (live(v, mx) && order_of(v) > o) {
      ++c;
      w += weight(v, mx, inv_t);
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
      above(l, n, mx, s.inv_t, mid, part, cnt, mass);
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
      above(l, n, mx, s.inv_t, ok, part, cnt, mass);
      uint64_t c1, m1;
      above(l, n, mx, s.inv_t, ok - 1, part, c1, m1);   // with the entries of order ok
      const uint64_t same = c1 - cnt, take = min((uint64_t)s.k - cnt, same);
      top = same ? mass + take * ((m1 - mass) / same) : mass;
    }
    limit = s.p * (double)top;
  }
  const uint32_t o = search(true, s.use_p ? limit : 1.0e300);
  above(l, n, mx, s.inv_t, o, part, cnt, mass);
  uint64_t c1, m1;
  above(l, n, mx, s.inv_t, o - 1, part, c1, m1);
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

__global__ __launch_bounds__(kThreads) void sample_choose_kernel(SampleArgs a, Ws ws, int chunks, int tiles) {
  __shared__ uint64_t part[kWaves];
  __shared__ int ipart[kWaves];
  __shared__ unsigned long long mass[kMaxTiles];
  __shared__ uint64_t key[kCand], wgt[kCand];
  __shared__ unsigned long long cut_key;
  const int row = blockIdx.x, t = threadIdx.x;
  const float2 st = row_stats(ws.stats + (int64_t)row * chunks, chunks);
  const float mx = st.x;
  if (!(mx > -INFINITY)) {   // nothing to choose from
    if (t == 0) {
      a.tokens[row] = -1;
      if (a.logprobs) a.logprobs[row] = -INFINITY;
    }
    return;
  }
  const Settings s = settings(a, row);
  const Binning b = binning(mx, st.y, s.t);
  const RowInfo r = ws.info[row];
  const float* l = a.logits + (int64_t)row * a.ld;
  Cut cut{0u, 0x7FFFFFFF, 0};
  if (!r.slow) {
    cut.lo = r.lo;
    for (int i = t; i < tiles; i += kThreads) mass[i] = ws.tile_mass[(int64_t)row * tiles + i];
    const int nc = min(r.listed, kCand);
    // Sort key: larger logit first, then lower index; ~index makes "greater is
    // ranked earlier" one comparison.
    for (int i = t; i < nc; i += kThreads) {
      const uint64_t e = ws.cand[(int64_t)row * kCand + i];
      key[i] = e ^ 0xFFFFFFFFull;
      wgt[i] = weight(logit_of((uint32_t)(e >> 32)), mx, s.inv_t);
    }
    if (t == 0) cut_key = ~0ull;
    __syncthreads();
    // Rank and preceding weight of each listed entry, among the listed ones.
    int my_rank[kCand / kThreads];
    uint64_t my_mass[kCand / kThreads];
    uint64_t bk_mass = 0;   // listed entries of bin bk that are among the top_k
#pragma unroll
    for (int e = 0; e < kCand / kThreads; ++e) {
      const int i = e * kThreads + t;
      my_rank[e] = 0;
      my_mass[e] = 0;
      if (i < nc) {
        const uint64_t k = key[i];
        int rank = 0;
        uint64_t before = 0;
        for (int j = 0; j < nc; ++j) {
          const bool g = key[j] > k;
          rank += g;
          before += g ? wgt[j] : 0;
        }
        my_rank[e] = rank;
        my_mass[e] = before;
      }
    }
    auto bin_at = [&](int i) { return bin_of(logit_of((uint32_t)(key[i] >> 32)), b); };
    // Entries listed in bins lo..hi come before those of bin bk.
    uint64_t inside = 0;
    if (r.want_bk) {
      uint64_t c = 0;
#pragma unroll
      for (int e = 0; e < kCand / kThreads; ++e) {
        const int i = e * kThreads + t;
        if (i < nc && bin_at(i) <= r.hi) ++c;
      }
      inside = block_sum(c, part);
    }
    uint64_t top = r.total;
    if (s.use_p && r.bk != kNone) {
#pragma unroll
      for (int e = 0; e < kCand / kThreads; ++e) {
        const int i = e * kThreads + t;
        if (i < nc && bin_at(i) == r.bk) {
          const int64_t rank = r.want_bk ? (int64_t)r.cnt_bk + my_rank[e] - (int64_t)inside
                                         : (int64_t)r.cnt_lo + my_rank[e];
          if (rank < s.k) bk_mass += wgt[i];
        }
      }
      top = r.mass_bk + block_sum(bk_mass, part);
    }
    const double limit = s.p * (double)top;
#pragma unroll
    for (int e = 0; e < kCand / kThreads; ++e) {
      const int i = e * kThreads + t;
      if (i < nc && bin_at(i) <= r.hi) {
        const int64_t rank = (int64_t)r.cnt_lo + my_rank[e];
        bool ok = rank < s.k;
        if (s.use_p) ok = ok && (rank == 0 || (double)(r.mass_lo + my_mass[e]) < limit);
        if (s.use_min) {
          const float v = logit_of((uint32_t)(key[i] >> 32));
          ok = ok && (v == mx || exp(((double)v - (double)mx) * s.inv_t) >= s.min_p);
        }
        if (ok) {
          const uint32_t index = ~(uint32_t)key[i];
          atomicAdd(&mass[index / kTile], (unsigned long long)wgt[i]);
          atomicMin(&cut_key, (unsigned long long)key[i]);
        }
      }
    }
    __syncthreads();
    if (r.lo != kNone) {
      cut.order = (uint32_t)(cut_key >> 32);   // none kept: above every logit
      cut.index = cut_key == ~0ull ? -1 : (int)~(uint32_t)cut_key;
    }
  } else {
    cut = bisect(a, l, mx, s, r.total, part);
    for (int tile = 0; tile < tiles; ++tile) {
      const int i = tile * kTile + t;
      const float v = i < a.n ? l[i] : -INFINITY;
      const uint64_t sum = block_sum(kept(v, i, mx, b, cut) ? weight(v, mx, s.inv_t) : 0, part);
      if (t == 0) mass[tile] = sum;
    }
    __syncthreads();
  }
  // The tile, then the entry, whose running sum exceeds u times the total.
  const uint64_t mine = t < tiles ? mass[t] : 0;
  const uint64_t run = block_scan(mine, part);
  const uint64_t total = block_sum(mine, part);
  float u = a.u[row];
  if (!(u > 0.f)) u = 0.f;
  const double want = (double)u * (double)total;
  int tile = block_min(mine && (double)run > want ? t : 0x7FFFFFFF, ipart);
  const bool over = tile == 0x7FFFFFFF;   // u >= 1: the last entry with weight
  if (over) tile = -block_min(mine ? -t : 0, ipart);
  __syncthreads();
  if (t == tile) part[0] = run - mine;
  __syncthreads();
  const uint64_t before = part[0];
  const int i = tile * kTile + t;
  const float v = i < a.n ? l[i] : -INFINITY;
  const uint64_t q = kept(v, i, mx, b, cut) ? weight(v, mx, s.inv_t) : 0;
  const uint64_t sum = before + block_scan(q, part);
  int pick = block_min(!over && q && (double)sum > want ? t : 0x7FFFFFFF, ipart);
  if (pick == 0x7FFFFFFF) pick = -block_min(q ? -t : 0, ipart);
  if (t == pick) {
    a.tokens[row] = i;
    if (a.logprobs)
      a.logprobs[row] =
          (float)((v == mx ? 0.0 : ((double)v - (double)mx) * s.inv_t) - log((double)total * (1.0 / kOne)));
  }
}

struct Plan {
  int tiles, tiles_per_chunk, chunks;
};
// Chunks for about 512 blocks over all rows (two per CU).
Plan plan(int64_t m, int64_t n) {
  Plan p;
  p.tiles = (int)((n + kTile - 1) / kTile);
  const int64_t want = (512 + m - 1) / m;
  p.tiles_per_chunk = (int)((p.tiles + want - 1) / want);
  p.chunks = (p.tiles + p.tiles_per_chunk - 1) / p.tiles_per_chunk;
  return p;
}
int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

int64_t sample_workspace_bytes(int64_t m, int64_t n) {
  const Plan p = plan(m, n);
  return align256(m * p.chunks * (int64_t)sizeof(float2)) + align256(m * (int64_t)sizeof(RowInfo)) +
         align256(m * p.chunks * kBins * 4) + align256(m * p.chunks * kBins * 8) + align256(m * p.tiles * 8) +
         align256(m * kCand * 8);
}

hipError_t launch_sample(const SampleArgs& a, void* workspace, hipStream_t s) {
  const Plan p = plan(a.m, a.n);
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
  ws.hist_cnt = reinterpret_cast<uint32_t*>(take(m * p.chunks * kBins * 4));
  ws.hist_mass = reinterpret_cast<uint64_t*>(take(m * p.chunks * kBins * 8));
  ws.tile_mass = reinterpret_cast<uint64_t*>(take(m * p.tiles * 8));
  ws.cand = reinterpret_cast<uint64_t*>(take(m * kCand * 8));
  const dim3 grid((unsigned)p.chunks, (unsigned)a.m), rows((unsigned)a.m), block(kThreads);
  hipLaunchKernelGGL(sample_stats_kernel, grid, block, 0, s, a, ws, p.tiles_per_chunk);
  hipLaunchKernelGGL(sample_hist_kernel, grid, block, 0, s, a, ws, p.tiles_per_chunk);
  hipLaunchKernelGGL(sample_border_kernel, rows, block, 0, s, a, ws, p.chunks);
  hipLaunchKernelGGL(sample_collect_kernel, grid, block, 0, s, a, ws, p.tiles_per_chunk, p.tiles);
  hipLaunchKernelGGL(sample_choose_kernel, rows, block, 0, s, a, ws, p.chunks, p.tiles);
  return hipGetLastError();
}

}  // namespace q3
