// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits, and their gradient.
//
// With c = 1 / temperature, M = max l, e_j = exp(c (l_j - M)):
//   S = sum e,  T = sum e c (l - M)
//   ln p_j = c (l_j - M) - ln S,  H = ln S - T / S
//   dl_j = c (g ([j == t] - p_j) - h p_j (ln p_j + H))
//
// Bound by memory: the forward reads each logit once.  A block holds 8192 of a
// row's logits in registers at a time and keeps the running M, S and T of every
// thread (rescaled where M grows; T in powers of two).  Differences to M are formed
// before they are scaled, so large logits lose nothing.  Rows are split over blocks
// where there are few; a second launch joins the parts in order.
//
// Top alternatives: each wave keeps the best `top` entries it has seen, sorted, in
// LDS.  An entry is one 64-bit key, the logit's order in the high word and the
// inverted index in the low one, so that a plain comparison ranks and no two are
// equal.  Most of 1024 new logits are below the list's last and cost the comparison
// with their lanes' maxima alone, which are there for the sums.  Where the list is
// not full yet, the top-th largest of the 64 lanes' maxima is a bound that at least
// that many entries reach (found bit by bit, 18 of 32 bits: a lower bound is one
// too).  What passes is packed behind one another and ranked by counting.
//
// Measured: 2048 rows of 151936 214 us (5.8 TB/s), 2047 of 50257 74 us.  64 rows of
// 151936 take 13 us without top alternatives, 20 with the best one and 26 with 20: 21
// in the parts and 6 in the join, a chain of lists rather than memory; one row of 32000
// 6.5, 11.5 and 13.  One list for a block, with a barrier for each chunk, took 29 for the
// 26 and 13.7 for the 13; packed bounds over the waves' lists instead of merges 26.6
// and 13.1.
#include "q3_device.h"
#include "../../include/q3_block.h"
#include "q3_internal.h"

namespace q3 {
namespace {

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kEach = 16;                     // logits of a thread
constexpr int kChunk = kThreads * kEach;      // of a block
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef unsigned long long Key;

// A logit's order as a number above 0 (for what is not NaN).
__device__ __forceinline__ uint32_t order_of(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.f);   // -0 as 0
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t order) {
  return __builtin_bit_cast(float, order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}
__device__ __forceinline__ Key key_of(float l, uint32_t index) { return (Key)order_of(l) << 32 | (uint32_t)~index; }
__device__ __forceinline__ Key max_key(Key a, Key b) { return a > b ? a : b; }
__device__ __forceinline__ Key min_key(Key a, Key b) { return a < b ? a : b; }
__device__ __forceinline__ void wave_sync() {   // the wave's own LDS, written before, read behind
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Two descending lists of 32, `k` in lanes 0..31 (and again in 32..63) of each: the
// best 32 of both, descending.
__device__ __forceinline__ Key merge_best(Key mine, Key other, int lane) {
  const Key back = __shfl(other, 31 - (lane & 31), 64);
  Key k = max_key(mine, back);   // the larger halves of a bitonic sequence
#pragma unroll
  for (int step = 16; step > 0; step /= 2) {
    const Key o = __shfl_xor(k, step, 64);
    k = (lane & step) == 0 ? max_key(k, o) : min_key(k, o);
  }
  return k;
}

struct Sums {
  float m, s, t;   // largest logit (raw), sum of weights, sum of weights * log2 of them
};
__device__ __forceinline__ Sums empty_sums() { return {-INFINITY, 0.f, 0.f}; }
// Sums under a larger maximum; c2 = log2(e) / temperature.
__device__ __forceinline__ void rise(Sums& a, float m, float c2) {
  if (!(m > a.m)) return;
  if (a.m > -INFINITY) {
    const float d = (a.m - m) * c2, f = __builtin_amdgcn_exp2f(d);
    a.t = f > 0.f ? f * (a.t + d * a.s) : 0.f;
    a.s *= f;
  }
  a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c2) {
  const float m = fmaxf(a.m, b.m);
  rise(a, m, c2);
  rise(b, m, c2);
  return {m, a.s + b.s, a.t + b.t};
}
__device__ __forceinline__ Sums join_wave(Sums a, float c2) {
#pragma unroll
  for (int off = 1; off < 64; off *= 2) {
    const Sums o = {__shfl_xor(a.m, off, 64), __shfl_xor(a.s, off, 64), __shfl_xor(a.t, off, 64)};
    a = join(a, o, c2);
  }
  return a;
}

// What a block found of its part of a row.
struct Part {
  float m, s, t, unused;
};

// Logits j..j+3 of a row of n; those past its end are 0.  `whole`: none is.
constexpr int kStreamed = 2;   // a load's mark: not to be kept in caches
template <int kMark = 0>
__device__ __forceinline__ f32x4 load4(rsrc_t row, const float* p, int j, int n, bool whole) {
  if (whole || j + 4 <= n)
    return __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(row, 4u * (uint32_t)j, 0, kMark));
  f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (j + i < n) v[i] = p[j + i];
  return v;
}

// The answers of a row from all its logits' sums.
__device__ __forceinline__ void finish(const LogprobArgs& a, int64_t row, Sums r, float target) {
  const bool some = r.m > -INFINITY;
  const float ln = some ? logf(r.s) : 0.f;
  const float h = some ? ln - r.t / r.s * kLn2 : 0.f;
  const int t = a.targets[row];
  float lp = 0.f;
  if (t >= 0 && t < a.n) {
    const float d = target == r.m ? 0.f : (target - r.m) * a.inv_t;   // +inf
    lp = some && target > -INFINITY ? d - ln : -INFINITY;
  }
  a.logprobs[row] = lp;
  if (a.entropy) a.entropy[row] = h;
  if (a.stats) reinterpret_cast<f32x4*>(a.stats)[row] = f32x4{r.m, ln, h, 0.f};
}
// Lane j < top writes place j.
__device__ __forceinline__ void finish_top(const LogprobArgs& a, int64_t row, Sums r, Key k, int lane) {
  if (lane >= a.top) return;
  const float l = logit_of((uint32_t)(k >> 32)), ln = logf(r.s);
  const float d = l == r.m ? 0.f : (l - r.m) * a.inv_t;
  a.top_ids[row * a.top + lane] = k ? (int32_t)~(uint32_t)k : -1;
  a.top_logprobs[row * a.top + lane] = k ? d - ln : -INFINITY;
}

// The waves' lists, `count` of them in LDS, into the first: a tree of merges.  Every
// thread of the block comes here.
__device__ __forceinline__ void merge_lists(Key (*list)[32], int count, int wave, int lane) {
  for (int half = count / 2; half > 0; half /= 2) {
    __syncthreads();
    if (wave < half) {
      const Key k = merge_best(list[wave][lane & 31], list[wave + half][lane & 31], lane);
      wave_sync();
      if (lane < 32) list[wave][lane] = k;
    }
  }
  __syncthreads();
}

// A chunk's logits into the wave's list: l[i] stands at first + i % 4 + (i / 4) * 4 *
// kThreads, m is the lane's largest.  `last` is the value in the list's last place
// (-inf: it is not full), `size` its entries, `shared` the order of the best of the
// block's last places.
struct Best {
  Key* list;     // the wave's 32
  Key* packed;   // and its 64 for new ones
  uint32_t* shared;
  int top, size;
  float last;

  __device__ __forceinline__ void add(const float (&l)[kEach], float m, int first, int lane) {
    // Of what stands in other waves' lists, an equal one may rank behind this one.
    const float others = logit_of(*shared);   // NaN (order 0): none is full
    const float floor_ = others > last ? others : last;
    if (__ballot(m > last && m >= floor_) == 0) return;
    float bound = floor_;
    if (size < top) {
      const uint32_t o = m > -INFINITY ? order_of(m) : 0;
      uint32_t t = 0;
#pragma unroll
      for (int bit = 31; bit > 13; --bit)
        if (__popcll(__ballot(o >= (t | 1u << bit))) >= top) t |= 1u << bit;
      if (t) bound = fmaxf(bound, logit_of(t));   // a number, or below all of them
    }
    int n = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool in = l[i] >= bound && l[i] > last;
      const uint64_t who = __ballot(in);
      if (who == 0) continue;
      const int place = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
      if (in && place < 64) packed[place] = key_of(l[i], first + (i / 4) * 4 * kThreads + i % 4);
      n += __popcll(who);
    }
    wave_sync();
    Key old = lane < size ? list[lane & 31] : 0, fresh = 0;
    if (n <= 64) {
      // Each entry's place is the number of entries above it.
      fresh = lane < n ? packed[lane] : 0;
      int a = lane, b = 0;
      for (int j = 0; j < n; ++j) {
        const Key k = packed[j];
        a += k > old;
        b += k > fresh;
      }
      for (int j = 0; j < size; ++j) b += list[j] > fresh;
      wave_sync();
      if (lane < size && a < top) list[a] = old;
      if (lane < n && b < top) list[b] = fresh;
      size = size + n < top ? size + n : top;
    } else {
      // Many equal ones, or many in few lanes: one at a time, best first.  `top`
      // steps are enough.
      Key below = ~0ull;   // the last one taken
      for (int step = 0; step < top; ++step) {
        Key k = 0;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
          const Key c = l[i] >= bound && l[i] > last ? key_of(l[i], first + (i / 4) * 4 * kThreads + i % 4) : 0;
          if (c < below) k = max_key(k, c);
        }
#pragma unroll
        for (int off = 1; off < 64; off *= 2) k = max_key(k, __shfl_xor(k, off, 64));
        if (k == 0 || k <= __shfl(old, top - 1, 64)) break;
        const int place = __popcll(__ballot(old > k));
        const Key up = __shfl_up(old, 1, 64);
        old = lane < place ? old : lane == place ? k : up;
        if (lane >= top) old = 0;
        below = k;
      }
      wave_sync();
      if (lane < 32) list[lane] = old;
      size = __popcll(__ballot(old != 0));
    }
    wave_sync();
    if (size == top) {
      const uint32_t o = (uint32_t)(list[top - 1] >> 32);
      last = logit_of(o);
      if (lane == 0) atomicMax(shared, o);
    }
  }
};

// Block (part, row): the logits [part * per, (part + 1) * per) of the row, per a
// multiple of kChunk.
template <bool kTop>
__global__ __launch_bounds__(kThreads) void logprobs_kernel(LogprobArgs a, int per, Part* parts, Key* lists) {
  __shared__ Sums red[kWaves];
  __shared__ Key list[kTop ? kWaves : 1][32];
  __shared__ Key packed[kTop ? kWaves : 1][64];
  __shared__ uint32_t shared;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.y;
  const int from = blockIdx.x * per, to = min(a.n, from + per);
  const float* logits = a.logits + row * a.ld;
  const rsrc_t src = make_rsrc(logits, (uint32_t)a.n * 4u);
  Sums sums = empty_sums();
  Best best{list[kTop ? wave : 0], packed[kTop ? wave : 0], &shared, a.top, 0, -INFINITY};
  if constexpr (kTop) {
    if (lane < 32) list[wave][lane] = 0;
    if (threadIdx.x == 0) shared = 0;
    __syncthreads();
  }
  const float c2 = a.inv_t * kLog2e;
  for (int at = from; at < to; at += kChunk) {
    float l[kEach];
    const int first = at + 4 * (int)threadIdx.x;   // four consecutive ones every 4 * kThreads
    const bool whole = at + kChunk <= a.n;
#pragma unroll
    for (int q = 0; q < kEach / 4; ++q) {
      const f32x4 v = load4(src, logits, first + q * 4 * kThreads, a.n, whole);
#pragma unroll
      for (int i = 0; i < 4; ++i) l[4 * q + i] = fmaxf(v[i], -INFINITY);   // NaN is masked
    }
    if (!whole) {
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (first + (i / 4) * 4 * kThreads + i % 4 >= a.n) l[i] = -INFINITY;
    }
    float m = l[0];
#pragma unroll
    for (int i = 1; i < kEach; ++i) m = fmaxf(m, l[i]);
    rise(sums, m, c2);
    if (m == INFINITY) {   // only these count in this row
#pragma unroll
      for (int i = 0; i < kEach; ++i) sums.s += l[i] == INFINITY ? 1.f : 0.f;
    } else if (sums.m > -INFINITY && sums.m < INFINITY) {
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const float d = fmaxf((l[i] - sums.m) * c2, -1000.f), e = __builtin_amdgcn_exp2f(d);
        sums.s += e;
        sums.t = fmaf(e, d, sums.t);
      }
    }
    if constexpr (kTop) best.add(l, m, first, lane);
  }

  sums = join_wave(sums, c2);
  if (lane == 0) red[wave] = sums;
  if constexpr (kTop) merge_lists(list, kWaves, wave, lane);
  else __syncthreads();
  if (wave != 0) return;
  sums = join_wave(lane < kWaves ? red[lane] : empty_sums(), c2);
  const int t = a.targets[row];
  if (!parts) {
    if (lane == 0) finish(a, row, sums, t >= 0 && t < a.n ? logits[t] : 0.f);
    if (kTop) finish_top(a, row, sums, list[0][lane & 31], lane);
    return;
  }
  const int64_t slot = row * gridDim.x + blockIdx.x;
  if (lane == 0) parts[slot] = {sums.m, sums.s, sums.t, 0.f};
  if (kTop && lane < a.top) lists[slot * a.top + lane] = list[0][lane];
}

// A block per row joins its parts in order.
template <bool kTop>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(LogprobArgs a, int count, const Part* parts,
                                                                 const Key* lists) {
  __shared__ Key list[kTop ? kWaves : 1][32];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const float c2 = a.inv_t * kLog2e;
  const int t = a.targets[row];
  const float target = t >= 0 && t < a.n ? a.logits[row * a.ld + t] : 0.f;
  Sums sums = empty_sums();
  if (wave == 0) {
    for (int i = lane; i < count; i += 64) {
      const Part p = parts[row * count + i];
      sums = join(sums, {p.m, p.s, p.t}, c2);
    }
  }
  if constexpr (kTop) {
    Key k = 0;
    const int j = lane & 31;
    for (int i = wave; i < count; i += kWaves)
      k = merge_best(k, j < a.top ? lists[(row * count + i) * a.top + j] : 0, lane);
    if (lane < 32) list[wave][lane] = k;
    merge_lists(list, kWaves, wave, lane);
  }
  if (wave != 0) return;
  sums = join_wave(sums, c2);
  if (lane == 0) finish(a, row, sums, target);
  if constexpr (kTop) finish_top(a, row, sums, list[0][lane & 31], lane);
}

// Four consecutive gradients a thread.  The last rows first: the forward pass has read
// them last, and the memory-side cache holds up to 256 MB of them; what is read and
// written here passes by that cache, so that it stays theirs (with the forward pass,
// 2047 rows of 50257: 218 us in the rows' order, 203 from the last, 192 with stores
// past the cache; 2048 of 151936: 589, 578, 559, and 544 with loads past it too).
template <typename E>
__global__ __launch_bounds__(256) void logprobs_back_kernel(LogprobBackArgs a, int vec) {
  const int64_t row = gridDim.y - 1 - blockIdx.y;
  const int j = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (j >= a.n) return;
  const f32x4 st = reinterpret_cast<const f32x4*>(a.stats)[row];
  const int t = a.targets && a.dlogprobs ? a.targets[row] : -1;
  const float g = t >= 0 && t < a.n ? a.dlogprobs[row] : 0.f;
  const float h = a.dentropy ? a.dentropy[row] : 0.f;
  const rsrc_t src = make_rsrc(a.logits + row * a.ld, (uint32_t)a.n * 4u);
  const f32x4 v = load4<kStreamed>(src, a.logits + row * a.ld, j, a.n, false);
  const bool finite = st.x < INFINITY;   // in a row with +inf only those entries count
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float l = v[i];
    const float lp = (l == st.x ? 0.f : (l - st.x) * a.inv_t) - st.y;
    const float p = l > -INFINITY ? __builtin_amdgcn_exp2f(lp * kLog2e) : 0.f;
    const float d = (j + i == t ? g : 0.f) - p * (g + h * (lp + st.z));
    o[i] = p > 0.f ? a.inv_t * d : finite && j + i == t && l > -INFINITY ? a.inv_t * g : 0.f;
  }
  E* to = static_cast<E*>(a.dlogits) + row * a.ld_d + j;
  if (vec && j + 4 <= a.n) {
    if constexpr (sizeof(E) == 4) {
      __builtin_nontemporal_store(f32x4{o[0], o[1], o[2], o[3]}, reinterpret_cast<f32x4*>(to));
    } else {
      const bf16x2 x = {static_cast<__bf16>(o[0]), static_cast<__bf16>(o[1])};
      const bf16x2 y = {static_cast<__bf16>(o[2]), static_cast<__bf16>(o[3])};
      __builtin_nontemporal_store(u32x2{__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, y)},
                                  reinterpret_cast<u32x2*>(to));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (j + i >= a.n) break;
      if constexpr (sizeof(E) == 4) to[i] = o[i];
      else to[i] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(o[i]));
    }
  }
}

// Parts of a row: blocks for the whole chip where rows are few, whole chunks each (64
// rows of 151936, best 20: 27 us a call with about 512 blocks or 1024, 29 with 2048,
// whose lists cost more to join; one row of 32000 20 to 22 with any).
int parts_of(int64_t m, int64_t n) {
  const int64_t chunks = (n + kChunk - 1) / kChunk, want = (1024 + m - 1) / m;
  const int64_t each = (chunks + want - 1) / want;
  return (int)((chunks + each - 1) / each);
}

}  // namespace

int64_t logprobs_workspace_bytes(int64_t m, int64_t n, int32_t top) {
  const int64_t parts = parts_of(m, n);
  return parts == 1 ? 0 : m * parts * ((int64_t)sizeof(Part) + 8 * top);
}

hipError_t launch_logprobs(const LogprobArgs& args, void* ws, hipStream_t s) {
  const int parts = parts_of(args.m, args.n);
  const int chunks = (args.n + kChunk - 1) / kChunk;
  const int per = (chunks + parts - 1) / parts * kChunk;
  Part* p = parts > 1 ? static_cast<Part*>(ws) : nullptr;
  Key* lists = p ? reinterpret_cast<Key*>(p + args.m * parts) : nullptr;
  // Rows of one launch: the grid's height (parts is 1 where there are more).
  constexpr int64_t most = 65535;
  for (int64_t at = 0; at < args.m; at += most) {
    LogprobArgs a = args;
    a.m = args.m - at < most ? args.m - at : most;
    a.logits += at * args.ld;
    a.targets += at;
    a.logprobs += at;
    if (a.entropy) a.entropy += at;
    if (a.stats) a.stats += 4 * at;
    if (a.top) {
      a.top_ids += at * a.top;
      a.top_logprobs += at * a.top;
    }
    const dim3 grid((unsigned)parts, (unsigned)a.m);
    if (a.top) hipLaunchKernelGGL(logprobs_kernel<true>, grid, dim3(kThreads), 0, s, a, per, p, lists);
    else hipLaunchKernelGGL(logprobs_kernel<false>, grid, dim3(kThreads), 0, s, a, per, p, lists);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!p) return hipSuccess;
  const dim3 join((unsigned)args.m);
  if (args.top) hipLaunchKernelGGL(logprobs_join_kernel<true>, join, dim3(kThreads), 0, s, args, parts, p, lists);
  else hipLaunchKernelGGL(logprobs_join_kernel<false>, join, dim3(64), 0, s, args, parts, p, lists);
  return hipGetLastError();
}

hipError_t launch_logprobs_back(const LogprobBackArgs& args, int32_t d_type, hipStream_t s) {
  const int e = d_type == Q3_BF16 ? 2 : 4;
  const int vec = args.ld_d % 4 == 0 && reinterpret_cast<uintptr_t>(args.dlogits) % (4 * e) == 0;
  const int64_t blocks = (args.n + 1023) / 1024;
  // Rows of one launch: the grid's height, and less than 2^32 threads.
  const int64_t most = 65535 < 0xFFFFFFFFll / (256 * blocks) ? 65535 : 0xFFFFFFFFll / (256 * blocks);
  for (int64_t end = args.m, at; end > 0; end = at) {
    LogprobBackArgs a = args;
    at = end > most ? end - most : 0;
    a.m = end - at;
    a.logits += at * args.ld;
    if (a.targets) a.targets += at;
    a.stats += 4 * at;
    if (a.dlogprobs) a.dlogprobs += at;
    if (a.dentropy) a.dentropy += at;
    a.dlogits = static_cast<char*>(args.dlogits) + at * args.ld_d * e;
    const dim3 grid((unsigned)blocks, (unsigned)a.m);
    if (d_type == Q3_BF16) hipLaunchKernelGGL(logprobs_back_kernel<uint16_t>, grid, dim3(256), 0, s, a, vec);
    else hipLaunchKernelGGL(logprobs_back_kernel<float>, grid, dim3(256), 0, s, a, vec);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  return hipSuccess;
}

}  // namespace q3
