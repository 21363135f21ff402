// Attention of new tokens over a paged cache.
//
//   S_j = scale q . k_j,  o = sum_j e^(S_j - max S) v_j / sum_j e^(S_j - max S)
//
// with the running maximum and sum of a softmax, one pass over the keys.  The
// rows of a sequence and kv head are its (token, head of the group) pairs, token
// by token, so that one decoded token, a few drafted ones and a long chunk are the
// same product with more or fewer rows, and keys are read once for a whole group.
//
// Few rows are bound by the cache's bytes (64 tokens over up to 16384, 8 kv heads of
// 128: 437 us, 5.6 TB/s), many by the products, the reads of their fragments and the
// exponentials (2048 over 32000, 32 heads of 128: 1.01 to 1.12 ms on several cards, 0.93
// to 1.03 PFLOP/s).
#include <type_traits>

#include "q3_device.h"
#include "q3_internal.h"
#include "q3_paged.h"
#include "q3_span.h"

namespace q3 {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// A tile of `size` rows of one sequence.  Tiles of sequence s are numbered from
// q_start[s] * group / size + s on: a sequence of n rows has at most n / size + 1
// of them and the next number is above all, so a tile finds its sequence by
// searching q_start, with no list made before.
struct Tile {
  int sequence;    // b.sequences: the tile is empty
  int start;       // the sequence's first row of q
  int end;         // one behind its last new token, as the batch says (positions count from it)
  int rows;        // (token, head) pairs of the sequence
  int first;       // the tile's first
  int length;      // the sequence's positions
};
__host__ __device__ __forceinline__ int64_t tiles_of(int64_t m, int64_t sequences, int group, int size) {
  return m * group / size + sequences;
}
__device__ __forceinline__ Tile find_tile(const AttendArgs& a, int64_t tile, int group, int size, int lane) {
  const BatchView& b = a.batch;
  auto number = [&](int s) { return (int64_t)b.q_start[s] * group / size + s; };
  int lo = 0, hi = b.sequences;   // sequences whose first number is at most `tile`
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int at = lo + (lane + 1) * step - 1;
    const bool below = at < hi && number(at < hi ? at : 0) <= tile;
    const int c = __popcll(__ballot(below));
    const int first = lo + c * step, last = lo + (c + 1) * step - 1;
    lo = first < hi ? first : hi;
    hi = last < hi ? last : hi;
  }
  Tile t{};
  t.sequence = b.sequences;
  if (lo == 0) return t;
  const int s = __builtin_amdgcn_readfirstlane(lo - 1);
  const int64_t m = a.m;
  const int64_t start = b.q_start[s], end = b.q_start[s + 1];
  const int length = b.kv_len[s];   // asked for beside the two above
  if (start < 0 || end <= start || start >= m) return t;
  const int64_t rows = ((end < m ? end : m) - start) * group;
  const int64_t first = (tile - number(s)) * size;
  if (first < 0 || first >= rows) return t;
  t.sequence = s;
  t.start = (int)start;
  t.end = (int)end;
  t.rows = (int)rows;   // m * heads_q < 2^31
  t.first = (int)first;
  t.length = length > 0 ? length : 0;
  return t;
}

// The position of a row's token, and the span of positions that rows [r0, r1) of
// the tile's sequence see between them.
__device__ __forceinline__ int position_of(const Tile& t, int row, int group) {
  return t.length - (t.end - (t.start + row / group));
}
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Tile& t, int r0, int r1, int group) {
  return span_between(position_of(t, r0, group), position_of(t, r1 - 1, group), a.window, a.batch.table_pages,
                      a.cache.shift);
}

// ---- keys and values on their way to LDS ------------------------------------------

// A tile of keys or values in LDS: rows of DT values (the head's, padded with zeros
// to one of the lengths that the kernels are made for), in chunks of 16 bytes.
// Keys are read 16 bytes a lane from 16 consecutive rows, values 8 bytes a lane
// from 4 rows and 64 consecutive bytes of each; place_k and place_v say which bits
// of a chunk's number are turned over in which row, so that the lanes of a step
// fall on all 64 banks either way.
template <int DT>
struct Layout {
  static constexpr int chunks = DT / 8;
  static constexpr uint32_t row = DT * 2;
  static __device__ __forceinline__ uint32_t place_k(uint32_t key) {
    if constexpr (chunks % 16 == 0) return key & 15u;
    else if constexpr (chunks % 8 == 0) return (key >> 1) & 7u;
    else return (key >> 2) & 3u;
  }
  static __device__ __forceinline__ uint32_t place_v(uint32_t key) {
    if constexpr (chunks % 16 == 0) return 4u * (key & 3u);
    else if constexpr (chunks % 8 == 0) return 4u * ((key >> 1) & 1u);
    else return 0u;
  }
};

__device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};   // what stands behind a head's last value

// One wave's 1 KB from memory to LDS: lane l's 16 bytes land at dst + 16 l.  As
// assembly, because the compiler would make every transposing LDS read wait for
// all of them; the kernels wait for the ones they need.  The target stands in m0,
// which the compiler sets (written here and named as such, heads of 256 in chunks
// lose 3%); the first instruction behind that has to wait a cycle.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)p);   // the low half of a generic address
}
__device__ __forceinline__ void load_lds(const void* base, uint32_t offset, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(dst), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds(const void* p, uint32_t dst) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"{m0}"(dst), "v"(p) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_loads() {   // until at most N are under way
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void reads_done() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The pages of a run of positions, checked once and kept in LDS (-1: not there),
// so that no load of a table stands between two of the cache.
constexpr int kListed = 2048;
struct Pages {
  int* id;
  int first;   // the page number that id[0] stands for
};
// Lists those of [key0, key1); whether all that this thread saw of positions below
// `hi` are there.
__device__ __forceinline__ bool list_pages(const AttendArgs& a, const Tile& t, int key0, int key1, int hi, Pages& pages,
                                           int thread, int threads) {
  pages.first = key0 >> a.cache.shift;
  const int count = key1 > key0 ? ((key1 - 1) >> a.cache.shift) - pages.first + 1 : 0;
  bool all = true;
  for (int i = thread; i < count && i < kListed; i += threads) {
    const int64_t key = (int64_t)(pages.first + i) << a.cache.shift;
    const int id = (int)find_page(a.batch, a.cache, t.sequence, key);
    pages.id[i] = id;
    all &= id >= 0 || key >= hi;
  }
  return all;
}
// Keys that a list takes, a multiple of `step`.
__device__ __forceinline__ int listed_keys(const AttendArgs& a, int step) {
  const int64_t n = (int64_t)(kListed - 1) << a.cache.shift;
  return (int)(n < (1 << 30) ? n : 1 << 30) / step * step;
}

// What a wave needs to bring KEYS consecutive keys (or values) of a head: for each
// load, which key and chunk the lane takes.
template <int DT, int KEYS>
struct Loader {
  using L = Layout<DT>;
  static constexpr int count = KEYS * L::chunks / 64;
  uint32_t off[2][count];   // bytes from the first key's row, heads of DT values: keys, values

  static __device__ __forceinline__ uint32_t key_of(int i, int lane) { return (uint32_t)(64 * i + lane) / L::chunks; }
  // `at`: the number of the first key's row in its LDS tile.
  static __device__ __forceinline__ uint32_t chunk_of(int i, int lane, int at, int which) {
    const uint32_t key = at + key_of(i, lane), c = (uint32_t)(64 * i + lane) % L::chunks;
    return c ^ (which ? L::place_v(key) : L::place_k(key));
  }
  __device__ __forceinline__ void init(int lane, int at) {
#pragma unroll
    for (int i = 0; i < count; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w) off[w][i] = (key_of(i, lane) * DT + 8 * chunk_of(i, lane, at, w)) * 2;
  }
  // The page of position key0, to be fetched some time before from() takes it.
  static __device__ __forceinline__ int page_of(const AttendArgs& a, const Pages& pages, int key0) {
    return pages.id[(key0 >> a.cache.shift) - pages.first];
  }
  // Where position key0 of `head` stands in the cache (key0 a multiple of KEYS).
  static __device__ __forceinline__ const uint16_t* from(const AttendArgs& a, int page, int head, int key0, int which) {
    const int shift = a.cache.shift;
    int id = __builtin_amdgcn_readfirstlane(page);
    id = id < 0 ? 0 : id;   // read, but never used
    return (which ? a.cache.v : a.cache.k) + (int64_t)id * a.cache.page_stride +
           (((int64_t)head << shift) + (key0 & ((1 << shift) - 1))) * DT;
  }
  // Load i of positions key0.. of `head`, which: 0 keys, 1 values, in one page from
  // `run` = from() on, rows of DT values;
  __device__ __forceinline__ void load_run(const uint16_t* run, int which, int i, uint32_t dst) const {
    load_lds(run, off[which][i], dst + 1024u * i);
  }
  // and wherever they are.
  static __device__ __forceinline__ void load_any(const AttendArgs& a, const Pages& pages, int head, int key0, int at,
                                                  int which, int i, uint32_t dst, int lane) {
    const int shift = a.cache.shift, mask = (1 << shift) - 1, d = a.cache.d;
    const int key = key0 + (int)key_of(i, lane);
    int id = pages.id[(key >> shift) - pages.first];
    id = id < 0 ? 0 : id;
    const uint32_t c = chunk_of(i, lane, at, which);
    const uint16_t* p = (which ? a.cache.v : a.cache.k) + (int64_t)id * a.cache.page_stride +
                        (((int64_t)head << shift) + (key & mask)) * d + 8 * c;
    load_lds(8 * c < (uint32_t)d ? (const void*)p : (const void*)&kZeros, dst + 1024u * i);
  }
};
// Whether `keys` consecutive positions lie in one page, in rows of DT values.
template <int DT>
__host__ __device__ __forceinline__ bool in_runs(const CacheView& c, int keys) {
  return c.d == DT && (1 << c.shift) >= keys;
}

// ---- the products of one wave -------------------------------------------------------

// A bit for each of the `keys` positions from key0 on that is there.
__device__ __forceinline__ uint64_t there_of(const AttendArgs& a, const Pages& pages, int key0, int hi, int keys,
                                             int lane) {
  const int key = key0 + lane;
  const bool in = lane < keys && key < hi;
  return __ballot(in && pages.id[in ? (key >> a.cache.shift) - pages.first : 0] >= 0);
}

// The lane's other half: the same row's value there.
__device__ __forceinline__ float other_half(float v) {
  const uint32_t u = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t low = r[0], high = r[1];   // lanes 0..31 and 32..63 of v, in both halves
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? low : high);
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}
// The finite halves of two bf16 values; the others as 0.
__device__ __forceinline__ uint32_t finite2(uint32_t u) {
  if ((u & 0x7F80u) == 0x7F80u) u &= 0xFFFF0000u;
  if ((u & 0x7F800000u) == 0x7F800000u) u &= 0xFFFFu;
  return u;
}

// Values that are not there, or that some row of the tile does not see, must not
// reach a product: weights of 0 would turn infinities and NaN there into NaN.  The
// absent ones become zeros, and so does what is not finite, which add_unseen adds
// again for the rows that see it.  KEYS rows from `v` on, a bit of `there` each;
// returns whether this lane took something out.
template <int DT, int KEYS>
__device__ __forceinline__ int clean_values(uint8_t* v, uint32_t there, int lane) {
  int bad = 0;
#pragma unroll
  for (int i = 0; i < KEYS * Layout<DT>::chunks / 64; ++i) {
    u32x4* p = reinterpret_cast<u32x4*>(v + 1024 * i + 16 * lane);
    u32x4 u = *p;
    if (!((there >> ((uint32_t)(64 * i + lane) / Layout<DT>::chunks)) & 1)) {
      u = u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t f = finite2(u[e]);
        bad |= f != u[e];
        u[e] = f;
      }
    }
    *p = u;
  }
  return bad;
}

// A wave's rows and its running sums: NT tiles of 32 rows, in each the lane's row
// is lane % 32.  The products are formed transposed, S^T = K Q^T and O^T = V^T P^T:
// a lane then holds half of the scores of its row (key 8 (i / 4) + 4 half + i % 4 of
// 32 in register i), so maxima and sums stay in the lane but for one exchange, and
// what it holds of P^T is the second product's operand as it is, the keys of a
// fragment being taken in the order in which the first product leaves them.
template <int DT, int NT>
struct Wave {
  bf16x8 q[NT][DT / 16];
  f32x16 o[NT][DT / 32];
  float top[NT], sum[NT];
  int position[NT], low[NT];   // the row sees low < key <= position
  float c;                     // |scale| log2(e)
  uint32_t value[DT / 32];     // byte of the lane's first transposing read, for each 32 values

  __device__ __forceinline__ void init(const AttendArgs& a, const Tile& t, int head, int group, int first, int live,
                                       int lane) {
    c = fabsf(a.scale) * kLog2e;
    const int half = lane >> 5, d = a.cache.d;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = first + 32 * n + (lane & 31);
      const bool mine = row < live;
      const int r = t.first + (mine ? row : 0);
      const int64_t token = t.start + r / group;
      const int qhead = head * group + r % group;
      position[n] = position_of(t, r, group);
      low[n] = below_window(a.window, position[n]);
#pragma unroll
      for (int k = 0; k < DT / 16; ++k) {
        u32x4 u = {0u, 0u, 0u, 0u};
        if (mine && 16 * k < d)
          u = *reinterpret_cast<const u32x4*>(a.q + token * a.ldq + (int64_t)qhead * d + 16 * k + 8 * half);
        if (a.scale < 0.f) u ^= 0x80008000u;   // the maximum is taken before scaling
        q[n][k] = __builtin_bit_cast(bf16x8, u);
      }
#pragma unroll
      for (int i = 0; i < DT / 32; ++i) o[n][i] = f32x16{};
      top[n] = -INFINITY;
      sum[n] = 0.f;
    }
    // A transposing read gives each lane one column of four rows: of 16 lanes, lane
    // i asks for row i / 4 and its bytes 8 (i % 4).. of 32.
    const uint32_t key = 4 * half + ((lane & 15) >> 2);
#pragma unroll
    for (int i = 0; i < DT / 32; ++i) {
      const uint32_t chunk = 4 * i + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
      value[i] = key * Layout<DT>::row + 16u * (chunk ^ Layout<DT>::place_v(key)) + 8u * (lane & 1);
    }
  }

  // Scores of 32 NB keys from the tile at `k`.  Six fragments are read ahead, one
  // beside each product: left to the compiler, every read is waited for at once.
  // beside(i) stands behind product i of kReads.
  template <int NB>
  static constexpr int score_products() { return NB * DT / 16; }
  template <int NB, typename Beside>
  __device__ __forceinline__ void scores(const uint8_t* k, f32x16 (&sc)[NT][NB], int lane, Beside&& beside) const {
    const int half = lane >> 5;
    constexpr int kReads = score_products<NB>(), kAhead = 6;
    auto read = [&](int i) {   // 16 values of 32 keys
      const uint32_t key = 32 * (i % NB) + (lane & 31);
      return *reinterpret_cast<const bf16x8*>(k + key * Layout<DT>::row +
                                              16u * ((2 * (i / NB) + half) ^ Layout<DT>::place_k(key)));
    };
    bf16x8 f[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead && i < kReads; ++i) f[i] = read(i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < NB; ++b) sc[n][b] = f32x16{};
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        sc[n][i % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[i % kAhead], q[n][i / NB], sc[n][i % NB], 0, 0, 0);
      if (i + kAhead < kReads) f[i % kAhead] = read(i + kAhead);
      beside(i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // -inf for what the row does not see: a bit per key, widened to a word each, so
  // that no comparison is kept per register.
  template <int NB>
  __device__ __forceinline__ void mask(f32x16 (&sc)[NT][NB], uint64_t there, int key0, int lane) const {
    const int half = lane >> 5;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int up = position[n] - (key0 + 32 * b) + 1, down = low[n] - (key0 + 32 * b) + 1;   // seen: [down, up)
        uint32_t seen = (uint32_t)(there >> (32 * b));
        seen &= up >= 32 ? ~0u : up <= 0 ? 0u : (1u << up) - 1u;
        seen &= down <= 0 ? ~0u : down >= 32 ? 0u : ~0u << down;
        seen >>= 4 * half;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)seen, 8 * (i / 4) + i % 4, 1);
          const float x = sc[n][b][i];
          sc[n][b][i] = __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, x) & keep) | (0xFF800000u & ~keep));
        }
      }
  }
  // Scores to weights, as bf16 operands of 16 keys each (what the second product
  // takes: a weight is then off by half a step, 2^-8 of itself, as the result is
  // once more.  The sum is that of the unrounded ones.  A second term for what the
  // rounding leaves would cost the narrow kernel nothing, but turns an infinite
  // value into NaN), and O^T += V^T P^T for 32 NB values from the tile at `v`.  The
  // products of one operand run beside the exponentials of the next.
  template <int NB>
  __device__ __forceinline__ void raise(const f32x16 (&sc)[NT][NB]) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float part[4];   // four chains side by side
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        part[i] = sc[n][0][4 * i];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int j = 0; j < 4; ++j) part[i] = fmaxf(part[i], sc[n][b][4 * i + j]);
      }
      float high = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
      high = fmaxf(top[n], fmaxf(high, other_half(high)) * c);
      if (__any(high > top[n])) {
        const float f = __builtin_amdgcn_exp2f(top[n] - (high == -INFINITY ? 0.f : high));
        sum[n] *= f;
#pragma unroll
        for (int i = 0; i < DT / 32; ++i) o[n][i] *= f;
        top[n] = high;
      }
    }
  }
  template <int NB>
  static constexpr int value_products() { return 2 * NB * (DT / 32); }
  template <int NB, typename Beside>
  __device__ __forceinline__ void values(const uint8_t* v, const f32x16 (&sc)[NT][NB], Beside&& beside) {
    constexpr int P = DT / 32, kFrags = value_products<NB>(), kAhead = 4;
    float base[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) base[n] = top[n] == -INFINITY ? 0.f : top[n];
    // Weights 2 i and 2 i + 1 of operand b.
    auto pair = [&](int n, int b, int i) {
      const float x = __builtin_amdgcn_exp2f(fmaf(sc[n][b / 2][8 * (b % 2) + 2 * i], c, -base[n]));
      const float y = __builtin_amdgcn_exp2f(fmaf(sc[n][b / 2][8 * (b % 2) + 2 * i + 1], c, -base[n]));
      sum[n] += x + y;
      return pack_bf16(x, y);
    };
    auto read = [&](int t) {   // 16 keys of 32 values
      union {
        s16x4 part[2];
        bf16x8 all;
      } f;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        f.part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
            v + value[t % P] + (16 * (t / P) + 8 * e) * Layout<DT>::row));
      return f.all;
    };
    bf16x8 f[kAhead];
#pragma unroll
    for (int t = 0; t < kAhead && t < kFrags; ++t) f[t] = read(t);
    __builtin_amdgcn_sched_barrier(0);
    u32x4 now[NT], next[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) now[n][i] = pair(n, 0, i);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int t = 0; t < kFrags; ++t) {
      const int b = t / P, i = t % P;
#pragma unroll
      for (int n = 0; n < NT; ++n)
        o[n][i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f[t % kAhead], __builtin_bit_cast(bf16x8, now[n]), o[n][i], 0, 0, 0);
      if (t + kAhead < kFrags) f[t % kAhead] = read(t + kAhead);
      if (b + 1 < 2 * NB) {
#pragma unroll
        for (int j = 4 * i / P; j < 4 * (i + 1) / P; ++j)
#pragma unroll
          for (int n = 0; n < NT; ++n) next[n][j] = pair(n, b + 1, j);
        if (i == P - 1) {
#pragma unroll
          for (int n = 0; n < NT; ++n) now[n] = next[n];
        }
      }
      beside(t);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // Values that clean_values took out, for the rows that see them (a weight times
  // an infinity or NaN is that again).
  __device__ __forceinline__ void add_unseen(const AttendArgs& a, const Pages& pages, uint64_t there, int head, int key0,
                                             int keys, int lane) {
    const int half = lane >> 5, shift = a.cache.shift, d = a.cache.d;
    for (int k = 0; k < keys; ++k) {
      const int key = key0 + k;
      if (!((there >> k) & 1)) continue;
      const uint16_t* from = a.cache.v + (int64_t)pages.id[(key >> shift) - pages.first] * a.cache.page_stride +
                             (((int64_t)head << shift) + (key & ((1 << shift) - 1))) * d;
#pragma unroll
      for (int i = 0; i < DT / 32; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int e = 32 * i + 8 * j + 4 * half;
          u32x2 u = {0u, 0u};
          if (e < d) u = *reinterpret_cast<const u32x2*>(from + e);
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const uint32_t pair = l < 2 ? u.x : u.y;
            const float x = __builtin_bit_cast(float, l & 1 ? pair & 0xFFFF0000u : pair << 16);
            const float add = fabsf(x) < INFINITY ? 0.f : x;
#pragma unroll
            for (int n = 0; n < NT; ++n) o[n][i][4 * j + l] += key <= position[n] && key > low[n] ? add : 0.f;
          }
          __builtin_amdgcn_sched_barrier(0);   // rare: one load at a time, no registers for more
        }
    }
  }
};

// A partial result's slot: unscaled sums [rows][DT], then maximum and sum of each row.
template <int DT>
constexpr int64_t slot_floats(int rows) { return (int64_t)rows * (DT + 2); }

__device__ __forceinline__ float lse_of(float top, float sum) {
  return sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}
__device__ __forceinline__ void store4(const AttendArgs& a, int64_t token, int qhead, int e, f32x4 v) {
  *reinterpret_cast<u32x2*>(a.out + token * a.ldo + (int64_t)qhead * a.cache.d + e) =
      u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
}

// A row's partial results, put together: a group of as many lanes as it has fours of
// values.
template <int DT>
struct Joined {
  static constexpr int L = DT <= 64 ? 16 : DT <= 128 ? 32 : 64;
  float top = -INFINITY, sum = 0.f;
  f32x4 o = {};

  __device__ __forceinline__ void add(float m, float s, f32x4 v) {
    const float high = fmaxf(top, m), base = high == -INFINITY ? 0.f : high;
    const float f = __builtin_amdgcn_exp2f(top - base), g = __builtin_amdgcn_exp2f(m - base);
    sum = f * sum + g * s;
    o = f * o + g * v;
    top = high;
  }
  // Parts first, first + stride, .. of `count` of row `row` of tiles of `rows`, each read
  // once, kAtOnce of them under way at a time (behind the last it is asked for again).
  template <int kAtOnce, typename Slot>
  __device__ __forceinline__ void gather(Slot&& slot, int first, int stride, int count, int rows, int row, int lane) {
    const int e = 4 * (lane % L) < DT ? 4 * (lane % L) : 0;
    for (int z0 = first; z0 < count; z0 += kAtOnce * stride) {
      float m[kAtOnce], s[kAtOnce];
      f32x4 v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int z = z0 + i * stride;
        const float* p = slot(z < count ? z : count - 1);
        m[i] = p[rows * DT + 2 * row];
        s[i] = p[rows * DT + 2 * row + 1];
        v[i] = *reinterpret_cast<const f32x4*>(p + row * DT + e);
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        if (z0 + i * stride < count) add(m[i], s[i], v[i]);
    }
  }
  // What the wave's groups hold of one row, in every group.
  __device__ __forceinline__ void add_groups() {
#pragma unroll
    for (int off = L; off < 64; off *= 2) {
      f32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __shfl_xor(o[e], off, 64);
      add(__shfl_xor(top, off, 64), __shfl_xor(sum, off, 64), v);
    }
  }
  __device__ __forceinline__ void write(const AttendArgs& a, const Tile& t, int head, int group, int row, int lane) const {
    const int r = t.first + row, l = lane % L;
    const int64_t token = t.start + r / group;
    const int qhead = head * group + r % group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (4 * l < a.cache.d) store4(a, token, qhead, 4 * l, o * inv);
    if (a.lse && l == 0) a.lse[token * a.hq + qhead] = lse_of(top, sum);
  }
};

// The rows of a tile from its parts: a wave a row, or, of more parts than a wave reads in
// two turns, a block a row, whose waves take every fourth turn and whose first adds the
// four up in order (3 sequences of 19 tokens over up to 92000, one kv head of 192
// values, 85 parts: 12.3 us, with a wave a row 38.6; 21 parts of 64 values: 13.5 with a
// block a row, 5.8 with a wave).  Blocks of four waves, blockIdx.y takes every
// gridDim.y-th of the rows, or of the fours of them.
template <int DT, typename Slot>
__device__ __forceinline__ void join_rows(const AttendArgs& a, const Tile& t, int head, int group, Slot&& slot, int count,
                                          int rows, int live) {
  constexpr int L = Joined<DT>::L, G = 64 / L;
  __shared__ f32x4 sums[3][L];
  __shared__ float marks[3][2];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (count <= 16 * G) {
    for (int row = blockIdx.y * 4 + wave; row < live; row += 4 * gridDim.y) {
      Joined<DT> j;
      j.template gather<8>(slot, lane / L, G, count, rows, row, lane);
      j.add_groups();
      if (lane < L) j.write(a, t, head, group, row, lane);
    }
    return;
  }
  for (int row = blockIdx.y; row < live; row += gridDim.y) {
    Joined<DT> j;
    j.template gather<8>(slot, wave * G + lane / L, 4 * G, count, rows, row, lane);
    j.add_groups();
    if (wave && lane < L) {
      sums[wave - 1][lane] = j.o;
      if (lane == 0) {
        marks[wave - 1][0] = j.top;
        marks[wave - 1][1] = j.sum;
      }
    }
    __syncthreads();
    if (threadIdx.x < L) {
#pragma unroll
      for (int w = 0; w < 3; ++w) j.add(marks[w][0], marks[w][1], sums[w][lane]);
      j.write(a, t, head, group, row, lane);
    }
    __syncthreads();
  }
}

// ---- many rows: tiles of 128 -----------------------------------------------------------

constexpr int kStep = 64, kWideRows = 128, kThreads = 256;   // keys of a step, rows of a tile
// Blocks of a CU: two where a wave's sums and queries leave room for a second one on
// its SIMD.  Steps that the LDS of a block holds.
__host__ __device__ constexpr int wide_blocks(int dim) { return dim > 128 ? 1 : 2; }
__host__ __device__ constexpr int wide_ring(int dim) { return dim > 192 ? 2 : dim > 128 ? 3 : dim > 64 ? 2 : 4; }

// Parts that a tile's steps go to: at most `splits`, of three steps at least (2 x 208
// tokens over 1233, 4 kv heads of 256: 40 us, with six 45, with one 58; 4 x 387 over up
// to 402, one head of 192: 26, 30 and 23).
__device__ __forceinline__ int parts_of(int steps, int splits) {
  const int most = (steps + 2) / 3;
  return most < splits ? (most > 0 ? most : 1) : splits;
}

// Whether XCDs share heads.  Not with a few tiles, whose parts have to go round (89 tokens
// over 16464, 2 heads of 192: 41 us, 62 with both heads' parts on an XCD each).
__host__ __device__ __forceinline__ bool heads_share(int64_t tiles, int hk) {
  return hk < 8 && 8 % hk == 0 && tiles * hk >= 64;
}
// Blocks of a launch for each part: those of (head, tile), and some that find nothing
// where XCDs share heads.
__host__ __device__ __forceinline__ uint32_t wide_units(int64_t tiles, int hk) {
  return (uint32_t)(heads_share(tiles, hk) ? (tiles + 8 / hk - 1) / (8 / hk) * 8 : tiles * hk);
}

// Four waves with 32 rows each share 64 keys at a time through a ring of LDS
// buffers.  The loads of a step are asked for beside the products of scores, up to
// three steps ahead.  kRuns: 16 keys are in one page, whole rows.
//
// Heads of 128, two waves a SIMD: for each pair of steps there the products take 2048
// cycles, the CU's reads of fragments from LDS 2048 and its writes 512, and the vector
// work about 2000, of which 1024 are the exponentials.  A step of 32000 keys' worth took
// 4500 cycles a pair, so that these still stand behind one another more than beside.
// Measured and not kept: 64 rows a wave, which halves the reads (its sums move between
// the register files: 2450 us for 1021), eight waves and 256 rows (1060 to 1110), the
// two waves' halves of a step apart (1110 to 1191), 32 keys a step for heads of 256
// (907 for 670).
template <int DT, bool kRuns>
__global__ __launch_bounds__(kThreads, wide_blocks(DT))
void attend_wide_kernel(AttendArgs a, int splits, float* parts) {
  constexpr int R = wide_ring(DT);
  constexpr uint32_t kTile = kStep * Layout<DT>::row, kBuf = 2 * kTile;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int list[kListed];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = a.cache.heads, group = a.hq / hk;

  // An XCD takes whole heads, or every so manieth tile of one: tiles that read the same
  // keys share an L2, and the XCDs have as much to do (4 kv heads of 256, 2048 tokens of
  // 16 heads over 16000: 674 us, with a run of tiles for each XCD, of which one had a
  // block more than CUs, 1282; 4096 over 4096: 218 and 406).
  const uint32_t tiles = (uint32_t)tiles_of(a.m, a.batch.sequences, group, kWideRows);
  const uint32_t total = wide_units(tiles, hk);   // below 2^24
  const int z = __builtin_amdgcn_readfirstlane(blockIdx.x / total);
  const uint32_t id = blockIdx.x - z * total, xcd = id & 7;
  uint32_t unit, place;
  if (heads_share(tiles, hk)) {
    const uint32_t each = 8 / hk;   // XCDs of a head
    unit = xcd / each;
    place = (id >> 3) * each + xcd % each;
  } else {
    const uint32_t per = total >> 3, rem = total & 7, at = xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
    unit = at / tiles;
    place = at - unit * tiles;
  }
  if (place >= tiles) return;
  const int head = __builtin_amdgcn_readfirstlane(unit);
  const int64_t tile = tiles - 1 - __builtin_amdgcn_readfirstlane(place);     // the long ones of a chunk first
  const Tile t = find_tile(a, tile, group, kWideRows, lane);
  if (t.sequence == a.batch.sequences) return;
  const int live = t.rows - t.first < kWideRows ? t.rows - t.first : kWideRows;
  const Span span = span_of(a, t, t.first, t.first + live, group);
  const int begin = first_of(span, kStep), steps = steps_of(span, kStep);
  const int count = parts_of(steps, splits);
  if (z >= count) return;
  const int s0 = (int)((int64_t)steps * z / count), s1 = (int)((int64_t)steps * (z + 1) / count);

  Wave<DT, 1> w;
  w.init(a, t, head, group, 32 * wave, live, lane);
  const int first_position = position_of(t, t.first, group);   // of the tile's rows
  const int last_low = below_window(a.window, position_of(t, t.first + live - 1, group));
  const bool mine = 32 * wave < live;
  // A wave brings 16 keys of a step, and their values.
  const int keys16 = 16 * wave;
  Loader<DT, 16> loader;
  loader.init(lane, keys16);
  constexpr int N = 2 * Loader<DT, 16>::count;   // a wave's loads of a step
  Pages pages{list, 0};
  const uint32_t base = lds_offset(lds) + keys16 * Layout<DT>::row;
  // Where this wave's part of step s stands, and load i of N of it.
  struct Where {
    int key0;
    const uint16_t* run[2];
  };
  auto where = [&](int s, int page) {
    Where o;
    o.key0 = begin + s * kStep + keys16;
#pragma unroll
    for (int i = 0; i < 2; ++i) o.run[i] = kRuns ? loader.from(a, page, head, o.key0, i) : nullptr;
    return o;
  };
  auto load = [&](const Where& o, int slot, int i) {
    const int which = i / loader.count, j = i % loader.count;
    const uint32_t dst = base + slot * kBuf + which * kTile;
    if (kRuns) loader.load_run(o.run[which], which, j, dst);
    else loader.load_any(a, pages, head, o.key0, keys16, which, j, dst, lane);
  };

  const int run_steps = listed_keys(a, kStep) / kStep;
  for (int w0 = s0; w0 < s1; w0 += run_steps) {
    const int w1 = s1 - w0 < run_steps ? s1 : w0 + run_steps;
    meet();   // the list and the ring are free
    bool all = list_pages(a, t, begin + w0 * kStep, begin + w1 * kStep, span.hi, pages, threadIdx.x, kThreads);
    __builtin_amdgcn_s_waitcnt(0x0F70);   // the compiler knows that queries are here (and waits in the loop for nothing)
    all = __syncthreads_and(all);
    // Behind the last step it is asked for again, and never used, so that every step
    // has the same loads under way.
    auto page_of = [&](int s) { return loader.page_of(a, pages, begin + (s < w1 ? s : w1 - 1) * kStep + keys16); };
#pragma unroll
    for (int i = 0; i < R - 1; ++i) {
      const Where o = where(w0 + i < w1 ? w0 + i : w1 - 1, page_of(w0 + i));
#pragma unroll
      for (int j = 0; j < N; ++j) load(o, i, j);
    }
    int page = page_of(w0 + R - 1);
    int slot = 0, free = R - 1;   // this step's, and the one that the step before has left
    // Steps that every row of the tile sees whole, all of them there.
    const int last = span.hi - 1 < first_position ? span.hi - 1 : first_position;
    for (int s = w0; s < w1; ++s) {
      wait_loads<(R - 2) * N>();   // this step's: all but those of the R - 2 behind it
      meet();                      // everyone's, and everyone has left the step before
      uint8_t* buf = lds + slot * kBuf;
      const int key0 = begin + s * kStep, next = s + R - 1 < w1 ? s + R - 1 : w1 - 1;
      const bool whole = all && key0 + kStep - 1 <= last && key0 > last_low;
      const Where o = where(next, page);
      uint64_t there = ~0ull;
      int bad = 0;
      if (!whole) {
        there = there_of(a, pages, key0, span.hi, kStep, lane);
        bad = clean_values<DT, 16>(buf + kTile + keys16 * Layout<DT>::row, (uint32_t)(there >> keys16), lane);
        bad = __syncthreads_or(bad);
      }
      f32x16 sc[1][2];
      if (mine) {
        constexpr int kProducts = w.template score_products<2>();
        w.scores(buf, sc, lane, [&](int i) {
#pragma unroll
          for (int j = i * N / kProducts; j < (i + 1) * N / kProducts; ++j) load(o, free, j);
        });
      } else {
#pragma unroll
        for (int j = 0; j < N; ++j) load(o, free, j);
      }
      page = page_of(s + R);
      if (mine) {
        if (!whole) w.mask(sc, there, key0, lane);
        w.raise(sc);
        w.values(buf + kTile, sc, [](int) {});
        if (bad) w.add_unseen(a, pages, there, head, key0, kStep, lane);
      }
      free = slot;
      slot = slot + 1 == R ? 0 : slot + 1;
    }
    wait_loads<0>();
  }

  const int row = 32 * wave + (lane & 31), half = lane >> 5;
  const float sum = w.sum[0] + other_half(w.sum[0]);
  if (row >= live) return;
  const int r = t.first + row;
  const int64_t token = t.start + r / group;
  const int qhead = head * group + r % group;
  if (count == 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int n = 0; n < DT / 32; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 32 * n + 8 * i + 4 * half;
        const f32x16& o = w.o[0][n];
        if (e < a.cache.d)
          store4(a, token, qhead, e, f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]} * inv);
      }
    if (a.lse && half == 0) a.lse[token * a.hq + qhead] = lse_of(w.top[0], sum);
    return;
  }
  float* slot = parts + ((tile * hk + head) * splits + z) * slot_floats<DT>(kWideRows);
#pragma unroll
  for (int n = 0; n < DT / 32; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x16& o = w.o[0][n];
      *reinterpret_cast<f32x4*>(slot + row * DT + 32 * n + 8 * i + 4 * half) =
          f32x4{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
    }
  if (half == 0) {
    slot[kWideRows * DT + 2 * row] = w.top[0];
    slot[kWideRows * DT + 2 * row + 1] = sum;
  }
}

// The parts of a tile's rows.  With few splits a wave has several rows (a chunk of 500
// and 8 tokens, heads of 64, three parts: 5.3 us, with a wave for each row 12.3).
constexpr int kFewSplits = 8;
template <int DT, bool kFew>
__global__ __launch_bounds__(kThreads) void attend_wide_join_kernel(AttendArgs a, int splits, const float* parts) {
  const int hk = a.cache.heads, group = a.hq / hk;
  const int tile = __builtin_amdgcn_readfirstlane(blockIdx.x / (uint32_t)hk), head = blockIdx.x - tile * hk;
  const Tile t = find_tile(a, tile, group, kWideRows, threadIdx.x & 63);
  if (t.sequence == a.batch.sequences) return;
  const int live = t.rows - t.first < kWideRows ? t.rows - t.first : kWideRows;
  const int count = parts_of(steps_of(span_of(a, t, t.first, t.first + live, group), kStep), splits);
  if (count == 1) return;
  const float* first = parts + ((int64_t)tile * hk + head) * splits * slot_floats<DT>(kWideRows);
  auto slot = [&](int z) { return first + z * slot_floats<DT>(kWideRows); };
  if constexpr (!kFew) {
    join_rows<DT>(a, t, head, group, slot, count, kWideRows, live);
  } else {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    constexpr int L = Joined<DT>::L, G = 64 / L;
    for (int row = (blockIdx.y * 4 + wave) * G + lane / L; row < live; row += 4 * gridDim.y * G) {
      Joined<DT> x;
      x.template gather<4>(slot, 0, 1, count, kWideRows, row, lane);
      x.write(a, t, head, group, row, lane);
    }
  }
}

// Splits of the keys of a tile: as many as there are blocks for at a time, if that is two
// or more (3 x 440 tokens over 3011, 8 heads of 64: 30 us, twice as many 40; 32 heads of
// 128 over 32000, 800 tokens, 208 units: 493 and 513); else as many as for twice over
// (1300 tokens, 336 units: 714, in one part 865), but in one part from three quarters on
// (1700 tokens, 432 units: 946, in two parts 987).
int wide_splits(int64_t units, int dim) {
  const int64_t want = 256 * wide_blocks(dim);
  if (4 * units >= 3 * want) return 1;
  const int64_t s = want / units > 1 ? want / units : 2 * want / units;
  return (int)(s < 64 ? s : 64);
}

// ---- few rows: tiles of 32 or 64 -----------------------------------------------------------

// Bound by the cache's bytes.  Each wave of a block streams keys and values of its
// own, 32 at a time, through its own part of LDS: no barrier stands in the stream,
// and while a wave computes on one tile, others are on their way.  The four
// waves take every fourth tile and join their sums through LDS at the end.
//
// A fixed number of blocks, one to three a CU, shares out the whole batch's work,
// counted in steps of 128 keys: sequences in order, in each the kv heads, in each
// the tiles of rows, in each the steps.  A block takes an equal run of steps,
// wherever it begins and ends, so that contexts of any lengths load the chip
// evenly.  A tile that is cut between blocks leaves a partial result in each (a
// block has at most one tile that it continues and one that others continue), and
// a second launch joins them in order.
constexpr int kNarrowStep = 128;
// Blocks of a CU, as many as registers allow, so that some stream while another begins
// or ends a tile, and how many tiles of keys, and of values, a wave's part of LDS holds.
// 8 kv heads of 128, two blocks with one tile each against one block with two: 64 single
// tokens over up to 500 positions 35 and 58 us, over up to 16384 436 and 455.  Heads of
// 64, three with one tile against two with two: 24 and 28, 230 and 234 (four spill).
template <int DT, int NT>
constexpr int per_cu() { return NT == 1 ? (DT <= 64 ? 3 : DT <= 128 ? 2 : 1) : DT <= 64 ? 2 : 1; }
template <int DT, int NT>
constexpr int ring_of() { return NT == 1 || DT > 128 ? 1 : 2; }
template <int DT, int NT>
constexpr size_t narrow_bytes() { return 4 * ring_of<DT, NT>() * 2 * 32 * Layout<DT>::row; }
template <int DT, int NT>
constexpr int narrow_blocks() { return 256 * per_cu<DT, NT>(); }

// A block's tile that others continue: what the second launch joins.
struct Cut {
  int start, rows;   // the sequence's first row of q and its rows (0: no tile)
  int first;         // the tile's first row
  int head;
  int last;          // the last block that has a part of it
};

// A sequence's share of the work.
struct Share {
  Tile t;
  Span span;
  int tiles, steps;
};
__device__ __forceinline__ Share share_of(const AttendArgs& a, int s, int group, int size) {
  Share w{};
  const int64_t start = a.batch.q_start[s], end = a.batch.q_start[s + 1];
  const int length = a.batch.kv_len[s];   // asked for beside the two above
  if (start < 0 || end <= start || start >= a.m) return w;
  w.t.sequence = s;
  w.t.start = (int)start;
  w.t.end = (int)end;
  w.t.rows = (int)(((end < a.m ? end : a.m) - start) * group);
  w.t.length = length > 0 ? length : 0;
  w.span = span_of(a, w.t, 0, w.t.rows, group);
  w.tiles = (w.t.rows + size - 1) / size;
  w.steps = steps_of(w.span, kNarrowStep);
  if (w.steps < 1) w.steps = 1;   // rows that see nothing are written too
  return w;
}
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)v), high = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return (int64_t)((uint64_t)high << 32 | low);
}
__device__ __forceinline__ int64_t wave_sum64(int64_t v) {
#pragma unroll
  for (int off = 1; off < 64; off *= 2) v += __shfl_xor(v, off, 64);
  return uniform(v);
}

template <int DT, int NT, bool kRuns>
__global__ __launch_bounds__(kThreads, (per_cu<DT, NT>()))
void attend_narrow_kernel(AttendArgs a, float* parts, Cut* cuts) {
  constexpr int kRows = 32 * NT, R = ring_of<DT, NT>();
  constexpr uint32_t kTile = 32 * Layout<DT>::row;
  constexpr int N = kTile / 1024;   // loads of a tile
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int list[kListed];
  __shared__ float marks[4][kRows][2];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = a.cache.heads, group = a.hq / hk, b = a.batch.sequences;
  auto work_of = [&](int s) {
    if (s >= b) return (int64_t)0;
    const Share w = share_of(a, s, group, kRows);
    return (int64_t)w.tiles * w.steps * hk;
  };

  // The block's run of steps [from, to), and the sequence that holds its first.
  constexpr int blocks = narrow_blocks<DT, NT>();
  auto running = [&](int64_t v) {   // sums of lanes 0..lane
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
      const int64_t up = __shfl_up(v, off, 64);
      if (lane >= off) v += up;
    }
    return v;
  };
  int64_t sums = running(work_of(lane)), total = uniform(__shfl(sums, 63, 64));   // of the first 64 sequences
  for (int s0 = 64; s0 < b; s0 += 64) total += wave_sum64(work_of(s0 + lane));
  const int64_t share = (total + blocks - 1) / blocks;
  const int64_t from = share * blockIdx.x, to = from + share < total ? from + share : total;
  Cut cut{};
  int s = 0;
  int64_t before = 0;   // steps of the sequences before s
  for (int s0 = 0; from < to && s0 < b; s0 += 64) {
    if (s0) sums = running(work_of(s0 + lane));
    const int64_t all = uniform(__shfl(sums, 63, 64));
    if (before + all > from) {
      const int n = __popcll(__ballot(before + sums <= from));   // sequences of these that end before
      const int64_t skipped = uniform(__shfl(sums, n > 0 ? n - 1 : 0, 64));
      before += n > 0 ? skipped : 0;
      s = s0 + n;
      break;
    }
    before += all;
  }
  s = __builtin_amdgcn_readfirstlane(s);

  uint8_t* mine = lds + wave * (R * 2) * kTile;   // [slot][keys, values]
  const uint32_t base = lds_offset(mine);
  Loader<DT, 32> loader;
  loader.init(lane, 0);
  Pages pages{list, 0};

  for (int64_t at = from; at < to;) {
    if (s >= b) break;
    const Share sh = share_of(a, s, group, kRows);
    const int64_t here = (int64_t)sh.tiles * sh.steps * hk, in = at - before;
    if (in >= here) {
      before += here;
      ++s;
      continue;
    }
    const int unit = in >> 32 ? (int)uniform(in / sh.steps)
                              : (int)__builtin_amdgcn_readfirstlane((uint32_t)in / (uint32_t)sh.steps);
    const int c0 = (int)(in - (int64_t)unit * sh.steps);
    const int n = (int)(sh.steps - c0 < to - at ? sh.steps - c0 : to - at);
    const int head = __builtin_amdgcn_readfirstlane(unit / sh.tiles);
    Tile t = sh.t;
    t.first = (unit - head * sh.tiles) * kRows;
    const int live = t.rows - t.first < kRows ? t.rows - t.first : kRows;
    const int begin = first_of(sh.span, kNarrowStep);
    const int first_position = position_of(t, t.first, group);
    const int last_position = position_of(t, t.first + live - 1, group);
    const int last_low = below_window(a.window, last_position);
    const bool complete = c0 == 0 && n == sh.steps;
    if (c0 == 0 && !complete) {
      const int64_t last = at + sh.steps - 1;   // the tile's last step
      cut = Cut{t.start, t.rows, t.first, head, (int)uniform(last / share)};
    }

    Wave<DT, NT> w;
    w.init(a, t, head, group, 0, live, lane);
    const int run = listed_keys(a, kNarrowStep) / kNarrowStep;
    for (int w0 = c0; w0 < c0 + n; w0 += run) {
      const int w1 = c0 + n - w0 < run ? c0 + n : w0 + run;
      meet();   // the list and the ring are free
      list_pages(a, t, begin + w0 * kNarrowStep, begin + w1 * kNarrowStep, sh.span.hi, pages, threadIdx.x, kThreads);
      // The stream counts its loads: nothing else is under way, and the compiler
      // knows that queries are here (it would wait for them inside the loop).
      __builtin_amdgcn_s_waitcnt(0x0F70);
      meet();
      // This wave's tiles: 32 keys from begin + 128 (w0 + i) + 32 wave on.
      const int key_w = begin + w0 * kNarrowStep + 32 * wave;
      int count = (sh.span.hi - key_w + kNarrowStep - 1) / kNarrowStep;
      count = count < 0 ? 0 : count < w1 - w0 ? count : w1 - w0;
      auto issue = [&](int i, int which) {
        const int key0 = key_w + i * kNarrowStep;
        const uint32_t dst = base + ((i & (R - 1)) * 2 + which) * kTile;
        if (kRuns) {
          const uint16_t* from = loader.from(a, loader.page_of(a, pages, key0), head, key0, which);
#pragma unroll
          for (int j = 0; j < N; ++j) loader.load_run(from, which, j, dst);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) loader.load_any(a, pages, head, key0, 0, which, j, dst, lane);
        }
      };
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (i < count) {
          issue(i, 0);
          issue(i, 1);
        }
      }
      for (int i = 0; i < count; ++i) {
        const int key0 = key_w + i * kNarrowStep, left = count - i;
        uint8_t* kt = mine + (i & (R - 1)) * 2 * kTile;
        uint8_t* vt = kt + kTile;
        const uint32_t there = (uint32_t)there_of(a, pages, key0, sh.span.hi, 32, lane);
        const bool none = there == 0 || key0 > last_position;
        const bool whole = ~there == 0 && key0 + 31 <= first_position && key0 > last_low;
        // Under way behind this tile's keys: its values and the R - 1 tiles after it.
        if (R == 2 && left >= 2) wait_loads<3 * N>();
        else wait_loads<N>();
        f32x16 sc[NT][1];
        if (!none) {
          w.scores(kt, sc, lane, [](int) {});
          if (!whole) w.mask(sc, there, key0, lane);
          w.raise(sc);
        }
        reads_done();
        if (left > R) issue(i + R, 0);
        if (R == 2) {
          if (left >= 3) wait_loads<3 * N>();
          else if (left == 2) wait_loads<2 * N>();
          else wait_loads<0>();
        } else {
          if (left >= 2) wait_loads<N>();
          else wait_loads<0>();
        }
        if (!none) {
          int bad = 0;
          if (!whole) {
            bad = __any(clean_values<DT, 32>(vt, there, lane));
            reads_done();
          }
          w.values(vt, sc, [](int) {});
          if (bad) w.add_unseen(a, pages, there, head, key0, 32, lane);
        }
        reads_done();
        if (left > R) issue(i + R, 1);
      }
    }

    // The four waves' sums: each scaled to the largest maximum, then added in order,
    // as many values of all rows at a time as the ring's LDS holds.
    meet();   // the ring is free
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const float sum = w.sum[i] + other_half(w.sum[i]);
      if (lane < 32) {
        marks[wave][32 * i + lane][0] = w.top[i];
        marks[wave][32 * i + lane][1] = sum;
      }
    }
    meet();
    float f[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int v = 0; v < 4; ++v) top = fmaxf(top, marks[v][32 * i + (lane & 31)][0]);
      f[i] = w.top[i] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(w.top[i] - top);
    }
    // Slots of what is continued, block by block, then of what is begun.
    float* slot = parts + (blockIdx.x + (c0 == 0 ? (int64_t)gridDim.x : 0)) * slot_floats<DT>(kRows);
    constexpr int kPitch = 36;   // floats of 32 values and room against bank conflicts
    constexpr int kAll = DT / 32, kSlice = 4 * kRows * kPitch;
    constexpr int kFit = (int)(narrow_bytes<DT, NT>() / (4 * kSlice));
    // (Two tiles of rows have no registers left for more than one slice.)
    constexpr int kSlices = NT > 1 ? 1 : kFit >= kAll ? kAll : kFit >= 2 && kAll % 2 == 0 ? 2 : 1;
    static_assert(kFit >= kSlices, "");
#pragma unroll
    for (int d1 = 0; d1 < kAll; d1 += kSlices) {
#pragma unroll
      for (int g = 0; g < kSlices; ++g)
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          float* to = reinterpret_cast<float*>(lds) + g * kSlice + (wave * kRows + 32 * i + (lane & 31)) * kPitch +
                      4 * (lane >> 5);
          const f32x16& o = w.o[i][d1 + g];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<f32x4*>(to + 8 * j) = f32x4{o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]} * f[i];
        }
      meet();
#pragma unroll
      for (int g = 0; g < kSlices; ++g) {
        const int d0 = d1 + g;
        const float* buf = reinterpret_cast<const float*>(lds) + g * kSlice;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int row = 32 * i + threadIdx.x / 8, e = 4 * (threadIdx.x % 8);
          if (row < live) {
            f32x4 v = {};
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v += *reinterpret_cast<const f32x4*>(buf + (k * kRows + row) * kPitch + e);
              top = fmaxf(top, marks[k][row][0]);
            }
            // (A wave whose scores are all NaN has the lowest maximum and a sum that counts.)
            const float floor_ = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              sum += marks[k][row][1] * __builtin_amdgcn_exp2f(marks[k][row][0] - floor_);
            if (complete) {
              const int r = t.first + row;
              const int64_t token = t.start + r / group;
              const int qhead = head * group + r % group;
              const float inv = sum == 0.f ? 0.f : 1.f / sum;
              if (32 * d0 + e < a.cache.d) store4(a, token, qhead, 32 * d0 + e, v * inv);
              if (a.lse && d0 == 0 && e == 0) a.lse[token * a.hq + qhead] = lse_of(top, sum);
            } else {
              *reinterpret_cast<f32x4*>(slot + row * DT + 32 * d0 + e) = v;
              if (d0 == 0 && e == 0) {
                slot[kRows * DT + 2 * row] = top;
                slot[kRows * DT + 2 * row + 1] = sum;
              }
            }
          }
        }
      }
      meet();
    }
    at += n;
  }
  if (threadIdx.x == 0) cuts[blockIdx.x] = cut;
}

// Blocks (x, y) join the tile that block x of the kernel above began and others went on
// with.
template <int DT, int NT>
__global__ __launch_bounds__(kThreads) void attend_narrow_join_kernel(AttendArgs a, const float* parts, const Cut* cuts) {
  constexpr int kRows = 32 * NT;
  const Cut cut = cuts[blockIdx.x];
  Tile t{};
  t.start = cut.start;
  t.rows = cut.rows;
  t.first = cut.first;
  const int live = t.rows - t.first < kRows ? t.rows - t.first : kRows;   // 0: no tile
  const int64_t x = blockIdx.x, blocks = gridDim.x;
  join_rows<DT>(a, t, cut.head, a.hq / a.cache.heads,
                [&](int z) { return parts + (z ? x + z : blocks + x) * slot_floats<DT>(kRows); }, cut.last - (int)x + 1,
                kRows, live);
}

// ---- which of them -----------------------------------------------------------------------

enum Form { kNarrow32, kNarrow64, kWide };
// By the rows that a sequence has on average.  8 sequences of 20000, 8 kv heads of 128
// values: at 32 rows 132 us (narrow, 32) and 135 (wide), at 64 rows 202 (narrow, 32), 146
// (narrow, 64) and 164, at 72 rows 230 (narrow, 64) and 166; of 256 values at 32 rows
// 247 and 299, at 48 (narrow, 32: two tiles) 556 and 388 (two tiles at a time do not fit
// a wave's registers there).  Unlike lengths are a reason for the narrow ones besides:
// 64 single tokens over up to 16384, 8 kv heads of 192, 660 us and 940.
Form form_of(int64_t m, int64_t sequences, int group, int dim) {
  const int64_t rows = m * group;
  if (rows <= 32 * sequences) return kNarrow32;
  return rows <= 64 * sequences && dim <= 128 ? kNarrow64 : kWide;
}

template <typename F>
auto by_dim(int d, F&& f) {
  if (d <= 64) return f(std::integral_constant<int, 64>{});
  if (d <= 96) return f(std::integral_constant<int, 96>{});
  if (d <= 128) return f(std::integral_constant<int, 128>{});
  if (d <= 192) return f(std::integral_constant<int, 192>{});
  return f(std::integral_constant<int, 256>{});
}

template <int DT>
hipError_t launch_wide(const AttendArgs& a, float* parts, hipStream_t s) {
  const int64_t units = tiles_of(a.m, a.batch.sequences, a.hq / a.cache.heads, kWideRows) * a.cache.heads;
  const int splits = wide_splits(units, DT);
  constexpr size_t shm = wide_ring(DT) * 2 * kStep * Layout<DT>::row;
  static LdsAllowance seen, seen_runs;
  const bool runs = in_runs<DT>(a.cache, 16);
  auto* kernel = runs ? attend_wide_kernel<DT, true> : attend_wide_kernel<DT, false>;
  const hipError_t ok = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), shm, runs ? seen_runs : seen);
  if (ok != hipSuccess) return ok;
  hipLaunchKernelGGL(kernel, dim3(wide_units(units / a.cache.heads, a.cache.heads) * splits), dim3(kThreads), shm, s, a,
                     splits, parts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  if (splits <= kFewSplits)
    hipLaunchKernelGGL((attend_wide_join_kernel<DT, true>), dim3((unsigned)units, kWideRows * Joined<DT>::L / 256),
                       dim3(kThreads), 0, s, a, splits, parts);
  else
    hipLaunchKernelGGL((attend_wide_join_kernel<DT, false>), dim3((unsigned)units, kWideRows / 4), dim3(kThreads), 0, s, a,
                       splits, parts);
  return hipGetLastError();
}

template <int DT, int NT>
hipError_t launch_narrow(const AttendArgs& a, float* parts, hipStream_t s) {
  constexpr int blocks = narrow_blocks<DT, NT>();
  constexpr size_t shm = narrow_bytes<DT, NT>();
  Cut* cuts = reinterpret_cast<Cut*>(parts + 2 * blocks * slot_floats<DT>(32 * NT));
  static LdsAllowance seen, seen_runs;
  const bool runs = in_runs<DT>(a.cache, 32);
  auto* kernel = runs ? attend_narrow_kernel<DT, NT, true> : attend_narrow_kernel<DT, NT, false>;
  const hipError_t ok = allow_dynamic_lds(reinterpret_cast<const void*>(kernel), shm, runs ? seen_runs : seen);
  if (ok != hipSuccess) return ok;
  hipLaunchKernelGGL(kernel, dim3(blocks), dim3(kThreads), shm, s, a, parts, cuts);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_narrow_join_kernel<DT, NT>), dim3(blocks, 8192 / blocks), dim3(kThreads), 0, s, a, parts, cuts);
  return hipGetLastError();
}

}  // namespace

int64_t attend_workspace_bytes(int64_t m, int64_t sequences, int32_t hq, int32_t hk, int32_t d) {
  return by_dim(d, [&](auto dim) -> int64_t {
    constexpr int DT = decltype(dim)::value;
    const Form form = form_of(m, sequences, hq / hk, DT);
    if (form != kWide) {
      const bool one = form == kNarrow32;
      const int64_t blocks = one ? narrow_blocks<DT, 1>() : narrow_blocks<DT, 2>();
      return blocks * (2 * 4 * slot_floats<DT>(one ? 32 : 64) + (int64_t)sizeof(Cut));
    }
    const int64_t units = tiles_of(m, sequences, hq / hk, kWideRows) * hk;
    const int splits = wide_splits(units, DT);
    return splits == 1 ? 0 : units * splits * slot_floats<DT>(kWideRows) * 4;
  });
}

hipError_t launch_attend(const AttendArgs& a, void* ws, hipStream_t s) {
  float* parts = static_cast<float*>(ws);
  return by_dim(a.cache.d, [&](auto dim) {
    constexpr int DT = decltype(dim)::value;
    const Form form = form_of(a.m, a.batch.sequences, a.hq / a.cache.heads, DT);
    if (form == kNarrow32) return launch_narrow<DT, 1>(a, parts, s);
    if constexpr (DT <= 128)
      if (form == kNarrow64) return launch_narrow<DT, 2>(a, parts, s);
    return launch_wide<DT>(a, parts, s);
  });
}

}  // namespace q3
