// Attention of new tokens over a paged cache.
//
//   S_j = scale q . k_j,  o = sum_j e^(S_j - max S) v_j / sum_j e^(S_j - max S)
//
// with the running maximum and sum of a softmax, one pass over the keys.  The
// rows of a sequence and kv head are its (token, head of the group) pairs, token
// by token, so that one decoded token, a few drafted ones and a long chunk are the
// same product with more or fewer rows, and keys are read once for a whole group.
#include <type_traits>

#include "q3_device.h"
#include "q3_internal.h"
#include "q3_paged.h"

namespace q3 {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxKey = 0x7FFFF000;   // positions stay below it, so sums with a step do not pass 2^31

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
  if (start < 0 || end <= start || start >= m) return t;
  const int64_t rows = ((end < m ? end : m) - start) * group;
  const int64_t first = (tile - number(s)) * size;
  if (first < 0 || first >= rows) return t;
  t.sequence = s;
  t.start = (int)start;
  t.end = (int)end;
  t.rows = (int)rows;   // m * heads_q < 2^31
  t.first = (int)first;
  t.length = b.kv_len[s] > 0 ? b.kv_len[s] : 0;
  return t;
}

// The position of a row's token, and the span of positions that rows [r0, r1) of
// the tile's sequence see between them.
__device__ __forceinline__ int position_of(const Tile& t, int row, int group) {
  return t.length - (t.end - (t.start + row / group));
}
// One below the first position that a token at `position` sees.
__device__ __forceinline__ int below_window(const AttendArgs& a, int position) {
  const int64_t low = a.window ? (int64_t)position - a.window : -1;
  return low > -1 ? (int)low : -1;
}
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, const Tile& t, int r0, int r1, int group) {
  const int64_t held = a.batch.table_pages << a.cache.shift;
  int64_t hi = (int64_t)position_of(t, r1 - 1, group) + 1;
  if (hi > held) hi = held;
  if (hi > kMaxKey) hi = kMaxKey;
  const int64_t lo = below_window(a, position_of(t, r0, group)) + 1;
  if (hi < lo) hi = lo;
  return {(int)lo, (int)hi};
}

// ---- tiles of 128 rows ----------------------------------------------------------

constexpr int kWideRows = 128, kStep = 64, kWideThreads = 256;

// Where chunk c (16 bytes) of key row `key` stands among the row's chunks in LDS.
// Keys are read 16 bytes a lane from 16 consecutive rows, values 8 bytes a lane
// from 4 rows and 64 consecutive bytes of each: either way the lanes of a step
// fall on all banks.
template <int DP>
__device__ __forceinline__ uint32_t place_k(uint32_t key) {
  return DP == 64 ? (key >> 1) & 7u : key & 15u;
}
template <int DP>
__device__ __forceinline__ uint32_t place_v(uint32_t key) {
  return DP == 64 ? 4u * ((key >> 1) & 1u) : 4u * (key & 3u);
}

// A partial result's slot: unscaled sums [rows][DP], then maximum and sum of each row.
template <int DP>
constexpr int64_t slot_floats(int rows) { return (int64_t)rows * (DP + 2); }

// Parts that a tile's steps go to: at most `splits`.
__device__ __forceinline__ int parts_of(int steps, int splits) { return steps < splits ? (steps > 0 ? steps : 1) : splits; }

// The same value of the lane's row in the wave's other half.
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

// Four waves with 32 rows each, 64 keys at a time through two LDS buffers.  The
// products are formed transposed, S^T = K Q^T and O^T = V^T P^T: a lane then
// holds half of the scores of one row, so that maxima and sums stay in the lane
// but for one exchange, and what it holds of P^T is the second product's operand
// as it is, the keys of a fragment being taken in the order in which the first
// product leaves them.
template <int DP, bool kExact>
__global__ __launch_bounds__(kWideThreads, DP > 128 ? 1 : 2)
void attend_wide_kernel(AttendArgs a, int splits, float* parts) {
  constexpr int CH = DP / 8;                         // chunks of a key row
  constexpr uint32_t kRow = DP * 2, kTileBytes = kStep * kRow, kBuf = 2 * kTileBytes;
  constexpr int kLoads = CH / 4;                     // of a wave: 16 keys
  constexpr int kKeysPerLoad = 64 / CH;
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ uint32_t held[2][4];                    // each wave's 16 keys: a bit for each that is there
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hk = a.cache.heads, group = a.hq / hk, d = a.cache.d;

  // Contiguous runs of (head, tile) to each XCD: tiles that read the same keys share an L2.
  const int64_t tiles = tiles_of(a.m, a.batch.sequences, group, kWideRows);
  const int64_t total = tiles * hk, id = blockIdx.x % total;
  const int z = (int)(blockIdx.x / total);
  const int64_t per = total >> 3, rem = total & 7, xcd = id & 7;
  const int64_t unit = xcd * per + (xcd < rem ? xcd : rem) + (id >> 3);
  const int head = __builtin_amdgcn_readfirstlane((int)(unit / tiles));
  const int64_t tile = tiles - 1 - unit % tiles;     // the long ones of a chunk first
  const Tile t = find_tile(a, tile, group, kWideRows, lane);
  if (t.sequence == a.batch.sequences) return;
  const int live = t.rows - t.first < kWideRows ? t.rows - t.first : kWideRows;
  const Span span = span_of(a, t, t.first, t.first + live, group);
  const int begin = span.lo & ~(kStep - 1);
  const int steps = (span.hi - begin + kStep - 1) / kStep;
  const int count = parts_of(steps, splits);
  if (z >= count) return;
  const int s0 = (int)((int64_t)steps * z / count), s1 = (int)((int64_t)steps * (z + 1) / count);

  // This lane's row, and its query in registers.
  const int row = 32 * wave + (lane & 31), half = lane >> 5;
  const bool mine = row < live;
  const int r = t.first + (mine ? row : 0);
  const int token = t.start + r / group, qhead = head * group + r % group;
  const int position = position_of(t, r, group), low = below_window(a, position);
  const float c = fabsf(a.scale) * kLog2e;
  bf16x8 q[DP / 16];
#pragma unroll
  for (int k = 0; k < DP / 16; ++k) {
    u32x4 u = {0u, 0u, 0u, 0u};
    if (mine && (kExact || 16 * k < d))
      u = *reinterpret_cast<const u32x4*>(a.q + (int64_t)token * a.ldq + (int64_t)qhead * d + 16 * k + 8 * half);
    if (a.scale < 0.f) u ^= 0x80008000u;             // the maximum is taken before scaling
    q[k] = __builtin_bit_cast(bf16x8, u);
  }

  // The page of one of the wave's 16 keys of a step (lane l: key l % 16), -1 where it is not there.
  auto page_of = [&](int s) {
    const int key = begin + s * kStep + 16 * wave + (lane & 15);
    return s < s1 && key < span.hi ? (int)find_page(a.batch, a.cache, t.sequence, key) : -1;
  };
  const int mask = (1 << a.cache.shift) - 1;
  auto issue = [&](int s, int page) {
    uint8_t* buf = lds + (s & 1) * kBuf + wave * 16 * kRow;
    const uint32_t there = (uint32_t)__ballot(page >= 0) & 0xFFFFu;
    if (lane == 0) held[s & 1][wave] = there;
    const int key0 = begin + s * kStep + 16 * wave;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int k = i * kKeysPerLoad + lane / CH;    // of the wave's 16
      const uint32_t key = 16 * wave + k, at = lane % CH;
      int p = __shfl(page, k, 64);
      p = p < 0 ? 0 : p;                             // read, but never used
      const int64_t from = (int64_t)p * a.cache.page_stride + (((int64_t)head << a.cache.shift) + ((key0 + k) & mask)) * d;
      uint32_t ck = at ^ place_k<DP>(key), cv = at ^ place_v<DP>(key);
      if (!kExact) {
        ck = 8 * ck < (uint32_t)d ? ck : 0;
        cv = 8 * cv < (uint32_t)d ? cv : 0;
      }
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(a.cache.k + from + 8 * ck),
          (__attribute__((address_space(3))) void*)(buf + i * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(a.cache.v + from + 8 * cv),
          (__attribute__((address_space(3))) void*)(buf + kTileBytes + i * 1024), 16, 0, 0);
    }
  };

  f32x16 o[DP / 32];
#pragma unroll
  for (int i = 0; i < DP / 32; ++i) o[i] = f32x16{};
  float top = -INFINITY, sum = 0.f;

  const int first_position = position_of(t, t.first, group);   // of the tile's rows
  const int last_low = below_window(a, position_of(t, t.first + live - 1, group));
  int page = page_of(s0);
  if (s0 < s1) issue(s0, page);
  page = page_of(s0 + 1);
  for (int s = s0; s < s1; ++s) {
    __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): this step's loads and the next one's pages
    __syncthreads();
    if (s + 1 < s1) issue(s + 1, page);
    page = page_of(s + 2);
    uint8_t* buf = lds + (s & 1) * kBuf;
    const int key0 = begin + s * kStep;
    uint64_t there = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) there |= (uint64_t)held[s & 1][w] << (16 * w);
    const bool whole = ~there == 0 && key0 + kStep - 1 <= first_position &&
                       key0 > last_low;
    int bad = 0;
    if (!whole) {
      // Values that are not there, or that some row does not see, must not reach
      // a product: weights of 0 would turn infinities and NaN there into NaN.
      // What is not finite is taken out here and added again below for the rows
      // that see it.
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int k = i * kKeysPerLoad + lane / CH;
        u32x4* p = reinterpret_cast<u32x4*>(buf + kTileBytes + wave * 16 * kRow + i * 1024 + lane * 16);
        u32x4 v = *p;
        if (!((held[s & 1][wave] >> k) & 1)) {
          v = u32x4{0u, 0u, 0u, 0u};
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t f = finite2(v[e]);
            bad |= f != v[e];
            v[e] = f;
          }
        }
        *p = v;
      }
      bad = __syncthreads_or(bad);
    }
    if (32 * wave >= live) continue;

    // S^T: keys of 32-key block b, 8 (i / 4) + 4 half + i % 4, of this lane's row.
    f32x16 sc[2] = {f32x16{}, f32x16{}};
#pragma unroll
    for (int k = 0; k < DP / 16; ++k) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        if (!kExact && 16 * k >= d) continue;
        const uint32_t key = 32 * b + (lane & 31);
        const bf16x8 f = *reinterpret_cast<const bf16x8*>(buf + key * kRow + 16u * ((2 * k + half) ^ place_k<DP>(key)));
        sc[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f, q[k], sc[b], 0, 0, 0);
      }
    }
    if (!whole) {
      const uint64_t seen = there >> (4 * half);
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int k = 32 * b + 8 * (i / 4) + i % 4, key = key0 + k + 4 * half;
          const bool sees = ((seen >> k) & 1) && key <= position && key > low;
          sc[b][i] = sees ? sc[b][i] : -INFINITY;
        }
    }
    float high = sc[0][0];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 16; ++i) high = fmaxf(high, sc[b][i]);
    high = fmaxf(top, fmaxf(high, other_half(high)) * c);
    const float base = high == -INFINITY ? 0.f : high;
    if (__any(high > top)) {
      const float f = __builtin_amdgcn_exp2f(top - base);
      sum *= f;
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) o[i] *= f;
      top = high;
    }
    bf16x8 p[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      u32x4 u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = __builtin_amdgcn_exp2f(fmaf(sc[b / 2][8 * (b % 2) + 2 * i], c, -base));
        const float y = __builtin_amdgcn_exp2f(fmaf(sc[b / 2][8 * (b % 2) + 2 * i + 1], c, -base));
        sum += x + y;
        u[i] = pack_bf16(x, y);
      }
      p[b] = __builtin_bit_cast(bf16x8, u);
    }
    // O^T += V^T P^T.  A transposing read gives each lane one column of four
    // rows: lanes 16 g + i ask for row i / 4 of four, 8 bytes i % 4 of 32.
#pragma unroll
    for (int b = 0; b < 4; ++b) {
#pragma unroll
      for (int n = 0; n < DP / 32; ++n) {
        if (!kExact && 32 * n >= d) continue;
        union {
          s16x4 part[2];
          bf16x8 all;
        } v;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t key = 16 * b + 8 * e + 4 * half + ((lane & 15) >> 2);
          const uint32_t chunk = 4 * n + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
          v.part[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)(
              buf + kTileBytes + key * kRow + 16u * (chunk ^ place_v<DP>(key)) + 8u * (lane & 1)));
        }
        o[n] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v.all, p[b], o[n], 0, 0, 0);
      }
    }
    if (bad) {
      for (int k = 0; k < kStep; ++k) {
        const int key = key0 + k;
        if (!((there >> k) & 1)) continue;
        const bool sees = mine && key <= position && key > low;
        const int64_t from = find_page(a.batch, a.cache, t.sequence, key) * a.cache.page_stride +
                             (((int64_t)head << a.cache.shift) + (key & mask)) * d;
#pragma unroll
        for (int n = 0; n < DP / 32; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int e = 32 * n + 8 * (i / 4) + 4 * half + i % 4;
            if (!kExact && e >= d) continue;
            const float v = __builtin_bit_cast(float, (uint32_t)a.cache.v[from + e] << 16);
            if (sees && !(fabsf(v) < INFINITY)) o[n][i] += v;
          }
      }
    }
  }

  sum += other_half(sum);
  if (!mine) return;
  if (count == 1) {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* to = a.out + (int64_t)token * a.ldo + (int64_t)qhead * d;
#pragma unroll
    for (int n = 0; n < DP / 32; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 32 * n + 8 * i + 4 * half;
        if (!kExact && e >= d) continue;
        *reinterpret_cast<u32x2*>(to + e) = u32x2{pack_bf16(o[n][4 * i] * inv, o[n][4 * i + 1] * inv),
                                                  pack_bf16(o[n][4 * i + 2] * inv, o[n][4 * i + 3] * inv)};
      }
    if (a.lse && half == 0) a.lse[(int64_t)token * a.hq + qhead] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
    return;
  }
  float* slot = parts + ((tile * hk + head) * splits + z) * slot_floats<DP>(kWideRows);
#pragma unroll
  for (int n = 0; n < DP / 32; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4*>(slot + row * DP + 32 * n + 8 * i + 4 * half) =
          f32x4{o[n][4 * i], o[n][4 * i + 1], o[n][4 * i + 2], o[n][4 * i + 3]};
  if (half == 0) {
    slot[kWideRows * DP + 2 * row] = top;
    slot[kWideRows * DP + 2 * row + 1] = sum;
  }
}

// The parts of a tile's rows, in order: eight rows a block, 32 lanes a row.
template <int DP>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int splits, const float* parts) {
  const int lane = threadIdx.x & 63;
  const int hk = a.cache.heads, group = a.hq / hk, d = a.cache.d;
  const int64_t tile = blockIdx.x / hk;
  const int head = blockIdx.x % hk;
  const Tile t = find_tile(a, tile, group, kWideRows, lane);
  if (t.sequence == a.batch.sequences) return;
  const int live = t.rows - t.first < kWideRows ? t.rows - t.first : kWideRows;
  const Span span = span_of(a, t, t.first, t.first + live, group);
  const int count = parts_of((span.hi - (span.lo & ~(kStep - 1)) + kStep - 1) / kStep, splits);
  const int row = blockIdx.y * 8 + threadIdx.x / 32, l = threadIdx.x % 32;
  if (count == 1 || row >= live) return;
  const float* slot = parts + (tile * hk + head) * splits * slot_floats<DP>(kWideRows);
  float top = -INFINITY, sum = 0.f;
  for (int z = 0; z < count; ++z) top = fmaxf(top, slot[z * slot_floats<DP>(kWideRows) + kWideRows * DP + 2 * row]);
  f32x4 o[(DP + 127) / 128] = {};
  for (int z = 0; z < count; ++z) {
    const float* p = slot + z * slot_floats<DP>(kWideRows);
    const float m = p[kWideRows * DP + 2 * row];
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
    sum += f * p[kWideRows * DP + 2 * row + 1];
#pragma unroll
    for (int i = 0; i < (DP + 127) / 128; ++i)
      if (128 * i + 4 * l < DP) o[i] += f * *reinterpret_cast<const f32x4*>(p + row * DP + 128 * i + 4 * l);
  }
  const int r = t.first + row;
  const int64_t token = t.start + r / group;
  const int qhead = head * group + r % group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < (DP + 127) / 128; ++i) {
    const int e = 128 * i + 4 * l;
    if (e < d)
      *reinterpret_cast<u32x2*>(a.out + token * a.ldo + (int64_t)qhead * d + e) =
          u32x2{pack_bf16(o[i][0] * inv, o[i][1] * inv), pack_bf16(o[i][2] * inv, o[i][3] * inv)};
  }
  if (a.lse && l == 0) a.lse[token * a.hq + qhead] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

int padded(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

// Splits of the keys: until every CU has two blocks.
int splits_of(int64_t m, int64_t sequences, int hq, int hk) {
  const int64_t units = tiles_of(m, sequences, hq / hk, kWideRows) * hk;
  if (units >= 384) return 1;
  const int64_t s = 1024 / units;
  return (int)(s < 64 ? s : 64);
}

template <int DP, bool kExact>
hipError_t launch_wide(const AttendArgs& a, float* parts, hipStream_t s) {
  const int hk = a.cache.heads, splits = splits_of(a.m, a.batch.sequences, a.hq, hk);
  const int64_t units = tiles_of(a.m, a.batch.sequences, a.hq / hk, kWideRows) * hk;
  constexpr size_t shm = 4 * kStep * DP * 2;
  static LdsAllowance seen;
  const hipError_t ok = allow_dynamic_lds(reinterpret_cast<const void*>(attend_wide_kernel<DP, kExact>), shm, seen);
  if (ok != hipSuccess) return ok;
  hipLaunchKernelGGL((attend_wide_kernel<DP, kExact>), dim3((unsigned)(units * splits)), dim3(kWideThreads), shm, s, a,
                     splits, parts);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || splits == 1) return e;
  hipLaunchKernelGGL(attend_join_kernel<DP>, dim3((unsigned)units, kWideRows / 8), dim3(256), 0, s, a, splits, parts);
  return hipGetLastError();
}

}  // namespace

int64_t attend_workspace_bytes(int64_t m, int64_t sequences, int32_t hq, int32_t hk, int32_t d) {
  const int splits = splits_of(m, sequences, hq, hk);
  if (splits == 1) return 0;
  const int dp = padded(d);
  return tiles_of(m, sequences, hq / hk, kWideRows) * hk * splits * kWideRows * (dp + 2) * 4;
}

hipError_t launch_attend(const AttendArgs& a, void* ws, hipStream_t s) {
  float* parts = static_cast<float*>(ws);
  switch (a.cache.d) {
    case 64: return launch_wide<64, true>(a, parts, s);
    case 128: return launch_wide<128, true>(a, parts, s);
    case 256: return launch_wide<256, true>(a, parts, s);
  }
  if (a.cache.d < 64) return launch_wide<64, false>(a, parts, s);
  if (a.cache.d < 128) return launch_wide<128, false>(a, parts, s);
  return launch_wide<256, false>(a, parts, s);
}

}  // namespace q3
