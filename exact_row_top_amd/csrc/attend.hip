// attend.hip -- decode attention over a paged cache for sequences that share
// a prefix, and the attention mass of cached positions.
//
// The queries of a group's sequences meet the group's prefix together: their
// rows (sequences x tokens x query heads of a key head) are the columns of one
// matrix product, so each key and value of the prefix is read once for all of
// them.  Each sequence's own positions follow in the same way by themselves.
// Keys are split over workgroups and a second launch joins the splits of a
// row by their largest scores and sums.
//
// Layout.  Scores are made transposed, S^T = K Q^T (32 keys x 32 queries): a
// lane then holds 16 scores of one query, its half wave's 16 of the 32 keys,
// so a row's maximum and sum stay in the lane but for one exchange between
// the halves, and S^T is, rounded, the right operand of O^T = V^T P^T as it
// stands: with i the register of a half h, the key is 8 (i / 4) + 4 h + i % 4,
// and the values are read in that order.  A half wave reads a value row side
// by side, dim / 32 neighbours a lane; eight rows' neighbours are regrouped
// in registers into the left operand.  Nothing goes through LDS before the
// four waves, which take every fourth key tile each, are joined.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "search.h"

namespace ert {

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef bf16x8 Vec;
  static __device__ __forceinline__ f32x16 mfma(const uint4& a, const uint4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  typedef __bf16 Value;
};
struct F16 {
  typedef f16x8 Vec;
  static __device__ __forceinline__ f32x16 mfma(const uint4& a, const uint4& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  typedef _Float16 Value;
};

constexpr float kNone = -__builtin_inff();

// n / d for n < 2^31.
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& d) {
  return (d.magic ? __umulhi(n, d.magic) : n) >> d.shift;
}

__device__ __forceinline__ float other_half(float x) { return __shfl_xor(x, 32); }

// A group's sequences.
__device__ __forceinline__ void group_range(const AttendParams& q, int g, int& s0, int& s1) {
  if (q.starts) {
    s0 = min(max(q.starts[g], 0), q.seqs);
    s1 = min(max(q.starts[g + 1], s0), q.seqs);
  } else {
    s0 = g * q.members;
    s1 = s0 + q.members;
  }
}

// The group and query tile of tile number `tile` among all groups', those of
// `cols` queries each; false if there are fewer.  Every lane of a wave takes
// part.
__device__ __forceinline__ bool find_tile(const AttendParams& q, int tile, int cols, int& group,
                                          int& first) {
  const int lane = threadIdx.x & 63, rows = q.next_n * q.per;
  int base = 0;
  for (int g0 = 0; g0 < q.groups; g0 += 64) {
    int n = 0;
    if (g0 + lane < q.groups) {
      int s0, s1;
      group_range(q, g0 + lane, s0, s1);
      n = (int)(((int64_t)(s1 - s0) * rows + cols - 1) / cols);
    }
    const int end = base + wave_scan(n);
    const uint64_t past = __ballot(end > tile);
    if (past) {
      const int at = __ffsll((unsigned long long)past) - 1;
      group = g0 + at;
      first = tile - __shfl(end - n, at);
      return true;
    }
    base = __shfl(end, 63);
  }
  return false;
}

// One workgroup's share: a range of keys of a table row against some queries.
struct Share {
  const int32_t* table;
  int len;        // positions of the table row that hold keys
  int begin, end; // keys of this share
  int head;       // key head
  int seq0;       // first sequence of the queries
  int rows;       // query rows of the entry
  int first;      // first query row of the tile
  int cut;        // rows see len - cut + token positions (0: len)
  int64_t slot;   // of the partial results
};

__device__ __forceinline__ int32_t block_at(const AttendParams& q, const Share& s, int width, int pos) {
  const uint32_t e = quotient((uint32_t)pos, q.by_block);
  const int32_t b = e < (uint32_t)width ? s.table[e] : -1;
  return b >= 0 && b < q.num_blocks ? b : -1;
}

}  // namespace

// ---------------------------------------------------------------------------
// One workgroup: a range of keys against 32 NT queries.
// ---------------------------------------------------------------------------
template <class T, int DIM, int NT>
__global__ void __launch_bounds__(kAttendBlock) attend_kernel(const AttendParams q) {
  constexpr int STEPS = DIM / 16;     // products of 16 deep a score tile
  constexpr int MT = DIM / 32;        // tiles of the output, values a lane loads of a row
  constexpr int WAVES = kAttendBlock / 64;
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  // what to do
  Share s;
  int width;
  {
    int64_t id = blockIdx.x;
    const bool shared = id < q.shared_wgs;
    int split;
    if (shared) {
      // tiles of one split and head follow each other on one of the eight dies
      const int64_t y = id >> 3;
      const int64_t strip = y / q.shared_tiles * 8 + (id & 7);
      if (strip >= (int64_t)q.shared_splits * q.kv_heads) return;
      split = (int)(strip / q.kv_heads);
      s.head = (int)(strip - (int64_t)split * q.kv_heads);
      int g, first;
      if (!find_tile(q, (int)(y % q.shared_tiles), 32 * NT, g, first)) return;
      g = __builtin_amdgcn_readfirstlane(g);
      first = __builtin_amdgcn_readfirstlane(first);
      int s1;
      group_range(q, g, s.seq0, s1);
      s.rows = (s1 - s.seq0) * q.next_n * q.per;
      s.first = first * 32 * NT;
      s.table = q.shared.tables + (int64_t)g * q.shared.stride;
      width = q.shared.width;
      s.len = min(max(q.shared.lens[g], 0), q.shared.limit);
      s.begin = split * q.shared_keys;
      s.end = s.begin + q.shared_keys;
      s.cut = 0;
      s.slot = (int64_t)split * q.rows;
    } else {
      id -= q.shared_wgs;
      const int tile = (int)(id % q.own_tiles);
      id /= q.own_tiles;
      s.head = (int)(id % q.kv_heads);
      id /= q.kv_heads;
      split = (int)(id % q.own_splits);
      s.seq0 = (int)(id / q.own_splits);
      s.rows = q.next_n * q.per;
      s.first = tile * 32 * NT;
      s.table = q.own.tables + (int64_t)s.seq0 * q.own.stride;
      width = q.own.width;
      s.len = min(max(q.own.lens[s.seq0], 0), q.own.limit);
      s.begin = split * q.own_keys;
      s.end = s.begin + q.own_keys;
      s.cut = q.next_n - 1;
      s.slot = (int64_t)(q.shared_splits + split) * q.rows;
    }
    if (s.begin >= s.len) return;
    s.end = min(s.end, s.len);
  }
  const int least = s.len - s.cut;    // positions that every query of the entry sees

  // the queries, as right operands
  uint4 query[NT][STEPS];
  int sees[NT];        // positions the lane's query sees
  int64_t out_row[NT]; // its row of the results, -1 none
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = s.first + n * 32 + col;
    const bool has = r < s.rows;
    const int rr = has ? r : 0;
    const int tok = rr / q.per, sub = rr - tok * q.per;
    const int64_t row = (int64_t)s.seq0 * q.next_n + tok;
    const int head = s.head * q.per + sub;
    out_row[n] = has ? row * q.heads + head : -1;
    sees[n] = least + (s.cut ? tok % q.next_n : 0);
    const unsigned char* p = q.q + row * q.q_stride + head * q.q_head_stride + half * 16;
#pragma unroll
    for (int d = 0; d < STEPS; ++d)
      query[n][d] = has ? *reinterpret_cast<const uint4*>(p + d * 32) : uint4{0, 0, 0, 0};
  }

  f32x16 acc[NT][MT];
  float top[NT], sum[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    top[n] = kNone;
    sum[n] = 0.0f;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[n][m][i] = 0.0f;
  }

  uint4 key[STEPS];
  uint32_t val[2][8][MT / 2];  // [group][row][two neighbours each]
  const int first_tile = s.begin + wv * kKeyTile;

  // keys: a lane reads its key's row, 16 bytes a product
  auto load_keys = [&](int p0) {
    const unsigned char* base = q.k.base + s.head * q.k.head_stride + half * 16;
    const int p = p0 + col;
    int32_t b = p < s.end ? block_at(q, s, width, p) : -1;
    const uint32_t off = (uint32_t)p - quotient((uint32_t)p, q.by_block) * (uint32_t)q.block_size;
    const unsigned char* a = base + (b >= 0 ? b * q.k.block_stride + off * q.k.slot_stride : 0);
#pragma unroll
    for (int d = 0; d < STEPS; ++d) key[d] = *reinterpret_cast<const uint4*>(a + d * 32);
    return b >= 0;
  };
  auto load_values = [&](int p0) {
    const unsigned char* base = q.v.base + s.head * q.v.head_stride + col * (MT * 2);
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int p = p0 + 16 * u + 8 * (e / 4) + 4 * half + e % 4;
        const int32_t b = p < s.end ? block_at(q, s, width, p) : -1;
        const uint32_t off = (uint32_t)p - quotient((uint32_t)p, q.by_block) * (uint32_t)q.block_size;
        const unsigned char* a = base + (b >= 0 ? b * q.v.block_stride + off * q.v.slot_stride : 0);
        if (b >= 0) {
          __builtin_memcpy(val[u][e], a, MT * 2);
        } else {
#pragma unroll
          for (int w = 0; w < MT / 2; ++w) val[u][e][w] = 0;
        }
      }
  };

  for (int p0 = first_tile; p0 < s.end; p0 += kAttendStep) {
    const bool there = load_keys(p0);
    load_values(p0);
    const uint64_t live = __ballot(there);
    const bool whole = live == ~0ull && p0 + kKeyTile <= least;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x16 sc;
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
#pragma unroll
      for (int d = 0; d < STEPS; ++d) sc = T::mfma(key[d], query[n][d], sc);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 8 * (i / 4) + 4 * half + i % 4;
          const bool on = (live >> j & 1) && p0 + j < sees[n];
          sc[i] = on ? sc[i] : kNone;
        }
      }
      float mx = sc[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
      mx = fmaxf(mx, other_half(mx)) * q.scale;
      // The weights' reference follows the largest score only once that is
      // over 2^8 times the reference's weight: weights of up to 2^8 lose
      // nothing, and sums are seldom scaled again.
      if (__ballot(mx > top[n] + 8.0f)) {
        const float now = fmaxf(mx, top[n]);
        const float f = now == kNone ? 0.0f : __builtin_amdgcn_exp2f(top[n] - now);
        top[n] = now;
        sum[n] *= f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[n][m][i] *= f;
      }
      const float ref = top[n] == kNone ? 0.0f : top[n];
      float part = 0.0f;
      typename T::Vec w[2];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], q.scale, -ref));
        part += p;
        w[i / 8][i % 8] = (typename T::Value)p;
      }
      sum[n] += part;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t a[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            a[e] = __builtin_amdgcn_perm(val[u][2 * e + 1][m / 2], val[u][2 * e][m / 2],
                                         m % 2 ? 0x07060302u : 0x05040100u);
          acc[n][m] = T::mfma(uint4{a[0], a[1], a[2], a[3]}, __builtin_bit_cast(uint4, w[u]), acc[n][m]);
        }
    }
  }

  // join the four waves
  __shared__ float lds_top[WAVES][NT * 32], lds_sum[WAVES][NT * 32];
  __shared__ float lds_acc[WAVES][16][64];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    sum[n] += other_half(sum[n]);
    if (half == 0) {
      lds_top[wv][n * 32 + col] = top[n];
      lds_sum[wv][n * 32 + col] = sum[n];
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float all = kNone, total = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) all = fmaxf(all, lds_top[w][n * 32 + col]);
    const float ref = all == kNone ? 0.0f : all;
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
      total += lds_sum[w][n * 32 + col] * __builtin_amdgcn_exp2f(lds_top[w][n * 32 + col] - ref);
    const float f = __builtin_amdgcn_exp2f(top[n] - ref);
    float res[4][MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 16; ++i) lds_acc[wv][i][lane] = acc[n][m][i] * f;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) v += lds_acc[w][4 * wv + i][lane];
        res[i][m] = v;
      }
    }
    if (out_row[n] >= 0) {
      const int64_t slot = s.slot + out_row[n];
      float* to = q.parts + slot * DIM + (8 * wv + 4 * half) * MT;
#pragma unroll
      for (int i = 0; i < 4 * MT; i += 4)
        *reinterpret_cast<float4*>(to + i) =
            float4{res[i / MT][i % MT], res[(i + 1) / MT][(i + 1) % MT], res[(i + 2) / MT][(i + 2) % MT],
                   res[(i + 3) / MT][(i + 3) % MT]};
      if (wv == 0 && half == 0) q.stats[slot] = float2{all, total};
    }
  }
}

// ---------------------------------------------------------------------------
// Joins a row's splits: dim / 4 threads a row.
// ---------------------------------------------------------------------------
template <class T, int DIM>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams q) {
  constexpr int LANES = DIM / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int d = (int)(threadIdx.x % LANES) * 4;
  if (row >= q.rows) return;
  const int seq = (int)(row / ((int64_t)q.next_n * q.heads));
  // live splits of both kinds
  int shared = 0;
  if (q.shared_splits > 0) {
    int g = -1;
    if (!q.starts) {
      g = seq / q.members;
    } else {
      int lo = 0, hi = q.groups;  // the last group that starts at or before seq
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.starts[mid] <= seq) lo = mid;
        else hi = mid;
      }
      int s0, s1;
      group_range(q, lo, s0, s1);
      if (seq >= s0 && seq < s1) g = lo;
    }
    if (g >= 0) {
      const int len = min(max(q.shared.lens[g], 0), q.shared.limit);
      shared = min((int)(((int64_t)len + q.shared_keys - 1) / q.shared_keys), q.shared_splits);
    }
  }
  const int len = min(max(q.own.lens[seq], 0), q.own.limit);
  const int own = min((int)(((int64_t)len + q.own_keys - 1) / q.own_keys), q.own_splits);
  const int n = shared + own;
  auto slot = [&](int i) {
    return (int64_t)(i < shared ? i : q.shared_splits + i - shared) * q.rows + row;
  };
  float top = kNone;
  for (int i = 0; i < n; ++i) top = fmaxf(top, q.stats[slot(i)].x);
  const float ref = top == kNone ? 0.0f : top;
  float total = 0.0f;
  float4 v{0.0f, 0.0f, 0.0f, 0.0f};
  for (int i = 0; i < n; ++i) {
    const float2 st = q.stats[slot(i)];
    const float f = __builtin_amdgcn_exp2f(st.x - ref);
    const float4 o = *reinterpret_cast<const float4*>(q.parts + slot(i) * DIM + d);
    total += st.y * f;
    v.x += o.x * f;
    v.y += o.y * f;
    v.z += o.z * f;
    v.w += o.w * f;
  }
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  typedef typename T::Value Value;
  Value* out = reinterpret_cast<Value*>(q.out) + row * DIM + d;
  Value r[4] = {(Value)(v.x * inv), (Value)(v.y * inv), (Value)(v.z * inv), (Value)(v.w * inv)};
  uint2 w;
  __builtin_memcpy(&w, r, 8);
  *reinterpret_cast<uint2*>(out) = w;
  if (q.lse && d == 0)
    q.lse[row] = total > 0.0f || total != total ? (top + __builtin_log2f(total)) * 0.69314718f : kNone;
}

// ---------------------------------------------------------------------------
// Attention mass: mass[h][p] = decay mass[h][p] + the weights of position p in
// every query of key head h.  A wave holds 32 keys and runs over the entry's
// queries, 32 at a time; each lane adds up its query column's weights, and the
// 32 columns are added at the end, so sums have one order.
// ---------------------------------------------------------------------------
template <class T, int DIM>
__global__ void __launch_bounds__(kAttendBlock) attend_mass_kernel(const MassParams mp) {
  constexpr int STEPS = DIM / 16;
  const AttendParams& q = mp.a;
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int64_t id = blockIdx.x;
  const bool shared = id < mp.shared_wgs;
  if (!shared) id -= mp.shared_wgs;
  const int tiles = shared ? mp.shared_tiles : mp.own_tiles;
  const int tile = (int)(id % tiles);
  id /= tiles;
  Share s;
  s.head = (int)(id % q.kv_heads);
  const int entry = (int)(id / q.kv_heads);
  const int row_len = shared ? mp.shared_width : mp.own_width;
  const PageTables& pt = shared ? q.shared : q.own;
  s.table = pt.tables + (int64_t)entry * pt.stride;
  s.len = min(max(pt.lens[entry], 0), pt.limit);
  if (shared) {
    int s1;
    group_range(q, entry, s.seq0, s1);
    s.rows = (s1 - s.seq0) * q.next_n * q.per;
    s.cut = 0;
  } else {
    s.seq0 = entry;
    s.rows = q.next_n * q.per;
    s.cut = q.next_n - 1;
  }
  const int p0 = (tile * (kAttendBlock / 64) + wv) * kKeyTile;
  if (p0 >= row_len) return;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  if (p0 < s.len) {
    uint4 key[STEPS];
    const int p = p0 + col;
    const int32_t b = p < s.len ? block_at(q, s, pt.width, p) : -1;
    const uint32_t off = (uint32_t)p - quotient((uint32_t)p, q.by_block) * (uint32_t)q.block_size;
    const unsigned char* a = q.k.base + s.head * q.k.head_stride + half * 16 +
                             (b >= 0 ? b * q.k.block_stride + off * q.k.slot_stride : 0);
#pragma unroll
    for (int d = 0; d < STEPS; ++d) key[d] = *reinterpret_cast<const uint4*>(a + d * 32);
    const uint64_t live = __ballot(b >= 0);
    for (int r0 = 0; r0 < s.rows; r0 += 32) {
      const int r = r0 + col;
      const bool has = r < s.rows;
      const int rr = has ? r : 0;
      const int tok = rr / q.per, sub = rr - tok * q.per;
      const int64_t row = (int64_t)s.seq0 * q.next_n + tok;
      const int head = s.head * q.per + sub;
      const unsigned char* at = q.q + row * q.q_stride + head * q.q_head_stride + half * 16;
      uint4 query[STEPS];
#pragma unroll
      for (int d = 0; d < STEPS; ++d) query[d] = *reinterpret_cast<const uint4*>(at + d * 32);
      // a row that saw nothing has a sum of nothing: its weights are none
      float lse = mp.lse[row * q.heads + head];
      const bool on = has && lse > kNone;
      lse = on ? lse * 1.44269504f : 0.0f;
      const int sees = s.len - s.cut + (s.cut ? tok % q.next_n : 0);
      f32x16 sc;
#pragma unroll
      for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
#pragma unroll
      for (int d = 0; d < STEPS; ++d) sc = T::mfma(key[d], query[d], sc);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int j = 8 * (i / 4) + 4 * half + i % 4;
        const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], q.scale, -lse));
        acc[i] += on && (live >> j & 1) && p0 + j < sees ? w : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) acc[i] += __shfl_xor(acc[i], d);
  }
  // lane j of the first 32 writes position j
  const int64_t base = ((int64_t)entry * q.kv_heads + s.head) * row_len + p0;
  const float* in = shared ? mp.shared_in : mp.own_in;
  float* out = shared ? mp.shared_out : mp.own_out;
  float mine = 0.0f;
  // position j = 8 (i / 4) + 4 h + i % 4 is held by half h: lane c of half h
  // takes register c % 16 if c < 16
#pragma unroll
  for (int i = 0; i < 16; ++i) mine = col == i ? acc[i] : mine;
  const int j = 8 * (col / 4) + 4 * half + col % 4;
  if (col < 16 && p0 + j < row_len) out[base + j] = (in ? in[base + j] * mp.decay : 0.0f) + mine;
}

namespace {

template <class T, int DIM>
const void* attend_ptr(int nt) {
  return nt == 1 ? reinterpret_cast<const void*>(&attend_kernel<T, DIM, 1>)
                 : reinterpret_cast<const void*>(&attend_kernel<T, DIM, 2>);
}

}  // namespace

const void* attend_kernel_ptr(int dtype, int dim, int nt) {
  if (dtype == 1) return dim == 64 ? attend_ptr<Bf16, 64>(nt) : attend_ptr<Bf16, 128>(nt);
  return dim == 64 ? attend_ptr<F16, 64>(nt) : attend_ptr<F16, 128>(nt);
}
const void* attend_join_kernel_ptr(int dtype, int dim) {
  if (dtype == 1)
    return dim == 64 ? reinterpret_cast<const void*>(&attend_join_kernel<Bf16, 64>)
                     : reinterpret_cast<const void*>(&attend_join_kernel<Bf16, 128>);
  return dim == 64 ? reinterpret_cast<const void*>(&attend_join_kernel<F16, 64>)
                   : reinterpret_cast<const void*>(&attend_join_kernel<F16, 128>);
}
const void* attend_mass_kernel_ptr(int dtype, int dim) {
  if (dtype == 1)
    return dim == 64 ? reinterpret_cast<const void*>(&attend_mass_kernel<Bf16, 64>)
                     : reinterpret_cast<const void*>(&attend_mass_kernel<Bf16, 128>);
  return dim == 64 ? reinterpret_cast<const void*>(&attend_mass_kernel<F16, 64>)
                   : reinterpret_cast<const void*>(&attend_mass_kernel<F16, 128>);
}

}  // namespace ert
