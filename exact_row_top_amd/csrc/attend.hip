// attend.hip -- decode attention over a paged cache for sequences that share
// a prefix, and the attention mass of cached positions.
//
// The queries of a group's sequences meet the group's prefix together: their
// rows (sequences x tokens x query heads of a key head) are the columns of one
// matrix product, so each key and value of the prefix is read once for up to
// 256 of them.  Each sequence's own positions follow in the same way by
// themselves.  Keys are split over workgroups, and a last launch joins the
// pieces of a row by their largest scores and sums.
//
// Layout.  Scores are made transposed, S^T = K Q^T (32 keys x 32 queries a
// wave): a lane then holds 16 scores of one query, its half wave's 16 of the 32
// keys, so a row's maximum and sum stay in the lane but for one exchange
// between the halves, and S^T is, rounded, the right operand of O^T = V^T P^T
// as it stands: register i of half h is key 8 (i / 4) + 4 h + i % 4, and the
// values are read from LDS in that order, four keys of one column a lane, by
// transposing reads.  Keys and values go through LDS in pieces of 16 bytes,
// swizzled so that both kinds of reads find all banks.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "search.h"

namespace ert {

namespace {

typedef uint32_t Piece __attribute__((ext_vector_type(4)));   // 16 bytes
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

struct Bf16 {
  typedef bf16x8 Vec;
  static __device__ __forceinline__ f32x16 mfma(const Piece& a, const Piece& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  typedef __bf16 Value;
};
struct F16 {
  typedef f16x8 Vec;
  static __device__ __forceinline__ f32x16 mfma(const Piece& a, const Piece& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  typedef _Float16 Value;
};

constexpr float kNone = -__builtin_inff();

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

// Sums over a wave's lanes up to each, and steps and strips of groups.
struct GroupScan {
  int steps, strips;      // of this lane's group
  int step_end, strip_end;
};

// Groups g0 .. g0 + 63, one a lane: a group has ceil(rows / cols) strips (query
// tiles) of ceil(len / keys) steps each, one strip behind the other.
__device__ __forceinline__ GroupScan scan_groups(const AttendParams& q, int g0, int cols, int keys,
                                                 int step0, int strip0) {
  const int g = g0 + (int)(threadIdx.x & 63);
  GroupScan s{0, 0, 0, 0};
  if (g < q.groups) {
    int s0, s1;
    group_range(q, g, s0, s1);
    s.strips = (int)(((int64_t)(s1 - s0) * q.next_n * q.per + cols - 1) / cols);
    const int len = min(max(q.shared.lens[g], 0), q.shared.limit);
    s.steps = s.strips * ((len + keys - 1) / keys);
  }
  s.step_end = step0 + wave_scan(s.steps);
  s.strip_end = strip0 + wave_scan(s.strips);
  return s;
}

// Steps that each workgroup of a key head takes of `all`.
__device__ __forceinline__ int share_of(const AttendParams& q, int all) {
  return max((all + q.shared_wgs - 1) / q.shared_wgs, q.shared_least);
}

// A range of keys of a table row against some queries.
struct Share {
  const int32_t* table;
  int width;
  int len;          // positions of the table row that hold keys
  int step0, step1; // the range in steps
  int head;         // key head
  int seq0;         // first sequence of the entry's queries
  int rows;         // query rows of the entry
  int first;        // first query row of the tile
  int cut;          // rows see len - cut + token positions (0: len)
};

__device__ __forceinline__ int32_t block_at(const AttendParams& q, const int32_t* table, int width, int pos) {
  const uint32_t e = q.by_block((uint32_t)pos);
  const int32_t b = e < (uint32_t)width ? table[e] : -1;
  return b < q.num_blocks ? b : -1;
}

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

// Where the 16-byte piece `piece` of row `row` lies in its row in LDS.  Keys:
// 16 lanes read one piece of 16 rows; values: 32 lanes read 64 bytes each of
// four rows.
template <int DIM>
__device__ __forceinline__ int key_piece(int row, int piece) {
  return DIM == 128 ? piece ^ (row & 15) : piece ^ ((row >> 1) & 7);
}
template <int DIM>
__device__ __forceinline__ int value_piece(int row, int piece) {
  return DIM == 128 ? piece ^ ((row & 3) << 2) : piece ^ (((row >> 1) & 1) << 2);
}

}  // namespace

// ---------------------------------------------------------------------------
// QW waves of 32 queries each share the keys and values of a step (KT of
// them); KW such sets take turns at the steps, and are joined at the end.
//
// A step's keys and values are on their way to registers while the step
// before is computed, and its block numbers one step ahead of that.
//
// Shared positions: the steps of all strips form one line, of which every
// workgroup of a key head takes an equal share, whatever the lengths; pieces
// of a strip are told apart by workgroup + strip, which no two pieces have in
// common.
// ---------------------------------------------------------------------------
template <class T, int DIM, int QW, int KW, int KT>
__global__ void __launch_bounds__(64 * QW * KW, QW == 1 ? 1 : 2) attend_kernel(const AttendParams q) {
  constexpr int STEPS = DIM / 16;          // products of 16 deep a score tile
  constexpr int MT = DIM / 32;             // tiles of the output
  constexpr int PIECES = DIM / 8;          // 16-byte pieces of a row
  constexpr int ROWS = 64 * QW / PIECES;   // rows that a set's threads load at once
  constexpr int PASSES = KT / ROWS;
  constexpr int BUFFERS = QW == 1 ? 1 : 2; // a wave alone reads what it wrote
  static_assert(KT % ROWS == 0 && (QW == 1 || KW == 1), "");
  struct Stage {
    Piece key[KT * PIECES];
    Piece value[KT * PIECES];
  };
  __shared__ Stage stages[KW][BUFFERS];
  __shared__ int32_t valid[KW][BUFFERS][KT];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = wave / QW, qw = wave % QW;
  const int lt = (int)threadIdx.x - set * QW * 64;
  const int lrow = lt / PIECES, lpiece = lt % PIECES;

  auto run = [&](const Share& s, float* parts, float2* stats) {
    const int least = s.len - s.cut;    // positions that every query of the entry sees
    // this wave's queries, as right operands
    Piece query[STEPS];
    const int r = s.first + qw * 32 + col;
    const bool has = r < s.rows;
    int sees;
    {
      const int rr = has ? r : 0;
      const int tok = rr / q.per, sub = rr - tok * q.per;
      sees = least + (s.cut ? tok % q.next_n : 0);
      const unsigned char* p = q.q + ((int64_t)s.seq0 * q.next_n + tok) * q.q_stride +
                               (s.head * q.per + sub) * q.q_head_stride + half * 16;
#pragma unroll
      for (int d = 0; d < STEPS; ++d)
        query[d] = has ? *reinterpret_cast<const Piece*>(p + d * 32) : Piece{0, 0, 0, 0};
    }
    f32x16 acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][i] = 0.0f;
    float top = kNone, sum = 0.0f;

    const unsigned char* kbase = q.k.base + s.head * q.k.head_stride + lpiece * 16;
    const unsigned char* vbase = q.v.base + s.head * q.v.head_stride + lpiece * 16;
    Piece kreg[PASSES], vreg[PASSES];
    int32_t block[PASSES];   // table entries of the step to be loaded next
    uint32_t live_row[PASSES];  // all ones where a position is there, else zero
    // (no branches around these loads: each would be waited for in its own)
    auto find = [&](int t) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const uint32_t p = (uint32_t)min(t * KT + i * ROWS + lrow, s.len - 1);
        block[i] = s.table[min(q.by_block(p), (uint32_t)s.width - 1u)];
      }
    };
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const uint32_t p = (uint32_t)(t * KT + i * ROWS + lrow);
        live_row[i] = p < (uint32_t)s.len && (uint32_t)block[i] < (uint32_t)q.num_blocks ? ~0u : 0u;
        // what is not there is read from the cache's first slot, and masked
        const uint32_t off = (p - q.by_block(p) * (uint32_t)q.block_size) & live_row[i];
        const uint32_t blk = (uint32_t)block[i] & live_row[i];
        kreg[i] = *reinterpret_cast<const Piece*>(kbase + (int64_t)blk * q.k.block_stride + (int64_t)off * q.k.slot_stride);
        vreg[i] = *reinterpret_cast<const Piece*>(vbase + (int64_t)blk * q.v.block_stride + (int64_t)off * q.v.slot_stride);
      }
    };

    int t = s.step0 + set, b = 0;
    find(t);
    fetch(t);
    find(t + KW);
    for (; t < s.step1; t += KW, b ^= BUFFERS - 1) {
      Stage& st = stages[set][b];
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int row = i * ROWS + lrow;
        st.key[row * PIECES + key_piece<DIM>(row, lpiece)] = kreg[i];
        // values that no weight counts must not be NaN or infinite
        st.value[row * PIECES + value_piece<DIM>(row, lpiece)] =
            vreg[i] & live_row[i];
        if (lpiece == 0) valid[set][b][row] = (int32_t)live_row[i];
      }
      fetch(t + KW);
      find(t + 2 * KW);
      if (QW > 1) {
        // the writes are done; what is on its way to registers need not be
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
      } else {
        wave_sync();
      }
      const uint64_t live = __ballot(valid[set][b][lane % KT] != 0);
      const bool whole = live == ~0ull && (t + 1) * KT <= least;
#pragma unroll 1
      for (int k0 = 0; k0 < KT; k0 += kKeyTile) {
        f32x16 sc;
#pragma unroll
        for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
#pragma unroll
        for (int d = 0; d < STEPS; ++d)
          sc = T::mfma(st.key[(k0 + col) * PIECES + key_piece<DIM>(col, 2 * d + half)], query[d], sc);
        if (!whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int j = k0 + 8 * (i / 4) + 4 * half + i % 4;
            sc[i] = (live >> j & 1) && t * KT + j < sees ? sc[i] : kNone;
          }
        }
        float mx = sc[0];
#pragma unroll
        for (int i = 1; i < 16; ++i) mx = fmaxf(mx, sc[i]);
        mx = fmaxf(mx, other_half(mx)) * q.scale;
        // The weights' reference follows the largest score only once that is
        // over 2^8 times the reference's weight: weights of up to 2^8 lose
        // nothing, and sums are seldom scaled again.
        if (__ballot(mx > top + 8.0f)) {
          const float now = fmaxf(mx, top);
          const float f = now == kNone ? 0.0f : __builtin_amdgcn_exp2f(top - now);
          top = now;
          sum *= f;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][i] *= f;
        }
        const float ref = top == kNone ? 0.0f : top;
        float part = 0.0f;
        typename T::Vec w[2];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i], q.scale, -ref));
          part += p;
          w[i / 8][i % 8] = (typename T::Value)p;
        }
        sum += part;
        // four keys of a column a read: lane l gives the address of row l % 16
        // / 4, columns 4 (l % 4) on, of its 16 lanes' columns
        const int vrow = k0 + 4 * half + ((lane & 15) >> 2);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            s16x4 a[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int row = vrow + 16 * u + 8 * e;
              const int piece = value_piece<DIM>((lane & 15) >> 2, 4 * m + 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1));
              a[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                  (__attribute__((address_space(3))) s16x4*)(reinterpret_cast<unsigned char*>(&st.value[row * PIECES + piece]) + 8 * (lane & 1)));
            }
            const s16x8 left = __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc[m] = T::mfma(__builtin_bit_cast(Piece, left), __builtin_bit_cast(Piece, w[u]), acc[m]);
          }
      }
      if (QW == 1) wave_sync();
    }

    sum += other_half(sum);
    if (KW == 1) {
      if (has) {
        float* to = parts + (int64_t)(qw * 32 + col) * DIM + 4 * half;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(to + 32 * m + 2 * i) =
                float4{acc[m][i], acc[m][i + 1], acc[m][i + 2], acc[m][i + 3]};
        if (half == 0) stats[qw * 32 + col] = float2{top, sum};
      }
      __syncthreads();   // before the next piece's first step is written
      return;
    }
    // join the sets' waves: each adds up a quarter of the registers
    __shared__ float lds_top[KW][32], lds_sum[KW][32];
    float (*lds_acc)[16][64] = reinterpret_cast<float (*)[16][64]>(&stages[0][0]);
    static_assert(KW == 1 || (KW == 4 && sizeof(stages) >= sizeof(float) * KW * 16 * 64), "");
    if (half == 0) {
      lds_top[set][col] = top;
      lds_sum[set][col] = sum;
    }
    __syncthreads();
    float all = kNone, total = 0.0f;
#pragma unroll
    for (int w = 0; w < KW; ++w) all = fmaxf(all, lds_top[w][col]);
    const float ref = all == kNone ? 0.0f : all;
#pragma unroll
    for (int w = 0; w < KW; ++w) total += lds_sum[w][col] * __builtin_amdgcn_exp2f(lds_top[w][col] - ref);
    const float f = __builtin_amdgcn_exp2f(top - ref);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < 16; ++i) lds_acc[set][i][lane] = acc[m][i] * f;
      __syncthreads();
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < KW; ++w)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += lds_acc[w][4 * set + i][lane];
      if (has)
        *reinterpret_cast<float4*>(parts + (int64_t)col * DIM + 32 * m + 8 * set + 4 * half) =
            float4{v[0], v[1], v[2], v[3]};
      __syncthreads();
    }
    if (has && set == 0 && half == 0) stats[col] = float2{all, total};
  };

  Share s;
  if (blockIdx.x < q.shared_grid) {
    const int wg = (int)(blockIdx.x / (uint32_t)q.kv_heads);
    s.head = (int)(blockIdx.x - (uint32_t)wg * (uint32_t)q.kv_heads);
    s.cut = 0;
    s.width = q.shared.width;
    int all = 0, strips = 0;
    for (int g0 = 0; g0 < q.groups; g0 += 64) {
      const GroupScan c = scan_groups(q, g0, 32 * QW, KT, all, strips);
      if (blockIdx.x == 0 && threadIdx.x < 64 && g0 + (int)threadIdx.x < q.groups)
        q.group_at[g0 + threadIdx.x] = int4{c.step_end - c.steps, c.strip_end - c.strips, 0, 0};
      all = __builtin_amdgcn_readlane(c.step_end, 63);
      strips = __builtin_amdgcn_readlane(c.strip_end, 63);
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) q.group_at[q.groups] = int4{all, strips, 0, 0};
    // (more strips than rising starts can have: the shared positions are left out)
    if (strips > q.strips) return;
    const int share = share_of(q, all);
    const int64_t from = (int64_t)wg * share;
    const int to = (int)min(from + share, (int64_t)all);
    for (int64_t at = from; at < to;) {
      // the strip that step `at` lies in
      int step0 = 0, strip0 = 0, g = 0;
      for (int g0 = 0; g0 < q.groups; g0 += 64) {
        const GroupScan c = scan_groups(q, g0, 32 * QW, KT, step0, strip0);
        const uint64_t past = __ballot(c.step_end > (int)at);
        if (past) {
          const int l = __ffsll((unsigned long long)past) - 1;
          g = g0 + l;
          step0 = __builtin_amdgcn_readlane(c.step_end - c.steps, l);
          strip0 = __builtin_amdgcn_readlane(c.strip_end - c.strips, l);
          break;
        }
        step0 = __builtin_amdgcn_readlane(c.step_end, 63);
        strip0 = __builtin_amdgcn_readlane(c.strip_end, 63);
      }
      int s1;
      group_range(q, g, s.seq0, s1);
      s.rows = (s1 - s.seq0) * q.next_n * q.per;
      s.table = q.shared.tables + (int64_t)g * q.shared.stride;
      s.len = min(max(q.shared.lens[g], 0), q.shared.limit);
      const int steps = (s.len + KT - 1) / KT;       // of a strip: not 0 where `at` lies in one
      const int tile = ((int)at - step0) / steps;
      s.first = tile * 32 * QW;
      s.step0 = (int)at - step0 - tile * steps;
      s.step1 = min(steps, s.step0 + to - (int)at);
      const int64_t slot = ((int64_t)s.head * (q.shared_wgs + q.strips) + wg + strip0 + tile) * 32 * QW;
      run(s, q.shared_parts + slot * DIM, q.shared_stats + slot);
      at += s.step1 - s.step0;
    }
    return;
  }
  if (QW > 1) return;
  int64_t id = (int64_t)blockIdx.x - q.shared_grid;
  s.head = (int)(id % q.kv_heads);
  id /= q.kv_heads;
  const int tile = (int)(id % q.own_tiles);
  id /= q.own_tiles;
  const int split = (int)(id % q.own_splits);
  s.seq0 = (int)(id / q.own_splits);
  s.rows = q.next_n * q.per;
  s.first = tile * 32;
  s.table = q.own.tables + (int64_t)s.seq0 * q.own.stride;
  s.width = q.own.width;
  s.len = min(max(q.own.lens[s.seq0], 0), q.own.limit);
  s.cut = q.next_n - 1;
  const int steps = (s.len + KT - 1) / KT;
  const int share = max((steps + q.own_splits - 1) / q.own_splits, KW);
  if ((int64_t)split * share >= steps) return;
  s.step0 = split * share;
  s.step1 = min(steps, s.step0 + share);
  const int64_t slot = (((int64_t)split * q.seqs + s.seq0) * q.kv_heads + s.head) * s.rows + s.first;
  run(s, q.own_parts + slot * DIM, q.own_stats + slot);
}

// ---------------------------------------------------------------------------
// Joins a row's pieces: dim / 4 threads a row.
// ---------------------------------------------------------------------------
template <class T, int DIM>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams q) {
  constexpr int LANES = DIM / 4;
  const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int d = (int)(threadIdx.x % LANES) * 4;
  if (row >= q.rows) return;
  const int tok = (int)(row / q.heads), head = (int)(row - (int64_t)tok * q.heads);
  const int seq = tok / q.next_n, kv = head / q.per, sub = head - kv * q.per;
  // the pieces of the shared positions: consecutive slots
  int shared = 0;
  int64_t shared_slot = 0;
  if (q.shared_wgs > 0) {
    int g = -1, s0 = 0, s1;
    if (!q.starts) {
      g = seq / q.members;
      group_range(q, g, s0, s1);
    } else {
      int lo = 0, hi = q.groups;  // the last group that starts at or before seq
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q.starts[mid] <= seq) lo = mid;
        else hi = mid;
      }
      group_range(q, lo, s0, s1);
      if (seq >= s0 && seq < s1) g = lo;
    }
    const int steps = g < 0 ? 0 : (min(max(q.shared.lens[g], 0), q.shared.limit) + q.shared_tile - 1) / q.shared_tile;
    if (steps > 0 && q.group_at[q.groups].y <= q.strips) {
      const int cols = 32 * q.query_waves;
      const int r = (tok - s0 * q.next_n) * q.per + sub, tile = r / cols;
      const int4 at = q.group_at[g];
      const int share = share_of(q, q.group_at[q.groups].x);
      const int a = at.x + tile * steps, first = a / share;
      shared = (a + steps - 1) / share - first + 1;
      shared_slot = ((int64_t)kv * (q.shared_wgs + q.strips) + first + at.y + tile) * cols + (r - tile * cols);
    }
  }
  const int own_rows = q.next_n * q.per;
  const int steps = (min(max(q.own.lens[seq], 0), q.own.limit) + kKeyTile - 1) / kKeyTile;
  const int share = q.own_splits > 0 ? max((steps + q.own_splits - 1) / q.own_splits, kOwnSets) : 1;
  const int own = q.own_splits > 0 ? (steps + share - 1) / share : 0;
  const int64_t own_slot = ((int64_t)seq * q.kv_heads + kv) * own_rows + (tok - seq * q.next_n) * q.per + sub;
  const int64_t own_stride = (int64_t)q.seqs * q.kv_heads * own_rows;

  float top = kNone, total = 0.0f;
  float4 v{0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const float2 st, const float4 o) {
    const float now = fmaxf(top, st.x), ref = now == kNone ? 0.0f : now;
    const float f = __builtin_amdgcn_exp2f(top - ref), g = __builtin_amdgcn_exp2f(st.x - ref);
    top = now;
    total = total * f + st.y * g;
    v.x = v.x * f + o.x * g;
    v.y = v.y * f + o.y * g;
    v.z = v.z * f + o.z * g;
    v.w = v.w * f + o.w * g;
  };
  for (int i = 0; i < shared; ++i) {
    const int64_t s = shared_slot + (int64_t)i * 32 * q.query_waves;
    add(q.shared_stats[s], *reinterpret_cast<const float4*>(q.shared_parts + s * DIM + d));
  }
  for (int i = 0; i < own; ++i) {
    const int64_t s = own_slot + i * own_stride;
    add(q.own_stats[s], *reinterpret_cast<const float4*>(q.own_parts + s * DIM + d));
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
__global__ void __launch_bounds__(kMassBlock) attend_mass_kernel(const MassParams mp) {
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
  const int p0 = (tile * (kMassBlock / 64) + wv) * kKeyTile;
  if (p0 >= row_len) return;
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
  if (p0 < s.len) {
    Piece key[STEPS];
    const int p = p0 + col;
    const int32_t b = p < s.len ? block_at(q, s.table, pt.width, p) : -1;
    const uint32_t off = (uint32_t)p - q.by_block((uint32_t)p) * (uint32_t)q.block_size;
    const unsigned char* a = q.k.base + s.head * q.k.head_stride + half * 16 +
                             (b >= 0 ? b * q.k.block_stride + off * q.k.slot_stride : 0);
#pragma unroll
    for (int d = 0; d < STEPS; ++d) key[d] = *reinterpret_cast<const Piece*>(a + d * 32);
    const uint64_t live = __ballot(b >= 0);
    for (int r0 = 0; r0 < s.rows; r0 += 32) {
      const int r = r0 + col;
      const bool has = r < s.rows;
      const int rr = has ? r : 0;
      const int tok = rr / q.per, sub = rr - tok * q.per;
      const int64_t row = (int64_t)s.seq0 * q.next_n + tok;
      const int head = s.head * q.per + sub;
      const unsigned char* at = q.q + row * q.q_stride + head * q.q_head_stride + half * 16;
      Piece query[STEPS];
#pragma unroll
      for (int d = 0; d < STEPS; ++d) query[d] = *reinterpret_cast<const Piece*>(at + d * 32);
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
const void* attend_ptr(int query_waves) {
  switch (query_waves) {
    case 8: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 8, 1, 64>);
    case 4: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 4, 1, 32>);
    case 2: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 2, 1, 32>);
    default: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 1, kOwnSets, kKeyTile>);
  }
}

}  // namespace

const void* attend_kernel_ptr(int dtype, int dim, int query_waves) {
  if (dtype == 1) return dim == 64 ? attend_ptr<Bf16, 64>(query_waves) : attend_ptr<Bf16, 128>(query_waves);
  return dim == 64 ? attend_ptr<F16, 64>(query_waves) : attend_ptr<F16, 128>(query_waves);
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
