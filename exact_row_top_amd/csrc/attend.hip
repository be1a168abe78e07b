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

#include <type_traits>

#include "search.h"

namespace ert {

namespace {

typedef uint32_t Piece __attribute__((ext_vector_type(4)));   // 16 bytes
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// kLift: the largest weights lie 2^kLift above 1 in the second product.  float16
// loses bits below 2^-14 and everything below 2^-25: with it, below 2^-21 and
// 2^-32 of the largest.  (With the 2^8 that the reference may lag, 2^15 at most.)
struct Bf16 {
  typedef bf16x8 Vec;
  static constexpr float kLift = 0.0f;
  static __device__ __forceinline__ f32x16 mfma(const Piece& a, const Piece& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
  typedef __bf16 Value;
};
struct F16 {
  typedef f16x8 Vec;
  static constexpr float kLift = 7.0f;
  static __device__ __forceinline__ f32x16 mfma(const Piece& a, const Piece& b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
  typedef _Float16 Value;
};

constexpr float kNone = -__builtin_inff();

// The two halves' values of a lane and its counterpart.
struct Pair {
  float a, b;
};
__device__ __forceinline__ Pair both_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return Pair{__uint_as_float(r[0]), __uint_as_float(r[1])};
}

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

namespace {

// 16 bytes a lane from memory into 1 KB of LDS from `to` on (uniform), lane by
// lane.  Written out so that reads of another part of LDS do not wait for it:
// whoever reads waits for vmcnt first.  m0, which holds where in LDS, is an
// operand, so that the compiler knows what is in it.
__device__ __forceinline__ void load_to_lds(const unsigned char* from, const Piece* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const Piece*)to);
  asm volatile(
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "{m0}"(at), "v"(from)
      : "memory");
}
// The same from a uniform base and a lane's own offset.  The base may come
// straight from v_readlane: a memory instruction that reads a scalar register
// which a vector instruction wrote needs five wait states between them, and the
// compiler puts none before inline assembly.
__device__ __forceinline__ void load_to_lds(const unsigned char* base, uint32_t lane_off, const Piece* to) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const Piece*)to);
  asm volatile(
      "s_nop 4\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "{m0}"(at), "v"(lane_off), "s"(base)
      : "memory");
}
// Waits until all but the last N loads are done.
template <int N>
__device__ __forceinline__ void loads_but() {
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}
// Waits for this wave's LDS reads and writes.
__device__ __forceinline__ void lds_done() { asm volatile("s_waitcnt lgkmcnt(0)" : : : "memory"); }
// A workgroup's LDS writes, and nothing on its way to LDS or registers.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

}  // namespace

// ---------------------------------------------------------------------------
// QW waves of 32 queries each share the keys and values of a step (KT of
// them); KW such sets take turns at the steps, and are joined at the end.
//
// Steps go straight from memory to LDS.  With QW > 1 one is on its way while
// the one before is computed; of eight waves, the second on each SIMD runs
// half a step behind the first, so that one's products meet the other's
// exponentials.  A wave alone (QW 1) has one buffer: the next step's keys are
// fetched once the products with this one's are done, and its values likewise.
//
// Shared positions: the steps of all strips form one line, of which every
// workgroup of a key head takes an equal share, whatever the lengths; pieces
// of a strip are told apart by workgroup + strip, which no two pieces have in
// common.
//
// Bound, with eight waves, by the matrix products and the LDS reads that feed
// them, which take about as long: 2 groups of 256 queries a key head (8 of them,
// dim 128) over some 24 thousand positions each, 51 GFLOP, take 84 us, 610
// TFLOP/s, of them about 20 for the first loads and the 33 MB of pieces.
// Bound, alone (QW 1), by memory and the waits for it: 64 sequences' own 1 to
// 512 positions, 67 MB, take 22 us (3.1 TB/s, the longest sequences last); four
// queries' 1000 positions take 8, the launch and the waits for lengths, tables,
// keys, values and the join of the four sets.
// ---------------------------------------------------------------------------
template <class T, int DIM, int QW, int KW, int KT, bool EVEN>
__global__ void __launch_bounds__(64 * QW * KW, 2) attend_kernel(const AttendParams q) {
  constexpr int STEPS = DIM / 16;          // products of 16 deep a score tile
  constexpr int MT = DIM / 32;             // tiles of the output
  constexpr int SUBS = KT / kKeyTile;      // score tiles of a step
  constexpr int PIECES = DIM / 8;          // 16-byte pieces of a row
  constexpr int ROWS = 64 / PIECES;        // rows that a wave loads at once
  constexpr int PASSES = KT / (ROWS * QW);
  constexpr bool LAG = QW == 8;
  constexpr int BUFFERS = QW == 1 ? 1 : (LAG ? 3 : 2);
  static_assert(PASSES * ROWS * QW == KT && (PASSES & (PASSES - 1)) == 0 && (QW == 1 || KW == 1), "");
  struct Stage {
    Piece key[KT * PIECES];
    Piece value[KT * PIECES];
  };
  __shared__ Stage stages[KW][BUFFERS];
  __shared__ int32_t valid[KW][BUFFERS][KT];

  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int set = wave / QW, qw = wave % QW;
  const int lrow = lane / PIECES, lpiece = lane % PIECES;
  const bool lag = LAG && qw >= QW / 2;

  auto run = [&](const Share& s, float* parts, float2* stats) {
    const int least = s.len - s.cut;    // positions that every query of the entry sees
    // Steps that the waves load: pass i of wave qw is rows row0(i) on.  EVEN:
    // blocks hold whole passes, so that a pass lies in one block; lane i < PASSES
    // makes the address of pass i's keys, lane i + PASSES that of its values.
    const unsigned char* kbase = q.k.base + s.head * q.k.head_stride;
    const unsigned char* vbase = q.v.base + s.head * q.v.head_stride;
    auto row0 = [&](int i) { return (i * QW + qw) * ROWS; };
    auto entry = [&](int p) {
      return s.table[min(q.by_block((uint32_t)min(p, s.len - 1)), (uint32_t)s.width - 1u)];
    };
    const bool for_values = lane & PASSES;
    const uint32_t my_block_stride = for_values ? q.v.block_stride : q.k.block_stride;
    const uint32_t my_slot_stride = for_values ? q.v.slot_stride : q.k.slot_stride;
    const uint64_t my_base = (uint64_t)(for_values ? vbase : kbase);
    int32_t ids = 0;     // table entries of the step to be fetched next
    uint64_t from = 0;   // where its passes lie
    auto find = [&](int t) {
      if (EVEN) ids = entry(t * KT + row0(lane % PASSES));
    };
    // What is not there is read from the cache's first slot, and masked.
    auto locate = [&](int t) {
      if (!EVEN) return;
      const uint32_t p = (uint32_t)(t * KT + row0(lane % PASSES));
      const uint32_t ok = p < (uint32_t)s.len && (uint32_t)ids < (uint32_t)q.num_blocks ? ~0u : 0u;
      const uint32_t off = (p - q.by_block(p) * (uint32_t)q.block_size) & ok;
      from = my_base + (uint64_t)((uint32_t)ids & ok) * my_block_stride + (uint64_t)off * my_slot_stride;
    };
    auto fetch = [&](int t, int b, bool keys) {
      const Pages& c = keys ? q.k : q.v;
      Piece* to = keys ? stages[set][b].key : stages[set][b].value;
      int r = lrow, x = lpiece;
      asm("" : "+v"(r), "+v"(x));   // (offsets of all passes would fill the registers)
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        const int row = row0(i) + r;
        const uint32_t piece = (uint32_t)(keys ? key_piece<DIM>(row, x) : value_piece<DIM>(row, x)) * 16;
        Piece* at = to + (i * QW + qw) * 64;
        if (EVEN) {
          const int l = keys ? i : i + PASSES;
          const uint64_t base = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(from >> 32), l) << 32 |
                                (uint32_t)__builtin_amdgcn_readlane((int)from, l);
          load_to_lds(reinterpret_cast<const unsigned char*>(base), (uint32_t)r * c.slot_stride + piece, at);
        } else {
          const uint32_t p = (uint32_t)(t * KT + row), id = (uint32_t)entry((int)p);
          const uint32_t ok = p < (uint32_t)s.len && id < (uint32_t)q.num_blocks ? ~0u : 0u;
          load_to_lds((keys ? kbase : vbase) + (uint64_t)(id & ok) * c.block_stride +
                          (uint64_t)((p - q.by_block(p) * (uint32_t)q.block_size) & ok) * c.slot_stride + piece,
                      at);
        }
      }
    };
    // Steps before `full` hold KT positions that are there, those before `seen`
    // no position that a query of the entry does not see.
    int full = 0, seen = 0;
    // For a step that lacks rows: marks them, and, once it has arrived, clears
    // their values, which must not be NaN or infinite even without a weight.
    auto mark = [&](int t, int b) {
      for (int r = lane; r < KT; r += 64) {
        const int p = t * KT + r;
        valid[set][b][r] = p < s.len && (uint32_t)entry(p) < (uint32_t)q.num_blocks ? 1 : 0;
      }
      wave_sync();
    };
    auto clear = [&](int b) {
#pragma unroll 1
      for (int i = 0; i < PASSES; ++i) {
        const int row = row0(i) + lrow;
        if (!valid[set][b][row]) stages[set][b].value[row * PIECES + lpiece] = Piece{0, 0, 0, 0};
      }
      wave_sync();
    };

    // A step's own part has arrived.
    auto settle = [&](int t, int b) {
      loads_but<0>();
      if (t >= full) {
        mark(t, b);   // (each wave all of them, the same)
        clear(b);
      }
    };

    int t = s.step0 + set;
    find(t);
    bool clean = true;   // every block of this share is there
    {
      const uint32_t e1 = min(q.by_block((uint32_t)min(s.step1 * KT, s.len) - 1u) + 1u, (uint32_t)s.width);
      for (uint32_t e = q.by_block((uint32_t)(s.step0 * KT)) + threadIdx.x; e < e1; e += 64 * QW * KW)
        clean = clean && (uint32_t)s.table[e] < (uint32_t)q.num_blocks;
    }
    if (t < s.step1) {
      locate(t);
      fetch(t, 0, true);
      fetch(t, 0, false);
      find(t + KW);
    }
    // this wave's queries, as right operands
    Piece query[STEPS];
    const int r = s.first + qw * 32 + col;
    const bool has = r < s.rows;
    int sees;
    {
      const int rr = has ? r : 0;
      const int tok = (int)((uint32_t)rr / (uint32_t)q.per), sub = rr - tok * q.per;
      sees = least + (s.cut ? tok % q.next_n : 0);
      const unsigned char* p = q.q + ((int64_t)s.seq0 * q.next_n + tok) * q.q_stride +
                               (s.head * q.per + sub) * q.q_head_stride + half * 16;
#pragma unroll
      for (int d = 0; d < STEPS; ++d) {
        query[d] = *reinterpret_cast<const Piece*>(p + d * 32);
        if (!has) query[d] = Piece{0, 0, 0, 0};
      }
    }
    if (__syncthreads_and(clean)) {
      full = s.len / KT;
      seen = max(least, 0) / KT;
    }

    f32x16 acc[MT], sc[SUBS];
    typename T::Vec w[2 * SUBS];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[m][i] = 0.0f;
    float top = kNone, sum = 0.0f;
    bool far = false;   // some query's reference lies beyond 2^16

    // Matrix products: the scores of the step in buffer bk (QK) and the values
    // of the one in buffer bv times its weights (PV), in turn; LDS reads run
    // AHEAD steps of either before their products.
    auto multiply = [&](auto qk, auto pv, int bk, int bv) {
      constexpr bool QK = decltype(qk)::value, PV = decltype(pv)::value;
      constexpr int AHEAD = PV ? 2 : 4, VALUES = 2 * SUBS * MT, VAHEAD = 4;
      // (made anew in every step: kept, these addresses fill the registers)
      int kcol = col, vlane = lane;
      asm("" : "+v"(kcol), "+v"(vlane));
      auto key = [&](int d, int n) {
        return stages[set][bk].key[(n * kKeyTile + kcol) * PIECES + key_piece<DIM>(kcol, 2 * d + half)];
      };
      // four keys of a column a read: lane l gives the address of row l % 16 /
      // 4, columns 4 (l % 4) on, of its 16 lanes' columns
      auto value = [&](int j) {
        const int row = 16 * (j / MT) + 4 * half + ((vlane & 15) >> 2);
        const int piece = value_piece<DIM>((vlane & 15) >> 2, 4 * (j % MT) + 2 * ((vlane >> 4) & 1) + ((vlane & 3) >> 1));
        s16x4 a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          a[e] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
              (__attribute__((address_space(3))) s16x4*)(reinterpret_cast<unsigned char*>(&stages[set][bv].value[(row + 8 * e) * PIECES + piece]) + 8 * (vlane & 1)));
        return __builtin_bit_cast(Piece, __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7));
      };
      Piece keys[AHEAD][SUBS], values[VAHEAD];
      if (QK) {
#pragma unroll
        for (int d = 0; d < AHEAD; ++d)
#pragma unroll
          for (int n = 0; n < SUBS; ++n) keys[d][n] = key(d, n);
#pragma unroll
        for (int n = 0; n < SUBS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[n][i] = 0.0f;
      }
      if (PV) {
#pragma unroll
        for (int j = 0; j < VAHEAD; ++j) values[j] = value(j);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < STEPS; ++d) {
        if (QK) {
#pragma unroll
          for (int n = 0; n < SUBS; ++n) {
            sc[n] = T::mfma(keys[d % AHEAD][n], query[d], sc[n]);
            if (d + AHEAD < STEPS) keys[d % AHEAD][n] = key(d + AHEAD, n);
          }
        }
        if (PV) {
#pragma unroll
          for (int j = d * VALUES / STEPS; j < (d + 1) * VALUES / STEPS; ++j) {
            acc[j % MT] = T::mfma(values[j % VAHEAD], __builtin_bit_cast(Piece, w[j / MT]), acc[j % MT]);
            if (j + VAHEAD < VALUES) values[j % VAHEAD] = value(j + VAHEAD);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};

    // From a step's scores to its weights.
    auto soften = [&](int t, int b) {
      if (t >= seen) {
        const uint64_t live = t < full ? ~0ull : __ballot(valid[set][b][lane % KT] != 0);
#pragma unroll
        for (int n = 0; n < SUBS; ++n) {
          // this half's keys from its first on that are there, and seen
          const int from = n * kKeyTile + 4 * half;
          const int ahead = min(max(sees - (t * KT + from), 0), 31);
          const uint32_t on = (uint32_t)(live >> from) & ((1u << ahead) - 1u);
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[n][i] = on >> (8 * (i / 4) + i % 4) & 1 ? sc[n][i] : kNone;
        }
      }
      float mx = kNone;
#pragma unroll
      for (int n = 0; n < SUBS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i) mx = fmaxf(mx, sc[n][i]);
      {
        const Pair h = both_halves(mx);
        mx = fmaxf(h.a, h.b) * q.scale;
      }
      // The weights' reference, the largest score less kLift, follows it only
      // once that is over 2^8 times what it was: weights of up to 2^8 more lose
      // nothing, and sums are seldom scaled again.
      if (__ballot(mx - top > 8.0f + T::kLift)) {   // (the difference is exact where it counts)
        const float now = fmaxf(mx - T::kLift, top);
        const float f = now == kNone ? 0.0f : __builtin_amdgcn_exp2f(top - now);
        top = now;
        sum *= f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[m][i] *= f;
        far = __ballot(__builtin_fabsf(top) > 0x1p16f && top > kNone) != 0;
      }
      float ref = top == kNone ? 0.0f : top, factor = q.scale;
      // The reference is a rounded score.  Beyond 2^16 its rounding would outgrow
      // the lag, and from 2^27 on overflow the weights: the scores are rounded
      // alike then, and none weighs more than the reference allows.
      if (__builtin_expect(far, 0)) {
#pragma unroll
        for (int n = 0; n < SUBS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) sc[n][i] = sc[n][i] * q.scale - ref;
        factor = 1.0f;
        ref = 0.0f;
      }
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < 2 * SUBS; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[u / 2][u % 2 * 8 + i], factor, -ref));
          part[i % 2] += p;
          // (to the cache's type, as the matrix instructions take them; the sum, which
          // the log-sum is made of, keeps 32 bits)
          w[u][i] = (typename T::Value)p;
        }
      sum += part[0] + part[1];
      if (LAG) {   // here, and not among the next phase's products
#pragma unroll
        for (int u = 0; u < 2 * SUBS; ++u) asm volatile("" : "+v"(w[u]));
      }
    };

    if (QW == 1) {
      for (; t < s.step1; t += KW) {
        const bool more = t + KW < s.step1;
        // all but the values have arrived, and the next step's table entries
        loads_but<PASSES + 1>();
        if (t >= full) mark(t, 0);
        multiply(yes, no, 0, 0);
        if (more) {
          lds_done();   // the keys are read
          locate(t + KW);
          fetch(t + KW, 0, true);
        }
        soften(t, 0);
        if (more) loads_but<PASSES>();
        else loads_but<0>();
        if (t >= full) clear(0);
        multiply(no, yes, 0, 0);
        if (more) {
          lds_done();   // the values are read
          fetch(t + KW, 0, false);
          find(t + 2 * KW);
        }
      }
    } else if (!LAG) {
      int b = 0;
      for (; t < s.step1; ++t) {
        // the step has arrived, and the next one's table entries
        settle(t, b);
        lds_barrier();
        if (t + 1 < s.step1) {
          locate(t + 1);
          fetch(t + 1, b ^ 1, true);
          fetch(t + 1, b ^ 1, false);
          find(t + 2);
        }
        multiply(yes, no, b, b);
        soften(t, b);
        multiply(no, yes, b, b);
        b ^= 1;
      }
    } else {
      // Two phases a step: in one the products of step t's keys and of step t
      // - 1's values, in the other step t's weights.  The first four waves are
      // a phase ahead of the others, so that each SIMD has one wave at either.
      // All waves fetch step t + 1 in phase 2 t, and wait for it at the end of
      // the next: of three buffers, t - 1 and t are read then.
      int b = 0;
      auto get = [&](int t, int b) {
        if (t < s.step1) {
          locate(t);
          fetch(t, b, true);
          fetch(t, b, false);
          find(t + 1);
        }
      };
      settle(t, 0);
      lds_barrier();
      if (lag) {
        get(t + 1, 1);
        lds_barrier();
      }
      for (; t < s.step1; ++t) {
        const int after = b == 2 ? 0 : b + 1, last = b == 0 ? 2 : b - 1;
        if (!lag) get(t + 1, after);
        if (t > s.step0) multiply(yes, yes, b, last);
        else multiply(yes, no, b, b);
        if (lag && t + 1 < s.step1) settle(t + 1, after);
        lds_barrier();
        if (lag) get(t + 2, last);
        soften(t, b);
        if (!lag && t + 1 < s.step1) settle(t + 1, after);
        lds_barrier();
        b = after;
      }
      if (!lag) lds_barrier();
      if (s.step1 > s.step0) multiply(no, yes, 0, b == 0 ? 2 : b - 1);
    }

    {
      const Pair h = both_halves(sum);
      sum = h.a + h.b;
    }
    if (KW == 1) {
      // Rows leave through LDS, 128 bytes of each at a time: 16 bytes of 64
      // rows, as the lanes hold them, would take several times as long.
      constexpr int PITCH = 36;
      static_assert(sizeof(stages) >= QW * 32 * PITCH * sizeof(float), "");
      float* rows = reinterpret_cast<float*>(&stages[0][0]) + qw * 32 * PITCH;
      const int r8 = lane >> 3, c8 = (lane & 7) * 4;
      __syncthreads();
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          *reinterpret_cast<float4*>(rows + col * PITCH + 2 * i + 4 * half) =
              float4{acc[m][i], acc[m][i + 1], acc[m][i + 2], acc[m][i + 3]};
        wave_sync();
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          if (s.first + qw * 32 + i + r8 < s.rows)
            *reinterpret_cast<float4*>(parts + (int64_t)(qw * 32 + i + r8) * DIM + 32 * m + c8) =
                *reinterpret_cast<const float4*>(rows + (i + r8) * PITCH + c8);
        wave_sync();
      }
      if (has && half == 0) stats[qw * 32 + col] = float2{top, sum};
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
    uint64_t falls = 0;
    for (int g0 = 0; g0 < q.groups; g0 += 64) {
      const int g = g0 + lane;
      falls |= __ballot(q.starts && g < q.groups && q.starts[g + 1] < q.starts[g]);
      const GroupScan c = scan_groups(q, g0, 32 * QW, KT, all, strips);
      if (blockIdx.x == 0 && threadIdx.x < 64 && g0 + (int)threadIdx.x < q.groups)
        q.group_at[g0 + threadIdx.x] = int4{c.step_end - c.steps, c.strip_end - c.strips, 0, 0};
      all = __builtin_amdgcn_readlane(c.step_end, 63);
      strips = __builtin_amdgcn_readlane(c.strip_end, 63);
    }
    // (starts that fall may have more strips than there is room for: no shared
    // positions then, which the join learns from here)
    if (falls) strips = q.strips + 1;
    if (blockIdx.x == 0 && threadIdx.x == 0) q.group_at[q.groups] = int4{all, strips, 0, 0};
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
  uint32_t id = blockIdx.x - (uint32_t)q.shared_grid;
  s.head = (int)(id % (uint32_t)q.kv_heads);
  id /= (uint32_t)q.kv_heads;
  const int tile = (int)(id % (uint32_t)q.own_tiles);
  id /= (uint32_t)q.own_tiles;
  const int split = (int)(id % (uint32_t)q.own_splits);
  s.seq0 = (int)(id / (uint32_t)q.own_splits);
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
// Joins a row's pieces: a wave a row, its lanes in 64 / (dim / 4) sets that
// take turns at the pieces.  Bound by reading them: 4096 rows of about 18
// pieces, 38 MB, take 10.8 us (3.5 TB/s), 128 rows 4.5, where the waits for
// what says where the pieces lie are the whole; a small row's pieces are asked
// for before its largest score is known (1120 rows 4.8 instead of 6.3).
// ---------------------------------------------------------------------------
template <class T, int DIM>
__global__ void __launch_bounds__(256) attend_join_kernel(const AttendParams q) {
  constexpr int LANES = DIM / 4, SETS = 64 / LANES;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
    } else {
      for (int g0 = 0; g0 < q.groups; g0 += 64) {  // the last group that starts at or before seq
        const uint64_t m = __ballot(g0 + lane < q.groups && q.starts[min(g0 + lane, q.groups)] <= seq);
        if (m) g = g0 + 63 - __builtin_clzll(m);
        if (m != ~0ull) break;
      }
    }
    if (g >= 0) {
      group_range(q, g, s0, s1);
      const int4 at = q.group_at[g], all = q.group_at[q.groups];
      const int steps = (min(max(q.shared.lens[g], 0), q.shared.limit) + q.shared_tile - 1) / q.shared_tile;
      if (seq >= s0 && seq < s1 && steps > 0 && all.y <= q.strips) {
        const int cols = 32 * q.query_waves;
        const int r = (tok - s0 * q.next_n) * q.per + sub, tile = r / cols;
        const int share = share_of(q, all.x);
        const int a = at.x + tile * steps, first = a / share;
        shared = (a + steps - 1) / share - first + 1;
        shared_slot = ((int64_t)kv * (q.shared_wgs + q.strips) + first + at.y + tile) * cols + (r - tile * cols);
      }
    }
  }
  const int own_rows = q.next_n * q.per;
  const int steps = (min(max(q.own.lens[seq], 0), q.own.limit) + kKeyTile - 1) / kKeyTile;
  const int share = q.own_splits > 0 ? max((steps + q.own_splits - 1) / q.own_splits, kOwnSets) : 1;
  const int own = q.own_splits > 0 ? (steps + share - 1) / share : 0;
  const int64_t own_slot = ((int64_t)seq * q.kv_heads + kv) * own_rows + (tok - seq * q.next_n) * q.per + sub;
  const int64_t own_stride = (int64_t)q.seqs * q.kv_heads * own_rows;
  const int n = shared + own;
  auto stat = [&](int i) {
    return i < shared ? q.shared_stats[shared_slot + (int64_t)i * 32 * q.query_waves]
                      : q.own_stats[own_slot + (i - shared) * own_stride];
  };

  const int set = lane / LANES, at = (lane % LANES) * 4;
  auto piece = [&](int i) {
    return *reinterpret_cast<const float4*>(
        (i < shared ? q.shared_parts + (shared_slot + (int64_t)i * 32 * q.query_waves) * DIM
                    : q.own_parts + (own_slot + (i - shared) * own_stride) * DIM) + at);
  };
  // (the first pieces are on their way while the largest score is found)
  constexpr int FIRST = 4;
  float4 x[FIRST];
  float2 st[FIRST];
#pragma unroll
  for (int a = 0; a < FIRST; ++a) {
    const int i = set + a * SETS;
    x[a] = float4{0.0f, 0.0f, 0.0f, 0.0f};
    st[a] = float2{kNone, 0.0f};
    if (i < n) {
      st[a] = stat(i);
      x[a] = piece(i);
    }
  }
  float top = kNone;
  for (int i = lane; i < n; i += 64) top = fmaxf(top, stat(i).x);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const float ref = top == kNone ? 0.0f : top;
  float total = 0.0f;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](const float2& st, const float4& x) {
    const float f = __builtin_amdgcn_exp2f(st.x - ref);
    total += st.y * f;
    v[0] += x.x * f;
    v[1] += x.y * f;
    v[2] += x.z * f;
    v[3] += x.w * f;
  };
#pragma unroll
  for (int a = 0; a < FIRST; ++a) add(st[a], x[a]);
#pragma unroll 4
  for (int i = set + FIRST * SETS; i < n; i += SETS) add(stat(i), piece(i));
#pragma unroll
  for (int d = LANES; d < 64; d <<= 1) {
    total += __shfl_xor(total, d);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += __shfl_xor(v[i], d);
  }
  if (set > 0) return;
  const float inv = total > 0.0f || total != total ? 1.0f / total : 0.0f;
  typedef typename T::Value Value;
  Value r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (Value)(v[i] * inv);
  uint2 w;
  __builtin_memcpy(&w, r, 8);
  *reinterpret_cast<uint2*>(reinterpret_cast<Value*>(q.out) + row * DIM + at) = w;
  if (q.lse && lane == 0)
    q.lse[row] = total > 0.0f || total != total ? (top + __builtin_log2f(total)) * 0.69314718f : kNone;
}

// ---------------------------------------------------------------------------
// Attention mass: mass[h][p] = decay mass[h][p] + the weights of position p in
// every query of key head h.  A wave holds two tiles of 32 keys and runs over
// the entry's queries, 32 at a time; each lane adds up its query column's
// weights, and the 32 columns are added at the end, so sums have one order.
// The next tiles are on their way to LDS while the last queries are computed
// and these are written.
//
// Bound by memory and by the exponentials, one a (position, query): 8 groups of
// 64 queries a key head over some 6 thousand positions each, and 64 sequences'
// own 1 to 256, 122 MB, take 32 us (3.8 TB/s): 28 for the reading alone, 22 for
// the products and exponentials alone.  Four tiles a wave: two take 36, for
// their first loads, eight the same and 15 instead of 9 where there are few.
// ---------------------------------------------------------------------------
namespace {

// Sums over a half wave: lane l of it gets that of value l % 16.  Lanes that
// differ in one more bit of l exchange the half of their values that the other
// keeps, so each step adds half as many.
template <int CTL>
__device__ __forceinline__ float from_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTL, 0xf, 0xf, true));
}
template <int CTL, int N>
__device__ __forceinline__ void halve(float (&v)[16], bool upper) {
#pragma unroll
  for (int x = 0; x < N; ++x) {
    const float keep = upper ? v[x + N] : v[x], send = upper ? v[x] : v[x + N];
    v[x] = keep + from_lane<CTL>(send);
  }
}
__device__ __forceinline__ float half_sums(float (&v)[16], int lane) {
  halve<0x140, 8>(v, lane & 8);   // row_mirror: lane ^ 15
  halve<0x141, 4>(v, lane & 4);   // row_half_mirror: lane ^ 7
  halve<0x1B, 2>(v, lane & 2);    // quad_perm 3 2 1 0
  halve<0xB1, 1>(v, lane & 1);    // quad_perm 1 0 3 2
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[0]), __float_as_uint(v[0]), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace

template <class T, int DIM>
__global__ void __launch_bounds__(kMassBlock, 2) attend_mass_kernel(const MassParams mp) {
  constexpr int STEPS = DIM / 16, TILES = kMassTiles, PAIR = 2;
  constexpr int PIECES = DIM / 8, ROWS = 64 / PIECES, PASSES = kKeyTile / ROWS;
  __shared__ Piece tiles[kMassBlock / 64][PAIR][kKeyTile * PIECES];
  const AttendParams& q = mp.a;
  const int lane = threadIdx.x & 63, col = lane & 31, half = lane >> 5;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint32_t id = blockIdx.x;
  const bool shared = id < (uint32_t)mp.shared_wgs;
  if (!shared) id -= (uint32_t)mp.shared_wgs;
  const uint32_t parts = (uint32_t)(shared ? mp.shared_tiles : mp.own_tiles);
  const int part = (int)(id % parts);
  id /= parts;
  const int head = (int)(id % (uint32_t)q.kv_heads);
  const int entry = (int)(id / (uint32_t)q.kv_heads);
  const int row_len = shared ? mp.shared_width : mp.own_width;
  const PageTables& pt = shared ? q.shared : q.own;
  const int32_t* table = pt.tables + (int64_t)entry * pt.stride;
  const int len = min(max(pt.lens[entry], 0), pt.limit);
  int seq0 = entry, seqs = 1, cut = q.next_n - 1;
  if (shared) {
    int s1;
    group_range(q, entry, seq0, s1);
    // where starts fall, the log-sums lack all prefixes
    const bool falls = q.starts && q.groups <= 64 && lane < q.groups && q.starts[lane + 1] < q.starts[lane];
    seqs = __ballot(falls) ? 0 : s1 - seq0;
    cut = 0;
  }
  // this wave's tiles: every fourth of the workgroup's
  auto first_of = [&](int i) { return ((part * TILES + i) * (kMassBlock / 64) + wv) * kKeyTile; };
  int rows = seqs * q.next_n * q.per;

  int32_t block[TILES];
#pragma unroll
  for (int i = 0; i < TILES; ++i) {
    const int p = first_of(i) + col;
    block[i] = p < len ? block_at(q, table, pt.width, p) : -1;
  }
  Piece key[PAIR][STEPS], query[STEPS];
  uint64_t live[PAIR];
  const int lrow = lane / PIECES, lpiece = lane % PIECES;
  // two tiles to LDS: whole rows, side by side; what is not there is read from
  // the cache's first slot, and masked
  auto fetch = [&](int i0) {
#pragma unroll
    for (int i = 0; i < PAIR; ++i) {
      const int32_t b = block[i0 + i];
      if (!__ballot(b >= 0)) continue;
      const uint32_t p = (uint32_t)(first_of(i0 + i) + col);
      const uint32_t off = p - q.by_block(p) * (uint32_t)q.block_size;
      const uint64_t from = b >= 0 ? (uint64_t)b * q.k.block_stride + (uint64_t)off * q.k.slot_stride : 0;
#pragma unroll
      for (int s = 0; s < PASSES; ++s) {
        const int row = s * ROWS + lrow;
        const uint32_t low = (uint32_t)__shfl((int)(uint32_t)from, row), high = (uint32_t)__shfl((int)(from >> 32), row);
        load_to_lds(q.k.base + head * q.k.head_stride + ((uint64_t)high << 32 | low) + key_piece<DIM>(row, lpiece) * 16,
                    &tiles[wv][i][s * 64]);
      }
    }
  };
  auto take = [&](int i0) {
    loads_but<0>();
#pragma unroll
    for (int i = 0; i < PAIR; ++i) {
      live[i] = __ballot(block[i0 + i] >= 0);
#pragma unroll
      for (int d = 0; d < STEPS; ++d) key[i][d] = tiles[wv][i][col * PIECES + key_piece<DIM>(col, 2 * d + half)];
    }
    lds_done();
  };
  // queries r0 .. r0 + 31: this lane's, its log-sum and the positions it sees
  float lse = 0.0f;
  int sees = 0;
  auto load_queries = [&](int r0) {
    const int r = r0 + col;
    const uint32_t rr = r < rows ? (uint32_t)r : 0u;
    const uint32_t tok = rr / (uint32_t)q.per, sub = rr - tok * (uint32_t)q.per;
    const int64_t row = (int64_t)seq0 * q.next_n + tok;
    const unsigned char* at = q.q + row * q.q_stride + (head * q.per + sub) * q.q_head_stride + half * 16;
#pragma unroll
    for (int d = 0; d < STEPS; ++d) query[d] = *reinterpret_cast<const Piece*>(at + d * 32);
    lse = mp.lse[row * q.heads + head * q.per + sub];
    // a row that saw nothing has a sum of nothing: its weights are none
    const bool on = r < rows && lse > kNone;
    lse = on ? lse * 1.44269504f : 0.0f;
    sees = on ? len - cut + (cut ? (int)(tok % (uint32_t)q.next_n) : 0) : 0;
  };
  if (rows > 0 && first_of(0) < min(len, row_len)) {
    fetch(0);
    load_queries(0);
  }
  // More groups than a wave has lanes: three pairs of neighbours a lane, the
  // workgroup's waves in turn, once the keys are on their way (4096 groups of a
  // sequence over 128 positions: 230 us without looking, 280 so, 680 with a
  // wave's pairs one load after the other).
  if (shared && q.starts && q.groups > 64 && rows > 0) {
    bool fall = false;
#pragma unroll 4
    for (int g = wv * 192; g < q.groups; g += 192 * (kMassBlock / 64)) {
      int4 s;
      __builtin_memcpy(&s, q.starts + min(g + 3 * lane, q.groups - 3), 16);
      fall |= s.y < s.x || s.z < s.y || s.w < s.z;
    }
    if (__syncthreads_or(fall)) {
      rows = 0;
      loads_but<0>();   // (nothing takes the keys)
    }
  }
  if (first_of(0) >= row_len) return;
  const float* in = shared ? mp.shared_in : mp.own_in;
  float* out = shared ? mp.shared_out : mp.own_out;
  const int64_t base = ((int64_t)entry * q.kv_heads + head) * row_len;
  // register i of a half is position 8 (i / 4) + 4 half + i % 4: lane i of the
  // half writes it
  const int mine = 8 * (col / 4) + 4 * half + col % 4;
#pragma unroll
  for (int i0 = 0; i0 < TILES; i0 += PAIR) {
    if (first_of(i0) >= row_len) break;
    float old[PAIR], acc[PAIR][16];
#pragma unroll
    for (int i = 0; i < PAIR; ++i) {
      const int p = first_of(i0 + i) + mine;
      old[i] = in && col < 16 && p < row_len ? in[base + p] : 0.0f;
#pragma unroll
      for (int x = 0; x < 16; ++x) acc[i][x] = 0.0f;
    }
    if (rows > 0 && first_of(i0) < len) {
      take(i0);
      for (int r0 = 0; r0 < rows; r0 += 32) {
        if (r0 > 0 || (i0 > 0 && rows > 32)) load_queries(r0);
        if (r0 + 32 >= rows && i0 + PAIR < TILES && first_of(i0 + PAIR) < min(len, row_len)) {
          loads_but<0>();   // (the queries: in order, they would wait for the keys as well)
          fetch(i0 + PAIR);
        }
#pragma unroll
        for (int i = 0; i < PAIR; ++i) {
          if (!live[i]) continue;
          f32x16 sc;
#pragma unroll
          for (int x = 0; x < 16; ++x) sc[x] = 0.0f;
#pragma unroll
          for (int d = 0; d < STEPS; ++d) sc = T::mfma(key[i][d], query[d], sc);
          if (live[i] == ~0ull && __ballot(sees >= first_of(i0 + i) + kKeyTile) == ~0ull) {   // all is seen
#pragma unroll
            for (int x = 0; x < 16; ++x)
              acc[i][x] += __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x], q.scale, -lse));
            continue;
          }
          const int ahead = min(max(sees - (first_of(i0 + i) + 4 * half), 0), 31);
          const uint32_t seen = (uint32_t)(live[i] >> (4 * half)) & ((1u << ahead) - 1u);
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const float w = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[x], q.scale, -lse));
            acc[i][x] += seen >> (8 * (x / 4) + x % 4) & 1 ? w : 0.0f;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < PAIR; ++i) {
      const float sum = half_sums(acc[i], lane);
      const int p = first_of(i0 + i) + mine;
      if (col < 16 && p < row_len) out[base + p] = old[i] * mp.decay + sum;
    }
  }
}

namespace {

template <class T, int DIM, bool EVEN>
const void* attend_ptr(int query_waves, int sets) {
  switch (query_waves) {
    case 8: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 8, 1, 64, EVEN>);
    case 4: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 4, 1, 64, EVEN>);
    case 2: return reinterpret_cast<const void*>(&attend_kernel<T, DIM, 2, 1, 32, EVEN>);
  }
  return sets == 1 ? reinterpret_cast<const void*>(&attend_kernel<T, DIM, 1, 1, kKeyTile, EVEN>)
                   : reinterpret_cast<const void*>(&attend_kernel<T, DIM, 1, kOwnSets, kKeyTile, EVEN>);
}
template <class T>
const void* attend_ptr(int dim, int query_waves, int sets, bool even) {
  if (dim == 64) return even ? attend_ptr<T, 64, true>(query_waves, sets) : attend_ptr<T, 64, false>(query_waves, sets);
  return even ? attend_ptr<T, 128, true>(query_waves, sets) : attend_ptr<T, 128, false>(query_waves, sets);
}

}  // namespace

const void* attend_kernel_ptr(int dtype, int dim, int query_waves, int sets, int block_size) {
  // rows that a wave loads at once
  const bool even = block_size % (64 / (dim / 8)) == 0;
  return dtype == 1 ? attend_ptr<Bf16>(dim, query_waves, sets, even) : attend_ptr<F16>(dim, query_waves, sets, even);
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
