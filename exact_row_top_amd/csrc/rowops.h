// rowops.h -- launch parameters and small device helpers of the row operators
// beside the top-K selection (sampling, expert routing, slot maps).
#pragma once

#include <hip/hip_runtime.h>
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <stdint.h>

namespace ert {

// ---- sampling --------------------------------------------------------------

constexpr int kSegment = 2048;    // scores one wave reads
constexpr int kSegSlots = 128;    // candidates a segment can hand on
constexpr int kMaxVocab = 1 << 20;

// One segment's findings, written by the segment kernel for the row kernel.
struct SegRecord {
  float best;       // largest live score, -inf if none
  int32_t first;    // greedy rows: the lowest position that holds it
  float floor;      // every live score >= floor is among the candidates
  int32_t count;    // candidates, -1 if they did not fit
  uint64_t mass;    // rows that need it: sum of the weights against `best`
  float low;        // rows with cuts: smallest live score
  float upper;      // rows with a top-p alone: the candidates' mass, rounded up
};

struct Candidate {
  float x;
  int32_t i;
};

// A row's way through the kernels after the row kernel.
constexpr int kWideBlock = 512;   // a wave for each segment
constexpr int kWideSegs = kWideBlock / 64;
constexpr int kRowBlock = kWideBlock;
constexpr int kBinsS = 1024;      // histogram bins
enum : uint32_t { kWideDone = 0, kWideMembers = 1, kWideWhole = 2 };
struct WideRow {
  uint32_t state;
  float m;              // the row's largest score
  uint64_t need;        // mass that top-p leaves to its crossing bins
  // Scores: the lowest above all crossing bins, the lowest in top-p's, and
  // the same two of top-k's.  NaN: none.
  float edge[4];
  uint32_t need_k;      // count that top-k leaves to its crossing bin
  uint64_t mass_k;      // with both: the mass above that bin
  uint64_t before;      // the mass above top-p's crossing bins
  uint32_t arrived[2];  // workgroups done with the bins, with the members
};

struct SampleParams {
  const void* logits;
  int64_t row_stride;  // elements
  int32_t vocab;
  int32_t rows;
  int32_t segments;    // per row
  const float* uniforms;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int32_t* tokens;
  float* logprobs;
  SegRecord* records;
  Candidate* candidates;  // [rows][segments][kSegSlots]; later the crossing bins' members
  WideRow* wide;          // null where no row can have a cut
  uint64_t* kept;         // [rows][segments + wide_wgs]: kept masses, member counts
  uint64_t* masses;       // [rows][wide_wgs][kBinsS]
  uint32_t* counts;       // the same
  int32_t wide_wgs;       // workgroups of a row in the wide kernel
  int32_t row_wgs;        // in the row kernel: as many if a top-k or top-p is given, else one
  int32_t whole_row;      // every row from memory
};

// ---- exponentials in 64 bits ---------------------------------------------------

constexpr double kLog2e = 1.4426950408889634;

// 2^f on [-1/2, 1/2]: interpolation at the ten Chebyshev nodes, relative
// error at most 2^-45.6.  The coefficients sit in scalar registers behind an
// empty asm: as known constants each would be moved into a vector register
// pair ahead of every multiply-add, two instructions to one.
struct Exp2Poly {
  double k0, k1, k2, k3, k4, k5, k6, k7, k8, k9;
  __device__ __forceinline__ Exp2Poly()
      : k0(0x1.000000000003dp+0), k1(0x1.62e42fefa39f7p-1), k2(0x1.ebfbdff8149f2p-3),
        k3(0x1.c6b08d7044119p-5), k4(0x1.3b2ab72b175eep-7), k5(0x1.5d87fe908f88ap-10),
        k6(0x1.43088e257f341p-13), k7(0x1.ffcb76789860fp-17), k8(0x1.63ef969a64d3cp-20),
        k9(0x1.b6571de2f2351p-24) {
    asm("" : "+s"(k0), "+s"(k1), "+s"(k2), "+s"(k3), "+s"(k4));
    asm("" : "+s"(k5), "+s"(k6), "+s"(k7), "+s"(k8), "+s"(k9));
  }
  __device__ __forceinline__ double operator()(double f) const {
    double p = __builtin_fma(f, k9, k8);
    p = __builtin_fma(p, f, k7);
    p = __builtin_fma(p, f, k6);
    p = __builtin_fma(p, f, k5);
    p = __builtin_fma(p, f, k4);
    p = __builtin_fma(p, f, k3);
    p = __builtin_fma(p, f, k2);
    p = __builtin_fma(p, f, k1);
    return __builtin_fma(p, f, k0);
  }
};

// 2^s for s <= 0; 0 for NaN.
__device__ __forceinline__ double exp2_64(double s, const Exp2Poly& poly) {
  s = __builtin_fmax(s, -1100.0);
  const double n = __builtin_rint(s);
  return __builtin_ldexp(poly(s - n), (int)n);
}

// A wave's LDS operations are done in order: this only keeps the compiler
// from moving them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---- 16-byte score groups ----------------------------------------------------

template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&x)[4]) {
    x[0] = __uint_as_float(q.x);
    x[1] = __uint_as_float(q.y);
    x[2] = __uint_as_float(q.z);
    x[3] = __uint_as_float(q.w);
  }
  __device__ static __forceinline__ void unpack_word(uint32_t w, float (&x)[1]) {
    x[0] = __uint_as_float(w);
  }
  __device__ static __forceinline__ float load(const void* base, int64_t i) {
    return static_cast<const float*>(base)[i];
  }
};
template <>
struct Elem<__hip_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
  __device__ static __forceinline__ void unpack_word(uint32_t w, float (&x)[2]) {
    x[0] = __uint_as_float(w << 16);
    x[1] = __uint_as_float(w & 0xFFFF0000u);
  }
  __device__ static __forceinline__ float load(const void* base, int64_t i) {
    return __uint_as_float((uint32_t)static_cast<const unsigned short*>(base)[i] << 16);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kVec = 8;
  __device__ static __forceinline__ void unpack(const uint4& q, float (&x)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __half2float(__ushort_as_half((unsigned short)(w[j] & 0xFFFFu)));
      x[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(w[j] >> 16)));
    }
  }
  __device__ static __forceinline__ void unpack_word(uint32_t w, float (&x)[2]) {
    x[0] = __half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu)));
    x[1] = __half2float(__ushort_as_half((unsigned short)(w >> 16)));
  }
  __device__ static __forceinline__ float load(const void* base, int64_t i) {
    return __half2float(static_cast<const __half*>(base)[i]);
  }
};

}  // namespace ert

namespace ert {

// ---- routing to experts ----------------------------------------------------

constexpr int kMaxExperts = 1024;
constexpr int kMaxGroups = 16;
constexpr int kMaxRouteK = 64;

struct RouteParams {
  const void* logits;
  int64_t row_stride;   // elements
  int32_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t sigmoid;      // else softmax
  const float* bias;    // null: none
  int32_t groups;
  int32_t group_size;
  uint32_t group_magic;  // e / group_size = the high word of e * group_magic
  int32_t group_lanes;   // log2 of the lanes that look at one group together
  int32_t vector;        // every row starts on 16 bytes and holds whole groups
  int32_t vector_bias;   // so does the bias, with groups of four
  int32_t topk_groups;
  int32_t top2;         // a group's score: its two largest summed, else its largest
  int32_t renormalize;
  float scale;
  int32_t* indices;     // [tokens][top_k]
  float* weights;
};

struct RouteGradParams {
  const void* logits;
  int64_t row_stride;
  int32_t tokens;
  int32_t experts;
  int32_t top_k;
  int32_t sigmoid;
  int32_t renormalize;
  float scale;
  const int32_t* indices;
  const float* grad_weights;
  void* grad_logits;
  int64_t grad_stride;
  int32_t vector;       // rows of both start on 16 bytes and hold whole groups
};

// ---- block tables and slots --------------------------------------------------

constexpr int kMaxRequests = 4096;
constexpr int kSlotBlock = 256;
constexpr int kSlotPart = 1024;    // entries of a row that a workgroup maps

// Division by d of numbers below 2^31: a shift for powers of two (magic 0),
// else the high word of the product with ceil(2^(31 + L) / d), L =
// ceil(log2 d), shifted by L - 1: the rounding adds less than n 2^L / 2^(31 +
// L) < 1 to n / d scaled by d, so the quotient is exact.
struct Divisor {
  uint32_t magic;
  uint32_t shift;
};

struct TableParams {
  int32_t* tables;
  int64_t table_stride;
  int32_t max_blocks;
  int32_t requests;
  const int32_t* kv_lens;
  const int32_t* new_tokens;
  const int32_t* free_blocks;
  int64_t num_free;
  const int32_t* free_start;
  int32_t block_size;
  Divisor by_block;
  int32_t vector;       // the token arrays start on 16 bytes
  int64_t max_tokens;
  int32_t* token_starts;
  int32_t* token_requests;
  int32_t* positions;
  void* slots;
  int32_t wide;         // slots are int64
  int32_t* free_next;
};

struct SlotParams {
  const int32_t* indices;
  int64_t rows;
  int32_t k;
  const int32_t* tables;
  int64_t table_stride;
  int32_t max_blocks;
  int32_t requests;
  const int32_t* row_requests;
  int32_t next_n;
  int32_t block_size;
  Divisor by_block;
  int32_t parts;        // workgroups of a row
  int32_t vector;       // rows of both start on 16 bytes and hold whole groups of four
  int32_t staged;       // the table goes through LDS
  void* slots;
  int32_t wide;
};

}  // namespace ert
