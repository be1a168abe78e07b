// search.h -- launch parameters of the operators of a beam search over a paged
// cache: the beams' choice, reordering, shared-prefix attention, attention
// mass and eviction.
#pragma once

#include "rowops.h"

namespace ert {

// Division by d of numbers below 2^31, without a branch: the high word of 2 n
// ceil(2^(31 + L) / d), L = ceil(log2 d), shifted by L (the rounding adds less
// than n 2^L / 2^(31 + L) < 1 to n / d scaled by d, so the quotient is exact).
struct Quotient {
  uint32_t magic;
  uint32_t shift;
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return __umulhi(n << 1, magic) >> shift; }
};

// ---- the beams' choice ---------------------------------------------------------

constexpr int kMaxBeams = 32;
constexpr int kMaxBeamK = 64;
constexpr int kChunk = 32;        // neighbouring scores that share one maximum
constexpr int kBeamBlock = 512;

// One of a beam's best continuations, in falling order.
struct BeamCandidate {
  double rank;
  float total;
  int32_t token;  // -1: none
};

struct BeamParams {
  const void* logits;
  int64_t row_stride;        // elements
  int32_t vocab;
  int32_t rows;              // requests * beams
  int32_t beams;
  int32_t k;
  int32_t segments;          // of a row
  const float* scores;       // [rows]
  const uint8_t* ended;      // [rows] or null
  int32_t end_token;
  const int32_t* lengths;    // [rows] or null
  double penalty;
  float* out_scores;         // [requests][k]
  int32_t* parents;
  int32_t* tokens;
  double* masses;            // [rows][segments]: a segment's weights against its best
  float* bests;              // [rows][segments]
  float* chunks;             // [rows][segments * 64]: the largest of 32 neighbours
  BeamCandidate* found;      // [rows][k]
  uint32_t* arrived;         // [requests]: rows done
  int32_t cap;               // chunks that a row can list
};

// ---- reordering --------------------------------------------------------------------

constexpr int kCopyBlock = 256;
constexpr int kMaxCopies = 32;    // arrays a launch reorders
constexpr int kMaxCaches = 64;    // caches a launch copies open blocks of

struct RowCopy {
  const unsigned char* src;
  unsigned char* dst;
  int64_t src_stride;   // bytes
  int64_t dst_stride;
  int64_t row_bytes;
  uint32_t tiles;       // workgroups of a request
  uint32_t first;       // workgroup of the launch
};

struct ReorderParams {
  const int32_t* parents;   // [requests][k]
  int32_t beams;
  int32_t k;
  int32_t copies;
  int32_t clear;            // rows without a parent are cleared, else left
  RowCopy copy[kMaxCopies];
};

struct ReorderBlocksParams {
  const int32_t* parents;
  int32_t requests;
  int32_t beams;
  int32_t k;
  const int32_t* tables;    // [requests * beams][max_blocks]
  int64_t table_stride;
  int32_t max_blocks;
  int32_t* out;             // [requests * k][max_blocks]
  int64_t out_stride;
  const int32_t* kv_lens;   // [requests]
  const int32_t* tail;      // [requests * k] or null: each row's own open block
  Quotient by_block;
  int32_t block_size;
  int64_t num_blocks;
  int64_t slot_bytes;       // of the caches
  int64_t block_stride;     // bytes
  int32_t caches;
  uint32_t tiles;           // workgroups that copy a request's open blocks in one cache
  uint32_t table_tiles;     // workgroups that make a request's table rows
  int32_t copying;          // this launch copies; else it makes tables only
  unsigned char* cache[kMaxCaches];
};

// ---- attention with a shared prefix ---------------------------------------------------

constexpr int kKeyTile = 32;        // keys of a score tile
constexpr int kMassBlock = 256;
constexpr int kMassTiles = 4;       // key tiles of a wave of the mass kernel
constexpr int kOwnSets = 4;         // waves that take turns at the keys of up to 32 queries

// Pages of one cache: position p of a table row lies in block table[p / size]
// at p % size.
struct Pages {
  const unsigned char* base;
  uint32_t block_stride;     // bytes
  uint32_t slot_stride;
  int64_t head_stride;
};

struct PageTables {
  const int32_t* tables;
  int64_t stride;
  int32_t width;
  int32_t limit;             // positions a row can hold, and lengths are cut to
  const int32_t* lens;
};

struct AttendParams {
  const unsigned char* q;    // [seqs * next_n][heads][dim]
  int64_t q_stride;          // bytes
  int64_t q_head_stride;
  Pages k, v;
  int64_t num_blocks;
  int32_t block_size;
  Quotient by_block;
  PageTables shared, own;    // [groups], [seqs]
  const int32_t* starts;     // [groups + 1]: a group's sequences; null: equal groups
  int32_t groups;
  int32_t seqs;
  int32_t members;           // of a group, without starts
  int32_t next_n;
  int32_t heads;
  int32_t kv_heads;
  int32_t per;               // heads / kv_heads
  float scale;               // log2(e) times the scores' scale
  // The shared kernel's work: `query_waves` waves of 32 queries to a workgroup,
  // shared_wgs of them to a key head; own positions in own_splits.
  int32_t query_waves;
  int32_t shared_tile;       // keys of its step
  int32_t shared_least;      // steps of a workgroup, at least
  int32_t shared_wgs;
  int32_t strips;            // query tiles of all groups, at most
  int32_t own_splits;
  int32_t own_tiles;         // query tiles of a sequence
  int64_t shared_grid;       // workgroups of this launch on shared positions
  int64_t rows;              // seqs * next_n * heads
  int4* group_at;            // [groups + 1]: first step, first strip; steps of all
  float* shared_parts;       // [kv_heads][shared_wgs + strips][32 query_waves][dim]: weighted values
  float2* shared_stats;      // the same rows: the weights' reference (log2), their sum
  float* own_parts;          // [own_splits][seqs][kv_heads][next_n * per][dim]
  float2* own_stats;
  unsigned char* out;        // [rows][dim]
  float* lse;                // [rows] or null
};

struct MassParams {
  AttendParams a;
  const float* lse;          // [rows]
  const float* shared_in;    // [groups][kv_heads][shared_width] or null
  float* shared_out;
  int32_t shared_width;      // positions of a mass row
  const float* own_in;       // [seqs][kv_heads][own_width] or null
  float* own_out;
  int32_t own_width;
  float decay;
  int32_t shared_tiles;      // workgroups of a (group, head)
  int32_t own_tiles;
  int64_t shared_wgs;
};

// ---- eviction ----------------------------------------------------------------------------

constexpr int kKeepBlock = 1024;
constexpr int kMoveBlock = 256;

struct KeepParams {
  const float* mass;         // [requests][heads][positions]
  int64_t request_stride;    // elements
  int64_t head_stride;
  int32_t positions;
  int32_t heads;
  const int32_t* kv_lens;    // [requests]
  int32_t budget;
  int32_t sinks;
  int32_t recent;
  int32_t* kept;             // [requests][heads][budget]
  float* mass_out;           // [requests][heads][out_positions] or null
  int32_t out_positions;
  int32_t* new_lens;         // [requests]
};

struct MoveParams {
  const int32_t* kept;       // [requests][heads][budget]
  int32_t requests;
  int32_t heads;
  int32_t budget;
  const int32_t* tables;
  int64_t table_stride;
  int32_t max_blocks;
  const int32_t* out_tables;
  int64_t out_stride;
  int32_t out_blocks;
  Quotient by_block;
  int32_t block_size;
  int64_t num_blocks;
  int64_t slot_bytes;        // of all heads
  int64_t row_bytes;         // of one head group: slot_bytes / heads
  int32_t columns;           // workgroups that share a row's bytes
  int32_t parts;             // workgroups that share a row's positions
  int32_t caches;
  unsigned char* cache[kMaxCaches];
};

}  // namespace ert
