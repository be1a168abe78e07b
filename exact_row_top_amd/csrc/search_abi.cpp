// search_abi.cpp -- C ABI of a beam search's operators over a paged cache:
// host-side validation (no device reads) and the kernel launches.  The
// contract is documented in include/exact_row_top.h.

#include <hip/hip_runtime.h>

#include <math.h>

#include "exact_row_top.h"
#include "rowops_host.h"
#include "search.h"

namespace ert {
const void* beam_segment_kernel_ptr(int dtype);
const void* beam_row_kernel_ptr(int dtype, int pieces);
const void* reorder_rows_kernel_ptr(int n);
const void* reorder_blocks_kernel_ptr(int n);
const void* attend_kernel_ptr(int dtype, int dim, int query_waves, int sets, int block_size);
const void* attend_join_kernel_ptr(int dtype, int dim);
const void* attend_mass_kernel_ptr(int dtype, int dim);
const void* evict_keep_kernel_ptr(int64_t positions);
const void* evict_move_kernel_ptr(bool in_place);
}  // namespace ert

using namespace ert;

namespace {

constexpr int64_t kMassStep = kKeyTile * kMassTiles * kMassBlock / 64;  // positions of a workgroup
constexpr int64_t kInt = ((int64_t)1 << 31) - 1;

Quotient quotient_of(uint32_t d) {
  uint32_t log = 0;
  while (((uint64_t)1 << log) < d) ++log;
  return Quotient{(uint32_t)((((uint64_t)1 << (31 + log)) + d - 1) / d), log};
}

// Whether [a, a + na) and [b, b + nb) share no byte (or one is not given).
bool clear_of(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return !a || !b || x + na <= y || y + nb <= x;
}

// Whether rows of na bytes, a stride apart from a on, and rows of nb bytes share
// no byte: side by side in rows of one stride, or apart.
bool rows_clear(const void* a, int64_t na, int64_t sa, int64_t ra, const void* b, int64_t nb, int64_t sb, int64_t rb) {
  if (clear_of(a, (uint64_t)((ra - 1) * sa + na), b, (uint64_t)((rb - 1) * sb + nb))) return true;
  if (sa != sb) return false;
  const int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t at = ((d % sa) + sa) % sa;   // b's first byte in a's rows
  return at >= na && sa - at >= nb;
}

// Whether caches of one size share no byte.
bool caches_apart(void* const* caches, int32_t n, int64_t blocks, int32_t block_size, int64_t slot_bytes) {
  const unsigned __int128 all = (unsigned __int128)blocks * (unsigned)block_size * (uint64_t)slot_bytes;
  const uint64_t bytes = all >> 62 ? (uint64_t)1 << 62 : (uint64_t)all;
  for (int32_t a = 1; a < n; ++a)
    for (int32_t b = 0; b < a; ++b)
      if (!clear_of(caches[a], bytes, caches[b], bytes)) return false;
  return true;
}

int64_t beam_segments(int32_t vocab) { return ((int64_t)vocab + kSegment - 1) / kSegment; }

// Chunk maxima that a thread holds, in 16-byte pieces.
int beam_pieces(int64_t segments) {
  const int64_t n = (segments * 64 + 4 * kBeamBlock - 1) / (4 * kBeamBlock);
  return n <= 1 ? 1 : (n <= 2 ? 2 : (n <= 4 ? 4 : 16));
}

// Chunks that a row can list: above the k-th largest of the threads' own
// maxima lie those of fewer than k threads, and each wave lists its first k
// that equal it.
int64_t beam_cap(int64_t segments, int32_t k) {
  return (int64_t)(k - 1) * beam_pieces(segments) * 4 + (int64_t)k * (kBeamBlock / 64);
}

struct AttendPlan {
  int32_t query_waves, tile, least, own_sets;
  int64_t strips, shared_wgs, own_splits, own_tiles, own_wgs;
};

// How the work is cut up.  A group's prefix is read once for up to 256 of its
// queries (8 waves of 32).  Groups of up to 32 queries, and all where prefixes
// take up to 2^27 products of a query's 32 (the strips of 32 queries times
// positions, key heads and dim), have a wave for each fourth key tile instead:
// prefixes and own positions are then one launch.  Kernel times of the two forms
// at 2^26, 2^27 and 2^28 products, 8 key heads, 100 own positions: dim 128, 4
// groups of 128 queries 55 / 60, 74 / 71 and 111 / 92 us, 8 of 64 queries 62 / 73,
// 83 / 95 and 137 / 145; dim 64, where exponentials weigh twice as much, 4 groups
// of 128 46 / 46 and 71 / 57 (2^26, 2^27).  With 2048 sequences times key heads or
// more, own positions are a launch of their own either way, and the shared reads
// are ahead from 2^26 on: 32 groups of 128 queries, dim 128, 84 / 77 and 102 / 86
// (2^26, 2^27), dim 64 73 / 63 and 103 / 77.  About 2048 waves in all, so that
// each of the chip's 1024 SIMDs has two.
constexpr int64_t kSetProducts = (int64_t)1 << 27;
bool attend_plan(int32_t groups, int32_t seqs, bool ragged, int32_t next_n, int32_t heads,
                 int32_t kv_heads, int32_t dim, int64_t max_shared, int64_t max_own, AttendPlan& p) {
  const int64_t per = heads / kv_heads, rows = (int64_t)next_n * per;
  const int64_t group_rows = groups > 0 ? (seqs + groups - 1) / groups * rows : 0;
  auto strips = [&](int64_t cols) {
    return ragged ? seqs * rows / cols + groups : groups * ((group_rows + cols - 1) / cols);
  };
  p.query_waves = group_rows > 128 ? 8 : (group_rows > 64 ? 4 : 2);
  const int64_t positions = max_shared * kv_heads;  // (below 2^62)
  if (group_rows <= 32 || positions <= kSetProducts / dim / strips(32)) p.query_waves = 1;
  p.tile = p.query_waves >= 4 ? 64 : 32;
  // (four steps a workgroup at least, where there are: 36 us instead of 40 for
  // one group of 32 sequences over a prefix of 8000; 8 and 16 are slower again)
  p.least = 4;
  p.strips = strips(32 * p.query_waves);
  p.shared_wgs = 0;
  if (groups > 0 && seqs > 0 && max_shared > 0) {
    const int64_t steps = (max_shared + p.tile - 1) / p.tile * p.strips;
    if (steps >= kInt) return false;
    const int64_t most = (steps + p.least - 1) / p.least;
    p.shared_wgs = 2048 / (p.query_waves == 1 ? kOwnSets : p.query_waves) / kv_heads;
    p.shared_wgs = p.shared_wgs < 1 ? 1 : (p.shared_wgs > most ? most : p.shared_wgs);
  }
  p.own_tiles = (rows + 31) / 32;
  p.own_splits = 0;
  const int64_t units = (int64_t)seqs * kv_heads * p.own_tiles;
  // (enough sequences fill the chip with a wave each: 1024 of up to 100
  // positions and 8 key heads, in groups of 16, took 242 us with four waves each
  // and take 201)
  p.own_sets = units >= 2048 ? 1 : kOwnSets;
  if (max_own > 0 && units > 0) {
    const int64_t steps = (max_own + kKeyTile - 1) / kKeyTile, most = (steps + kOwnSets - 1) / kOwnSets;
    p.own_splits = 2048 / kOwnSets / units;
    p.own_splits = p.own_splits < 1 ? 1 : (p.own_splits > most ? most : p.own_splits);
  }
  p.own_wgs = units * p.own_splits;
  return p.shared_wgs * kv_heads + p.own_wgs < kInt;
}

int64_t shared_rows(const AttendPlan& p, int32_t kv_heads) {
  return p.shared_wgs > 0 ? kv_heads * (p.shared_wgs + p.strips) * 32 * p.query_waves : 0;
}

size_t attend_bytes(const AttendPlan& p, int32_t groups, int32_t kv_heads, int64_t rows, int32_t dim) {
  return (size_t)(shared_rows(p, kv_heads) + p.own_splits * rows) * ((size_t)dim * 4 + 8) +
         (size_t)(groups + 1) * sizeof(int4);
}

// What attention and mass share.
struct AttendShape {
  int32_t dtype, groups, seqs, next_n, heads, kv_heads, dim, block_size;
  int64_t num_blocks;
};

bool attend_shape_ok(const AttendShape& s, const int32_t* starts) {
  return (s.dtype == TOPK_DT_BF16 || s.dtype == TOPK_DT_F16) && s.groups >= 0 && s.seqs >= 0 &&
         s.next_n >= 1 && s.next_n <= 1024 && s.heads >= 1 && s.kv_heads >= 1 && s.heads % s.kv_heads == 0 &&
         (s.dim == 64 || s.dim == 128) && s.block_size >= 1 && s.block_size <= (1 << 20) &&
         s.num_blocks >= 0 && s.num_blocks < kInt &&
         (int64_t)s.seqs * s.next_n * s.heads < kInt &&
         (starts || s.groups == 0 || s.seqs % s.groups == 0);
}

bool pages_ok(const void* base, int64_t block, int64_t slot, int64_t head, int64_t num_blocks) {
  return (base || num_blocks == 0) && block >= 0 && block < kInt && slot >= 0 && slot < (1 << 27) && head >= 0 &&
         head < kInt;
}

bool pages_at(const void* base, int64_t block, int64_t slot, int64_t head) {
  return at(base, 16) && block % 8 == 0 && slot % 8 == 0 && head % 8 == 0;
}

Pages pages(const void* base, int64_t block, int64_t slot, int64_t head) {
  return Pages{static_cast<const unsigned char*>(base), (uint32_t)block * 2, (uint32_t)slot * 2, head * 2};
}

int tables_ok(const int32_t* tables, int64_t stride, int32_t width, const int32_t* lens, int32_t rows) {
  if (width < 0 || stride < width || (rows > 0 && (!lens || (width > 0 && !tables)))) return TOPK_EINVAL;
  return at(tables, 4) && at(lens, 4) ? TOPK_OK : TOPK_ELAYOUT;
}

void attend_params(AttendParams& p, const AttendShape& s, const void* q, int64_t q_stride,
                   int64_t q_head_stride, const void* k, int64_t k_block, int64_t k_slot, int64_t k_head,
                   const int32_t* shared_tables, int64_t shared_stride, int32_t shared_width,
                   const int32_t* shared_lens, int64_t shared_limit, const int32_t* starts,
                   const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                   const int32_t* own_lens, int64_t own_limit, float scale) {
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const unsigned char*>(q);
  p.q_stride = q_stride * 2;
  p.q_head_stride = q_head_stride * 2;
  p.k = pages(k, k_block, k_slot, k_head);
  p.num_blocks = s.num_blocks;
  p.block_size = s.block_size;
  p.by_block = quotient_of((uint32_t)s.block_size);
  p.shared = PageTables{shared_tables, shared_stride, shared_width, (int32_t)shared_limit, shared_lens};
  p.own = PageTables{own_tables, own_stride, own_width, (int32_t)own_limit, own_lens};
  p.starts = starts;
  p.groups = s.groups;
  p.seqs = s.seqs;
  p.members = s.groups > 0 ? s.seqs / s.groups : 1;
  p.next_n = s.next_n;
  p.heads = s.heads;
  p.kv_heads = s.kv_heads;
  p.per = s.heads / s.kv_heads;
  // (a scale of zero, too, has to leave -inf where positions are masked)
  p.scale = fmaxf(scale * 1.44269504f, 1e-30f);
  p.rows = (int64_t)s.seqs * s.next_n * s.heads;
}

// The positions that rows of a table can hold, cut to the caller's bound; -1
// if there are too many.
constexpr int64_t kMaxPositions = (int64_t)1 << 30;
int64_t longest_of(int32_t width, int64_t block_size, int64_t num_blocks, int64_t bound) {
  const int64_t most = num_blocks > 0 ? (int64_t)width * block_size : 0;
  if (most > kMaxPositions) return -1;
  return bound > 0 && bound < most ? bound : most;
}

}  // namespace

extern "C" {

size_t topk_beams_workspace_bytes(int32_t num_requests, int32_t beams, int32_t k, int32_t vocab) {
  if (num_requests < 1 || beams < 1 || beams > kMaxBeams || k < 1 || k > kMaxBeamK || vocab < 1 ||
      vocab > kMaxVocab)
    return 0;
  const size_t rows = (size_t)num_requests * beams, seg = (size_t)beam_segments(vocab);
  return rows * (seg * (8 + 4 + 64 * 4) + (size_t)k * sizeof(BeamCandidate)) + (size_t)num_requests * 4 + 16;
}

int topk_beams(const void* logits, int32_t dtype, int64_t row_stride, int32_t vocab, int32_t num_requests,
               int32_t beams, int32_t k, const float* scores, const uint8_t* ended, int32_t end_token,
               const int32_t* lengths, float length_penalty, float* out_scores, int32_t* parents,
               int32_t* tokens, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (num_requests < 0 || beams < 1 || beams > kMaxBeams || k < 1 || k > kMaxBeamK || !dtype_ok(dtype) ||
      vocab < 1 || vocab > kMaxVocab || row_stride < vocab || !isfinite(length_penalty) ||
      (ended && (end_token < 0 || end_token >= vocab)))
    return TOPK_EINVAL;
  if (num_requests == 0) return TOPK_OK;
  if (!logits || !scores || !out_scores || !parents || !tokens) return TOPK_EINVAL;
  if (!at(logits, elem(dtype)) || !at(scores, 4) || !at(lengths, 4) || !at(out_scores, 4) ||
      !at(parents, 4) || !at(tokens, 4) || !at(workspace, 16))
    return TOPK_ELAYOUT;
  const int64_t rows = (int64_t)num_requests * beams, segments = beam_segments(vocab);
  if (rows * segments >= kInt) return TOPK_EINVAL;
  // a request's workgroups read its settings while another's may be done
  const uint64_t in = (uint64_t)rows * 4, out = (uint64_t)num_requests * k * 4;
  const void* outs[] = {out_scores, parents, tokens};
  for (int i = 0; i < 3; ++i) {
    if (!clear_of(outs[i], out, scores, in) || !clear_of(outs[i], out, lengths, in) ||
        !clear_of(outs[i], out, ended, (uint64_t)rows) || !clear_of(outs[i], out, outs[(i + 1) % 3], out))
      return TOPK_EINVAL;
  }
  if (!workspace || workspace_bytes < topk_beams_workspace_bytes(num_requests, beams, k, vocab))
    return TOPK_EWORKSPACE;
  int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  BeamParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.row_stride = row_stride;
  p.vocab = vocab;
  p.rows = (int32_t)rows;
  p.beams = beams;
  p.k = k;
  p.segments = (int32_t)segments;
  p.scores = scores;
  p.ended = ended;
  p.end_token = end_token;
  p.lengths = lengths;
  p.penalty = (double)length_penalty;
  p.out_scores = out_scores;
  p.parents = parents;
  p.tokens = tokens;
  p.found = static_cast<BeamCandidate*>(workspace);
  p.chunks = reinterpret_cast<float*>(p.found + rows * k);
  p.masses = reinterpret_cast<double*>(p.chunks + rows * segments * 64);
  p.bests = reinterpret_cast<float*>(p.masses + rows * segments);
  p.arrived = reinterpret_cast<uint32_t*>(p.bests + rows * segments);
  p.cap = (int32_t)beam_cap(segments, k);
  rc = launch(beam_segment_kernel_ptr(dtype), (rows * segments + 3) / 4, 256, &p, 0, stream);
  if (rc != TOPK_OK) return rc;
  size_t lds = (size_t)p.cap * 8;
  const size_t gather = (size_t)k * kChunk * 8, merge = (size_t)beams * k * 16;
  lds = lds > gather ? lds : gather;
  lds = lds > merge ? lds : merge;
  return launch(beam_row_kernel_ptr(dtype, beam_pieces(segments)), rows, kBeamBlock, &p, lds, stream);
}

int topk_reorder_rows(int32_t num_arrays, const void* const* sources, void* const* targets,
                      const int64_t* source_strides, const int64_t* target_strides,
                      const int64_t* row_bytes, const int32_t* parents, int32_t num_requests,
                      int32_t beams, int32_t k, int32_t clear, hipStream_t stream) {
  if (num_arrays < 0 || num_requests < 0 || beams < 1 || k < 1 || k > kMaxBeams || beams > kMaxBeams ||
      (clear != 0 && clear != 1))
    return TOPK_EINVAL;
  if (num_arrays == 0 || num_requests == 0) return TOPK_OK;
  if (!sources || !targets || !source_strides || !target_strides || !row_bytes || !parents)
    return TOPK_EINVAL;
  if (!at(parents, 4)) return TOPK_ELAYOUT;
  for (int32_t a = 0; a < num_arrays; ++a) {
    const int64_t n = row_bytes[a], ss = source_strides[a], ts = target_strides[a];
    const int64_t rows = (int64_t)num_requests * beams, outs = (int64_t)num_requests * k;
    if (n < 0 || n > ((int64_t)1 << 40) || ss < n || ts < n || ss > ((int64_t)1 << 62) / rows ||
        ts > ((int64_t)1 << 62) / outs)
      return TOPK_EINVAL;
    if (n == 0) continue;
    if (!sources[a] || !targets[a]) return TOPK_EINVAL;
    const uint64_t sb = (uint64_t)((rows - 1) * ss + n), tb = (uint64_t)((outs - 1) * ts + n);
    const bool in_place = sources[a] == targets[a] && ss == ts && beams == k;
    if (!in_place && !clear_of(sources[a], sb, targets[a], tb)) return TOPK_EINVAL;
    if (!clear_of(parents, (uint64_t)outs * 4, targets[a], tb)) return TOPK_EINVAL;
    if ((n + 16 * kCopyBlock - 1) / (16 * kCopyBlock) * num_requests >= kInt) return TOPK_EINVAL;
    // what one array's rows are moved to is no other's source or target
    for (int32_t b = 0; b < num_arrays; ++b) {
      const int64_t m = row_bytes[b];
      if (b == a || m <= 0 || source_strides[b] < m || source_strides[b] > ((int64_t)1 << 62) / rows ||
          target_strides[b] < m || target_strides[b] > ((int64_t)1 << 62) / outs)
        continue;
      if (!rows_clear(sources[b], m, source_strides[b], rows, targets[a], n, ts, outs) ||
          !rows_clear(targets[b], m, target_strides[b], outs, targets[a], n, ts, outs))
        return TOPK_EINVAL;
    }
  }
  int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  ReorderParams p;
  memset(&p, 0, sizeof(p));
  p.parents = parents;
  p.beams = beams;
  p.k = k;
  p.clear = clear;
  int64_t grid = 0;
  auto flush = [&]() -> int {
    if (p.copies == 0) return TOPK_OK;
    const int status = launch(reorder_rows_kernel_ptr(k <= 8 ? 8 : 32), grid, kCopyBlock, &p, 0, stream);
    p.copies = 0;
    grid = 0;
    return status;
  };
  for (int32_t a = 0; a < num_arrays; ++a) {
    if (row_bytes[a] == 0) continue;
    const int64_t tiles = (row_bytes[a] + 16 * kCopyBlock - 1) / (16 * kCopyBlock);
    if (p.copies == kMaxCopies || grid + tiles * num_requests >= kInt) {
      rc = flush();
      if (rc != TOPK_OK) return rc;
    }
    p.copy[p.copies++] = RowCopy{static_cast<const unsigned char*>(sources[a]),
                                 static_cast<unsigned char*>(targets[a]), source_strides[a],
                                 target_strides[a], row_bytes[a], (uint32_t)tiles, (uint32_t)grid};
    grid += tiles * num_requests;
  }
  return flush();
}

int topk_reorder_blocks(const int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                        const int32_t* kv_lens, const int32_t* parents, int32_t num_requests,
                        int32_t beams, int32_t k, int32_t block_size, const int32_t* tail_blocks,
                        int32_t* out_tables, int64_t out_stride, int32_t num_caches, void* const* caches,
                        int64_t num_blocks, int64_t slot_bytes, hipStream_t stream) {
  if (num_requests < 0 || beams < 1 || beams > kMaxBeams || k < 1 || k > kMaxBeams || max_blocks < 0 ||
      table_stride < max_blocks || out_stride < max_blocks || block_size < 1 || block_size > (1 << 20) ||
      num_caches < 0 || num_caches > kMaxCaches || num_blocks < 0 || num_blocks > kInt || slot_bytes < 0 ||
      slot_bytes > ((int64_t)1 << 31) || (!tail_blocks && beams != k))
    return TOPK_EINVAL;
  if (num_requests == 0) return TOPK_OK;
  if (!kv_lens || !parents || (max_blocks > 0 && (!block_tables || !out_tables)) ||
      (num_caches > 0 && !caches))
    return TOPK_EINVAL;
  if (!at(block_tables, 4) || !at(kv_lens, 4) || !at(parents, 4) || !at(tail_blocks, 4) || !at(out_tables, 4))
    return TOPK_ELAYOUT;
  for (int32_t c = 0; c < num_caches; ++c)
    if (!caches[c] && num_blocks > 0 && slot_bytes > 0) return TOPK_EINVAL;
  if (num_caches > 1 && !caches_apart(caches, num_caches, num_blocks, block_size, slot_bytes))
    return TOPK_EINVAL;
  const int64_t rows = (int64_t)num_requests * beams, outs = (int64_t)num_requests * k;
  const bool in_place = block_tables == out_tables && table_stride == out_stride && beams == k;
  const uint64_t out_bytes = max_blocks > 0 ? (uint64_t)((outs - 1) * out_stride + max_blocks) * 4 : 0;
  if (!in_place && max_blocks > 0 &&
      !clear_of(block_tables, (uint64_t)((rows - 1) * table_stride + max_blocks) * 4, out_tables, out_bytes))
    return TOPK_EINVAL;
  if (max_blocks > 0 && (!clear_of(out_tables, out_bytes, parents, (uint64_t)outs * 4) ||
                         !clear_of(out_tables, out_bytes, kv_lens, (uint64_t)num_requests * 4) ||
                         !clear_of(out_tables, out_bytes, tail_blocks, (uint64_t)outs * 4)))
    return TOPK_EINVAL;
  int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  if (max_blocks == 0) return TOPK_OK;
  ReorderBlocksParams p;
  memset(&p, 0, sizeof(p));
  p.parents = parents;
  p.requests = num_requests;
  p.beams = beams;
  p.k = k;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.max_blocks = max_blocks;
  p.out = out_tables;
  p.out_stride = out_stride;
  p.kv_lens = kv_lens;
  p.tail = tail_blocks;
  p.by_block = quotient_of((uint32_t)block_size);
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.slot_bytes = slot_bytes;
  p.block_stride = slot_bytes * block_size;
  p.caches = num_blocks > 0 && slot_bytes > 0 ? num_caches : 0;
  const int64_t tiles = (p.block_stride + 16 * kCopyBlock - 1) / (16 * kCopyBlock);
  p.tiles = (uint32_t)(tiles < 1 ? 1 : (tiles > 64 ? 64 : tiles));
  p.table_tiles = (uint32_t)((max_blocks + kCopyBlock - 1) / kCopyBlock);
  for (int32_t c = 0; c < p.caches; ++c) p.cache[c] = static_cast<unsigned char*>(caches[c]);
  const int64_t copying = (int64_t)p.caches * num_requests * p.tiles;
  const int64_t making = (int64_t)num_requests * p.table_tiles;
  if (copying + making >= kInt) return TOPK_EINVAL;
  const void* kernel = reorder_blocks_kernel_ptr(k <= 8 ? 8 : 32);
  p.copying = copying > 0 ? 1 : 0;
  // In place, given blocks take the place of the table entries that say where
  // the parents' open blocks lie: copied first, then written.
  if (in_place && tail_blocks && copying > 0) {
    rc = launch(kernel, copying, kCopyBlock, &p, 0, stream);
    if (rc != TOPK_OK) return rc;
    p.copying = 0;
  }
  return launch(kernel, (p.copying ? copying : 0) + making, kCopyBlock, &p, 0, stream);
}

size_t topk_attend_workspace_bytes(int32_t num_groups, int32_t num_seqs, int32_t ragged, int32_t next_n,
                                   int32_t num_heads, int32_t num_kv_heads, int32_t dim,
                                   int64_t max_shared_len, int64_t max_own_len) {
  if (num_groups < 0 || num_seqs < 1 || next_n < 1 || num_heads < 1 || num_kv_heads < 1 ||
      num_heads % num_kv_heads || (dim != 64 && dim != 128) || max_shared_len < 0 || max_own_len < 0 ||
      (int64_t)num_seqs * next_n >= kInt || (int64_t)num_seqs * next_n * num_heads >= kInt ||
      max_shared_len > kInt || max_own_len > kInt)
    return 0;
  AttendPlan plan;
  if (!attend_plan(num_groups, num_seqs, ragged != 0, next_n, num_heads, num_kv_heads, dim, max_shared_len,
                   max_own_len, plan))
    return 0;
  return attend_bytes(plan, num_groups, num_kv_heads, (int64_t)num_seqs * next_n * num_heads, dim);
}

int topk_attend(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride, int32_t num_seqs,
                int32_t next_n, int32_t num_heads, int32_t num_kv_heads, int32_t dim, const void* k_cache,
                int64_t k_block_stride, int64_t k_slot_stride, int64_t k_head_stride, const void* v_cache,
                int64_t v_block_stride, int64_t v_slot_stride, int64_t v_head_stride, int64_t num_blocks,
                int32_t block_size, const int32_t* shared_tables, int64_t shared_stride,
                int32_t shared_width, const int32_t* shared_lens, const int32_t* group_starts,
                int32_t num_groups, const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                const int32_t* own_lens, float scale, int64_t max_shared_len, int64_t max_own_len,
                void* out, float* lse, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  const AttendShape s{dtype, num_groups, num_seqs, next_n, num_heads, num_kv_heads, dim, block_size, num_blocks};
  if (!attend_shape_ok(s, group_starts) || !(scale >= 0.0f) || isinf(scale) || q_stride < 0 || q_head_stride < 0 ||
      max_shared_len < 0 || max_own_len < 0)
    return TOPK_EINVAL;
  if (num_seqs == 0) return TOPK_OK;
  if (!q || !out || !pages_ok(k_cache, k_block_stride, k_slot_stride, k_head_stride, num_blocks) ||
      !pages_ok(v_cache, v_block_stride, v_slot_stride, v_head_stride, num_blocks))
    return TOPK_EINVAL;
  if (!at(q, 16) || q_stride % 8 || q_head_stride % 8 || !at(out, 16) || !at(lse, 4) || !at(group_starts, 4) ||
      !pages_at(k_cache, k_block_stride, k_slot_stride, k_head_stride) ||
      !pages_at(v_cache, v_block_stride, v_slot_stride, v_head_stride) || !at(workspace, 16))
    return TOPK_ELAYOUT;
  int rc = tables_ok(shared_tables, shared_stride, shared_width, shared_lens, num_groups);
  if (rc != TOPK_OK) return rc;
  rc = tables_ok(own_tables, own_stride, own_width, own_lens, num_seqs);
  if (rc != TOPK_OK) return rc;
  const int64_t most_shared = longest_of(num_groups > 0 ? shared_width : 0, block_size, num_blocks, max_shared_len);
  const int64_t most_own = longest_of(own_width, block_size, num_blocks, max_own_len);
  AttendPlan plan;
  if (most_shared < 0 || most_own < 0 ||
      !attend_plan(num_groups, num_seqs, group_starts != nullptr, next_n, num_heads, num_kv_heads, dim,
                   most_shared, most_own, plan))
    return TOPK_EINVAL;
  const int64_t rows = (int64_t)num_seqs * next_n * num_heads;
  if (!workspace || workspace_bytes < attend_bytes(plan, num_groups, num_kv_heads, rows, dim)) return TOPK_EWORKSPACE;
  rc = device_ok();
  if (rc != TOPK_OK) return rc;
  AttendParams p;
  attend_params(p, s, q, q_stride, q_head_stride, k_cache, k_block_stride, k_slot_stride, k_head_stride,
                shared_tables, shared_stride, shared_width, shared_lens, most_shared, group_starts, own_tables,
                own_stride, own_width, own_lens, most_own, scale);
  p.v = pages(v_cache, v_block_stride, v_slot_stride, v_head_stride);
  p.query_waves = plan.query_waves;
  p.shared_tile = plan.tile;
  p.shared_least = plan.least;
  p.shared_wgs = (int32_t)plan.shared_wgs;
  p.strips = (int32_t)plan.strips;
  p.own_splits = (int32_t)plan.own_splits;
  p.own_tiles = (int32_t)plan.own_tiles;
  const int64_t shared = shared_rows(plan, num_kv_heads), own = plan.own_splits * rows;
  p.group_at = static_cast<int4*>(workspace);
  p.shared_parts = reinterpret_cast<float*>(p.group_at + num_groups + 1);
  p.own_parts = p.shared_parts + shared * dim;
  p.shared_stats = reinterpret_cast<float2*>(p.own_parts + own * dim);
  p.own_stats = p.shared_stats + shared;
  p.out = static_cast<unsigned char*>(out);
  p.lse = lse;
  p.shared_grid = plan.shared_wgs * num_kv_heads;
  const bool together = plan.query_waves == 1 && plan.own_sets == kOwnSets;
  const int64_t first = p.shared_grid + (together ? plan.own_wgs : 0);
  if (first > 0) {
    const int sets = plan.query_waves == 1 ? kOwnSets : 1;
    rc = launch(attend_kernel_ptr(dtype, dim, plan.query_waves, sets, block_size), first,
                64 * plan.query_waves * sets, &p, 0, stream);
    if (rc != TOPK_OK) return rc;
  }
  if (!together && plan.own_wgs > 0) {
    p.shared_grid = 0;
    rc = launch(attend_kernel_ptr(dtype, dim, 1, plan.own_sets, block_size), plan.own_wgs, 64 * plan.own_sets, &p, 0,
                stream);
    if (rc != TOPK_OK) return rc;
  }
  return launch(attend_join_kernel_ptr(dtype, dim), (rows + 3) / 4, 256, &p, 0, stream);
}

int topk_attend_mass_bounded(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride, int32_t num_seqs,
                             int32_t next_n, int32_t num_heads, int32_t num_kv_heads, int32_t dim, const void* k_cache,
                             int64_t k_block_stride, int64_t k_slot_stride, int64_t k_head_stride, int64_t num_blocks,
                             int32_t block_size, const int32_t* shared_tables, int64_t shared_stride,
                             int32_t shared_width, const int32_t* shared_lens, const int32_t* group_starts,
                             int32_t num_groups, const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                             const int32_t* own_lens, float scale, int64_t max_shared_len, int64_t max_own_len,
                             const float* lse, float decay, const float* shared_mass, float* shared_out,
                             int32_t shared_positions, const float* own_mass, float* own_out, int32_t own_positions,
                             hipStream_t stream) {
  const AttendShape s{dtype, num_groups, num_seqs, next_n, num_heads, num_kv_heads, dim, block_size, num_blocks};
  if (!attend_shape_ok(s, group_starts) || !(scale >= 0.0f) || isinf(scale) || q_stride < 0 || q_head_stride < 0 ||
      max_shared_len < 0 || max_own_len < 0 || !isfinite(decay) || shared_positions < 0 || shared_positions > kMaxPositions || own_positions < 0 ||
      own_positions > kMaxPositions)
    return TOPK_EINVAL;
  if (num_seqs > 0 && (!q || !lse)) return TOPK_EINVAL;
  if (!pages_ok(k_cache, k_block_stride, k_slot_stride, k_head_stride, num_blocks)) return TOPK_EINVAL;
  const uint64_t sb = (uint64_t)num_groups * num_kv_heads * shared_positions * 4;
  const uint64_t ob = (uint64_t)num_seqs * num_kv_heads * own_positions * 4;
  const uint64_t lb = (uint64_t)num_seqs * next_n * num_heads * 4;
  if ((sb > 0 && !shared_out) || (ob > 0 && !own_out)) return TOPK_EINVAL;
  if (!at(q, 16) || q_stride % 8 || q_head_stride % 8 || !at(lse, 4) || !at(group_starts, 4) ||
      !at(shared_mass, 4) || !at(shared_out, 4) || !at(own_mass, 4) || !at(own_out, 4) ||
      !pages_at(k_cache, k_block_stride, k_slot_stride, k_head_stride))
    return TOPK_ELAYOUT;
  if ((shared_mass != shared_out && !clear_of(shared_mass, sb, shared_out, sb)) ||
      (own_mass != own_out && !clear_of(own_mass, ob, own_out, ob)) || !clear_of(shared_out, sb, own_out, ob) ||
      !clear_of(shared_out, sb, own_mass, ob) || !clear_of(own_out, ob, shared_mass, sb) ||
      !clear_of(shared_out, sb, lse, lb) || !clear_of(own_out, ob, lse, lb))
    return TOPK_EINVAL;
  int rc = tables_ok(shared_tables, shared_stride, shared_width, shared_lens, num_groups);
  if (rc != TOPK_OK) return rc;
  rc = tables_ok(own_tables, own_stride, own_width, own_lens, num_seqs);
  if (rc != TOPK_OK) return rc;
  const int64_t most_shared = longest_of(num_groups > 0 ? shared_width : 0, block_size, num_blocks, max_shared_len);
  const int64_t most_own = longest_of(own_width, block_size, num_blocks, max_own_len);
  if (most_shared < 0 || most_own < 0) return TOPK_EINVAL;
  const int64_t shared_tiles = ((int64_t)shared_positions + kMassStep - 1) / kMassStep;
  const int64_t own_tiles = ((int64_t)own_positions + kMassStep - 1) / kMassStep;
  const int64_t shared_wgs = shared_tiles * num_groups * num_kv_heads;
  const int64_t own_wgs = own_tiles * num_seqs * num_kv_heads;
  if (shared_wgs + own_wgs >= kInt) return TOPK_EINVAL;
  if (shared_wgs + own_wgs == 0) return TOPK_OK;
  rc = device_ok();
  if (rc != TOPK_OK) return rc;
  MassParams p;
  attend_params(p.a, s, q, q_stride, q_head_stride, k_cache, k_block_stride, k_slot_stride, k_head_stride,
                shared_tables, shared_stride, shared_width, shared_lens, most_shared, group_starts, own_tables,
                own_stride, own_width, own_lens, most_own, scale);
  p.lse = lse;
  p.shared_in = shared_mass;
  p.shared_out = shared_out;
  p.shared_width = shared_positions;
  p.own_in = own_mass;
  p.own_out = own_out;
  p.own_width = own_positions;
  p.decay = decay;
  p.shared_tiles = (int32_t)shared_tiles;
  p.own_tiles = (int32_t)own_tiles;
  p.shared_wgs = shared_wgs;
  return launch(attend_mass_kernel_ptr(dtype, dim), shared_wgs + own_wgs, kMassBlock, &p, 0, stream);
}

int topk_attend_mass(const void* q, int32_t dtype, int64_t q_stride, int64_t q_head_stride, int32_t num_seqs,
                     int32_t next_n, int32_t num_heads, int32_t num_kv_heads, int32_t dim, const void* k_cache,
                     int64_t k_block_stride, int64_t k_slot_stride, int64_t k_head_stride, int64_t num_blocks,
                     int32_t block_size, const int32_t* shared_tables, int64_t shared_stride,
                     int32_t shared_width, const int32_t* shared_lens, const int32_t* group_starts,
                     int32_t num_groups, const int32_t* own_tables, int64_t own_stride, int32_t own_width,
                     const int32_t* own_lens, float scale, const float* lse, float decay,
                     const float* shared_mass, float* shared_out, int32_t shared_positions,
                     const float* own_mass, float* own_out, int32_t own_positions, hipStream_t stream) {
  return topk_attend_mass_bounded(q, dtype, q_stride, q_head_stride, num_seqs, next_n, num_heads, num_kv_heads, dim,
                                  k_cache, k_block_stride, k_slot_stride, k_head_stride, num_blocks, block_size,
                                  shared_tables, shared_stride, shared_width, shared_lens, group_starts, num_groups,
                                  own_tables, own_stride, own_width, own_lens, scale, 0, 0, lse, decay, shared_mass,
                                  shared_out, shared_positions, own_mass, own_out, own_positions, stream);
}

int topk_evict_keep(const float* mass, int64_t request_stride, int64_t head_stride, int32_t positions,
                    int32_t num_requests, int32_t num_heads, const int32_t* kv_lens, int32_t budget,
                    int32_t sinks, int32_t recent, int32_t* kept, float* mass_out, int32_t out_positions,
                    int32_t* new_lens, hipStream_t stream) {
  if (num_requests < 0 || num_heads < 1 || positions < 0 || request_stride < 0 || head_stride < 0 ||
      budget < 1 || sinks < 0 || recent < 0 || (int64_t)sinks + recent > budget ||
      (mass_out && out_positions < budget) || positions > (1 << 30) || budget > (1 << 30) ||
      (int64_t)num_requests * num_heads >= kInt)
    return TOPK_EINVAL;
  if (num_requests == 0) return TOPK_OK;
  if ((!mass && positions > 0) || !kv_lens || !kept || !new_lens || kv_lens == new_lens) return TOPK_EINVAL;
  if (!at(mass, 4) || !at(kv_lens, 4) || !at(kept, 4) || !at(mass_out, 4) || !at(new_lens, 4)) return TOPK_ELAYOUT;
  const int64_t rows = (int64_t)num_requests * num_heads;
  const uint64_t in = positions > 0 ? (uint64_t)((num_requests - 1) * request_stride + (num_heads - 1) * head_stride + positions) * 4 : 0;
  const uint64_t kb = (uint64_t)rows * budget * 4, mb = (uint64_t)rows * out_positions * 4, nb = (uint64_t)num_requests * 4;
  if (!clear_of(mass, in, kept, kb) || !clear_of(mass, in, mass_out, mb) || !clear_of(mass, in, new_lens, nb) ||
      !clear_of(kv_lens, nb, kept, kb) || !clear_of(kv_lens, nb, mass_out, mb) || !clear_of(kv_lens, nb, new_lens, nb) ||
      !clear_of(kept, kb, mass_out, mb) || !clear_of(kept, kb, new_lens, nb) || !clear_of(mass_out, mb, new_lens, nb))
    return TOPK_EINVAL;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  KeepParams p;
  memset(&p, 0, sizeof(p));
  p.mass = mass;
  p.request_stride = request_stride;
  p.head_stride = head_stride;
  p.positions = positions;
  p.heads = num_heads;
  p.kv_lens = kv_lens;
  p.budget = budget;
  p.sinks = sinks;
  p.recent = recent;
  p.kept = kept;
  p.mass_out = mass_out;
  p.out_positions = out_positions;
  p.new_lens = new_lens;
  return launch(evict_keep_kernel_ptr(positions), rows, kKeepBlock, &p, 0, stream);
}

int topk_evict_move(const int32_t* kept, int32_t num_requests, int32_t num_heads, int32_t budget,
                    const int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                    const int32_t* out_tables, int64_t out_stride, int32_t out_blocks, int32_t block_size,
                    int32_t num_caches, void* const* caches, int64_t num_blocks, int64_t slot_bytes,
                    hipStream_t stream) {
  if (num_requests < 0 || num_heads < 1 || budget < 1 || budget > (1 << 30) || max_blocks < 0 || table_stride < max_blocks ||
      out_blocks < 0 || out_stride < out_blocks || block_size < 1 || block_size > (1 << 20) || num_caches < 0 ||
      num_caches > kMaxCaches || num_blocks < 0 || num_blocks > kInt || slot_bytes < 0 ||
      slot_bytes > ((int64_t)1 << 31) || slot_bytes % num_heads || (slot_bytes / num_heads) % 16)
    return TOPK_EINVAL;
  if (num_requests == 0 || num_caches == 0 || slot_bytes == 0 || num_blocks == 0) return TOPK_OK;
  if (!kept || !caches || (max_blocks > 0 && !block_tables) || (out_blocks > 0 && !out_tables) ||
      (block_tables == out_tables && table_stride != out_stride && num_requests > 1))
    return TOPK_EINVAL;
  if (!at(kept, 4) || !at(block_tables, 4) || !at(out_tables, 4)) return TOPK_ELAYOUT;
  for (int32_t c = 0; c < num_caches; ++c) {
    if (!caches[c]) return TOPK_EINVAL;
    if (!at(caches[c], 16)) return TOPK_ELAYOUT;
  }
  if (!caches_apart(caches, num_caches, num_blocks, block_size, slot_bytes)) return TOPK_EINVAL;
  if (max_blocks == 0 || out_blocks == 0) return TOPK_OK;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  MoveParams p;
  memset(&p, 0, sizeof(p));
  p.kept = kept;
  p.requests = num_requests;
  p.heads = num_heads;
  p.budget = budget;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.max_blocks = max_blocks;
  p.out_tables = out_tables;
  p.out_stride = out_stride;
  p.out_blocks = out_blocks;
  p.by_block = quotient_of((uint32_t)block_size);
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.slot_bytes = slot_bytes;
  p.row_bytes = slot_bytes / num_heads;
  p.caches = num_caches;
  for (int32_t c = 0; c < num_caches; ++c) p.cache[c] = static_cast<unsigned char*>(caches[c]);
  // Other bytes of a row are another workgroup's, 256 of them at least; rows
  // are split too where targets are not sources.
  const int64_t rows = (int64_t)num_caches * num_requests * num_heads;
  const int64_t pieces = p.row_bytes / 16;
  int64_t columns = (pieces + 15) / 16;
  while (columns > 1 && rows * columns > 4096) columns = (columns + 1) / 2;
  p.columns = (int32_t)columns;
  int64_t parts = 1;
  const bool in_place = block_tables == out_tables;
  if (!in_place) {
    parts = 8192 / (rows * columns);
    const int64_t most = ((int64_t)budget + 63) / 64;
    parts = parts < 1 ? 1 : (parts > most ? most : parts);
  }
  p.parts = (int32_t)parts;
  return launch(evict_move_kernel_ptr(in_place), rows * columns * parts, kMoveBlock, &p, 0, stream);
}

}  // extern "C"
