// rowops_abi.cpp -- C ABI of the row operators beside the selection: host-side
// validation (no device reads) and the kernel launches.  The contract is
// documented in include/exact_row_top.h.

#include <hip/hip_runtime.h>

#include <string.h>

#include "exact_row_top.h"
#include "rowops.h"
#include "rowops_host.h"

namespace ert {
const void* sample_segment_kernel_ptr(int dtype, bool cuts);
const void* sample_row_kernel_ptr(int dtype);
const void* sample_wide_kernel_ptr(int dtype);
const void* route_kernel_ptr(int dtype, int lanes, int per_lane);
const void* route_grad_kernel_ptr(int dtype, int lanes, int per_lane);
const void* block_table_kernel_ptr(int per_thread);
const void* topk_slots_kernel_ptr();
}  // namespace ert

using namespace ert;

namespace {

// Segments of a row whose first score may lie up to one 16-byte group past
// an aligned boundary.
int64_t segments_of(int32_t vocab) { return ((int64_t)vocab + 7 + kSegment - 1) / kSegment; }

int64_t wide_wgs_of(int64_t segments) { return (segments + kWideSegs - 1) / kWideSegs; }

bool route_shape_ok(int32_t tokens, int32_t experts, int32_t top_k) {
  return tokens >= 0 && experts >= 1 && experts <= kMaxExperts && top_k >= 1 && top_k <= kMaxRouteK &&
         top_k <= experts;
}

Divisor divisor(uint32_t d) {
  uint32_t log = 0;
  while (((uint64_t)1 << log) < d) ++log;
  if (((uint64_t)1 << log) == d) return Divisor{0, log};
  return Divisor{(uint32_t)((((uint64_t)1 << (31 + log)) + d - 1) / d), log - 1};
}

// How a token's experts are spread: 16 lanes up to 256 experts (four tokens a
// wave share each step of the selection), a whole wave above.
struct Spread {
  int lanes, per_lane;
};
Spread route_spread(int experts, int vec) {
  Spread s{experts <= 256 ? 16 : 64, vec};
  while (s.per_lane * s.lanes < experts || (s.lanes == 64 && s.per_lane < 16)) s.per_lane *= 2;
  return s;
}

}  // namespace

extern "C" {

size_t topk_sample_workspace_bytes(int32_t num_rows, int32_t vocab) {
  if (num_rows < 1 || vocab < 1 || vocab > kMaxVocab) return 0;
  const size_t seg = (size_t)segments_of(vocab);
  return (size_t)num_rows * (seg * (sizeof(SegRecord) + kSegSlots * sizeof(Candidate) + 8) +
                             wide_wgs_of(seg) * (kBinsS * 12 + 8) + sizeof(WideRow));
}

int topk_sample(const void* logits, int32_t dtype, int64_t row_stride, int32_t vocab,
                int32_t num_rows, const float* uniforms, const float* temperature,
                const int32_t* top_k, const float* top_p, const float* min_p, int32_t* tokens,
                float* logprobs, uint32_t flags, void* workspace, size_t workspace_bytes,
                hipStream_t stream) {
  if (num_rows < 0 || !dtype_ok(dtype) || vocab < 1 || vocab > kMaxVocab || row_stride < vocab ||
      (flags & ~(uint32_t)TOPK_SAMPLE_WHOLE_ROW))
    return TOPK_EINVAL;
  if (num_rows == 0) return TOPK_OK;
  if (!logits || !uniforms || !tokens) return TOPK_EINVAL;
  if (!at(logits, elem(dtype)) || !at(uniforms, 4) || !at(temperature, 4) || !at(top_k, 4) ||
      !at(top_p, 4) || !at(min_p, 4) || !at(tokens, 4) || !at(logprobs, 4) || !at(workspace, 16))
    return TOPK_ELAYOUT;
  // a row's workgroups read its settings while one of them may be done
  const void* settings[] = {uniforms, temperature, top_k, top_p, min_p};
  bool clear = apart(tokens, logprobs, (uint64_t)num_rows * 4);
  for (const void* in : settings)
    clear = clear && apart(in, tokens, (uint64_t)num_rows * 4) && apart(in, logprobs, (uint64_t)num_rows * 4);
  if (!clear) return TOPK_EINVAL;
  const int64_t segments = segments_of(vocab);
  const int64_t waves = segments * num_rows;
  if (waves >= ((int64_t)1 << 31)) return TOPK_EINVAL;
  if (!workspace || workspace_bytes < topk_sample_workspace_bytes(num_rows, vocab))
    return TOPK_EWORKSPACE;
  int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  SampleParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.row_stride = row_stride;
  p.vocab = vocab;
  p.rows = num_rows;
  p.segments = (int32_t)segments;
  p.uniforms = uniforms;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.tokens = tokens;
  p.logprobs = logprobs;
  // the row's settings alone say whether it has a cut; without any, no row has
  const bool cuts = top_k || top_p || min_p;
  const bool whole = (flags & TOPK_SAMPLE_WHOLE_ROW) != 0;
  const int64_t wgs = wide_wgs_of(segments);
  p.records = static_cast<SegRecord*>(workspace);
  p.candidates = reinterpret_cast<Candidate*>(p.records + waves);
  p.kept = reinterpret_cast<uint64_t*>(p.candidates + waves * kSegSlots);
  p.masses = p.kept + waves + num_rows * wgs;
  p.counts = reinterpret_cast<uint32_t*>(p.masses + num_rows * wgs * kBinsS);
  p.wide = (cuts || whole) ? reinterpret_cast<WideRow*>(p.counts + num_rows * wgs * kBinsS) : nullptr;
  p.wide_wgs = (int32_t)wgs;
  p.row_wgs = (top_k || top_p) && !whole ? (int32_t)wgs : 1;
  p.whole_row = whole ? 1 : 0;
  rc = launch(sample_segment_kernel_ptr(dtype, cuts || whole), (waves + 3) / 4, 256, &p, 0, stream);
  if (rc == TOPK_OK)
    rc = launch(sample_row_kernel_ptr(dtype), num_rows * p.row_wgs, kRowBlock, &p, 0, stream);
  if (rc == TOPK_OK && (cuts || whole))
    rc = launch(sample_wide_kernel_ptr(dtype), num_rows * wgs, kWideBlock, &p, 0, stream);
  return rc;
}

int topk_route(const void* logits, int32_t dtype, int64_t row_stride, int32_t num_tokens,
               int32_t num_experts, int32_t top_k, const float* bias, int32_t num_groups,
               int32_t topk_groups, uint32_t flags, float scale, int32_t* indices, float* weights,
               hipStream_t stream) {
  if (!route_shape_ok(num_tokens, num_experts, top_k) || !dtype_ok(dtype) ||
      row_stride < num_experts || num_groups < 1 || num_groups > kMaxGroups ||
      num_experts % num_groups || topk_groups < 1 || topk_groups > num_groups ||
      (flags & ~(uint32_t)(TOPK_ROUTE_SIGMOID | TOPK_ROUTE_TOP2 | TOPK_ROUTE_RENORMALIZE)))
    return TOPK_EINVAL;
  if (num_tokens == 0) return TOPK_OK;
  if (!logits || !indices || !weights) return TOPK_EINVAL;
  if (!at(logits, elem(dtype)) || !at(bias, 4) || !at(indices, 4) || !at(weights, 4))
    return TOPK_ELAYOUT;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  RouteParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.row_stride = row_stride;
  p.tokens = num_tokens;
  p.experts = num_experts;
  p.top_k = top_k;
  p.sigmoid = (flags & TOPK_ROUTE_SIGMOID) ? 1 : 0;
  p.bias = bias;
  p.groups = num_groups;
  p.group_size = num_experts / num_groups;
  // exact for e < 1024 with sizes of 2 and more: the quotient's error, below
  // e / 2^32, is less than the 1 / size to the next whole number
  p.group_magic = p.group_size > 1 ? (uint32_t)((((uint64_t)1 << 32) + p.group_size - 1) / p.group_size) : 0;
  p.topk_groups = topk_groups;
  p.top2 = (flags & TOPK_ROUTE_TOP2) ? 1 : 0;
  p.renormalize = (flags & TOPK_ROUTE_RENORMALIZE) ? 1 : 0;
  p.scale = scale;
  p.indices = indices;
  p.weights = weights;
  const int vec = dtype == TOPK_DT_F32 ? 4 : 8;
  p.vector = at(logits, 16) && (num_tokens == 1 || row_stride % vec == 0) && num_experts % vec == 0;
  p.vector_bias = bias && at(bias, 16) && num_experts % 4 == 0;
  const Spread sp = route_spread(num_experts, vec);
  while ((num_groups << (p.group_lanes + 1)) <= sp.lanes) ++p.group_lanes;
  const int per = 256 / sp.lanes;
  // the groups' scores go through LDS
  return launch(route_kernel_ptr(dtype, sp.lanes, sp.per_lane),
                ((int64_t)num_tokens + per - 1) / per, 256, &p,
                num_groups > 1 ? (size_t)per * num_experts * sizeof(double) : 0, stream);
}

int topk_route_backward(const void* logits, int32_t dtype, int64_t row_stride, int32_t num_tokens,
                        int32_t num_experts, int32_t top_k, uint32_t flags, float scale,
                        const int32_t* indices, const float* grad_weights, void* grad_logits,
                        int64_t grad_row_stride, hipStream_t stream) {
  if (!route_shape_ok(num_tokens, num_experts, top_k) || !dtype_ok(dtype) ||
      row_stride < num_experts || grad_row_stride < num_experts ||
      (flags & ~(uint32_t)(TOPK_ROUTE_SIGMOID | TOPK_ROUTE_TOP2 | TOPK_ROUTE_RENORMALIZE)))
    return TOPK_EINVAL;
  if (num_tokens == 0) return TOPK_OK;
  if (!logits || !indices || !grad_weights || !grad_logits) return TOPK_EINVAL;
  if (!at(logits, elem(dtype)) || !at(indices, 4) || !at(grad_weights, 4) ||
      !at(grad_logits, elem(dtype)))
    return TOPK_ELAYOUT;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  RouteGradParams p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.row_stride = row_stride;
  p.tokens = num_tokens;
  p.experts = num_experts;
  p.top_k = top_k;
  p.sigmoid = (flags & TOPK_ROUTE_SIGMOID) ? 1 : 0;
  p.renormalize = (flags & TOPK_ROUTE_RENORMALIZE) ? 1 : 0;
  p.scale = scale;
  p.indices = indices;
  p.grad_weights = grad_weights;
  p.grad_logits = grad_logits;
  p.grad_stride = grad_row_stride;
  const int vec = dtype == TOPK_DT_F32 ? 4 : 8;
  p.vector = at(logits, 16) && at(grad_logits, 16) && num_experts % vec == 0 &&
             (num_tokens == 1 || (row_stride % vec == 0 && grad_row_stride % vec == 0));
  const Spread sp = route_spread(num_experts, vec);
  const int per = 256 / sp.lanes;
  return launch(route_grad_kernel_ptr(dtype, sp.lanes, sp.per_lane),
                ((int64_t)num_tokens + per - 1) / per, 256, &p,
                (size_t)256 * sp.per_lane * sizeof(float), stream);
}

int topk_block_tables(int32_t* block_tables, int64_t table_stride, int32_t max_blocks,
                      int32_t num_requests, const int32_t* kv_lens, const int32_t* new_tokens,
                      const int32_t* free_blocks, int64_t num_free, const int32_t* free_start,
                      int32_t block_size, int64_t max_tokens, int32_t* token_starts,
                      int32_t* token_requests, int32_t* positions, void* slots, int32_t slots_64,
                      int32_t* free_next, hipStream_t stream) {
  if (num_requests < 0 || num_requests > kMaxRequests || max_blocks < 0 ||
      table_stride < max_blocks || num_free < 0 || block_size < 1 || block_size > (1 << 30) ||
      max_tokens < 0 || max_tokens >= ((int64_t)1 << 31) || (slots_64 != 0 && slots_64 != 1))
    return TOPK_EINVAL;
  if (!free_start || !free_next || free_start == free_next || !token_starts) return TOPK_EINVAL;
  if (num_requests > 0 && (!kv_lens || !new_tokens || (max_blocks > 0 && !block_tables)))
    return TOPK_EINVAL;
  if (num_free > 0 && !free_blocks) return TOPK_EINVAL;
  if (max_tokens > 0 && (!token_requests || !positions || !slots)) return TOPK_EINVAL;
  if (!at(block_tables, 4) || !at(kv_lens, 4) || !at(new_tokens, 4) || !at(free_blocks, 4) ||
      !at(free_start, 4) || !at(token_starts, 4) || !at(token_requests, 4) || !at(positions, 4) ||
      !at(slots, slots_64 ? 8 : 4) || !at(free_next, 4))
    return TOPK_ELAYOUT;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  TableParams p;
  memset(&p, 0, sizeof(p));
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.max_blocks = max_blocks;
  p.requests = num_requests;
  p.kv_lens = kv_lens;
  p.new_tokens = new_tokens;
  p.free_blocks = free_blocks;
  p.num_free = num_free;
  p.free_start = free_start;
  p.block_size = block_size;
  p.max_tokens = max_tokens;
  p.token_starts = token_starts;
  p.token_requests = token_requests;
  p.positions = positions;
  p.slots = slots;
  p.wide = slots_64;
  p.free_next = free_next;
  p.by_block = divisor((uint32_t)block_size);
  p.vector = at(token_requests, 16) && at(positions, 16) && at(slots, 16);
  // Four tokens a thread once 1024 workgroups of single ones are full (one
  // behind the other in a graph, a million tokens: 7.2 us against 7.8; 244000:
  // 5.3 either way; 32768: 4.8 against 3.9; 64: 5.0 against 3.6); beyond 1024
  // workgroups another round costs less than another workgroup's sums over the
  // requests.
  const int per_thread = max_tokens > 1024 * kSlotBlock ? 4 : 1;
  int64_t grid = (max_tokens + kSlotBlock * per_thread - 1) / (kSlotBlock * per_thread);
  grid = grid < 1 ? 1 : (grid > 1024 ? 1024 : grid);
  return launch(block_table_kernel_ptr(per_thread), grid, kSlotBlock, &p,
                (size_t)(3 * num_requests + 1) * 4, stream);
}

int topk_slots(const int32_t* indices, int64_t num_rows, int32_t k, const int32_t* block_tables,
               int64_t table_stride, int32_t max_blocks, int32_t num_requests,
               const int32_t* row_requests, int32_t next_n, int32_t block_size, void* slots,
               int32_t slots_64, hipStream_t stream) {
  if (num_rows < 0 || num_rows >= ((int64_t)1 << 31) || k < 1 || max_blocks < 0 ||
      table_stride < max_blocks || num_requests < 0 || block_size < 1 || block_size > (1 << 30) ||
      (slots_64 != 0 && slots_64 != 1) || (!row_requests && next_n < 1))
    return TOPK_EINVAL;
  if (num_rows == 0) return TOPK_OK;
  if (!indices || !slots || (num_requests > 0 && max_blocks > 0 && !block_tables)) return TOPK_EINVAL;
  if (slots_64 && slots == indices) return TOPK_EINVAL;
  if (!at(indices, 4) || !at(block_tables, 4) || !at(row_requests, 4) || !at(slots, slots_64 ? 8 : 4))
    return TOPK_ELAYOUT;
  const int rc = device_ok();
  if (rc != TOPK_OK) return rc;
  SlotParams p;
  memset(&p, 0, sizeof(p));
  p.indices = indices;
  p.rows = num_rows;
  p.k = k;
  p.tables = block_tables;
  p.table_stride = table_stride;
  p.max_blocks = max_blocks;
  p.requests = num_requests;
  p.row_requests = row_requests;
  p.next_n = row_requests ? 1 : next_n;
  p.block_size = block_size;
  p.slots = slots;
  p.wide = slots_64;
  p.by_block = divisor((uint32_t)block_size);
  p.vector = k % 4 == 0 && at(indices, 16) && at(slots, 16);
  p.parts = (int32_t)(((int64_t)k + kSlotPart - 1) / kSlotPart);
  // Where a part maps at least twice as many positions as its table has
  // entries, and workgroups hide the copy's latency: 4096 rows of 2048 over
  // 256 entries 13.4 us against 16.0, 4096 x 1024 over 512 8.7 against 9.1,
  // 512 x 1024 over 256 2.87 against 2.99; 4096 x 1024 over 1000 10.4 either
  // way, 64 x 1024 over 1000 2.8 against 2.55.
  p.staged = 2 * (int64_t)max_blocks <= (k < kSlotPart ? k : kSlotPart) && num_rows * p.parts >= 512;
  return launch(topk_slots_kernel_ptr(), num_rows * p.parts, kSlotBlock, &p,
                p.staged ? (size_t)max_blocks * 4 : 0, stream);
}

}  // extern "C"
