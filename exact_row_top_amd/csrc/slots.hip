// slots.hip -- block tables and slot maps of a paged cache, made on the device
// from request lengths, and the slots of selected positions.
//
// A request's cache of n tokens lies in ceil(n / block_size) blocks; entry b
// of its block table names the block of positions [b * block_size, (b + 1) *
// block_size), and position p has the slot table[p / block_size] * block_size
// + p % block_size.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rowops.h"

namespace ert {

namespace {

constexpr int kSlotBlock = 256;

__device__ __forceinline__ int64_t slot_of(int32_t block, uint32_t bs, uint32_t off, int wide) {
  if (block < 0) return -1;
  const int64_t s = (int64_t)block * bs + off;
  return (wide || s <= 0x7FFFFFFF) ? s : -1;
}

}  // namespace

// One launch: every workgroup makes the two running sums over the requests
// itself (tokens, and blocks to take from the free list) and keeps them in
// LDS, then maps its share of the step's tokens.  Blocks a step adds are
// found in the free list by those sums, never read back from the table, so
// nothing waits for another workgroup; a new block's table entry is written
// by the token that opens it.
__global__ void __launch_bounds__(kSlotBlock) block_table_kernel(const TableParams q) {
  extern __shared__ int32_t lds_i[];
  int32_t* starts = lds_i;                    // first token of each request
  int32_t* fresh = lds_i + q.requests + 1;    // first free-list place of each
  __shared__ int64_t wave_tok[kSlotBlock / 64], wave_blk[kSlotBlock / 64];
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const uint32_t bs = (uint32_t)q.block_size;

  auto lens = [&](int r, int& kv, int& add) {
    kv = max(q.kv_lens[r], 0);
    add = min(max(q.new_tokens[r], 0), kv);
  };
  auto blocks = [&](int n) { return (int)min((uint32_t)q.max_blocks, ((uint32_t)n + bs - 1u) / bs); };

  int64_t tok0 = 0, blk0 = 0;
  for (int r0 = 0; r0 < q.requests; r0 += kSlotBlock) {
    const int r = r0 + t;
    int kv = 0, add = 0;
    if (r < q.requests) lens(r, kv, add);
    const int need = blocks(kv) - blocks(kv - add);
    int64_t a = add, b = need;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t oa = __shfl_up(a, d), ob = __shfl_up(b, d);
      if (lane >= d) {
        a += oa;
        b += ob;
      }
    }
    if (lane == 63) {
      wave_tok[wv] = a;
      wave_blk[wv] = b;
    }
    __syncthreads();
    int64_t ta = 0, tb = 0;
#pragma unroll
    for (int w = 0; w < kSlotBlock / 64; ++w) {
      if (w < wv) {
        a += wave_tok[w];
        b += wave_blk[w];
      }
      ta += wave_tok[w];
      tb += wave_blk[w];
    }
    if (r < q.requests) {
      starts[r] = (int32_t)min(tok0 + a - add, (int64_t)0x7FFFFFFF);
      fresh[r] = (int32_t)min(blk0 + b - need, (int64_t)0x7FFFFFFF);
    }
    tok0 += ta;
    blk0 += tb;
    __syncthreads();
  }
  const int64_t total = min(tok0, (int64_t)0x7FFFFFFF);
  if (t == 0) starts[q.requests] = (int32_t)total;
  __syncthreads();
  const int64_t first_free = max(q.free_start[0], 0);
  if (blockIdx.x == 0) {
    for (int r = t; r <= q.requests; r += kSlotBlock) q.token_starts[r] = starts[r];
    if (t == 0) q.free_next[0] = (int32_t)min(first_free + blk0, (int64_t)0x7FFFFFFF);
  }

  const int64_t end = max(total, q.max_tokens);
  for (int64_t n = (int64_t)blockIdx.x * kSlotBlock + t; n < end; n += (int64_t)gridDim.x * kSlotBlock) {
    int32_t req = -1, pos = -1;
    int64_t slot = -1;
    if (n < total) {
      int lo = 0, hi = q.requests;  // the last request that starts at or before n
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (starts[mid] <= (int32_t)n) lo = mid;
        else hi = mid;
      }
      req = lo;
      int kv, add;
      lens(req, kv, add);
      pos = kv - add + ((int32_t)n - starts[req]);
      const uint32_t blk = (uint32_t)pos / bs, off = (uint32_t)pos - blk * bs;
      const uint32_t held = (uint32_t)blocks(kv - add);
      if (blk < (uint32_t)q.max_blocks) {
        int32_t* entry = q.tables + (int64_t)req * q.table_stride + blk;
        int32_t id;
        if (blk < held) {
          id = *entry;
        } else {
          const int64_t at = first_free + fresh[req] + (blk - held);
          id = at < q.num_free ? q.free_blocks[at] : -1;
          if (off == 0) *entry = id;
        }
        slot = slot_of(id, bs, off, q.wide);
      }
    }
    if (n < q.max_tokens) {
      q.token_requests[n] = req;
      q.positions[n] = pos;
      if (q.wide) static_cast<int64_t*>(q.slots)[n] = slot;
      else static_cast<int32_t*>(q.slots)[n] = (int32_t)slot;
    }
  }
}

// Slots of selected positions: one entry a thread.
__global__ void __launch_bounds__(kSlotBlock) topk_slots_kernel(const SlotParams q) {
  const int64_t n = (int64_t)blockIdx.x * kSlotBlock + threadIdx.x;
  if (n >= q.rows * q.k) return;
  const int64_t row = n / q.k;
  const int64_t req = q.row_requests ? (int64_t)q.row_requests[row] : row / q.next_n;
  const int32_t i = q.indices[n];
  int64_t slot = -1;
  if (i >= 0 && req >= 0 && req < q.requests) {
    const uint32_t bs = (uint32_t)q.block_size;
    const uint32_t blk = (uint32_t)i / bs, off = (uint32_t)i - blk * bs;
    if (blk < (uint32_t)q.max_blocks)
      slot = slot_of(q.tables[req * q.table_stride + blk], bs, off, q.wide);
  }
  if (q.wide) static_cast<int64_t*>(q.slots)[n] = slot;
  else static_cast<int32_t*>(q.slots)[n] = (int32_t)slot;
}

const void* block_table_kernel_ptr() { return reinterpret_cast<const void*>(&block_table_kernel); }
const void* topk_slots_kernel_ptr() { return reinterpret_cast<const void*>(&topk_slots_kernel); }

}  // namespace ert
