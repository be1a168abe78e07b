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

// n / d for n < 2^31.
__device__ __forceinline__ uint32_t quotient(uint32_t n, const Divisor& d) {
  return (d.magic ? __umulhi(n, d.magic) : n) >> d.shift;
}

__device__ __forceinline__ int64_t slot_of(int32_t block, uint32_t bs, uint32_t off, int wide) {
  if (block < 0) return -1;
  const int64_t s = (int64_t)block * bs + off;
  return (wide || s <= 0x7FFFFFFF) ? s : -1;
}

}  // namespace

// One launch: every workgroup makes the two running sums over the requests
// itself (tokens, and blocks to take from the free list) and keeps them in
// LDS, then maps its share of the step's tokens, N neighbours a thread (four
// where there are enough to fill the chip with: one search and mostly one
// table entry for the four, and 16-byte stores).
// Blocks a step adds are found in the free list by those sums, never read
// back from the table, so nothing waits for another workgroup; a new block's
// table entry is written by the token that opens it.
//
// Bound by the sums over the requests, which every workgroup waits for, and
// then by writing: a million tokens of 61 prompts, 12 MB, take 7.7 us, 64
// decode tokens 3.2.
template <int N>
__global__ void __launch_bounds__(kSlotBlock) block_table_kernel(const TableParams q) {
  extern __shared__ int32_t lds_i[];
  int32_t* starts = lds_i;                       // first token of each request, and the total
  int32_t* first = starts + q.requests + 1;      // its position
  int32_t* fresh = first + q.requests;           // the request's first place in the free list
  __shared__ int64_t wave_tok[kSlotBlock / 64], wave_blk[kSlotBlock / 64];
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const uint32_t bs = (uint32_t)q.block_size;
  // blocks that hold n tokens, within the table
  auto blocks = [&](int n) {
    return n > 0 ? (int)min((uint32_t)q.max_blocks, quotient((uint32_t)n - 1u, q.by_block) + 1u) : 0;
  };

  int64_t tok0 = 0, blk0 = 0;
  for (int r0 = 0; r0 < q.requests; r0 += kSlotBlock) {
    const int r = r0 + t;
    int kv = 0, add = 0;
    if (r < q.requests) {
      kv = max(q.kv_lens[r], 0);
      add = min(max(q.new_tokens[r], 0), kv);
    }
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
      first[r] = kv - add;
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
  for (int64_t n0 = ((int64_t)blockIdx.x * kSlotBlock + t) * N; n0 < end;
       n0 += (int64_t)gridDim.x * kSlotBlock * N) {
    int req = 0;
    if (n0 < total) {
      int hi = q.requests;  // the last request that starts at or before n0
      while (hi - req > 1) {
        const int mid = (req + hi) >> 1;
        if (starts[mid] <= (int32_t)n0) req = mid;
        else hi = mid;
      }
    }
    int32_t owner[N], place[N];
    int64_t slot[N];
    uint32_t known = 0xFFFFFFFFu;  // the block looked up last, of this request
    int32_t id = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int64_t n = n0 + i;
      owner[i] = place[i] = -1;
      slot[i] = -1;
      if (n >= total) continue;
      while (starts[req + 1] <= (int32_t)n) {
        ++req;
        known = 0xFFFFFFFFu;
      }
      const int pos = first[req] + ((int32_t)n - starts[req]);
      const uint32_t blk = quotient((uint32_t)pos, q.by_block), off = (uint32_t)pos - blk * bs;
      owner[i] = req;
      place[i] = pos;
      if (blk >= (uint32_t)q.max_blocks) continue;
      if (blk != known) {
        known = blk;
        int32_t* entry = q.tables + (int64_t)req * q.table_stride + blk;
        const uint32_t held = (uint32_t)blocks(first[req]);
        if (blk < held) {
          id = *entry;
        } else {
          const int64_t at = first_free + fresh[req] + (blk - held);
          id = at < q.num_free ? q.free_blocks[at] : -1;
          if (off == 0) *entry = id;
        }
      }
      slot[i] = slot_of(id, bs, off, q.wide);
    }
    if (N == 4 && q.vector && n0 + 4 <= q.max_tokens) {
      *reinterpret_cast<int4*>(q.token_requests + n0) =
          int4{owner[0], owner[1 % N], owner[2 % N], owner[3 % N]};
      *reinterpret_cast<int4*>(q.positions + n0) =
          int4{place[0], place[1 % N], place[2 % N], place[3 % N]};
      if (!q.wide) {
        *reinterpret_cast<int4*>(static_cast<int32_t*>(q.slots) + n0) =
            int4{(int32_t)slot[0], (int32_t)slot[1 % N], (int32_t)slot[2 % N], (int32_t)slot[3 % N]};
      } else {
        longlong2* out = reinterpret_cast<longlong2*>(static_cast<int64_t*>(q.slots) + n0);
        out[0] = longlong2{slot[0], slot[1 % N]};
        out[1] = longlong2{slot[2 % N], slot[3 % N]};
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (n0 + i < q.max_tokens) {
          q.token_requests[n0 + i] = owner[i];
          q.positions[n0 + i] = place[i];
          if (q.wide) static_cast<int64_t*>(q.slots)[n0 + i] = slot[i];
          else static_cast<int32_t*>(q.slots)[n0 + i] = (int32_t)slot[i];
        }
    }
  }
}

// Slots of selected positions: kSlotPart entries of one row a workgroup, four
// neighbours a thread.  The row's table goes through LDS where that pays:
// its entries are then read once, side by side, and the scattered look-ups
// stay on the compute unit.  Bound by reading and writing: 4096 rows of 1024
// positions over 256 entries, 33.6 MB, take 8.4 us alone and 7.6 one behind
// the other (4.4 TB/s); 64 rows of 2048 take 3.2, half of it the launch.
__global__ void __launch_bounds__(kSlotBlock) topk_slots_kernel(const SlotParams q) {
  extern __shared__ int32_t table_lds[];
  const uint32_t row = blockIdx.x / (uint32_t)q.parts;
  const int j0 = (int)(blockIdx.x - row * (uint32_t)q.parts) * kSlotPart;
  const int64_t req = q.row_requests ? (int64_t)q.row_requests[row] : (int64_t)(row / (uint32_t)q.next_n);
  const bool known = req >= 0 && req < q.requests;
  const int32_t* table = q.tables + (known ? req * q.table_stride : 0);
  const int n = known ? q.max_blocks : 0;
  const int64_t base = (int64_t)row * q.k;
  const uint32_t bs = (uint32_t)q.block_size;
  // (k < 2^31 and parts of a power of two: no position passes 2^31 - 1)
  int32_t i[kSlotPart / kSlotBlock / 4][4];
#pragma unroll
  for (int g = 0; g < kSlotPart / kSlotBlock / 4; ++g) {
    const int j = j0 + (g * kSlotBlock + (int)threadIdx.x) * 4;
    if (q.vector) {
      int4 v{-1, -1, -1, -1};
      if (j < q.k) v = *reinterpret_cast<const int4*>(q.indices + base + j);
      i[g][0] = v.x, i[g][1] = v.y, i[g][2] = v.z, i[g][3] = v.w;
    } else {
#pragma unroll
      for (int o = 0; o < 4; ++o) i[g][o] = j + o < q.k ? q.indices[base + j + o] : -1;
    }
  }
  if (q.staged) {
    for (int b = threadIdx.x; b < n; b += kSlotBlock) table_lds[b] = table[b];
    __syncthreads();
  }
#pragma unroll
  for (int g = 0; g < kSlotPart / kSlotBlock / 4; ++g) {
    const int j = j0 + (g * kSlotBlock + (int)threadIdx.x) * 4;
    int64_t slot[4];
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const uint32_t p = (uint32_t)i[g][o];
      const uint32_t blk = quotient(p & 0x7FFFFFFFu, q.by_block), off = p - blk * bs;
      slot[o] = -1;
      if (i[g][o] >= 0 && blk < (uint32_t)n)
        slot[o] = slot_of(q.staged ? table_lds[blk] : table[blk], bs, off, q.wide);
    }
    if (q.vector) {
      if (j >= q.k) continue;
      if (!q.wide) {
        *reinterpret_cast<int4*>(static_cast<int32_t*>(q.slots) + base + j) =
            int4{(int32_t)slot[0], (int32_t)slot[1], (int32_t)slot[2], (int32_t)slot[3]};
      } else {
        longlong2* out = reinterpret_cast<longlong2*>(static_cast<int64_t*>(q.slots) + base + j);
        out[0] = longlong2{slot[0], slot[1]};
        out[1] = longlong2{slot[2], slot[3]};
      }
    } else {
#pragma unroll
      for (int o = 0; o < 4; ++o)
        if (j + o < q.k) {
          if (q.wide) static_cast<int64_t*>(q.slots)[base + j + o] = slot[o];
          else static_cast<int32_t*>(q.slots)[base + j + o] = (int32_t)slot[o];
        }
    }
  }
}

const void* block_table_kernel_ptr(int per_thread) {
  return per_thread == 4 ? reinterpret_cast<const void*>(&block_table_kernel<4>)
                         : reinterpret_cast<const void*>(&block_table_kernel<1>);
}
const void* topk_slots_kernel_ptr() { return reinterpret_cast<const void*>(&topk_slots_kernel); }

}  // namespace ert
