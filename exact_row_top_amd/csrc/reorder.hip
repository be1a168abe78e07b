// reorder.hip -- after a beam search's choice: each child takes over what its
// parent holds.
//
// Rows of any state move by gathering, out[child] = state[parent of child].  A
// paged cache moves without its full blocks: children share them through
// their table rows, and only the open block, which the next token is written
// into, is copied to the block that the child's row owns.
//
// A thread owns 16 bytes of every row of a request: it loads its piece of all
// parents' rows and stores its piece of all children's, so moving in place
// needs no barrier and no second buffer, whatever the parents.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "search.h"

namespace ert {

namespace {

// 16 bytes at any address.  Stored with the hint that nothing reads them soon:
// a step moves more than the caches keep until the next (256 rows of 260 KB and
// as many open blocks took 59 us without it, 51 to 56 with it).
typedef uint32_t Loose16 __attribute__((ext_vector_type(4), aligned(1)));

// The last bytes of a row, fewer than 16, in pieces of 8, 4, 2 and 1.
__device__ __forceinline__ Loose16 load_tail(const unsigned char* p, uint32_t n) {
  unsigned char b[16] = {};
  if (n & 8) __builtin_memcpy(b, p, 8), p += 8;
  if (n & 4) __builtin_memcpy(b + 8, p, 4), p += 4;
  if (n & 2) __builtin_memcpy(b + 12, p, 2), p += 2;
  if (n & 1) b[14] = *p;
  Loose16 v;
  __builtin_memcpy(&v, b, 16);
  return v;
}
__device__ __forceinline__ void store_tail(unsigned char* p, uint32_t n, const Loose16& v) {
  unsigned char b[16];
  __builtin_memcpy(b, &v, 16);
  if (n & 8) __builtin_memcpy(p, b, 8), p += 8;
  if (n & 4) __builtin_memcpy(p, b + 8, 4), p += 4;
  if (n & 2) __builtin_memcpy(p, b + 12, 2), p += 2;
  if (n & 1) *p = b[14];
}

// A number that lane j holds, in all lanes.
__device__ __forceinline__ uint64_t of_lane(uint64_t v, int j) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), j) << 32 |
         (uint32_t)__builtin_amdgcn_readlane((int)v, j);
}

// Moves this thread's piece of a request's rows: lane j holds child j's source
// and target (0: none; a target without a source is cleared).  With k <= N
// everything is read before anything is written.
template <int N>
__device__ __forceinline__ void move_rows(int k, int64_t bytes, int64_t off, uint64_t src, uint64_t dst) {
  const int64_t left = bytes - off;
  const uint32_t tail = left < 16 ? (uint32_t)max(left, (int64_t)0) : 0u;
  for (int j0 = 0; j0 < k; j0 += N) {
    Loose16 v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      v[j] = Loose16{0, 0, 0, 0};
      const unsigned char* p = reinterpret_cast<const unsigned char*>(of_lane(src, j0 + j));
      if (p && left > 0) {
        if (!tail) v[j] = *reinterpret_cast<const Loose16*>(p + off);
        else v[j] = load_tail(p + off, tail);
      }
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      unsigned char* p = reinterpret_cast<unsigned char*>(of_lane(dst, j0 + j));
      if (p && left > 0) {
        if (!tail) __builtin_nontemporal_store(v[j], reinterpret_cast<Loose16*>(p + off));
        else store_tail(p + off, tail, v[j]);
      }
    }
  }
}

}  // namespace

// Rows of up to kMaxCopies arrays in one launch; a workgroup takes 4 KB of
// every row of a request.  Bound by memory: 256 rows of 260 KB, 68 MB written
// and, by the children's parents, up to as much read, take 20 us where the
// last-level cache holds them; 8 small rows 3.3, the launch and the wait for
// the parents.
template <int N>
__global__ void __launch_bounds__(kCopyBlock) reorder_rows_kernel(const ReorderParams q) {
  int a = 0;
  while (a + 1 < q.copies && blockIdx.x >= q.copy[a + 1].first) ++a;
  const RowCopy c = q.copy[a];
  const uint32_t at = blockIdx.x - c.first;
  const uint32_t req = at / c.tiles;
  const int64_t off = ((int64_t)(at - req * c.tiles) * kCopyBlock + threadIdx.x) * 16;
  const int j = (int)(threadIdx.x & 63);
  uint64_t src = 0, dst = 0;
  if (j < q.k) {
    const int p = q.parents[(int64_t)req * q.k + j];
    const bool has = (unsigned)p < (unsigned)q.beams;
    if (has) src = (uint64_t)(c.src + ((int64_t)req * q.beams + p) * c.src_stride);
    dst = (uint64_t)(c.dst + ((int64_t)req * q.k + j) * c.dst_stride);
    // nothing to do for a row that stays where it is
    if (has ? dst == src : !q.clear) src = dst = 0;
  }
  move_rows<N>(q.k, c.row_bytes, off, src, dst);
}

// Table rows and open blocks.  The launch's first workgroups copy: a request's
// open blocks in one cache each, 4 KB of a block at a time; the others make
// its table rows, a thread an entry of every row.  Bound by memory: 32 requests
// of 8 beams, blocks of 64 slots of 2 KB about half full, four caches, 67 MB
// written, take 20 us where the last-level cache holds what is read; 8 rows 4.
template <int N>
__global__ void __launch_bounds__(kCopyBlock) reorder_blocks_kernel(const ReorderBlocksParams q) {
  const uint32_t copying = q.copying ? (uint32_t)q.caches * q.requests * q.tiles : 0u;
  const uint32_t w = blockIdx.x;
  const bool copy = w < copying;
  const uint32_t per = copy ? q.tiles : q.table_tiles;
  const uint32_t unit = (copy ? w : w - copying) / per;
  const uint32_t tile = (copy ? w : w - copying) - unit * per;
  const uint32_t req = copy ? unit % (uint32_t)q.requests : unit;
  const int32_t* tables = q.tables + (int64_t)req * q.beams * q.table_stride;
  const uint32_t len = (uint32_t)max(q.kv_lens[req], 0);
  const uint32_t full = q.by_block(len), part = len - full * (uint32_t)q.block_size;
  const bool open = part > 0 && full < (uint32_t)q.max_blocks;
  // lane j: child j
  const int j = (int)(threadIdx.x & 63);
  const int parent = j < q.k ? q.parents[(int64_t)req * q.k + j] : -1;
  const bool has = (unsigned)parent < (unsigned)q.beams;
  if (copy) {
    if (!open) return;
    unsigned char* cache = q.cache[unit / (uint32_t)q.requests];
    uint64_t src = 0, dst = 0;
    if (has) {
      const int32_t from = tables[parent * q.table_stride + full];
      // the block that the child's open one becomes
      const int32_t own = q.tail ? q.tail[(int64_t)req * q.k + j] : tables[j * q.table_stride + full];
      if (from >= 0 && from < q.num_blocks && own >= 0 && own < q.num_blocks && own != from) {
        src = (uint64_t)(cache + from * q.block_stride);
        dst = (uint64_t)(cache + own * q.block_stride);
      }
    }
    const int64_t bytes = (int64_t)part * q.slot_bytes;
    for (int64_t off = (int64_t)tile * kCopyBlock * 16; off < bytes; off += (int64_t)q.tiles * kCopyBlock * 16)
      move_rows<N>(q.k, bytes, off + threadIdx.x * 16, src, dst);
    return;
  }
  const uint32_t e = tile * kCopyBlock + threadIdx.x;
  const int own = has && open && q.tail ? q.tail[(int64_t)req * q.k + j] : -1;
  int32_t* out = q.out + (int64_t)req * q.k * q.out_stride + e;
  const bool rows_stay = q.beams == q.k, inside = e < (uint32_t)q.max_blocks;
  for (int j0 = 0; j0 < q.k; j0 += N) {
    int32_t v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = -1;
      const int p = __builtin_amdgcn_readlane(parent, j0 + i), tail = __builtin_amdgcn_readlane(own, j0 + i);
      if (j0 + i >= q.k || !inside) continue;
      const bool child = (unsigned)p < (unsigned)q.beams;
      if (child && e < full) v[i] = tables[p * q.table_stride + e];
      else if (child && open && e == full && q.tail) v[i] = tail;
      else if (rows_stay) v[i] = tables[(j0 + i) * q.table_stride + e];
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (j0 + i < q.k && inside) out[(j0 + i) * q.out_stride] = v[i];
  }
}

const void* reorder_rows_kernel_ptr(int n) {
  return n == 8 ? reinterpret_cast<const void*>(&reorder_rows_kernel<8>)
                : reinterpret_cast<const void*>(&reorder_rows_kernel<32>);
}
const void* reorder_blocks_kernel_ptr(int n) {
  return n == 8 ? reinterpret_cast<const void*>(&reorder_blocks_kernel<8>)
                : reinterpret_cast<const void*>(&reorder_blocks_kernel<32>);
}

}  // namespace ert
