// evict.hip -- eviction from a cache by accumulated attention mass: which
// positions of each (request, head) stay, and the move of their rows to the
// front of the cache.
//
// The positions that stay are the first `sinks`, the last `recent` and, of the
// others, those with the largest mass (equal masses: the lower position; NaN
// below all), listed in rising order.  So the j-th of them comes from position
// kept[j] >= j, and rows can move in place from the front on.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gvr_device.h"
#include "search.h"

namespace ert {

namespace {

constexpr int kKeepWaves = kKeepBlock / 64;
constexpr int kDigitBins = 2048;

struct KeepShared {
  uint32_t count[kDigitBins];
  uint32_t wave[kKeepWaves];
  uint32_t wave2[kKeepWaves];
  uint32_t digit;
  uint32_t need;
  uint32_t whole;
};

}  // namespace

// ---------------------------------------------------------------------------
// One workgroup a row: the key of the last position that stays, digit by
// digit from the top (11, 11 and 10 bits, counted in LDS), then one pass that
// writes what stays in order, each wave its own range.  The row's mass sits in
// registers, HELD values a thread, and is read once; rows longer than 1024
// HELD are read again in every pass (HELD 0).
//
// Bound by the passes' waits and by the counting: 128 rows of 8192, which leave
// half of the compute units idle, take 11 us, one row of 5003 positions 8.  Rows
// in memory, four passes by one workgroup each: one of 65536 takes 67 us, 128 of
// them 98, one of 131072 126.
// ---------------------------------------------------------------------------
template <int HELD>
__global__ void __launch_bounds__(kKeepBlock) evict_keep_kernel(const KeepParams q) {
  __shared__ KeepShared sh;
  const int t = threadIdx.x, lane = t & 63;
  const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
  const int req = blockIdx.x / q.heads, head = blockIdx.x - req * q.heads;
  const float* mass = q.mass + req * q.request_stride + head * q.head_stride;
  const int n = min(max(q.kv_lens[req], 0), q.positions);
  const int stay = min(n, q.budget);
  int32_t* kept = q.kept + (int64_t)blockIdx.x * q.budget;
  float* out = q.mass_out ? q.mass_out + (int64_t)blockIdx.x * q.out_positions : nullptr;
  if (head == 0 && t == 0) q.new_lens[req] = stay;
  for (int j = stay + t; j < q.budget; j += kKeepBlock) kept[j] = -1;
  if (out)
    for (int j = stay + t; j < q.out_positions; j += kKeepBlock) out[j] = 0.0f;
  if (n <= q.budget) {
    for (int j = t; j < n; j += kKeepBlock) {
      kept[j] = j;
      if (out) out[j] = mass[j];
    }
    return;
  }
  const int lo = q.sinks, hi = n - q.recent;   // lo < hi: sinks + recent <= budget < n
  const int span = ((n + kKeepBlock - 1) / kKeepBlock) * 64;  // a wave's positions
  const int w0 = wv * span, steps = span / 64;
  // Keys: what always stays is above all masses (the largest of which is
  // 0xFF800000); NaN and what is behind the last position are zero.
  auto key_of = [&](int i, float m) { return i >= n ? 0u : (i < lo || i >= hi ? ~0u : rkey(m)); };
  float held[HELD > 0 ? HELD : 1];
  uint32_t keys[HELD > 0 ? HELD : 1];
  if (HELD > 0) {
#pragma unroll
    for (int s = 0; s < HELD; ++s) {
      const int i = w0 + s * 64 + lane;
      held[s] = s < steps && i < n ? mass[i] : 0.0f;
    }
#pragma unroll
    for (int s = 0; s < HELD; ++s) keys[s] = key_of(w0 + s * 64 + lane, held[s]);
  }
  // f(position, its mass, its key) for the wave's positions in order; the same
  // number of calls in every lane
  auto each = [&](auto&& f) {
    if (HELD > 0) {
#pragma unroll
      for (int s = 0; s < HELD; ++s)
        if (s < steps) f(w0 + s * 64 + lane, held[s], keys[s]);
    } else {
      for (int s = 0; s < steps; ++s) {
        const int i = w0 + s * 64 + lane;
        const float m = i < n ? mass[i] : 0.0f;
        f(i, m, key_of(i, m));
      }
    }
  };
  uint32_t need = (uint32_t)(q.budget - q.sinks - q.recent);
  // prefix: the digits found so far, all but the lowest `below` bits
  uint32_t prefix = need > 0 ? 0u : ~1u;
  int below = need > 0 ? 32 : 0;
  if (need > 0) {
#pragma unroll 1
    for (int level = 0; level < 3; ++level) {
      const int width = level < 2 ? 11 : 10, shift = below - width;
      for (int b = t; b < kDigitBins; b += kKeepBlock) sh.count[b] = 0;
      __syncthreads();
      // Positions without any mass count in registers first: their adds to one
      // address would wait for each other.
      uint32_t zeros = 0;
      each([&](int i, float m, uint32_t key) {
        if (i >= lo && i < hi && (level == 0 || (key >> (below & 31)) == prefix)) {
          if (m == 0.0f) ++zeros;
          else atomicAdd(&sh.count[(key >> shift) & ((1u << width) - 1)], 1u);
        }
      });
      zeros = wave_sum(zeros);
      if (lane == 0 && zeros) atomicAdd(&sh.count[(rkey(0.0f) >> shift) & ((1u << width) - 1)], zeros);
      __syncthreads();
      // from the largest digit down: thread t holds digits 2047 - 2t and 2046 - 2t
      const uint32_t a = sh.count[kDigitBins - 1 - 2 * t], b = sh.count[kDigitBins - 2 - 2 * t];
      uint32_t sum = wave_scan(a + b);
      if (lane == 63) sh.wave[wv] = sum;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kKeepWaves; ++w) sum += w < wv ? sh.wave[w] : 0u;
      const uint32_t above = sum - a - b;
      if (above < need && need <= above + a) {
        sh.digit = (uint32_t)(kDigitBins - 1 - 2 * t);
        sh.need = need - above;
        sh.whole = need == above + a;
      } else if (above + a < need && need <= sum) {
        sh.digit = (uint32_t)(kDigitBins - 2 - 2 * t);
        sh.need = need - above - a;
        sh.whole = need == sum;
      }
      __syncthreads();
      prefix = (prefix << width) | sh.digit;
      need = sh.need;
      below = shift;
      if (sh.whole) break;   // all that share these digits stay
    }
  }
  // Now `prefix` are the first digits of the last keys that stay, `need` how
  // many of their positions.
  uint32_t counts = 0;   // this lane's larger ones, and from bit 16 on its even ones
  uint32_t larger = 0, even = 0;
  each([&](int i, float, uint32_t key) {
    const uint32_t d = key >> below;
    if (HELD > 0) {
      counts += (d > prefix ? 1u : 0u) + (d == prefix && i < n ? 0x10000u : 0u);
    } else {
      larger += d > prefix ? 1u : 0u;
      even += d == prefix && i < n ? 1u : 0u;
    }
  });
  if (HELD > 0) {
    counts = wave_sum(counts);
    larger = counts & 0xFFFFu, even = counts >> 16;
  } else {
    larger = wave_sum(larger), even = wave_sum(even);
  }
  if (lane == 0) {
    sh.wave[wv] = larger;
    sh.wave2[wv] = even;
  }
  __syncthreads();
  uint32_t larger_before = 0, even_before = 0;
#pragma unroll
  for (int w = 0; w < kKeepWaves; ++w) {
    larger_before += w < wv ? sh.wave[w] : 0u;
    even_before += w < wv ? sh.wave2[w] : 0u;
  }
  uint32_t at = larger_before + min(even_before, need);
  each([&](int i, float m, uint32_t key) {
    const uint32_t d = key >> below;
    bool in = d > prefix;
    const uint64_t evens = __ballot(d == prefix && i < n);
    if (evens) {
      const uint32_t turn = even_before + __builtin_amdgcn_mbcnt_hi(
                                              (uint32_t)(evens >> 32),
                                              __builtin_amdgcn_mbcnt_lo((uint32_t)evens, 0u));
      in = in || ((evens >> lane & 1) && turn < need);
      even_before += (uint32_t)__popcll(evens);
    }
    const uint64_t ins = __ballot(in);
    if (!ins) return;
    const uint32_t j = at + __builtin_amdgcn_mbcnt_hi(
                                (uint32_t)(ins >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)ins, 0u));
    if (in) {
      kept[j] = i;
      if (out) out[j] = m;
    }
    at += (uint32_t)__popcll(ins);
  });
}

// ---------------------------------------------------------------------------
// Moves the kept rows, 16 bytes a thread, a step of rows at a time.  In place,
// all of a step's loads are done before its first store, and a later step
// reads positions behind everything that was stored (kept[j] >= j); between
// different blocks nothing waits, and workgroups share a row's positions.
//
// Bound by memory: rows of 256 bytes from all over a cache.  16 x 8192 positions
// to 1024, 8 heads of 256 bytes, two caches, 134 MB from and to memory, take 44
// us with the choice (27 at a copy's rate); 48 without the stores' hint, which
// keeps what is moved out of the caches' way.  Four rows in flight a thread:
// with 8 the same took 68 where four took 56, with 16 (fewer waves) 124.  In place
// a workgroup takes all of a row's positions, and its next loads wait for the last
// stores: the same move, 64 us.
// ---------------------------------------------------------------------------
namespace {
constexpr int kMoveRows = 4;   // rows in flight a thread
typedef uint32_t Four __attribute__((ext_vector_type(4)));
}

template <bool IN_PLACE>
__global__ void __launch_bounds__(kMoveBlock) evict_move_kernel(const MoveParams q) {
  uint32_t id = blockIdx.x;
  const int part = (int)(id % (uint32_t)q.parts);
  id /= (uint32_t)q.parts;
  const int column = (int)(id % (uint32_t)q.columns);
  id /= (uint32_t)q.columns;
  const int head = (int)(id % (uint32_t)q.heads);
  id /= (uint32_t)q.heads;
  const int req = (int)(id % (uint32_t)q.requests);
  unsigned char* cache = q.cache[id / (uint32_t)q.requests];
  const int32_t* kept = q.kept + ((int64_t)req * q.heads + head) * q.budget;
  const int32_t* from = q.tables + (int64_t)req * q.table_stride;
  const int32_t* to = q.out_tables + (int64_t)req * q.out_stride;
  const int64_t pieces = q.row_bytes / 16;
  const int wide = (int)((pieces + q.columns - 1) / q.columns);   // this workgroup's pieces of a row
  const int64_t c0 = (int64_t)column * wide;
  const int mine = (int)(pieces - c0 < wide ? pieces - c0 : (int64_t)wide);
  if (mine <= 0) return;
  // threads side by side on a row's pieces, the rest on further rows
  const int across = min(mine, kMoveBlock), down = kMoveBlock / across;
  const int x = (int)threadIdx.x % across, y = (int)threadIdx.x / across;
  const int step = down * kMoveRows;
  const int span = (((q.budget + q.parts - 1) / q.parts + step - 1) / step) * step;
  const int j1 = min(q.budget, (part + 1) * span);
  auto address = [&](const int32_t* table, int width, int p) -> unsigned char* {
    const uint32_t e = q.by_block((uint32_t)p);
    if (e >= (uint32_t)width) return nullptr;
    const int32_t b = table[e];
    if (b < 0 || b >= q.num_blocks) return nullptr;
    const int64_t slot = (int64_t)b * q.block_size + ((uint32_t)p - e * (uint32_t)q.block_size);
    return cache + slot * q.slot_bytes + head * q.row_bytes + c0 * 16;
  };
  for (int j0 = part * span; j0 < j1; j0 += step) {
    for (int x0 = 0; x0 < mine; x0 += across) {
      Four v[kMoveRows];
      unsigned char* dst[kMoveRows];
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i) {
        const int j = j0 + i * down + y;
        dst[i] = nullptr;
        v[i] = Four{0, 0, 0, 0};
        if (y < down && j < j1 && x0 + x < mine) {
          const int p = kept[j];
          const unsigned char* src = p >= 0 ? address(from, q.max_blocks, p) : nullptr;
          dst[i] = src ? address(to, q.out_blocks, j) : nullptr;
          if (dst[i] == src) dst[i] = nullptr;
          if (dst[i]) {
            v[i] = *reinterpret_cast<const Four*>(src + (int64_t)(x0 + x) * 16);
            dst[i] += (int64_t)(x0 + x) * 16;
          }
        }
      }
      if (IN_PLACE) {
        __builtin_amdgcn_s_waitcnt(0x0F70);  // the loads are done
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < kMoveRows; ++i)
        if (dst[i]) __builtin_nontemporal_store(v[i], reinterpret_cast<Four*>(dst[i]));
      if (IN_PLACE) __syncthreads();
    }
  }
}

const void* evict_keep_kernel_ptr(int64_t positions) {
  if (positions <= 8 * kKeepBlock) return reinterpret_cast<const void*>(&evict_keep_kernel<8>);
  if (positions <= 32 * kKeepBlock) return reinterpret_cast<const void*>(&evict_keep_kernel<32>);
  return reinterpret_cast<const void*>(&evict_keep_kernel<0>);
}
const void* evict_move_kernel_ptr(bool in_place) {
  return in_place ? reinterpret_cast<const void*>(&evict_move_kernel<true>)
                  : reinterpret_cast<const void*>(&evict_move_kernel<false>);
}

}  // namespace ert
