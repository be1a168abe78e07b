// beams.hip -- one step of a beam search: the k best continuations of a
// request's beams over the vocabulary.
//
// A beam b with score s_b and logits x offers every token i with the total
// s_b + x_i - ln sum_j exp(x_j); totals (divided by a power of the length
// where one is asked for) are ranked over the request's beams.  Within a beam
// the order is that of the logits, so its own k best logits are all that can
// be chosen, and the sum of exponentials is one number a beam.
//
// The sum's weights are whole multiples of 2^-43 of a segment's largest, added
// up exactly, and segments are counted from the row's own start whatever its
// alignment: rows with the same scores have the same sum to the bit, and ties
// between them go to the lower index.
//
// Two launches: the segment kernel reads the logits once, the row kernel finds
// each beam's k best and, in a request's last workgroup, the request's.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gvr_device.h"
#include "search.h"

namespace ert {

namespace {

// 16 bytes from any address that is aligned to an element.
__device__ __forceinline__ uint4 load16(const unsigned char* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

__device__ __forceinline__ bool offers(float score) { return __builtin_fabsf(score) < __builtin_inff(); }

}  // namespace

// ---------------------------------------------------------------------------
// Segment kernel: a wave reads 2048 scores of a row and writes the largest,
// the weights' sum against it, and the largest of each 32 neighbours.
// ---------------------------------------------------------------------------
template <class T>
__global__ void __launch_bounds__(256) beam_segment_kernel(const BeamParams q) {
  constexpr int V = Elem<T>::kVec;
  constexpr int G = kSegment / (64 * V);
  constexpr int L = kChunk / V;  // lanes of a chunk
  static_assert(G == L, "a lane keeps one chunk");
  const int lane = threadIdx.x & 63;
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (id >= (uint32_t)q.rows * (uint32_t)q.segments) return;
  const int row = (int)(id / (uint32_t)q.segments);
  const int seg = (int)(id - (uint32_t)row * (uint32_t)q.segments);
  if (seg == 0 && row % q.beams == 0 && lane == 0) q.arrived[row / q.beams] = 0;
  if ((q.ended && q.ended[row]) || !offers(q.scores[row])) return;

  const unsigned char* base =
      static_cast<const unsigned char*>(q.logits) + (int64_t)row * q.row_stride * (int64_t)sizeof(T);
  const int pos0 = seg * kSegment + lane * V;
  float x[G][V];
  if ((seg + 1) * kSegment <= q.vocab) {
#pragma unroll
    for (int g = 0; g < G; ++g)
      Elem<T>::unpack(load16(base + (int64_t)(pos0 + g * 64 * V) * (int64_t)sizeof(T)), x[g]);
  } else {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const int pos = pos0 + g * 64 * V + e;
        x[g][e] = pos < q.vocab ? Elem<T>::load(base, pos) : -__builtin_inff();
      }
  }
  float top = -__builtin_inff(), mine = -__builtin_inff();
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float m = -__builtin_inff();
#pragma unroll
    for (int e = 0; e < V; ++e) {
      x[g][e] = x[g][e] > -__builtin_inff() ? x[g][e] : -__builtin_inff();  // NaN too
      m = fmaxf(m, x[g][e]);
    }
#pragma unroll
    for (int d = 1; d < L; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    top = fmaxf(top, m);
    if ((lane & (L - 1)) == g) mine = m;
  }
  float low = top, best = top;
  wave_minmax(low, best);
  q.chunks[(int64_t)id * 64 + (lane & (L - 1)) * (64 / L) + lane / L] = mine;

  uint64_t mass = 0;
  if (best == __builtin_inff()) {
    uint32_t n = 0;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) n += x[g][e] == best ? 1u : 0u;
    mass = wave_sum((uint64_t)n * kOne);
  } else if (best > -__builtin_inff()) {
    // (four scores at a time: with more in flight the registers leave room
    // for fewer waves)
    const Weigher w(best, kLog2e);
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        mass += w.raw(x[g][e]);
        if (e % 4 == 3) {
          asm("" : "+v"(mass));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    mass = wave_sum(mass - (uint64_t)(G * V) * kRaw);
  }
  if (lane == 0) {
    q.bests[id] = best;
    q.masses[id] = mass;
  }
}

// ---------------------------------------------------------------------------
// Row kernel: one workgroup a beam.
//
// Of the chunks ordered by (largest score falling, position) the first k hold
// the beam's k best: were one of those in another chunk, the k chunks before
// that one would each hold a score before it.  A bound for the k-th chunk is
// the k-th largest of the threads' own maxima; what lies above it goes to LDS
// and is ranked by counting, as are the chosen chunks' scores from the k-th
// chunk's largest up.  So equal scores cost no more than others.
// ---------------------------------------------------------------------------

namespace {

constexpr int kBeamWaves = kBeamBlock / 64;

struct BeamShared {
  uint32_t keys[kBeamBlock];
  int32_t chosen[kMaxBeamK];
  float top[kMaxBeamK];
  float redf[kBeamWaves];
  double redd[kBeamWaves];
  uint32_t n;
  uint32_t turn;
  BeamCandidate out[kMaxBeamK];
};

__device__ __forceinline__ float block_max(float v, BeamShared& sh) {
  float low = v;
  wave_minmax(low, v);
  if ((threadIdx.x & 63) == 0) sh.redf[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh.redf[0];
#pragma unroll
  for (int w = 1; w < kBeamWaves; ++w) v = fmaxf(v, sh.redf[w]);
  return v;
}

// Added up in one fixed order.
__device__ __forceinline__ double block_sum(double v, BeamShared& sh) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  if ((threadIdx.x & 63) == 0) sh.redd[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sh.redd[0];
#pragma unroll
  for (int w = 1; w < kBeamWaves; ++w) v += sh.redd[w];
  return v;
}

// Appends what is `in` to a list in LDS; returns the place.
__device__ __forceinline__ uint32_t append(bool in, uint32_t* n) {
  const uint64_t mask = __ballot(in);
  if (mask == 0) return 0;
  uint32_t base = 0;
  if ((threadIdx.x & 63) == 0) base = atomicAdd(n, (uint32_t)__popcll(mask));
  base = __builtin_amdgcn_readfirstlane(base);
  return base + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32),
                                          __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
}

// How many of the list's n entries come before (x, i).
__device__ __forceinline__ int before(const float* lx, const int32_t* li, int n, float x, int i) {
  int c = 0;
  for (int j = 0; j < n; ++j) c += (lx[j] > x || (lx[j] == x && li[j] < i)) ? 1 : 0;
  return c;
}

}  // namespace

template <class T>
__global__ void __launch_bounds__(kBeamBlock) beam_row_kernel(const BeamParams q) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ BeamShared sh;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const int row = blockIdx.x, req = row / q.beams, beam = row - req * q.beams;
  const int k = q.k, segs = q.segments;
  const float score = q.scores[row];
  const bool ended = q.ended && q.ended[row];
  double norm = 1.0;
  if (q.lengths && q.penalty != 0.0)
    norm = pow((double)max((int64_t)q.lengths[row] + (ended ? 0 : 1), (int64_t)1), q.penalty);
  if (t < k) sh.out[t] = BeamCandidate{-__builtin_inf(), -__builtin_inff(), -1};
  if (t == 0) sh.n = 0;
  __syncthreads();

  if (offers(score)) {
    if (ended) {
      if (t == 0) sh.out[0] = BeamCandidate{(double)score / norm, score, q.end_token};
    } else {
      const float* bests = q.bests + (int64_t)row * segs;
      const uint64_t* masses = q.masses + (int64_t)row * segs;
      float m = -__builtin_inff();
      for (int s = t; s < segs; s += kBeamBlock) m = fmaxf(m, bests[s]);
      // the largest chunk of each thread's own
      const float* chunks = q.chunks + (int64_t)row * segs * 64 + (int64_t)wv * (segs * 64 / kBeamWaves);
      const int mine = segs * 64 / kBeamWaves;  // a wave's chunks
      float top = -__builtin_inff();
      for (int c = lane; c < mine; c += 64) top = fmaxf(top, chunks[c]);
      sh.keys[t] = fkey(top);
      m = block_max(m, sh);
      if (m > -__builtin_inff()) {
        const Exp2Poly poly;
        double sum = 0.0;
        for (int s = t; s < segs; s += kBeamBlock) {
          const float b = bests[s];
          const double w = b == m ? 1.0 : exp2_64(((double)b - (double)m) * kLog2e, poly);
          sum += (double)masses[s] * w;
        }
        sum = block_sum(sum, sh) * 0x1p-43;
        const double lse = m == __builtin_inff() ? log(sum) : (double)m + log(sum);

        uint32_t key[kBeamWaves], thr = 0;
#pragma unroll
        for (int i = 0; i < kBeamWaves; ++i) key[i] = sh.keys[i * 64 + lane];
#pragma unroll 1
        for (int b = 31; b >= 0; --b) {
          const uint32_t at = thr | (1u << b);
          int n = 0;
#pragma unroll
          for (int i = 0; i < kBeamWaves; ++i) n += __popcll(__ballot(key[i] >= at));
          if (n >= k) thr = at;
        }
        const float floor = from_key(thr);
        float* lx = reinterpret_cast<float*>(lds);
        int32_t* li = reinterpret_cast<int32_t*>(lx + q.cap);
        int ties = 0;  // this wave's, in the order of the row
        for (int c0 = 0; c0 < mine; c0 += 64) {
          const float v = c0 + lane < mine ? chunks[c0 + lane] : -__builtin_inff();
          const uint64_t even = __ballot(v == floor && v > -__builtin_inff());
          const int rank = ties + (int)__builtin_amdgcn_mbcnt_hi(
                                      (uint32_t)(even >> 32),
                                      __builtin_amdgcn_mbcnt_lo((uint32_t)even, 0u));
          const bool in = v > floor || ((even >> lane & 1) && rank < k);
          ties += __popcll(even);
          const uint32_t at = append(in, &sh.n);
          if (in) {
            lx[at] = v;
            li[at] = wv * mine + c0 + lane;
          }
        }
        __syncthreads();
        const int n = (int)sh.n, picked = min(n, k);
        for (int i = t; i < n; i += kBeamBlock) {
          const int r = before(lx, li, n, lx[i], li[i]);
          if (r < k) {
            sh.chosen[r] = li[i];
            sh.top[r] = lx[i];
          }
        }
        __syncthreads();
        if (t == 0) sh.n = 0;
        const float least = n >= k ? sh.top[k - 1] : -__builtin_inff();
        __syncthreads();
        int32_t* gi = reinterpret_cast<int32_t*>(lx + k * kChunk);
        const unsigned char* base = static_cast<const unsigned char*>(q.logits) +
                                    (int64_t)row * q.row_stride * (int64_t)sizeof(T);
        for (int i0 = 0; i0 < picked * kChunk; i0 += kBeamBlock) {
          const int i = i0 + t;
          float v = -__builtin_inff();
          int pos = 0;
          if (i < picked * kChunk) {
            pos = sh.chosen[i / kChunk] * kChunk + i % kChunk;
            if (pos < q.vocab) v = Elem<T>::load(base, pos);
          }
          const bool in = v > -__builtin_inff() && v >= least && (m < __builtin_inff() || v == m);
          const uint32_t at = append(in, &sh.n);
          if (in) {
            lx[at] = v;
            gi[at] = pos;
          }
        }
        __syncthreads();
        const int found = (int)sh.n;
        for (int i = t; i < found; i += kBeamBlock) {
          const float v = lx[i];
          const int r = before(lx, gi, found, v, gi[i]);
          if (r < k) {
            const double total = (double)score + (m == __builtin_inff() ? -lse : (double)v - lse);
            sh.out[r] = BeamCandidate{total / norm, (float)total, gi[i]};
          }
        }
      }
    }
  }
  __syncthreads();

  // The request's last beam merges them all.  What crosses between workgroups
  // goes through agent-scope atomics, complete before their workgroup counts
  // itself.
  if (t < k) {
    uint64_t w[2];
    __builtin_memcpy(w, &sh.out[t], 16);
    uint64_t* to = reinterpret_cast<uint64_t*>(q.found + (int64_t)row * k + t);
    agent_store(to, w[0]);
    agent_store(to + 1, w[1]);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);
  __syncthreads();
  if (t == 0) {
    sh.turn = __hip_atomic_fetch_add(q.arrived + req, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    sh.n = 0;
  }
  __syncthreads();
  if (sh.turn != (uint32_t)q.beams - 1) return;
  const int all = q.beams * k;
  double* rank = reinterpret_cast<double*>(lds);
  uint64_t* rest = reinterpret_cast<uint64_t*>(rank + all);
  const uint64_t* from = reinterpret_cast<const uint64_t*>(q.found + (int64_t)req * all);
  for (int i = t; i < all; i += kBeamBlock) {
    rank[i] = __longlong_as_double((long long)agent_load(from + 2 * i));
    rest[i] = agent_load(from + 2 * i + 1);
  }
  __syncthreads();
  for (int i = t; i < all; i += kBeamBlock) {
    BeamCandidate c;
    c.rank = rank[i];
    __builtin_memcpy(&c.total, &rest[i], 8);
    if (c.token < 0) continue;
    atomicAdd(&sh.n, 1u);
    const int b = i / k;
    int place = i - b * k;
    for (int o = 0; o < q.beams && place < k; ++o) {
      if (o == b) continue;
      // entries of beam o before c: in falling order, and the same from an
      // earlier beam first
      int lo = 0, hi = k;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        const double r = rank[o * k + mid];
        if (r > c.rank || (r == c.rank && o < b)) lo = mid + 1;
        else hi = mid;
      }
      place += lo;
    }
    if (place < k) {
      const int64_t at = (int64_t)req * k + place;
      q.out_scores[at] = c.total;
      q.parents[at] = b;
      q.tokens[at] = c.token;
    }
  }
  __syncthreads();
  for (int i = (int)sh.n + t; i < k; i += kBeamBlock) {
    const int64_t at = (int64_t)req * k + i;
    q.out_scores[at] = -__builtin_inff();
    q.parents[at] = -1;
    q.tokens[at] = -1;
  }
}

const void* beam_segment_kernel_ptr(int dtype) {
  return dtype == 0 ? reinterpret_cast<const void*>(&beam_segment_kernel<float>)
         : dtype == 1 ? reinterpret_cast<const void*>(&beam_segment_kernel<__hip_bfloat16>)
                      : reinterpret_cast<const void*>(&beam_segment_kernel<__half>);
}
const void* beam_row_kernel_ptr(int dtype) {
  return dtype == 0 ? reinterpret_cast<const void*>(&beam_row_kernel<float>)
         : dtype == 1 ? reinterpret_cast<const void*>(&beam_row_kernel<__hip_bfloat16>)
                      : reinterpret_cast<const void*>(&beam_row_kernel<__half>);
}

}  // namespace ert
