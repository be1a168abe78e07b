// beams.hip -- one step of a beam search: the k best continuations of a
// request's beams over the vocabulary.
//
// A beam b with score s_b and logits x offers every token i with the total
// s_b + x_i - ln sum_j exp(x_j); totals (divided by a power of the length
// where one is asked for) are ranked over the request's beams.  Within a beam
// the order is that of the logits, so its own k best logits are all that can
// be chosen, and the sum of exponentials is one number a beam.
//
// The sum is made in 64 bits, in one order that is counted from the row's own
// start whatever its alignment: rows with the same scores have the same sum to
// the bit, and ties between them go to the lower index.
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

// 2^s for s <= 0 (-1000 and less, and NaN, as 2^-1000): interpolation of 2^f at
// the nine Chebyshev nodes of [-1/2, 1/2], relative error at most 2^-39.7, and
// 1 for s = 0.  Adding 1.5 * 2^52 rounds s to a whole n, which then stands in
// the sum's low bits and is added to the result's exponent.  (The coefficients
// in scalar registers, as in Exp2Poly.)  Ranks need totals far better than
// 32-bit sums would make them, and this is a third cheaper than weights that
// are whole numbers, which add up exactly in any order.
constexpr double kShift = 6755399441055744.0;
struct Exp2Short {
  double k1, k2, k3, k4, k5, k6, k7, k8;
  __device__ __forceinline__ Exp2Short()
      : k1(0x1.62e42fef84cf0p-1), k2(0x1.ebfbdff823cedp-3), k3(0x1.c6b08dd6fd234p-5),
        k4(0x1.3b2ab7181b755p-7), k5(0x1.5d8745a728441p-10), k6(0x1.4308ac85aa947p-13),
        k7(0x1.00dc4a532fb8ep-16), k8(0x1.63d136366db24p-20) {
    asm("" : "+s"(k1), "+s"(k2), "+s"(k3), "+s"(k4));
    asm("" : "+s"(k5), "+s"(k6), "+s"(k7), "+s"(k8));
  }
  __device__ __forceinline__ double operator()(double s) const {
    s = __builtin_fmax(s, -1000.0);
    const double sm = s + kShift;
    return scaled(s - (sm - kShift), sm);
  }
  // 2^f times 2 to the power of the whole number in sm's low bits.
  __device__ __forceinline__ double scaled(double f, double sm) const {
    double p = __builtin_fma(f, k8, k7);
    p = __builtin_fma(p, f, k6);
    p = __builtin_fma(p, f, k5);
    p = __builtin_fma(p, f, k4);
    p = __builtin_fma(p, f, k3);
    p = __builtin_fma(p, f, k2);
    p = __builtin_fma(p, f, k1);
    p = __builtin_fma(p, f, 1.0);
    const uint64_t bits = (uint64_t)__double_as_longlong(p);
    return __hiloint2double((int)((uint32_t)(bits >> 32) + ((uint32_t)__double_as_longlong(sm) << 20)),
                            (int)(uint32_t)bits);
  }
};

__device__ __forceinline__ bool offers(float score) { return __builtin_fabsf(score) < __builtin_inff(); }

}  // namespace

// ---------------------------------------------------------------------------
// Segment kernel: a wave reads 2048 scores of a row and writes the largest,
// the weights' sum against it, and the largest of each 32 neighbours.
//
// Bound by the 64-bit exponentials where the scores are 16 bits wide: 240 rows
// of 50001, 24 MB, take 13.9 us (1.7 TB/s); and nearly by memory where they
// are 32: 256 rows of 131072, a tenth of them ended, 121 MB, take 27 us (4.5
// TB/s).
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
    for (int e = 0; e < V; ++e) m = fmaxf(m, x[g][e]);  // (passes over NaN)
#pragma unroll
    for (int d = 1; d < L; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
    top = fmaxf(top, m);
    if ((lane & (L - 1)) == g) mine = m;
  }
  float low = top, best = top;
  wave_minmax(low, best);
  q.chunks[(int64_t)id * 64 + (lane & (L - 1)) * (64 / L) + lane / L] = mine;

  double mass = 0.0;
  if (best == __builtin_inff()) {
    uint32_t n = 0;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) n += x[g][e] == best ? 1u : 0u;
    mass = (double)wave_sum(n);
  } else if (best > -__builtin_inff()) {
    // (four scores at a time: with more in flight the registers leave room
    // for fewer waves)
    const Exp2Short exp2;
    auto add_all = [&](auto&& weight) {
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          mass += weight(x[g][e]);
          if (e % 4 == 3) {
            asm("" : "+v"(mass));
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      mass = wave_sum(mass);
    };
    if (__builtin_fabsf(best) < 0x1p20f) {
      // 2^((x - best) log2(e)) as 2^(x log2(e) + whole) times the rest of -best
      // log2(e), once for all; what is 690 below the largest weighs nothing
      const float low = best - 690.0f;
      const double whole = __builtin_rint(-(double)best * kLog2e), shift = kShift + whole;
      add_all([&](float v) {
        const double d = (double)fmaxf(v, low), sm = __builtin_fma(d, kLog2e, shift);
        return exp2.scaled(__builtin_fma(d, kLog2e, -(sm - shift)), sm);
      });
      mass *= exp2(__builtin_fma(-(double)best, kLog2e, -whole));
    } else {
      // (too large for products apart: the difference first)
      add_all([&](float v) { return exp2(((double)v - (double)best) * kLog2e); });
    }
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
// that one would each hold a score before it.  The chunks' maxima sit in
// registers; a bound for the k-th of them is the k-th largest of 128 sets' own
// maxima, found to 16 bits of its key with ballots.  What reaches it goes to
// LDS and is ranked by counting, as are the chosen chunks' scores from the
// k-th chunk's largest up.  Where more reach it than fit (equal or nearly
// equal maxima), the bound is the k-th largest of the 512 threads' maxima to
// the bit: fewer than k threads hold any above it, and of those that equal it
// each wave takes its first k.
//
// Bound by the waits between these steps, and in a batch by its rankings, which
// grow with k: 4 rows of 32768, best 8, take 7.1 us, 240 of 50001, best 10, 8.7,
// 256 of 131072 9.1, 11.7 and 19.1 for the best 4, 16 and 32 of 8 beams each, 9.7
// for the best 16 of 4 beams; the vocabulary adds little (256 rows of 32768 10.6).
// ---------------------------------------------------------------------------

namespace {

constexpr int kBeamWaves = kBeamBlock / 64;

struct ListEntry {
  float x;
  int32_t i;
};

struct BeamShared {
  uint32_t keys[kBeamBlock];
  int32_t chosen[kMaxBeamK];
  float least;
  float best[kBeamWaves];
  double weight;   // ln of the row's weights' sum against its largest score
  uint32_t n[3];
  uint32_t turn;
  BeamCandidate out[kMaxBeamK];
};

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

// f(entry, how many of the list's n come before it) for each entry of which
// fewer than k do: by one wave in registers where they fit one, else by all.
template <class F>
__device__ __forceinline__ void rank_list(const ListEntry* list, int n, int k, F&& f) {
  const int t = threadIdx.x;
  if (n <= 64) {
    if (t >= 64) return;
    const ListEntry e = t < n ? list[t] : ListEntry{0.0f, 0};
    const uint64_t mine = t < n ? (uint64_t)fkey(e.x) << 32 | (0xFFFFFFFFu - (uint32_t)e.i) : 0u;
    int c = 0;
    // (lanes by number: eight at a time take what one did with a running index)
#pragma unroll
    for (int j0 = 0; j0 < 64; j0 += 8) {
      if (j0 >= n) break;
#pragma unroll
      for (int j = j0; j < j0 + 8; ++j) {
        const uint64_t other = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine >> 32), j) << 32 |
                               (uint32_t)__builtin_amdgcn_readlane((int)mine, j);
        c += other > mine ? 1 : 0;
      }
    }
    if (t < n && c < k) f(e, c);
    return;
  }
  for (int o = t; o < n; o += kBeamBlock) {
    const ListEntry e = list[o];
    int c = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const ListEntry b = list[j];
      c += (b.x > e.x || (b.x == e.x && b.i < e.i)) ? 1 : 0;
    }
    if (c < k) f(e, c);
  }
}

// The largest value whose lowest `low` bits are zero that at least k of the
// wave's keys (N a lane) reach: two bits at a time.
template <int N>
__device__ __forceinline__ uint32_t kth_key(const uint32_t (&key)[N], int k, int low) {
  uint32_t thr = 0;
#pragma unroll 1
  for (int b = 30; b >= low; b -= 2) {
    int n[3] = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int d = 0; d < 3; ++d) n[d] += __popcll(__ballot(key[i] >= (thr | ((uint32_t)(d + 1) << b))));
    thr |= (uint32_t)((n[0] >= k) + (n[1] >= k) + (n[2] >= k)) << b;
  }
  return thr;
}

}  // namespace

// NV: 16-byte pieces of chunk maxima that a thread holds.
template <class T, int NV>
__global__ void __launch_bounds__(kBeamBlock) beam_row_kernel(const BeamParams q) {
  extern __shared__ __align__(16) unsigned char lds[];
  __shared__ BeamShared sh;
  const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
  const int row = blockIdx.x, req = row / q.beams, beam = row - req * q.beams;
  const int k = q.k, segs = q.segments;
  // a wave holds NV * 256 neighbouring chunks, a lane four in each piece (asked
  // for before it is known whether the beam reads them)
  const int chunks = segs * 64, c0 = wv * NV * 256 + lane * 4;
  const float* maxima = q.chunks + (int64_t)row * chunks;
  float v[NV][4];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float4 x{-__builtin_inff(), -__builtin_inff(), -__builtin_inff(), -__builtin_inff()};
    if (c0 + j * 256 < chunks) x = *reinterpret_cast<const float4*>(maxima + c0 + j * 256);
    v[j][0] = x.x, v[j][1] = x.y, v[j][2] = x.z, v[j][3] = x.w;
  }
  const float score = q.scores[row];
  const bool ended = q.ended && q.ended[row];
  const bool reads = offers(score) && !ended;
  double norm = 1.0;
  // (within bounds that leave every rank a number)
  if (q.lengths && q.penalty != 0.0)
    norm = fmin(fmax(pow((double)max((int64_t)q.lengths[row] + (ended ? 0 : 1), (int64_t)1), q.penalty), 0x1p-500),
                0x1p500);
  if (t < k) sh.out[t] = BeamCandidate{-__builtin_inf(), -__builtin_inff(), -1};
  if (t < 3) sh.n[t] = 0;

  ListEntry* list = reinterpret_cast<ListEntry*>(lds);
  if (offers(score) && ended) {
    __syncthreads();
    if (t == 0) sh.out[0] = BeamCandidate{(double)score / norm, score, q.end_token};
  } else if (reads) {
    float top = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) top = fmaxf(top, v[j][e]);
    float four = fmaxf(top, __shfl_xor(top, 1));
    four = fmaxf(four, __shfl_xor(four, 2));
    if ((lane & 3) == 0) sh.keys[t >> 2] = fkey(four);
    float low = top, best = top;
    wave_minmax(low, best);
    if (lane == 0) sh.best[wv] = best;
    __syncthreads();
    float m = sh.best[0];
#pragma unroll
    for (int w = 1; w < kBeamWaves; ++w) m = fmaxf(m, sh.best[w]);
    if (m > -__builtin_inff()) {
      const uint32_t sets[2] = {sh.keys[lane], sh.keys[64 + lane]};
      const uint32_t thr = max(kth_key(sets, k, 16), fkey(-__builtin_inff()) + 1u);
      const uint32_t room = (uint32_t)q.cap;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        // the four of a piece together: one count of the list's entries
        uint64_t in[4];
        uint32_t all = 0, at = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          in[e] = __ballot(fkey(v[j][e]) >= thr);
          all += (uint32_t)__popcll(in[e]);
        }
        if (all == 0) continue;
        if (lane == 0) at = atomicAdd(&sh.n[0], all);
        at = __builtin_amdgcn_readfirstlane(at);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t mine = at + __builtin_amdgcn_mbcnt_hi((uint32_t)(in[e] >> 32),
                                                               __builtin_amdgcn_mbcnt_lo((uint32_t)in[e], 0u));
          if ((in[e] >> lane & 1) && mine < room) list[mine] = ListEntry{v[j][e], c0 + j * 256 + e};
          at += (uint32_t)__popcll(in[e]);
        }
      }
      __syncthreads();
      int n = (int)sh.n[0];
      if (n > q.cap) {
        // too many: to the bit, and of equal ones each wave's first k
        sh.keys[t] = fkey(top);
        __syncthreads();
        uint32_t all[kBeamWaves];
#pragma unroll
        for (int i = 0; i < kBeamWaves; ++i) all[i] = sh.keys[i * 64 + lane];
        const float floor = from_key(kth_key(all, k, 0));
        int ties = 0;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          uint64_t even[4];
          int rank = ties;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            even[e] = __ballot(v[j][e] == floor && v[j][e] > -__builtin_inff());
            rank += (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(even[e] >> 32),
                                                   __builtin_amdgcn_mbcnt_lo((uint32_t)even[e], 0u));
            ties += __popcll(even[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool tie = even[e] >> lane & 1;
            const bool in = v[j][e] > floor || (tie && rank < k);
            rank += tie ? 1 : 0;
            const uint32_t at = append(in, &sh.n[1]);
            if (in) list[at] = ListEntry{v[j][e], c0 + j * 256 + e};
          }
        }
        __syncthreads();
        n = (int)sh.n[1];
      }
      const int picked = min(n, k);
      rank_list(list, n, k, [&](const ListEntry& e, int r) {
        sh.chosen[r] = e.i;
        if (r == picked - 1) sh.least = n >= k ? e.x : -__builtin_inff();
      });
      if (wv == 1) {
        // the row's sum, segment by segment in one order
        const float* bests = q.bests + (int64_t)row * segs;
        const double* masses = q.masses + (int64_t)row * segs;
        const Exp2Poly poly;
        double sum = 0.0;
        for (int s = lane; s < segs; s += 64) {
          const float b = bests[s];
          const double w = b == m ? 1.0 : exp2_64(((double)b - (double)m) * kLog2e, poly);
          sum += w > 0.0 ? masses[s] * w : 0.0;
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
        if (lane == 0) sh.weight = log(sum);
      }
      __syncthreads();
      const float least = sh.least;
      const unsigned char* base = static_cast<const unsigned char*>(q.logits) +
                                  (int64_t)row * q.row_stride * (int64_t)sizeof(T);
      for (int i0 = 0; i0 < picked * kChunk; i0 += kBeamBlock) {
        const int i = i0 + t;
        float x = -__builtin_inff();
        int pos = 0;
        if (i < picked * kChunk) {
          pos = sh.chosen[i / kChunk] * kChunk + i % kChunk;
          if (pos < q.vocab) x = Elem<T>::load(base, pos);
        }
        const bool in = x > -__builtin_inff() && x >= least && (m < __builtin_inff() || x == m);
        const uint32_t at = append(in, &sh.n[2]);
        if (in) list[at] = ListEntry{x, pos};
      }
      __syncthreads();
      const double weight = sh.weight;
      rank_list(list, (int)sh.n[2], k, [&](const ListEntry& e, int r) {
        // (differences first: the largest score may be far larger than they are)
        const double total = (double)score + ((m == __builtin_inff() ? 0.0 : (double)e.x - (double)m) - weight);
        sh.out[r] = BeamCandidate{total / norm, (float)total, e.i};
      });
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
    sh.n[0] = 0;
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
  // up to 512 are counted: those before one in the list that are not less, those
  // behind it that are more (lists stand in falling order, ties by beam), by up
  // to 32 neighbouring threads each
  int sharers = 1;
  while (sharers < 32 && 2 * sharers * all <= kBeamBlock) sharers *= 2;
  for (int n = t; n < all * sharers; n += kBeamBlock) {
    const int i = n / sharers, first = n - i * sharers;
    BeamCandidate c;
    c.rank = rank[i];
    __builtin_memcpy(&c.total, &rest[i], 8);
    const int b = i / k;
    int place = 0;
    if (all <= kBeamBlock) {
#pragma unroll 4
      for (int j = first; j < all; j += sharers)
        place += (rank[j] > c.rank || (rank[j] == c.rank && j < i)) ? 1 : 0;
      for (int d = 1; d < sharers; d <<= 1) place += __shfl_xor(place, d);
    }
    if (first > 0 || c.token < 0) continue;
    atomicAdd(&sh.n[0], 1u);
    if (all > kBeamBlock) {
      place = i - b * k;
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
    }
    if (place < k) {
      const int64_t at = (int64_t)req * k + place;
      q.out_scores[at] = c.total;
      q.parents[at] = b;
      q.tokens[at] = c.token;
    }
  }
  __syncthreads();
  for (int i = (int)sh.n[0] + t; i < k; i += kBeamBlock) {
    const int64_t at = (int64_t)req * k + i;
    q.out_scores[at] = -__builtin_inff();
    q.parents[at] = -1;
    q.tokens[at] = -1;
  }
}

namespace {

template <class T>
const void* beam_row_ptr(int pieces) {
  switch (pieces) {
    case 1: return reinterpret_cast<const void*>(&beam_row_kernel<T, 1>);
    case 2: return reinterpret_cast<const void*>(&beam_row_kernel<T, 2>);
    case 4: return reinterpret_cast<const void*>(&beam_row_kernel<T, 4>);
    default: return reinterpret_cast<const void*>(&beam_row_kernel<T, 16>);
  }
}

}  // namespace

const void* beam_segment_kernel_ptr(int dtype) {
  return dtype == 0 ? reinterpret_cast<const void*>(&beam_segment_kernel<float>)
         : dtype == 1 ? reinterpret_cast<const void*>(&beam_segment_kernel<__hip_bfloat16>)
                      : reinterpret_cast<const void*>(&beam_segment_kernel<__half>);
}
const void* beam_row_kernel_ptr(int dtype, int pieces) {
  return dtype == 0 ? beam_row_ptr<float>(pieces)
         : dtype == 1 ? beam_row_ptr<__hip_bfloat16>(pieces) : beam_row_ptr<__half>(pieces);
}

}  // namespace ert
