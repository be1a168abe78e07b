// sample.hip -- one token per row from its logits: temperature, top-k, top-p,
// min-p and a given uniform number.
//
// With m the row's largest live score (NaN and -inf are not live) and weights
// w_i = exp((x_i - m) / T), all three cuts keep a prefix of one order (score
// descending, then index ascending), and the token is the first index at
// which the kept weights' running sum in INDEX order passes u times their
// total.  So a row needs its maximum, one or two crossings in value order and
// one crossing in index order; nothing is sorted.
//
// Weights are whole numbers: 2^43 times the value, rounded once, from an
// exponential good to 46 bits in 64-bit arithmetic.  Their sums are exact in
// 64 bits (at most 2^20 weights of at most 2^43) and the same in every order,
// so atomics and splits never change a token.  Weights of 2^-44 of the largest
// and less are zero, and such a token is never drawn.
//
// A weight is off by at most half a unit, 2^-44 of the largest (equal scores
// all to the same side), and 2^-45 of itself, so a token differs from the
// real-number definition only if u Z lies within vocab * 2^-44 and 2^-44 Z of
// a border: 6e-8 for 2^20 equal scores at worst, about 1e-11 for ordinary
// rows.  Two sums are taken before the row's largest score is known, each
// segment against its own and then brought to the row's unit: the total of a
// row without a cut, and the total that a top-p without a top-k takes its
// share of.  They are off by no more than that either, but not by the same
// amount as a sum of the row's weights.  Segments whose largest score weighs
// nothing in the row add nothing to them.
//
// Three launches, the third only where a row may have a cut: the segment
// kernel reads the logits once, a wave for each 2048 scores; the row kernel
// finishes every row whose cuts lie among the candidates the segments hand
// on (or that has none); the wide kernel finishes rows whose cut lies lower.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gvr_device.h"
#include "rowops.h"

namespace ert {

namespace {

constexpr uint64_t kOne = 1ull << 43;   // the weight of a row's largest score
constexpr double kLn2 = 0.6931471805599453;
constexpr double kTmax = 44.0;          // weights of 2^-44 and less are zero

// The weights of a row's scores against m >= x.
//
// raw(x): round(2^43 * 2^s), s = (x - m) log2(e) / T <= 0, under the exponent
// bits of 2^52: adding 1.5 * 2^52 rounds s to a whole n, which then stands in
// the sum's low bits; adding 2^52 to the scaled value rounds it to a whole
// number in the low 52 bits.  s below -60 (or NaN) is taken as -60 and gives
// zero.  Callers that add many of them up take the exponent bits out once.
constexpr uint64_t kRaw = 0x4330000000000000ull;
struct Weigher {
  Exp2Poly poly;
  float m;
  double md, c;
  __device__ __forceinline__ Weigher(float m_, double c_) : m(m_), md((double)m_), c(c_) {}
  __device__ __forceinline__ void against(float m_) {
    m = m_;
    md = (double)m_;
  }
  __device__ __forceinline__ double log2_of(float x) const { return ((double)x - md) * c; }
  __device__ __forceinline__ uint64_t raw_of(double s) const {
    const double magic = 6755399441055744.0;
    s = __builtin_fmax(s, -60.0);
    const double sm = s + magic;
    const double p = poly(s - (sm - magic));
    const uint32_t hi = ((uint32_t)__double_as_longlong(sm) << 20) + ((1023u + 43u) << 20);
    return (uint64_t)__double_as_longlong(
        __builtin_fma(p, __hiloint2double((int)hi, 0), 4503599627370496.0));
  }
  __device__ __forceinline__ uint64_t raw(float x) const { return raw_of(log2_of(x)); }
  // x == m also covers m = +inf, beside which nothing else weighs anything
  __device__ __forceinline__ uint64_t operator()(float x) const {
    return x == m ? kOne : raw(x) - kRaw;
  }
  // scores that take part in cuts: weights above 2^-44
  __device__ __forceinline__ bool drawable(float x) const { return x == m || log2_of(x) > -kTmax; }
  // the weight of a drawable score, zero for others
  __device__ __forceinline__ uint64_t drawn(float x) const {
    const double s = log2_of(x);
    return x == m ? kOne : s > -kTmax ? raw_of(s) - kRaw : 0ull;
  }
};

// What a row asks for.
struct RowAsk {
  bool greedy;      // T is not > 0: the first of the order
  bool cut_k;       // 0 < top_k < vocab
  bool cut_p;       // top_p < 1
  int k;
  double p;
  uint64_t min_w;   // weights below this are cut by min-p (0: none)
  double c;         // log2(e) / T

  __device__ __forceinline__ bool cuts() const { return cut_k || cut_p || min_w > 0; }
};

__device__ __forceinline__ RowAsk row_ask(const SampleParams& q, int row) {
  RowAsk a;
  const float T = q.temperature ? q.temperature[row] : 1.0f;
  const float p = q.top_p ? q.top_p[row] : 1.0f;
  const float mp = q.min_p ? q.min_p[row] : 0.0f;
  a.k = q.top_k ? q.top_k[row] : 0;
  a.greedy = !(T > 0.0f);
  a.c = a.greedy ? 0.0 : kLog2e / (double)T;
  a.cut_k = a.k > 0 && a.k < q.vocab;
  a.cut_p = p < 1.0f;
  a.p = p > 0.0f ? (double)p : 0.0;
  a.min_w = mp > 0.0f ? (uint64_t)__builtin_ceil((mp < 1.0f ? (double)mp : 1.0) * (double)kOne) : 0ull;
  return a;
}

// A row's scores as whole 16-byte groups from the boundary at or below its
// first score; positions outside [0, vocab) read as -inf.
template <class T>
struct RowView {
  const unsigned char* base;  // 16-byte aligned
  int lead;                   // scores between base and the row's first
  int vocab;

  __device__ __forceinline__ RowView(const SampleParams& q, int row) {
    const unsigned char* p =
        static_cast<const unsigned char*>(q.logits) + (int64_t)row * q.row_stride * (int64_t)sizeof(T);
    lead = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    base = p - lead * (int)sizeof(T);
    vocab = q.vocab;
  }
  // Group g of those that lie inside the row: its scores, NaN as -inf.
  __device__ __forceinline__ void inner_group(int g, float (&x)[Elem<T>::kVec]) const {
    Elem<T>::unpack(*reinterpret_cast<const uint4*>(base + (int64_t)g * 16), x);
#pragma unroll
    for (int e = 0; e < Elem<T>::kVec; ++e)
      x[e] = x[e] > -__builtin_inff() ? x[e] : -__builtin_inff();
  }
  // whether groups [g, g + n) lie inside the row
  __device__ __forceinline__ bool inside(int g, int n) const {
    return g * Elem<T>::kVec >= lead && (g + n) * Elem<T>::kVec - lead <= vocab;
  }
  // One wave's segment, all its loads at once.
  static constexpr int kGroups = kSegment / (64 * Elem<T>::kVec);
  __device__ __forceinline__ void segment(int seg, int lane, float (&x)[kGroups][Elem<T>::kVec]) const {
    const int g0 = seg * (kSegment / Elem<T>::kVec);
    if (inside(g0, kSegment / Elem<T>::kVec)) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) inner_group(g0 + g * 64 + lane, x[g]);
    } else {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) group(g0 + g * 64 + lane, x[g]);
    }
  }
  // Group g: its scores, NaN as -inf, and the position of the first.
  __device__ __forceinline__ int group(int g, float (&x)[Elem<T>::kVec]) const {
    constexpr int V = Elem<T>::kVec;
    const int pos = g * V - lead;
    uint4 raw{0, 0, 0, 0};
    if (pos < vocab && pos + V > 0) raw = *reinterpret_cast<const uint4*>(base + (int64_t)g * 16);
    Elem<T>::unpack(raw, x);
#pragma unroll
    for (int e = 0; e < V; ++e)
      x[e] = ((unsigned)(pos + e) < (unsigned)vocab && x[e] > -__builtin_inff()) ? x[e]
                                                                               : -__builtin_inff();
    return pos;
  }
};

// Prefix sums over a wave of 4- and 8-byte values with DPP row shifts and
// broadcasts (no LDS: a 64-bit scan by ds_bpermute takes six times as long).
template <int CTL, int ROWS, class V>
__device__ __forceinline__ V dpp_from(V v) {  // 0 where there is no source lane
  uint32_t w[sizeof(V) / 4];
  __builtin_memcpy(w, &v, sizeof(V));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i)
    w[i] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[i], CTL, ROWS, 0xf, false);
  __builtin_memcpy(&v, w, sizeof(V));
  return v;
}
template <class V>
__device__ __forceinline__ V wave_scan(V v) {
  v += dpp_from<0x111, 0xf>(v);  // row_shr 1, 2, 4, 8
  v += dpp_from<0x112, 0xf>(v);
  v += dpp_from<0x114, 0xf>(v);
  v += dpp_from<0x118, 0xf>(v);
  v += dpp_from<0x142, 0xa>(v);  // row_bcast 15, 31
  v += dpp_from<0x143, 0xc>(v);
  return v;
}
// The sum, in every lane.
template <class V>
__device__ __forceinline__ V wave_sum(V v) {
  v = wave_scan(v);
  uint32_t w[sizeof(V) / 4];
  __builtin_memcpy(w, &v, sizeof(V));
#pragma unroll
  for (int i = 0; i < (int)(sizeof(V) / 4); ++i)
    w[i] = (uint32_t)__builtin_amdgcn_readlane((int)w[i], 63);
  __builtin_memcpy(&v, w, sizeof(V));
  return v;
}
__device__ __forceinline__ int wave_min(int v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d));
  return v;
}

}  // namespace

// ---------------------------------------------------------------------------
// Segment kernel: one wave reads 2048 scores of a row into registers, once,
// and writes what the row kernel needs of them: the largest, the weights'
// sum against it (rows whose draw or top-p needs the whole row's), and the
// candidates of a row with cuts.
//
// Candidates: the j-th largest of the 64 lanes' maxima is at most the
// segment's j-th largest score, so at least j scores lie at or above it; an
// 18-bit prefix of its key, found with ballots, is a floor that needs no
// barrier and no atomics.  All live scores at or above the floor are handed
// on.
//
// Bound by 64-bit arithmetic where the weights are summed (about 20
// instructions a score), close behind it by reading: 256 x 131072 fp32, 134
// MB, 31.0 us, where a copy of as much runs at 5.2 TB/s (26 us) and the
// instructions alone take about 22; with weights in flight for all of a
// lane's 32 scores and constants in vector registers it took 54.  CUTS false
// leaves the candidates' code out where no row of the call can have a cut (74
// registers, six waves a SIMD, instead of 108 and four).
// ---------------------------------------------------------------------------
template <class T, bool CUTS>
__global__ void __launch_bounds__(256) sample_segment_kernel(const SampleParams q) {
  constexpr int V = Elem<T>::kVec;
  constexpr int G = kSegment / (64 * V);
  const int lane = threadIdx.x & 63;
  const uint32_t id = __builtin_amdgcn_readfirstlane(blockIdx.x * 4u + (threadIdx.x >> 6));
  if (id >= (uint32_t)q.rows * (uint32_t)q.segments) return;
  const int row = (int)(id / (uint32_t)q.segments);
  const int seg = (int)(id - (uint32_t)row * (uint32_t)q.segments);
  const RowAsk ask = row_ask(q, row);
  const RowView<T> view(q, row);

  float x[G][V];
  const int g0 = seg * (kSegment / V);
  view.segment(seg, lane, x);

  float top = -__builtin_inff();
#pragma unroll
  for (int g = 0; g < G; ++g)
#pragma unroll
    for (int e = 0; e < V; ++e) top = fmaxf(top, x[g][e]);
  float best = top, low = __builtin_inff();
  if (CUTS && ask.cuts() && !ask.greedy) {
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e)
        low = fminf(low, x[g][e] > -__builtin_inff() ? x[g][e] : __builtin_inff());
  }
  wave_minmax(low, best);

  SegRecord rec;
  rec.best = best;
  rec.first = 0x7FFFFFFF;
  rec.floor = -__builtin_inff();
  rec.count = 0;
  rec.mass = 0;
  rec.low = low;
  rec.upper = 0.0f;
  if (best > -__builtin_inff()) {
    if (ask.greedy) {
      int first = 0x7FFFFFFF;
#pragma unroll
      for (int g = G - 1; g >= 0; --g)
#pragma unroll
        for (int e = V - 1; e >= 0; --e)
          if (x[g][e] == best) first = (g0 + g * 64 + lane) * V + e - view.lead;
      rec.first = wave_min(first);
    } else {
      float floor = __builtin_inff();
      if (CUTS && ask.cuts()) {
        // How many candidates a segment should hand on: its share of a row's
        // best k and room for an uneven spread, within what fits; 16 where
        // only the weights say how many are needed.  With j of the 64 lane
        // maxima at or above the floor, about -64 ln(1 - j / 64) scores are.
        // (64 x 16000: top-k 300, whose candidates fit, takes 20 us, top-k
        // 1000, whose do not, 33.)
        float want = 16.0f;
        if (ask.cut_k) {
          const float share = (float)ask.k / (float)q.segments;
          want = fminf(share + 4.0f * __builtin_sqrtf(share) + 4.0f, 88.0f);
        }
        const int j = 1 + (int)(64.0f * (1.0f - __expf(want * (-1.0f / 64.0f))));
        const uint32_t key = fkey(top);
        uint32_t thr = 0;
#pragma unroll
        for (int b = 31; b >= 14; --b) {
          const uint32_t t = thr | (1u << b);
          if (__popcll(__ballot(key >= t)) >= j) thr = t;
        }
        floor = thr > fkey(-__builtin_inff()) ? from_key(thr) : -__builtin_inff();
        Candidate* out = q.candidates + (int64_t)id * kSegSlots;
        int n = 0;
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const bool in = x[g][e] >= floor && x[g][e] > -__builtin_inff();
            const uint64_t mask = __ballot(in);
            if (mask == 0) continue;
            const int at = n + (int)__builtin_amdgcn_mbcnt_hi(
                                   (uint32_t)(mask >> 32),
                                   __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
            if (in && at < kSegSlots)
              out[at] = Candidate{x[g][e], (g0 + g * 64 + lane) * V + e - view.lead};
            n += __popcll(mask);
          }
        rec.floor = floor;
        rec.count = n <= kSegSlots ? n : -1;
      }
      if (!CUTS || !ask.cut_k) {
        if (best == __builtin_inff()) {
          uint32_t n = 0;
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < V; ++e) n += x[g][e] == best ? 1u : 0u;
          rec.mass = wave_sum((uint64_t)n * kOne);
        } else {
          // Four scores at a time (the empty asm keeps the additions where
          // they are): with all of them in flight, and added up at the end,
          // the registers would leave room for three waves a SIMD, not six
          // (four with the cuts' code).  (One loop for all rows: of two, the
          // compiler shares the conversions, which then stay in registers
          // across both.)
          uint64_t mass = 0, top_mass = 0;
          const Weigher w(best, ask.c);
#pragma unroll
          for (int g = 0; g < G; ++g)
#pragma unroll
            for (int e = 0; e < V; ++e) {
              const uint64_t v = w.raw(x[g][e]);
              mass += v;
              if (CUTS) top_mass += x[g][e] >= floor ? v : kRaw;
              if (e % 4 == 3) {
                asm("" : "+v"(mass), "+v"(top_mass));
                __builtin_amdgcn_sched_barrier(0);
              }
            }
          rec.mass = wave_sum(mass - (uint64_t)(G * V) * kRaw);
          if (CUTS) rec.upper = (float)wave_sum(top_mass - (uint64_t)(G * V) * kRaw) * 1.000001f;
        }
      }
    }
  }
  if (lane == 0) {
    q.records[id] = rec;
    if (CUTS && seg == 0) {
      q.wide[row].state = kWideDone;
      q.wide[row].arrived[0] = 0;
      q.wide[row].arrived[1] = 0;
    }
  }
}

// ---------------------------------------------------------------------------
// Row kernel: one workgroup per row, or one per kWideSegs segments for rows
// whose top-k or top-p may lie below the candidates.
//
// Bound by its own chain of scans and barriers, not by work: one row of 32768
// with all cuts takes 9.2 us, of which reading the records is 1.3, the
// candidates 1.8, ranking them with both cuts 2.5 and the draw 1.5 (11 us with
// a histogram for each cut, which longer lists take).
// ---------------------------------------------------------------------------

namespace {

constexpr int kShort = 256;    // members of a bin that are ranked directly
constexpr int kListS = 2048;   // candidates held in LDS
constexpr int kMaxSegments = (kMaxVocab + 7 + kSegment - 1) / kSegment;
static_assert(kMaxSegments <= kBinsS, "the bins hold a row's segments");

struct RowShared {
  uint32_t cnt[kBinsS];
  uint64_t mass[kBinsS];
  uint64_t sk[kShort];  // sort keys, larger first
  uint64_t sw[kShort];
  uint64_t red[32];
  double redd[32];
  float redf[64];
  uint32_t n;
  int32_t bin;
  int32_t found_i;
  float found_x;
  uint64_t before;
  uint32_t list_n;
  union {
    struct {
      float lx[kListS];
      int32_t li[kListS];
      uint64_t lw[kListS];
    };
    float dense[kWideSegs][64 + 256];  // each wave's scores on their way to a weight
  };
  float seg_best[kMaxSegments];
  uint64_t seg_mass[kMaxSegments];
  float seg_upper[kMaxSegments];
  int32_t seg_count[kMaxSegments];
};

// Everything of the order up to and including (x, i).
struct Cut {
  float x;
  int32_t i;
  __device__ __forceinline__ bool holds(float y, int j) const { return y > x || (y == x && j <= i); }
};

// The candidates in LDS.
struct ListSource {
  const float* x;
  const int32_t* i;
  const uint64_t* v;  // their weights
  int n;
  template <int BLOCK, class F>
  __device__ __forceinline__ void visit(F&& f) const {
    for (int t = threadIdx.x; t < n; t += BLOCK) f(x[t], i[t], [&] { return v[t]; });
  }
};

// The live scores of a row in memory, of `groups` groups.
template <class T>
struct RowSource {
  RowView<T> view;
  const Weigher& weigh;
  int groups;
  template <int BLOCK, class F>
  __device__ __forceinline__ void visit(F&& f) const {
    constexpr int V = Elem<T>::kVec;
    for (int g = threadIdx.x; g < groups; g += BLOCK) {
      const int pos = g * V - view.lead;
      uint4 raw = *reinterpret_cast<const uint4*>(view.base + (int64_t)g * 16);
      // one 32-bit word at a time: the callers' code appears once or twice,
      // not once for each score of the group
#pragma unroll 1
      for (int w = 0; w < 4; ++w) {
        float x[V / 4];
        Elem<T>::unpack_word(raw.x, x);
#pragma unroll
        for (int e = 0; e < V / 4; ++e) {
          const int i = pos + w * (V / 4) + e;
          if ((unsigned)i < (unsigned)view.vocab && x[e] > -__builtin_inff())
            f(x[e], i, [&] { return weigh(x[e]); });
        }
        raw.x = raw.y;
        raw.y = raw.z;
        raw.z = raw.w;
      }
    }
  }
};

template <int BLOCK, class V>
__device__ __forceinline__ V block_sum(V v, V* red) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  V s = red[0];
#pragma unroll
  for (int w = 1; w < BLOCK / 64; ++w) s += red[w];
  return s;
}

template <int BLOCK>
__device__ __forceinline__ void block_sum2(double& a, double& b, double* red) {
  a = wave_sum(a);
  b = wave_sum(b);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = a;
    red[BLOCK / 64 + (threadIdx.x >> 6)] = b;
  }
  __syncthreads();
  a = red[0];
  b = red[BLOCK / 64];
#pragma unroll
  for (int w = 1; w < BLOCK / 64; ++w) {
    a += red[w];
    b += red[BLOCK / 64 + w];
  }
}

template <int BLOCK>
__device__ __forceinline__ void block_min_max(float& lo, float& hi, float* red) {
  wave_minmax(lo, hi);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = lo;
    red[32 + (threadIdx.x >> 6)] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < BLOCK / 64; ++w) {
    lo = fminf(lo, red[w]);
    hi = fmaxf(hi, red[32 + w]);
  }
}

// Inclusive prefix sum over the workgroup in thread order.
template <int BLOCK, class V>
__device__ __forceinline__ V block_scan(V v, V* red) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  v = wave_scan(v);
  __syncthreads();
  if (lane == 63) red[wv] = v;
  __syncthreads();
  V off = 0;
#pragma unroll
  for (int w = 0; w < BLOCK / 64; ++w) off += w < wv ? red[w] : (V)0;
  return off + v;
}

template <int BLOCK>
__device__ __forceinline__ void clear_bins(RowShared& sh) {
  __syncthreads();
  for (int b = threadIdx.x; b < kBinsS; b += BLOCK) {
    sh.cnt[b] = 0;
    sh.mass[b] = 0;
  }
  if (threadIdx.x == 0) {
    sh.n = 0;
    sh.bin = -1;
  }
  __syncthreads();
}

// The first bin at which the running sum of the counts (or masses) reaches
// `need`, and the sum before it; false if the total stays below.
template <int BLOCK, bool MASS>
__device__ __forceinline__ bool cross_bins(RowShared& sh, uint64_t need, int& bin, uint64_t& before) {
  constexpr int PER = kBinsS / BLOCK;
  __syncthreads();
  uint64_t own = 0;
#pragma unroll
  for (int e = 0; e < PER; ++e) {
    const int b = threadIdx.x * PER + e;
    own += MASS ? sh.mass[b] : (uint64_t)sh.cnt[b];
  }
  const uint64_t incl = block_scan<BLOCK>(own, sh.red);
  uint64_t run = incl - own;
  if (run < need && need <= incl) {
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int b = threadIdx.x * PER + e;
      const uint64_t v = MASS ? sh.mass[b] : (uint64_t)sh.cnt[b];
      if (run < need && need <= run + v) {
        sh.bin = b;
        sh.before = run;
      }
      run += v;
    }
  }
  __syncthreads();
  bin = sh.bin;
  before = sh.before;
  return bin >= 0;
}

// Sort keys of the order (score descending, index ascending) and of index
// order alone; the larger key comes first.
__device__ __forceinline__ uint64_t order_key(float x, int i) {
  return ((uint64_t)fkey(x) << 32) | (uint32_t)~i;
}
__device__ __forceinline__ uint64_t index_key(float x, int i) {
  return ((uint64_t)(uint32_t)~i << 32) | fkey(x);
}

// The short list's member at which the running sum by falling key reaches
// `need`, left in found_x / found_i.
template <bool MASS, bool BY_INDEX = false>
__device__ __forceinline__ void rank_short(RowShared& sh, int m, uint64_t need) {
  __syncthreads();
  const int t = threadIdx.x;
  if (t < m) {
    const uint64_t key = sh.sk[t];
    uint64_t run = 0;
#pragma unroll 8
    for (int o = 0; o < m; ++o) {
      const uint64_t v = MASS ? sh.sw[o] : 1ull;
      run += sh.sk[o] > key ? v : 0ull;
    }
    const uint64_t own = MASS ? sh.sw[t] : 1ull;
    if (run < need && need <= run + own) {
      const uint32_t hi = (uint32_t)(key >> 32), lo = (uint32_t)key;
      sh.found_x = from_key(BY_INDEX ? lo : hi);
      sh.found_i = (int)~(BY_INDEX ? hi : lo);
    }
  }
  __syncthreads();
}

// The lowest index at which the running count (or mass) of the scores that
// `pred` admits reaches `need`, in index order over [0, vocab); -1 if the
// total stays below.
template <int BLOCK, bool MASS, class Src, class Pred>
__device__ int find_index(const Src& src, RowShared& sh, int vocab, Pred&& pred, uint64_t need) {
  int i0 = 0, width = (vocab + kBinsS - 1) / kBinsS;
  for (;;) {
    clear_bins<BLOCK>(sh);
    src.template visit<BLOCK>([&](float x, int i, auto&& v) {
      const int d = i - i0;
      if (d >= 0 && d < width * kBinsS && pred(x, i)) {
        const int b = (int)((unsigned)d / (unsigned)width);
        atomicAdd(&sh.cnt[b], 1u);
        if (MASS) atomicAdd((unsigned long long*)&sh.mass[b], (unsigned long long)v());
      }
    });
    int bin;
    uint64_t before;
    if (!cross_bins<BLOCK, MASS>(sh, need, bin, before)) return -1;
    need -= before;
    i0 += bin * width;
    const int members = (int)sh.cnt[bin];
    if (width == 1 || members <= kShort) {
      src.template visit<BLOCK>([&](float x, int i, auto&& v) {
        const int d = i - i0;
        if (d >= 0 && d < width && pred(x, i)) {
          const uint32_t s = atomicAdd(&sh.n, 1u);
          if (s < (uint32_t)kShort) {
            sh.sk[s] = index_key(x, i);
            if (MASS) sh.sw[s] = v();
          }
        }
      });
      rank_short<MASS, true>(sh, min(members, kShort), need);
      return sh.found_i;
    }
    width = (width + kBinsS - 1) / kBinsS;
  }
}

// The lowest index of a segment at which the running mass of the scores that
// `pred` admits reaches `need` (or their total, which is not zero, if that is
// less), with its score: every thread's scores lie side by side, so one prefix
// sum over the workgroup finds the thread and a walk over its registers the
// score.
template <int BLOCK, class T, class Pred>
__device__ __forceinline__ void pick_in_segment(const RowView<T>& view, int seg, RowShared& sh,
                                                const Weigher& w, Pred&& pred, uint64_t need) {
  constexpr int V = Elem<T>::kVec;
  constexpr int N = kSegment / V;  // groups
  constexpr int PER = (N + BLOCK - 1) / BLOCK;
  float x[PER][V];
  uint64_t own = 0;
  const int g0 = threadIdx.x * PER;
#pragma unroll
  for (int g = 0; g < PER; ++g) {
    if (g0 + g < N) {
      view.group(seg * N + g0 + g, x[g]);
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[g][e] = -__builtin_inff();
    }
  }
  uint64_t v[PER][V];
#pragma unroll
  for (int g = 0; g < PER; ++g)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int i = (seg * N + g0 + g) * V + e - view.lead;
      v[g][e] = pred(x[g][e], i) ? w(x[g][e]) : 0ull;
      own += v[g][e];
    }
  const uint64_t incl = block_scan<BLOCK>(own, sh.red);
  uint64_t run = incl - own, total = 0;
#pragma unroll
  for (int o = 0; o < BLOCK / 64; ++o) total += sh.red[o];
  need = need < total ? need : total;
  if (run < need && need <= incl) {
#pragma unroll
    for (int g = 0; g < PER; ++g)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (run < need && need <= run + v[g][e]) {
          sh.found_i = (seg * N + g0 + g) * V + e - view.lead;
          sh.found_x = x[g][e];
        }
        run += v[g][e];
      }
  }
  __syncthreads();
}

// The place in the order (score descending, index ascending) at which the
// running count (or mass) of the drawable scores inside `within` reaches
// `need` (>= 1); `within` itself if the total stays below.  Each round splits
// the class's value range into equal bins, finds the crossing bin, and
// narrows the range to that bin's own extremes, which land in different bins
// next time; a class of one value is split by index.
template <int BLOCK, bool MASS, class Src>
__device__ Cut find_cut(const Src& src, RowShared& sh, const Weigher& w, float lo, float hi,
                        const Cut& within,
                        int vocab, uint64_t need) {
  for (;;) {
    clear_bins<BLOCK>(sh);
    const double range = (double)hi - (double)lo;
    const double s = (range > 0.0 && range < 1e300) ? (double)kBinsS / range : 0.0;
    auto bin_of = [&](float x) {
      if (!(s > 0.0)) return 0;
      const double b = ((double)hi - (double)x) * s;
      return b < (double)(kBinsS - 1) ? (int)b : kBinsS - 1;
    };
    auto admitted = [&](float x, int i) {
      return x <= hi && x >= lo && w.drawable(x) && within.holds(x, i);
    };
    src.template visit<BLOCK>([&](float x, int i, auto&& v) {
      if (admitted(x, i)) {
        const int b = bin_of(x);
        atomicAdd(&sh.cnt[b], 1u);
        if (MASS) atomicAdd((unsigned long long*)&sh.mass[b], (unsigned long long)v());
      }
    });
    int bin;
    uint64_t before;
    if (!cross_bins<BLOCK, MASS>(sh, need, bin, before)) return within;
    need -= before;
    const int members = (int)sh.cnt[bin];
    float mn = __builtin_inff(), mx = -__builtin_inff();
    src.template visit<BLOCK>([&](float x, int i, auto&& v) {
      if (admitted(x, i) && bin_of(x) == bin) {
        mn = fminf(mn, x);
        mx = fmaxf(mx, x);
        const uint32_t s = atomicAdd(&sh.n, 1u);
        if (s < (uint32_t)kShort) {
          sh.sk[s] = order_key(x, i);
          if (MASS) sh.sw[s] = v();
        }
      }
    });
    if (members <= kShort) {
      rank_short<MASS>(sh, members, need);
      return Cut{sh.found_x, sh.found_i};
    }
    block_min_max<BLOCK>(mn, mx, sh.redf);
    if (mn == mx) {
      // one value: its first `count` indices
      const uint64_t one = MASS ? w(mn) : 1ull;
      const uint64_t count = MASS ? (need + one - 1) / one : need;
      const int at = find_index<BLOCK, false>(
          src, sh, vocab, [&](float x, int i) { return x == mn && within.holds(x, i); }, count);
      return Cut{mn, at};
    }
    hi = mx;
    lo = mn;
  }
}

__device__ __forceinline__ uint64_t ceil_share(double p, double total) {
  const double need = __builtin_ceil(p * total);
  return need < 1.0 ? 1ull : (need >= total ? (uint64_t)total : (uint64_t)need);
}

__device__ __forceinline__ double clamp_uniform(float u) {
  return u > 0.0f ? (u < 0.99999994f ? (double)u : 0.99999994039535522) : 0.0;
}

// The drawn token, its score in the row, and the kept total.
__device__ __forceinline__ void put_token(const SampleParams& q, int row, int token, float x,
                                          const Weigher& w, double total) {
  if (threadIdx.x != 0) return;
  q.tokens[row] = token;
  if (q.logprobs)
    q.logprobs[row] =
        (float)((x == w.m ? 0.0 : w.log2_of(x) * kLn2) - log(total * (1.0 / (double)kOne)));
}

// The sum of the weights of a source's scores inside a cut that min-p keeps.
template <int BLOCK, class Src>
__device__ __forceinline__ uint64_t mass_in(const Src& src, RowShared& sh, const Weigher& w,
                                            const Cut& cut, uint64_t min_w) {
  uint64_t s = 0;
  src.template visit<BLOCK>([&](float x, int i, auto&& v) {
    if (cut.holds(x, i) && w.drawable(x)) {
      const uint64_t own = v();
      s += own >= min_w ? own : 0ull;
    }
  });
  return block_sum<BLOCK>(s, sh.red);
}

// The draw over a source's kept scores, left in found_i / found_x.
template <int BLOCK, class Src>
__device__ void draw_from(const Src& src, RowShared& sh, const Weigher& w, const Cut& cut,
                          uint64_t min_w, int vocab, double u, double& total) {
  const uint64_t z = mass_in<BLOCK>(src, sh, w, cut, min_w);
  total = (double)z;
  uint64_t need = (uint64_t)(u * total) + 1;
  if (need > z) need = z;
  find_index<BLOCK, true>(
      src, sh, vocab,
      [&](float x, int i) { return cut.holds(x, i) && w.drawn(x) >= (min_w ? min_w : 1ull); }, need);
}

// The same over a list: a few kept scores are ranked by index directly.
template <int BLOCK>
__device__ void draw_from_list(const ListSource& list, RowShared& sh, const Weigher& w, const Cut& cut,
                               uint64_t min_w, int vocab, double u, double& total) {
  __syncthreads();
  if (threadIdx.x == 0) sh.n = 0;
  __syncthreads();
  uint64_t s = 0;
  list.visit<BLOCK>([&](float x, int i, auto&& weight) {
    if (!cut.holds(x, i)) return;
    const uint64_t v = weight();
    if (v < min_w) return;
    s += v;
    const uint32_t at = atomicAdd(&sh.n, 1u);
    if (at < (uint32_t)kShort) {
      sh.sk[at] = index_key(x, i);
      sh.sw[at] = v;
    }
  });
  const uint64_t z = block_sum<BLOCK>(s, sh.red);
  const int n = (int)sh.n;
  if (n > kShort) {
    draw_from<BLOCK>(list, sh, w, cut, min_w, vocab, u, total);
    return;
  }
  total = (double)z;
  uint64_t need = (uint64_t)(u * total) + 1;
  if (need > z) need = z;
  rank_short<true, true>(sh, n, need);
}

// Of n >= 1 distinct keys (at most kShort; one a thread, 0 in the threads
// behind them, and equal zeros among them), how many are larger than this
// thread's.  All waves share the comparisons: each takes 64 keys against a
// part of the list.
template <int BLOCK>
__device__ __forceinline__ int rank_of(RowShared& sh, uint64_t key, int n) {
  const int t = threadIdx.x, wave = t >> 6;
  __syncthreads();
  if (t < kShort) {
    sh.sk[t] = key;
    sh.cnt[t] = 0;
  }
  __syncthreads();
  const int chunks = (n + 63) / 64;  // 1 .. 4
  const int slices = chunks == 1 ? BLOCK / 64 : chunks == 2 ? BLOCK / 128 : BLOCK / 256;
  const int slice = chunks == 1 ? wave : chunks == 2 ? wave >> 1 : wave >> 2;
  const int e = (chunks == 1 ? 0 : chunks == 2 ? wave & 1 : wave & 3) * 64 + (t & 63);
  const uint64_t own = sh.sk[e];
  const int per = ((n + slices - 1) / slices + 7) & ~7;
  uint32_t count = 0;
  for (int s = slice * per; s < min((slice + 1) * per, n); s += 8) {
#pragma unroll
    for (int o = 0; o < 8; ++o) count += sh.sk[s + o] > own ? 1u : 0u;
  }
  if (e < n && count) atomicAdd(&sh.cnt[e], count);
  __syncthreads();
  return t < kShort ? (int)sh.cnt[t] : 0;
}

// Cuts and draw over a list of at most kShort candidates: ranked against each
// other, one prefix sum of their weights gives the cuts; the kept ones ranked
// by index, another one the token.  `need` is top-p's mass where no top-k
// comes before it.
template <int BLOCK>
__device__ __forceinline__ void draw_ranked(const ListSource& list, RowShared& sh, const RowAsk& ask,
                                            uint64_t need, double u, double& total) {
  const int t = threadIdx.x, n = list.n;
  uint64_t key = t < n ? order_key(list.x[t], list.i[t]) : 0ull;
  uint64_t weight = t < n ? list.v[t] : 0ull;
  int at = rank_of<BLOCK>(sh, key, n);
  if (t < n) {
    sh.sk[at] = key;
    sh.mass[at] = weight;
  }
  __syncthreads();
  // from here on thread t holds the t-th of the order
  key = t < n ? sh.sk[t] : 0ull;
  weight = t < n ? sh.mass[t] : 0ull;
  int keep = ask.cut_k ? min(ask.k, n) : n;
  const uint64_t to = block_scan<BLOCK>(weight, sh.red);
  if (t == keep - 1) {
    sh.before = to;
    sh.bin = t;
  }
  __syncthreads();
  if (ask.cut_p) {
    if (ask.cut_k) need = ceil_share(ask.p, (double)sh.before);
    if (t < keep && to >= need && to - weight < need) sh.bin = t;
  }
  __syncthreads();
  keep = sh.bin + 1;
  if (t >= keep || weight < ask.min_w) weight = 0;
  at = rank_of<BLOCK>(sh, t < keep ? (uint64_t)(uint32_t)key : 0ull, keep);  // by ~index
  if (t < keep) sh.mass[at] = weight;
  __syncthreads();
  const uint64_t part = t < keep ? sh.mass[t] : 0ull;
  const uint64_t run = block_scan<BLOCK>(part, sh.red);
  if (t == keep - 1) sh.before = run;
  __syncthreads();
  const uint64_t z = sh.before;
  total = (double)z;
  uint64_t pick = (uint64_t)(u * total) + 1;
  if (pick > z) pick = z;
  if (run >= pick && run - part < pick) sh.bin = t;
  __syncthreads();
  if (t < keep && at == sh.bin) {
    sh.found_x = from_key((uint32_t)(key >> 32));
    sh.found_i = (int)~(uint32_t)key;
  }
  __syncthreads();
}

// What a segment's weights against its own best score come to against the
// row's: 2^(best - m), or nothing if even that score's weight is zero.
__device__ __forceinline__ double below_best(float best, const Weigher& w) {
  return best == w.m ? 1.0 : w(best) > 0 ? exp2_64(w.log2_of(best), w.poly) : 0.0;
}

// ---------------------------------------------------------------------------
// Rows whose cut lies below the candidates (flat rows with a top-p, a large
// top-k, a small min-p), kWideSegs segments a workgroup:
//  1. in the row kernel, the row's masses (top-p) and counts (top-k) in kBinsS
//     equal bins of score from the largest down; the row's last workgroup
//     adds the others' bins up and finds the crossing bins;
//  2. sample_wide_kernel: each segment's kept mass above those bins, and the
//     bins' members; the row's last workgroup finds the exact cut among the
//     members, adds the kept ones to their segments, finds the segment in
//     which the draw falls, and the token in it.
// Sums are whole numbers, so which workgroup is last changes nothing.  What
// crosses between workgroups goes through agent-scope atomics, complete
// before their workgroup counts itself; nobody waits for anybody.
// Of more members than fit, all of one value, the first so many are kept, found
// by their counts in the segments.  Rows with cuts and more +inf scores than
// are handed on, and bins with more members than fit of several values, are
// selected by one workgroup from memory, pass by pass.
//
// Both steps are bound by the exponentials (64 x 131072 with mixed cuts: row
// kernel 18.2 us, wide kernel 19.6, of which 8 each are the waves' work and
// the rest the last workgroup's chain of scans and look-ups).  One workgroup
// a row, from memory, took 395 us for the same rows, and 480 to 670 where
// both cuts lie low (now 78 to 88, the whole call).
// ---------------------------------------------------------------------------


// The bin of log2-weight s <= 0; `rate` bins an octave.
__device__ __forceinline__ int wide_bin(double s, double rate) {
  return min((int)(s * -rate), kBinsS - 1);
}

template <class V>
__device__ __forceinline__ V agent_load(const V* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <class V>
__device__ __forceinline__ void agent_store(V* p, V v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Counts this workgroup in; true in the row's last one.
__device__ __forceinline__ bool last_in(uint32_t* counter, int workgroups, RowShared& sh) {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // this wave's stores and atomics are done
  __syncthreads();
  if (threadIdx.x == 0)
    sh.bin = (int)__hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __syncthreads();
  const bool last = sh.bin == workgroups - 1;
  __syncthreads();
  return last;
}

// One wave's segment, as the segment kernel reads it, dead scores as -inf: f
// of four neighbouring scores of every lane and the first one's index, the
// code once with the scores moving up (unrolled, the callers' conversions to
// 64 bits are all made first and fill the registers; the times are the same).
template <class T, class F>
__device__ __forceinline__ void visit_fours(const RowView<T>& view, int seg, F&& f) {
  constexpr int V = Elem<T>::kVec;
  constexpr int G = RowView<T>::kGroups;
  const int lane = threadIdx.x & 63;
  float x[G][V], y[G * V];
  view.segment(seg, lane, x);
#pragma unroll
  for (int i = 0; i < G * V; ++i) y[i] = x[i / V][i % V];
#pragma unroll 1
  for (int r = 0; r < G * V / 4; ++r) {
    f(y, (seg * (kSegment / V) + r / (V / 4) * 64 + lane) * V + r % (V / 4) * 4 - view.lead);
#pragma unroll
    for (int i = 0; i + 4 < G * V; ++i) y[i] = y[i + 4];
  }
}

// One wave's segment again: f(x) for the scores that `take` admits, 64 at a
// time (-inf in the lanes behind the last), so that the exponentials run on
// full waves however few scores pass.  `buf` holds what is left over and four
// scores of every lane.
template <class T, class Take, class F>
__device__ __forceinline__ void visit_dense(const RowView<T>& view, int seg, float* buf, Take&& take,
                                            F&& f) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  visit_fours(view, seg, [&](const float* y, int pos) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool in = take(y[e], pos + e);
      const uint64_t mask = __ballot(in);
      const int at = n + (int)__builtin_amdgcn_mbcnt_hi(
                             (uint32_t)(mask >> 32),
                             __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0u));
      if (in) buf[at] = y[e];
      n += __popcll(mask);
    }
    wave_sync();
    while (n >= 64) {
      n -= 64;
      f(buf[n + lane]);
    }
    wave_sync();
  });
  if (n > 0) f(lane < n ? buf[lane] : -__builtin_inff());
}

// A drawable score's weight, else 0, for finite m: what Weigher::drawn gives.
__device__ __forceinline__ uint64_t drawn_at(const Weigher& w, double s) {
  const uint64_t v = w.raw_of(s) - kRaw;
  return s > -kTmax ? v : 0ull;
}

// This workgroup's wave adds its segment to the bins: the masses of the scores
// at or above `from` (top-p), counts (top-k), or both.
template <class T>
__device__ __forceinline__ void fill_bins(const RowView<T>& view, int seg, int nseg, RowShared& sh,
                                          const Weigher& w, double rate, float from, bool by_count,
                                          bool by_mass) {
  clear_bins<kWideBlock>(sh);
  if (seg < nseg) {
    if (!by_count)
      visit_dense(
          view, seg, sh.dense[threadIdx.x >> 6], [&](float x, int) { return x >= from; },
          [&](float x) {
            const double s = w.log2_of(x);
            const unsigned long long v = drawn_at(w, s);
            if (v) atomicAdd((unsigned long long*)&sh.mass[wide_bin(s, rate)], v);
          });
    else
      visit_fours(view, seg, [&](const float* y, int) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double s = w.log2_of(y[e]);
          if (s > -kTmax) {
            const int b = wide_bin(s, rate);
            atomicAdd(&sh.cnt[b], 1u);
            if (by_mass)
              atomicAdd((unsigned long long*)&sh.mass[b], (unsigned long long)drawn_at(w, s));
          }
        }
      });
  }
  __syncthreads();
}

// The lowest score of the bins up to `last`, by one wave: 64 probes a round
// over the keys.  NaN if there is no such bin, -inf for the last one.
__device__ __forceinline__ float bin_begin(int last, const Weigher& w, double rate) {
  if (last < 0) return __builtin_nanf("");
  if (!(rate > 0.0) || last >= kBinsS - 1) return -__builtin_inff();
  const uint32_t lane = threadIdx.x & 63;
  auto inside = [&](uint32_t key) { return wide_bin(w.log2_of(from_key(key)), rate) <= last; };
  uint32_t lo = fkey(-__FLT_MAX__), hi = fkey(w.m);  // hi lies in bin 0
  // mostly within 32 floats of where real arithmetic has it
  const double guess = (double)w.m - (double)(last + 1) / (rate * w.c);
  if (guess > -1e38) {
    const uint32_t probe = min(fkey((float)guess) - 32 + lane, hi);
    const uint64_t ok = __ballot(inside(probe));
    if (!(ok & 1) && ok) return from_key(__shfl(probe, __ffsll((unsigned long long)ok) - 1));
  }
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 64 + 1;
    const uint32_t probe = min(lo + lane * step, hi);
    const uint64_t ok = __ballot(inside(probe));
    const uint32_t f = (uint32_t)__ffsll((unsigned long long)ok);  // 1-based, 0: none
    const uint32_t old = lo;
    if (f == 1) hi = old;
    else if (f == 0) lo = min(old + 63 * step, hi) + 1;
    else {
      lo = old + (f - 2) * step + 1;
      hi = min(old + (f - 1) * step, hi);
    }
  }
  return from_key(hi);
}

// The crossing bins of a row's whole bins, handed to the wide kernel as the
// scores at which they begin and end.
//
// With both cuts, top-p's share is of the top-k's mass, which is known but for
// the count's crossing bin: the mass above it, and with all of it, bound the
// share, and the mass's crossing lies in the bins from the one bound's to the
// other's (mostly one bin).  The wide kernel lists the members of both and
// settles the count first.
__device__ __forceinline__ void cross_wide(RowShared& sh, const Weigher& w, double rate,
                                           const RowAsk& ask, uint64_t need_p, WideRow* wr) {
  const int t = threadIdx.x;
  auto cross = [&](auto mass, uint64_t need, int& bin, uint64_t& before) {
    __syncthreads();
    if (t == 0) sh.bin = -1;
    return cross_bins<kWideBlock, decltype(mass)::value>(sh, need, bin, before);
  };
  using Counts = std::false_type;
  using Masses = std::true_type;
  int bin_k = kBinsS, first = kBinsS, last = kBinsS;
  uint64_t before_k = 0, before = 0, mass_k = 0, need = 0;
  bool by_count = ask.cut_k && cross(Counts{}, (uint64_t)ask.k, bin_k, before_k);
  if (!by_count) bin_k = kBinsS;
  bool by_mass = ask.cut_p;
  if (by_mass) {
    uint64_t lo = need_p, hi = need_p;
    if (ask.cut_k) {
      uint64_t above = 0;
      __syncthreads();
      for (int b = t; b < kBinsS; b += kWideBlock) above += b < bin_k ? sh.mass[b] : 0ull;
      mass_k = block_sum<kWideBlock>(above, sh.red);
      lo = ceil_share(ask.p, (double)mass_k);
      hi = ceil_share(ask.p, (double)(mass_k + (by_count ? sh.mass[bin_k] : 0ull)));
    }
    uint64_t unused;
    by_mass = cross(Masses{}, lo, first, before);
    if (by_mass) {
      need = lo - before;
      if (!cross(Masses{}, hi, last, unused)) last = kBinsS - 1;
    }
  }
  const int wave = t >> 6;
  if (wave < 4) {
    // what lies above all crossing bins, top-p's, above top-k's, top-k's;
    // nothing is cut unless the bins say so
    const int end = wave == 0 ? (by_mass ? first : bin_k) - 1 : wave == 1 ? last : wave == 2 ? bin_k - 1 : bin_k;
    const bool known = wave == 0 ? by_mass || by_count : wave == 1 ? by_mass : by_count;
    float edge = wave == 0 ? -__builtin_inff() : __builtin_nanf("");
    if (known) edge = bin_begin(end, w, rate);
    if ((t & 63) == 0) wr->edge[wave] = edge;
  }
  if (t == 0) {
    wr->m = w.m;
    wr->need = need;
    wr->need_k = by_count ? (uint32_t)(ask.k - before_k) : 0u;
    wr->mass_k = mass_k;
    wr->before = before;
    wr->state = kWideMembers;
  }
}

}  // namespace

template <class T, int BLOCK>
__global__ void __launch_bounds__(BLOCK) sample_row_kernel(const SampleParams q) {
  __shared__ RowShared sh;
  const int t = threadIdx.x;
  const int row = blockIdx.x / q.row_wgs, part = blockIdx.x % q.row_wgs;
  const RowAsk ask = row_ask(q, row);
  // only rows whose cut may lie low need more than one workgroup
  const bool binned = (ask.cut_p || ask.cut_k) && !ask.greedy && !q.whole_row;
  if (part > 0 && !binned) return;
  const RowView<T> view(q, row);
  const int nseg = q.segments;
  const SegRecord* recs = q.records + (int64_t)row * nseg;
  const float ninf = -__builtin_inff();

  // The row's largest score, the candidates' common floor, and whether every
  // segment's candidates fitted.
  float m = ninf, floor = ninf, low = __builtin_inff();
  bool fits = true;
  int listed = 0;
  int first = 0x7FFFFFFF;
  for (int s = t; s < nseg; s += BLOCK) {
    const SegRecord r = recs[s];
    if (ask.greedy && (r.best > m || (r.best == m && r.first < first))) first = r.first;
    m = fmaxf(m, r.best);
    floor = fmaxf(floor, r.floor);
    low = r.best > ninf ? fminf(low, r.low) : low;
    fits = fits && r.count >= 0;
    listed += r.count;
    sh.seg_best[s] = r.best;
    sh.seg_mass[s] = r.mass;
    sh.seg_upper[s] = r.upper;
    sh.seg_count[s] = r.count;
  }
  const float own_best = m;
  block_min_max<BLOCK>(low, m, sh.redf);
  float unused = 0.0f;
  block_min_max<BLOCK>(unused, floor, sh.redf);
  fits = __syncthreads_and(fits);
  if (m == ninf) {  // nothing to draw from
    if (t == 0 && part == 0) {
      q.tokens[row] = -1;
      if (q.logprobs) q.logprobs[row] = ninf;
    }
    return;
  }
  if (ask.greedy) {
    if (t == 0) sh.found_i = 0x7FFFFFFF;
    __syncthreads();
    if (own_best == m && first != 0x7FFFFFFF) atomicMin(&sh.found_i, first);
    __syncthreads();
    if (t == 0) {
      q.tokens[row] = sh.found_i;
      if (q.logprobs) q.logprobs[row] = 0.0f;
    }
    return;
  }
  if (q.whole_row) {
    if (t == 0) q.wide[row].state = kWideWhole;
    return;
  }

  Weigher w(m, ask.c);
  const double u = clamp_uniform(q.uniforms[row]);
  double total = 0.0;  // the kept weights' sum, in units of 2^-43 of the largest

  if (!ask.cuts()) {
    // The whole vocabulary: the segment in which the running sum passes
    // u * total, then the place inside it.
    double* seg_m = reinterpret_cast<double*>(sh.mass);  // kBinsS entries >= segments
    for (int s = t; s < nseg; s += BLOCK)
      seg_m[s] = below_best(sh.seg_best[s], w) * (double)sh.seg_mass[s];
    __syncthreads();
    double own = 0.0;
    const int per = (nseg + BLOCK - 1) / BLOCK;
    for (int e = 0; e < per; ++e) {
      const int s = t * per + e;
      if (s < nseg) own += seg_m[s];
    }
    const double incl = block_scan<BLOCK>(own, sh.redd);
    if (t == 0) sh.found_i = 0x7FFFFFFF;
    if (t == BLOCK - 1) sh.redd[31] = incl;
    __syncthreads();
    total = sh.redd[31];
    const double y = u * total;
    double run = incl - own;
    // u is at most 1 - 2^-24, far further below 1 than these sums' rounding,
    // so some segment's running sum lies above y
    int mine = 0x7FFFFFFF;
    double mine_before = 0.0;
    for (int e = 0; e < per; ++e) {
      const int s = t * per + e;
      if (s < nseg) {
        if (mine == 0x7FFFFFFF && seg_m[s] > 0.0 && run + seg_m[s] > y) {
          mine = s;
          mine_before = run;
        }
        run += seg_m[s];
      }
    }
    if (mine != 0x7FFFFFFF) atomicMin(&sh.found_i, mine);
    __syncthreads();
    const int seg = sh.found_i;
    if (mine == seg) sh.redd[30] = mine_before;
    __syncthreads();
    // inside it the weights are the row's again
    const double rest = y - sh.redd[30];
    pick_in_segment<BLOCK>(view, seg, sh, w, [](float, int) { return true; },
                           rest > 0.0 ? (uint64_t)rest + 1 : 1ull);
    put_token(q, row, sh.found_i, sh.found_x, w, total);
    return;
  }

  // no drawable score lies below the floor (beside +inf nothing else is drawable)
  const bool complete = floor == ninf || m == __builtin_inff() || !w.drawable(floor);
  // at or below every drawable score
  const float least = (float)fmax((double)m - 1.0001 * kTmax / ask.c, -(double)__FLT_MAX__);
  WideRow* wr = q.wide + row;
  double rate = 0.0;
  float lowest = ninf;
  uint64_t need = 0;  // top-p's mass
  if (binned && m < __builtin_inff()) {
    // The cut's count or mass, and whether the candidates can hold it at all.
    double span = fmax(w.log2_of(low), -kTmax);
    bool low_cut;
    if (!ask.cut_k) {
      double z = 0.0, top = 0.0;
      for (int s = t; s < nseg; s += BLOCK) {
        const double unit = below_best(sh.seg_best[s], w);
        z += unit * (double)sh.seg_mass[s];
        top += unit * (double)sh.seg_upper[s];
      }
      block_sum2<BLOCK>(z, top, sh.redd);
      need = ceil_share(ask.p, z);
      low_cut = top < (double)need;
      // All scores whose weight is below (1 - p) / vocab of the total weigh
      // less than 1 - p of it together: the cut lies above them (by 0.02
      // octaves, so that no sum's rounding matters).
      const float share = (float)((1.0 - ask.p) * z * (1.0 / (double)kOne)) / (float)q.vocab;
      const double t = (double)__log2f(share) - 0.02;
      if (t > span) {
        span = fmin(t, 0.0);
        lowest = (float)((double)m + span / ask.c);
      }
    } else {
      low_cut = block_sum<BLOCK>(listed, reinterpret_cast<int*>(sh.redf)) < ask.k && !complete;
    }
    fits = fits && !low_cut;
    rate = span < 0.0 ? (double)kBinsS / -span : 0.0;
  }
  // This workgroup's share of the bins; the row's last one finds the crossing.
  auto bin_row = [&] {
    fill_bins(view, part * kWideSegs + (t >> 6), nseg, sh, w, rate, lowest, ask.cut_k, ask.cut_p);
    uint64_t* masses = q.masses + (int64_t)row * q.row_wgs * kBinsS;
    uint32_t* counts = q.counts + (int64_t)row * q.row_wgs * kBinsS;
    for (int b = t; b < kBinsS; b += BLOCK) {
      if (ask.cut_p) agent_store(&masses[part * kBinsS + b], sh.mass[b]);
      if (ask.cut_k) agent_store(&counts[part * kBinsS + b], sh.cnt[b]);
    }
    if (!last_in(&wr->arrived[0], q.row_wgs, sh)) return;
    auto add_up = [&](const auto* slices, auto* to) {
      constexpr int PER = kBinsS / BLOCK, FLY = 8 / PER;  // 8 loads in flight
      uint64_t sum[PER] = {};
      for (int p0 = 0; p0 < q.row_wgs; p0 += FLY) {
#pragma unroll
        for (int f = 0; f < FLY; ++f)
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const int p = min(p0 + f, q.row_wgs - 1);
            const uint64_t v = agent_load(&slices[p * kBinsS + e * BLOCK + t]);
            sum[e] += p0 + f < q.row_wgs ? v : 0;
          }
      }
#pragma unroll
      for (int e = 0; e < PER; ++e) to[e * BLOCK + t] = sum[e];
    };
    if (ask.cut_p) add_up(masses, sh.mass);
    if (ask.cut_k) add_up(counts, sh.cnt);
    cross_wide(sh, w, rate, ask, need, wr);
  };

  // Candidates at or above the common floor: every such score of the row.
  bool covered = fits;
  ListSource list{sh.lx, sh.li, sh.lw, 0};
  if (covered) {
    if (t == 0) sh.list_n = 0;
    __syncthreads();
    const int lane = t & 63;
    static_assert(kSegSlots == 128, "two rounds");
    constexpr int W = BLOCK / 64, FLY = 8;  // segments a wave has in flight
    // a segment's first 64 places, and the rest if one of the wave's uses them
    int more = 0;
    for (int s0 = t >> 6, from = 0; s0 < nseg;) {
      Candidate cd[FLY];
      int n[FLY];
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        const int s = min(s0 + f * W, nseg - 1);
        n[f] = s0 + f * W < nseg ? sh.seg_count[s] - from : 0;
        more = max(more, n[f]);
        cd[f] = q.candidates[((int64_t)row * nseg + s) * kSegSlots + from + lane];
      }
      uint64_t in[FLY];
      int all = 0;
#pragma unroll
      for (int f = 0; f < FLY; ++f) {
        in[f] = __ballot(lane < n[f] && cd[f].x >= floor && w.drawable(cd[f].x));
        all += __popcll(in[f]);
      }
      if (all > 0) {
        uint32_t base = 0;
        if (lane == 0) base = atomicAdd(&sh.list_n, (uint32_t)all);
        base = __builtin_amdgcn_readfirstlane(base);
#pragma unroll
        for (int f = 0; f < FLY; ++f) {
          const uint32_t at = base + __builtin_amdgcn_mbcnt_hi(
                                         (uint32_t)(in[f] >> 32),
                                         __builtin_amdgcn_mbcnt_lo((uint32_t)in[f], 0u));
          if ((in[f] >> lane & 1) && at < (uint32_t)kListS) {
            sh.lx[at] = cd[f].x;
            sh.li[at] = cd[f].i;
          }
          base += (uint32_t)__popcll(in[f]);
        }
      }
      s0 += W * FLY;
      if (s0 >= nseg && more > 64 && from == 0) {
        s0 = t >> 6;
        from = 64;
      }
    }
    __syncthreads();
    list.n = (int)sh.list_n;
    covered = list.n <= kListS;
  }
  // Whether the cut lies among them; each of the row's workgroups comes to the
  // same answer.
  Cut cut{ninf, 0x7FFFFFFF};
  const float from = complete ? least : floor;
  if (covered && ask.cut_k) covered = list.n >= ask.k || complete;
  if (covered)
    for (int i = t; i < list.n; i += BLOCK) sh.lw[i] = w(sh.lx[i]);
  __syncthreads();
  if (covered && ask.cut_p && !ask.cut_k) {
    const uint64_t have = mass_in<BLOCK>(list, sh, w, cut, 0);
    if (complete) need = ceil_share(ask.p, (double)have);
    covered = have >= need;
  }
  if (binned && !covered && m < __builtin_inff()) {
    bin_row();
    return;
  }
  if (part > 0) return;
  if (covered && !ask.cut_k && !ask.cut_p) covered = complete || w(floor) < ask.min_w;
  if (covered && list.n <= kShort) {
    draw_ranked<BLOCK>(list, sh, ask, need, u, total);
    put_token(q, row, sh.found_i, sh.found_x, w, total);
    return;
  }
  if (covered) {
    if (ask.cut_k && list.n >= ask.k)
      cut = find_cut<BLOCK, false>(list, sh, w, from, m, cut, q.vocab, (uint64_t)ask.k);
    if (ask.cut_p) {
      if (ask.cut_k) need = ceil_share(ask.p, (double)mass_in<BLOCK>(list, sh, w, cut, 0));
      cut = find_cut<BLOCK, true>(list, sh, w, from, m, cut, q.vocab, need);
    }
    draw_from_list<BLOCK>(list, sh, w, cut, ask.min_w, q.vocab, u, total);
    put_token(q, row, sh.found_i, sh.found_x, w, total);
    return;
  }

  // +inf scores that were not all handed on, or (needing no bins) min-p alone
  if (t == 0) {
    wr->edge[0] = ninf;
    wr->edge[1] = wr->edge[2] = wr->edge[3] = __builtin_nanf("");
    wr->m = m;
    wr->need = 0;
    wr->need_k = 0;
    wr->state = m == __builtin_inff() ? kWideWhole : kWideMembers;
  }
}

template <class T>
__global__ void __launch_bounds__(kWideBlock) sample_wide_kernel(const SampleParams q) {
  __shared__ RowShared sh;
  constexpr int V = Elem<T>::kVec;
  const int t = threadIdx.x;
  const int row = blockIdx.x / q.wide_wgs, part = blockIdx.x % q.wide_wgs;
  WideRow* wr = q.wide + row;
  const uint32_t state = wr->state;  // kWideWhole rows: the first workgroup alone
  if (state == kWideDone) return;
  const RowAsk ask = row_ask(q, row);
  const RowView<T> view(q, row);
  const double u = clamp_uniform(q.uniforms[row]);
  const int nseg = q.segments;
  const Cut all{-__builtin_inff(), 0x7FFFFFFF};
  Cut cut = all;
  float m = wr->m;
  Weigher w(m, ask.c);

  if (state == kWideMembers) {
    const float above = wr->edge[0], from = wr->edge[1], above_k = wr->edge[2], from_k = wr->edge[3];
    const uint32_t need_k = wr->need_k;
    uint64_t need_cut = wr->need;
    // each part's members in the places of its segments' candidates, its count
    // behind the segments' kept masses
    const int room = kWideSegs * kSegSlots;
    uint64_t* members = reinterpret_cast<uint64_t*>(q.candidates + (int64_t)row * nseg * kSegSlots);
    uint64_t* kept = q.kept + (int64_t)row * (nseg + q.wide_wgs);
    const int seg = part * kWideSegs + (t >> 6);
    const uint64_t least = ask.min_w ? ask.min_w : 1ull;
    const int mine = min(nseg - part * kWideSegs, kWideSegs) * kSegSlots;  // places for this part's
    if (t == 0) sh.list_n = 0;
    __syncthreads();
    SegRecord* recs = q.records + (int64_t)row * nseg;  // free again: the members' count and extremes
    if (seg < nseg) {
      uint64_t mass = 0;
      int own = 0;
      float lo = __builtin_inff(), hi = -__builtin_inff();
      visit_dense(
          view, seg, sh.dense[t >> 6],
          [&](float x, int i) {
            const bool kept_above = x >= above;
            const bool member = (x >= from && !kept_above) || (x >= from_k && !(x >= above_k));
            if (member && w.drawable(x)) {
              ++own;
              lo = fminf(lo, x);
              hi = fmaxf(hi, x);
              const int at = (int)atomicAdd(&sh.list_n, 1u);
              if (at < mine)
                agent_store(&members[part * room + at],
                            ((uint64_t)(uint32_t)i << 32) | __float_as_uint(x));
            }
            return kept_above;
          },
          [&](float x) {
            const uint64_t v = drawn_at(w, w.log2_of(x));
            mass += v >= least ? v : 0ull;
          });
      mass = wave_sum(mass);
      own = wave_sum(own);
      wave_minmax(lo, hi);
      if ((t & 63) == 0) {
        agent_store(&kept[seg], mass);
        agent_store(&recs[seg].count, own);
        agent_store(&recs[seg].mass,
                    ((uint64_t)__float_as_uint(hi) << 32) | (uint64_t)__float_as_uint(lo));
      }
    }
    __syncthreads();
    if (t == 0) agent_store(&kept[nseg + part], (uint64_t)sh.list_n);
    if (!last_in(&wr->arrived[1], q.wide_wgs, sh)) return;
    // the parts' counts, and their members one behind the other
    for (int p = t; p < q.wide_wgs; p += kWideBlock) sh.cnt[p] = (uint32_t)agent_load(&kept[nseg + p]);
    __syncthreads();
    int n = 0;
    bool fits = true;
    for (int p = 0; p < q.wide_wgs; ++p) {
      const int c = (int)sh.cnt[p];
      fits = fits && c <= min(nseg - p * kWideSegs, kWideSegs) * kSegSlots;
      n += c;
    }
    bool ready = fits && n <= kListS;  // each segment's kept mass, in the bins
    if (ready) {
      const ListSource list{sh.lx, sh.li, sh.lw, n};
      // the extremes of top-p's members and of top-k's
      float low = __builtin_inff(), high = -__builtin_inff(), low_k = low, high_k = high;
      int p = 0, base = 0;
      for (int i = t; i < n; i += kWideBlock) {
        while (i - base >= (int)sh.cnt[p]) base += (int)sh.cnt[p++];
        const uint64_t both = agent_load(&members[p * room + i - base]);
        const float x = __uint_as_float((uint32_t)both);
        sh.lx[i] = x;
        sh.li[i] = (int32_t)(both >> 32);
        sh.lw[i] = w(x);
        if (x >= from && !(x >= above)) {
          low = fminf(low, x);
          high = fmaxf(high, x);
        }
        if (x >= from_k && !(x >= above_k)) {
          low_k = fminf(low_k, x);
          high_k = fmaxf(high_k, x);
        }
      }
      if (need_k > 0) {
        block_min_max<kWideBlock>(low_k, high_k, sh.redf);
        cut = find_cut<kWideBlock, false>(list, sh, w, low_k, high_k, all, q.vocab, need_k);
        if (ask.cut_p) {
          uint64_t mass = 0;
          list.visit<kWideBlock>([&](float x, int i, auto&& weight) {
            if (x <= high_k && cut.holds(x, i)) mass += weight();
          });
          mass = wr->mass_k + block_sum<kWideBlock>(mass, sh.red);
          need_cut = ceil_share(ask.p, (double)mass) - wr->before;
        }
      }
      if (need_cut > 0) {
        block_min_max<kWideBlock>(low, high, sh.redf);
        cut = find_cut<kWideBlock, true>(list, sh, w, low, high, cut, q.vocab, need_cut);
      }
      clear_bins<kWideBlock>(sh);
      for (int s = t; s < nseg; s += kWideBlock) sh.mass[s] = agent_load(&kept[s]);
      __syncthreads();
      list.visit<kWideBlock>([&](float x, int i, auto&& weight) {
        const uint64_t v = weight();
        if (cut.holds(x, i) && v >= ask.min_w)
          atomicAdd((unsigned long long*)&sh.mass[(i + view.lead) / kSegment], (unsigned long long)v);
      });
    } else {
      // Too many to list, which mostly are equal scores (16-bit logits far
      // from zero, or a constant row): of one value, the first so many.
      float lo = __builtin_inff(), hi = -__builtin_inff();
      clear_bins<kWideBlock>(sh);
      for (int s = t; s < nseg; s += kWideBlock) {
        const uint64_t ends = agent_load(&recs[s].mass);
        sh.cnt[s] = (uint32_t)agent_load(&recs[s].count);
        lo = fminf(lo, __uint_as_float((uint32_t)ends));
        hi = fmaxf(hi, __uint_as_float((uint32_t)(ends >> 32)));
      }
      block_min_max<kWideBlock>(lo, hi, sh.redf);
      ready = lo == hi;
      if (ready) {
        const uint64_t one = w.drawn(lo);
        uint64_t take = (uint64_t)n, before;
        if (need_k > 0) {
          take = min(take, (uint64_t)need_k);
          if (ask.cut_p) need_cut = ceil_share(ask.p, (double)(wr->mass_k + take * one)) - wr->before;
        }
        if (need_cut > 0 && one > 0) take = min(take, (need_cut + one - 1) / one);
        int at;
        cross_bins<kWideBlock, false>(sh, take, at, before);
        take -= before;
        cut.x = lo;
        if (one > 0) {  // (else it makes no difference which of them are kept)
          pick_in_segment<kWideBlock>(
              view, at, sh, w, [&](float x, int) { return x == lo; }, take * one);
          cut.i = sh.found_i;
        }
        for (int s = t; s < nseg; s += kWideBlock) {
          const uint64_t count = s < at ? sh.cnt[s] : s == at ? take : 0ull;
          sh.mass[s] = agent_load(&kept[s]) + (one >= least ? count * one : 0ull);
        }
      }
    }
    if (ready) {
      __syncthreads();
      uint64_t z = 0;
      for (int s = t; s < nseg; s += kWideBlock) z += sh.mass[s];
      z = block_sum<kWideBlock>(z, sh.red);
      uint64_t need = (uint64_t)(u * (double)z) + 1, before;
      if (need > z) need = z;
      int at;
      cross_bins<kWideBlock, true>(sh, need, at, before);
      pick_in_segment<kWideBlock>(
          view, at, sh, w, [&](float x, int i) { return cut.holds(x, i) && w.drawn(x) >= least; },
          need - before);
      put_token(q, row, sh.found_i, sh.found_x, w, (double)z);
      return;
    }
  } else if (part != 0 || state != kWideWhole) {
    return;
  }

  // The whole row from memory, by this workgroup alone.
  const RowSource<T> src{view, w, (q.vocab + view.lead + V - 1) / V};
  float low = __builtin_inff(), high = -__builtin_inff();
  src.template visit<kWideBlock>([&](float x, int, auto&&) { high = fmaxf(high, x); });
  block_min_max<kWideBlock>(low, high, sh.redf);
  m = high;
  low = m;
  w.against(m);
  src.template visit<kWideBlock>([&](float x, int, auto&&) {
    if (w.drawable(x)) low = fminf(low, x);
  });
  block_min_max<kWideBlock>(low, high, sh.redf);
  cut = all;
  if (ask.cut_k)
    cut = find_cut<kWideBlock, false>(src, sh, w, low, high, all, q.vocab, (uint64_t)ask.k);
  if (ask.cut_p) {
    const uint64_t z = mass_in<kWideBlock>(src, sh, w, cut, 0);
    cut = find_cut<kWideBlock, true>(src, sh, w, low, high, cut, q.vocab, ceil_share(ask.p, (double)z));
  }
  double total;
  draw_from<kWideBlock>(src, sh, w, cut, ask.min_w, q.vocab, u, total);
  put_token(q, row, sh.found_i, sh.found_x, w, total);
}

const void* sample_segment_kernel_ptr(int dtype, bool cuts) {
  switch (dtype * 2 + (cuts ? 1 : 0)) {
    case 0: return reinterpret_cast<const void*>(&sample_segment_kernel<float, false>);
    case 1: return reinterpret_cast<const void*>(&sample_segment_kernel<float, true>);
    case 2: return reinterpret_cast<const void*>(&sample_segment_kernel<__hip_bfloat16, false>);
    case 3: return reinterpret_cast<const void*>(&sample_segment_kernel<__hip_bfloat16, true>);
    case 4: return reinterpret_cast<const void*>(&sample_segment_kernel<__half, false>);
    case 5: return reinterpret_cast<const void*>(&sample_segment_kernel<__half, true>);
    default: return nullptr;
  }
}

#define ERT_SAMPLE_PTR(NAME, ...)                                                      \
  const void* NAME##_ptr(int dtype) {                                                  \
    switch (dtype) {                                                                   \
      case 0: return reinterpret_cast<const void*>(&NAME<float __VA_ARGS__>);          \
      case 1: return reinterpret_cast<const void*>(&NAME<__hip_bfloat16 __VA_ARGS__>); \
      case 2: return reinterpret_cast<const void*>(&NAME<__half __VA_ARGS__>);         \
      default: return nullptr;                                                         \
    }                                                                                  \
  }
ERT_SAMPLE_PTR(sample_row_kernel, , kRowBlock)
ERT_SAMPLE_PTR(sample_wide_kernel)

}  // namespace ert
