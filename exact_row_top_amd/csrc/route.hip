// route.hip -- routing to experts: which top_k experts each token goes to, the
// weights they get, and the weights' gradient.
//
// s = sigmoid(x) or softmax(x) over the token's E logits, c = s + bias (the
// bias takes part in the choice only; without one the order of c is that of
// x, which is used as it is).  Experts may lie in equal groups, of which the
// topk_groups with the largest score (largest c, or the two largest summed)
// stay; the top_k largest c among them are chosen, in falling order.  Equal
// scores go to the lower index.  The weights are s at the chosen experts,
// divided by their sum if asked, times a scale.  Experts whose logit is -inf
// or NaN are never chosen; slots without an expert hold -1 and weight 0.
//
// The choice is a whole number that has to come out the same wherever it is
// made, so it is the choice on 64-bit scores.  It is made on 32-bit ones
// first: where every score that was taken stands clear of the next one by
// more than both can be off, the 64-bit order is the same; the experts near
// the last one of the few tokens (and ties under a bias) where it does not
// are ranked again by 64-bit scores, and so are the groups near the last one
// that stays, by the experts that can be their largest (a token's whole 64-bit
// scores instead cost 2 us of the 16384 x 256 call, whose waves all run at
// once and wait for the slowest).

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gvr_device.h"
#include "rowops.h"

namespace ert {

namespace {

constexpr int kRouteBlock = 256;
constexpr int kNear = 16;  // experts that are ranked one a lane

// Sums and least values over the L lanes that share a token.
template <int L, class V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
template <int L>
__device__ __forceinline__ int lanes_min(int v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d));
  return v;
}

// All-lane reductions of 32-bit values by rotations within rows of 16 lanes
// (no LDS), and for L = 64 over the four rows' results.
template <int N>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x120 + N, 0xf, 0xf, false);
}
template <int L, class Op>
__device__ __forceinline__ uint32_t lanes_fold(uint32_t v, Op&& op) {
  v = op(v, ror<8>(v));
  v = op(v, ror<4>(v));
  v = op(v, ror<2>(v));
  v = op(v, ror<1>(v));
  if (L == 64) {
    const uint32_t a = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
    const uint32_t b = (uint32_t)__builtin_amdgcn_readlane((int)v, 16);
    const uint32_t c = (uint32_t)__builtin_amdgcn_readlane((int)v, 32);
    const uint32_t d = (uint32_t)__builtin_amdgcn_readlane((int)v, 48);
    v = op(op(a, b), op(c, d));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t fold_max(uint32_t v) {
  return lanes_fold<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int L>
__device__ __forceinline__ float fold_maxf(float v) {
  return __uint_as_float(lanes_fold<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t fold_sum(uint32_t v) {
  return lanes_fold<L>(v, [](uint32_t a, uint32_t b) { return a + b; });
}

__device__ __forceinline__ bool live(float x) { return x > -__builtin_inff(); }

// The group of expert e < 1024.
__device__ __forceinline__ uint32_t group_of(const RouteParams& q, int e) {
  return q.group_size > 1 ? __umulhi((uint32_t)e, q.group_magic) : (uint32_t)e & 31u;
}

// Scores in 64 bits, to 2^-45 of themselves.
struct Score64 {
  Exp2Poly poly;
  float top;      // softmax: the largest of the logits that share the mass
  double inv_z;
  bool sigmoid;
  __device__ __forceinline__ double share(float x) const {
    const double v = exp2_64(((double)x - (double)top) * kLog2e, poly);  // 0 at -inf
    return x == top ? 1.0 : v;
  }
  __device__ __forceinline__ double operator()(float x) const {
    if (!sigmoid) return share(x) * inv_z;
    double e = exp2_64(-__builtin_fabs((double)x) * kLog2e, poly);
    if (e < 0x1p-1022) e = 0.0;  // (a sum of subnormals has no reciprocal)
    return (x < 0.0f ? e : 1.0) / (1.0 + e);
  }
};

__device__ __forceinline__ double ror64(double v, int n) {
  const uint32_t lo = (uint32_t)__double2loint(v), hi = (uint32_t)__double2hiint(v);
  uint32_t a, b;
  switch (n) {
    case 8: a = ror<8>(lo); b = ror<8>(hi); break;
    case 4: a = ror<4>(lo); b = ror<4>(hi); break;
    case 2: a = ror<2>(lo); b = ror<2>(hi); break;
    default: a = ror<1>(lo); b = ror<1>(hi); break;
  }
  return __hiloint2double((int)b, (int)a);
}
template <int L>
__device__ __forceinline__ double fold_max64(double v) {
  v = fmax(v, ror64(v, 8));
  v = fmax(v, ror64(v, 4));
  v = fmax(v, ror64(v, 2));
  v = fmax(v, ror64(v, 1));
  if (L == 64) {
    v = fmax(v, __shfl_xor(v, 16));
    v = fmax(v, __shfl_xor(v, 32));
  }
  return v;
}

// One token's scores in 64 bits; -inf for experts that cannot be chosen.
template <class T, int L, int EPL>
__device__ __forceinline__ void scores64(const RouteParams& q, const float (&x)[EPL],
                                         const Score64& score, int l, double (&d)[EPL]) {
  constexpr int V = Elem<T>::kVec;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = (i / V * L + l) * V + i % V;
    const double v = q.bias ? score(x[i]) + (double)q.bias[min(e, q.experts - 1)] : (double)x[i];
    d[i] = (live(x[i]) && v > -__builtin_inf()) ? v : -__builtin_inf();
  }
}

// The groups that stay, in 64 bits; `c` and `group_score` in LDS.
template <class T, int L, int EPL>
__device__ __forceinline__ uint32_t groups64(const RouteParams& q, const float (&x)[EPL],
                                             const Score64& score, int l, double* c,
                                             double* group_score) {
  constexpr int V = Elem<T>::kVec;
  const double ninf = -__builtin_inf();
  double d[EPL];
  scores64<T, L, EPL>(q, x, score, l, d);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = (i / V * L + l) * V + i % V;
    if (e < q.experts) c[e] = d[i];
  }
  wave_sync();
  if (l < q.groups) {
    double a = ninf, b = ninf;
#pragma unroll 4
    for (int n = 0; n < q.group_size; ++n) {
      const double v = c[l * q.group_size + n];
      b = fmax(b, fmin(a, v));
      a = fmax(a, v);
    }
    double v = a;
    if (q.top2 && a > ninf) {
      v = q.bias ? a : score((float)a);
      if (b > ninf) v += q.bias ? b : score((float)b);
    }
    group_score[l] = v;
  }
  wave_sync();
  bool stay = false;
  if (l < q.groups) {
    const double own = group_score[l];
    int better = 0;
    for (int h = 0; h < q.groups; ++h) {
      const double o = group_score[h];
      better += (o > own || (o == own && h < l)) ? 1 : 0;
    }
    stay = better < q.topk_groups;
  }
  wave_sync();
  return (uint32_t)(__ballot(stay) >> ((threadIdx.x & 63) / L * L)) & 0xFFFFu;
}

// The choice of one token in 64 bits by its L lanes, among the groups kept.
template <class T, int L, int EPL>
__device__ __forceinline__ void choose64(const RouteParams& q, const float (&x)[EPL],
                                         const Score64& score, int l, uint32_t keep, int32_t* chosen) {
  constexpr int V = Elem<T>::kVec;
  const double ninf = -__builtin_inf();
  double d[EPL];
  scores64<T, L, EPL>(q, x, score, l, d);
  if (q.groups > 1) {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (!((keep >> group_of(q, (i / V * L + l) * V + i % V)) & 1u)) d[i] = ninf;
  }
  for (int j = 0; j < q.top_k; ++j) {
    double best = ninf;
#pragma unroll
    for (int i = 0; i < EPL; ++i) best = fmax(best, d[i]);
    best = fold_max64<L>(best);
    int i = EPL;
#pragma unroll
    for (int o = EPL - 1; o >= 0; --o) i = d[o] == best ? o : i;
    if (!(best > ninf)) i = EPL;
    const int own = i < EPL ? (i / V * L + l) * V + i % V : 0x7FFFFFFF;
    const int at = lanes_min<L>(own);  // the lowest of equals
    if (l == 0) chosen[j] = at == 0x7FFFFFFF ? -1 : at;
    const int gone = at == own ? i : EPL;
#pragma unroll
    for (int o = 0; o < EPL; ++o) d[o] = o == gone ? ninf : d[o];
  }
}

}  // namespace

// L lanes a token, up to EPL experts a lane in 16-byte groups: group v of lane
// l holds experts (v * L + l) * V ... of the token, so a token's loads are one
// piece.  Waves work alone.
//
// The chosen scores come off in falling order as 31-bit keys: with M the last
// key taken, key - M as an unsigned number is at least 2^31 exactly for the
// keys below M and larger the nearer they are, so the next one is the largest
// difference, and nothing needs marking.  16-bit logits without a bias carry
// the expert's number in the key's low bits and are unique; other equal keys
// are found by counting, at the end, the keys at or above the last.
//
// Bound by the chain of top_k selections, each a maximum over the token's
// lanes that the next one waits for (about 0.65 us of a token's time), not by
// the 17.8 MB read: 16384 x 256 fp32, top 8, takes 11 us with softmax and 18.4
// with sigmoid, bias and 4 of 8 groups; 64 x 128 bf16 5.5.  16 lanes a token
// let four tokens share each step of a wave: with a wave a token the same
// softmax calls take 35 and 7.1 us.
//
// A group's two largest summed without a bias are sums of scores while the
// order is that of the logits, and 32 bits would need a bound for each: such
// calls settle the groups in 64 bits for every token (the 16384 x 256 call
// with 4 of 8 groups 19.9 us, 13.4 by each group's largest).
template <class T, int L, int EPL>
__global__ void __launch_bounds__(kRouteBlock) route_kernel(const RouteParams q) {
  constexpr int TOKENS = kRouteBlock / L;
  constexpr int V = Elem<T>::kVec;
  constexpr int NV = EPL / V;
  constexpr bool NARROW = V == 8;
  extern __shared__ double lds[];
  __shared__ double group_score[TOKENS][kMaxGroups];
  __shared__ int32_t chosen[TOKENS][kMaxRouteK];
  const int l = threadIdx.x % L;
  const int slot = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
  const bool on = token < q.tokens;
  const int E = q.experts, K = q.top_k;
  const float ninf = -__builtin_inff();
  const T* row = static_cast<const T*>(q.logits) + (on ? token : (int64_t)q.tokens - 1) * q.row_stride;
  int32_t* mine = chosen[slot];

  float x[EPL];
  if (q.vector) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e0 = (v * L + l) * V;
      float y[V];
      uint4 raw{0, 0, 0, 0};
      if (e0 < E) raw = *reinterpret_cast<const uint4*>(row + e0);
      Elem<T>::unpack(raw, y);
#pragma unroll
      for (int i = 0; i < V; ++i) x[v * V + i] = (e0 < E && live(y[i])) ? y[i] : ninf;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = (v * L + l) * V + i;
        const float y = e < E ? Elem<T>::load(row, e) : ninf;
        x[v * V + i] = live(y) ? y : ninf;
      }
  }

  Score64 score;
  score.sigmoid = q.sigmoid;
  score.inv_z = 1.0;
  float top = ninf;
#pragma unroll
  for (int i = 0; i < EPL; ++i) top = fmaxf(top, x[i]);
  top = fold_maxf<L>(top);
  score.top = top;
  if (!q.sigmoid && (!q.renormalize || q.bias)) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += live(x[i]) ? score.share(x[i]) : 0.0;
    z = lanes_sum<L>(z);
    score.inv_z = z > 0.0 ? 1.0 / z : 0.0;
  }

  // 32-bit scores, how far two of them may be off against each other, and
  // whether that bound does not hold
  float c[EPL];
  float eps = 0.0f;
  bool hard = false;
  if (q.bias) {
    const float log2e = 1.44269504f;
    float scale = (float)score.inv_z, best;
    if (q.sigmoid) {
      best = 1.0f / (1.0f + __builtin_amdgcn_exp2f(-top * log2e));
      // below, the exponential's own error would no longer be small beside
      // the largest score
      hard = top < -16.0f;
    } else {
      best = scale;
      hard = !(top < __builtin_inff());
    }
    // A sigmoid is off by at most (|x| + 4) 2^-24 of itself (the product with
    // log2(e), one unit each of v_exp_f32 and v_rcp_f32, two sums) while |x|
    // <= 16, and beyond by less than that of the largest; a softmax share by
    // (1.5 |x - top| + 4) 2^-24 of itself.  Two of
    // either differ by less than 2^-17 of the largest.  Adding the bias costs
    // 2^-24 of the result, the bits that the key gives up 2^-18, each of two.
    eps = best * 0x1p-17f;
    float widest = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e0 = (v * L + l) * V;
      float b[V];
      if (q.vector_bias) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const f4 y = *reinterpret_cast<const f4*>(q.bias + min(e0 + i, E - 4));
#pragma unroll
          for (int o = 0; o < 4; ++o) b[i + o] = y[o];
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = q.bias[min(e0 + i, E - 1)];
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = v * V + i;
        const float s = q.sigmoid ? __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-x[j] * log2e))
                                  : __builtin_amdgcn_exp2f((x[j] - top) * log2e) * scale;
        const float sum = s + b[i];
        const bool in = live(x[j]) && sum > ninf;
        c[j] = in ? sum : ninf;
        widest = fmaxf(widest, in ? __builtin_fabsf(sum) : 0.0f);
      }
    }
    eps += fold_maxf<L>(widest) * 0x1p-17f;
    hard = hard || !(eps < 1e30f);
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = x[i];
  }

  uint32_t keep = 0xFFFFFFFFu;  // the groups that stay
  bool unsure = hard || (!q.bias && q.top2);  // (sums of two logits are no scores)
  if (q.groups > 1 && !unsure) {
    float* cc = reinterpret_cast<float*>(lds + (int64_t)slot * E);
    float* gs = reinterpret_cast<float*>(group_score[slot]);
    const int size = q.group_size;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e0 = (v * L + l) * V;
      if (E % V == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4)
          if (e0 < E)
            *reinterpret_cast<f4*>(cc + e0 + i) =
                f4{c[v * V + i], c[v * V + i + 1], c[v * V + i + 2], c[v * V + i + 3]};
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (e0 + i < E) cc[e0 + i] = c[v * V + i];
      }
    }
    if (l >= q.groups && l < kMaxGroups) gs[l] = ninf;  // read four at a time below
    wave_sync();
    // `split` neighbouring lanes a group, each over every split-th part of it
    const int split = 1 << q.group_lanes, g = l >> q.group_lanes, part = l & (split - 1);
    float a = ninf, b = ninf;
    if (g < q.groups) {
      const float* own_c = cc + g * size;
      if (size % 4 == 0) {
        for (int n = part * 4; n < size; n += split * 4) {
          const f4 y = *reinterpret_cast<const f4*>(own_c + n);
#pragma unroll
          for (int o = 0; o < 4; ++o) {
            b = fmaxf(b, fminf(a, y[o]));
            a = fmaxf(a, y[o]);
          }
        }
      } else {
        for (int n = part; n < size; n += split) {
          const float y = own_c[n];
          b = fmaxf(b, fminf(a, y));
          a = fmaxf(a, y);
        }
      }
    }
    for (int d = 1; d < split; d <<= 1) {
      const float oa = __shfl_xor(a, d), ob = __shfl_xor(b, d);
      b = fmaxf(fmaxf(b, ob), fminf(a, oa));
      a = fmaxf(a, oa);
    }
    float* lowest_in = gs + kMaxGroups;  // below these, no expert is one of its group's largest
    if (g < q.groups && part == 0) {
      gs[g] = (q.top2 && live(b)) ? a + b : a;
      lowest_in[g] = (q.top2 ? b : a) - eps;
    }
    wave_sync();
    const float own = l < q.groups ? gs[l] : ninf;
    bool stay = false;
    if (l < q.groups) {
      int better = 0;
      for (int h = 0; h < q.groups; h += 4) {
        const f4 y = *reinterpret_cast<const f4*>(gs + h);
#pragma unroll
        for (int o = 0; o < 4; ++o)
          better += (y[o] > own || (y[o] == own && h + o < l)) ? 1 : 0;
      }
      stay = better < q.topk_groups;
    }
    const float last = -fold_maxf<L>(stay && live(own) ? -own : ninf);
    const float next = fold_maxf<L>(l < q.groups && !stay ? own : ninf);
    unsure = q.bias && live(next) && last - next <= 2.0f * eps;
    const int base = (int)(threadIdx.x & 63) / L * L;  // the token's first lane
    auto token_mask = [&](bool p) { return (uint32_t)(__ballot(p) >> base) & 0xFFFFu; };
    keep = token_mask(stay);
    wave_sync();
    if (unsure) {
      // Only groups as near to the border as two sums can be off are open, and
      // of them only the experts that can be their largest: one a lane, in 64
      // bits.  More of those than kNear: all of the token's, below.
      const bool open = live(own) && own >= last - 2.0f * eps && own <= next + 2.0f * eps;
      const uint32_t opened = token_mask(open), sure = token_mask(stay && !open);
      int32_t* near = mine;
      int n = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int e = (i / V * L + l) * V + i % V;
        const uint32_t h = group_of(q, e) & 15u;
        const bool in = live(c[i]) && ((opened >> h) & 1u) && c[i] >= lowest_in[h];
        const uint64_t bits = __ballot(in) >> base;
        const uint64_t m = L == 64 ? bits : bits & ((1ull << (L & 63)) - 1);
        const int at = n + __popcll(m & ((1ull << l) - 1));
        if (in && at < kNear) near[at] = e;
        n += __popcll(m);
      }
      wave_sync();
      if (n <= kNear) {
        unsure = false;
        const int e = l < n ? near[l] : 0;
        const double d = l < n ? score(Elem<T>::load(row, e)) + (double)q.bias[e] : 0.0;
        const int of = (int)group_of(q, e);
        double first = -__builtin_inf(), second = -__builtin_inf();
        for (int o = 0; o < n; ++o) {
          const double y = __shfl(d, base + o);
          if (__shfl(of, base + o) == l) {
            second = fmax(second, fmin(first, y));
            first = fmax(first, y);
          }
        }
        if (q.top2 && second > -__builtin_inf()) first += second;
        int better = 0;
        for (int h = 0; h < q.groups; ++h) {
          const double y = __shfl(first, base + h);
          if ((opened >> h) & 1u) better += (y > first || (y == first && h < l)) ? 1 : 0;
        }
        keep = sure | token_mask(open && better < q.topk_groups - __popc(sure));
      }
      wave_sync();
    }
  }
  if (q.groups > 1 && unsure)
    keep = groups64<T, L, EPL>(q, x, score, l, lds + (int64_t)slot * E, group_score[slot]);

  // Keys: a 16-bit logit's 19 leading bits (all a bfloat16 or float16 has) and
  // the expert's number; under a bias 27 bits and the score's place in the
  // lane; else 31 bits.
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = (i / V * L + l) * V + i % V;
    uint32_t k = fkey(c[i]) >> 1;
    if (q.bias) k = (k & ~15u) | (uint32_t)(EPL - 1 - i);
    else if (NARROW) k = (k >> 12) << 10 | (uint32_t)(1023 - e);
    key[i] = live(c[i]) ? k : 0u;
  }
  if (q.groups > 1) {
    if (q.group_size % V == 0) {  // neighbours share their group
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const bool in = (keep >> group_of(q, (v * L + l) * V)) & 1u;
#pragma unroll
        for (int i = 0; i < V; ++i) key[v * V + i] = in ? key[v * V + i] : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!((keep >> group_of(q, (i / V * L + l) * V + i % V)) & 1u)) key[i] = 0u;
    }
  }

  // one more than asked for, to see that the last one stands clear
  unsure = false;
  uint32_t last = 0x80000000u;  // above every key
  uint32_t lowest = 0x80000000u;
  int taken = 0;
  float before = 0.0f;
  for (int j = 0; j <= K; ++j) {
    uint32_t own = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) own = max(own, key[i] - last);
    const uint32_t d = fold_max<L>(own);
    const uint32_t now = last + d;
    const bool any = d >= 0x80000000u && now > 0u;
    if (q.bias) {
      const float f = from_key((now & ~15u) << 1);
      unsure = unsure || (any && j > 0 && before - f <= eps);
      before = f;
    }
    last = any ? now : 0u;
    if (j == K) break;
    if (!any) {
      if (l == 0) mine[j] = -1;
      continue;
    }
    lowest = last;
    ++taken;
    if (NARROW && !q.bias) {
      if (l == 0) mine[j] = 1023 - (int)(now & 1023u);
    } else if (own == d) {  // this lane's; two lanes with one key are found below
      int i = EPL - 1 - (int)(now & 15u);
      if (!q.bias) {
        i = 0;
#pragma unroll
        for (int o = 1; o < EPL; ++o) i = key[o] == last ? o : i;
      }
      mine[j] = (i / V * L + l) * V + i % V;
    }
  }
  if (q.bias || !NARROW) {
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) n += key[i] >= lowest ? 1u : 0u;
    unsure = unsure || fold_sum<L>(n) != (uint32_t)taken;
  }
  wave_sync();

  if (unsure || hard) {
    // Every expert whose 32-bit score is within eps of the last one taken:
    // one a lane, ranked by 64-bit scores.  More than kNear, or scores too
    // far down for eps to hold: all of them in 64 bits.
    int n = 0;
    int32_t* near = reinterpret_cast<int32_t*>(group_score[slot]);
    if (!hard) {
      const float thr = taken ? (q.bias ? from_key((lowest & ~15u) << 1) - eps : from_key(lowest << 1))
                              : __builtin_inff();
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const bool in = key[i] > 0u && (c[i] >= thr || key[i] >= lowest);
        const uint64_t all = __ballot(in) >> ((threadIdx.x & 63) / L * L);
        const uint64_t m = L == 64 ? all : all & ((1ull << (L & 63)) - 1);
        const int at = n + __popcll(m & ((1ull << l) - 1));
        if (in && at < kNear) near[at] = (i / V * L + l) * V + i % V;
        n += __popcll(m);
      }
      wave_sync();
    }
    if (hard || n > kNear) {
      choose64<T, L, EPL>(q, x, score, l, keep, mine);
    } else {
      const int e = l < n ? near[l] : 0x7FFFFFFF;
      double d = -__builtin_inf();
      if (l < n) {
        const float v = Elem<T>::load(row, e);
        d = q.bias ? score(v) + (double)q.bias[e] : (double)v;
      }
      int rank = 0;
      for (int o = 0; o < n; ++o) {
        const int from = (int)(threadIdx.x & 63) / L * L + o;
        const double y = __shfl(d, from);
        const int f = __shfl(e, from);
        rank += (y > d || (y == d && f < e)) ? 1 : 0;
      }
      if (l < n && rank < K) mine[rank] = e;
      for (int j = n + l; j < K; j += L) mine[j] = -1;
    }
  }
  wave_sync();

  // The weights, in 64 bits.  Softmax scores that are divided by their sum are
  // taken against the largest of the chosen, which a bias may have kept far
  // below the token's largest.
  constexpr int R = kMaxRouteK / L;
  int named[R];
  float logit[R];
  float best = ninf;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = r * L + l;
    named[r] = j < K ? mine[j] : -1;
    logit[r] = named[r] >= 0 ? Elem<T>::load(row, named[r]) : ninf;
    best = fmaxf(best, logit[r]);
  }
  if (!q.sigmoid && q.renormalize) {
    score.top = fold_maxf<L>(best);
    score.inv_z = 1.0;
  }
  double s[R], sum = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = 0.0;
    if (r * L >= K) continue;
    if (named[r] >= 0) s[r] = score(logit[r]);
    sum += s[r];
  }
  if (q.renormalize) {
    sum = lanes_sum<L>(sum);
    sum = sum > 0.0 ? 1.0 / sum : 0.0;
  } else {
    sum = 1.0;
  }
  if (!on) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = r * L + l;
    if (j >= K) continue;
    q.indices[token * K + j] = named[r];
    q.weights[token * K + j] = (float)(s[r] * sum * (double)q.scale);
  }
}

// ---------------------------------------------------------------------------
// The gradient of the weights in the logits.  With g the incoming gradient
// times the scale and s the chosen scores: where the weights were divided by
// their sum W, ds_j = (g_j - sum_i g_i s_i / W) / W, else ds_j = g_j; then
// dx_j = ds_j s_j (1 - s_j) for the sigmoid and dx_e = s_e (ds_e - sum_j ds_j
// s_j) for the softmax, where renormalised weights make that sum zero, so
// only the chosen experts' logits get a gradient and only theirs are read.
// ---------------------------------------------------------------------------

namespace {

template <class T>
__device__ __forceinline__ void store_as(T* p, float v);
template <>
__device__ __forceinline__ void store_as<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store_as<__hip_bfloat16>(__hip_bfloat16* p, float v) { *p = __float2bfloat16(v); }
template <>
__device__ __forceinline__ void store_as<__half>(__half* p, float v) { *p = __float2half(v); }

}  // namespace

// A token's row of changes is put together in LDS: zeros, the chosen
// experts' changes (at most K), and out in 16-byte pieces.  Bound by the
// chain of dependent steps at few tokens and by writing at many: 16384 x 256
// fp32 sigmoid, whose 18.4 MB are written and hardly read, take 8.9 us (2.1
// TB/s; a store per chosen expert over rows of zeros took 11), 4097 x 64 bf16
// with the whole softmax 6.2.
template <class T, int L, int EPL>
__global__ void __launch_bounds__(kRouteBlock) route_grad_kernel(const RouteGradParams q) {
  constexpr int TOKENS = kRouteBlock / L;
  constexpr int V = Elem<T>::kVec;
  extern __shared__ float row_lds[];
  __shared__ double change[TOKENS][kMaxRouteK];
  __shared__ int32_t names[TOKENS][kMaxRouteK];
  const int l = threadIdx.x % L;
  const int slot = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
  const bool on = token < q.tokens;
  const int E = q.experts, K = q.top_k;
  const float ninf = -__builtin_inff();
  float* d = row_lds + (int64_t)slot * (L * EPL);
  const int64_t tk = on ? token : (int64_t)q.tokens - 1;
  const T* row = static_cast<const T*>(q.logits) + tk * q.row_stride;
  const int32_t* idx = q.indices + tk * K;
  const float* grad = q.grad_weights + tk * K;

#pragma unroll
  for (int i = 0; i < EPL; i += 4) *reinterpret_cast<f4*>(d + (i / 4 * L + l) * 4) = f4{0, 0, 0, 0};

  const bool whole = !q.sigmoid && !q.renormalize;
  Score64 score;
  score.sigmoid = q.sigmoid;
  score.inv_z = 1.0;
  float top = ninf;
  float x[EPL];
  if (whole) {
#pragma unroll
    for (int v = 0; v < EPL / V; ++v) {
      const int e0 = (v * L + l) * V;
      float y[V];
      if (q.vector) {
        uint4 raw{0, 0, 0, 0};
        if (e0 < E) raw = *reinterpret_cast<const uint4*>(row + e0);
        Elem<T>::unpack(raw, y);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) y[i] = e0 + i < E ? Elem<T>::load(row, e0 + i) : ninf;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[v * V + i] = (e0 + i < E && live(y[i])) ? y[i] : ninf;
        top = fmaxf(top, x[v * V + i]);
      }
    }
  }

  // this lane's share of the chosen: expert (-1 for none), logit, gradient
  constexpr int R = kMaxRouteK / L;
  int named[R];
  float logit[R], g[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = r * L + l;
    named[r] = -1;
    logit[r] = ninf;
    g[r] = 0.0f;
    if (j < K) {
      const int e = idx[j];
      if ((unsigned)e < (unsigned)E) {
        named[r] = e;
        g[r] = grad[j];
        const float y = Elem<T>::load(row, e);
        logit[r] = live(y) ? y : ninf;
      }
      names[slot][j] = named[r];
    }
    if (!whole) top = fmaxf(top, logit[r]);
  }
  score.top = fold_maxf<L>(top);
  if (whole) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z += live(x[i]) ? score.share(x[i]) : 0.0;
    z = lanes_sum<L>(z);
    score.inv_z = z > 0.0 ? 1.0 / z : 0.0;
  }

  // sigmoids near the end of their range are raised, so that their products
  // with small gradients and their sum's reciprocal stay inside it
  const int raise = q.sigmoid && q.renormalize && score.top < -200.0f ? 500 : 0;
  double s[R], sum = 0.0, dot = 0.0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    s[r] = 0.0;
    if (r * L >= K) continue;
    if (live(logit[r])) s[r] = __builtin_ldexp(score(logit[r]), raise);
    sum += s[r];
    dot += (double)g[r] * s[r];
  }
  sum = lanes_sum<L>(sum);
  dot = lanes_sum<L>(dot);
  const double scale = (double)q.scale;
  // a token whose chosen scores sum to zero has no weights to change
  const double inv = q.renormalize ? (sum > 0.0 ? 1.0 / sum : 0.0) : 1.0;
  const double mean = q.renormalize ? dot * inv : 0.0;
  double both[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = r * L + l;
    both[r] = 0.0;
    if (j >= K) continue;
    double v = ((double)g[r] - mean) * inv * scale * s[r];
    if (q.sigmoid) v *= live(logit[r]) ? score(-logit[r]) : 0.0;
    both[r] = whole ? (double)g[r] : v;
    change[slot][j] = both[r];
  }
  wave_sync();
  // an expert that a caller names twice gets both changes, added in order by
  // the first slot that names it
  bool first[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int j = r * L + l;
    first[r] = j < K && named[r] >= 0;
    if (!first[r]) continue;
    for (int o = 0; o < K; ++o)
      if (names[slot][o] == named[r] && o != j) {  // rarely any
        first[r] = first[r] && o > j;
        both[r] += change[slot][o];
      }
  }
  wave_sync();
  // Through the whole softmax a chosen expert's gradient less `dot` may be far
  // smaller than either, so the row gets the chosen one's slot, from which the
  // difference is taken in 64 bits below.
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (!first[r]) continue;
    const int j = r * L + l;
    if (whole) change[slot][j] = both[r];
    d[named[r]] = whole ? __int_as_float(j + 1) : (float)both[r];
  }
  wave_sync();
  if (!on) return;
  T* out = static_cast<T*>(q.grad_logits) + token * q.grad_stride;
#pragma unroll
  for (int v = 0; v < EPL / V; ++v) {
    const int e0 = (v * L + l) * V;
    if (e0 >= E) continue;
    float y[V];
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f4 part = *reinterpret_cast<const f4*>(d + e0 + i);
#pragma unroll
      for (int o = 0; o < 4; ++o) y[i + o] = part[o];
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int j = __float_as_int(y[i]);
        const double own = j > 0 ? change[slot][j - 1] : 0.0;
        y[i] = live(x[v * V + i]) ? (float)(score(x[v * V + i]) * (own - dot) * scale) : 0.0f;
      }
    }
    if (q.vector) {
      T packed[V];
#pragma unroll
      for (int i = 0; i < V; ++i) store_as(packed + i, y[i]);
      *reinterpret_cast<uint4*>(out + e0) = *reinterpret_cast<const uint4*>(packed);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (e0 + i < E) store_as(out + e0 + i, y[i]);
    }
  }
}

#define ERT_ROUTE(NAME, T, L, N) \
  if (lanes == L && per_lane == N) return reinterpret_cast<const void*>(&NAME<T, L, N>)
#define ERT_ROUTE_PTR(NAME)                                              \
  const void* NAME##_ptr(int dtype, int lanes, int per_lane) {           \
    if (dtype == 0) {                                                    \
      ERT_ROUTE(NAME, float, 16, 4);                                     \
      ERT_ROUTE(NAME, float, 16, 8);                                     \
      ERT_ROUTE(NAME, float, 16, 16);                                    \
      ERT_ROUTE(NAME, float, 64, 16);                                    \
    } else if (dtype == 1) {                                             \
      ERT_ROUTE(NAME, __hip_bfloat16, 16, 8);                            \
      ERT_ROUTE(NAME, __hip_bfloat16, 16, 16);                           \
      ERT_ROUTE(NAME, __hip_bfloat16, 64, 16);                           \
    } else {                                                             \
      ERT_ROUTE(NAME, __half, 16, 8);                                    \
      ERT_ROUTE(NAME, __half, 16, 16);                                   \
      ERT_ROUTE(NAME, __half, 64, 16);                                   \
    }                                                                    \
    return nullptr;                                                      \
  }
ERT_ROUTE_PTR(route_kernel)
ERT_ROUTE_PTR(route_grad_kernel)

}  // namespace ert
