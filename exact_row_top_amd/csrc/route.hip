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
// The choice is a whole number that has to be the same wherever it is made,
// so it is made on 64-bit scores.

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "rowops.h"

namespace ert {

namespace {

constexpr int kRouteBlock = 256;

// Sums and maxima over the L lanes that share a token.
template <int L, class V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
template <int L, class V>
__device__ __forceinline__ V lanes_max(V v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) {
    const V o = __shfl_xor(v, d);
    v = o > v ? o : v;
  }
  return v;
}
template <int L>
__device__ __forceinline__ int lanes_min(int v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = min(v, __shfl_xor(v, d));
  return v;
}

__device__ __forceinline__ bool live(float x) { return x > -__builtin_inff(); }

__device__ __forceinline__ double sigmoid64(double x) {
  const double e = exp(-__builtin_fabs(x));
  return (x < 0.0 ? e : 1.0) / (1.0 + e);
}

}  // namespace

template <class T, int L>
__global__ void __launch_bounds__(kRouteBlock) route_kernel(const RouteParams q) {
  constexpr int TOKENS = kRouteBlock / L;
  extern __shared__ double lds[];
  __shared__ double group_score[TOKENS][kMaxGroups];
  __shared__ int32_t chosen[TOKENS][kMaxRouteK];
  const int l = threadIdx.x % L;
  const int slot = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
  const bool on = token < q.tokens;
  const int E = q.experts;
  const double ninf = -__builtin_inf();
  double* c = lds + (int64_t)slot * E;
  const T* row = static_cast<const T*>(q.logits) + (on ? token : 0) * q.row_stride;

  // scores of the choice
  float top = -__builtin_inff();
  for (int e = l; e < E; e += L) {
    const float x = Elem<T>::load(row, e);
    if (live(x)) top = fmaxf(top, x);
  }
  top = lanes_max<L>(top);
  auto share = [&](float x) { return x == top ? 1.0 : exp((double)x - (double)top); };
  double z = 1.0;
  const bool whole = !q.sigmoid && (q.bias || !q.renormalize);
  if (whole) {
    z = 0.0;
    for (int e = l; e < E; e += L) {
      const float x = Elem<T>::load(row, e);
      if (live(x)) z += share(x);
    }
    z = lanes_sum<L>(z);
  }
  // without a bias the order is that of the logits
  auto score = [&](float x) { return q.sigmoid ? sigmoid64((double)x) : share(x) / z; };
  for (int e = l; e < E; e += L) {
    const float x = Elem<T>::load(row, e);
    double v = ninf;
    if (live(x)) v = q.bias ? score(x) + (double)q.bias[e] : (double)x;
    c[e] = v;
  }
  __syncthreads();

  if (q.groups > 1) {
    const int size = E / q.groups;
    for (int g = l; g < q.groups; g += L) {
      double a = ninf, b = ninf;
      for (int i = 0; i < size; ++i) {
        const double v = c[g * size + i];
        if (v > a) {
          b = a;
          a = v;
        } else if (v > b) {
          b = v;
        }
      }
      double v = a;
      if (q.top2 && a > ninf) {
        v = q.bias ? a : score((float)a);
        if (b > ninf) v += q.bias ? b : score((float)b);
      }
      group_score[slot][g] = v;
    }
    __syncthreads();
    for (int g = l; g < q.groups; g += L) {
      const double own = group_score[slot][g];
      int better = 0;
      for (int h = 0; h < q.groups; ++h) {
        const double o = group_score[slot][h];
        better += (o > own || (o == own && h < g)) ? 1 : 0;
      }
      if (better >= q.topk_groups)
        for (int i = 0; i < size; ++i) c[g * size + i] = ninf;
    }
    __syncthreads();
  }

  for (int j = 0; j < q.top_k; ++j) {
    double best = ninf;
    int at = 0x7FFFFFFF;
    for (int e = l; e < E; e += L)
      if (c[e] > best) {
        best = c[e];
        at = e;
      }
    const double all = lanes_max<L>(best);
    at = lanes_min<L>(best == all && all > ninf ? at : 0x7FFFFFFF);
    if (l == 0) {
      chosen[slot][j] = at == 0x7FFFFFFF ? -1 : at;
      if (at != 0x7FFFFFFF) c[at] = ninf;
    }
    __syncthreads();
  }

  // weights of the chosen
  double sum = 0.0;
  for (int j = l; j < q.top_k; j += L) {
    const int e = chosen[slot][j];
    if (e >= 0) {
      const float x = Elem<T>::load(row, e);
      sum += q.sigmoid ? sigmoid64((double)x) : share(x);
    }
  }
  sum = lanes_sum<L>(sum);
  const double over = q.renormalize ? sum : (q.sigmoid ? 1.0 : z);
  if (on)
    for (int j = l; j < q.top_k; j += L) {
      const int e = chosen[slot][j];
      double w = 0.0;
      if (e >= 0 && over > 0.0) {
        const float x = Elem<T>::load(row, e);
        w = (q.sigmoid ? sigmoid64((double)x) : share(x)) / over * (double)q.scale;
      }
      q.indices[token * q.top_k + j] = e;
      q.weights[token * q.top_k + j] = (float)w;
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

template <class T, int L>
__global__ void __launch_bounds__(kRouteBlock) route_grad_kernel(const RouteGradParams q) {
  constexpr int TOKENS = kRouteBlock / L;
  extern __shared__ float row_lds[];
  __shared__ float change[TOKENS][kMaxRouteK];
  const int l = threadIdx.x % L;
  const int slot = threadIdx.x / L;
  const int64_t token = (int64_t)blockIdx.x * TOKENS + slot;
  const bool on = token < q.tokens;
  const int E = q.experts, K = q.top_k;
  float* d = row_lds + (int64_t)slot * E;
  const int64_t tk = on ? token : 0;
  const T* row = static_cast<const T*>(q.logits) + tk * q.row_stride;
  const int32_t* idx = q.indices + tk * K;
  const float* grad = q.grad_weights + tk * K;

  for (int e = l; e < E; e += L) d[e] = 0.0f;
  __syncthreads();

  const bool whole = !q.sigmoid && !q.renormalize;
  float top = -__builtin_inff();
  double z = 1.0;
  if (whole) {
    for (int e = l; e < E; e += L) {
      const float x = Elem<T>::load(row, e);
      if (live(x)) top = fmaxf(top, x);
    }
  } else if (!q.sigmoid) {
    for (int j = l; j < K; j += L) {
      const int e = idx[j];
      if ((unsigned)e < (unsigned)E) {
        const float x = Elem<T>::load(row, e);
        if (live(x)) top = fmaxf(top, x);
      }
    }
  }
  top = lanes_max<L>(top);
  auto share = [&](float x) { return x == top ? 1.0 : exp((double)x - (double)top); };
  if (whole) {
    z = 0.0;
    for (int e = l; e < E; e += L) {
      const float x = Elem<T>::load(row, e);
      if (live(x)) z += share(x);
    }
    z = lanes_sum<L>(z);
  }
  auto score = [&](float x) { return !live(x) ? 0.0 : q.sigmoid ? sigmoid64((double)x) : share(x) / z; };

  double sum = 0.0, dot = 0.0;
  for (int j = l; j < K; j += L) {
    const int e = idx[j];
    if ((unsigned)e < (unsigned)E) {
      const double s = score(Elem<T>::load(row, e));
      sum += s;
      dot += (double)grad[j] * s;
    }
  }
  sum = lanes_sum<L>(sum);
  dot = lanes_sum<L>(dot);
  const double scale = (double)q.scale;
  // a token whose chosen scores sum to zero has no weights to change
  const double inv = q.renormalize ? (sum > 0.0 ? 1.0 / sum : 0.0) : 1.0;
  const double mean = q.renormalize ? dot * inv : 0.0;
  for (int j = l; j < K; j += L) {
    const int e = idx[j];
    change[slot][j] = 0.0f;
    if ((unsigned)e < (unsigned)E) {
      const float x = Elem<T>::load(row, e);
      const double s = score(x);
      double v = ((double)grad[j] - mean) * inv * scale * s;
      if (q.sigmoid) v *= live(x) ? sigmoid64(-(double)x) : 0.0;
      change[slot][j] = (float)v;
    }
  }
  __syncthreads();
  // an expert that a caller names twice gets both changes, added in order by
  // the first slot that names it
  for (int j = l; j < K; j += L) {
    const int e = idx[j];
    if ((unsigned)e >= (unsigned)E) continue;
    float v = 0.0f;
    bool first = true;
    for (int o = 0; o < K; ++o) {
      if (idx[o] != e) continue;
      first = first && o >= j;
      v += change[slot][o];
    }
    if (first) d[e] = v;
  }
  __syncthreads();
  if (on) {
    T* out = static_cast<T*>(q.grad_logits) + token * q.grad_stride;
    for (int e = l; e < E; e += L) {
      float v = d[e];
      if (whole) v -= (float)(score(Elem<T>::load(row, e)) * dot * scale);
      store_as(out + e, v);
    }
  }
}

#define ERT_ROUTE_PTR(NAME)                                                              \
  const void* NAME##_ptr(int dtype, int lanes) {                                         \
    switch (dtype * 2 + (lanes == 64 ? 1 : 0)) {                                         \
      case 0: return reinterpret_cast<const void*>(&NAME<float, 16>);                    \
      case 1: return reinterpret_cast<const void*>(&NAME<float, 64>);                    \
      case 2: return reinterpret_cast<const void*>(&NAME<__hip_bfloat16, 16>);           \
      case 3: return reinterpret_cast<const void*>(&NAME<__hip_bfloat16, 64>);           \
      case 4: return reinterpret_cast<const void*>(&NAME<__half, 16>);                   \
      case 5: return reinterpret_cast<const void*>(&NAME<__half, 64>);                   \
      default: return nullptr;                                                           \
    }                                                                                    \
  }
ERT_ROUTE_PTR(route_kernel)
ERT_ROUTE_PTR(route_grad_kernel)

}  // namespace ert
