// Routing to experts (include/mok_ops.h, mok_route and mok_route_bwd): softmax or sigmoid
// scores, a bias that steers the choice only, expert groups, top-k, gates renormalised or
// not; and the gradient of the gates with respect to the logits.
//
// One warp per token. Lane l holds the logits of experts l, l + 32, ...: coalesced loads,
// every step of the choice a register loop plus a warp reduction, nothing shared between
// warps. Comparisons run on 32-bit keys with the order of the fp32 scores, so a maximum over
// the warp is one integer reduction instruction and a second one finds the lowest id that
// has it. Bound by latency for few tokens and by instruction issue for many (the T E logits
// are read once, a few microseconds' worth of HBM).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mok_internal.h"
#include "mok_ops.h"

namespace mok {
namespace {

constexpr int kWarps = 4;   // tokens per CTA
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float load(const float* p) { return *p; }
__device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }

// A logit as the rule reads it: NaN masks like -inf, +inf is the largest finite value.
__device__ __forceinline__ float clean(float l) { return l > -INFINITY ? fminf(l, FLT_MAX) : -INFINITY; }

// Unsigned key in the order of v (equal for -0 and +0; -inf lowest, above 0 = "no candidate").
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {   // no NaN among the values
  return key_value(__reduce_max_sync(kAll, order_key(v)));
}

struct Rule {
  int T, E, k, groups, per, top_groups;
  bool sigmoid, top2, renorm;
  float scale;
};

// 1 - sigmoid(l) is sigmoid(-l): no cancellation near 1
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

template <int NV, typename LT>
__global__ void __launch_bounds__(32 * kWarps)
    route_kernel(const Rule q, const LT* __restrict__ logits, const float* __restrict__ bias,
                 int32_t* __restrict__ topk_idx, float* __restrict__ gates) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= q.T) return;
  const LT* row = logits + (size_t)t * q.E;

  // scores; key = 0: no candidate (past E, in a dropped group, or taken)
  float s[NV];
  uint32_t key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    s[i] = e < q.E ? clean(load(row + e)) : -INFINITY;
  }
  float m = 0.f, z = 1.f;   // softmax statistics
  const bool on_logits = !q.sigmoid && bias == nullptr;
#pragma unroll
  for (int i = 0; i < NV; ++i) key[i] = order_key(s[i]);
  if (!q.sigmoid) {
    m = s[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, s[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;   // every expert masked: all scores 0
    z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = expf(s[i] - m);
      z += s[i];
    }
    z = warp_sum(z);
    const float d = z > 0.f ? z : 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = s[i] / d;
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = sigmoid(s[i]);
  }
  // choice scores: s becomes s + bias, -inf for masked experts
  const uint32_t masked = order_key(-INFINITY);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (key[i] == masked) {
      s[i] = -INFINITY;
    } else if (bias != nullptr) {
      const float c = s[i] + bias[e];
      s[i] = c > -INFINITY ? c : -INFINITY;   // a NaN bias masks too
    }
    if (!on_logits) key[i] = order_key(s[i]);
    if (e >= q.E) key[i] = 0;
  }

  if (q.top_groups < q.groups) {
    // score of group g in lane g
    float gs = -INFINITY;
    for (int g = 0; g < q.groups; ++g) {
      const int e0 = g * q.per, e1 = e0 + q.per;
      float v;
      if (!q.top2) {
        uint32_t b = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane + 32 * i;
          if (e >= e0 && e < e1) b = max(b, key[i]);
        }
        v = key_value(__reduce_max_sync(kAll, b));
      } else {
        // the two largest choice scores of this lane, then of the warp
        uint32_t b1 = 0, b2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = lane + 32 * i;
          if (e >= e0 && e < e1) {
            const uint32_t x = order_key(s[i]);
            b2 = max(b2, min(b1, x));
            b1 = max(b1, x);
          }
        }
        const uint32_t w1 = __reduce_max_sync(kAll, b1);
        const unsigned have = __ballot_sync(kAll, b1 == w1);
        const uint32_t w2 = __reduce_max_sync(kAll, lane == __ffs(have) - 1 ? b2 : b1);
        v = key_value(w1);
        if (w2 > masked) v += key_value(w2);   // masked experts add nothing
      }
      if (lane == g) gs = v;
    }
    uint32_t gkey = lane < q.groups ? order_key(gs) : 0;
    uint32_t live = 0;
    for (int j = 0; j < q.top_groups; ++j) {
      const uint32_t w = __reduce_max_sync(kAll, gkey);
      const int g = __ffs(__ballot_sync(kAll, gkey == w)) - 1;
      live |= 1u << g;
      if (lane == g) gkey = 0;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      if (e < q.E && !((live >> (e / q.per)) & 1u)) key[i] = 0;
    }
  }

  // the k largest; lane j keeps the j-th id
  int mine = 0;
  for (int j = 0; j < q.k; ++j) {
    uint32_t b = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) b = max(b, key[i]);
    const uint32_t w = __reduce_max_sync(kAll, b);
    int e = 0x7fffffff;
#pragma unroll
    for (int i = NV - 1; i >= 0; --i)
      if (key[i] == w) e = lane + 32 * i;
    e = __reduce_min_sync(kAll, e);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 32 * i) key[i] = 0;
    if (lane == j) mine = e;
  }

  // gates from the scores without the bias, one lane per slot
  const bool on = lane < q.k;
  const float l = on ? clean(load(row + mine)) : -INFINITY;
  float w;
  if (q.sigmoid) {
    w = on ? sigmoid(l) : 0.f;
  } else if (q.renorm) {   // relative to the largest chosen logit: no underflow of the sum
    const float mc = warp_max(l);
    w = l > -INFINITY ? expf(l - mc) : 0.f;
  } else {
    w = l > -INFINITY ? expf(l - m) / z : 0.f;
  }
  if (q.renorm) {
    const float sum = warp_sum(w);
    w = sum > 0.f ? w / sum : 0.f;
  }
  if (on) {
    topk_idx[(size_t)t * q.k + lane] = mine;
    gates[(size_t)t * q.k + lane] = q.scale * w;
  }
}

// dlogits of one token per warp, at the fixed choice S:
//   softmax, renormalised   scale w_j (dg_j - sum_S w dg),               w = s / sum_S s
//   sigmoid, renormalised   scale w_j (1 - s_j) (dg_j - sum_S w dg)
//   sigmoid                 scale s_j (1 - s_j) dg_j
//   softmax                 scale s_e ([e in S] dg_e - sum_S s dg)       for every expert e
// Slot j's value d_j lives in lane j; the row is written once, zeros included.
template <int NV, typename LT, typename DT>
__global__ void __launch_bounds__(32 * kWarps)
    route_bwd_kernel(const Rule q, const LT* __restrict__ logits,
                     const int32_t* __restrict__ topk_idx, const float* __restrict__ dgates,
                     DT* __restrict__ dlogits) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= q.T) return;
  const LT* row = logits + (size_t)t * q.E;
  DT* out = dlogits + (size_t)t * q.E;

  int id = lane < q.k ? topk_idx[(size_t)t * q.k + lane] : -1;
  if (id < 0 || id >= q.E) id = -1;
  const float dg = id >= 0 ? q.scale * dgates[(size_t)t * q.k + lane] : 0.f;
  const float l = id >= 0 ? clean(load(row + id)) : -INFINITY;

  const bool dense = !q.sigmoid && !q.renorm;
  float d;              // lane j: the gradient of slot j's expert (dense: its own part)
  float p[NV];          // dense: s_e
  float dot = 0.f;
  if (dense) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 32 * i;
      p[i] = e < q.E ? clean(load(row + e)) : -INFINITY;
    }
    float m = p[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, p[i]);
    m = warp_max(m);
    if (m == -INFINITY) m = 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] = expf(p[i] - m);
      z += p[i];
    }
    z = warp_sum(z);
    if (!(z > 0.f)) z = 1.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = p[i] / z;
    const float s = l > -INFINITY ? expf(l - m) / z : 0.f;
    dot = warp_sum(s > 0.f ? s * dg : 0.f);   // a gate of 0 takes no part, whatever its dg
    d = s > 0.f ? s * (dg - dot) : 0.f;
  } else {
    float w, part = 1.f;
    if (q.sigmoid) {
      w = id >= 0 ? sigmoid(l) : 0.f;
      part = sigmoid(-l);
    } else {
      const float mc = warp_max(l);
      w = l > -INFINITY ? expf(l - mc) : 0.f;
    }
    if (q.renorm) {
      const float sum = warp_sum(w);
      w = sum > 0.f ? w / sum : 0.f;
      d = w * (dg - warp_sum(w > 0.f ? w * dg : 0.f));
    } else {
      d = w * dg;
    }
    d = w > 0.f ? d * part : 0.f;
  }

#pragma unroll
  for (int i = 0; i < NV; ++i) p[i] = dense ? -p[i] * dot : 0.f;
  for (int j = 0; j < q.k; ++j) {
    const int e = __shfl_sync(kAll, id, j);
    const float v = __shfl_sync(kAll, d, j);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e == lane + 32 * i) p[i] = v;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = lane + 32 * i;
    if (e < q.E) store(out + e, p[i]);
  }
}

template <typename LT, int NV>
void launch_fwd(const Rule& q, const void* logits, const float* bias, int32_t* idx, float* gates,
                cudaStream_t s) {
  const unsigned blocks = (unsigned)((q.T + kWarps - 1) / kWarps);
  route_kernel<NV, LT><<<blocks, 32 * kWarps, 0, s>>>(q, static_cast<const LT*>(logits), bias, idx,
                                                      gates);
}
template <typename LT, typename DT, int NV>
void launch_bwd(const Rule& q, const void* logits, const int32_t* idx, const float* dg, void* dl,
                cudaStream_t s) {
  const unsigned blocks = (unsigned)((q.T + kWarps - 1) / kWarps);
  route_bwd_kernel<NV, LT, DT><<<blocks, 32 * kWarps, 0, s>>>(
      q, static_cast<const LT*>(logits), idx, dg, static_cast<DT*>(dl));
}

// Registers per lane: the smallest of the built sizes that holds E / 32 logits.
template <class F>
void by_width(int E, F f) {
  const int nv = (E + 31) / 32;
  if (nv <= 1) f(std::integral_constant<int, 1>{});
  else if (nv <= 2) f(std::integral_constant<int, 2>{});
  else if (nv <= 4) f(std::integral_constant<int, 4>{});
  else if (nv <= 8) f(std::integral_constant<int, 8>{});
  else if (nv <= 12) f(std::integral_constant<int, 12>{});
  else f(std::integral_constant<int, 16>{});
}

bool is_type(mok_out_dtype t) { return t == MOK_OUT_BF16 || t == MOK_OUT_F32; }
bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool make_rule(const mok_routing* r, int T, Rule* q) {
  if (!r || T < 0) return false;
  if (r->E < 1 || r->E > 512 || r->k < 1 || r->k > 32) return false;
  if (r->score != MOK_SCORE_SOFTMAX && r->score != MOK_SCORE_SIGMOID) return false;
  if (r->group_score != MOK_GROUP_MAX && r->group_score != MOK_GROUP_TOP2) return false;
  if (r->groups < 1 || r->groups > 32 || r->E % r->groups) return false;
  if (r->top_groups < 1 || r->top_groups > r->groups) return false;
  if (r->k > r->top_groups * (r->E / r->groups)) return false;
  if (!std::isfinite(r->scale)) return false;
  *q = Rule{T, r->E, r->k, r->groups, r->E / r->groups, r->top_groups,
            r->score == MOK_SCORE_SIGMOID, r->group_score == MOK_GROUP_TOP2, r->renormalize != 0,
            r->scale};
  return true;
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_route(const mok_routing* rule, int T, const void* logits,
                                mok_out_dtype logits_type, const float* bias, int32_t* topk_idx,
                                float* gates, void* stream) {
  using namespace mok;
  Rule q;
  if (!make_rule(rule, T, &q) || !is_type(logits_type)) return MOK_ERR_INVALID_ARG;
  if (T == 0) return MOK_OK;
  if (!logits || !topk_idx || !gates) return MOK_ERR_INVALID_ARG;
  if (!aligned_to(logits, logits_type == MOK_OUT_BF16 ? 2 : 4) || !aligned_to(bias, 4) ||
      !aligned_to(topk_idx, 4) || !aligned_to(gates, 4))
    return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_width(q.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (logits_type == MOK_OUT_BF16)
      launch_fwd<__nv_bfloat16, NV>(q, logits, bias, topk_idx, gates, s);
    else
      launch_fwd<float, NV>(q, logits, bias, topk_idx, gates, s);
  });
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_route_bwd(const mok_routing* rule, int T, const void* logits,
                                    mok_out_dtype logits_type, const int32_t* topk_idx,
                                    const float* dgates, void* dlogits,
                                    mok_out_dtype dlogits_type, void* stream) {
  using namespace mok;
  Rule q;
  if (!make_rule(rule, T, &q) || !is_type(logits_type) || !is_type(dlogits_type))
    return MOK_ERR_INVALID_ARG;
  if (T == 0) return MOK_OK;
  if (!logits || !topk_idx || !dgates || !dlogits) return MOK_ERR_INVALID_ARG;
  if (!aligned_to(logits, logits_type == MOK_OUT_BF16 ? 2 : 4) || !aligned_to(topk_idx, 4) ||
      !aligned_to(dgates, 4) || !aligned_to(dlogits, dlogits_type == MOK_OUT_BF16 ? 2 : 4))
    return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_width(q.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    if (logits_type == MOK_OUT_BF16 && dlogits_type == MOK_OUT_BF16)
      launch_bwd<__nv_bfloat16, __nv_bfloat16, NV>(q, logits, topk_idx, dgates, dlogits, s);
    else if (logits_type == MOK_OUT_BF16)
      launch_bwd<__nv_bfloat16, float, NV>(q, logits, topk_idx, dgates, dlogits, s);
    else if (dlogits_type == MOK_OUT_BF16)
      launch_bwd<float, __nv_bfloat16, NV>(q, logits, topk_idx, dgates, dlogits, s);
    else
      launch_bwd<float, float, NV>(q, logits, topk_idx, dgates, dlogits, s);
  });
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
