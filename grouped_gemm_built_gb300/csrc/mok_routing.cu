// Routing to experts (include/mok_ops.h, mok_route and mok_route_bwd): softmax or sigmoid
// scores, a bias that steers the choice only, expert groups, top-k, gates renormalised or
// not; and the gradient of the gates with respect to the logits.
//
// One warp per token; lane l holds the NV consecutive logits l NV .. l NV + NV - 1 (16-byte
// loads), so lower lanes hold lower ids and the lowest id among equal scores is the lowest
// lane of a ballot. Scores are compared through 32-bit keys in the order of the fp32 values:
// the maximum over the warp is one integer reduction instruction per chosen expert. A group
// of experts is a run of lanes, its score a lane-local pass and a few shuffles. Bound by
// latency for few tokens (one token over 384 experts 3.4 us, the launch included) and by
// instruction issue for many: 16384 tokens over 256 experts in 8 groups with a bias 16.4 us, about
// 840 instructions a token, where reading the logits once would take 2.6 (15.0 and 770 with the fast
// exponential, see the choice scores). 8192 tokens over 384 experts and their dense gradient 13.0
// us; the gradient's launch mostly waits for its loads.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

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
__device__ __forceinline__ float clean(float l) { return fminf(fmaxf(l, -INFINITY), FLT_MAX); }

// Unsigned key in the order of v (equal for -0 and +0; -inf lowest, above 0 = "no candidate").
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
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
  bool vec;          // rows of logits (and gradients) allow vector accesses
  bool vec_bias;
  int lanes_shift;   // log2 of the lanes per group, -1: groups do not fall on such runs
  float scale;
};

// 1 - sigmoid(l) is sigmoid(-l): no cancellation near 1
__device__ __forceinline__ float sigmoid(float l) { return 1.f / (1.f + expf(-l)); }

// The NV consecutive elements from e0 of a row of E; `fill` past its end. vec: e0 NV-aligned,
// E a multiple of NV, addresses aligned for the widest access that divides NV elements.
template <int NV, typename T>
__device__ __forceinline__ void load_row(const T* row, int e0, int E, bool vec, float fill,
                                         float* v) {
  constexpr int bytes = NV * (int)sizeof(T);
  if constexpr (bytes % 4 == 0) {
    if (vec) {
      if (e0 < E) {
        uint32_t w[bytes / 4];
        if constexpr (bytes % 16 == 0) {
#pragma unroll
          for (int i = 0; i < bytes / 16; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(row + e0)[i];
            w[4 * i] = q.x; w[4 * i + 1] = q.y; w[4 * i + 2] = q.z; w[4 * i + 3] = q.w;
          }
        } else if constexpr (bytes % 8 == 0) {
#pragma unroll
          for (int i = 0; i < bytes / 8; ++i) {
            const uint2 q = reinterpret_cast<const uint2*>(row + e0)[i];
            w[2 * i] = q.x; w[2 * i + 1] = q.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < bytes / 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(row + e0)[i];
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
          else v[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = fill;
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = e0 + i < E ? load(row + e0 + i) : fill;
}
template <int NV, typename T>
__device__ __forceinline__ void store_row(T* row, int e0, int E, bool vec, const float* v) {
  constexpr int bytes = NV * (int)sizeof(T);
  if constexpr (bytes % 4 == 0) {
    if (vec) {
      if (e0 >= E) return;
      uint32_t w[bytes / 4];
#pragma unroll
      for (int i = 0; i < bytes / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          w[i] = __float_as_uint(v[i]);
        } else {
          const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
      }
      if constexpr (bytes % 16 == 0) {
#pragma unroll
        for (int i = 0; i < bytes / 16; ++i)
          reinterpret_cast<uint4*>(row + e0)[i] =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
      } else if constexpr (bytes % 8 == 0) {
#pragma unroll
        for (int i = 0; i < bytes / 8; ++i)
          reinterpret_cast<uint2*>(row + e0)[i] = make_uint2(w[2 * i], w[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < bytes / 4; ++i) reinterpret_cast<uint32_t*>(row + e0)[i] = w[i];
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if (e0 + i < E) store(row + e0 + i, v[i]);
}

// Softmax over the warp's logits s (cleaned): s becomes the scores, m and 1 / z its
// statistics. A fully masked row has scores 0. expf, not __expf, whose error grows with the
// argument (to 1e-5 of the smallest scores, all of which the dense gradient writes).
template <int NV>
__device__ __forceinline__ void warp_softmax(float* s, float& m, float& inv_z) {
  m = s[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, s[i]);
  m = warp_max(m);
  if (m == -INFINITY) m = 0.f;
  float z = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    s[i] = expf(s[i] - m);
    z += s[i];
  }
  z = warp_sum(z);
  inv_z = z > 0.f ? 1.f / z : 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] *= inv_z;
}

// Renormalised gates from the chosen logits, one per lane (-inf: none): each score over the sum of
// all. Softmax scores are taken relative to the largest chosen one, so that their sum cannot
// underflow; so are sigmoid scores where the largest chosen logit is below -17 (there 1 + e^l is 1
// in fp32 and sigmoid(l) is e^l, which is 0 below -104).
__device__ __forceinline__ float renormalized(bool is_sigmoid, float l) {
  const float mc = warp_max(l);
  float w;
  if (is_sigmoid && mc > -17.f) w = sigmoid(l);
  else w = l > -INFINITY ? expf(l - mc) : 0.f;
  const float sum = warp_sum(w);
  return sum > 0.f ? w / sum : 0.f;
}

template <int NV, typename LT>
__global__ void __launch_bounds__(32 * kWarps)
    route_kernel(const Rule q, const LT* __restrict__ logits, const float* __restrict__ bias,
                 int32_t* __restrict__ topk_idx, float* __restrict__ gates) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= q.T) return;
  const LT* row = logits + (size_t)t * q.E;
  const int e0 = lane * NV;
  const uint32_t masked = order_key(-INFINITY);
  __shared__ uint2 s_list[kWarps][32];

  // scores; key = 0: no candidate (past E, in a dropped group, or taken)
  float s[NV];
  uint32_t key[NV];
  load_row<NV>(row, e0, q.E, q.vec, -INFINITY, s);
#pragma unroll
  for (int i = 0; i < NV; ++i) s[i] = clean(s[i]);
  float m = 0.f, inv_z = 0.f;
  // without a bias the logits have the scores' order, and keep it where scores round to one value
  const bool on_logits = bias == nullptr;
  const bool group_sums = q.top_groups < q.groups && q.top2;
  if (on_logits) {
#pragma unroll
    for (int i = 0; i < NV; ++i) key[i] = order_key(s[i]);
  }
  if (!on_logits || group_sums || (!q.sigmoid && !q.renorm)) {
    unsigned off = 0;   // masked experts of this lane
#pragma unroll
    for (int i = 0; i < NV; ++i) off |= s[i] == -INFINITY ? 1u << i : 0u;
    if (q.sigmoid) {
      // The choice needs the scores to a few ulp (the gates below are full precision): 4, of which
      // the quotient takes 2 (IEEE division: 0.5). __expf's documented error grows with the
      // argument instead, 13 ulp at a logit of -10.
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = __fdividef(1.f, 1.f + expf(-s[i]));
    } else {
      warp_softmax<NV>(s, m, inv_z);
    }
    // choice scores: s becomes s + bias, -inf for masked experts
    if (bias != nullptr) {
      float c[NV];
      load_row<NV>(bias, e0, q.E, q.vec_bias, 0.f, c);
#pragma unroll
      for (int i = 0; i < NV; ++i) s[i] = fmaxf(s[i] + c[i], -INFINITY);   // a NaN bias masks the choice too
    }
    if (off) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (off >> i & 1u) s[i] = -INFINITY;
    }
    if (!on_logits) {
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = order_key(s[i]);
    }
  }
  if (e0 + NV > q.E) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (e0 + i >= q.E) key[i] = 0;
  }

  if (q.top_groups < q.groups) {
    uint32_t gkey;      // of the group of this lane (lanes_shift >= 0), else of group `lane`
    if (q.lanes_shift >= 0) {
      uint32_t b1 = 0, b2 = 0;   // the group's two largest choice scores
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const uint32_t x = on_logits && q.top2 && key[i] ? order_key(s[i]) : key[i];
        b2 = max(b2, min(b1, x));
        b1 = max(b1, x);
      }
      for (int sh = 0; sh < q.lanes_shift; ++sh) {
        const uint32_t o1 = __shfl_xor_sync(kAll, b1, 1 << sh);
        const uint32_t o2 = __shfl_xor_sync(kAll, b2, 1 << sh);
        b2 = max(max(b2, o2), min(b1, o1));
        b1 = max(b1, o1);
      }
      // masked experts add nothing to a sum
      gkey = q.top2 && b2 > masked ? order_key(key_value(b1) + key_value(b2)) : b1;
    } else {
      gkey = 0;
      for (int g = 0; g < q.groups; ++g) {
        const int g0 = g * q.per, g1 = g0 + q.per;
        uint32_t b1 = 0, b2 = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = e0 + i;
          const uint32_t x = e < g0 || e >= g1 ? 0u : on_logits && q.top2 ? order_key(s[i]) : key[i];
          b2 = max(b2, min(b1, x));
          b1 = max(b1, x);
        }
        uint32_t w = __reduce_max_sync(kAll, b1);
        if (q.top2) {
          const unsigned have = __ballot_sync(kAll, b1 == w);
          const uint32_t w2 = __reduce_max_sync(kAll, lane == __ffs(have) - 1 ? b2 : b1);
          if (w2 > masked) w = order_key(key_value(w) + key_value(w2));
        }
        if (lane == g) gkey = w;
      }
    }
    // the best groups; every lane of a run carries its group's key, the lowest lane wins ties
    uint32_t live = 0;
    const int shift = q.lanes_shift >= 0 ? q.lanes_shift : 0;
    for (int j = 0; j < q.top_groups; ++j) {
      const uint32_t w = __reduce_max_sync(kAll, gkey);
      const int g = (__ffs(__ballot_sync(kAll, gkey == w)) - 1) >> shift;
      live |= 1u << g;
      if ((lane >> shift) == g) gkey = 0;
    }
    if (q.lanes_shift >= 0) {
      if (!((live >> (lane >> shift)) & 1u)) {
#pragma unroll
        for (int i = 0; i < NV; ++i) key[i] = 0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = e0 + i;
        if (e < q.E && !((live >> (e / q.per)) & 1u)) key[i] = 0;
      }
    }
  }

  // the k largest; lane j keeps the j-th id
  int mine = 0;
  uint32_t b = 0;   // this lane's largest
#pragma unroll
  for (int i = 0; i < NV; ++i) b = max(b, key[i]);
  // The k-th largest of the lanes' maxima bounds the k-th largest score from below; what
  // reaches it, little more than k, usually fits one candidate per lane. (Lanes with equal
  // maxima leave together: the bound may come out lower, never higher.)
  uint32_t bound = 0, left = b;
  for (int j = 0; j < q.k; ++j) {
    bound = __reduce_max_sync(kAll, left);
    if (left == bound) left = 0;
  }
  bound = max(bound, 1u);
  int have = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) have += key[i] >= bound;
  int upto = have;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kAll, upto, off);
    if (lane >= off) upto += o;
  }
  const int total = __shfl_sync(kAll, upto, 31);
  if (total <= 32) {
    uint2* list = s_list[threadIdx.x >> 5];
    int at = upto - have;   // candidates in ascending id
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (key[i] >= bound) list[at++] = make_uint2(key[i], (uint32_t)(e0 + i));
    __syncwarp();
    const uint2 c = lane < total ? list[lane] : make_uint2(0u, 0u);
    uint32_t mykey = c.x;
    for (int j = 0; j < q.k; ++j) {
      const uint32_t w = __reduce_max_sync(kAll, mykey);
      const int win = __ffs(__ballot_sync(kAll, mykey == w)) - 1;
      const int e = __shfl_sync(kAll, (int)c.y, win);
      if (lane == j) mine = e;
      if (lane == win) mykey = 0;
    }
  } else {   // many equal scores: one maximum of all at a time
    for (int j = 0; j < q.k; ++j) {
      const uint32_t w = __reduce_max_sync(kAll, b);
      const int win = __ffs(__ballot_sync(kAll, b == w)) - 1;
      int at = 0;
      if (lane == win) {
#pragma unroll
        for (int i = NV - 1; i >= 0; --i)
          if (key[i] == w) at = i;
        b = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (i == at) key[i] = 0;
          b = max(b, key[i]);
        }
      }
      at = __shfl_sync(kAll, at, win);
      if (lane == j) mine = win * NV + at;
    }
  }

  // gates from the scores without the bias, one lane per slot
  const bool on = lane < q.k;
  const float l = on ? clean(load(row + mine)) : -INFINITY;
  float w;
  if (q.renorm) w = renormalized(q.sigmoid, l);
  else if (q.sigmoid) w = sigmoid(l);
  else w = l > -INFINITY ? expf(l - m) * inv_z : 0.f;
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
// The whole row is written first (zeros, or the dense part), then lane j puts slot j's value
// in its place.
template <int NV, typename LT, typename DT>
__global__ void __launch_bounds__(32 * kWarps)
    route_bwd_kernel(const Rule q, const LT* __restrict__ logits,
                     const int32_t* __restrict__ topk_idx, const float* __restrict__ dgates,
                     DT* dlogits) {
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= q.T) return;
  const LT* row = logits + (size_t)t * q.E;
  DT* out = dlogits + (size_t)t * q.E;
  const int e0 = lane * NV;

  int id = lane < q.k ? topk_idx[(size_t)t * q.k + lane] : -1;
  if (id < 0 || id >= q.E) id = -1;
  const float dg = id >= 0 ? q.scale * dgates[(size_t)t * q.k + lane] : 0.f;
  const float l = id >= 0 ? clean(load(row + id)) : -INFINITY;

  float d;              // lane j: the gradient of slot j's expert
  float p[NV];
  if (!q.sigmoid && !q.renorm) {
    load_row<NV>(row, e0, q.E, q.vec, -INFINITY, p);
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = clean(p[i]);
    float m, inv_z;
    warp_softmax<NV>(p, m, inv_z);
    const float s = l > -INFINITY ? expf(l - m) * inv_z : 0.f;
    const float dot = warp_sum(s > 0.f ? s * dg : 0.f);   // a gate of 0 takes no part, whatever its dg
    d = s > 0.f ? s * (dg - dot) : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = -p[i] * dot;
  } else {
    const float part = q.sigmoid ? sigmoid(-l) : 1.f;
    float w;
    if (q.renorm) {
      w = renormalized(q.sigmoid, l);
      d = w * (dg - warp_sum(w > 0.f ? w * dg : 0.f));
    } else {
      w = sigmoid(l);
      d = w * dg;
    }
    d = w > 0.f ? d * part : 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) p[i] = 0.f;
  }
  store_row<NV>(out, e0, q.E, q.vec, p);
  __syncwarp();   // orders the row's stores before the slots'
  if (id >= 0) store(out + id, d);
}

template <typename LT, int NV>
void launch_fwd(const Rule& q, const void* logits, const float* bias, int32_t* idx, float* gates,
                cudaStream_t s) {
  const unsigned blocks = ((unsigned)q.T + kWarps - 1) / kWarps;
  route_kernel<NV, LT><<<blocks, 32 * kWarps, 0, s>>>(q, static_cast<const LT*>(logits), bias, idx,
                                                      gates);
}
template <typename LT, typename DT, int NV>
void launch_bwd(const Rule& q, const void* logits, const int32_t* idx, const float* dg, void* dl,
                cudaStream_t s) {
  const unsigned blocks = ((unsigned)q.T + kWarps - 1) / kWarps;
  route_bwd_kernel<NV, LT, DT><<<blocks, 32 * kWarps, 0, s>>>(
      q, static_cast<const LT*>(logits), idx, dg, static_cast<DT*>(dl));
}

// Logits per lane: the smallest of the built widths that holds a row in 32 lanes.
int lane_width(int E) {
  const int nv = (E + 31) / 32;
  return nv <= 2 ? nv : nv <= 4 ? 4 : nv <= 8 ? 8 : nv <= 12 ? 12 : 16;
}
template <class F>
void by_width(int E, F f) {
  switch (lane_width(E)) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 8: f(std::integral_constant<int, 8>{}); break;
    case 12: f(std::integral_constant<int, 12>{}); break;
    default: f(std::integral_constant<int, 16>{}); break;
  }
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
            false, false, -1, r->scale};
  const int nv = lane_width(r->E);
  if (q->per % nv == 0)
    for (int s = 0; s <= 5; ++s)
      if (q->per / nv == 1 << s) q->lanes_shift = s;
  return true;
}
// Vector accesses to the rows of [T][E]: whole lanes only, aligned to the widest power of
// two that divides a lane's bytes (at most 16).
bool rows_vectorize(int E, const void* p, mok_out_dtype type) {
  const int nv = lane_width(E), es = type == MOK_OUT_BF16 ? 2 : 4;
  const int width = std::min(16, (nv * es) & -(nv * es));
  return E % nv == 0 && (long long)E * es % width == 0 && aligned_to(p, width);
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
  q.vec = rows_vectorize(q.E, logits, logits_type);
  q.vec_bias = bias && rows_vectorize(q.E, bias, MOK_OUT_F32);
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
  q.vec = rows_vectorize(q.E, logits, logits_type) && rows_vectorize(q.E, dlogits, dlogits_type);
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
