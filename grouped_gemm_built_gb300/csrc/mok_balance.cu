// Balance loss of a router (include/mok_ops.h, mok_balance_fwd and mok_balance_bwd).
//
//   losses[0] = sum_t f_s (p_t . c_s),  f_s = coef E / (k T_s Tv),  s: row t's sequence
//   losses[1] = z_coef / Tv sum_t lse_t^2
// With the choices c_s counted first, the loss is a sum over rows: one pass over the logits and
// no sums over columns, however many sequences there are.
//
// Two launches: the choices are counted by a cluster of CTAs per sequence, which joins its counts
// through distributed shared memory and so needs no zeroed memory and no atomics on it; then a warp
// per row takes the scores and the product with its sequence's counts. The rows' kernel starts
// while the choices are still counted and has its first logits by then; its last CTA adds the CTAs'
// sums in their order.
#include <climits>

#include "mok_internal.h"
#include "mok_launch.cuh"
#include "mok_ops.h"
#include "mok_ptx.cuh"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kWarps = 8;
constexpr int kCountThreads = 1024;
constexpr int kMaxS = 1 << 20;
constexpr int kParts = 152 * 8;   // CTAs of the rows' kernels at most

struct Args {
  int T, E, k, S;
  bool vec, vec_out;
  float coef, z;             // coef E / k, z_coef
  const int32_t* idx;
  const int32_t* seqs;
  int32_t* seq_counts;       // [S][E]
  int32_t* counts;           // [E]
  float* losses;
  double2* part;             // one per CTA of the forward
  unsigned* ticket;          // CTAs of the forward that are done
  const float* dlosses;
  int rows;                  // rows per CTA
};

// The last sequence that begins at or before row t (-1: none, S: behind the last), by a whole warp:
// 32 offsets at a time.
__device__ __forceinline__ int find_sequence(const Args& q, int t) {
  if (!q.seqs) return 0;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = q.S + 1;   // the first offset above t lies in [lo, hi]
  while (true) {
    const int step = (hi - lo + 31) / 32, i = lo + lane * step;
    const int below = __popc(__ballot_sync(kAll, i < hi && q.seqs[min(i, q.S)] <= t));
    if (below == 0) return lo - 1;
    lo += (below - 1) * step + 1;
    hi = min(hi, lo + step - 1);
    if (lo >= hi) return lo - 1;
  }
}

// Counts of the choices of one sequence by a cluster. Rank r takes the r-th share of the ids.
__global__ void __launch_bounds__(kCountThreads) count_kernel(const Args q, int ctas) {
  launch_dependents();
  __shared__ int32_t hist[512];
  const int s = blockIdx.x / ctas, rank = blockIdx.x % ctas;
  for (int e = threadIdx.x; e < 512; e += kCountThreads) hist[e] = 0;
  int begin = 0, end = q.T;
  if (q.seqs) {   // offsets outside the batch are cut off
    begin = max(q.seqs[s], 0);
    end = min(q.seqs[s + 1], q.T);
  }
  __syncthreads();
  if (end > begin) {
    const size_t first = (size_t)begin * q.k, n = (size_t)(end - begin) * q.k;
    const size_t lo = first + n * rank / ctas, hi = first + n * (rank + 1) / ctas;
    auto count = [&](int e) {
      if (e >= 0 && e < q.E) atomicAdd(&hist[e], 1);
    };
    // whole groups of four, and the ids before and behind them
    const size_t a = min((lo + 3) & ~(size_t)3, hi), b = max(hi & ~(size_t)3, a);
    if ((reinterpret_cast<uintptr_t>(q.idx) & 15) == 0) {
      if (lo + threadIdx.x < a) count(q.idx[lo + threadIdx.x]);
      if (b + threadIdx.x < hi) count(q.idx[b + threadIdx.x]);
      const int4* v = reinterpret_cast<const int4*>(q.idx);
#pragma unroll 8
      for (size_t i = a / 4 + threadIdx.x; i < b / 4; i += kCountThreads) {
        const int4 x = v[i];
        count(x.x), count(x.y), count(x.z), count(x.w);
      }
    } else {
#pragma unroll 8
      for (size_t i = lo + threadIdx.x; i < hi; i += kCountThreads) count(q.idx[i]);
    }
  }
  if (ctas > 1) cluster_sync_all();
  else __syncthreads();
  // the ranks' counts of a share of the experts each
  for (int e = rank + threadIdx.x * ctas; e < q.E; e += kCountThreads * ctas) {
    int c = 0;
    for (int r = 0; r < ctas; ++r) {
      int x = hist[e];
      if (ctas > 1)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(mapa_rank(&hist[e], r)) : "memory");
      c += x;
    }
    q.seq_counts[(size_t)s * q.E + e] = c;
    if (s == 0) q.counts[e] = q.S == 1 ? c : 0;   // several: the rows' kernel adds them up
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *q.ticket = 0;
    if (q.T == 0) q.losses[0] = q.losses[1] = 0.f;
  }
  if (ctas > 1) cluster_sync_all();   // nobody leaves while its counts are read
}

constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float exp2_fast(float t) {   // 2^t to 2 ulp, 0 below 2^-126
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  return e;
}
__device__ __forceinline__ float inverse(float x) {     // to 1 ulp; 0 above 2^126
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// e^x of NV values, x clamped to +-200 (NaN: the lower limit). One product x log2 e would leave
// an error of |x| / 2 ulp; what its rounding cut off comes back as a factor.
template <int NV>
__device__ __forceinline__ Vec<NV> exp_vec(Vec<NV> x) {
#pragma unroll
  for (int i = 0; i < NV; ++i) x.v[i] = fminf(fmaxf(x.v[i], -200.f), 200.f);
  const Vec<NV> k = Vec<NV>::all(kLog2e), t = x * k;
  const Vec<NV> cut = fma(x, k, t * Vec<NV>::all(-1.f)) * Vec<NV>::all(0.693147182f);
  Vec<NV> e;
#pragma unroll
  for (int i = 0; i < NV; ++i) e.v[i] = exp2_fast(t.v[i]);
  return fma(e, cut, e);
}

// a and b summed over the warp: the lower half goes on with a, the upper with b.
__device__ __forceinline__ float2 warp_sum2(float a, float b) {
  const bool low = (threadIdx.x & 16) == 0;
  const float other = __shfl_xor_sync(kAll, low ? b : a, 16);
  a = (low ? a : b) + other;
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) a += __shfl_xor_sync(kAll, a, off);
  return make_float2(__shfl_sync(kAll, a, 0), __shfl_sync(kAll, a, 16));
}

// The largest logit of the warp's row, as the rule reads it: NaN is none, +inf becomes the largest
// finite value, also in l.
template <int NV>
__device__ __forceinline__ float row_max(Vec<NV>& l) {
  float m = l.v[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l.v[i]);
  m = warp_max(m == m ? m : -INFINITY);
  if (m == INFINITY) {
    m = FLT_MAX;
#pragma unroll
    for (int i = 0; i < NV; ++i) l.v[i] = fminf(l.v[i], FLT_MAX);
  }
  return m;
}

// What the rows of one sequence share, held by a warp while it stays in the sequence.
template <int NV>
struct Sequence {
  int s = -2, end = 0;        // rows up to `end` belong to it
  bool live = false;
  float factor = 0.f;
  // Whether row t begins another sequence; its counts are then the caller's to load.
  __device__ __forceinline__ bool move_to(const Args& q, int t, int tv) {
    if (s != -2 && t < end) return false;
    s = find_sequence(q, t);
    const int begin = !q.seqs ? 0 : s >= 0 ? q.seqs[s] : 0;
    end = !q.seqs || s >= q.S ? q.T : q.seqs[s + 1];
    live = s >= 0 && s < q.S && end > begin && tv > 0;
    factor = live ? q.coef / ((float)(end - begin) * (float)tv) : 0.f;
    return live;
  }
};
template <int NV>
__device__ __forceinline__ void load_counts(const Args& q, int s, int e0, int32_t* c) {
  const int32_t* row = q.seq_counts + (size_t)s * q.E;
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = e0 + i < q.E ? row[e0 + i] : 0;
}
__device__ __forceinline__ int valid_rows(const Args& q) {
  return q.seqs ? q.seqs[q.S] - q.seqs[0] : q.T;
}
template <int NV, typename LT>
__device__ __forceinline__ void load_logits(const Args& q, const LT* logits, long long t, int e0, float* l) {
  load_row<NV>(logits + (size_t)t * q.E, e0, q.E, q.vec, -INFINITY, l);
}

// Sigmoid scores whose sum is below this are taken relative to the largest logit: there each is e^l
// to 32 bits, and the smallest would underflow.
constexpr float kTiny = 1e-20f;

// One product with log2 e: an exponential is off by up to |x| / 2 ulp, which the loss, a sum in which
// the largest scores weigh most, does not show.
template <int NV, bool SIGMOID, typename LT>
__global__ void __launch_bounds__(32 * kWarps) loss_kernel(const Args q, const LT* logits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * NV;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  Vec<NV> next;
  if (first + warp < end) load_logits<NV>(q, logits, first + warp, e0, next.v);
  const int tv = valid_rows(q);
  Sequence<NV> seq;
  if (first + warp < end) seq.move_to(q, (int)first + warp, tv);
  bool fresh = seq.live;
  wait_prerequisites();
  // with several sequences, this CTA's share of them into the counts of all
  if (q.S > 1) {
    for (int s = blockIdx.x; s < q.S; s += gridDim.x) {
      for (int e = threadIdx.x; e < q.E; e += 32 * kWarps) {
        const int c = q.seq_counts[(size_t)s * q.E + e];
        if (c) atomicAdd(&q.counts[e], c);   // integers: any order, one result
      }
    }
  }
  float sum = 0.f, sum_z = 0.f;
  Vec<NV> c;
  for (int t = (int)first + warp; t < end; t += kWarps) {
    Vec<NV> l = next;
    if (end - t > kWarps) load_logits<NV>(q, logits, t + kWarps, e0, next.v);
    fresh |= seq.move_to(q, t, tv);
    if (!seq.live) continue;
    if (fresh) {
      int32_t n[NV];
      load_counts<NV>(q, seq.s, e0, n);
#pragma unroll
      for (int i = 0; i < NV; ++i) c.v[i] = (float)n[i];
      fresh = false;
    }
    float2 w;        // sum of the scores, their product with the counts
    bool tiny = false;
    if constexpr (SIGMOID) {
      const Vec<NV> x = l * Vec<NV>::all(-kLog2e);
      Vec<NV> p;
#pragma unroll
      for (int i = 0; i < NV; ++i) p.v[i] = inverse(1.f + exp2_fast(fminf(x.v[i], 200.f)));
      w = warp_sum2(p.sum(), dot(p, c));
      tiny = w.x < kTiny;
    }
    if (!SIGMOID || tiny || q.z > 0.f) {
      const float m = row_max<NV>(l);
      if (m == -INFINITY) continue;
      const Vec<NV> x = (l + Vec<NV>::all(-m)) * Vec<NV>::all(kLog2e);
      Vec<NV> p;
#pragma unroll
      for (int i = 0; i < NV; ++i) p.v[i] = exp2_fast(fmaxf(x.v[i], -200.f));
      const float2 v = warp_sum2(p.sum(), dot(p, c));
      if (!SIGMOID || tiny) w = v;
      const float lse = m + __logf(v.x);
      sum_z = fmaf(lse, lse, sum_z);
    }
    sum += seq.factor * __fdividef(w.y, w.x);
  }
  __shared__ double2 s[kWarps];
  __shared__ bool last;
  if (lane == 0) s[warp] = make_double2(sum, sum_z);
  __syncthreads();
  if (threadIdx.x == 0) {
    double2 t = make_double2(0., 0.);
    for (int i = 0; i < kWarps; ++i) {
      t.x += s[i].x;
      t.y += s[i].y;
    }
    q.part[blockIdx.x] = t;
    __threadfence();
    last = atomicAdd(q.ticket, 1u) + 1 == gridDim.x;
  }
  __syncthreads();
  if (!last) return;
  // the last CTA: everyone's sums, in their order
  __threadfence();
  double2 t = make_double2(0., 0.);
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 32 * kWarps) {
    t.x += __ldcg(&q.part[i].x);
    t.y += __ldcg(&q.part[i].y);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    t.x += __shfl_xor_sync(kAll, t.x, off);
    t.y += __shfl_xor_sync(kAll, t.y, off);
  }
  if (lane == 0) s[warp] = t;
  __syncthreads();
  if (threadIdx.x == 0) {
    t = make_double2(0., 0.);
    for (int i = 0; i < kWarps; ++i) {
      t.x += s[i].x;
      t.y += s[i].y;
    }
    q.losses[0] = (float)t.x;
    q.losses[1] = tv > 0 && q.z > 0.f ? (float)(t.y * q.z / tv) : 0.f;
  }
}

// softmax  p_e (u_e - p.u + 2 z / Tv lse);  sigmoid  p_e (1 - s_e) (u_e - p.u), the penalty apart
template <int NV, bool SIGMOID, typename LT, typename DT>
__global__ void __launch_bounds__(32 * kWarps)
    balance_bwd_kernel(const Args q, const LT* logits, const DT* add, DT* dlogits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * NV;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  Vec<NV> next, next_add = Vec<NV>::all(0.f);
  auto load_next = [&](long long t) {
    load_logits<NV>(q, logits, t, e0, next.v);
    if (add) load_row<NV>(add + (size_t)t * q.E, e0, q.E, q.vec_out, 0.f, next_add.v);
  };
  if (first + warp < end) load_next(first + warp);
  const int tv = valid_rows(q);
  const float d0 = q.dlosses ? q.dlosses[0] : 1.f, d1 = q.dlosses ? q.dlosses[1] : 1.f;
  const float fz = q.z > 0.f && tv > 0 ? 2.f * q.z / (float)tv * d1 : 0.f;
  Sequence<NV> seq;
  Vec<NV> u;
  for (int t = (int)first + warp; t < end; t += kWarps) {
    Vec<NV> l = next, d = next_add;
    if (end - t > kWarps) load_next(t + kWarps);
    if (seq.move_to(q, t, tv)) {
      // counts relative to their mean, an integer: sum_e p_e = 1, so the gradient is the same,
      // without the cancellation of nearly even counts
      int32_t c[NV];
      load_counts<NV>(q, seq.s, e0, c);
      int total = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) total += c[i];
      const int mean = __reduce_add_sync(kAll, total) / q.E;
#pragma unroll
      for (int i = 0; i < NV; ++i) u.v[i] = (float)(c[i] - mean) * (seq.factor * d0);
    }
    bool tiny = false;
    if (SIGMOID && seq.live) {
      Vec<NV> e = exp_vec<NV>(l * Vec<NV>::all(-1.f)), p;   // e^-l, at most e^88
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        e.v[i] = l.v[i] > -88.f ? e.v[i] : FLT_MAX;   // and masked: a score of 0
        p.v[i] = inverse(1.f + e.v[i]);
      }
      const float2 w = warp_sum2(p.sum(), dot(p, u));
      tiny = w.x < kTiny;
      if (!tiny) {
        const float inv = 1.f / w.x;
        // sigmoid (1 - sigmoid) = (e^-l sigmoid) sigmoid
        d = fma((e * p) * (p * Vec<NV>::all(inv)), u + Vec<NV>::all(-w.y * inv), d);
      }
    }
    if (seq.live && (!SIGMOID || tiny || fz != 0.f)) {
      const float m = row_max<NV>(l);
      if (m > -INFINITY) {
        const Vec<NV> p = exp_vec<NV>(l + Vec<NV>::all(-m));
        const float2 w = warp_sum2(p.sum(), dot(p, u));
        const float inv = 1.f / w.x;
        const float shift = fz != 0.f ? fz * (m + logf(w.x)) : 0.f;
        const Vec<NV> scores = p * Vec<NV>::all(inv);
        if (!SIGMOID || tiny) d = fma(scores, u + Vec<NV>::all(shift - w.y * inv), d);
        else d = fma(scores, Vec<NV>::all(shift), d);
      }
    }
    store_row<NV>(dlogits + (size_t)t * q.E, e0, q.E, q.vec_out, d.v);
  }
}

bool make_args(const mok_balance* r, int T, int S, Args* q) {
  if (!r || T < 0 || S < 1 || S > kMaxS) return false;
  if (r->E < 1 || r->E > 512 || r->k < 1 || r->k > 32) return false;
  if (r->score != MOK_SCORE_SOFTMAX && r->score != MOK_SCORE_SIGMOID) return false;
  if (!std::isfinite(r->coef) || r->coef < 0.f || !std::isfinite(r->z_coef) || r->z_coef < 0.f)
    return false;
  *q = Args{};
  q->T = T; q->E = r->E; q->k = r->k; q->S = S;
  q->coef = (float)((double)r->coef * r->E / r->k);
  q->z = r->z_coef;
  // rows per CTA: whole rounds of its warps, at most kParts CTAs
  const long long per = ((long long)T + kParts - 1) / kParts;
  q->rows = (int)((per + kWarps - 1) / kWarps * kWarps);
  if (q->rows < kWarps) q->rows = kWarps;
  return true;
}
size_t counts_bytes(const mok_balance* r, int S) { return align_up((size_t)S * r->E * 4, 256); }

}  // namespace
}  // namespace mok

extern "C" mok_status mok_balance_get_sizes(const mok_balance* rule, int T, int S,
                                            size_t* saved_bytes) {
  using namespace mok;
  Args q;
  if (!make_args(rule, T, S, &q) || !saved_bytes) return MOK_ERR_INVALID_ARG;
  *saved_bytes = counts_bytes(rule, S) + kParts * sizeof(double2) + 256;
  return MOK_OK;
}

extern "C" mok_status mok_balance_fwd(const mok_balance* rule, int T, const void* logits,
                                      mok_out_dtype logits_type, const int32_t* topk_idx,
                                      const int32_t* seqs, int S, float* losses, int32_t* counts,
                                      void* saved, void* stream) {
  using namespace mok;
  Args q;
  if (!make_args(rule, T, S, &q) || !is_type(logits_type)) return MOK_ERR_INVALID_ARG;
  if (!losses || !counts || (T > 0 && (!logits || !topk_idx)) || (!seqs && S != 1))
    return MOK_ERR_INVALID_ARG;
  if (!aligned_to(logits, logits_type == MOK_OUT_BF16 ? 2 : 4) || !aligned_to(topk_idx, 4) ||
      !aligned_to(seqs, 4) || !aligned_to(losses, 4) || !aligned_to(counts, 4))
    return MOK_ERR_INVALID_ARG;
  if (!saved || !aligned_to(saved, 256)) return MOK_ERR_WORKSPACE;
  q.idx = topk_idx; q.seqs = seqs; q.counts = counts; q.losses = losses;
  q.seq_counts = static_cast<int32_t*>(saved);
  q.part = reinterpret_cast<double2*>(static_cast<char*>(saved) + counts_bytes(rule, S));
  q.ticket = reinterpret_cast<unsigned*>(q.part + kParts);
  q.vec = rows_vectorize(q.E, logits, logits_type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a sequence's CTAs: eight, but one where sequences are short or many
  const int ctas = (long long)T / S * q.k >= 4096 && S <= 4096 ? 8 : 1;
  cudaError_t e = launch(count_kernel, dim3((unsigned)S * ctas), dim3(kCountThreads), 0, ctas, false, s,
                         q, ctas);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  if (T > 0) {
    const unsigned parts = ((unsigned)T + q.rows - 1) / q.rows;
    by_width(q.E, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      auto go = [&](auto kernel, auto* l) {
        e = launch(kernel, dim3(parts), dim3(32 * kWarps), 0, 1, true, s, q, l);
      };
      const auto* lb = static_cast<const __nv_bfloat16*>(logits);
      const auto* lf = static_cast<const float*>(logits);
      const bool sg = rule->score == MOK_SCORE_SIGMOID, b = logits_type == MOK_OUT_BF16;
      if (sg && b) go(loss_kernel<NV, true, __nv_bfloat16>, lb);
      else if (sg) go(loss_kernel<NV, true, float>, lf);
      else if (b) go(loss_kernel<NV, false, __nv_bfloat16>, lb);
      else go(loss_kernel<NV, false, float>, lf);
    });
  }
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_balance_bwd(const mok_balance* rule, int T, const void* logits,
                                      mok_out_dtype logits_type, const int32_t* seqs, int S,
                                      const void* saved, const float* dlosses, const void* add,
                                      void* dlogits, mok_out_dtype dlogits_type, void* stream) {
  using namespace mok;
  Args q;
  if (!make_args(rule, T, S, &q) || !is_type(logits_type) || !is_type(dlogits_type))
    return MOK_ERR_INVALID_ARG;
  if (!seqs && S != 1) return MOK_ERR_INVALID_ARG;
  if (T == 0) return MOK_OK;
  if (!logits || !dlogits) return MOK_ERR_INVALID_ARG;
  const uintptr_t out = dlogits_type == MOK_OUT_BF16 ? 2 : 4;
  if (!aligned_to(logits, logits_type == MOK_OUT_BF16 ? 2 : 4) || !aligned_to(seqs, 4) ||
      !aligned_to(dlosses, 4) || !aligned_to(add, out) || !aligned_to(dlogits, out))
    return MOK_ERR_INVALID_ARG;
  if (!saved || !aligned_to(saved, 256)) return MOK_ERR_WORKSPACE;
  q.seqs = seqs; q.dlosses = dlosses;
  q.seq_counts = static_cast<int32_t*>(const_cast<void*>(saved));
  q.vec = rows_vectorize(q.E, logits, logits_type);
  q.vec_out = rows_vectorize(q.E, dlogits, dlogits_type) &&
              (!add || rows_vectorize(q.E, add, dlogits_type));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned ctas = ((unsigned)T + q.rows - 1) / q.rows;
  by_width(q.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    auto go = [&](auto lt, auto dt) {
      using LT = decltype(lt);
      using DT = decltype(dt);
      auto* kernel = rule->score == MOK_SCORE_SIGMOID ? balance_bwd_kernel<NV, true, LT, DT>
                                                      : balance_bwd_kernel<NV, false, LT, DT>;
      kernel<<<ctas, 32 * kWarps, 0, s>>>(q, static_cast<const LT*>(logits),
                                          static_cast<const DT*>(add), static_cast<DT*>(dlogits));
    };
    const bool lb = logits_type == MOK_OUT_BF16, db = dlogits_type == MOK_OUT_BF16;
    if (lb && db) go(__nv_bfloat16{}, __nv_bfloat16{});
    else if (lb) go(__nv_bfloat16{}, 0.f);
    else if (db) go(0.f, __nv_bfloat16{});
    else go(0.f, 0.f);
  });
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
