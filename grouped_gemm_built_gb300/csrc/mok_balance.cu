// Balance loss of a router (include/mok_ops.h, mok_balance_fwd and mok_balance_bwd).
//
//   losses[0] = sum_t f_s (p_t . c_s),  f_s = coef E / (k T_s Tv),  s: row t's sequence
//   losses[1] = z_coef / Tv sum_t lse_t^2
// With the choices c_s counted first, the loss is a sum over rows: one pass over the logits and
// no sums over columns, however many sequences there are.
#include "mok_internal.h"
#include "mok_ops.h"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kWarps = 8;
constexpr int kCountRows = 256;   // rows per CTA that counts
constexpr int kMaxS = 1 << 20;

struct Args {
  int T, E, k, S;
  bool sigmoid, vec, vec_out;
  float coef, z;             // coef E / k, z_coef
  const int32_t* idx;
  const int32_t* seqs;
  int32_t* seq_counts;       // [S][E]
  int32_t* counts;           // [E]
  float* losses;
  double2* part;             // one per CTA of the forward
  const float* dlosses;
  int rows;                  // rows per CTA
};

// The last sequence that begins at or before row t (-1: none, S: behind the last).
__device__ __forceinline__ int find_sequence(const Args& q, int t) {
  if (!q.seqs) return 0;
  int lo = -1, hi = q.S + 1;
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (q.seqs[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void count_kernel(const Args q) {
  __shared__ int32_t hist[512];
  for (int e = threadIdx.x; e < q.E; e += blockDim.x) hist[e] = 0;
  const long long first = (long long)blockIdx.x * kCountRows;
  const int end = (int)min(first + kCountRows, (long long)q.T);
  __syncthreads();
  for (int a = (int)first; a < end;) {
    const int s = find_sequence(q, a);
    int b = end;
    if (q.seqs && s < q.S) b = max(a + 1, min(end, q.seqs[s + 1]));
    if (s >= 0 && s < q.S) {
      for (int i = threadIdx.x; i < (b - a) * q.k; i += blockDim.x) {
        const int e = q.idx[(size_t)a * q.k + i];
        if (e >= 0 && e < q.E) atomicAdd(&hist[e], 1);
      }
      __syncthreads();
      for (int e = threadIdx.x; e < q.E; e += blockDim.x) {
        const int c = hist[e];
        if (c) {
          atomicAdd(&q.seq_counts[(size_t)s * q.E + e], c);   // integers: any order, one result
          atomicAdd(&q.counts[e], c);
        }
        hist[e] = 0;
      }
      __syncthreads();
    }
    a = b;
  }
}

// A row's scores. In: cleaned logits (-inf past E). Out: p, and soft, lse where `z` is needed.
template <int NV>
struct RowScores {
  float p[NV], slope[NV], soft[NV], lse;
  __device__ __forceinline__ void make(const float* l, bool is_sigmoid, bool z, bool gradient) {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    lse = 0.f;
    if (m == -INFINITY) {
#pragma unroll
      for (int i = 0; i < NV; ++i) p[i] = slope[i] = soft[i] = 0.f;
      return;
    }
    if (!is_sigmoid || z) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        soft[i] = expf(l[i] - m);
        sum += soft[i];
      }
      sum = warp_sum(sum);
      lse = m + logf(sum);
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < NV; ++i) soft[i] *= inv;
    }
    if (!is_sigmoid) {
#pragma unroll
      for (int i = 0; i < NV; ++i) p[i] = slope[i] = soft[i];
      return;
    }
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // below -17, 1 + e^l is 1 in fp32 and sigmoid(l) is e^l: relative to the largest, as
      // their sum would underflow
      p[i] = m > -17.f ? sigmoid(l[i]) : expf(l[i] - m);
      if (l[i] == -INFINITY) p[i] = 0.f;
      sum += p[i];
    }
    sum = warp_sum(sum);
    const float inv = 1.f / sum;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      p[i] *= inv;
      slope[i] = gradient && p[i] > 0.f ? p[i] * sigmoid(-l[i]) : 0.f;
    }
  }
};

// What the rows of one sequence share, held by a warp while it stays in the sequence.
template <int NV>
struct Sequence {
  int s = -2, end = 0;        // rows up to `end` belong to it
  bool live = false;
  float factor = 0.f;
  int32_t c[NV];
  __device__ __forceinline__ void move_to(const Args& q, int t, int e0, int tv) {
    if (s != -2 && t < end) return;
    s = find_sequence(q, t);
    const int begin = !q.seqs ? 0 : s >= 0 ? q.seqs[s] : 0;
    end = !q.seqs || s >= q.S ? q.T : q.seqs[s + 1];
    live = s >= 0 && s < q.S && end > begin && tv > 0;
    if (!live) return;
    factor = q.coef / ((float)(end - begin) * (float)tv);
    load_counts(q, e0);
  }
  __device__ __forceinline__ void load_counts(const Args& q, int e0) {
    const int32_t* row = q.seq_counts + (size_t)s * q.E;
#pragma unroll
    for (int i = 0; i < NV; ++i) c[i] = e0 + i < q.E ? row[e0 + i] : 0;
  }
};

__device__ __forceinline__ int valid_rows(const Args& q) {
  return q.seqs ? q.seqs[q.S] - q.seqs[0] : q.T;
}

template <int NV, typename LT>
__global__ void __launch_bounds__(32 * kWarps) loss_kernel(const Args q, const LT* logits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * NV;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  const int tv = valid_rows(q);
  Sequence<NV> seq;
  double sum = 0., sum_z = 0.;
  for (long long t = first + warp; t < end; t += kWarps) {
    seq.move_to(q, (int)t, e0, tv);
    if (!seq.live) continue;
    float l[NV];
    load_row<NV>(logits + (size_t)t * q.E, e0, q.E, q.vec, -INFINITY, l);
#pragma unroll
    for (int i = 0; i < NV; ++i) l[i] = clean(l[i]);
    RowScores<NV> r;
    r.make(l, q.sigmoid, q.z > 0.f, false);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) dot += r.p[i] * (float)seq.c[i];
    sum += (double)(seq.factor * warp_sum(dot));
    sum_z += (double)(r.lse * r.lse);
  }
  __shared__ double2 s[kWarps];
  if (lane == 0) s[warp] = make_double2(sum, sum_z);
  __syncthreads();
  if (threadIdx.x == 0) {
    double2 t = make_double2(0., 0.);
    for (int i = 0; i < kWarps; ++i) {
      t.x += s[i].x;
      t.y += s[i].y;
    }
    q.part[blockIdx.x] = t;
  }
}

__global__ void loss_sum_kernel(const Args q, int parts) {
  __shared__ double2 s[256];
  double2 t = make_double2(0., 0.);
  for (int i = threadIdx.x; i < parts; i += 256) {
    t.x += q.part[i].x;
    t.y += q.part[i].y;
  }
  s[threadIdx.x] = t;
  __syncthreads();
  for (int n = 128; n > 0; n >>= 1) {
    if (threadIdx.x < n) {
      s[threadIdx.x].x += s[threadIdx.x + n].x;
      s[threadIdx.x].y += s[threadIdx.x + n].y;
    }
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int tv = valid_rows(q);
    q.losses[0] = (float)s[0].x;
    q.losses[1] = tv > 0 && q.z > 0.f ? (float)(s[0].y * q.z / tv) : 0.f;
  }
}

template <int NV, typename LT, typename DT>
__global__ void __launch_bounds__(32 * kWarps)
    balance_bwd_kernel(const Args q, const LT* logits, const DT* add, DT* dlogits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = lane * NV;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  const int tv = valid_rows(q);
  const float d0 = q.dlosses ? q.dlosses[0] : 1.f, d1 = q.dlosses ? q.dlosses[1] : 1.f;
  const float fz = q.z > 0.f && tv > 0 ? 2.f * q.z / (float)tv * d1 : 0.f;
  Sequence<NV> seq;
  float u[NV];
  int of = -2;
  for (long long t = first + warp; t < end; t += kWarps) {
    seq.move_to(q, (int)t, e0, tv);
    float d[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) d[i] = 0.f;
    if (add) load_row<NV>(add + (size_t)t * q.E, e0, q.E, q.vec_out, 0.f, d);
    if (seq.live) {
      if (of != seq.s) {
        // counts relative to their mean, an integer: sum_e p_e = 1, so the gradient is the same,
        // without the cancellation of nearly even counts
        int total = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i) total += seq.c[i];
        total = __reduce_add_sync(kAll, total);
        const int mean = total / q.E;
#pragma unroll
        for (int i = 0; i < NV; ++i) u[i] = (float)(seq.c[i] - mean) * (seq.factor * d0);
        of = seq.s;
      }
      float l[NV];
      load_row<NV>(logits + (size_t)t * q.E, e0, q.E, q.vec, -INFINITY, l);
#pragma unroll
      for (int i = 0; i < NV; ++i) l[i] = clean(l[i]);
      RowScores<NV> r;
      r.make(l, q.sigmoid, fz != 0.f, true);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) dot += r.p[i] * u[i];
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        d[i] += r.slope[i] * (u[i] - dot);
        if (fz != 0.f) d[i] += fz * r.lse * r.soft[i];
      }
    }
    store_row<NV>(dlogits + (size_t)t * q.E, e0, q.E, q.vec_out, d);
  }
}

constexpr int kParts = 152 * 8;

bool make_args(const mok_balance* r, int T, int S, Args* q) {
  if (!r || T < 0 || S < 1 || S > kMaxS) return false;
  if (r->E < 1 || r->E > 512 || r->k < 1 || r->k > 32) return false;
  if (r->score != MOK_SCORE_SOFTMAX && r->score != MOK_SCORE_SIGMOID) return false;
  if (!std::isfinite(r->coef) || r->coef < 0.f || !std::isfinite(r->z_coef) || r->z_coef < 0.f)
    return false;
  *q = Args{};
  q->T = T; q->E = r->E; q->k = r->k; q->S = S;
  q->sigmoid = r->score == MOK_SCORE_SIGMOID;
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
  *saved_bytes = counts_bytes(rule, S) + kParts * sizeof(double2);
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
  q.vec = rows_vectorize(q.E, logits, logits_type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(saved, 0, (size_t)S * q.E * 4, s) != cudaSuccess) return MOK_ERR_CUDA;
  if (cudaMemsetAsync(counts, 0, (size_t)q.E * 4, s) != cudaSuccess) return MOK_ERR_CUDA;
  unsigned parts = 0;
  if (T > 0) {
    count_kernel<<<((unsigned)T + kCountRows - 1) / kCountRows, 256, 0, s>>>(q);
    parts = ((unsigned)T + q.rows - 1) / q.rows;
    by_width(q.E, [&](auto nv) {
      constexpr int NV = decltype(nv)::value;
      if (logits_type == MOK_OUT_BF16)
        loss_kernel<NV><<<parts, 32 * kWarps, 0, s>>>(q, static_cast<const __nv_bfloat16*>(logits));
      else
        loss_kernel<NV><<<parts, 32 * kWarps, 0, s>>>(q, static_cast<const float*>(logits));
    });
  }
  loss_sum_kernel<<<1, 256, 0, s>>>(q, (int)parts);
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
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
      balance_bwd_kernel<NV><<<ctas, 32 * kWarps, 0, s>>>(
          q, static_cast<const LT*>(logits), static_cast<const DT*>(add), static_cast<DT*>(dlogits));
    };
    const bool lb = logits_type == MOK_OUT_BF16, db = dlogits_type == MOK_OUT_BF16;
    if (lb && db) go(__nv_bfloat16{}, __nv_bfloat16{});
    else if (lb) go(__nv_bfloat16{}, 0.f);
    else if (db) go(0.f, __nv_bfloat16{});
    else go(0.f, 0.f);
  });
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
