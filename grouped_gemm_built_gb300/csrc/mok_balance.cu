// Balance loss of a router (include/mok_ops.h, mok_balance_fwd and mok_balance_bwd).
//
//   losses[0] = sum_t f_s (p_t . c_s),  f_s = coef E / (k T_s Tv),  s: row t's sequence
//   losses[1] = z_coef / Tv sum_t lse_t^2
// With the choices c_s counted, the loss is a sum over rows: one pass over the logits, however many
// sequences there are. A warp adds up the scores of its rows per expert, and multiplies by the counts
// when it leaves a sequence.
//
// Two launches: the choices are counted by a cluster of CTAs per sequence, which joins its counts
// through distributed shared memory and so needs no zeroed memory and no atomics on it; then a warp
// per row takes the scores. The rows' kernel runs while the choices are still counted, and waits for
// the counts when it has its scores; its last CTA adds the CTAs' sums in their order.
#include <climits>

#include "mok_internal.h"
#include "mok_launch.cuh"
#include "mok_ops.h"
#include "mok_ptx.cuh"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kWarps = 8;
constexpr int kCountThreads = 512;   // at most
constexpr int kMaxS = 1 << 20;
constexpr int kSmallCtas = 8, kSmallWarps = 16;
constexpr int kSmallIds = 8192, kSmallRows = 1024, kSmallScores = 1 << 18;
constexpr int kGroups = 16;        // clusters that count one sequence at most
constexpr int kSms = 152;
constexpr int kLossCtas = 4;       // CTAs a SM
constexpr int kParts = kSms * kLossCtas;
template <int NV, bool SIGMOID>       // ... and of the backward: what the registers allow
constexpr int kBwdCtas = NV <= 8 ? (SIGMOID ? 3 : 4) : NV <= 12 && !SIGMOID ? 3 : 2;

struct Args {
  int T, E, k, S;
  bool vec;                  // a lane's elements of a row lie side by side, in vectors
  float coef, z;             // coef E / k, z_coef
  const int32_t* idx;
  const int32_t* seqs;
  int32_t* seq_counts;       // [S][E]
  int32_t* counts;           // [E]
  float* losses;
  int32_t* group_counts;     // [groups][E]: one sequence's counts, by several clusters
  int groups;
  float2* part;              // one per CTA of the forward
  unsigned* ticket;          // CTAs of the forward that are done
  const float* dlosses;
  int rows;                  // rows per CTA
};

// Counts of the choices of one sequence by a cluster, whose CTAs take a share of the ids each; a long
// batch without offsets is shared by `groups` clusters, whose counts the rows' kernel adds up.
__global__ void __launch_bounds__(kCountThreads) count_kernel(const Args q, int ctas) {
  launch_dependents();
  const int threads = blockDim.x;
  __shared__ int32_t hist[512];
  const int s = q.groups > 1 ? 0 : blockIdx.x / ctas, rank = blockIdx.x % ctas;
  const int share = q.groups > 1 ? blockIdx.x : rank, shares = q.groups * ctas;
  for (int e = threadIdx.x; e < 512; e += threads) hist[e] = 0;
  int begin = 0, end = q.T;
  if (q.seqs) {   // offsets outside the batch are cut off
    begin = max(q.seqs[s], 0);
    end = min(q.seqs[s + 1], q.T);
  }
  __syncthreads();
  if (end > begin) {
    const size_t first = (size_t)begin * q.k, n = (size_t)(end - begin) * q.k;
    const size_t lo = first + n * share / shares, hi = first + n * (share + 1) / shares;
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
      for (size_t i = a / 4 + threadIdx.x; i < b / 4; i += threads) {
        const int4 x = v[i];
        count(x.x), count(x.y), count(x.z), count(x.w);
      }
    } else {
#pragma unroll 8
      for (size_t i = lo + threadIdx.x; i < hi; i += threads) count(q.idx[i]);
    }
  }
  if (ctas > 1) cluster_sync_all();
  else __syncthreads();
  // the ranks' counts of a share of the experts each
  for (int e = rank + threadIdx.x * ctas; e < q.E; e += threads * ctas) {
    int c = 0;
    for (int r = 0; r < ctas; ++r) {
      int x = hist[e];
      if (ctas > 1)
        asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(x) : "r"(mapa_rank(&hist[e], r)) : "memory");
      c += x;
    }
    if (q.groups > 1) {
      q.group_counts[blockIdx.x / ctas * q.E + e] = c;
    } else {
      q.seq_counts[(size_t)s * q.E + e] = c;
      if (s == 0) q.counts[e] = q.S == 1 ? c : 0;   // several: the rows' kernel adds them up
    }
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
// e^x of NV values to 5 u + |x| u / 20, u = 2^-24: 2^t with t = x log2 e rounded down, from a little below, and
// what that cut off, x - t ln 2, as a factor. It lies in (0, 2^-16) for -88 <= x <= 88, so that a saturated
// sum gives it; which is 0, not NaN, for x = -inf, and e^x is 0. NaN for NaN, inf or NaN for inf.
template <int NV>
__device__ __forceinline__ Vec<NV> exp_vec(const Vec<NV>& x) {
  Vec<NV> t, e, cut;
  if constexpr (NV == 1) t.v[0] = __fmaf_rd(x.v[0], kLog2e, -0x1p-19f);
#pragma unroll
  for (int i = 0; i + 1 < NV; i += 2)
    t.set(i, __ffma2_rd(x.pair(i), make_float2(kLog2e, kLog2e), make_float2(-0x1p-19f, -0x1p-19f)));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    e.v[i] = exp2_fast(t.v[i]);
    cut.v[i] = __saturatef(fmaf(-t.v[i], 0.693147182f, x.v[i]));
  }
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

// The largest of the warp's cleaned logits; and e^(l - m), at least e^-200, which is 0: 1 for the largest.
template <int NV>
__device__ __forceinline__ float row_max(const Vec<NV>& l) {
  float m = l.v[0];
#pragma unroll
  for (int i = 1; i < NV; ++i) m = fmaxf(m, l.v[i]);
  return warp_max(m);
}
template <int NV>
__device__ __forceinline__ Vec<NV> exp_below(Vec<NV> l, float m) {
#pragma unroll
  for (int i = 0; i < NV; ++i) l.v[i] = fmaxf(l.v[i] - m, -200.f);
  const Vec<NV> minus = l * Vec<NV>::all(-kLog2e), cut = fma(minus, Vec<NV>::all(0.693147182f), l);
  Vec<NV> e;
#pragma unroll
  for (int i = 0; i < NV; ++i) e.v[i] = exp2_fast(-minus.v[i]);
  return fma(e, cut, e);
}

// Where the warp's row lies, and what the rows of its sequence share. Up to 32 offsets stay in the
// lanes, read once; more are searched 32 at a time.
struct Sequence {
  int off;                    // lane i: offset i
  int s = -2, end = 0;        // rows up to `end` belong to sequence s (-1: before the first, S: behind)
  int valid;                  // rows of all sequences
  bool live = false;
  float factor = 0.f;
  __device__ __forceinline__ explicit Sequence(const Args& q) {
    const int lane = threadIdx.x & 31;
    off = q.seqs ? q.seqs[min(lane, q.S)] : 0;
    const int last = !q.seqs ? q.T : q.S < 32 ? __shfl_sync(kAll, off, q.S & 31) : q.seqs[q.S];
    valid = last - __shfl_sync(kAll, off, 0);
  }
  // The number of offsets at or before t, less one.
  __device__ __forceinline__ int find(const Args& q, int t) const {
    const int lane = threadIdx.x & 31;
    if (q.S < 32) return __popc(__ballot_sync(kAll, lane <= q.S && off <= t)) - 1;
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
  __device__ __forceinline__ bool ends_before(int t) const { return s == -2 || t >= end; }
  // Whether row t begins another sequence; its counts are then the caller's to load.
  __device__ __forceinline__ bool move_to(const Args& q, int t) {
    if (!ends_before(t)) return false;
    int begin = 0;
    if (!q.seqs) {
      s = 0;
      end = q.T;
    } else {
      s = find(q, t);
      if (q.S < 32) {
        begin = __shfl_sync(kAll, off, s & 31);
        end = __shfl_sync(kAll, off, (s + 1) & 31);
      } else {
        begin = q.seqs[max(s, 0)];
        end = q.seqs[min(s + 1, q.S)];
      }
      if (s >= q.S) end = q.T;
    }
    live = s >= 0 && s < q.S && end > begin && valid > 0;
    factor = live ? q.coef / ((float)(end - begin) * (float)valid) : 0.f;
    return live;
  }
};
// A lane's i-th element of a row: the NV elements from NV lane on, where rows allow such accesses; else
// every 32nd.
template <int NV>
__device__ __forceinline__ int element(bool vec, int i) {
  const int lane = threadIdx.x & 31;
  return vec ? lane * NV + i : lane + 32 * i;
}
template <int NV>
__device__ __forceinline__ void load_counts(const int32_t* row, int E, bool vec, int32_t* c) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = element<NV>(vec, i);
    c[i] = e < E ? row[e] : 0;
  }
}
// A lane's elements of a row as they lie in memory (past the row's end: `fill`'s bits), loaded a row
// ahead of their use. (Three rows ahead, through shared memory, were no faster: 65536 rows of 384 22.8 us
// backward both ways.)
template <int NV, typename T>
struct RawRow {
  static constexpr int kBytes = NV * (int)sizeof(T), kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* row, int E, bool vec, uint32_t fill) {
    const int lane = threadIdx.x & 31;
    if constexpr (kBytes % 4 == 0) {
      if (vec) {
        if (lane * NV < E) {
          constexpr int kWide = kBytes % 16 == 0 ? 4 : kBytes % 8 == 0 ? 2 : 1;
          using Word = std::conditional_t<kWide == 4, uint4, std::conditional_t<kWide == 2, uint2, uint32_t>>;
          const Word* from = reinterpret_cast<const Word*>(row + lane * NV);
#pragma unroll
          for (int i = 0; i < kWords / kWide; ++i) {
            const Word x = from[i];
            if constexpr (kWide == 4) {
              w[4 * i] = x.x; w[4 * i + 1] = x.y; w[4 * i + 2] = x.z; w[4 * i + 3] = x.w;
            } else if constexpr (kWide == 2) {
              w[2 * i] = x.x; w[2 * i + 1] = x.y;
            } else {
              w[i] = x;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < kWords; ++i) w[i] = sizeof(T) == 4 ? fill : fill | fill << 16;
        }
        return;
      }
    }
    if constexpr (sizeof(T) == 4) {
      const uint32_t* from = reinterpret_cast<const uint32_t*>(row) + lane;
#pragma unroll
      for (int i = 0; i < NV; ++i) w[i] = lane + 32 * i < E ? from[32 * i] : fill;
    } else {
      const uint16_t* from = reinterpret_cast<const uint16_t*>(row) + lane;
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const uint32_t lo = lane + 64 * i < E ? from[64 * i] : fill;
        const uint32_t hi = 2 * i + 1 < NV && lane + 64 * i + 32 < E ? from[64 * i + 32] : fill;
        w[i] = lo | hi << 16;
      }
    }
  }
  __device__ __forceinline__ Vec<NV> values() const {
    Vec<NV> v;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (sizeof(T) == 4) v.v[i] = __uint_as_float(w[i]);
      else v.v[i] = __uint_as_float((i & 1) ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    return v;
  }
};
template <int NV, typename T>
__device__ __forceinline__ void store_values(T* row, int E, bool vec, const Vec<NV>& v) {
  if (vec) {
    store_row<NV>(row, (int)(threadIdx.x & 31) * NV, E, true, v.v);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = element<NV>(false, i);
      if (e < E) store(row + e, v.v[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ constexpr uint32_t minus_infinity() { return sizeof(T) == 4 ? 0xff800000u : 0xff80u; }

// The scores of a row first come straight from its logits, without their maximum: e^l, or sigmoid(l);
// masked ones, and what lies past the row's end, are 0. A sum of them in these bounds says that none
// overflowed, that what underflowed is below 1e-32 of it, and that no softmax logit was NaN or +inf.
// Any other row is read again as the rule says: NaN masks, +inf is the largest finite value, softmax
// scores relative to the largest logit; and sigmoid scores too where all are tiny: there each is
// e^l to 32 bits. So is a row whose log sum e^l is wanted and lies near 0, where its digits cancel.
__device__ __forceinline__ bool plain_sum(float z) { return z > 1e-6f && z < 1e30f; }
__device__ __forceinline__ bool near_one(float z) { return z > 0.5f && z < 2.f; }
constexpr float kTiny = 1e-20f;

template <int NV>
__device__ __forceinline__ void clean_row(Vec<NV>& l) {
#pragma unroll
  for (int i = 0; i < NV; ++i) l.v[i] = clean(l.v[i]);
}

// The scores of any row over their sum (0 where all is masked) added to p; log sum e^l squared.
template <int NV, bool SIGMOID>
__device__ __noinline__ Vec<NV> careful_scores(Vec<NV> l, Vec<NV> p, bool scores, float* lse_squared) {
  clean_row(l);
  const float m = row_max(l);
  if (m == -INFINITY) return p;
  Vec<NV> s = exp_below(l, m);
  float z = warp_sum(s.sum());
  const float lse = m + logf(z);
  *lse_squared += lse * lse;
  if (!scores) return p;
  if (SIGMOID && m > -17.f) {
#pragma unroll
    for (int i = 0; i < NV; ++i) s.v[i] = sigmoid(l.v[i]);
    z = warp_sum(s.sum());
  }
  return fma(s, Vec<NV>::all(1.f / z), p);
}

// e^-l, at most e^88, whose sigmoid is 0: that of masked logits.
template <int NV>
__device__ __forceinline__ Vec<NV> exp_minus(const Vec<NV>& l) {
  Vec<NV> x;
#pragma unroll
  for (int i = 0; i < NV; ++i) x.v[i] = fminf(-l.v[i], 88.f);
  return exp_vec(x);
}

// Adds a row's scores over their sum to p, and its log sum e^l squared to sum_z.
template <int NV, bool SIGMOID>
__device__ __forceinline__ void add_row(const Args& q, const Vec<NV>& l, Vec<NV>& p, float& sum_z) {
  Vec<NV> s;
  if constexpr (SIGMOID) {
    s = exp_minus(l);
#pragma unroll
    for (int i = 0; i < NV; ++i) s.v[i] = inverse(1.f + s.v[i]);
  } else {
    s = exp_vec(l);
  }
  const float z = warp_sum(s.sum());
  const bool plain = SIGMOID ? z > kTiny && z < 1e30f : plain_sum(z) && !(q.z > 0.f && near_one(z));
  if (plain) {
    p = fma(s, Vec<NV>::all(inverse(z)), p);
    const float lse = SIGMOID ? 0.f : __logf(z);   // to 3 ulp
    sum_z = fmaf(lse, lse, sum_z);
  }
  if (!plain || (SIGMOID && q.z > 0.f)) {
    float more = 0.f;
    p = careful_scores<NV, SIGMOID>(l, p, !plain, &more);
    sum_z += more;
  }
}

// Scores summed per expert times the experts' counts, over the warp.
template <int NV>
__device__ __forceinline__ float counted(const Args& q, const Vec<NV>& p, const int32_t* counts) {
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = element<NV>(q.vec, i);
    if (e < q.E) t = fmaf(p.v[i], (float)counts[e], t);
  }
  return warp_sum(t);
}

// Few rows in one sequence: one launch of one cluster. Every CTA counts all choices by itself and takes
// its share of the rows; the cluster's sums meet in distributed shared memory.
template <int NV, bool SIGMOID, typename LT>
__global__ void __launch_bounds__(32 * kSmallWarps) small_loss_kernel(const Args q, const LT* logits) {
  __shared__ int32_t hist[512];
  __shared__ float2 s[kSmallWarps], mine;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)blockIdx.x, first = rank * kSmallWarps + warp;
  RawRow<NV, LT> next;
  auto load = [&](int t) { next.load(logits + (size_t)t * q.E, q.E, q.vec, minus_infinity<LT>()); };
  if (first < q.T) load(first);
  for (int e = threadIdx.x; e < 512; e += 32 * kSmallWarps) hist[e] = 0;
  __syncthreads();
#pragma unroll 4
  for (int i = threadIdx.x; i < q.T * q.k; i += 32 * kSmallWarps) {
    const int e = q.idx[i];
    if (e >= 0 && e < q.E) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = rank + kSmallCtas * threadIdx.x; e < q.E; e += kSmallCtas * 32 * kSmallWarps)
    q.counts[e] = q.seq_counts[e] = hist[e];
  float sum_z = 0.f;
  Vec<NV> p = Vec<NV>::all(0.f);
  for (int t = first; t < q.T; t += kSmallCtas * kSmallWarps) {
    const Vec<NV> l = next.values();
    if (t + kSmallCtas * kSmallWarps < q.T) load(t + kSmallCtas * kSmallWarps);
    add_row<NV, SIGMOID>(q, l, p, sum_z);
  }
  const float sum = q.coef / ((float)q.T * (float)q.T) * counted(q, p, hist);
  if (lane == 0) s[warp] = make_float2(sum, sum_z);
  __syncthreads();
  if (warp == 0) {
    const float2 v = lane < kSmallWarps ? s[lane] : make_float2(0.f, 0.f), t = warp_sum2(v.x, v.y);
    if (lane == 0) mine = t;
  }
  cluster_sync_all();
  if (rank == 0 && warp == 0) {
    float2 v = make_float2(0.f, 0.f);
    if (lane < kSmallCtas) {
      const uint32_t at = mapa_rank(&mine, lane);
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    }
    v = warp_sum2(v.x, v.y);
    if (lane == 0) {
      q.losses[0] = v.x;
      q.losses[1] = q.z > 0.f ? v.y / (float)q.T * q.z : 0.f;
    }
  }
  cluster_sync_all();   // nobody leaves while its sums are read
}

// A warp a row at a time, rows a CTA apart. Bound by instruction issue (170 a row of 384 bf16, 63% of
// the slots). With the counts: 65536 rows of 384 bf16, softmax and z, 21.4 us (2.4 TB/s), 16384 of 256
// fp32 sigmoid in one sequence 10.5 us.
template <int NV, bool SIGMOID, typename LT>
__global__ void __launch_bounds__(32 * kWarps, kLossCtas) loss_kernel(const Args q, const LT* logits) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  RawRow<NV, LT> next;
  const LT* row = logits + (size_t)(first + warp) * q.E;
  auto load_next = [&] { next.load(row, q.E, q.vec, minus_infinity<LT>()); };
  if (first + warp < end) load_next();
  Sequence seq(q);
  float sum = 0.f, sum_z = 0.f;
  Vec<NV> p = Vec<NV>::all(0.f);
  for (int left = end - (int)first - warp; left > 0; left -= kWarps) {
    const int t = end - left;
    const Vec<NV> l = next.values();
    row += (size_t)kWarps * q.E;
    if (left > kWarps) load_next();
    if (seq.ends_before(t)) {
      if (seq.live) {
        wait_prerequisites();
        sum = fmaf(seq.factor, counted(q, p, q.seq_counts + (size_t)seq.s * q.E), sum);
      }
      p = Vec<NV>::all(0.f);
      seq.move_to(q, t);
    }
    if (seq.live) add_row<NV, SIGMOID>(q, l, p, sum_z);
  }
  wait_prerequisites();
  if (q.groups > 1) {   // all rows are one sequence, counted in parts
    __shared__ int32_t all[512];
    for (int e = threadIdx.x; e < q.E; e += 32 * kWarps) {
      int n = 0;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) n += g < q.groups ? q.group_counts[g * q.E + e] : 0;
      all[e] = n;
      if (blockIdx.x == 0) q.seq_counts[e] = q.counts[e] = n;
    }
    __syncthreads();
    sum = seq.factor * counted(q, p, all);
  } else {
    if (seq.live) sum = fmaf(seq.factor, counted(q, p, q.seq_counts + (size_t)seq.s * q.E), sum);
    // with several sequences, this CTA's share of them into the counts of all
    for (int s = blockIdx.x; q.S > 1 && s < q.S; s += gridDim.x) {
      for (int e = threadIdx.x; e < q.E; e += 32 * kWarps) {
        const int c = q.seq_counts[(size_t)s * q.E + e];
        if (c) atomicAdd(&q.counts[e], c);   // integers: any order, one result
      }
    }
  }
  // The sums of a CTA, then of all by the last CTA to arrive, in a fixed order. Positive terms, a few
  // after one another: fp32 keeps them to some ulp.
  __shared__ float2 s[kWarps];
  __shared__ bool last;
  auto cta_sum = [&](float2 v) {
    if (lane == 0) s[warp] = v;
    __syncthreads();
    const float2 t = lane < kWarps ? s[lane] : make_float2(0.f, 0.f);
    return warp_sum2(t.x, t.y);
  };
  float2 t = cta_sum(make_float2(sum, sum_z));
  if (threadIdx.x == 0) {
    q.part[blockIdx.x] = t;
    __threadfence();
    last = atomicAdd(q.ticket, 1u) + 1 == gridDim.x;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  t = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < (int)gridDim.x; i += 32 * kWarps) {
    const float2 v = __ldcg(&q.part[i]);
    t.x += v.x;
    t.y += v.y;
  }
  t = cta_sum(warp_sum2(t.x, t.y));
  if (threadIdx.x == 0) {
    q.losses[0] = t.x;
    q.losses[1] = seq.valid > 0 && q.z > 0.f ? t.y / (float)seq.valid * q.z : 0.f;
  }
}

// e = e^-l; p = 1 / (1 + e); the sums of p and p u.
template <int NV>
__device__ __forceinline__ float2 sigmoids(const Vec<NV>& l, const Vec<NV>& u, Vec<NV>& e, Vec<NV>& p) {
  e = exp_minus(l);
#pragma unroll
  for (int i = 0; i < NV; ++i) p.v[i] = inverse(1.f + e.v[i]);
  return warp_sum2(p.sum(), dot(p, u));
}
// d + sigmoid (1 - sigmoid) / sum (u - p.u) = d + (e^-l p) (p / sum) (u - p.u)
template <int NV>
__device__ __forceinline__ Vec<NV> sigmoid_gradient(const Vec<NV>& d, const Vec<NV>& u, const Vec<NV>& e,
                                                    const Vec<NV>& p, float2 w) {
  const float inv = inverse(w.x);
  return fma((e * p) * (p * Vec<NV>::all(inv)), u + Vec<NV>::all(-w.y * inv), d);
}

// d plus a row's gradient, for any row: that of the loss where `loss`, and fz lse softmax.
template <int NV, bool SIGMOID>
__device__ __noinline__ Vec<NV> careful_gradient(Vec<NV> l, Vec<NV> u, Vec<NV> d, float fz, bool loss) {
  clean_row(l);
  const float m = row_max(l);
  if (m == -INFINITY) return d;
  bool relative = loss;
  if (SIGMOID && loss && m > -17.f) {
    Vec<NV> e, p;
    const float2 w = sigmoids(l, u, e, p);
    d = sigmoid_gradient(d, u, e, p, w);
    relative = false;
  }
  if (relative || fz != 0.f) {
    const Vec<NV> p = exp_below(l, m);
    const float2 w = warp_sum2(p.sum(), dot(p, u));
    const float inv = 1.f / w.x, shift = fz != 0.f ? fz * (m + logf(w.x)) : 0.f;
    const Vec<NV> scores = p * Vec<NV>::all(inv);
    d = relative ? fma(scores, u + Vec<NV>::all(shift - w.y * inv), d)
                 : fma(scores, Vec<NV>::all(shift), d);
  }
  return d;
}

// softmax  p_e (u_e - p.u + 2 z / Tv lse);  sigmoid  p_e (1 - s_e) (u_e - p.u), the penalty apart
// Bound by instruction issue (219 a row of 384 bf16 with z, 63% of the slots): 65536 of those 20.9 us
// (4.8 TB/s), 16384 rows of 256 fp32, sigmoid, 7.7 us (4.4 TB/s).
template <int NV, bool SIGMOID, typename LT, typename DT>
__global__ void __launch_bounds__(32 * kWarps, kBwdCtas<NV, SIGMOID>)
    balance_bwd_kernel(const Args q, const LT* logits, const DT* add, DT* dlogits) {
  const int warp = threadIdx.x >> 5;
  const long long first = (long long)blockIdx.x * q.rows;
  const int end = (int)min(first + q.rows, (long long)q.T);
  RawRow<NV, LT> next;
  RawRow<NV, DT> next_add;
  size_t at = (size_t)(first + warp) * q.E;
  auto load_next = [&] {
    next.load(logits + at, q.E, q.vec, minus_infinity<LT>());
    if (add) next_add.load(add + at, q.E, q.vec, 0u);
  };
  if (first + warp < end) load_next();
  const float d0 = q.dlosses ? q.dlosses[0] : 1.f, d1 = q.dlosses ? q.dlosses[1] : 1.f;
  Sequence seq(q);
  const float fz = q.z > 0.f && seq.valid > 0 ? 2.f * q.z / (float)seq.valid * d1 : 0.f;
  Vec<NV> u;
  for (int left = end - (int)first - warp; left > 0; left -= kWarps) {
    const int t = end - left;
    const Vec<NV> l = next.values();
    Vec<NV> d = add ? next_add.values() : Vec<NV>::all(0.f);
    DT* to = dlogits + at;
    at += (size_t)kWarps * q.E;
    if (left > kWarps) load_next();
    if (seq.move_to(q, t)) {
      // counts relative to their mean, an integer: sum_e p_e = 1, so the gradient is the same,
      // without the cancellation of nearly even counts
      int32_t c[NV];
      load_counts<NV>(q.seq_counts + (size_t)seq.s * q.E, q.E, q.vec, c);
      long long total = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) total += c[i];
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(kAll, total, off);
      const int mean = (int)(total / q.E);
#pragma unroll
      for (int i = 0; i < NV; ++i) u.v[i] = (float)(c[i] - mean) * (seq.factor * d0);
    }
    if (seq.live) {
      bool plain;
      if constexpr (SIGMOID) {
        Vec<NV> e, p;
        const float2 w = sigmoids(l, u, e, p);
        plain = w.x > kTiny && w.x < 1e30f;
        if (plain) d = sigmoid_gradient(d, u, e, p, w);
      } else {
        const Vec<NV> p = exp_vec(l);
        const float2 w = warp_sum2(p.sum(), dot(p, u));
        plain = plain_sum(w.x) && !(fz != 0.f && near_one(w.x));
        if (plain) {
          const float inv = inverse(w.x), shift = fz * __logf(w.x);   // fz 0: w.x is finite
          d = fma(p * Vec<NV>::all(inv), u + Vec<NV>::all(shift - w.y * inv), d);
        }
      }
      if (!plain || (SIGMOID && fz != 0.f)) d = careful_gradient<NV, SIGMOID>(l, u, d, fz, !plain);
    }
    store_values<NV>(to, q.E, q.vec, d);
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
  return true;
}
// Rows per CTA: whole rounds of its warps, one wave of `ctas` CTAs a SM at most.
int cta_rows(int T, int ctas) {
  const long long per = ((long long)T + kSms * ctas - 1) / (kSms * ctas);
  return (int)std::max<long long>((per + kWarps - 1) / kWarps * kWarps, kWarps);
}
size_t counts_bytes(const mok_balance* r, int S) { return align_up((size_t)S * r->E * 4, 256); }

}  // namespace
}  // namespace mok

extern "C" mok_status mok_balance_get_sizes(const mok_balance* rule, int T, int S,
                                            size_t* saved_bytes) {
  using namespace mok;
  Args q;
  if (!make_args(rule, T, S, &q) || !saved_bytes) return MOK_ERR_INVALID_ARG;
  *saved_bytes = counts_bytes(rule, S) + kParts * sizeof(float2) + 256 + (size_t)kGroups * rule->E * 4;
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
  q.part = reinterpret_cast<float2*>(static_cast<char*>(saved) + counts_bytes(rule, S));
  q.ticket = reinterpret_cast<unsigned*>(q.part + kParts);
  q.group_counts = reinterpret_cast<int32_t*>(q.ticket + 64);
  q.vec = rows_vectorize(q.E, logits, logits_type);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto by_score = [&](auto f) {   // f(score is a sigmoid, the logits)
    const auto* lb = static_cast<const __nv_bfloat16*>(logits);
    const auto* lf = static_cast<const float*>(logits);
    const bool sg = rule->score == MOK_SCORE_SIGMOID, b = logits_type == MOK_OUT_BF16;
    if (sg && b) f(std::true_type{}, lb);
    else if (sg) f(std::true_type{}, lf);
    else if (b) f(std::false_type{}, lb);
    else f(std::false_type{}, lf);
  };
  cudaError_t e = cudaSuccess;
  // One launch against two, top-8 fp32, us: 128 x 256 6.3 and 8.4, 1024 x 256 9.0 and 9.6, 2048 x 256
  // 12.6 and 10.5, 1024 x 512 12.7 and 10.6.
  if (!seqs && T > 0 && T <= kSmallRows && T * q.k <= kSmallIds && T * q.E <= kSmallScores) {
    by_width(q.E, [&](auto nv) {
      by_score([&](auto sg, const auto* l) {
        using LT = std::remove_const_t<std::remove_pointer_t<decltype(l)>>;
        e = launch(small_loss_kernel<decltype(nv)::value, decltype(sg)::value, LT>, dim3(kSmallCtas),
                   dim3(32 * kSmallWarps), 0, kSmallCtas, false, s, q, l);
      });
    });
    return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
  }
  // A sequence's CTAs: eight, but one where sequences are short or many; and several clusters for a
  // long batch without offsets, 32 K ids each (65536 rows of 8: 10.6 us by one cluster, 6.8 by 16).
  const long long ids = (long long)T / S * q.k;
  const int ctas = ids >= 4096 && S <= 4096 ? 8 : 1;
  q.groups = seqs ? 1 : (int)std::max(1ll, std::min<long long>(kGroups, ids >> 15));
  // Few threads, so that the rows' kernel has room beside them. Forward with 1024 a CTA and now, us: 16384
  // rows of 256 in one sequence 11.3 and 9.9, in 512 16.6 and 12.7. Clusters keep 512, as sequences
  // differ (24 of 16384 rows, forward and backward: 22.3, with 256 22.4, 128 24.0, 1024 23.5).
  const long long share = ids / ctas;
  const unsigned threads = ctas > 1 || share >= 2048 ? kCountThreads : share >= 1024 ? 256 : 128;
  e = launch(count_kernel, dim3((unsigned)(S * q.groups) * ctas), dim3(threads), 0, ctas, false, s, q, ctas);
  if (e != cudaSuccess) return MOK_ERR_CUDA;
  if (T > 0) {
    q.rows = cta_rows(T, kLossCtas);
    const unsigned parts = ((unsigned)T + q.rows - 1) / q.rows;
    by_width(q.E, [&](auto nv) {
      by_score([&](auto sg, const auto* l) {
        using LT = std::remove_const_t<std::remove_pointer_t<decltype(l)>>;
        e = launch(loss_kernel<decltype(nv)::value, decltype(sg)::value, LT>, dim3(parts), dim3(32 * kWarps),
                   0, 1, true, s, q, l);
      });
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
  // one placement of a row's elements for all its tensors
  q.vec = q.vec && rows_vectorize(q.E, dlogits, dlogits_type) &&
          (!add || rows_vectorize(q.E, add, dlogits_type));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  by_width(q.E, [&](auto nv) {
    constexpr int NV = decltype(nv)::value;
    const bool sg = rule->score == MOK_SCORE_SIGMOID;
    q.rows = cta_rows(T, sg ? kBwdCtas<NV, true> : kBwdCtas<NV, false>);
    const unsigned ctas = ((unsigned)T + q.rows - 1) / q.rows;
    auto go = [&](auto lt, auto dt) {
      using LT = decltype(lt);
      using DT = decltype(dt);
      e = launch(sg ? balance_bwd_kernel<NV, true, LT, DT> : balance_bwd_kernel<NV, false, LT, DT>, dim3(ctas),
                 dim3(32 * kWarps), 0, 1, false, s, q, static_cast<const LT*>(logits),
                 static_cast<const DT*>(add), static_cast<DT*>(dlogits));
    };
    const bool lb = logits_type == MOK_OUT_BF16, db = dlogits_type == MOK_OUT_BF16;
    if (lb && db) go(__nv_bfloat16{}, __nv_bfloat16{});
    else if (lb) go(__nv_bfloat16{}, 0.f);
    else if (db) go(0.f, __nv_bfloat16{});
    else go(0.f, 0.f);
  });
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
