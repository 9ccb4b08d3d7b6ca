// Layer norm and RMS norm of rows, with the residual sum in front, and their gradients
// (include/mok_ops.h, mok_norm_fwd and mok_norm_bwd).
//
//   h = x + add;  xh = (h - m) r;  y = xh w + b
//   dX = r (t - [mean t] - xh mean(t xh)) + add,  t = dY w;   dW = sum dY xh,  dB = sum dY
//
// Bound by memory. A team of threads, from a warp (H <= 1024) to a whole CTA, goes through rows
// a grid apart, so that a thread keeps the same columns throughout: dW and dB stay in its registers
// and leave as one partial row per CTA, which a second, overlapped kernel sums up. Each thread
// copies its own part of the next row to shared memory (cp.async: asynchronous, and nobody else
// reads it, so there is no barrier and no wait on another thread) while the team reduces this one.
#include <climits>

#include "mok_internal.h"
#include "mok_launch.cuh"
#include "mok_ops.h"
#include "mok_ptx.cuh"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kMaxH = 32768;
constexpr int kSms = 152;
constexpr int kMaxParts = kSms * 4;    // partial rows of dW and dB
constexpr int kRingBytes = 220 * 1024; // shared memory of an SM for rows in flight

struct NormArgs {
  int T, H;
  float eps;
  bool rms, w_bf16;
  int stages;                    // rows in flight per team; 0: no ring
  const void *x, *add, *w, *b;   // the backward: h in place of x, add the gradient's
  const void* dy;
  void *h, *y;                   // the backward: dX in place of y
  float2* stats;
  float *part_w, *part_b;        // [parts][H]
  void *dw, *db;
  int parts;
};

// V consecutive elements of a tensor or of shared memory
template <int V, typename E>
__device__ __forceinline__ void get(const E* p, float* v) {
  if constexpr (V == 8) {
    load8(p, v);
  } else if constexpr (V == 4 && sizeof(E) == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
  } else if constexpr (V == 4) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
  } else {
    v[0] = load(p);
  }
}
template <int V, typename E>
__device__ __forceinline__ void put(E* p, const float* v) {
  if constexpr (V == 8) {
    store8(p, v);
  } else if constexpr (V == 4 && sizeof(E) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (V == 4) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    store(p, v[0]);
  }
}
template <int V>
__device__ __forceinline__ void get_w(const NormArgs& q, const void* p, int c, float* v) {
  if (q.w_bf16) get<V>(static_cast<const __nv_bfloat16*>(p) + c, v);
  else get<V>(static_cast<const float*>(p) + c, v);
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// At most the newest `n` (0 or 1) groups still in flight.
__device__ __forceinline__ void copies_wait(int n) {
  if (n) asm volatile("cp.async.wait_group 1;" ::: "memory");
  else asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// Sums of a and b over the threads of a team. `turn` alternates between two places, so that one
// barrier a sum is enough.
__device__ __forceinline__ float2 row_sum(float a, float b, int& turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (blockDim.x == 32) return make_float2(a, b);
  __shared__ float2 s[2][32];
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31, first = threadIdx.y * warps;
  turn ^= 1;
  if (lane == 0) s[turn][first + (threadIdx.x >> 5)] = make_float2(a, b);
  if (blockDim.y == 1) __syncthreads();
  else named_bar_sync(1 + threadIdx.y, blockDim.x);   // teams differ in their rows
  const float2 t = lane < warps ? s[turn][first + lane] : make_float2(0.f, 0.f);
  return make_float2(warp_sum(t.x), warp_sum(t.y));
}

// A thread's places in shared memory: `stages` rows of K tensors, N accesses of 16 bytes.
extern __shared__ __align__(16) char ring[];
template <int N>
__device__ __forceinline__ char* slot(int stage, int K, int tensor, int i) {
  const int threads = blockDim.x * blockDim.y, me = threadIdx.y * blockDim.x + threadIdx.x;
  return ring + (size_t)(((stage * K + tensor) * N + i) * threads + me) * 16;
}
// Starts the copies of this thread's part of a row.
template <int N, int V, typename E>
__device__ __forceinline__ void fetch(const void* p, size_t row, int H, int stage, int K, int tensor) {
  const E* from = static_cast<const E*>(p) + row * H;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
    if (c < H) copy_async<V * (int)sizeof(E)>(smem_u32(slot<N>(stage, K, tensor, i)), from + c);
  }
}

// RING: V elements a copy, 16 bytes at most; else V = 1, any alignment.
template <int N, int V, typename X, typename Y, bool RING, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_fwd_kernel(const NormArgs q) {
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int K = q.add ? 2 : 1;
  const float inv_h = 1.f / (float)q.H;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        fetch<N, V, X>(q.x, r, q.H, stage, K, 0);
        if (q.add) fetch<N, V, X>(q.add, r, q.H, stage, K, 1);
      }
      copies_commit();
    }
  };
  int stage = 0, turn = 0;
  for (int s = 0; s < q.stages; ++s) start(row + s * step, s);
  for (; row < (size_t)q.T; row += step) {
    const size_t at = row * q.H;
    float v[N][V];
    float sum = 0.f;
    if constexpr (RING) copies_wait(q.stages - 1);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = 0.f;
      if (c < q.H)
        get<V>(RING ? reinterpret_cast<const X*>(slot<N>(stage, K, 0, i))
                    : static_cast<const X*>(q.x) + at + c, v[i]);
    }
    if (q.add) {
      float kept[RING ? 1 : N][V];   // without a ring: all loads before the first store
      if constexpr (!RING) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
          if (c < q.H) get<V>(static_cast<const X*>(q.add) + at + c, kept[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c < q.H) {
          float a[V];
          if constexpr (RING) get<V>(reinterpret_cast<const X*>(slot<N>(stage, K, 1, i)), a);
#pragma unroll
          for (int j = 0; j < V; ++j) {
            v[i][j] += RING ? a[j] : kept[RING ? 0 : i][j];
            // the norm is that of the stored h
            if constexpr (sizeof(X) == 2) v[i][j] = __bfloat162float(__float2bfloat16_rn(v[i][j]));
          }
          put<V>(static_cast<X*>(q.h) + at + c, v[i]);
        }
      }
    }
    start(row + q.stages * step, stage);
    if (++stage >= q.stages) stage = 0;
    float mean = 0.f;
    if (!q.rms) {
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) sum += v[i][j];
      mean = row_sum(sum, 0.f, turn).x * inv_h;
    }
    float sq = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
      if (c < q.H) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] -= mean;
          sq += v[i][j] * v[i][j];
        }
      }
    }
    const float r = 1.f / sqrtf(row_sum(sq, 0.f, turn).x * inv_h + q.eps);
    if (q.stats && threadIdx.x == 0) q.stats[row] = make_float2(mean, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
      if (c < q.H) {
        float w[V], b[V];
        get_w<V>(q, q.w, c, w);
        if (q.b) get_w<V>(q, q.b, c, b);
#pragma unroll
        for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * w[j] + (q.b ? b[j] : 0.f);
        put<V>(static_cast<Y*>(q.y) + at + c, v[i]);
      }
    }
  }
}

template <int N, int V, typename X, typename Y, bool RING, bool DB, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) norm_bwd_kernel(const NormArgs q) {
  launch_dependents();
  const size_t step = (size_t)gridDim.x * blockDim.y;
  size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int K = q.add ? 3 : 2;
  const float inv_h = 1.f / (float)q.H;
  auto start = [&](size_t r, int stage) {
    if constexpr (RING) {
      if (r < (size_t)q.T) {
        fetch<N, V, Y>(q.dy, r, q.H, stage, K, 0);
        fetch<N, V, X>(q.x, r, q.H, stage, K, 1);
        if (q.add) fetch<N, V, X>(q.add, r, q.H, stage, K, 2);
      }
      copies_commit();
    }
  };
  float acc_w[N][V], acc_b[DB ? N : 1][V];
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      acc_w[i][j] = 0.f;
      if (DB) acc_b[i][j] = 0.f;
    }
  int stage = 0, turn = 0;
  for (int s = 0; s < q.stages; ++s) start(row + s * step, s);
  float2 st = row < (size_t)q.T ? q.stats[row] : make_float2(0.f, 0.f);
  for (; row < (size_t)q.T; row += step) {
    const size_t at = row * q.H;
    const float mean = st.x, r = st.y;
    if (row + step < (size_t)q.T) st = q.stats[row + step];
    if constexpr (RING) copies_wait(q.stages - 1);
    float s1 = 0.f, s2 = 0.f;
    // what the second pass needs again: kept in registers without a ring
    float kept_t[RING ? 1 : N][V], kept_x[RING ? 1 : N][V];
    if constexpr (!RING) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c < q.H) {
          get<V>(static_cast<const Y*>(q.dy) + at + c, kept_t[i]);
          get<V>(static_cast<const X*>(q.x) + at + c, kept_x[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
      if (c < q.H) {
        float dy[V], x[V], w[V];
        if constexpr (RING) {
          get<V>(reinterpret_cast<const Y*>(slot<N>(stage, K, 0, i)), dy);
          get<V>(reinterpret_cast<const X*>(slot<N>(stage, K, 1, i)), x);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            dy[j] = kept_t[i][j];
            x[j] = kept_x[i][j];
          }
        }
        get_w<V>(q, q.w, c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (x[j] - mean) * r, t = dy[j] * w[j];
          acc_w[i][j] += dy[j] * xh;
          if (DB) acc_b[i][j] += dy[j];
          s1 += t;
          s2 += t * xh;
        }
      }
    }
    float2 s = row_sum(q.rms ? 0.f : s1, s2, turn);
    s.x *= inv_h;
    s.y *= inv_h;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
      if (c < q.H) {
        float dy[V], x[V], a[V], w[V];
        if constexpr (RING) {
          get<V>(reinterpret_cast<const Y*>(slot<N>(stage, K, 0, i)), dy);
          get<V>(reinterpret_cast<const X*>(slot<N>(stage, K, 1, i)), x);
          if (q.add) get<V>(reinterpret_cast<const X*>(slot<N>(stage, K, 2, i)), a);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            dy[j] = kept_t[i][j];
            x[j] = kept_x[i][j];
          }
          if (q.add) get<V>(static_cast<const X*>(q.add) + at + c, a);
        }
        get_w<V>(q, q.w, c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xh = (x[j] - mean) * r;
          x[j] = r * (dy[j] * w[j] - s.x - xh * s.y) + (q.add ? a[j] : 0.f);
        }
        put<V>(static_cast<X*>(q.y) + at + c, x);
      }
    }
    start(row + q.stages * step, stage);
    if (++stage >= q.stages) stage = 0;
  }
  // this CTA's partial rows: its teams' sums one after another through shared memory
  float* sum_w = reinterpret_cast<float*>(ring);
  float* sum_b = sum_w + q.H;
  if (blockDim.y > 1) {
    if constexpr (RING) copies_wait(0);
    __syncthreads();
  }
  for (int team = 0; team < (int)blockDim.y; ++team) {
    if ((int)threadIdx.y == team) {
      const bool last = team + 1 == (int)blockDim.y;
      float* to_w = last ? q.part_w + (size_t)blockIdx.x * q.H : sum_w;
      float* to_b = last ? q.part_b + (size_t)blockIdx.x * q.H : sum_b;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int c = (i * (int)blockDim.x + (int)threadIdx.x) * V;
        if (c < q.H) {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            to_w[c + j] = acc_w[i][j] + (team ? sum_w[c + j] : 0.f);
            if (DB) to_b[c + j] = acc_b[i][j] + (team ? sum_b[c + j] : 0.f);
          }
        }
      }
    }
    if (blockDim.y > 1) __syncthreads();
  }
}

// dW and dB from the partial rows: 32 columns a CTA, 16 rows at a time.
__global__ void __launch_bounds__(512) norm_dw_kernel(const NormArgs q) {
  wait_prerequisites();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float w = 0.f, b = 0.f;
  if (c < q.H) {
#pragma unroll 4
    for (int i = threadIdx.y; i < q.parts; i += 16) {
      w += q.part_w[(size_t)i * q.H + c];
      if (q.db) b += q.part_b[(size_t)i * q.H + c];
    }
  }
  __shared__ float2 s[16][32];
  s[threadIdx.y][threadIdx.x] = make_float2(w, b);
  __syncthreads();
  if (threadIdx.y || c >= q.H) return;
  w = b = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w += s[i][threadIdx.x].x;
    b += s[i][threadIdx.x].y;
  }
  if (q.w_bf16) {
    store(static_cast<__nv_bfloat16*>(q.dw) + c, w);
    if (q.db) store(static_cast<__nv_bfloat16*>(q.db) + c, b);
  } else {
    store(static_cast<float*>(q.dw) + c, w);
    if (q.db) store(static_cast<float*>(q.db) + c, b);
  }
}

bool check(const mok_norm_dims* d) {
  return d && d->T >= 0 && d->H >= 1 && d->H <= kMaxH &&
         (d->kind == MOK_NORM_LAYER || d->kind == MOK_NORM_RMS) && std::isfinite(d->eps) &&
         d->eps >= 0.f && is_type(d->x_type) && is_type(d->y_type) && is_type(d->w_type);
}
uintptr_t size_of(mok_out_dtype t) { return t == MOK_OUT_BF16 ? 2 : 4; }
bool whole(const void* p) { return aligned_to(p, 16); }


// How a call runs: teams of bx threads a row, by teams a CTA, `stages` rows of `tensors` tensors in
// flight per team.
struct Form {
  unsigned bx, by, grid;
  int stages;
  size_t smem;
};
// n accesses of v elements a thread; `threads` a SM is what the registers allow.
Form form(const mok_norm_dims* d, int n, int v, int tensors, int threads, int most_ctas) {
  Form f{};
  f.bx = ((d->H + n * v - 1) / (n * v) + 31) / 32 * 32;
  f.by = std::max(1u, 256 / f.bx);
  const size_t row = (size_t)f.bx * f.by * n * tensors * 16;
  f.stages = v == 1 ? 0 : row * 2 <= kRingBytes ? 2 : 1;
  f.smem = row * f.stages;
  int ctas = std::max(1, threads / (int)(f.bx * f.by));
  if (f.smem) ctas = std::max(1, std::min(ctas, (int)(kRingBytes / f.smem)));
  f.grid = (unsigned)std::min<size_t>(((size_t)d->T + f.by - 1) / f.by,
                                      std::min(kSms * ctas, most_ctas));
  return f;
}
// Partial rows of dW and dB at most.
int most_parts(const mok_norm_dims* d) { return std::min(d->T, d->H <= 2048 ? kMaxParts : kMaxParts / 2); }

template <typename K>
cudaError_t run(K kernel, const Form& f, const NormArgs& q, cudaStream_t s) {
  if (f.smem > 40 * 1024) {   // 48 KB with the static part
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)f.smem);
    if (e != cudaSuccess) return e;
  }
  return launch(kernel, dim3(f.grid), dim3(f.bx, f.by), f.smem, 1, false, s, q);
}

template <int N, int V, int THREADS, typename F>
cudaError_t by_types(const mok_norm_dims* d, F f) {
  using B = __nv_bfloat16;
  constexpr std::integral_constant<int, N> n{};
  constexpr std::integral_constant<int, V> v{};
  constexpr std::integral_constant<int, THREADS> t{};
  const bool xb = d->x_type == MOK_OUT_BF16, yb = d->y_type == MOK_OUT_BF16;
  if constexpr (V != 4)
    if (xb && yb) return f(n, v, t, B{}, B{});
  if constexpr (V != 8) {
    if (xb && !yb) return f(n, v, t, B{}, 0.f);
    if (yb && !xb) return f(n, v, t, 0.f, B{});
    return f(n, v, t, 0.f, 0.f);
  }
  return cudaErrorInvalidValue;
}
// f(accesses a thread, elements an access, most threads of a CTA, X, Y) for the call's types, width
// and alignment. `vec`: 32 elements a thread (8 for narrow rows) in accesses of 16 bytes of the
// widest type, through the ring; element by element where rows are not aligned, or too wide for
// it.
template <typename F>
cudaError_t by_form(const mok_norm_dims* d, bool vec, int tensors, F f) {
  const bool wide = d->x_type != MOK_OUT_BF16 || d->y_type != MOK_OUT_BF16;
  const int bx = ((d->H + 31) / 32 + 31) / 32 * 32;
  if ((size_t)bx * (wide ? 8 : 4) * tensors * 16 > kRingBytes) vec = false;
  if (!vec) {
    if (d->H <= 2048) return by_types<8, 1, 256>(d, f);
    if (d->H <= 8192) return by_types<8, 1, 1024>(d, f);
    return by_types<32, 1, 1024>(d, f);
  }
  if (wide) {
    if (d->H <= 256) return by_types<2, 4, 256>(d, f);
    if (d->H <= 8192) return by_types<8, 4, 256>(d, f);
    return by_types<8, 4, 1024>(d, f);
  }
  if (d->H <= 256) return by_types<1, 8, 256>(d, f);
  if (d->H <= 8192) return by_types<4, 8, 256>(d, f);
  return by_types<4, 8, 1024>(d, f);
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_norm_get_sizes(const mok_norm_dims* d, mok_norm_sizes* out) {
  using namespace mok;
  if (!check(d) || !out) return MOK_ERR_INVALID_ARG;
  out->stats_bytes = (size_t)d->T * sizeof(float2);
  out->workspace_bytes = align_up((size_t)most_parts(d) * d->H * sizeof(float2), 256) + 256;
  return MOK_OK;
}

extern "C" mok_status mok_norm_fwd(const mok_norm_dims* d, const void* x, const void* add,
                                   const void* w, const void* b, void* h, void* y, float* stats,
                                   void* stream) {
  using namespace mok;
  if (!check(d)) return MOK_ERR_INVALID_ARG;
  if (d->T == 0) return MOK_OK;
  if (!x || !w || !y || (add == nullptr) != (h == nullptr)) return MOK_ERR_INVALID_ARG;
  const uintptr_t xs = size_of(d->x_type), ws = size_of(d->w_type);
  if (!aligned_to(x, xs) || !aligned_to(add, xs) || !aligned_to(h, xs) || !aligned_to(w, ws) ||
      !aligned_to(b, ws) || !aligned_to(y, size_of(d->y_type)) || !aligned_to(stats, 8))
    return MOK_ERR_INVALID_ARG;
  NormArgs q{};
  q.T = d->T; q.H = d->H; q.eps = d->eps;
  q.rms = d->kind == MOK_NORM_RMS; q.w_bf16 = d->w_type == MOK_OUT_BF16;
  q.x = x; q.add = add; q.w = w; q.b = b; q.h = h; q.y = y;
  q.stats = reinterpret_cast<float2*>(stats);
  const bool vec = d->H % 8 == 0 && whole(x) && whole(add) && whole(w) && whole(b) && whole(h) &&
                   whole(y);
  const int tensors = add ? 2 : 1;
  const cudaError_t e = by_form(d, vec, tensors, [&](auto n, auto v, auto threads, auto xt, auto yt) {
    constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
    constexpr int CTAS = THREADS == 1024 ? 1 : V == 1 ? 6 : 3;
    const Form f = form(d, N, V, tensors, THREADS * CTAS, INT_MAX);
    q.stages = f.stages;
    return run(norm_fwd_kernel<N, V, decltype(xt), decltype(yt), (V > 1), THREADS, CTAS>, f, q,
               static_cast<cudaStream_t>(stream));
  });
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

extern "C" mok_status mok_norm_bwd(const mok_norm_dims* d, const void* dY, const void* h,
                                   const void* w, const float* stats, const void* add, void* dX,
                                   void* dW, void* dB, void* workspace, void* stream) {
  using namespace mok;
  if (!check(d)) return MOK_ERR_INVALID_ARG;
  const uintptr_t xs = size_of(d->x_type), ws = size_of(d->w_type);
  if (!dW || !aligned_to(dW, ws) || !aligned_to(dB, ws)) return MOK_ERR_INVALID_ARG;
  if (d->T > 0) {
    if (!dY || !h || !w || !stats || !dX) return MOK_ERR_INVALID_ARG;
    if (!aligned_to(dY, size_of(d->y_type)) || !aligned_to(h, xs) || !aligned_to(add, xs) ||
        !aligned_to(dX, xs) || !aligned_to(w, ws) || !aligned_to(stats, 8))
      return MOK_ERR_INVALID_ARG;
  }
  if (!workspace || !aligned_to(workspace, 256)) return MOK_ERR_WORKSPACE;
  NormArgs q{};
  q.T = d->T; q.H = d->H;
  q.rms = d->kind == MOK_NORM_RMS; q.w_bf16 = d->w_type == MOK_OUT_BF16;
  q.dy = dY; q.x = h; q.w = w; q.add = add; q.y = dX; q.dw = dW; q.db = dB;
  q.stats = reinterpret_cast<float2*>(const_cast<float*>(stats));
  q.part_w = static_cast<float*>(workspace);
  q.part_b = q.part_w + (size_t)most_parts(d) * d->H;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->T) {
    const bool vec = d->H % 8 == 0 && whole(dY) && whole(h) && whole(w) && whole(add) && whole(dX);
    const int tensors = add ? 3 : 2;
    const cudaError_t e = by_form(d, vec, tensors, [&](auto n, auto v, auto threads, auto xt, auto yt) {
      constexpr int N = decltype(n)::value, V = decltype(v)::value, THREADS = decltype(threads)::value;
      constexpr int CTAS = THREADS == 1024 ? 1 : V == 1 ? 3 : 2;
      Form f = form(d, N, V, tensors, THREADS * CTAS, most_parts(d));
      if (f.by > 1) f.smem = std::max(f.smem, (size_t)d->H * sizeof(float2));   // joins the teams
      q.stages = f.stages;
      q.parts = (int)f.grid;
      if (dB)
        return run(norm_bwd_kernel<N, V, decltype(xt), decltype(yt), (V > 1), true, THREADS, CTAS>, f, q, s);
      return run(norm_bwd_kernel<N, V, decltype(xt), decltype(yt), (V > 1), false, THREADS, CTAS>, f, q, s);
    });
    if (e != cudaSuccess) return MOK_ERR_CUDA;
  }
  const cudaError_t e = launch(norm_dw_kernel, dim3((d->H + 31) / 32), dim3(32, 16), 0, 1, d->T > 0, s, q);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
