// Layer norm and RMS norm of rows, with the residual sum in front, and their gradients
// (include/mok_ops.h, mok_norm_fwd and mok_norm_bwd).
//
//   h = x + add;  xh = (h - m) r;  y = xh w + b
//   dX = r (t - [mean t] - xh mean(t xh)) + add,  t = dY w;   dW = sum dY xh,  dB = sum dY
#include "mok_internal.h"
#include "mok_ops.h"
#include "mok_rows.cuh"

namespace mok {
namespace {

constexpr int kMaxH = 32768;

struct NormArgs {
  int T, H;
  float eps;
  bool rms, w_bf16;
  const void *x, *add, *w, *b;   // the backward: dY and h in place of x, add the gradient's
  const void* dy;
  void *h, *y;                   // the backward: dX in place of y
  float2* stats;
  float2* part;                  // [chunks][H] (dW, dB)
  void *dw, *db;
  int chunks;
};

// V consecutive elements from element i of a tensor (V = 8: 16-byte accesses)
template <int V, typename E>
__device__ __forceinline__ void get(const void* p, size_t i, float* v) {
  if constexpr (V == 8) load8(static_cast<const E*>(p) + i, v);
  else v[0] = load(static_cast<const E*>(p) + i);
}
template <int V, typename E>
__device__ __forceinline__ void put(void* p, size_t i, const float* v) {
  if constexpr (V == 8) store8(static_cast<E*>(p) + i, v);
  else store(static_cast<E*>(p) + i, v[0]);
}
template <int V>
__device__ __forceinline__ void get_w(const NormArgs& q, const void* p, size_t i, float* v) {
  if (q.w_bf16) get<V, __nv_bfloat16>(p, i, v);
  else get<V, float>(p, i, v);
}

// Sums of a and b over the threads of a row: a warp (one row per warp), or the whole CTA.
__device__ __forceinline__ float2 row_sum(float a, float b) {
  a = warp_sum(a);
  b = warp_sum(b);
  if (blockDim.x == 32) return make_float2(a, b);
  __shared__ float2 s[32];
  const int warps = blockDim.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  float2 t = make_float2(0.f, 0.f);
  for (int i = 0; i < warps; ++i) {
    t.x += s[i].x;
    t.y += s[i].y;
  }
  return t;
}

// One row per blockDim.x threads; thread i holds the accesses i, i + blockDim.x, ... of the row.
template <int N, int V, typename X, typename Y>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const NormArgs q) {
  const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= (size_t)q.T) return;
  const size_t at = row * q.H;
  float v[N][V];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) v[i][j] = 0.f;
    if (c < q.H) {
      get<V, X>(q.x, at + c, v[i]);
      if (q.add) {
        float a[V];
        get<V, X>(q.add, at + c, a);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          v[i][j] += a[j];
          if constexpr (sizeof(X) == 2) v[i][j] = __bfloat162float(__float2bfloat16_rn(v[i][j]));
        }
        put<V, X>(q.h, at + c, v[i]);
      }
#pragma unroll
      for (int j = 0; j < V; ++j) sum += v[i][j];
    }
  }
  const float inv_h = 1.f / (float)q.H;
  const float mean = q.rms ? 0.f : row_sum(sum, 0.f).x * inv_h;
  float sq = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < q.H) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        v[i][j] -= mean;
        sq += v[i][j] * v[i][j];
      }
    }
  }
  const float r = 1.f / sqrtf(row_sum(sq, 0.f).x * inv_h + q.eps);
  if (q.stats && threadIdx.x == 0) q.stats[row] = make_float2(mean, r);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < q.H) {
      float w[V], b[V];
      get_w<V>(q, q.w, c, w);
      if (q.b) get_w<V>(q, q.b, c, b);
#pragma unroll
      for (int j = 0; j < V; ++j) v[i][j] = v[i][j] * r * w[j] + (q.b ? b[j] : 0.f);
      put<V, Y>(q.y, at + c, v[i]);
    }
  }
}

template <int N, int V, typename X, typename Y>
__global__ void __launch_bounds__(1024) norm_dx_kernel(const NormArgs q) {
  const size_t row = (size_t)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= (size_t)q.T) return;
  const size_t at = row * q.H;
  const float2 st = q.stats[row];
  float t[N][V], xh[N][V];
  float s1 = 0.f, s2 = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < q.H) {
      float w[V];
      get<V, Y>(q.dy, at + c, t[i]);
      get<V, X>(q.x, at + c, xh[i]);
      get_w<V>(q, q.w, c, w);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        t[i][j] *= w[j];
        xh[i][j] = (xh[i][j] - st.x) * st.y;
        s1 += t[i][j];
        s2 += t[i][j] * xh[i][j];
      }
    }
  }
  float2 s = row_sum(s1, s2);
  const float inv_h = 1.f / (float)q.H;
  s.x = q.rms ? 0.f : s.x * inv_h;
  s.y *= inv_h;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = (i * blockDim.x + threadIdx.x) * V;
    if (c < q.H) {
      float a[V];
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] = 0.f;
      if (q.add) get<V, X>(q.add, at + c, a);
#pragma unroll
      for (int j = 0; j < V; ++j) a[j] += st.y * (t[i][j] - s.x - xh[i][j] * s.y);
      put<V, X>(q.y, at + c, a);
    }
  }
}

// dW and dB over a chunk of rows: a CTA holds 32 columns and 8 rows at a time.
template <typename X, typename Y>
__global__ void norm_dw_kernel(const NormArgs q) {
  const int c = blockIdx.x * 32 + threadIdx.x;
  const size_t per = ((size_t)q.T + q.chunks - 1) / q.chunks;
  const size_t r0 = blockIdx.y * per, r1 = min(r0 + per, (size_t)q.T);
  float dw = 0.f, db = 0.f;
  if (c < q.H) {
    for (size_t r = r0 + threadIdx.y; r < r1; r += 8) {
      const float2 st = q.stats[r];
      const float dy = load(static_cast<const Y*>(q.dy) + r * q.H + c);
      dw += dy * ((load(static_cast<const X*>(q.x) + r * q.H + c) - st.x) * st.y);
      db += dy;
    }
  }
  __shared__ float2 s[8][32];
  s[threadIdx.y][threadIdx.x] = make_float2(dw, db);
  __syncthreads();
  if (threadIdx.y == 0 && c < q.H) {
    float2 t = make_float2(0.f, 0.f);
    for (int i = 0; i < 8; ++i) {
      t.x += s[i][threadIdx.x].x;
      t.y += s[i][threadIdx.x].y;
    }
    q.part[(size_t)blockIdx.y * q.H + c] = t;
  }
}

__global__ void norm_dw_sum_kernel(const NormArgs q) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= q.H) return;
  float2 t = make_float2(0.f, 0.f);
  for (int i = 0; i < q.chunks; ++i) {
    const float2 p = q.part[(size_t)i * q.H + c];
    t.x += p.x;
    t.y += p.y;
  }
  if (q.w_bf16) {
    store(static_cast<__nv_bfloat16*>(q.dw) + c, t.x);
    if (q.db) store(static_cast<__nv_bfloat16*>(q.db) + c, t.y);
  } else {
    store(static_cast<float*>(q.dw) + c, t.x);
    if (q.db) store(static_cast<float*>(q.db) + c, t.y);
  }
}

bool check(const mok_norm_dims* d) {
  return d && d->T >= 0 && d->H >= 1 && d->H <= kMaxH &&
         (d->kind == MOK_NORM_LAYER || d->kind == MOK_NORM_RMS) && std::isfinite(d->eps) &&
         d->eps >= 0.f && is_type(d->x_type) && is_type(d->y_type) && is_type(d->w_type);
}
uintptr_t size_of(mok_out_dtype t) { return t == MOK_OUT_BF16 ? 2 : 4; }
bool whole(const void* p) { return aligned_to(p, 16); }

// Chunks of rows whose sums of dW and dB are kept apart.
int row_chunks(int T) { return std::max(1, std::min(64, T / 16)); }

template <int N, int V, typename F>
void by_types(const mok_norm_dims* d, F f) {
  using B = __nv_bfloat16;
  constexpr auto n = std::integral_constant<int, N>{};
  constexpr auto v = std::integral_constant<int, V>{};
  if (d->x_type == MOK_OUT_BF16 && d->y_type == MOK_OUT_BF16) f(n, v, B{}, B{});
  else if (d->x_type == MOK_OUT_BF16) f(n, v, B{}, 0.f);
  else if (d->y_type == MOK_OUT_BF16) f(n, v, 0.f, B{});
  else f(n, v, 0.f, 0.f);
}
// Accesses per thread, elements per access.
template <typename F>
void by_width(const mok_norm_dims* d, bool vec, F f) {
  if (vec) {
    if (d->H <= 8 * 32) by_types<1, 8>(d, f);
    else by_types<4, 8>(d, f);
  } else {
    if (d->H <= 4096) by_types<4, 1>(d, f);
    else by_types<32, 1>(d, f);
  }
}

}  // namespace
}  // namespace mok

extern "C" mok_status mok_norm_get_sizes(const mok_norm_dims* d, mok_norm_sizes* out) {
  using namespace mok;
  if (!check(d) || !out) return MOK_ERR_INVALID_ARG;
  out->stats_bytes = (size_t)d->T * sizeof(float2);
  out->workspace_bytes = align_up((size_t)row_chunks(d->T) * d->H * sizeof(float2), 256);
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
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_width(d, vec, [&](auto n, auto v, auto xt, auto yt) {
    constexpr int per = decltype(n)::value * decltype(v)::value;
    const unsigned bx = ((d->H + per - 1) / per + 31) / 32 * 32, by = bx == 32 ? 8 : 1;
    norm_fwd_kernel<decltype(n)::value, decltype(v)::value, decltype(xt), decltype(yt)>
        <<<((unsigned)d->T + by - 1) / by, dim3(bx, by), 0, s>>>(q);
  });
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
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
  q.part = static_cast<float2*>(workspace);
  q.chunks = d->T ? row_chunks(d->T) : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (d->T) {
    const bool vec = d->H % 8 == 0 && whole(dY) && whole(h) && whole(w) && whole(add) && whole(dX);
    by_width(d, vec, [&](auto n, auto v, auto xt, auto yt) {
      constexpr int per = decltype(n)::value * decltype(v)::value;
      const unsigned bx = ((d->H + per - 1) / per + 31) / 32 * 32, by = bx == 32 ? 8 : 1;
      norm_dx_kernel<decltype(n)::value, decltype(v)::value, decltype(xt), decltype(yt)>
          <<<((unsigned)d->T + by - 1) / by, dim3(bx, by), 0, s>>>(q);
    });
    by_types<1, 1>(d, [&](auto, auto, auto xt, auto yt) {
      norm_dw_kernel<decltype(xt), decltype(yt)>
          <<<dim3((d->H + 31) / 32, q.chunks), dim3(32, 8), 0, s>>>(q);
    });
  }
  norm_dw_sum_kernel<<<(d->H + 255) / 256, 256, 0, s>>>(q);
  return cudaGetLastError() == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}
