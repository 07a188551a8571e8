// attn_rows.cu -- attention of one query row and head per block, on the CUDA
// cores in fp32: one pass over the keys with the running maximum and sum of
// the softmax, each of the block's warps over every eighth group of keys, and
// the warps' parts joined at the end.
#include <cuda_bf16.h>

#include <cmath>

#include "attention.h"
#include "internal.h"
#include "sm100.cuh"

namespace li {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxKey = 576, kMaxValue = 512;
constexpr int kKeys = 4;   // keys a warp takes at once

template <typename T>
__device__ __forceinline__ void load16(const T* p, float (&v)[16 / sizeof(T)]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  if constexpr (sizeof(T) == 4) {
    const float* f = reinterpret_cast<const float*>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f[e];
  } else {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __bfloat1622float2(h[e]);
      v[2 * e] = f.x;
      v[2 * e + 1] = f.y;
    }
  }
}

template <typename T>
struct KeyRow {
  const T *k1, *k2, *v;   // key in two parts, value; v null: skipped
};

// q: the query in shared memory.  rows(i) gives key i of n.  Every thread of
// the block calls it.
template <typename T, typename Rows>
__device__ __forceinline__ void attend(const float* q, int d1, int d2, int d_v, int64_t n, float scale, Rows rows, T* out,
                                       float* lse) {
  constexpr int V = 16 / sizeof(T);
  constexpr int NK = (kMaxKey / V + 31) / 32, NV = (kMaxValue / V + 31) / 32;
  __shared__ float part[kWarps][kMaxValue], pm[kWarps], pl[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c1 = d1 / V, ck = (d1 + d2) / V, cv = (d_v + V - 1) / V;
  float acc[NV][V] = {};
  float m = -INFINITY, l = 0.f;
  for (int64_t i0 = static_cast<int64_t>(warp) * kKeys; i0 < n; i0 += kWarps * kKeys) {
    KeyRow<T> mine{};
    if (lane < kKeys && i0 + lane < n) mine = rows(i0 + lane);
    KeyRow<T> r[kKeys];
    float z[kKeys];
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      r[u].k1 = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.k1), u));
      r[u].k2 = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.k2), u));
      r[u].v = reinterpret_cast<const T*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(mine.v), u));
      z[u] = 0.f;
      if (r[u].v) {
#pragma unroll
        for (int j = 0; j < NK; ++j) {
          const int c = lane + 32 * j;
          if (c < ck) {
            float k[V];
            load16<T>(c < c1 ? r[u].k1 + c * V : r[u].k2 + (c - c1) * V, k);
#pragma unroll
            for (int e = 0; e < V; ++e) z[u] = fmaf(q[c * V + e], k[e], z[u]);
          }
        }
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) z[u] += __shfl_xor_sync(0xffffffffu, z[u], o);
      z[u] = r[u].v ? z[u] * scale : -INFINITY;
      mn = fmaxf(mn, z[u]);
    }
    if (mn == -INFINITY) continue;
    const float keep = expf(m - mn);
    m = mn;
    l *= keep;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) acc[j][e] *= keep;
#pragma unroll
    for (int u = 0; u < kKeys; ++u) {
      if (!r[u].v) continue;
      const float p = expf(z[u] - m);
      l += p;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = lane + 32 * j;
        if (c < cv) {
          float v[V];
          load16<T>(r[u].v + c * V, v);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[j][e] = fmaf(p, v[e], acc[j][e]);
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e)
      if ((lane + 32 * j) * V + e < d_v) part[warp][(lane + 32 * j) * V + e] = acc[j][e];
  if (lane == 0) {
    pm[warp] = m;
    pl[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, w[kWarps];
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, pm[i]);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    w[i] = pm[i] == -INFINITY ? 0.f : expf(pm[i] - M);
    L = fmaf(w[i], pl[i], L);
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
  for (int i = threadIdx.x; i < d_v; i += kWarps * 32) {
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) s = fmaf(w[u], part[u][i], s);
    out[i] = static_cast<T>(s * inv);
  }
  if (lse && threadIdx.x == 0) *lse = L > 0.f ? M + logf(L) : -INFINITY;
}

// One block per (sequence, query, head).
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) latent_rows_kernel(const __grid_constant__ LatentAttnArgs a) {
  pdl_begin();
  __shared__ float q[kMaxKey];
  const int64_t row = blockIdx.x;              // (b * T + t) * H + h
  const int64_t bt = row / a.H;
  const int b = static_cast<int>(bt / a.T);
  for (int i = threadIdx.x; i < a.dim; i += blockDim.x) q[i] = static_cast<float>(static_cast<const T*>(a.q)[row * a.dim + i]);
  __syncthreads();
  int64_t n = min(static_cast<int64_t>(max(a.lengths[b], 0)), static_cast<int64_t>(a.max_pages) * a.page_size);
  if (a.q_pos) n = min(n, max(static_cast<int64_t>(a.q_pos[bt]) + 1, int64_t(0)));
  const int32_t* table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  const int32_t* sel = a.sel ? a.sel + bt * a.k : nullptr;
  auto rows = [&](int64_t i) {
    KeyRow<T> r{};
    const int64_t s = sel ? sel[i] : i;
    if (s < 0) return r;
    if (s >= n) {
      record_status(a.status, kStatusIndex);
      return r;
    }
    const int page = table[s / a.page_size];
    if (page < 0 || page >= a.n_pages) {
      record_status(a.status, kStatusIndex);
      return r;
    }
    r.k1 = r.v = static_cast<const T*>(a.data) + (static_cast<int64_t>(page) * a.page_size + s % a.page_size) * a.dim;
    return r;
  };
  attend<T>(q, a.dim, 0, a.d_v, sel ? a.k : n, a.scale, rows, static_cast<T*>(a.out) + row * a.d_v,
            a.lse ? a.lse + row : nullptr);
}

// One block per (sequence, query, head); queries past the sequence's end return.
template <typename T>
__global__ void __launch_bounds__(kWarps * 32) prompt_rows_kernel(const __grid_constant__ li_prompt p, T* out, float* lse) {
  pdl_begin();
  __shared__ float q[kMaxKey];
  const int h = blockIdx.y % p.H, b = blockIdx.z;
  const int q0 = min(max(p.cu_q[b], 0), p.total_q), q1 = min(max(p.cu_q[b + 1], q0), p.total_q);
  const int k0 = min(max(p.cu_k[b], 0), p.total_k), k1 = min(max(p.cu_k[b + 1], k0), p.total_k);
  const int i = blockIdx.x;
  if (i >= q1 - q0) return;
  const T* qr = static_cast<const T*>(p.q) + (q0 + i) * p.q_tok_stride + h * p.q_head_stride;
  for (int j = threadIdx.x; j < p.d_nope + p.d_rope; j += blockDim.x) q[j] = static_cast<float>(qr[j]);
  __syncthreads();
  int64_t n = k1 - k0;
  if (p.causal) n = max(min(n, static_cast<int64_t>(i) + 1 + n - (q1 - q0)), int64_t(0));
  auto rows = [&](int64_t j) {
    KeyRow<T> r;
    r.k1 = static_cast<const T*>(p.k_nope) + (k0 + j) * p.k_tok_stride + h * p.k_head_stride;
    r.k2 = static_cast<const T*>(p.k_rope) + (k0 + j) * p.kr_tok_stride;
    r.v = static_cast<const T*>(p.v) + (k0 + j) * p.v_tok_stride + h * p.v_head_stride;
    return r;
  };
  const int64_t row = static_cast<int64_t>(q0 + i) * p.H + h;
  attend<T>(q, p.d_nope, p.d_rope, p.d_v, n, p.scale, rows, out + row * p.d_v, lse ? lse + row : nullptr);
}

}  // namespace

cudaError_t launch_latent_attn_rows(const LatentAttnArgs& a, li_dtype dtype, cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(static_cast<int64_t>(a.batch) * a.T * a.H)), b(kWarps * 32);
  return dtype == LI_F32 ? launch_pdl(latent_rows_kernel<float>, g, b, 0, st, 1, a)
                         : launch_pdl(latent_rows_kernel<__nv_bfloat16>, g, b, 0, st, 1, a);
}

cudaError_t launch_prompt_attn_rows(const li_prompt& p, void* out, float* lse, cudaStream_t st) {
  const dim3 g(p.max_q, p.H, p.batch), b(kWarps * 32);
  return p.dtype == LI_F32 ? launch_pdl(prompt_rows_kernel<float>, g, b, 0, st, 1, p, static_cast<float*>(out), lse)
                           : launch_pdl(prompt_rows_kernel<__nv_bfloat16>, g, b, 0, st, 1, p,
                                        static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace li
