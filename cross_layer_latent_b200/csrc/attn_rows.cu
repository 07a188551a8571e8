// attn_rows.cu -- attention of one fp32 query row and head per block, on the
// CUDA cores: one pass over the keys with the running maximum and sum of the
// softmax, each of the block's warps over its share of the keys, 32 at a time,
// and the warps' parts joined at the end.  Everything stays fp32: tensor-core
// fp32 products (tf32) would round the operands to 11 bits.
//
// Within a warp, eight lanes take a key (four keys at a time): the products of
// a key need three shuffles, its value rows are read in full lines, and small
// dimensions keep most lanes busy.  A warp a key at a time took 33 us for 2 x 8
// heads over 512 rows of 48 (five shuffles and a dependent load a key); this
// takes 15.
// No block shares what another reads, and none splits a query's keys: made for
// small configurations.  64 heads over 8192 rows of 576 take 620 us (14 of
// arithmetic), a prompt of 2048 x 16 heads 6.3 ms.
#include <cmath>

#include "attention.h"
#include "internal.h"
#include "sm100.cuh"

namespace li {

namespace {

constexpr int kWarps = 8;
constexpr int kMaxKey = 576, kMaxValue = 512;
constexpr int kNV = kMaxValue / 32;   // 4-value pieces of a lane

struct KeyRow {
  const float *k1, *k2, *v;   // key in two parts, value; v null: skipped
};

__device__ __forceinline__ const float* from_lane(const float* p, int lane) {
  return reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(p), lane));
}

// q: the query in shared memory, 16-byte aligned.  rows(i) gives key i of n.
// d1, d2 and the readable part of a value row are multiples of 4.  Every
// thread of the block calls it.
template <typename Rows>
__device__ __forceinline__ void attend(const float* q, int d1, int d2, int d_v, int64_t n, float scale, Rows rows, float* out,
                                       float* lse) {
  __shared__ float part[kWarps][kMaxValue], pm[kWarps], pl[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, g = lane >> 3;
  const int c1 = d1 / 4, ck = (d1 + d2) / 4, cv = (d_v + 3) / 4;
  float4 acc[kNV];
#pragma unroll
  for (int j = 0; j < kNV; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, s = 0.f;
  KeyRow next{};
  const int64_t step = kWarps * 32;
  int64_t i0 = static_cast<int64_t>(warp) * 32;
  if (i0 + lane < n) next = rows(i0 + lane);
  for (; i0 < n; i0 += step) {
    const KeyRow mine = next;
    next = KeyRow{};
    if (i0 + step + lane < n) next = rows(i0 + step + lane);   // found while these are worked on
    // scores: lane i ends up with key i's
    float z = -INFINITY;
#pragma unroll 2
    for (int u = 0; u < 8; ++u) {
      const float *k1 = from_lane(mine.k1, 4 * u + g), *k2 = from_lane(mine.k2, 4 * u + g), *v = from_lane(mine.v, 4 * u + g);
      float d = 0.f;
      if (v) {
#pragma unroll 4
        for (int c = l; c < ck; c += 8) {
          const float4 k = __ldg(reinterpret_cast<const float4*>(c < c1 ? k1 + c * 4 : k2 + (c - c1) * 4));
          const float4 x = *reinterpret_cast<const float4*>(q + c * 4);
          d = fmaf(x.x, k.x, fmaf(x.y, k.y, fmaf(x.z, k.z, fmaf(x.w, k.w, d))));
        }
      }
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
      const float mine_d = __shfl_sync(0xffffffffu, d, (lane & 3) * 8);
      if ((lane >> 2) == u && mine.v) z = mine_d * scale;
    }
    float top = z;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float now = fmaxf(m, top);
    // fmaxf passes over a NaN: such a score goes on, and makes the row's sums NaN
    if (now == -INFINITY && !__any_sync(0xffffffffu, z != z)) continue;
    const float keep = expf(m - now), p = expf(z - now);
    m = now;
    s = fmaf(s, keep, p);                        // a lane's own share of the sum
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      acc[j].x *= keep;
      acc[j].y *= keep;
      acc[j].z *= keep;
      acc[j].w *= keep;
    }
#pragma unroll 2
    for (int u = 0; u < 8; ++u) {
      const float* v = from_lane(mine.v, 4 * u + g);
      const float w = __shfl_sync(0xffffffffu, p, 4 * u + g);
      if (v) {
#pragma unroll
        for (int j = 0; j < kNV; ++j) {
          const int c = l + 8 * j;
          if (c < cv) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(v + c * 4));
            acc[j].x = fmaf(w, x.x, acc[j].x);
            acc[j].y = fmaf(w, x.y, acc[j].y);
            acc[j].z = fmaf(w, x.z, acc[j].z);
            acc[j].w = fmaf(w, x.w, acc[j].w);
          }
        }
      }
    }
  }
  // the warp's four key groups, then the block's warps
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
#pragma unroll
  for (int j = 0; j < kNV; ++j) {
    if (8 * j >= cv) break;
    float a[4] = {acc[j].x, acc[j].y, acc[j].z, acc[j].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      a[e] += __shfl_xor_sync(0xffffffffu, a[e], 8);
      a[e] += __shfl_xor_sync(0xffffffffu, a[e], 16);
      if (g == 0 && (l + 8 * j) * 4 + e < d_v) part[warp][(l + 8 * j) * 4 + e] = a[e];
    }
  }
  if (lane == 0) {
    pm[warp] = m;
    pl[warp] = s;
  }
  __syncthreads();
  float M = -INFINITY, L = 0.f, w[kWarps];
#pragma unroll
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, pm[i]);
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    w[i] = pm[i] == -INFINITY ? 0.f : expf(pm[i] - M);
    L = fmaf(w[i], pl[i], L);
  }
  const float inv = inverse_sum(L);
  for (int i = threadIdx.x; i < d_v; i += kWarps * 32) {
    float x = 0.f;
#pragma unroll
    for (int u = 0; u < kWarps; ++u) x = fmaf(w[u], part[u][i], x);
    out[i] = x * inv;
  }
  if (lse && threadIdx.x == 0) *lse = row_lse(L, M + logf(L));
}

// One block per (sequence, query, head).
__global__ void __launch_bounds__(kWarps * 32) latent_rows_kernel(const __grid_constant__ LatentAttnArgs a) {
  pdl_begin();
  __shared__ __align__(16) float q[kMaxKey];
  const int64_t row = blockIdx.x;              // (b * T + t) * H + h
  const int64_t bt = row / a.H;
  const int b = static_cast<int>(bt / a.T);
  for (int i = threadIdx.x; i < a.dim; i += blockDim.x) q[i] = a.q[row * a.dim + i];
  int64_t n = min(static_cast<int64_t>(max(a.lengths[b], 0)), static_cast<int64_t>(a.max_pages) * a.page_size);
  if (a.q_pos) n = min(n, max(static_cast<int64_t>(a.q_pos[bt]) + 1, int64_t(0)));
  __syncthreads();
  const int32_t* table = a.page_table + static_cast<int64_t>(b) * a.max_pages;
  const int32_t* sel = a.sel ? a.sel + bt * a.k : nullptr;
  auto rows = [&](int64_t i) {
    KeyRow r{};
    const int s = sel ? sel[i] : static_cast<int>(i);
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
    r.k1 = r.v = a.data + (static_cast<int64_t>(page) * a.page_size + s % a.page_size) * a.dim;
    return r;
  };
  attend(q, a.dim, 0, a.d_v, sel ? a.k : n, a.scale, rows, a.out + row * a.d_v, a.lse ? a.lse + row : nullptr);
}

// One block per (query, head, sequence); queries past the sequence's end return.
__global__ void __launch_bounds__(kWarps * 32) prompt_rows_kernel(const __grid_constant__ li_prompt p, float* out, float* lse) {
  pdl_begin();
  __shared__ __align__(16) float q[kMaxKey];
  const int h = blockIdx.y, b = blockIdx.z;
  const int q0 = min(max(p.cu_q[b], 0), p.total_q), q1 = min(max(p.cu_q[b + 1], q0), p.total_q);
  const int k0 = min(max(p.cu_k[b], 0), p.total_k), k1 = min(max(p.cu_k[b + 1], k0), p.total_k);
  const int i = blockIdx.x;
  if (i >= q1 - q0) return;
  const float* qr = static_cast<const float*>(p.q) + (q0 + i) * p.q_tok_stride + h * p.q_head_stride;
  for (int j = threadIdx.x; j < p.d_nope + p.d_rope; j += blockDim.x) q[j] = qr[j];
  __syncthreads();
  int64_t n = k1 - k0;
  if (p.causal) n = max(min(n, static_cast<int64_t>(i) + 1 + n - (q1 - q0)), int64_t(0));
  auto rows = [&](int64_t j) {
    KeyRow r;
    r.k1 = static_cast<const float*>(p.k_nope) + (k0 + j) * p.k_tok_stride + h * p.k_head_stride;
    r.k2 = static_cast<const float*>(p.k_rope) + (k0 + j) * p.kr_tok_stride;
    r.v = static_cast<const float*>(p.v) + (k0 + j) * p.v_tok_stride + h * p.v_head_stride;
    return r;
  };
  const int64_t row = static_cast<int64_t>(q0 + i) * p.H + h;
  attend(q, p.d_nope, p.d_rope, p.d_v, n, p.scale, rows, out + row * p.d_v, lse ? lse + row : nullptr);
}

}  // namespace

cudaError_t launch_latent_attn_rows(const LatentAttnArgs& a, cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(static_cast<int64_t>(a.batch) * a.T * a.H)), b(kWarps * 32);
  return launch_pdl(latent_rows_kernel, g, b, 0, st, 1, a);
}

cudaError_t launch_prompt_attn_rows(const li_prompt& p, float* out, float* lse, cudaStream_t st) {
  return launch_pdl(prompt_rows_kernel, dim3(p.max_q, p.H, p.batch), dim3(kWarps * 32), 0, st, 1, p, out, lse);
}

}  // namespace li
