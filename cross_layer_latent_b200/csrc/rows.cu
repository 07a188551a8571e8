// rows.cu -- row transforms around the attention: the norm of a head (or of a
// latent) and the rotation of its rotary part in one pass over the row,
// either from tensor to tensor (li_norm_rope) or into a paged cache
// (li_append_paged).
//
// A row is read once, held in registers as fp32, reduced across the lanes
// that share it, turned, rounded once and written once: the bytes of the rows
// are the bound.  Angles are formed as position * inv_freq in double
// precision and reduced to a turn there (an fp32 angle at position 1e6 is off
// by 0.03), once per token and frequency, in shared memory.
#include <cuda_bf16.h>

#include "attention.h"
#include "internal.h"
#include "sm100.cuh"

namespace li {

namespace {

// cos and sin of pos * f.  The turn's fraction is exact to 2^-50 of the
// angle; sincospif takes its fp32 value and the remainder enters to first
// order, so both are good to fp32 rounding at any position.
__device__ __forceinline__ float2 turn(int pos, float f) {
  const double turns = static_cast<double>(pos) * static_cast<double>(f) * 0.15915494309189533577;   // 1 / (2 pi)
  const double x = 2.0 * (turns - rint(turns));   // half turns, [-1, 1]
  const float hi = static_cast<float>(x);
  const float lo = static_cast<float>(x - static_cast<double>(hi)) * 3.14159265f;
  float sn, cs;
  sincospif(hi, &sn, &cs);
  return make_float2(fmaf(-lo, sn, cs), fmaf(lo, cs, sn));
}

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Eight consecutive elements as they lie in memory (16 or 32 bytes).
template <typename T>
struct Raw8 {
  uint4 u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) r.u[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float (&v)[8]) {
  const T* t = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f<T>(t[e]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  Raw8<T> r;
  T* t = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = from_f<T>(v[e]);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) reinterpret_cast<uint4*>(p)[i] = r.u[i];
}

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The transforms on a row spread over LPR lanes in chunks of 8 elements: lane
// `l` of the row holds chunks l, l + LPR, ...  Both ranges start and end on
// chunks; with halves NC is 1 (the partner chunk is then another lane's).
// tab: cos and sin of each rotary slot.  Every lane of the warp calls it.
template <int NC, int LPR>
__device__ __forceinline__ void transform_chunks(float (&v)[NC][8], int l, const li_row_transform& tf, const float2* tab) {
  if (tf.norm != LI_NORM_NONE) {
    const int c0 = tf.norm_offset / 8, c1 = c0 + tf.norm_dim / 8;
    const float inv_n = 1.f / static_cast<float>(tf.norm_dim);
    float mean = 0.f;
    if (tf.norm == LI_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (l + LPR * j >= c0 && l + LPR * j < c1)
#pragma unroll
          for (int e = 0; e < 8; ++e) s += v[j][e];
      mean = group_sum<LPR>(s) * inv_n;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (l + LPR * j >= c0 && l + LPR * j < c1)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = v[j][e] - mean;
          ss = fmaf(d, d, ss);
        }
    const float r = __frsqrt_rn(fmaf(group_sum<LPR>(ss), inv_n, tf.eps));
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = l + LPR * j;
      if (c >= c0 && c < c1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = (c - c0) * 8 + e;
          v[j][e] = (v[j][e] - mean) * r * (tf.gamma ? __ldg(tf.gamma + i) : 1.f) + (tf.beta ? __ldg(tf.beta + i) : 0.f);
        }
      }
    }
  }
  if (tf.rope_dim > 0) {
    const int c0 = tf.rope_offset / 8, nc = tf.rope_dim / 8;
    if (!tf.rope_halves) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int rc = l + LPR * j - c0;
        if (rc >= 0 && rc < nc) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float2 t = tab[rc * 4 + e / 2];
            const float x = v[j][e], y = v[j][e + 1];
            v[j][e] = x * t.x - y * t.y;
            v[j][e + 1] = x * t.y + y * t.x;
          }
        }
      }
    } else if constexpr (NC == 1) {
      const int rc = l - c0, hc = nc / 2;
      const bool in = rc >= 0 && rc < nc, first = rc < hc;
      const int src = in ? (first ? l + hc : l - hc) : l;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float o = __shfl_sync(0xffffffffu, v[0][e], src, LPR);
        if (in) {
          const float2 t = tab[(first ? rc : rc - hc) * 8 + e];
          v[0][e] = first ? v[0][e] * t.x - o * t.y : o * t.y + v[0][e] * t.x;
        }
      }
    }
  }
}

// The same for rows of any size and alignment, one warp a row, the row in
// shared memory (rotary partners are any distance apart).
__device__ __forceinline__ void transform_smem(float* row, int lane, const li_row_transform& tf, const float2* tab) {
  if (tf.norm != LI_NORM_NONE) {
    float* x = row + tf.norm_offset;
    const float inv_n = 1.f / static_cast<float>(tf.norm_dim);
    float mean = 0.f, ss = 0.f;
    if (tf.norm == LI_NORM_LAYER) {
      float s = 0.f;
      for (int i = lane; i < tf.norm_dim; i += 32) s += x[i];
      mean = group_sum<32>(s) * inv_n;
    }
    for (int i = lane; i < tf.norm_dim; i += 32) ss = fmaf(x[i] - mean, x[i] - mean, ss);
    const float r = __frsqrt_rn(fmaf(group_sum<32>(ss), inv_n, tf.eps));
    for (int i = lane; i < tf.norm_dim; i += 32)
      x[i] = (x[i] - mean) * r * (tf.gamma ? __ldg(tf.gamma + i) : 1.f) + (tf.beta ? __ldg(tf.beta + i) : 0.f);
    __syncwarp();
  }
  if (tf.rope_dim > 0) {
    float* x = row + tf.rope_offset;
    const int half = tf.rope_dim / 2;
    for (int p = lane; p < half; p += 32) {
      const int i = tf.rope_halves ? p : 2 * p, k = tf.rope_halves ? p + half : 2 * p + 1;
      const float2 t = tab[p];
      const float a = x[i], b = x[k];
      x[i] = a * t.x - b * t.y;
      x[k] = a * t.y + b * t.x;
    }
    __syncwarp();
  }
}

constexpr int kVecThreads = 256;
constexpr int kAnyWarps = 4;

// Which set a head index of all sets together falls into, and the first head
// of that set.
__device__ __forceinline__ int find_set(const NormRopeArgs& a, int h, int* first) {
  int s = 0, f = 0;
  while (s + 1 < a.n_sets && h >= f + a.set[s].H) f += a.set[s++].H;
  *first = f;
  return s;
}

// cos / sin tables of the sets that heads [h0, h1) touch; a set with the
// same frequencies as an earlier one shares its table.
__device__ __forceinline__ int table_of(const NormRopeArgs& a, int s) {
  for (int u = 0; u < s; ++u)
    if (a.set[u].tf.inv_freq == a.set[s].tf.inv_freq && a.set[u].tf.rope_dim >= a.set[s].tf.rope_dim) return u;
  return s;
}
__device__ __forceinline__ void fill_tables(const NormRopeArgs& a, int64_t tok, float2 (*tab)[kMaxRowDim / 2]) {
  for (int s = 0; s < a.n_sets; ++s) {
    const li_row_transform& tf = a.set[s].tf;
    if (tf.rope_dim == 0 || table_of(a, s) != s) continue;
    const int pos = __ldg(a.pos + tok);
    for (int p = threadIdx.x; p < tf.rope_dim / 2; p += blockDim.x) tab[s][p] = turn(pos, __ldg(tf.inv_freq + p));
  }
}

// One block: heads_per_block heads of one token, so that a token's angles are
// computed once for many heads.  U rows a lane group are in flight at once.
template <typename T, int NC, int LPR>
__global__ void __launch_bounds__(kVecThreads) norm_rope_vec_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_begin();
  pdl_release();
  __shared__ float2 tab[kMaxRowSets][kMaxRowDim / 2];
  constexpr int U = NC == 1 ? 4 : 1;
  constexpr int kRows = kVecThreads / LPR;
  const int hblocks = (a.heads + a.heads_per_block - 1) / a.heads_per_block;
  const int64_t tok = blockIdx.x / hblocks;
  const int h0 = static_cast<int>(blockIdx.x - tok * hblocks) * a.heads_per_block;
  const int h1 = min(h0 + a.heads_per_block, a.heads);
  const int l = threadIdx.x % LPR, g = threadIdx.x / LPR;
  bool ready = false;
  for (int hb = h0; hb < h1; hb += kRows * U) {
    Raw8<T> raw[U][NC];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = hb + u * kRows + g;
      if (h < h1) {
        int first;
        const li_head_rows& s = a.set[find_set(a, h, &first)];
        const T* x = static_cast<const T*>(s.x) + tok * s.tok_stride + (h - first) * s.head_stride;
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if ((l + LPR * j) * 8 < s.dim) raw[u][j] = load_raw8(x + (l + LPR * j) * 8);
      }
    }
    if (!ready) {
      fill_tables(a, tok, tab);
      __syncthreads();
      ready = true;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // lanes without a row run along on zeros (the shuffles need every lane)
      const int h = hb + u * kRows + g, hc = min(h, h1 - 1);
      if (__all_sync(0xffffffffu, h >= h1)) continue;
      int first;
      const int si = find_set(a, hc, &first);
      const li_head_rows& s = a.set[si];
      float v[NC][8];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        if (h < h1 && (l + LPR * j) * 8 < s.dim) {
          unpack8<T>(raw[u][j], v[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = 0.f;
        }
      }
      transform_chunks<NC, LPR>(v, l, s.tf, tab[table_of(a, si)]);
      if (h < h1) {
        T* o = static_cast<T*>(s.out) + tok * s.out_tok_stride + (h - first) * s.out_head_stride;
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if ((l + LPR * j) * 8 < s.dim) store8<T>(o + (l + LPR * j) * 8, v[j]);
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kAnyWarps * 32) norm_rope_any_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_begin();
  pdl_release();
  __shared__ float2 tab[kMaxRowSets][kMaxRowDim / 2];
  __shared__ float rows[kAnyWarps][kMaxRowDim];
  const int hblocks = (a.heads + a.heads_per_block - 1) / a.heads_per_block;
  const int64_t tok = blockIdx.x / hblocks;
  const int h0 = static_cast<int>(blockIdx.x - tok * hblocks) * a.heads_per_block;
  const int h1 = min(h0 + a.heads_per_block, a.heads);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  fill_tables(a, tok, tab);
  __syncthreads();
  for (int h = h0 + warp; h < h1; h += kAnyWarps) {
    int first;
    const int si = find_set(a, h, &first);
    const li_head_rows& s = a.set[si];
    const T* x = static_cast<const T*>(s.x) + tok * s.tok_stride + (h - first) * s.head_stride;
    for (int i = lane; i < s.dim; i += 32) rows[warp][i] = to_f<T>(x[i]);
    __syncwarp();
    transform_smem(rows[warp], lane, s.tf, tab[table_of(a, si)]);
    T* o = static_cast<T*>(s.out) + tok * s.out_tok_stride + (h - first) * s.out_head_stride;
    for (int i = lane; i < s.dim; i += 32) o[i] = from_f<T>(rows[warp][i]);
    __syncwarp();
  }
}

// ------------------------------------------------------------------ paged append

struct NewRows {
  int64_t start;   // first position written
  int n;           // rows of the sequence
  bool ok;         // they fit
};
__device__ __forceinline__ NewRows new_rows(const AppendPagedArgs& a, int b) {
  NewRows r;
  r.n = a.n_new ? min(max(a.n_new[b], 0), a.T) : a.T;
  r.start = a.start ? a.start[b] : a.lengths[b];
  r.ok = r.start >= 0 && r.start + r.n <= static_cast<int64_t>(a.max_pages) * a.page_size;
  return r;
}

// One warp a row.  Sequence lengths advance after every row's start has been
// read: at once when the starts come from `start`, else in the last block to
// finish (a counter in the workspace, which that block resets).
template <typename T, int NC>   // NC = 0: any size and alignment, by shared memory
__global__ void __launch_bounds__(kAnyWarps * 32) append_paged_kernel(const __grid_constant__ AppendPagedArgs a) {
  pdl_begin();
  pdl_release();
  __shared__ float2 tab[kAnyWarps][kMaxRowDim / 2];
  __shared__ float rows[kAnyWarps][NC == 0 ? kMaxRowDim : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * a.T;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * kAnyWarps + warp; r < n_rows; r += static_cast<int64_t>(gridDim.x) * kAnyWarps) {
    const T* x = static_cast<const T*>(a.x) + r * a.tok_stride;
    constexpr int kN = NC == 0 ? 1 : NC;
    Raw8<T> raw[kN];
    if constexpr (NC > 0) {
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if ((lane + 32 * j) * 8 < a.dim) raw[j] = load_raw8(x + (lane + 32 * j) * 8);
    }
    const float f0 = lane < a.tf.rope_dim / 2 ? __ldg(a.tf.inv_freq + lane) : 0.f;
    const int b = static_cast<int>(r / a.T), t = static_cast<int>(r - static_cast<int64_t>(b) * a.T);
    const NewRows nr = new_rows(a, b);
    if (t == 0 && lane == 0) {
      if (!nr.ok) record_status(a.status, kStatusCapacity);
      else if (a.start) a.lengths[b] = static_cast<int>(nr.start) + nr.n;
    }
    if (!nr.ok || t >= nr.n) continue;
    const int pos = static_cast<int>(nr.start) + t;
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / a.page_size];
    for (int p = lane; p < a.tf.rope_dim / 2; p += 32) tab[warp][p] = turn(pos, p < 32 ? f0 : __ldg(a.tf.inv_freq + p));
    __syncwarp();
    T* o = static_cast<T*>(a.data) + (static_cast<int64_t>(page) * a.page_size + pos % a.page_size) * a.dim;
    const bool there = page >= 0 && page < a.n_pages;
    if (!there && lane == 0) record_status(a.status, kStatusIndex);
    if constexpr (NC > 0) {
      float v[kN][8];
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        if ((lane + 32 * j) * 8 < a.dim) {
          unpack8<T>(raw[j], v[j]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = 0.f;
        }
      }
      transform_chunks<kN, 32>(v, lane, a.tf, tab[warp]);
      if (there) {
#pragma unroll
        for (int j = 0; j < NC; ++j)
          if ((lane + 32 * j) * 8 < a.dim) store8<T>(o + (lane + 32 * j) * 8, v[j]);
      }
    } else {
      for (int i = lane; i < a.dim; i += 32) rows[warp][i] = to_f<T>(x[i]);
      __syncwarp();
      transform_smem(rows[warp], lane, a.tf, tab[warp]);
      if (there)
        for (int i = lane; i < a.dim; i += 32) o[i] = from_f<T>(rows[warp][i]);
    }
    __syncwarp();
  }
  if (a.start) return;
  __shared__ unsigned last;
  __syncthreads();
  if (threadIdx.x == 0) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.done) : "memory");
    last = prev == gridDim.x - 1 ? 1u : 0u;
  }
  __syncthreads();
  if (!last) return;
  for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
    const NewRows nr = new_rows(a, b);
    if (nr.ok) a.lengths[b] = static_cast<int>(nr.start) + nr.n;
  }
  if (threadIdx.x == 0) *a.done = 0u;
}

template <typename T>
cudaError_t norm_rope_t(const NormRopeArgs& a, bool vec, int max_dim, int64_t grid, cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(grid));
  if (!vec) return launch_pdl(norm_rope_any_kernel<T>, g, dim3(kAnyWarps * 32), 0, st, 1, a);
  const dim3 b(kVecThreads);
  if (max_dim <= 64) return launch_pdl(norm_rope_vec_kernel<T, 1, 8>, g, b, 0, st, 1, a);
  if (max_dim <= 128) return launch_pdl(norm_rope_vec_kernel<T, 1, 16>, g, b, 0, st, 1, a);
  if (max_dim <= 256) return launch_pdl(norm_rope_vec_kernel<T, 1, 32>, g, b, 0, st, 1, a);
  if (max_dim <= 512) return launch_pdl(norm_rope_vec_kernel<T, 2, 32>, g, b, 0, st, 1, a);
  return launch_pdl(norm_rope_vec_kernel<T, 4, 32>, g, b, 0, st, 1, a);
}

template <typename T>
cudaError_t append_paged_t(const AppendPagedArgs& a, bool vec, unsigned grid, cudaStream_t st) {
  const dim3 g(grid), b(kAnyWarps * 32);
  if (!vec) return launch_pdl(append_paged_kernel<T, 0>, g, b, 0, st, 1, a);
  if (a.dim <= 256) return launch_pdl(append_paged_kernel<T, 1>, g, b, 0, st, 1, a);
  if (a.dim <= 768) return launch_pdl(append_paged_kernel<T, 3>, g, b, 0, st, 1, a);
  return launch_pdl(append_paged_kernel<T, 4>, g, b, 0, st, 1, a);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, li_dtype dtype, bool vec, int max_dim, int64_t grid, cudaStream_t st) {
  return dtype == LI_F32 ? norm_rope_t<float>(a, vec, max_dim, grid, st)
                         : norm_rope_t<__nv_bfloat16>(a, vec, max_dim, grid, st);
}

cudaError_t launch_append_paged(const AppendPagedArgs& a, li_dtype dtype, bool vec, int num_sms, cudaStream_t st) {
  const int64_t blocks = (static_cast<int64_t>(a.batch) * a.T + kAnyWarps - 1) / kAnyWarps;
  const unsigned grid = static_cast<unsigned>(blocks < 16 * num_sms ? blocks : 16 * num_sms);
  return dtype == LI_F32 ? append_paged_t<float>(a, vec, grid, st) : append_paged_t<__nv_bfloat16>(a, vec, grid, st);
}

}  // namespace li
