// rows.cu -- row transforms around the attention: the norm of a head (or of a
// latent) and the rotation of its rotary part in one pass over the row,
// either from tensor to tensor (li_norm_rope) or into a paged cache
// (li_append_paged).
//
// A row is read once, held in registers, reduced in fp32 across the lanes that
// share it, turned, rounded once and written once: the bytes of the rows are
// the bound.  Angles are formed modulo a turn in 64-bit integers (an fp32
// angle at position 1e6 is off by 0.03).
#include <cuda_bf16.h>

#include "attention.h"
#include "attn_sm100.cuh"
#include "internal.h"

namespace li {

namespace {

// cos and sin of pos * f.  The angle is formed in turns modulo 1, as 64-bit
// fractions: f = m 2^e with a 24-bit m, so f / (2 pi) is m times the digits of
// 1 / (2 pi), shifted, and whole turns fall off the top of the products.  It is
// off by 2^-62 of itself (the digits end) and by |pos| 2^-64 of a turn (the
// shift cuts), 2^-33 at most, and its 32 leading bits are used: 2^-31 of a turn
// and 2^-62 of the angle in all.  (Double precision gives the same to 2^-52, but
// its conversions and roundings go through the narrow transcendental pipe:
// with them the append spent 700 instructions a row.)  The fraction's upper 24
// bits make an exact fp32 argument of sincospif, the next 8 enter to first
// order.
__device__ __forceinline__ uint64_t turns_of(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>(u >> 23 & 0xFFu);
  const uint64_t m = e ? (u & 0x7FFFFFu) | 0x800000u : (u & 0x7FFFFFu);
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;          // 2^64 / (2 pi)
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int shift = 150 - max(e, 1);                           // m 2^(e - 150) = |f|
  const uint64_t t = shift <= 0     ? (shift > -64 ? lo << -shift : 0ull)
                     : shift < 64   ? (lo >> shift) | (hi << (64 - shift))
                     : shift < 128  ? hi >> (shift - 64)
                                    : 0ull;
  return u >> 31 ? 0ull - t : t;
}
__device__ __forceinline__ float2 turn(int pos, uint64_t turns) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const int h = static_cast<int>(t >> 32);                     // [-1/2, 1/2) turn in 2^-32
  const float hi = static_cast<float>(h >> 8) * 0x1p-23f;      // half turns, exact
  const float lo = static_cast<float>(h & 0xFF) * (0x1p-31f * 3.14159265f);
  float sn, cs;
  sincospif(hi, &sn, &cs);
  return make_float2(fmaf(-lo, sn, cs), fmaf(lo, cs, sn));
}
// For rows that are rounded to bf16: the special-function unit's cosine and
// sine, off by 2^-21, a thousandth of that rounding.
__device__ __forceinline__ float2 turn_short(int pos, uint64_t turns) {
  const uint64_t t = turns * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const float x = static_cast<float>(static_cast<int>(t >> 32)) * (0x1p-31f * 3.14159265f);
  return make_float2(__cosf(x), __sinf(x));
}
template <typename T>
__device__ __forceinline__ float2 turn_for(int pos, float f) {
  return sizeof(T) == 2 ? turn_short(pos, turns_of(f)) : turn(pos, turns_of(f));
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
// The same to shared memory, by copies that the lane waits for.
template <typename T>
__device__ __forceinline__ void copy_raw8(Raw8<T>* to, const T* p) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(&to->u[i])), "l"(reinterpret_cast<const uint4*>(p) + i) : "memory");
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = reinterpret_cast<const float*>(&r)[e];
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = __uint_as_float(w[e] << 16);
    v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  // two values a conversion: single ones go through the narrow pipe
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// The hardware's reciprocal root and one Newton step; an infinity (a zero row
// without eps) stays one.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x), better = r * fmaf(-0.5f * x * r, r, 1.5f);
  return fabsf(better) <= 3.4e38f ? better : r;
}

// Eight fp32 parameters.
__device__ __forceinline__ void load_params(const float* p, float (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __ldg(p + e);
  }
}

template <int LPR>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The transforms on a row spread over LPR lanes in chunks of 8 elements: lane
// `l` of the row holds chunks l, l + LPR, ... in raw, zeros where it has none.
// Both ranges start and end on chunks, and a rotation by halves has its
// partners either in the same register of another lane or in another register
// of the same lane (halves_in_reach).  turns(i, out) gives cos and sin of the
// 8 / 2 (pairs) or 8 (halves) slots from slot i on; store(chunk, values) takes
// the results.  The row stays packed between the norm's sums and the stores,
// which halves its registers.  Every lane of the warp calls it.
// NORM is the li_norm, ROPE 0 none, 1 pairs, 2 halves: one body a kind, as the
// whole of it would cost every row its tests.
template <typename T, int NC, int LPR, int NORM, int ROPE, typename Turns, typename Store>
__device__ __forceinline__ void transform_kind(const Raw8<T> (&raw)[NC], int l, const li_row_transform& tf, Turns turns, Store store) {
  const int n0 = tf.norm_offset / 8, n1 = n0 + tf.norm_dim / 8;
  float mean = 0.f, r = 1.f;
  if constexpr (NORM != LI_NORM_NONE) {
    const float inv_n = __frcp_rn(static_cast<float>(tf.norm_dim));
    if constexpr (NORM == LI_NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (l + LPR * j >= n0 && l + LPR * j < n1) {
          float v[8];
          unpack8(raw[j], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) s += v[e];
        }
      mean = group_sum<LPR>(s) * inv_n;
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (l + LPR * j >= n0 && l + LPR * j < n1) {
        float v[8];
        unpack8(raw[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = NORM == LI_NORM_LAYER ? v[e] - mean : v[e];
          ss = fmaf(d, d, ss);
        }
      }
    r = inverse_root(fmaf(group_sum<LPR>(ss), inv_n, tf.eps));
  }
  // chunk c, held in `x`, after the norm
  auto value = [&](const Raw8<T>& x, int c, float (&v)[8]) {
    unpack8(x, v);
    if constexpr (NORM != LI_NORM_NONE) {
      if (c >= n0 && c < n1) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (NORM == LI_NORM_LAYER ? v[e] - mean : v[e]) * r;
        if (tf.gamma) {
          float g[8];
          load_params(tf.gamma + (c - n0) * 8, g);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= g[e];
        }
        if (tf.beta) {
          float b[8];
          load_params(tf.beta + (c - n0) * 8, b);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += b[e];
        }
      }
    }
  };
  const int r0 = tf.rope_offset / 8, nc = tf.rope_dim / 8, hc = nc / 2;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = l + LPR * j, rc = c - r0;
    float v[8];
    value(raw[j], c, v);
    if (ROPE != 0 && LPR * (j + 1) > r0 && LPR * j < r0 + nc) {   // this register row holds rotary chunks
      const bool in = rc >= 0 && rc < nc;
      if constexpr (ROPE == 1) {
        if (in) {
          float2 t[4];
          turns(rc * 4, t);
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float x = v[e], y = v[e + 1];
            v[e] = x * t[e / 2].x - y * t[e / 2].y;
            v[e + 1] = x * t[e / 2].y + y * t[e / 2].x;
          }
        }
      } else if constexpr (ROPE == 2) {
        const bool first = rc < hc;
        const float sign = first ? -1.f : 1.f;
        float o[8];                              // the slot's other half
        if (nc <= LPR) {
          const int src = in ? (first ? l + hc : l - hc) : l;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __shfl_sync(0xffffffffu, v[e], src, LPR);
        } else {
          const int d = hc / LPR;
#pragma unroll
          for (int k = 0; k < NC; ++k)
            if (k == (first ? j + d : j - d)) value(raw[k], l + LPR * k, o);
        }
        if (in) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float2 t[4];
            turns((first ? rc : rc - hc) * 8 + 4 * q, t);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[4 * q + e] = fmaf(sign * t[e].y, o[4 * q + e], v[4 * q + e] * t[e].x);
          }
        }
      }
    }
    store(c, v);
  }
}

template <typename T, int NC, int LPR, int NORM, typename Turns, typename Store>
__device__ __forceinline__ void transform_norm(const Raw8<T> (&raw)[NC], int l, const li_row_transform& tf, Turns turns, Store store) {
  if (tf.rope_dim == 0) transform_kind<T, NC, LPR, NORM, 0>(raw, l, tf, turns, store);
  else if (!tf.rope_halves) transform_kind<T, NC, LPR, NORM, 1>(raw, l, tf, turns, store);
  else transform_kind<T, NC, LPR, NORM, 2>(raw, l, tf, turns, store);
}
template <typename T, int NC, int LPR, typename Turns, typename Store>
__device__ __forceinline__ void transform_chunks(const Raw8<T> (&raw)[NC], int l, const li_row_transform& tf, Turns turns, Store store) {
  if (tf.norm == LI_NORM_RMS) transform_norm<T, NC, LPR, LI_NORM_RMS>(raw, l, tf, turns, store);
  else if (tf.norm == LI_NORM_LAYER) transform_norm<T, NC, LPR, LI_NORM_LAYER>(raw, l, tf, turns, store);
  else transform_norm<T, NC, LPR, LI_NORM_NONE>(raw, l, tf, turns, store);
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
    const float r = inverse_root(fmaf(group_sum<32>(ss), inv_n, tf.eps));
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

// Two warps a block: a token's tasks are few (17 for 64 + 1 heads of 192), and
// what a warp sets up for a set pays from several tasks on (256 threads: 183 us
// for 8192 tokens, 128: 125, 64: 106, before rows came through shared memory).
constexpr int kVecThreads = 64;
constexpr int kAnyWarps = 4;

// cos / sin tables of the sets; a set with the same frequencies as an earlier
// one shares its table.
__device__ __forceinline__ int table_of(const NormRopeArgs& a, int s) {
  for (int u = 0; u < s; ++u)
    if (a.set[u].tf.inv_freq == a.set[s].tf.inv_freq && a.set[u].tf.rope_dim >= a.set[s].tf.rope_dim) return u;
  return s;
}
template <typename T>
__device__ __forceinline__ void fill_tables(const NormRopeArgs& a, int64_t tok, float2* tab) {
  for (int s = 0; s < a.n_sets; ++s) {
    const li_row_transform& tf = a.set[s].tf;
    if (tf.rope_dim == 0 || table_of(a, s) != s) continue;
    const int pos = __ldg(a.pos + tok);
    for (int p = threadIdx.x; p < tf.rope_dim / 2; p += blockDim.x) tab[s * a.tab_stride + p] = turn_for<T>(pos, __ldg(tf.inv_freq + p));
  }
}

// One block works on one token, so that its angles are computed once for many
// heads.  A row belongs to LPR lanes, as few as hold it in NC <= 4 chunks
// each: the reductions, address arithmetic and parameter loads are shared by
// the 32 / LPR rows of a warp, a task.  (With a warp a row the kernel was bound
// by its instructions: 300 us for 8192 x 65 rows of 192, against 62 us for
// their bytes.)  Tasks do not mix sets.  A warp's next task is loaded
// while it works on one, its first before the angles are formed.
// A launch with one layer norm, beta or longer rotation has all its sets here:
// 8192 x (64 RMS heads of 192 + 1 layer-normed key) bf16 take 113 to 130 us,
// 78 with an RMS key (norm_rope_plain_kernel).
template <typename T, int NC, int LPR>
__global__ void __launch_bounds__(kVecThreads) norm_rope_vec_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_begin();
  pdl_release();
  extern __shared__ __align__(16) float2 tab[];  // [n_sets][tab_stride]
  constexpr int G = 32 / LPR, kWarps = kVecThreads / 32;
  const int64_t tok = blockIdx.x / a.blocks;
  const int t0 = static_cast<int>(blockIdx.x - tok * a.blocks) * a.per_block, t1 = min(t0 + a.per_block, a.tasks);
  const int l = threadIdx.x % LPR, g = (threadIdx.x & 31) / LPR;
  int task = t0 + (threadIdx.x >> 5);
  Raw8<T> next[NC];
  int next_set = 0, next_head = 0;
  // a lane's chunks of the task's rows (zeros where there are none)
  auto load = [&]() {
    if (task >= t1) return;
    int si = 0, t = task;
    for (int n = (a.set[0].H + G - 1) / G; t >= n; n = (a.set[si].H + G - 1) / G) {
      t -= n;
      ++si;
    }
    const li_head_rows& s = a.set[si];
    next_set = si;
    next_head = t * G + g;
    const T* x = static_cast<const T*>(s.x) + tok * s.tok_stride + next_head * s.head_stride;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      next[j] = Raw8<T>{};
      if (next_head < s.H && (l + LPR * j) * 8 < s.dim) next[j] = load_raw8(x + (l + LPR * j) * 8);
    }
  };
  load();
  fill_tables<T>(a, tok, tab);
  __syncthreads();
  while (task < t1) {
    Raw8<T> raw[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) raw[j] = next[j];
    const int head = next_head, si = next_set;
    task += kWarps;
    load();                                      // on its way while this one is worked on
    const li_head_rows& s = a.set[si];
    const float2* t = tab + table_of(a, si) * a.tab_stride;
    T* out = static_cast<T*>(s.out) + tok * s.out_tok_stride + head * s.out_head_stride;
    const bool there = head < s.H;
    const int dim = s.dim;
    transform_chunks<T, NC, LPR>(
        raw, l, s.tf,
        [t](int i, float2 (&o)[4]) {
          // i is even and so is tab_stride: 16-byte loads
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float4 two = *reinterpret_cast<const float4*>(t + i + k);
            o[k] = make_float2(two.x, two.y);
            o[k + 1] = make_float2(two.z, two.w);
          }
        },
        [=](int c, const float (&v)[8]) {
          if (there && c * 8 < dim) store8(out + c * 8, v);
        });
  }
}

// The common kind of head rows: RMS norm without beta or no norm, rotary chunks
// in one register row.  What a lane needs of the parameters and angles then
// stays in its registers for all tasks of a set, and a row costs little more
// than its arithmetic.  Registers leave 20 warps to an SM, so each keeps the rows
// of several tasks on their way, in shared memory (one task, in registers, and
// 16 warps: 104 us for 8192 x 65 rows of 192, most of them waiting for loads).
constexpr int kAhead = 3, kSlots = kAhead + 1;
template <typename T, int NC, int LPR, int ROPE, typename Angles>
__device__ __forceinline__ void plain_set(const li_head_rows& s, int64_t tok, const float2* tab, int t0, int t1, int l, int g,
                                          Raw8<T> (*ring)[NC][32], Angles angles) {
  constexpr int G = 32 / LPR, kWarps = kVecThreads / 32;
  const int lane = threadIdx.x & 31;
  int at = 0;
  const li_row_transform& tf = s.tf;
  const bool normed = tf.norm != LI_NORM_NONE;
  const int n0 = tf.norm_offset / 8, n1 = normed ? n0 + tf.norm_dim / 8 : n0;
  float gamma[NC][8];
  bool in_norm[NC], in_row[NC];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int c = l + LPR * j;
    in_row[j] = c * 8 < s.dim;
    in_norm[j] = c >= n0 && c < n1;
#pragma unroll
    for (int e = 0; e < 8; ++e) gamma[j][e] = 1.f;
    if (in_norm[j] && tf.gamma) load_params(tf.gamma + (c - n0) * 8, gamma[j]);
  }
  const T* x = static_cast<const T*>(s.x) + tok * s.tok_stride + l * 8;
  int task = t0 + (threadIdx.x >> 5);
  // the rows of the next kAhead tasks are on their way to shared memory, each lane's chunks by its own copies
  auto load = [&](int n) {
    const int h = (task + n * kWarps) * G + g;
#pragma unroll
    for (int j = 0; j < NC; ++j)
      if (task + n * kWarps < t1 && h < s.H && in_row[j]) copy_raw8(&ring[(at + n) % kSlots][j][lane], x + h * s.head_stride + LPR * 8 * j);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int n = 0; n < kAhead; ++n) load(n);
  angles();                                      // the block's, if this is its first set
  if (task >= t1) return;
  // rotary chunks are register row j0 of lanes [first, first + nc)
  const int r0 = tf.rope_offset / 8, nc = tf.rope_dim / 8, hc = nc / 2, j0 = r0 / LPR;
  const int rc = l - (r0 - j0 * LPR);
  const bool in = rc >= 0 && rc < nc;
  const bool low = rc < hc;
  const int src = in ? (low ? l + hc : l - hc) : l;
  float co[8], si[8];
  if constexpr (ROPE != 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // pairs: slot e / 2 of the chunk; halves: slot e of the chunk or of its partner
      const int slot = ROPE == 1 ? rc * 4 + e / 2 : (low ? rc : rc - hc) * 8 + e;
      const float2 t = in ? tab[slot] : make_float2(1.f, 0.f);
      co[e] = t.x;
      si[e] = (ROPE == 1 ? (e & 1) == 0 : low) ? -t.y : t.y;
    }
  }
  const float inv_n = normed ? __frcp_rn(static_cast<float>(tf.norm_dim)) : 0.f;
  T* out = static_cast<T*>(s.out) + tok * s.out_tok_stride + l * 8;
  for (; task < t1; task += kWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
    const int h = task * G + g;
    Raw8<T> raw[NC];
#pragma unroll
    for (int j = 0; j < NC; ++j) raw[j] = ring[at][j][lane];
    load(kAhead);                                // to the slot that was read one task ago
    at = (at + 1) % kSlots;
    float r = 1.f;
    if (normed) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < NC; ++j)
        if (in_norm[j]) {
          float v[8];
          unpack8(raw[j], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(v[e], v[e], ss);
        }
      r = inverse_root(fmaf(group_sum<LPR>(ss), inv_n, tf.eps));
    }
    T* o = out + h * s.out_head_stride;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      float v[8];
      unpack8(raw[j], v);
      const float k = in_norm[j] ? r : 1.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= k * gamma[j][e];
      if (ROPE != 0 && j == j0) {
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = ROPE == 1 ? v[e ^ 1] : __shfl_sync(0xffffffffu, v[e], src, LPR);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = in ? fmaf(si[e], w[e], co[e] * v[e]) : v[e];
      }
      if (h < s.H && in_row[j]) store8(o + LPR * 8 * j, v);
    }
  }
}

// Ten blocks an SM where 96 registers hold a lane's part (8192 x 65 rows of 192:
// 82 us, 85 with eight blocks of 121 registers, 87 with twelve that spill).
template <typename T, int NC, int LPR>
__global__ void __launch_bounds__(kVecThreads, sizeof(T) == 2 && NC <= 3 ? 10 : 6) norm_rope_plain_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_begin();
  pdl_release();
  extern __shared__ __align__(16) float2 tab[];  // [n_sets][tab_stride]
  __shared__ Raw8<T> rings[kVecThreads / 32][kSlots][NC][32];
  constexpr int G = 32 / LPR;
  const int64_t tok = blockIdx.x / a.blocks;
  const int b0 = static_cast<int>(blockIdx.x - tok * a.blocks) * a.per_block, b1 = min(b0 + a.per_block, a.tasks);
  const int l = threadIdx.x % LPR, g = (threadIdx.x & 31) / LPR;
  bool filled = false;
  auto angles = [&]() {
    if (filled) return;
    fill_tables<T>(a, tok, tab);
    __syncthreads();
    filled = true;
  };
  int first = 0;                                 // first task of the set
  for (int i = 0; i < a.n_sets; ++i) {
    const li_head_rows& s = a.set[i];
    const int n = (s.H + G - 1) / G, t0 = max(b0 - first, 0), t1 = min(b1 - first, n);
    first += n;
    if (t0 >= t1) continue;
    const float2* t = tab + table_of(a, i) * a.tab_stride;
    if (s.tf.rope_dim == 0) plain_set<T, NC, LPR, 0>(s, tok, t, t0, t1, l, g, rings[threadIdx.x >> 5], angles);
    else if (!s.tf.rope_halves) plain_set<T, NC, LPR, 1>(s, tok, t, t0, t1, l, g, rings[threadIdx.x >> 5], angles);
    else plain_set<T, NC, LPR, 2>(s, tok, t, t0, t1, l, g, rings[threadIdx.x >> 5], angles);
  }
}

// Rows of any size and alignment: a warp a row, a task, by way of shared memory.
template <typename T>
__global__ void __launch_bounds__(kAnyWarps * 32) norm_rope_any_kernel(const __grid_constant__ NormRopeArgs a) {
  pdl_begin();
  pdl_release();
  extern __shared__ __align__(16) float2 tab[];
  __shared__ float rows[kAnyWarps][kMaxRowDim];
  const int64_t tok = blockIdx.x / a.blocks;
  const int t0 = static_cast<int>(blockIdx.x - tok * a.blocks) * a.per_block, t1 = min(t0 + a.per_block, a.tasks);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  fill_tables<T>(a, tok, tab);
  __syncthreads();
  for (int t = t0 + warp; t < t1; t += kAnyWarps) {
    int h = t, si = 0;
    while (h >= a.set[si].H) h -= a.set[si++].H;
    const li_head_rows& s = a.set[si];
    const T* x = static_cast<const T*>(s.x) + tok * s.tok_stride + h * s.head_stride;
    for (int i = lane; i < s.dim; i += 32) rows[warp][i] = to_f<T>(x[i]);
    __syncwarp();
    transform_smem(rows[warp], lane, s.tf, tab + table_of(a, si) * a.tab_stride);
    T* o = static_cast<T*>(s.out) + tok * s.out_tok_stride + h * s.out_head_stride;
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

constexpr int kAppendLanes = 16;

// Sixteen lanes a row in NC chunks each, two rows a warp (eight lanes were no
// faster at 576: their registers left too few rows in flight); NC = 0: any size and
// alignment, a warp a row by way of shared memory.  Every row has a position
// of its own, so a lane forms the angles of its own slots.  Sequence lengths
// advance after every row's start and number have been read: at once when
// both come from elsewhere, else in the last block to finish (a counter in
// the workspace, which that block resets).
// PLAIN: RMS or no norm and pairs or no rotation, the one body of
// transform_kind that covers those (its ranges are empty where a part is off).
// 4 x 4096 to 8192 rows of 576 take 19 us (3 TB/s read and written), bound by
// the chain of loads start, page, row, and rows past n_new are loaded before
// that is known; one row each of 8 sequences 7 us.  4 x 8192 whole: 22 us, with
// a layer norm 34, with a rotation by halves 35 to 38; fp32 32, 46, 51 to 54.
template <typename T, int NC, bool PLAIN>
__global__ void __launch_bounds__(kAnyWarps * 32) append_paged_kernel(const __grid_constant__ AppendPagedArgs a) {
  pdl_begin();
  pdl_release();
  constexpr int kLanes = NC == 0 ? 32 : kAppendLanes;
  constexpr int kPer = kAnyWarps * 32 / kLanes;  // rows of a block at a time
  __shared__ float2 tab[NC == 0 ? kAnyWarps : 1][NC == 0 ? kMaxRowDim / 2 : 1];
  __shared__ float rows[NC == 0 ? kAnyWarps : 1][NC == 0 ? kMaxRowDim : 1];
  const int l = threadIdx.x % kLanes;
  const int64_t n_rows = static_cast<int64_t>(a.batch) * a.T;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * kPer; r0 < n_rows; r0 += static_cast<int64_t>(gridDim.x) * kPer) {
    const int64_t r = r0 + threadIdx.x / kLanes;
    const bool row = r < n_rows;
    const T* x = static_cast<const T*>(a.x) + (row ? r : 0) * a.tok_stride;
    Raw8<T> raw[NC == 0 ? 1 : NC];
    if constexpr (NC > 0) {
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        raw[j] = Raw8<T>{};
        if (row && (l + kLanes * j) * 8 < a.dim) raw[j] = load_raw8(x + (l + kLanes * j) * 8);
      }
    }
    const int b = row ? static_cast<int>(r / a.T) : 0, t = row ? static_cast<int>(r - static_cast<int64_t>(b) * a.T) : 0;
    const NewRows nr = new_rows(a, b);
    if (row && t == 0 && l == 0) {
      if (!nr.ok) record_status(a.status, kStatusCapacity);
      else if (!a.lengths_last) a.lengths[b] = static_cast<int>(nr.start) + nr.n;
    }
    const bool mine = row && nr.ok && t < nr.n;
    const int pos = mine ? static_cast<int>(nr.start) + t : 0;
    const int page = mine ? a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / a.page_size] : -1;
    if (__all_sync(0xffffffffu, !mine)) continue;
    const bool there = page >= 0 && page < a.n_pages;
    if (mine && !there && l == 0) record_status(a.status, kStatusIndex);
    T* o = static_cast<T*>(a.data) + (static_cast<int64_t>(there ? page : 0) * a.page_size + pos % a.page_size) * a.dim;
    if constexpr (NC > 0) {
      auto turns = [&](int i, float2 (&out)[4]) {
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k] = turn_for<T>(pos, __ldg(a.tf.inv_freq + i + k));
      };
      auto store = [&](int c, const float (&v)[8]) {
        if (there && c * 8 < a.dim) store8(o + c * 8, v);
      };
      if constexpr (PLAIN) transform_kind<T, NC, kLanes, LI_NORM_RMS, 1>(raw, l, a.tf, turns, store);
      else transform_chunks<T, NC, kLanes>(raw, l, a.tf, turns, store);
    } else if (there) {
      const int warp = threadIdx.x >> 5;
      for (int p = l; p < a.tf.rope_dim / 2; p += 32) tab[warp][p] = turn_for<T>(pos, __ldg(a.tf.inv_freq + p));
      for (int i = l; i < a.dim; i += 32) rows[warp][i] = to_f<T>(x[i]);
      __syncwarp();
      transform_smem(rows[warp], l, a.tf, tab[warp]);
      for (int i = l; i < a.dim; i += 32) o[i] = from_f<T>(rows[warp][i]);
      __syncwarp();
    }
  }
  if (!a.lengths_last) return;
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
cudaError_t norm_rope_t(const NormRopeArgs& a, const NormRopePlan& p, int64_t grid, cudaStream_t st) {
  const dim3 g(static_cast<unsigned>(grid)), b(kVecThreads);
  const size_t smem = static_cast<size_t>(a.n_sets) * a.tab_stride * sizeof(float2);
  if (p.lanes == 0) return launch_pdl(norm_rope_any_kernel<T>, g, dim3(kAnyWarps * 32), smem, st, 1, a);
  if (p.plain) {
    if (p.lanes == 16) return launch_pdl(norm_rope_plain_kernel<T, 4, 16>, g, b, smem, st, 1, a);
    if (p.lanes == 32) return launch_pdl(norm_rope_plain_kernel<T, 4, 32>, g, b, smem, st, 1, a);
    if (p.chunks == 1) return launch_pdl(norm_rope_plain_kernel<T, 1, 8>, g, b, smem, st, 1, a);
    if (p.chunks == 2) return launch_pdl(norm_rope_plain_kernel<T, 2, 8>, g, b, smem, st, 1, a);
    if (p.chunks == 3) return launch_pdl(norm_rope_plain_kernel<T, 3, 8>, g, b, smem, st, 1, a);
    return launch_pdl(norm_rope_plain_kernel<T, 4, 8>, g, b, smem, st, 1, a);
  }
  if (p.lanes == 16) return launch_pdl(norm_rope_vec_kernel<T, 4, 16>, g, b, smem, st, 1, a);
  if (p.lanes == 32) return p.chunks == 1 ? launch_pdl(norm_rope_vec_kernel<T, 1, 32>, g, b, smem, st, 1, a)
                                          : launch_pdl(norm_rope_vec_kernel<T, 4, 32>, g, b, smem, st, 1, a);
  if (p.chunks == 1) return launch_pdl(norm_rope_vec_kernel<T, 1, 8>, g, b, smem, st, 1, a);
  if (p.chunks == 2) return launch_pdl(norm_rope_vec_kernel<T, 2, 8>, g, b, smem, st, 1, a);
  if (p.chunks == 3) return launch_pdl(norm_rope_vec_kernel<T, 3, 8>, g, b, smem, st, 1, a);
  return launch_pdl(norm_rope_vec_kernel<T, 4, 8>, g, b, smem, st, 1, a);
}

template <typename T>
cudaError_t append_paged_t(const AppendPagedArgs& a, bool vec, int num_sms, cudaStream_t st) {
  const int64_t per = vec ? kAnyWarps * 32 / kAppendLanes : kAnyWarps;
  const int64_t blocks = (static_cast<int64_t>(a.batch) * a.T + per - 1) / per;
  const dim3 g(static_cast<unsigned>(blocks < 64 * num_sms ? blocks : 64 * num_sms)), b(kAnyWarps * 32);
  const bool plain = a.tf.norm != LI_NORM_LAYER && (a.tf.rope_dim == 0 || !a.tf.rope_halves);
  if (!vec) return launch_pdl(append_paged_kernel<T, 0, false>, g, b, 0, st, 1, a);
  if (!plain) return launch_pdl(append_paged_kernel<T, 5, false>, g, b, 0, st, 1, a);
  if (a.dim <= 128) return launch_pdl(append_paged_kernel<T, 1, true>, g, b, 0, st, 1, a);
  if (a.dim <= 384) return launch_pdl(append_paged_kernel<T, 3, true>, g, b, 0, st, 1, a);
  return launch_pdl(append_paged_kernel<T, 5, true>, g, b, 0, st, 1, a);
}

}  // namespace

// Whether transform_chunks reaches the partners of a rotation by halves with
// `lanes` lanes a row.
static bool halves_in_reach(const li_row_transform& tf, int lanes) {
  if (tf.rope_dim == 0 || !tf.rope_halves) return true;
  const int c0 = tf.rope_offset / 8, nc = tf.rope_dim / 8;
  if (nc <= lanes) return c0 % lanes + nc <= lanes;
  return c0 % lanes == 0 && (nc / 2) % lanes == 0;
}

NormRopePlan plan_norm_rope(const li_head_rows* sets, int n_sets, bool chunked, int max_dim) {
  // as few lanes a row as hold it in four chunks each, more where a rotation's partners would be out of reach
  static const int kForms[][2] = {{8, 1}, {8, 2}, {8, 3}, {8, 4}, {16, 4}, {32, 1}, {32, 4}};
  if (chunked)
    for (const auto& f : kForms) {
      bool ok = f[0] * f[1] * 8 >= max_dim, plain = f[0] * f[1] != 32 || f[1] == 4;
      for (int i = 0; i < n_sets; ++i) {
        const li_row_transform& t = sets[i].tf;
        ok = ok && halves_in_reach(t, f[0]);
        plain = plain && t.norm != LI_NORM_LAYER && !t.beta &&
                (t.rope_dim == 0 || t.rope_offset / 8 % f[0] + t.rope_dim / 8 <= f[0]);
      }
      if (ok) return {f[0], f[1], 32 / f[0], kVecThreads / 32, plain};
    }
  return {0, 0, 1, kAnyWarps, false};
}

bool append_in_chunks(const li_row_transform& tf, int dim) { return dim <= 640 && halves_in_reach(tf, kAppendLanes); }

cudaError_t launch_norm_rope(const NormRopeArgs& a, li_dtype dtype, const NormRopePlan& p, int64_t grid, cudaStream_t st) {
  return dtype == LI_F32 ? norm_rope_t<float>(a, p, grid, st) : norm_rope_t<__nv_bfloat16>(a, p, grid, st);
}

cudaError_t launch_append_paged(const AppendPagedArgs& a, li_dtype dtype, bool vec, int num_sms, cudaStream_t st) {
  return dtype == LI_F32 ? append_paged_t<float>(a, vec, num_sms, st) : append_paged_t<__nv_bfloat16>(a, vec, num_sms, st);
}

}  // namespace li
