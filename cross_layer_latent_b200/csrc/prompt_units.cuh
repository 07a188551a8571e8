// prompt_units.cuh -- what the two prompt attention kernels share: how the
// queries of ragged sequences are cut into units of work.
//
// A unit is kRows queries of one head, as two query tiles of kRows / 2.  Units
// of a sequence are ordered by groups of heads whose keys and values fit the
// L2 together, longest first within a group.
#pragma once

#include "attention.h"

namespace li {
namespace prompt {

constexpr int kTile = 128;                       // keys of a tile
constexpr int64_t kL2Share = int64_t(48) << 20;  // keys and values of the heads that run together

struct alignas(16) Unit {
  int q0, nq, k0, nk;    // rows of the sequence in q and k
  int row0, h;           // first query of the unit; h < 0: no more units
  int pad[2];
};

// Keys that query i of the sequence sees.
__device__ __forceinline__ int key_limit(const PromptMmaArgs& a, const Unit& u, int i) {
  if (!a.causal) return u.nk;
  const int64_t n = static_cast<int64_t>(i) + 1 + u.nk - u.nq;
  return static_cast<int>(max(min(n, static_cast<int64_t>(u.nk)), int64_t(0)));
}
// Key tiles of query tile q (0 or 1) of a unit of kRows queries: those that its last row sees.
template <int kRows>
__device__ __forceinline__ int key_tiles(const PromptMmaArgs& a, const Unit& u, int q) {
  const int first = u.row0 + q * (kRows / 2);
  if (first >= u.nq) return 0;
  return (key_limit(a, u, min(first + kRows / 2, u.nq) - 1) + kTile - 1) / kTile;
}

__device__ __forceinline__ int seq_rows(const int32_t* cu, int b, int total, int* first) {
  const int x = min(max(cu[b], 0), total);
  *first = x;
  return min(max(cu[b + 1], x), total) - x;
}
__device__ __forceinline__ int seq_queries(const PromptMmaArgs& a, int b, int* first) {
  return min(seq_rows(a.cu_q, b, a.total_q, first), a.max_q);
}
template <int kRows>
__device__ __forceinline__ int seq_units(const PromptMmaArgs& a, int b) {
  int f;
  return (seq_queries(a, b, &f) + kRows - 1) / kRows;
}

// Unit number x of all `total` (the whole warp calls it).
template <int kRows>
__device__ __forceinline__ Unit find_unit(const PromptMmaArgs& a, int64_t x, int64_t total, int lane) {
  Unit u;
  u.h = -1;
  if (x >= total) return u;
  int b = a.batch - 1;
  for (int b0 = 0; b0 < a.batch; b0 += 32) {
    const int64_t c = b0 + lane < a.batch ? static_cast<int64_t>(seq_units<kRows>(a, b0 + lane)) * a.H : 0;
    int64_t end = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    const int past = __popc(__ballot_sync(0xffffffffu, b0 + lane < a.batch && end <= x));
    if (past < min(32, a.batch - b0)) {
      b = b0 + past;
      x -= __shfl_sync(0xffffffffu, end - c, past);
      break;
    }
    x -= __shfl_sync(0xffffffffu, end, 31);
  }
  u.nq = seq_queries(a, b, &u.q0);
  u.nk = seq_rows(a.cu_k, b, a.total_k, &u.k0);
  // causal limits go by the whole sequence, also where max_q cuts it
  int f;
  const int whole = seq_rows(a.cu_q, b, a.total_q, &f);
  if (a.causal && whole > u.nq) u.nk = max(u.nk - (whole - u.nq), 0);
  const int tiles = (u.nq + kRows - 1) / kRows;
  const int64_t per_head = static_cast<int64_t>(max(u.nk, 1)) * (a.d_nope + a.d_v) * 2;
  const int hg = static_cast<int>(max(min(kL2Share / per_head, static_cast<int64_t>(a.H)), int64_t(1)));
  const int64_t per_group = static_cast<int64_t>(hg) * tiles;
  const int g = static_cast<int>(x / per_group);
  const int r = static_cast<int>(x - g * per_group);
  const int heads = min(hg, a.H - g * hg);
  u.h = g * hg + r % heads;
  u.row0 = (tiles - 1 - r / heads) * kRows;
  return u;
}

// Units of all sequences (the whole warp calls it).
template <int kRows>
__device__ __forceinline__ int64_t all_units(const PromptMmaArgs& a, int lane) {
  int64_t units = 0;
  for (int b = lane; b < a.batch; b += 32) units += seq_units<kRows>(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
  return units * a.H;
}

// 32 bytes in one store (p 32-byte aligned).
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// The first min(n, 32) of 32 output columns of a row (n a multiple of 8, of 16 if wide).  Rows lie apart, so a store
// takes as many cycles as it has rows: 32 bytes a thread where rows are aligned to them (8192 tokens of 32 heads: 694
// us with 16 bytes, 682 with 32).
__device__ __forceinline__ void store_row32(__nv_bfloat16* out, const uint32_t* w, int n, int wide) {
  if (wide) {
#pragma unroll
    for (int e = 0; e < 16; e += 8)
      if (2 * e < n) st_global_32(out + 2 * e, &w[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 16; e += 4)
      if (2 * e < n) *reinterpret_cast<uint4*>(out + 2 * e) = make_uint4(w[e], w[e + 1], w[e + 2], w[e + 3]);
  }
}

}  // namespace prompt
}  // namespace li
