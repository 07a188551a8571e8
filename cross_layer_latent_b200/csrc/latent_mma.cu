// latent_mma.cu -- latent attention in absorbed form on the tensor cores.
//
// For a group of up to N = 64 query rows of one sequence (heads, and without a
// selection also neighbouring queries) and 64 cached rows C a tile:
//     S^T = C Q^T          [64 tokens x N]    A = C (K-major),   B = Q
//     P^T = exp2(S^T - m)
//     O^T += C[:, :d_v]^T P^T [d_v x N]       A = C (MN-major),  B = P^T
// Tokens lie along the scores' M, so the N dimension and the work shrink with
// the head count (16, 32 or 64), the same tile in shared memory serves as key
// and as value, and O^T takes 4 N <= 256 tensor-memory columns, which leaves
// room for two S^T.  (Heads along M would put 512 columns of output next to
// the scores, more than there are.)  The tile is 64 tokens because two then
// fit next to the queries (2 x 72 KB + 72 KB at 576 x 64): one is loaded while
// the other is worked on.  With one tile of 128 tokens the loads waited for
// the products and the products for the loads: 10,200 cycles a tile of 128
// against 5,000 of MMA, 189 us for 4 x 131072 rows, against 152 us now.  Cost
// of the small tile: the scores' MMAs run at M = 64, 32 cycles for half the
// tokens (48 at M = 128).
//
// The running maximum m is kept per head and moves only when a score exceeds
// it by more than 8 (in powers of two): then weights stay below 256 and
// neither their bf16 rounding (relative) nor the fp32 sums lose anything, and
// the common tile needs no reduction over the tokens, which lie across lanes.
// The sums of the weights are taken before they are rounded to bf16.
//
// P^T (64 tokens x N) overwrites the tile's last 64-column block, which holds
// rotary columns only and is no longer needed once S^T is complete; where
// the last block belongs to the values, a spare block is set aside.
//
// Each CTA takes an equal, contiguous share of all tiles of all groups, so
// ragged lengths balance; a group cut by a share's border is written as fp32
// partial sums with their maxima, which a second kernel joins in a fixed order.
#include <algorithm>

#include "attention.h"
#include "attn_sm100.cuh"
#include "internal.h"

namespace li {

namespace {

constexpr int kTile = 64;                        // tokens per tile
constexpr int kBlockBytes = kTile * 128;         // 64 tokens x 64 bf16
constexpr int kSoftWarps = 8;                    // two warpgroups, half of the N columns each
constexpr int kMmaWarp = kSoftWarps;
constexpr int kLookWarp = kMmaWarp + 1;           // finds the pool rows of tiles ahead
constexpr int kLoadWarps = 4;
constexpr int kLook = 4;                         // tiles that it may be ahead (a power of two)
constexpr int kThreads = 32 * (kSoftWarps + 2 + kLoadWarps);
constexpr int kMaxBufs = 4;
constexpr int kMaxSlots = 9;
constexpr float kGrow = 8.f;                     // log2 by which a score may exceed the kept maximum
constexpr float kNoMax = -1e30f;
constexpr uint64_t kDrainNs = 1000ull * 1000ull;

struct Smem {
  uint64_t full[kMaxBufs], empty[kMaxBufs];      // a tile arrived, is free again
  uint64_t look_full[kLook], look_empty[kLook];  // pool rows of a tile's tokens
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done, o_full, o_empty, drain;
  uint32_t tmem;
  int abort_flag;
  int first_b, first_g, first_tile;
  int64_t total;
  alignas(8) uint32_t valid[kLook][2];           // tokens that are there
  alignas(16) int row[kLook][kTile];             // their pool rows, -1: nobody attends the token
  alignas(16) float m[64];
  alignas(16) float alpha[64];
  alignas(16) float part[4][64];
  int limit[64];
};

// One group's share of this CTA.
struct Seg {
  int b, g;        // sequence (with a selection: sequence and query), group of rows
  int tiles;       // of the whole group
  int t0, t1;      // this CTA's
};

__device__ __forceinline__ int prefix_len(const LatentMmaArgs& a, int b) {
  const int64_t cap = static_cast<int64_t>(a.max_pages) * a.page_size;
  return static_cast<int>(min(static_cast<int64_t>(max(a.lengths[b], 0)), cap));
}

// A group without positions still gets a tile, which writes its zeros.
__device__ __forceinline__ int group_tiles(const LatentMmaArgs& a, int b) {
  return a.sel ? (a.k + kTile - 1) / kTile : max((prefix_len(a, b) + kTile - 1) / kTile, 1);
}

// Positions that query row r of sequence b sees (r = t * H + h).
__device__ __forceinline__ int row_limit(const LatentMmaArgs& a, int b, int r, int n) {
  if (!a.q_pos) return n;
  const int64_t p = static_cast<int64_t>(a.q_pos[static_cast<int64_t>(b) * a.T + r / a.H]) + 1;
  return static_cast<int>(max(min(p, static_cast<int64_t>(n)), int64_t(0)));
}

// Tiles of all groups of all sequences (the whole warp calls it).
__device__ __forceinline__ int64_t total_tiles(const LatentMmaArgs& a, int lane) {
  if (a.sel) return static_cast<int64_t>(a.seqs) * a.groups * group_tiles(a, 0);
  int64_t n = 0;
  for (int b = lane; b < a.seqs; b += 32) n += group_tiles(a, b);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n * a.groups;
}

// Where tile number x of all lies (the whole warp calls it).
struct Place {
  int b, g, tile, tiles;
};
__device__ __forceinline__ Place locate(const LatentMmaArgs& a, int64_t x, int lane) {
  Place p;
  int b = a.seqs - 1;
  if (a.sel) {
    const int64_t per = static_cast<int64_t>(a.groups) * group_tiles(a, 0);
    b = static_cast<int>(min(x / per, static_cast<int64_t>(b)));
    x -= b * per;
  } else {
    for (int b0 = 0; b0 < a.seqs; b0 += 32) {
      // tiles of 32 sequences, and how many of those end at or before x
      const int64_t c = b0 + lane < a.seqs ? static_cast<int64_t>(group_tiles(a, b0 + lane)) * a.groups : 0;
      int64_t end = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += u;
      }
      const int past = __popc(__ballot_sync(0xffffffffu, b0 + lane < a.seqs && end <= x));
      if (past < min(32, a.seqs - b0)) {
        b = b0 + past;
        x -= __shfl_sync(0xffffffffu, end - c, past);
        break;
      }
      if (b0 + 32 < a.seqs) x -= __shfl_sync(0xffffffffu, end, 31);
    }
  }
  p.b = b;
  p.tiles = group_tiles(a, b);
  p.g = static_cast<int>(min(x / p.tiles, static_cast<int64_t>(a.groups - 1)));
  p.tile = static_cast<int>(x - static_cast<int64_t>(p.g) * p.tiles);
  return p;
}

// CTAs that work: share i is the tiles [total i / n, total (i + 1) / n), none
// of them empty.
__device__ __forceinline__ int64_t shares(const LatentMmaArgs& a, int64_t total) {
  return min(static_cast<int64_t>(a.grid), total);
}

// Walks the groups of this CTA's share.
struct Walk {
  Seg s;
  int64_t left;
  __device__ __forceinline__ bool start(const LatentMmaArgs& a, const Smem& sm) {
    const int64_t n = shares(a, sm.total);
    if (blockIdx.x >= n) return false;
    left = sm.total * (blockIdx.x + 1) / n - sm.total * blockIdx.x / n;
    s.b = sm.first_b;
    s.g = sm.first_g;
    s.tiles = group_tiles(a, s.b);
    s.t0 = sm.first_tile;
    s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), s.t0 + left));
    return true;
  }
  __device__ __forceinline__ bool next(const LatentMmaArgs& a) {
    left -= s.t1 - s.t0;
    if (left <= 0) return false;
    if (++s.g == a.groups) {
      s.g = 0;
      ++s.b;
      s.tiles = group_tiles(a, s.b);
    }
    s.t0 = 0;
    s.t1 = static_cast<int>(min(static_cast<int64_t>(s.tiles), left));
    return true;
  }
};

// Position in the ring of tile buffers, and the phase of its barriers.
struct Ring {
  int buf = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void step(int bufs) {
    if (++buf == bufs) {
      buf = 0;
      ph ^= 1u;
    }
  }
};

// Arrives `n` times at once.
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

// 16 bytes from global to shared memory, zeros where src_bytes is 0.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(src_bytes) : "memory");
}

// Reads a 64-row accumulator: 16 lanes x 8 K columns, rows lane / 4 and
// lane / 4 + 8, columns 8 i + 2 (lane % 4) + {0, 1} in r[4 i ...].
template <int K>
__device__ __forceinline__ void tmem_ld_rows16(uint32_t taddr, uint32_t (&r)[4 * K]) {
  static_assert(K == 1 || K == 2 || K == 4, "8, 16 or 32 columns");
  if constexpr (K == 1) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x1.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(taddr)
                 : "memory");
  } else if constexpr (K == 2) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr)
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1) latent_mma_kernel(const __grid_constant__ LatentMmaArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  constexpr int CW = N / 2;                      // columns of a softmax warpgroup
  const uint32_t q_smem = smem_addr(base);
  const uint32_t tiles_smem = q_smem + a.nb * N * 128;
  Smem& sm = *reinterpret_cast<Smem*>(base + a.nb * N * 128 + static_cast<size_t>(a.bufs) * a.slots * kBlockBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{&sm.abort_flag, a.status, a.wait_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.bufs; ++i) {
      mbar_init(&sm.full[i], 32 * kLoadWarps);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kLook; ++i) {
      mbar_init(&sm.look_full[i], 1);
      mbar_init(&sm.look_empty[i], kSoftWarps + kLoadWarps);
    }
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.p_full[0], kSoftWarps);
    mbar_init(&sm.p_full[1], kSoftWarps);
    mbar_init(&sm.pv_done, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_empty, kSoftWarps);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&a.map_q);
    if (a.box) tma_prefetch_desc(&a.map_box);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&sm.tmem, a.tmem_cols);
    tmem_relinquish();
  }
  pdl_begin();
  if (warp == 0) {
    const int64_t total = total_tiles(a, lane);
    const int64_t n = shares(a, total);
    const Place at = locate(a, total * min(static_cast<int64_t>(blockIdx.x), n - 1) / n, lane);
    if (lane == 0) {
      sm.total = total;
      sm.first_b = at.b;
      sm.first_g = at.g;
      sm.first_tile = at.tile;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_release();
  const uint32_t tmem = sm.tmem;
  const uint32_t o_tmem = tmem, s_tmem = tmem + a.m_blocks * N;

  if (warp < kSoftWarps) {
    // ------------------------------------------------ softmax and output
    const int wg = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int c0 = wg * CW;                      // first column
    constexpr int K = CW / 8;
    // M = 64 accumulators lie in 16 lanes of each quarter; read in 16-lane rows a thread has tokens tok and
    // tok + 8 and of every eight columns two
    const int tok = quad * 16 + (lane >> 2), cl = (lane & 3) * 2;
    const int bar = 1 + wg;
    Walk w;
    Ring ring, sring;                            // tile buffers, score buffers
    uint32_t tile = 0, seg = 0;                  // parities over the CTA's share
    bool dead = false;
    for (bool more = w.start(a, sm); more && !dead; more = w.next(a), ++seg) {
      const int r0 = w.s.g * N;                  // first query row of the group
      const int rows = min(N, a.rows - r0);
      const int n = a.sel ? 0 : prefix_len(a, w.s.b);
      const bool column_limits = !a.sel && a.q_pos && a.T > 1;
      if (threadIdx.x % 128 < CW) {
        const int c = c0 + threadIdx.x % 128;
        sm.m[c] = kNoMax;
        if (column_limits) sm.limit[c] = c < rows ? row_limit(a, w.s.b, r0 + c, n) : 0;
      }
      named_bar_sync(bar, 128);
      float sum[K][2];                           // of this thread's two rows, by column
#pragma unroll
      for (int i = 0; i < K; ++i) sum[i][0] = sum[i][1] = 0.f;
      for (int t = w.s.t0; t < w.s.t1; ++t, ++tile) {
        const int buf = ring.buf, sb = sring.buf;
        const int lk = tile % kLook;
        bool ok = bounded_wait(&sm.look_full[lk], (tile / kLook) & 1u, wc);
        ok = bounded_wait(&sm.s_full[sb], sring.ph, wc) && ok;
        ring.step(a.bufs);
        sring.step(a.s_bufs);
        __syncwarp();
        tc_fence_after();
        uint32_t xr[4 * K];
        tmem_ld_rows16<K>(s_tmem + sb * N + c0 + lanes, xr);
        const uint64_t valid = *reinterpret_cast<const uint64_t*>(sm.valid[lk]) >> tok;
        const bool live[2] = {(valid & 1u) != 0, (valid >> 8 & 1u) != 0};
        tmem_wait_ld();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.look_empty[lk]);
        // x[i][e]: token tok + 8 (e / 2), column c0 + 8 i + cl + e % 2
        float x[K][4];
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[i][e] = live[e >> 1] ? __uint_as_float(xr[4 * i + e]) * a.scale_log2 : -INFINITY;
        if (column_limits) {
          const int at = t * kTile + tok;
#pragma unroll
          for (int i = 0; i < K; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at + 8 * (e >> 1) >= sm.limit[c0 + 8 * i + cl + (e & 1)]) x[i][e] = -INFINITY;
        }
        bool grow = t == w.s.t0;
        if (!grow) {
          float over = -INFINITY;
#pragma unroll
          for (int i = 0; i < K; ++i) {
            const float2 m = *reinterpret_cast<const float2*>(&sm.m[c0 + 8 * i + cl]);
            over = fmaxf(over, fmaxf(fmaxf(x[i][0], x[i][2]) - m.x, fmaxf(x[i][1], x[i][3]) - m.y));
          }
          grow = named_bar_any(bar, 128, over > kGrow || !ok);
        }
        if (grow) {
          // new maxima over the tile's tokens, and what they make of the old sums
          if (named_bar_any(bar, 128, !ok)) {
            dead = true;
            break;
          }
#pragma unroll
          for (int i = 0; i < K; ++i) {
            float2 top = make_float2(fmaxf(x[i][0], x[i][2]), fmaxf(x[i][1], x[i][3]));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
              top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
            }
            if (lane < 4) *reinterpret_cast<float2*>(&sm.part[quad][c0 + 8 * i + cl]) = top;
          }
          named_bar_sync(bar, 128);
          if (threadIdx.x % 128 < CW) {
            const int c = c0 + threadIdx.x % 128;
            const float old = sm.m[c];
            const float now = fmaxf(fmaxf(fmaxf(sm.part[0][c], sm.part[1][c]), fmaxf(sm.part[2][c], sm.part[3][c])), old);
            sm.alpha[c] = exp2_fast(old - now);
            sm.m[c] = now;
          }
          named_bar_sync(bar, 128);
          if (t > w.s.t0) {
            ok = bounded_wait(&sm.pv_done, (tile - 1) & 1u, wc);
            if (named_bar_any(bar, 128, !ok)) {
              dead = true;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int i = 0; i < K; ++i) {
              const float2 f = *reinterpret_cast<const float2*>(&sm.alpha[c0 + 8 * i + cl]);
              sum[i][0] *= f.x;
              sum[i][1] *= f.y;
            }
            constexpr int R = CW < 16 ? CW : 16;   // columns in registers at a time
            for (int u = 0; u < a.m_blocks * (CW / R); ++u) {
              const int cc = (u % (CW / R)) * R;
              const uint32_t at = o_tmem + (u / (CW / R)) * N + c0 + cc + lanes;
              uint32_t o[R];
              tmem_ld<R>(at, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < R; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&sm.alpha[c0 + cc + i]);
                o[i] = __float_as_uint(__uint_as_float(o[i]) * f.x);
                o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) * f.y);
                o[i + 2] = __float_as_uint(__uint_as_float(o[i + 2]) * f.z);
                o[i + 3] = __float_as_uint(__uint_as_float(o[i + 3]) * f.w);
              }
              tmem_st<R>(at, o);
            }
            tmem_wait_st();
          }
        }
        // weights, their sums, and P^T: a token is a row of 128 bytes, heads along it
        const uint32_t p_row = tiles_smem + (buf * a.slots + a.slots - 1) * kBlockBytes + tok * 128 + cl * 2;
#pragma unroll
        for (int i = 0; i < K; ++i) {
          const float2 m = *reinterpret_cast<const float2*>(&sm.m[c0 + 8 * i + cl]);
          const float p0 = exp2_fast(x[i][0] - m.x), p1 = exp2_fast(x[i][1] - m.y);
          const float p2 = exp2_fast(x[i][2] - m.x), p3 = exp2_fast(x[i][3] - m.y);
          sum[i][0] += p0 + p2;
          sum[i][1] += p1 + p3;
          const uint32_t at = p_row + (static_cast<uint32_t>((c0 / 8 + i) ^ (lane >> 2)) << 4);
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(pack_bf16(p0, p1)) : "memory");
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 8 * 128), "r"(pack_bf16(p2, p3)) : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[sb]);
      }
      if (dead) break;
      // ---- sums over the tokens
#pragma unroll
      for (int i = 0; i < K; ++i)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          sum[i][0] += __shfl_xor_sync(0xffffffffu, sum[i][0], o);
          sum[i][1] += __shfl_xor_sync(0xffffffffu, sum[i][1], o);
        }
      named_bar_sync(bar, 128);                  // the last maxima have been read
      if (lane < 4) {
#pragma unroll
        for (int i = 0; i < K; ++i) *reinterpret_cast<float2*>(&sm.part[quad][c0 + 8 * i + cl]) = make_float2(sum[i][0], sum[i][1]);
      }
      named_bar_sync(bar, 128);
      const bool whole = w.s.t0 == 0 && w.s.t1 == w.s.tiles;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.s.t0 == 0 ? 1 : 0);
      const int64_t row0 = static_cast<int64_t>(w.s.b) * a.rows + r0;
      if (threadIdx.x % 128 < CW) {
        const int c = c0 + threadIdx.x % 128;
        const float l = sm.part[0][c] + sm.part[1][c] + sm.part[2][c] + sm.part[3][c];
        sm.alpha[c] = whole ? inverse_sum(l) : 1.f;
        if (whole) {
          if (a.lse && c < rows) a.lse[row0 + c] = row_lse(l, (sm.m[c] + log2f(l)) * 0.69314718056f);
        } else {
          a.part_ml[(slot * 64 + c) * 2] = sm.m[c];
          a.part_ml[(slot * 64 + c) * 2 + 1] = l;
        }
      }
      bool ok = bounded_wait(&sm.o_full, seg & 1u, wc);
      if (named_bar_any(bar, 128, !ok)) {
        dead = true;
        break;
      }
      tc_fence_after();
      for (int mb = 0; mb < a.m_blocks; ++mb) {
        uint32_t o[CW];
        tmem_ld<CW>(o_tmem + mb * N + c0 + lanes, o);
        tmem_wait_ld();
        const int d = mb * 128 + quad * 32 + lane;
        if (d < a.d_v) {
          if (whole) {
            __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + (row0 + c0) * a.d_v + d;
#pragma unroll
            for (int i = 0; i < CW; ++i)
              if (c0 + i < rows) out[static_cast<int64_t>(i) * a.d_v] = __float2bfloat16_rn(__uint_as_float(o[i]) * sm.alpha[c0 + i]);
          } else {
            float* out = a.part_o + (slot * 64 + c0) * a.part_stride + d;
#pragma unroll
            for (int i = 0; i < CW; ++i) out[static_cast<int64_t>(i) * a.part_stride] = __uint_as_float(o[i]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_empty);
      named_bar_sync(bar, 128);                  // m and alpha may be written again
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issue, one lane
    if (elect_one()) {
      const uint32_t id_s = make_instr_desc(1, 64, N);
      const uint32_t id_o = make_instr_desc(1, 128, N) | kMajorMnA | kMajorMnB;
      Walk w;
      Ring sr, ssr, vr, vsr;                     // tile and score buffers of the next scores, of the next values
      uint32_t seg = 0;
      bool ok = true;
      const uint32_t c0 = desc_lo(tiles_smem, 0), q0 = desc_lo(q_smem, 0), v0 = desc_lo(tiles_smem, kBlockBytes);
      constexpr uint32_t kBlockStep = kBlockBytes >> 4, kQStep = (N * 128) >> 4;
      const uint32_t tile_step = a.slots * kBlockStep;
      for (bool more = w.start(a, sm); more && ok; more = w.next(a), ++seg) {
        if (!(ok = bounded_wait(&sm.q_full, seg & 1u, wc))) break;
        if (seg > 0 && !(ok = bounded_wait(&sm.o_empty, (seg - 1) & 1u, wc))) break;
        const int nt = w.s.t1 - w.s.t0;
        // One step at a time, so that each kind's code stays small and warm: the products with the values as
        // soon as the weights are there, else the next tile's scores once it is here.  (Tiles in two to four parts,
        // each loaded and freed by itself, gained nothing and cost up to a tenth.)
        int st = 0, vt = 0;                      // tiles whose scores are issued, tiles done
        uint64_t idle = cycles();
        while (vt < nt) {
          if (vt < st && mbar_test_wait(&sm.p_full[vsr.buf], vsr.ph)) {
            tc_fence_after();
            const uint32_t v = v0 + vr.buf * tile_step, pt = v + (a.slots - 1) * kBlockStep;
            for (int mb = 0; mb < a.m_blocks; ++mb)
              umma_ss_steps<kTile / 16, 128, 128>(o_tmem + mb * N, v + 2 * mb * kBlockStep, pt, id_o, vt > 0 ? 1u : 0u);
            umma_commit(&sm.empty[vr.buf]);
            umma_commit(&sm.pv_done);
            vr.step(a.bufs);
            vsr.step(a.s_bufs);
            if (++vt == nt) umma_commit(&sm.o_full);
          } else if (st < nt && st < vt + a.s_bufs && mbar_test_wait(&sm.full[sr.buf], sr.ph)) {
            fence_proxy_async_smem();            // rows gathered by cp.async are read by the tensor cores
            tc_fence_after();
            const uint32_t d = s_tmem + ssr.buf * N;
            uint32_t c = c0 + sr.buf * tile_step, q = q0;
            for (int j = 0; j < a.nb; ++j, c += kBlockStep, q += kQStep) {
              if (j < a.nb - 1 || a.last_ksteps == 4) {
                umma_ss_steps<4, 2, 2>(d, c, q, id_s, j > 0 ? 1u : 0u);
              } else {
                for (int k = 0; k < a.last_ksteps; ++k) umma_ss_steps<1, 2, 2>(d, c + 2 * k, q + 2 * k, id_s, j + k > 0 ? 1u : 0u);
              }
            }
            umma_commit(&sm.s_full[ssr.buf]);
            sr.step(a.bufs);
            ssr.step(a.s_bufs);
            if (++st == nt) umma_commit(&sm.q_empty);
          } else {
            if (!*wc.abort_flag && cycles() - idle <= a.wait_ns * kCyclesPerNs) continue;
            ok = give_up(wc);
            break;
          }
          idle = cycles();
        }
      }
      // nothing is in flight when the CTA ends, whichever role gave up
      umma_commit(&sm.drain);
      drain_wait(&sm.drain, 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kLookWarp) {
    // ------------------------------------------------ pool rows of the tiles
    Walk w;
    uint32_t tile = 0;
    bool ok = true;
    // the CTAs behind this one that work on its last group, for the join
    if (!a.cuts_by_group && lane == 0 && static_cast<int>(blockIdx.x) < a.n_cuts) a.cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    for (bool more = w.start(a, sm); more && ok; more = w.next(a)) {
      if (lane == 0 && w.s.t0 == 0 && a.n_cuts > 0) {
        const int64_t group = static_cast<int64_t>(w.s.b) * a.groups + w.s.g;
        const bool cut = w.s.t1 < w.s.tiles;
        int4 c = make_int4(0, 0, 0, 0);
        if (cut) {
          // the share that holds tile x is the largest i with total * i / n <= x
          const int64_t n = shares(a, sm.total), last = sm.total * (blockIdx.x + 1) / n - w.s.t1 + w.s.tiles - 1;
          c = make_int4(static_cast<int>(w.s.b * static_cast<int64_t>(a.rows) + w.s.g * N), min(N, a.rows - w.s.g * N), blockIdx.x,
                        static_cast<int>(((last + 1) * n - 1) / sm.total));
        }
        if (a.cuts_by_group) a.cuts[group] = c;
        else if (cut) a.cuts[blockIdx.x] = c;
      }
      // what the group's rows see at most; positions and pages of a tile are read two and one tiles ahead
      const int seq = a.sel ? w.s.b / a.T : w.s.b;
      int lim = prefix_len(a, seq);
      if (a.q_pos) {
        int top = 0;
        const int qa = a.sel ? w.s.b % a.T : w.s.g * N / a.H;
        const int qb = a.sel ? qa : (min(a.rows, (w.s.g + 1) * N) - 1) / a.H;
        for (int t = qa + lane; t <= qb; t += 32) top = max(top, row_limit(a, seq, t * a.H, lim));
        lim = __reduce_max_sync(0xffffffffu, top);
      }
      const int32_t* table = a.page_table + static_cast<int64_t>(seq) * a.max_pages;
      const int32_t* sel = a.sel ? a.sel + static_cast<int64_t>(w.s.b) * a.k : nullptr;
      // a lane looks after tokens lane and lane + 32 of a tile
      auto position = [&](int t, int half) {     // -1: none
        const int64_t i = static_cast<int64_t>(t) * kTile + half * 32 + lane;
        if (t >= w.s.t1) return -1;
        if (!sel) return i < lim ? static_cast<int>(i) : -1;
        return i < a.k ? sel[i] : -1;
      };
      // selected positions outside the prefix are reported and skipped
      auto checked = [&](int s) {
        if (s >= lim) {
          record_status(a.status, kStatusIndex);
          return -1;
        }
        return s < 0 ? -1 : s;
      };
      auto page_of = [&](int s) { return s >= 0 ? table[s / a.page_size] : 0; };
      int s0[2], pg[2], s1[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s0[h] = checked(position(w.s.t0, h));
        s1[h] = position(w.s.t0 + 1, h);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) pg[h] = page_of(s0[h]);
      for (int t = w.s.t0; t < w.s.t1; ++t, ++tile) {
        const int lk = tile % kLook;
        int row[2];
        unsigned valid[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (s0[h] >= 0 && (pg[h] < 0 || pg[h] >= a.n_pages)) {
            record_status(a.status, kStatusIndex);
            s0[h] = -1;
          }
          row[h] = s0[h] >= 0 ? pg[h] * a.page_size + s0[h] % a.page_size : -1;
          valid[h] = __ballot_sync(0xffffffffu, s0[h] >= 0);
          // next tile's pages, and the positions after that
          s0[h] = checked(s1[h]);
          pg[h] = page_of(s0[h]);
          s1[h] = position(t + 2, h);
        }
        if (tile >= kLook) ok = __all_sync(0xffffffffu, bounded_wait(&sm.look_empty[lk], (tile / kLook - 1) & 1u, wc));
        if (!ok) break;
        sm.row[lk][lane] = row[0];
        sm.row[lk][lane + 32] = row[1];
        if (lane == 0) {
          sm.valid[lk][0] = valid[0];
          sm.valid[lk][1] = valid[1];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.look_full[lk]);
      }
    }
  } else {
    // ------------------------------------------------ loads
    const int lw = warp - kLookWarp - 1;
    Walk w;
    Ring ring;
    uint32_t seg = 0, queries = 0;
    int64_t tile = 0;
    bool ok = true;
    // a box of rows to a lane, or eight lanes a row, four rows at a time, in 16-byte pieces (rows 16 lw ... of a
    // tile); 128-byte swizzle: piece c of row r lies at c ^ (r mod 8)
    const int per = kTile >> a.box_shift, at = (lane & (per - 1)) << a.box_shift;
    const int c = lane & 7, r4 = lane >> 3;
    const uint32_t even = (16 * lw + r4) * 128 + ((c ^ r4) << 4), odd = (16 * lw + r4) * 128 + ((c ^ (4 + r4)) << 4);
    for (bool more = w.start(a, sm); more && ok; more = w.next(a), ++seg) {
      // queries of the group (one lane), once the previous group's scores are done
      if (lw == 0) {
        if (seg > 0) ok = __all_sync(0xffffffffu, bounded_wait(&sm.q_empty, (seg - 1) & 1u, wc));
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&sm.q_full, a.nb * N * 128);
          for (int j = 0; j < a.nb; ++j)
            tma_load_3d(base + j * N * 128, &a.map_q, &sm.q_full, 64 * j, w.s.g * N, w.s.b);
        }
        ++queries;
        __syncwarp();
      }
      for (int t = w.s.t0; t < w.s.t1; ++t, ++tile) {
        const int buf = ring.buf;
        const uint32_t free_phase = ring.ph ^ 1u;
        ring.step(a.bufs);
        const int lk = static_cast<int>(tile & (kLook - 1));
        ok = __all_sync(0xffffffffu, bounded_wait(&sm.look_full[lk], static_cast<uint32_t>(tile / kLook) & 1u, wc));
        if (!ok) break;
        const bool boxes = a.box && (sm.valid[lk][0] & sm.valid[lk][1]) == 0xffffffffu;
        int box_row = 0;
        const uint8_t* src[4];
        uint32_t there = 0;
        if (boxes) {
          box_row = sm.row[lk][at & (kTile - 1)];
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = sm.row[lk][16 * lw + 4 * i + r4];
            if (r >= 0) there |= 1u << i;
            src[i] = static_cast<const uint8_t*>(a.data) + static_cast<int64_t>(max(r, 0)) * a.dim * 2 + c * 16;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.look_empty[lk]);
        const uint32_t dst = tiles_smem + buf * a.slots * kBlockBytes;
        if (tile >= a.bufs) ok = __all_sync(0xffffffffu, bounded_wait(&sm.empty[buf], free_phase, wc));
        if (!ok) break;
        if (boxes) {
          // blocks lw, lw + 4, ... are this warp's
          const int mine = lw < a.nb ? (a.nb - lw + kLoadWarps - 1) / kLoadWarps : 0;
          if (lane == 0) {
            mbar_arrive_n(&sm.full[buf], 31);
            mbar_arrive_expect_tx(&sm.full[buf], mine * kBlockBytes);
          }
          if (lane < per)
            for (int j = lw; j < a.nb; j += kLoadWarps)
              tma_load_2d(base + (dst - q_smem) + j * kBlockBytes + at * 128, &a.map_box, &sm.full[buf], 64 * j, box_row);
        } else {
          // tokens that nobody attends, and columns past the row, become zeros
          uint32_t n[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) n[i] = (there >> i) & 1u ? 16u : 0u;
          uint32_t to = dst + even, to_odd = dst + odd;
#pragma unroll 4
          for (int j = 0; j < a.nb - 1; ++j, to += kBlockBytes, to_odd += kBlockBytes) {
#pragma unroll
            for (int i = 0; i < 4; ++i) cp_async_16_or_zero((i & 1 ? to_odd : to) + i * 512, src[i] + j * 128, n[i]);
          }
          const bool in_row = 64 * (a.nb - 1) + c * 8 < a.dim;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            cp_async_16_or_zero((i & 1 ? to_odd : to) + i * 512, in_row ? src[i] + (a.nb - 1) * 128 : static_cast<const uint8_t*>(a.data),
                                in_row ? n[i] : 0u);
          cp_async_arrive_noinc(&sm.full[buf]);
        }
      }
    }
    // the copies that were issued land before the CTA ends, whichever role gave up
    cp_async_wait_all();
    for (int64_t i = max(tile - a.bufs, int64_t(0)); i < tile; ++i)
      drain_wait(&sm.full[i % a.bufs], static_cast<uint32_t>(i / a.bufs) & 1u, kDrainNs);
    if (lw == 0 && queries > 0) drain_wait(&sm.q_full, (queries - 1) & 1u, kDrainNs);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, a.tmem_cols);
}

// Joins the parts of the groups that more than one CTA worked on, one row a
// block, four values a thread; the first CTA of every such group has left in
// `cuts` which CTAs those are.
__global__ void __launch_bounds__(128) latent_join_kernel(const __grid_constant__ LatentMmaArgs a) {
  pdl_begin();
  const int4 cut = a.cuts[blockIdx.x];            // first row, rows, first CTA, last CTA
  const int c = blockIdx.y, lane = threadIdx.x & 31;
  // after a wait that ran out, a group may have left no entry
  if (c >= cut.y || cut.x < 0 || cut.x + static_cast<int64_t>(cut.y) > static_cast<int64_t>(a.seqs) * a.rows || cut.z < 0 ||
      cut.w >= a.grid)
    return;
  const int64_t i0 = cut.z, i1 = cut.w;
  auto slot = [&](int64_t i) { return 2 * i + (i == i0 ? 1 : 0); };
  const int d = threadIdx.x * 4;
  float M = kNoMax, L = 0.f;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int64_t j0 = i0; j0 <= i1; j0 += 32) {
    // the maxima and sums of 32 parts, one a lane; what came before is rescaled to the new maximum
    const int cnt = static_cast<int>(min(i1 - j0 + 1, int64_t(32)));
    float2 ml = make_float2(kNoMax, 0.f);
    if (lane < cnt) ml = *reinterpret_cast<const float2*>(a.part_ml + (slot(j0 + lane) * 64 + c) * 2);
    const float now = fmaxf(M, warp_max_f32(ml.x));
    const float keep = exp2_fast(M - now), mine = exp2_fast(ml.x - now);
    M = now;
    float l = mine * ml.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    L = fmaf(L, keep, l);
    s.x *= keep;
    s.y *= keep;
    s.z *= keep;
    s.w *= keep;
    for (int j1 = 0; j1 < cnt; j1 += 8) {
      float4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (d < a.d_v && j1 + u < cnt) v[u] = *reinterpret_cast<const float4*>(a.part_o + (slot(j0 + j1 + u) * 64 + c) * a.part_stride + d);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float f = __shfl_sync(0xffffffffu, mine, j1 + u);
        if (d < a.d_v && j1 + u < cnt) {
          s.x = fmaf(f, v[u].x, s.x);
          s.y = fmaf(f, v[u].y, s.y);
          s.z = fmaf(f, v[u].z, s.z);
          s.w = fmaf(f, v[u].w, s.w);
        }
      }
    }
  }
  const int64_t row = static_cast<int64_t>(cut.x) + c;
  const float inv = inverse_sum(L);
  const float v[4] = {s.x * inv, s.y * inv, s.z * inv, s.w * inv};
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.d_v + d;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (d + e < a.d_v) out[e] = __float2bfloat16_rn(v[e]);
  if (threadIdx.x == 0 && a.lse) a.lse[row] = row_lse(L, (M + log2f(L)) * 0.69314718056f);
}

template <int N>
cudaError_t launch_n(const LatentMmaArgs& a, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(latent_mma_kernel<N>);
  const cudaError_t e = raise_smem_limit(fn, static_cast<int>(a.smem_bytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(latent_mma_kernel<N>, dim3(a.grid), dim3(kThreads), a.smem_bytes, st, 1, a);
}

}  // namespace

size_t latent_part_bytes(int num_sms, int d_v) {
  return static_cast<size_t>(num_sms) * 2 * 64 * (static_cast<size_t>(latent_part_stride(d_v)) + 2) * 4;
}

bool latent_mma_layout(LatentMmaArgs* a, int num_sms, int max_smem) {
  const int nv = (a->d_v + 63) / 64;
  a->nb = (a->dim + 63) / 64;
  a->last_ksteps = (a->dim - 64 * (a->nb - 1) + 15) / 16;
  a->m_blocks = (a->d_v + 127) / 128;
  // P^T takes the place of the last block if that holds no values
  a->slots = a->nb > nv ? a->nb : a->nb + 1;
  a->N = a->rows > 32 ? 64 : (a->rows > 16 ? 32 : 16);
  const int64_t cap = a->sel ? a->k : static_cast<int64_t>(a->max_pages) * a->page_size;
  const int64_t tiles = static_cast<int64_t>(a->seqs) * ((cap + kTile - 1) / kTile);   // of each group of rows
  // Few tiles leave SMs idle: narrower groups share the rows' work among more of them, and every one writes and joins
  // less, but each reads the tiles again.  Measured (N = 64, narrower): 64 heads x 2048 tokens 16.0, 14.8 us; 64 x 512
  // 13.6, 11.7; 2 x 64 x 500 13.8, 11.9; 128 x 2048 16.4, 17.3, so not where that would leave few SMs idle.
  while (a->N > 16 && tiles * ((a->rows + a->N - 1) / a->N) * 3 <= num_sms) a->N /= 2;
  a->groups = (a->rows + a->N - 1) / a->N;
  const int64_t q = static_cast<int64_t>(a->nb) * a->N * 128;
  const int64_t room = static_cast<int64_t>(max_smem) - 1024 - q - static_cast<int64_t>(sizeof(Smem));
  a->bufs = static_cast<int>(std::min<int64_t>(kMaxBufs, room / (static_cast<int64_t>(a->slots) * kBlockBytes)));
  if (a->bufs < 1 || a->slots > kMaxSlots) return false;
  a->s_bufs = a->bufs >= 2 ? 2 : 1;
  // one CTA an SM: tensor memory is taken in full
  a->smem_bytes = static_cast<uint32_t>(std::max<int64_t>(
      1024 + q + static_cast<int64_t>(a->bufs) * a->slots * kBlockBytes + static_cast<int64_t>(sizeof(Smem)), 120 * 1024));
  a->tmem_cols = 32;
  while (a->tmem_cols < static_cast<uint32_t>((a->m_blocks + a->s_bufs) * a->N)) a->tmem_cols <<= 1;
  const int64_t most = tiles * a->groups;
  a->grid = static_cast<int>(std::min<int64_t>(num_sms, most));
  // a cut for every border between shares, or for every group where those are fewer
  const int64_t n_groups = static_cast<int64_t>(a->seqs) * a->groups;
  a->cuts_by_group = n_groups < a->grid - 1;
  a->n_cuts = static_cast<int>(std::min<int64_t>(n_groups, a->grid - 1));
  return true;
}

cudaError_t launch_latent_mma(const LatentMmaArgs& a, cudaStream_t st) {
  return a.N == 64 ? launch_n<64>(a, st) : (a.N == 32 ? launch_n<32>(a, st) : launch_n<16>(a, st));
}

cudaError_t launch_latent_join(const LatentMmaArgs& a, cudaStream_t st) {
  return launch_pdl(latent_join_kernel, dim3(a.n_cuts, std::min(a.N, a.rows)), dim3(128), 0, st, 1, a);
}

}  // namespace li
