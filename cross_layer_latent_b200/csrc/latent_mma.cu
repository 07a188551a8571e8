// latent_mma.cu -- latent attention in absorbed form on the tensor cores.
//
// For a group of up to N = 64 query rows of one sequence (heads, and without a
// selection also neighbouring queries) and 128 cached rows C a tile:
//     S^T = C Q^T          [128 tokens x N]   A = C (K-major),   B = Q
//     P^T = exp2(S^T - m)                     one token a thread
//     O^T += C[:, :d_v]^T P^T [d_v x N]       A = C (MN-major),  B = P^T
// Tokens lie along the MMA's M, so the N dimension and the work shrink with
// the head count (16, 32 or 64), the same tile in shared memory serves as key
// and as value, and O^T takes 4 N <= 256 tensor-memory columns, which leaves
// room for S^T.  (Heads along M would put 512 columns of output next to the
// scores, more than there are.)  Cost: at N = 64 an MMA is bound by its 6 KB of
// shared-memory operands, 48 cycles instead of 32.
//
// The running maximum m is kept per head and moves only when a score exceeds
// it by more than 8 (in powers of two): then weights stay below 256 and
// neither their bf16 rounding (relative) nor the fp32 sums lose anything, and
// the common tile needs no reduction over the tokens, which lie across lanes.
// The sums of the weights are taken before they are rounded to bf16.
//
// P^T (128 tokens x N) overwrites the tile's last 64-column block, which holds
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

constexpr int kTile = 128;                       // tokens per tile
constexpr int kBlockBytes = kTile * 128;         // 128 tokens x 64 bf16
constexpr int kSoftWarps = 8;                    // two warpgroups, half of the N columns each
constexpr int kMmaWarp = kSoftWarps;
constexpr int kLoadWarps = 4;                    // 32 tokens of a tile each
constexpr int kThreads = 32 * (kSoftWarps + 1 + kLoadWarps);
constexpr int kMaxBufs = 4;
constexpr int kMaxBlocks = 10;
constexpr float kGrow = 8.f;                     // log2 by which a score may exceed the kept maximum
constexpr float kNoMax = -1e30f;
constexpr uint64_t kDrainNs = 1000ull * 1000ull;

struct Smem {
  uint64_t full[kMaxBufs][kMaxBlocks / 2];       // two blocks (a pair) arrived
  uint64_t empty[kMaxBufs][kMaxBlocks / 2];      // they are free again
  uint64_t meta[kMaxBufs];                       // tokens' valid bits written
  uint64_t q_full, q_empty, s_full[2], p_full[2], pv_done, o_full, o_empty, drain;
  uint32_t tmem;
  int abort_flag;
  int first_b, first_g, first_tile;
  int64_t total;
  uint32_t valid[kMaxBufs][4];
  alignas(16) float m[64];
  alignas(16) float alpha[64];
  float part[4][64];
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

template <int N>
__global__ void __launch_bounds__(kThreads, 1) latent_mma_kernel(const __grid_constant__ LatentMmaArgs a) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  constexpr int CW = N / 2;                      // columns of a softmax warpgroup
  const uint32_t q_smem = smem_addr(base);
  const uint32_t tiles_smem = q_smem + a.nb * N * 128;
  Smem& sm = *reinterpret_cast<Smem*>(base + a.nb * N * 128 + static_cast<size_t>(a.bufs) * a.slots * kBlockBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pairs = (a.slots + 1) / 2;
  const WaitCtl wc{&sm.abort_flag, a.status, a.wait_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < a.bufs; ++i) {
      for (int j = 0; j < pairs; ++j) {
        mbar_init(&sm.full[i][j], 32 * kLoadWarps);
        mbar_init(&sm.empty[i][j], 1);
      }
      mbar_init(&sm.meta[i], kLoadWarps);
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
  const uint32_t tmem = sm.tmem;
  const uint32_t o_tmem = tmem, s_tmem = tmem + a.m_blocks * N;

  if (warp < kSoftWarps) {
    // ------------------------------------------------ softmax and output
    const int wg = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const int c0 = wg * CW;                      // first column
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
      float sum[CW];
#pragma unroll
      for (int i = 0; i < CW; ++i) sum[i] = 0.f;
      for (int t = w.s.t0; t < w.s.t1; ++t, ++tile) {
        const int buf = ring.buf, sb = sring.buf;
        bool ok = bounded_wait(&sm.meta[buf], ring.ph, wc);
        ok = bounded_wait(&sm.s_full[sb], sring.ph, wc) && ok;
        ring.step(a.bufs);
        sring.step(a.s_bufs);
        __syncwarp();
        tc_fence_after();
        uint32_t xr[CW];
        tmem_ld<CW>(s_tmem + sb * N + c0 + lanes, xr);
        const bool live = (sm.valid[buf][quad] >> lane) & 1u;
        tmem_wait_ld();
        float x[CW];
#pragma unroll
        for (int i = 0; i < CW; ++i) x[i] = live ? __uint_as_float(xr[i]) * a.scale_log2 : -INFINITY;
        if (column_limits) {
          const int s = t * kTile + quad * 32 + lane;
#pragma unroll
          for (int i = 0; i < CW; ++i)
            if (s >= sm.limit[c0 + i]) x[i] = -INFINITY;
        }
        bool grow = t == w.s.t0;
        if (!grow) {
          float over = -INFINITY;
#pragma unroll
          for (int i = 0; i < CW; i += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&sm.m[c0 + i]);
            over = fmaxf(over, fmaxf(fmaxf(x[i] - m.x, x[i + 1] - m.y), fmaxf(x[i + 2] - m.z, x[i + 3] - m.w)));
          }
          grow = named_bar_any(bar, 128, over > kGrow || !ok);
        }
        if (grow) {
          // new maxima over the tile's 128 tokens, and what they make of the old sums
          if (named_bar_any(bar, 128, !ok)) {
            dead = true;
            break;
          }
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < CW; ++i) {
            const float r = warp_max_f32(x[i]);
            if (lane == i) top = r;
          }
          if (lane < CW) sm.part[quad][c0 + lane] = top;
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
            for (int i = 0; i < CW; i += 4) {
              const float4 f = *reinterpret_cast<const float4*>(&sm.alpha[c0 + i]);
              sum[i] *= f.x;
              sum[i + 1] *= f.y;
              sum[i + 2] *= f.z;
              sum[i + 3] *= f.w;
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
        // weights, their sums, and P^T: token = row of 128 bytes, heads along it
        const uint32_t p_row = tiles_smem + (buf * a.slots + a.slots - 1) * kBlockBytes + (quad * 32 + lane) * 128;
#pragma unroll
        for (int i = 0; i < CW; i += 8) {
          float p[8], m[8];
          *reinterpret_cast<float4*>(&m[0]) = *reinterpret_cast<const float4*>(&sm.m[c0 + i]);
          *reinterpret_cast<float4*>(&m[4]) = *reinterpret_cast<const float4*>(&sm.m[c0 + i + 4]);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = exp2_fast(x[i + e] - m[e]);
            sum[i + e] += p[e];
          }
          const uint32_t chunk = static_cast<uint32_t>((c0 + i) / 8) ^ static_cast<uint32_t>(lane & 7);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(p_row + chunk * 16), "r"(pack_bf16(p[0], p[1])),
                       "r"(pack_bf16(p[2], p[3])), "r"(pack_bf16(p[4], p[5])), "r"(pack_bf16(p[6], p[7]))
                       : "memory");
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[sb]);
      }
      if (dead) break;
      // ---- sums over the tokens
#pragma unroll
      for (int i = 0; i < CW; ++i) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
      }
      named_bar_sync(bar, 128);                  // the last maxima have been read
      if (lane == 0) {
#pragma unroll
        for (int i = 0; i < CW; ++i) sm.part[quad][c0 + i] = sum[i];
      }
      named_bar_sync(bar, 128);
      const bool whole = w.s.t0 == 0 && w.s.t1 == w.s.tiles;
      const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.s.t0 == 0 ? 1 : 0);
      const int64_t row0 = static_cast<int64_t>(w.s.b) * a.rows + r0;
      if (threadIdx.x % 128 < CW) {
        const int c = c0 + threadIdx.x % 128;
        const float l = sm.part[0][c] + sm.part[1][c] + sm.part[2][c] + sm.part[3][c];
        sm.alpha[c] = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
        if (whole) {
          if (a.lse && c < rows) a.lse[row0 + c] = l > 0.f ? (sm.m[c] + log2f(l)) * 0.69314718056f : -INFINITY;
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
      const uint32_t id_s = make_instr_desc(1, 128, N);
      const uint32_t id_o = id_s | kMajorMnA | kMajorMnB;
      Walk w;
      Ring sr, ssr, vr, vsr;                     // tile and score buffers of the next scores, of the next values
      uint32_t seg = 0;
      bool ok = true;
      const uint64_t da0 = desc_sw128(tiles_smem, 16, 1024), db0 = desc_sw128(q_smem, 16, 1024);
      const uint64_t dv0 = desc_sw128(tiles_smem, kBlockBytes, 1024);
      constexpr uint64_t kBlockDesc = kBlockBytes >> 4, kQDesc = (N * 128) >> 4;
      // S^T of the next tile
      auto scores = [&]() {
        const uint32_t d = s_tmem + ssr.buf * N;
        uint64_t da = da0 + sr.buf * a.slots * kBlockDesc, db = db0;
        uint32_t acc = 0;
        for (int p = 0; p < pairs; ++p) {
          const int nblk = min(2, a.nb - 2 * p);
          if (nblk <= 0) break;
          if (!bounded_wait(&sm.full[sr.buf][p], sr.ph, wc)) return false;
          fence_proxy_async_smem();              // rows gathered by cp.async are read by the tensor cores
          tc_fence_after();
          for (int j = 0; j < nblk; ++j, da += kBlockDesc, db += kQDesc) {
            const int ks = 2 * p + j == a.nb - 1 ? a.last_ksteps : 4;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < ks) umma<kKindBF16>(d, da + 2 * kk, db + 2 * kk, id_s, acc);
              acc = 1;
            }
          }
        }
        umma_commit(&sm.s_full[ssr.buf]);
        sr.step(a.bufs);
        ssr.step(a.s_bufs);
        return true;
      };
      for (bool more = w.start(a, sm); more && ok; more = w.next(a), ++seg) {
        if (!(ok = bounded_wait(&sm.q_full, seg & 1u, wc))) break;
        const int nt = w.s.t1 - w.s.t0;
        const int ahead = a.s_bufs - 1;          // scores run one tile ahead where there are two buffers
        int issued = 0;
        for (int t = 0; t < nt && ok; ++t) {
          while (ok && issued < nt && issued <= t + ahead) {
            ok = scores();
            if (++issued == nt) umma_commit(&sm.q_empty);
          }
          if (!ok) break;
          if (t == 0 && seg > 0 && !(ok = bounded_wait(&sm.o_empty, (seg - 1) & 1u, wc))) break;
          if (!(ok = bounded_wait(&sm.p_full[vsr.buf], vsr.ph, wc))) break;
          tc_fence_after();
          const uint64_t dt = dv0 + vr.buf * a.slots * kBlockDesc;
          const uint64_t dp = dt + (a.slots - 1) * kBlockDesc;
          uint64_t* const empty = sm.empty[vr.buf];
          for (int mb = 0; mb < a.m_blocks; ++mb) {
            const uint64_t dv = dt + 2 * mb * kBlockDesc;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma<kKindBF16>(o_tmem + mb * N, dv + kk * 128, dp + kk * 128, id_o, (t > 0 || kk > 0) ? 1u : 0u);
            if (mb < a.m_blocks - 1) umma_commit(&empty[mb]);
          }
          for (int p = a.m_blocks - 1; p < pairs; ++p) umma_commit(&empty[p]);
          umma_commit(&sm.pv_done);
          if (t == nt - 1) umma_commit(&sm.o_full);
          vr.step(a.bufs);
          vsr.step(a.s_bufs);
        }
      }
      // nothing is in flight when the CTA ends, whichever role gave up
      umma_commit(&sm.drain);
      drain_wait(&sm.drain, 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ loads
    const int lw = warp - kMmaWarp - 1;          // 32 tokens of every tile
    Walk w;
    Ring ring;
    uint32_t seg = 0, queries = 0;
    int64_t tile = 0;
    bool ok = true;
    const uint32_t my_rows = tiles_smem + lw * 32 * 128;
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
      auto position = [&](int t) {               // of this lane's token in tile t; -1: none
        const int64_t i = static_cast<int64_t>(t) * kTile + lw * 32 + lane;
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
      int s0 = checked(position(w.s.t0));
      int pg0 = page_of(s0);
      int s1 = position(w.s.t0 + 1);
      for (int t = w.s.t0; t < w.s.t1; ++t, ++tile) {
        const int buf = ring.buf;
        const uint32_t free_phase = ring.ph ^ 1u;
        ring.step(a.bufs);
        if (s0 >= 0 && (pg0 < 0 || pg0 >= a.n_pages)) {
          record_status(a.status, kStatusIndex);
          s0 = -1;
        }
        const int row = s0 >= 0 ? pg0 * a.page_size + s0 % a.page_size : -1;
        const unsigned valid = __ballot_sync(0xffffffffu, s0 >= 0);
        const bool boxes = a.box && valid == 0xffffffffu;
        // next tile's pages, and the positions after that
        s0 = checked(s1);
        pg0 = page_of(s0);
        s1 = position(t + 2);
        const uint32_t dst = my_rows + buf * a.slots * kBlockBytes;
        const bool wait = tile >= a.bufs;
        if (boxes) {
          // lane i < 32 / box loads box i of every block
          const int i = lane & (32 / a.box - 1);
          const int r = __shfl_sync(0xffffffffu, row, i * a.box);
          uint8_t* to = base + (dst - q_smem) + i * a.box * 128;
          for (int p = 0; p < pairs && ok; ++p) {
            const int nblk = min(2, a.nb - 2 * p);
            if (wait) ok = __all_sync(0xffffffffu, bounded_wait(&sm.empty[buf][p], free_phase, wc));
            if (!ok) break;
            if (lane == 0) {
              if (p == 0) {
                sm.valid[buf][lw] = valid;
                mbar_arrive(&sm.meta[buf]);
              }
              if (nblk > 0) {
                mbar_arrive_n(&sm.full[buf][p], 31);
                mbar_arrive_expect_tx(&sm.full[buf][p], nblk * 32 * 128);
              }
            }
            if (lane < 32 / a.box)
              for (int j = 2 * p; j < 2 * p + nblk; ++j) tma_load_2d(to + j * kBlockBytes, &a.map_box, &sm.full[buf][p], 64 * j, r);
          }
        } else {
          // eight lanes a row, four rows at a time, in 16-byte pieces; tokens that nobody attends become zeros
          const int c = lane & 7;
          const uint8_t* src[8];
          uint32_t there = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = __shfl_sync(0xffffffffu, row, 4 * i + (lane >> 3));
            if (r >= 0) there |= 1u << i;
            src[i] = static_cast<const uint8_t*>(a.data) + static_cast<int64_t>(max(r, 0)) * a.dim * 2 + c * 16;
          }
          // 128-byte swizzle: piece c of row r lies at c ^ (r mod 8); rows 4 i + lane / 8
          const uint32_t even = dst + (lane >> 3) * 128 + ((c ^ (lane >> 3)) << 4);
          const uint32_t odd = dst + (lane >> 3) * 128 + ((c ^ (4 + (lane >> 3))) << 4);
          for (int p = 0; p < pairs && ok; ++p) {
            const int nblk = min(2, a.nb - 2 * p);
            if (wait) ok = __all_sync(0xffffffffu, bounded_wait(&sm.empty[buf][p], free_phase, wc));
            if (!ok) break;
            if (p == 0 && lane == 0) {
              sm.valid[buf][lw] = valid;
              mbar_arrive(&sm.meta[buf]);
            }
            if (nblk <= 0) continue;
            for (int j = 2 * p; j < 2 * p + nblk; ++j) {
              const bool in_row = 64 * j + c * 8 < a.dim;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const bool on = in_row && ((there >> i) & 1u);
                cp_async_16_or_zero((i & 1 ? odd : even) + j * kBlockBytes + i * 512, on ? src[i] + j * 128 : static_cast<const uint8_t*>(a.data),
                                    on ? 16u : 0u);
              }
            }
            cp_async_arrive_noinc(&sm.full[buf][p]);
          }
        }
        if (!ok) break;
      }
    }
    // the copies that were issued land before the CTA ends, whichever role gave up
    cp_async_wait_all();
    for (int64_t i = max(tile - a.bufs, int64_t(0)); i < tile; ++i)
      for (int p = 0; 2 * p < a.nb; ++p)
        drain_wait(&sm.full[i % a.bufs][p], static_cast<uint32_t>(i / a.bufs) & 1u, kDrainNs);
    if (lw == 0 && queries > 0) drain_wait(&sm.q_full, (queries - 1) & 1u, kDrainNs);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, a.tmem_cols);
}

// Joins the parts of the groups that more than one CTA worked on.  Block
// (i, c) joins row c of the group that the border after CTA i's share cuts,
// if CTA i is the first to work on that group; four values a thread.
__global__ void __launch_bounds__(128) latent_join_kernel(const __grid_constant__ LatentMmaArgs a) {
  pdl_begin();
  const int64_t i0 = blockIdx.x;
  const int c = blockIdx.y, lane = threadIdx.x & 31;
  const int64_t total = total_tiles(a, lane);
  const int64_t n = shares(a, total);
  if (i0 >= n) return;
  const int64_t border = total * (i0 + 1) / n;
  const Place p = locate(a, border - 1, lane);
  if (p.tile + 1 == p.tiles || p.g * a.N + c >= a.rows) return;
  // the share that holds tile x is the largest i with total * i / n <= x
  const int64_t first = border - 1 - p.tile, last = first + p.tiles - 1;
  if (((first + 1) * n - 1) / total != i0) return;
  const int64_t i1 = ((last + 1) * n - 1) / total;
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
  const int64_t row = static_cast<int64_t>(p.b) * a.rows + p.g * a.N + c;
  const float inv = L > 0.f ? 1.f / L : 0.f;
  const float v[4] = {s.x * inv, s.y * inv, s.z * inv, s.w * inv};
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out) + row * a.d_v + d;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (d + e < a.d_v) out[e] = __float2bfloat16_rn(v[e]);
  if (threadIdx.x == 0 && a.lse) a.lse[row] = L > 0.f ? (M + log2f(L)) * 0.69314718056f : -INFINITY;
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
  a->groups = (a->rows + a->N - 1) / a->N;
  const int64_t q = static_cast<int64_t>(a->nb) * a->N * 128;
  const int64_t room = static_cast<int64_t>(max_smem) - 1024 - q - static_cast<int64_t>(sizeof(Smem));
  a->bufs = static_cast<int>(std::min<int64_t>(kMaxBufs, room / (static_cast<int64_t>(a->slots) * kBlockBytes)));
  if (a->bufs < 1 || a->slots > kMaxBlocks) return false;
  a->s_bufs = a->bufs >= 2 ? 2 : 1;
  // one CTA an SM: tensor memory is taken in full
  a->smem_bytes = static_cast<uint32_t>(std::max<int64_t>(
      1024 + q + static_cast<int64_t>(a->bufs) * a->slots * kBlockBytes + static_cast<int64_t>(sizeof(Smem)), 120 * 1024));
  a->tmem_cols = 32;
  while (a->tmem_cols < static_cast<uint32_t>((a->m_blocks + a->s_bufs) * a->N)) a->tmem_cols <<= 1;
  const int64_t cap = a->sel ? a->k : static_cast<int64_t>(a->max_pages) * a->page_size;
  const int64_t most = static_cast<int64_t>(a->seqs) * a->groups * ((cap + kTile - 1) / kTile);
  a->grid = static_cast<int>(std::min<int64_t>(num_sms, most));
  return true;
}

cudaError_t launch_latent_mma(const LatentMmaArgs& a, cudaStream_t st) {
  return a.N == 64 ? launch_n<64>(a, st) : (a.N == 32 ? launch_n<32>(a, st) : launch_n<16>(a, st));
}

cudaError_t launch_latent_join(const LatentMmaArgs& a, cudaStream_t st) {
  return launch_pdl(latent_join_kernel, dim3(a.grid - 1, std::min(a.N, a.rows)), dim3(128), 0, st, 1, a);
}

}  // namespace li
