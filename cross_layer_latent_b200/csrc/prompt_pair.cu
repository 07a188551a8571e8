// prompt_pair.cu -- latent attention in expanded form for long prompts: the work
// of prompt_mma.cu by pairs of CTAs.
//
// Two CTAs on neighbouring SMs work as a pair (cta_group::2 MMAs of M = 256).
// A unit of work is 512 queries of one head, as two tiles of 256, half of the
// rows of each in either CTA, and a walk over the keys in tiles of 128:
//     S_q = Q_q K^T      [256 x 128]   A = Q, B = K (both K-major in shared memory)
//     P_q = exp2(S_q - m)              one query row to two threads
//     O_q += P_q V       [256 x 128]   A = P from tensor memory, B = V (MN-major)
// The two tiles alternate: while one's scores are turned into weights, the
// other's products run.  At d_nope + d_rope = 192, d_v = 128 two tiles cost
// 2560 cycles of MMA (12 steps of 64 and 8 of 64 for each).
// The pair halves what an SM holds and reads of the keys and values: 64 keys
// of K and 64 columns of V, 40 KB a key tile instead of 80.  Single CTAs with
// 256 queries have room for 1.6 key tiles next to their queries, and their
// loads, issued 1300 cycles ahead, come 800 too late: 4,100 cycles for the two
// tiles without any softmax, against 2,560 here, which the softmax's chain
// lengthens to about 3,600.  8192 tokens of 32 heads: 682 us (1.01 PFLOP/s).
// Tensor memory is full: S0, S1 (P takes the place of S), O0, O1.  Shared
// memory holds the CTA's rows of both query tiles (96 KB) and a ring of 8 KB
// blocks of 64 rows x 64 columns.  A key tile has two parts in the ring, its K
// blocks (k_nope of the head, then the k_rope that all heads share) and its V
// blocks, each with one barrier in the even CTA, which issues the MMAs.
//
// The running maximum moves only when a row exceeds it by more than 8 (in
// powers of two): weights stay below 256, which costs their bf16 rounding
// (relative) and the fp32 sums nothing, and the outputs are seldom rescaled.
// The sums are taken before the weights are rounded.
//
// The pairs are persistent and take units (prompt_units.cuh) from a counter
// that the even CTA draws on for both (dealt out in turn, the slowest pair had
// 20% more work).
#include <math_constants.h>

#include <algorithm>

#include "attention.h"
#include "attn_sm100.cuh"
#include "internal.h"
#include "prompt_units.cuh"

namespace li {

namespace {

using namespace prompt;

constexpr int kPairRows = 2 * kTile;             // queries of a tile of the pair
constexpr int kRows = 2 * kPairRows;             // and of a unit
constexpr int kQBlockBytes = kTile * 128;        // 128 rows x 64 bf16
constexpr int kBlockBytes = 64 * 128;            // 64 rows x 64 bf16
constexpr int kVBlocks = 2;                      // blocks of a V part: 128 keys x 64 columns
constexpr int kSoftWarps = 16;                   // two warpgroups for each query tile, half of the keys each
constexpr int kMmaWarp = 16, kLoadWarp = 17, kUnitWarp = 18;   // and one that zeroes
constexpr int kThreads = 32 * 20;
constexpr int kMaxRing = 24;
constexpr int kParts = 8;                        // parts in flight at most (a power of two)
constexpr int kPolyOf = 4;                       // of so many pairs of exponentials one is computed on the FMA pipes
constexpr float kGrow = 8.f;
constexpr float kNoMax = -1e30f;
constexpr uint64_t kDrainNs = 1000ull * 1000ull;

struct Smem {
  uint64_t full[kParts], empty[kParts], raw[kParts];   // full, q_full, p_full, o_empty, unit_empty: the even CTA's count
  uint64_t unit_full[2], unit_empty[2];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], o_empty[2], drain;
  Unit unit[2];
  float part[2][2][kTile];                       // by query tile, half of the keys and row
  uint32_t tmem;
  int abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1) prompt_pair_kernel(const __grid_constant__ PromptMmaArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int nkb = a.nope_blocks + a.rope_blocks;
  uint8_t* ring = base + 2 * nkb * kQBlockBytes;
  Smem& sm = *reinterpret_cast<Smem*>(ring + a.ring * kBlockBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const WaitCtl wc{&sm.abort_flag, a.status, a.wait_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sm.full[i], 2);
      mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.raw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      // MMA issue; softmax, loads and zeroes of both CTAs; the odd CTA's unit warp
      mbar_init(&sm.unit_empty[i], 1 + 2 * (kSoftWarps + 2) + 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 16);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_empty[i], 16);
    }
    mbar_init(&sm.q_full, 2);
    mbar_init(&sm.q_empty, 1);
    mbar_init(&sm.drain, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&a.map_q);
    if (a.total_k > 0) {
      tma_prefetch_desc(&a.map_k);
      tma_prefetch_desc(&a.map_v);
    }
  }
  if (warp == kMmaWarp) {
    tmem2_alloc(&sm.tmem, 512);
  }
  pdl_begin();
  tc_fence_before();
  cluster_sync();                                // the barriers of both CTAs are there
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < kSoftWarps) {
    // ------------------------------------------------ softmax and output of query tile q
    // A row has two threads, one for 64 of a tile's keys: with 128 keys a thread, a warp alone on its scheduler
    // took 2100 cycles a tile, most of them waiting for its own results.
    const int q = warp >> 3, half = (warp >> 2) & 1, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_tm = tmem + q * 128 + lanes, o_tm = tmem + 256 + q * 128 + lanes;
    const int r = quad * 32 + lane;
    const int bar = 1 + q * 4 + quad;            // the two warps of these 32 rows
    const uint32_t u_bar[2] = {cluster_addr(&sm.unit_empty[0], 0), cluster_addr(&sm.unit_empty[1], 0)};
    constexpr int my_cols = 64;                  // output columns of a half
    const uint32_t p_bar = cluster_addr(&sm.p_full[q], 0), o_bar = cluster_addr(&sm.o_empty[q], 0);
    uint32_t tile = 0, outs = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      ok = bounded_wait_cluster(&sm.unit_full[un & 1], (un >> 1) & 1u, wc);
      ok = !named_bar_any(bar, 64, !ok);
      if (!ok) break;
      const Unit u = sm.unit[un & 1];
      if (u.h < 0) break;
      const int n = key_tiles<kRows>(a, u, q);
      const int i = u.row0 + q * kPairRows + rank * kTile + r;
      const int lim = i < u.nq ? key_limit(a, u, i) : u.nk;
      float m = kNoMax, l = 0.f;
      for (int t = 0; t < n; ++t, ++tile) {
        ok = bounded_wait(&sm.s_full[q], tile & 1u, wc);
        __syncwarp();
        tc_fence_after();
        float x[64];
        {
          uint32_t xr[2][32];
          tmem_ld<32>(s_tm + 64 * half, xr[0]);
          tmem_ld<32>(s_tm + 64 * half + 32, xr[1]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 64; ++c) x[c] = __uint_as_float(xr[c / 32][c % 32]);
        }
        if (a.negate) {
#pragma unroll
          for (int c = 0; c < 64; ++c) x[c] = -x[c];
        }
        const int left = lim - t * kTile - 64 * half;
        if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= left) x[c] = -INFINITY;
        }
        float top4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 60; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top4[e] = fmaxf(fmaxf(top4[e], x[c + e]), x[c + 4 + e]);
        float top = fmaxf(fmaxf(fmaxf(top4[0], x[60]), fmaxf(top4[1], x[61])), fmaxf(fmaxf(top4[2], x[62]), fmaxf(top4[3], x[63])));
        // every score of the tile has been read when this returns
        if (named_bar_any(bar, 64, (top - m) * a.scale_log2 > kGrow || !ok)) {
          sm.part[q][half][r] = top;
          if (named_bar_any(bar, 64, !ok)) {
            ok = false;
            break;
          }
          top = fmaxf(top, sm.part[q][half ^ 1][r]);
          const bool grow = (top - m) * a.scale_log2 > kGrow;
          if (__any_sync(0xffffffffu, grow)) {
            const float now = grow ? top : m;
            const float keep = exp2_fast((m - now) * a.scale_log2);
            m = now;
            l *= keep;
            if (t > 0) {
              // the previous tile's product is complete: s_full was committed after it
#pragma unroll 1
              for (int c = half * my_cols; c < (half + 1) * my_cols; c += 16) {
                uint32_t o[16];
                tmem_ld<16>(o_tm + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
                tmem_st<16>(o_tm + c, o);
              }
            }
          }
        }
        const float ms = m * a.scale_log2;
        const uint64_t sc = pair(a.scale_log2, a.scale_log2), off = pair(-ms, -ms);
        uint64_t s0 = 0, s1 = 0;                 // pairs of zeros
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const uint64_t y = fma2(pair(x[32 * c + 2 * e], x[32 * c + 2 * e + 1]), sc, off);
            float2 p;
            if (e % kPolyOf == kPolyOf - 1) {
              p = exp2_poly(y);
            } else {
              const float2 v = unpair(y);
              p = make_float2(exp2_fast(v.x), exp2_fast(v.y));
            }
            if (e & 1) s1 = add2(s1, pair(p.x, p.y));
            else s0 = add2(s0, pair(p.x, p.y));
            pk[e] = pack_bf16(p.x, p.y);
          }
          tmem_st<16>(s_tm + 32 * half + 16 * c, pk);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_at(p_bar);
        const float2 sum = unpair(add2(s0, s1));
        l += sum.x + sum.y;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed_at(u_bar[un & 1]);   // the unit's numbers have been used
      if (u.row0 + q * kPairRows >= u.nq) continue;
      // the row's sum: both halves, after the last tile's maxima have been read
      named_bar_sync(bar, 64);
      sm.part[q][half][r] = l;
      ok = n == 0 || bounded_wait(&sm.o_full[q], outs & 1u, wc);
      if (named_bar_any(bar, 64, !ok)) {
        ok = false;
        break;
      }
      l += sm.part[q][half ^ 1][r];
      // What exp2_poly makes of scores that are not finite shows in the sum, which is 1 or nearly, its maximum's weight,
      // to 256 a key for a row that has a softmax.  Below: hidden keys alone, or scores that are all -inf.  Above: a NaN.
      if (l < 0x1p-64f) l = 0.f;
      if (m == INFINITY || l > 0x1p100f) l = CUDART_NAN_F;
      tc_fence_after();
      const float inv = inverse_sum(l);
      const int64_t row = static_cast<int64_t>(u.q0 + i) * a.H + u.h;
      for (int c = half * my_cols; c < min((half + 1) * my_cols, a.d_v); c += 32) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld<32>(o_tm + c, o);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (i < u.nq) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
          store_row32(static_cast<__nv_bfloat16*>(a.out) + row * a.d_v + c, w, a.d_v - c, a.wide_out);
        }
      }
      if (a.lse && half == 0 && i < u.nq) a.lse[row] = row_lse(l, (m * a.scale_log2 + log2f(l)) * 0.69314718056f);
      if (n > 0) {
        ++outs;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_at(o_bar);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issue, one lane of the even CTA
    if (rank == 0 && elect_one()) {
      const uint32_t id_s = make_instr_desc(1, 256, 128);
      const uint32_t id_o = id_s | kMajorMnB;
      const uint32_t q0 = desc_lo(smem_addr(base), 0), r0 = desc_lo(smem_addr(ring), 0);
      constexpr uint32_t kBlockStep = kBlockBytes >> 4, kQStep = kQBlockBytes >> 4;
      const int per = nkb + kVBlocks;
      int kc = 0, vc = nkb;                      // ring positions of the next K part and V part
      uint32_t kp = 0, vp = 1;                   // and their numbers
      auto advance = [&](int& c, uint32_t& p) {
        c += per;
        if (c >= a.ring) c -= a.ring;
        p += 2;
      };
      uint32_t ptile[2] = {0, 0}, outs[2] = {0, 0};
      bool ok = true;
      if (vc >= a.ring) vc -= a.ring;
      uint32_t busy = 0;
      for (uint32_t un = 0; ok; ++un) {
        if (!(ok = bounded_wait(&sm.unit_full[un & 1], (un >> 1) & 1u, wc))) break;
        const Unit u = sm.unit[un & 1];
        if (u.h < 0) break;
        const int n0 = key_tiles<kRows>(a, u, 0), n1 = key_tiles<kRows>(a, u, 1), nt = max(n0, n1);
        mbar_arrive(&sm.unit_empty[un & 1]);
        if (nt == 0) continue;
        if (!(ok = bounded_wait_cluster(&sm.q_full, busy & 1u, wc))) break;
        ++busy;
        bool k_here = false, v_here = false;
        // S_q of the next K part; `last`: no other tile needs the part
        auto scores = [&](int q, bool last) {
          if (!k_here && !bounded_wait_cluster(&sm.full[kp % kParts], (kp / kParts) & 1u, wc)) return false;
          k_here = true;
          tc_fence_after();
          uint32_t da = q0 + q * nkb * kQStep;
          int s = kc;
          for (int j = 0; j < nkb; ++j, da += kQStep) {
            const uint32_t db = r0 + s * kBlockStep;
            if (++s == a.ring) s = 0;
            const int ks = j == a.nope_blocks - 1 ? a.nope_ksteps : (j == nkb - 1 ? a.rope_ksteps : 4);
            if (ks == 4) {
              umma2_ss_steps<4, 2, 2>(tmem + q * 128, da, db, id_s, j > 0 ? 1u : 0u);
            } else {
              for (int k = 0; k < ks; ++k) umma2_ss_steps<1, 2, 2>(tmem + q * 128, da + 2 * k, db + 2 * k, id_s, j + k > 0 ? 1u : 0u);
            }
          }
          if (last) {
            umma2_commit(&sm.empty[kp % kParts]);
            advance(kc, kp);
            k_here = false;
          }
          umma2_commit(&sm.s_full[q]);
          return true;
        };
        // O_q of the next V part
        auto values = [&](int q, bool first, bool final, bool last) {
          if (first && outs[q] > 0 && !bounded_wait_cluster(&sm.o_empty[q], (outs[q] - 1) & 1u, wc)) return false;
          if (!v_here && !bounded_wait_cluster(&sm.full[vp % kParts], (vp / kParts) & 1u, wc)) return false;
          v_here = true;
          if (!bounded_wait_cluster(&sm.p_full[q], ptile[q] & 1u, wc)) return false;
          ++ptile[q];
          tc_fence_after();
          int s = vc;
          for (int j = 0; j < kVBlocks; ++j) {   // 64 keys each
            umma2_ts_steps<4, 128>(tmem + 256 + q * 128, tmem + q * 128 + j * 32, r0 + s * kBlockStep, id_o, first && j == 0 ? 0u : 1u);
            if (++s == a.ring) s = 0;
          }
          if (last) {
            umma2_commit(&sm.empty[vp % kParts]);
            advance(vc, vp);
            v_here = false;
          }
          if (final) {
            umma2_commit(&sm.o_full[q]);
            ++outs[q];
          }
          return true;
        };
        for (int t = -1; t < nt && ok; ++t) {
          for (int q = 0; q < 2 && ok; ++q) {
            const int n = q == 0 ? n0 : n1;
            if (t >= 0 && t < n) ok = values(q, t == 0, t == n - 1, q == 1 || t >= n1);
            if (ok && t + 1 < n) ok = scores(q, q == 1 || t + 1 >= n1);
          }
          if (ok && t + 2 == nt) umma2_commit(&sm.q_empty);
        }
      }
      // nothing is in flight when the CTA ends, whichever role gave up
      umma2_commit(&sm.drain);
      drain_wait(&sm.drain, 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------ loads
    uint32_t part = 0, tail = 0, busy = 0;       // parts loaded, parts known to be free again, units with keys
    int free_blocks = a.ring, slot = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      ok = __all_sync(0xffffffffu, bounded_wait_cluster(&sm.unit_full[un & 1], (un >> 1) & 1u, wc));
      if (!ok) break;
      const Unit u = sm.unit[un & 1];
      if (u.h < 0) break;
      const int n0 = key_tiles<kRows>(a, u, 0), n1 = key_tiles<kRows>(a, u, 1), nt = max(n0, n1);
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed_at(cluster_addr(&sm.unit_empty[un & 1], 0));
      if (nt == 0) continue;
      int good = 1;
      if (lane == 0) {
        // a part of `blocks` blocks of the ring, once they are free
        auto room = [&](int blocks) {
          while (free_blocks < blocks || part - tail >= kParts) {
            if (!bounded_wait(&sm.empty[tail % kParts], (tail / kParts) & 1u, wc)) return false;
            free_blocks += tail & 1 ? kVBlocks : nkb;
            ++tail;
          }
          free_blocks -= blocks;
          return true;
        };
        auto next_slot = [&]() {
          uint8_t* p = ring + slot * kBlockBytes;
          if (++slot == a.ring) slot = 0;
          return p;
        };
        if (busy > 0) good = bounded_wait(&sm.q_empty, (busy - 1) & 1u, wc);
        if (good) {
          const int tiles = n1 > 0 ? 2 : 1;
          const uint32_t q_bar = cluster_addr(&sm.q_full, 0);
          mbar_arrive_expect_tx_at(q_bar, tiles * nkb * kQBlockBytes);
          ++busy;
          for (int q = 0; q < tiles; ++q)
            for (int j = 0; j < nkb; ++j)
              tma2_load_3d(base + (q * nkb + j) * kQBlockBytes, &a.map_q, q_bar,
                           j < a.nope_blocks ? 64 * j : a.d_nope + 64 * (j - a.nope_blocks), u.h,
                           u.q0 + u.row0 + q * kPairRows + rank * kTile);
          for (int t = 0; t < nt; ++t) {
            const int row = u.k0 + t * kTile;
            if (!(good = room(nkb))) break;
            uint32_t bar = cluster_addr(&sm.full[part % kParts], 0);
            mbar_arrive_expect_tx_at(bar, nkb * kBlockBytes);
            for (int j = 0; j < nkb; ++j) {
              if (j < a.nope_blocks) tma2_load_3d(next_slot(), &a.map_k, bar, 64 * j, u.h, row + rank * 64);
              else tma2_load_2d(next_slot(), &a.map_kr, bar, 64 * (j - a.nope_blocks), row + rank * 64);
            }
            ++part;
            if (!(good = room(kVBlocks))) break;
            // values past the sequence's end are zeroed before anyone reads them
            bar = (t + 1) * kTile > u.nk ? smem_addr(&sm.raw[part % kParts]) : cluster_addr(&sm.full[part % kParts], 0);
            mbar_arrive_expect_tx_at(bar, kVBlocks * kBlockBytes);
            for (int j = 0; j < kVBlocks; ++j) tma2_load_3d(next_slot(), &a.map_v, bar, 64 * rank, u.h, row + 64 * j);
            ++part;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, good, 0) != 0;
    }
    if (lane == 0) {
      // the copies that were issued land before the pair ends, whichever role gave up (the even CTA's barriers
      // count both CTAs' copies, and both stay until the end)
      if (rank == 0) {
        for (uint32_t f = part > kParts ? part - kParts : 0; f < part; ++f)
          drain_wait(&sm.full[f % kParts], (f / kParts) & 1u, kDrainNs);
        if (busy > 0) drain_wait(&sm.q_full, (busy - 1) & 1u, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == kUnitWarp) {
    // ------------------------------------------------ units, found ahead by the even CTA for both
    if (rank == 0) {
      const int64_t total = all_units<kRows>(a, lane);
      int64_t next = blockIdx.x / 2;
      for (uint32_t un = 0;; ++un) {
        const Unit u = find_unit<kRows>(a, next, total, lane);
        if (u.h >= 0 && lane == 0) next = static_cast<int64_t>(gridDim.x / 2) + atomicAdd(a.next_unit, 1u);
        next = __shfl_sync(0xffffffffu, next, 0);
        if (un >= 2 && !__all_sync(0xffffffffu, bounded_wait_cluster(&sm.unit_empty[un & 1], ((un >> 1) - 1) & 1u, wc))) break;
        if (lane == 0) {
          sm.unit[un & 1] = u;
          mbar_arrive(&sm.unit_full[un & 1]);
          const uint32_t to = cluster_addr(&sm.unit[un & 1], 1), bar = cluster_addr(&sm.unit_full[un & 1], 1);
          st_async_v4(to, make_uint4(u.q0, u.nq, u.k0, u.nk), bar);
          st_async_v4(to + 16, make_uint4(u.row0, u.h, 0u, 0u), bar);
        }
        if (u.h < 0) break;
      }
    } else {
      // the odd CTA expects them
      for (uint32_t un = 0;; ++un) {
        if (lane == 0) mbar_arrive_expect_tx(&sm.unit_full[un & 1], sizeof(Unit));
        if (!__all_sync(0xffffffffu, bounded_wait_cluster(&sm.unit_full[un & 1], (un >> 1) & 1u, wc))) break;
        if (sm.unit[un & 1].h < 0) break;
        // read: the unit after the next may take its place
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed_at(cluster_addr(&sm.unit_empty[un & 1], 0));
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ zeroes behind a sequence's last values
    int vc = nkb % a.ring;                       // ring position of the unit's first V part
    uint32_t vp = 1, raw_phase = 0;
    const int per = nkb + kVBlocks;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      ok = __all_sync(0xffffffffu, bounded_wait_cluster(&sm.unit_full[un & 1], (un >> 1) & 1u, wc));
      if (!ok) break;
      const Unit u = sm.unit[un & 1];
      if (u.h < 0) break;
      const int nt = max(key_tiles<kRows>(a, u, 0), key_tiles<kRows>(a, u, 1));
      if (nt > 0 && nt * kTile > u.nk) {
        const uint32_t p = vp + 2 * (nt - 1);
        const int keep = u.nk - (nt - 1) * kTile;
        int s = (vc + (nt - 1) * per) % a.ring;
        ok = __all_sync(0xffffffffu, bounded_wait_sleep(&sm.raw[p % kParts], (raw_phase >> (p % kParts)) & 1u, wc));
        if (!ok) break;
        raw_phase ^= 1u << (p % kParts);
        for (int j = 0; j < kVBlocks; ++j) {
          uint4* rows = reinterpret_cast<uint4*>(ring + s * kBlockBytes);
          for (int x = max(keep - 64 * j, 0) * 8 + lane; x < 64 * 8; x += 32) rows[x] = make_uint4(0u, 0u, 0u, 0u);
          if (++s == a.ring) s = 0;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_release_at(cluster_addr(&sm.full[p % kParts], 0));
      }
      vc = (vc + nt * per) % a.ring;
      vp += 2 * nt;
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed_at(cluster_addr(&sm.unit_empty[un & 1], 0));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // nothing of the other CTA reaches this one any more, but for the last commit's arrival, which the even CTA has seen
  cluster_sync();
  if (rank == 1 && threadIdx.x == 0) {
    drain_wait(&sm.drain, 0, kDrainNs);
    // after a wait that ran out, copies that only the even CTA's barriers count may be under way to this one
    if (sm.abort_flag) delay_ns(kDrainNs);
  }
  if (warp == kMmaWarp) tmem2_dealloc(tmem, 512);
  // the last pair leaves the counters as it found them
  if (rank == 0 && threadIdx.x == 0) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.done) : "memory");
    if (prev == gridDim.x / 2 - 1) {
      *a.next_unit = 0u;
      *a.done = 0u;
    }
  }
}

}  // namespace

bool prompt_pair_layout(PromptMmaArgs* a, int num_sms, int max_smem) {
  a->nope_blocks = (a->d_nope + 63) / 64;
  a->rope_blocks = (a->d_rope + 63) / 64;
  a->box_rows = 64;
  a->nope_ksteps = (a->d_nope - 64 * (a->nope_blocks - 1) + 15) / 16;
  a->rope_ksteps = (a->d_rope + 15) / 16;
  const int nkb = a->nope_blocks + a->rope_blocks;
  const int64_t q = 2ll * nkb * kQBlockBytes;
  const int64_t room = static_cast<int64_t>(max_smem) - 1024 - q - static_cast<int64_t>(sizeof(Smem));
  a->ring = static_cast<int>(std::min<int64_t>(kMaxRing, room / kBlockBytes));
  if (a->ring < nkb + kVBlocks) return false;
  a->smem_bytes = static_cast<uint32_t>(1024 + q + a->ring * kBlockBytes + sizeof(Smem));
  const int64_t units = (static_cast<int64_t>(a->total_q) / kRows + a->batch) * a->H;
  a->grid = 2 * static_cast<int>(std::min<int64_t>(num_sms / 2, units));
  return true;
}

cudaError_t launch_prompt_pair(const PromptMmaArgs& a, cudaStream_t st) {
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prompt_pair_kernel), static_cast<int>(a.smem_bytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_pair_kernel, dim3(a.grid), dim3(kThreads), a.smem_bytes, st, 2, a);
}

}  // namespace li
