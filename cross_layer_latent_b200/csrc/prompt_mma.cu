// prompt_mma.cu -- latent attention in expanded form on the tensor cores:
// causal (or full) attention of ragged prompts, head by head.
//
// A unit of work is 256 queries of one head, as two tiles of 128, and a walk
// over the keys in tiles of 128:
//     S_q = Q_q K^T      [128 x 128]   A = Q, B = K (both K-major in shared memory)
//     P_q = exp2(S_q - m)              one query row a thread
//     O_q += P_q V       [128 x d_v]   A = P from tensor memory, B = V (MN-major)
// The two tiles alternate: while one's scores are turned into weights, the
// other's products run, so the tensor cores wait for neither.  At d_nope +
// d_rope = 192, d_v = 128 a tile pair costs 2560 cycles of MMA (12 steps of 64
// and 8 of 64 for each tile) against 2048 cycles of special-function unit (128
// x 128 exponentials a tile at 16 a cycle): the MMAs bound it.
// Tensor memory is full: S0, S1 (P takes the place of S), O0, O1.  Shared
// memory holds both query tiles (96 KB) and a ring of 16 KB blocks, 128
// tokens x 64 columns of K (k_nope of the head, then the k_rope that all heads
// share) or of V.  A key tile has two parts in the ring, its K blocks and its
// V blocks, each with one barrier: eight blocks hold 1.6 tiles, and a part is
// loaded at least 1280 cycles of MMA before it is needed.
//
// The running maximum moves only when a row exceeds it by more than 8 (in
// powers of two): weights stay below 256, which costs their bf16 rounding
// (relative) and the fp32 sums nothing, and the outputs are seldom rescaled.
// The sums are taken before the weights are rounded.
//
// CTAs are persistent and take the next unit (prompt_units.cuh) from a counter.
// 4 sequences of 1500 to 2048 x 32 heads take 190 us (0.68 PFLOP/s), 8 of up to
// 257 x 16 heads 16 us.
// prompt_pair.cu does the same work by pairs of CTAs, better for long
// sequences: there the loads of this kernel, of whole key tiles for one SM,
// come too late.
#include <algorithm>

#include "attention.h"
#include "attn_sm100.cuh"
#include "internal.h"
#include "prompt_units.cuh"

namespace li {

namespace {

using namespace prompt;

constexpr int kRows = 2 * kTile;                 // queries of a unit
constexpr int kBlockBytes = kTile * 128;
constexpr int kSoftWarps = 8;                    // a warpgroup for each query tile
constexpr int kMmaWarp = 8, kLoadWarp = 9;      // and one that zeroes
constexpr int kThreads = 32 * 11;
constexpr int kMaxRing = 13;
constexpr int kParts = 8;                        // parts in flight at most (a power of two)
constexpr float kGrow = 8.f;
constexpr float kNoMax = -1e30f;
constexpr uint64_t kDrainNs = 1000ull * 1000ull;

struct Smem {
  uint64_t full[kParts], empty[kParts], raw[kParts];
  uint64_t unit_full[2], unit_empty[2];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], o_empty[2], drain;
  Unit unit[2];
  uint32_t tmem;
  int abort_flag;
};

__global__ void __launch_bounds__(kThreads, 1) prompt_mma_kernel(const __grid_constant__ PromptMmaArgs a) {
  extern __shared__ uint8_t raw_smem[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
  const int nkb = a.nope_blocks + a.rope_blocks;
  uint8_t* ring = base + 2 * nkb * kBlockBytes;
  Smem& sm = *reinterpret_cast<Smem*>(ring + a.ring * kBlockBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtl wc{&sm.abort_flag, a.status, a.wait_ns};

  if (threadIdx.x == 0) {
    for (int i = 0; i < kParts; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
      mbar_init(&sm.raw[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_empty[i], kSoftWarps + 2);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_empty[i], 4);
    }
    mbar_init(&sm.q_full, 1);
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
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
  }
  pdl_begin();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;

  if (warp < kSoftWarps) {
    // ------------------------------------------------ softmax and output of query tile q
    const int q = warp >> 2, quad = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_tm = tmem + q * 128 + lanes, o_tm = tmem + 256 + q * 128 + lanes;
    const int r = quad * 32 + lane;
    uint32_t tile = 0, outs = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      ok = __all_sync(0xffffffffu, bounded_wait_sleep(&sm.unit_full[un & 1], (un >> 1) & 1u, wc));
      if (!ok) break;
      const Unit u = sm.unit[un & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[un & 1]);
      if (u.h < 0) break;
      const int first = u.row0 + q * kTile;
      const int n = key_tiles<kRows>(a, u, q);
      const int i = first + r;
      const int lim = i < u.nq ? key_limit(a, u, i) : u.nk;
      float m = kNoMax, l = 0.f;
      for (int t = 0; t < n; ++t, ++tile) {
        ok = __all_sync(0xffffffffu, bounded_wait(&sm.s_full[q], tile & 1u, wc));
        if (!ok) break;
        tc_fence_after();
        float x[128];
        {
          uint32_t xr[4][32];
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld<32>(s_tm + 32 * c, xr[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = __uint_as_float(xr[c / 32][c % 32]);
        }
        if (a.negate) {
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] = -x[c];
        }
        if (__any_sync(0xffffffffu, (t + 1) * kTile > lim)) {
          const int left = lim - t * kTile;
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= left) x[c] = -INFINITY;
        }
        float top4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) top4[e] = fmaxf(fmaxf(top4[e], x[c + e]), x[c + 4 + e]);
        const float top = fmaxf(fmaxf(fmaxf(top4[0], x[124]), fmaxf(top4[1], x[125])), fmaxf(fmaxf(top4[2], x[126]), fmaxf(top4[3], x[127])));
        const bool grow = (top - m) * a.scale_log2 > kGrow;
        if (__any_sync(0xffffffffu, grow)) {
          const float now = grow ? top : m;
          const float keep = exp2_fast((m - now) * a.scale_log2);
          m = now;
          l *= keep;
          if (t > 0) {
            // the previous tile's product is complete: s_full was committed after it
#pragma unroll 1
            for (int c = 0; c < a.v_blocks * 64; c += 16) {
              uint32_t o[16];
              tmem_ld<16>(o_tm + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * keep);
              tmem_st<16>(o_tm + c, o);
            }
          }
        }
        const float ms = m * a.scale_log2;
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int c = 0; c < 128; c += 32) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float p0 = exp2_fast(fmaf(x[c + e], a.scale_log2, -ms));
            const float p1 = exp2_fast(fmaf(x[c + e + 1], a.scale_log2, -ms));
            s0 += p0;
            s1 += p1;
            pk[e / 2] = pack_bf16(p0, p1);
          }
          tmem_st<16>(s_tm + c / 2, pk);
        }
        l += s0 + s1;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[q]);
      }
      if (!ok) break;
      if (first >= u.nq) continue;
      if (n > 0) {
        ok = __all_sync(0xffffffffu, bounded_wait(&sm.o_full[q], outs & 1u, wc));
        if (!ok) break;
        ++outs;
        tc_fence_after();
      }
      const float inv = inverse_sum(l);
      const int64_t row = static_cast<int64_t>(u.q0 + i) * a.H + u.h;
      for (int c = 0; c < a.d_v; c += 32) {
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
      if (a.lse && i < u.nq) a.lse[row] = row_lse(l, (m * a.scale_log2 + log2f(l)) * 0.69314718056f);
      if (n > 0) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_empty[q]);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------ MMA issue, one lane
    if (elect_one()) {
      const uint32_t id_s = make_instr_desc(1, 128, 128);
      const uint32_t id_o = make_instr_desc(1, 128, 64) | kMajorMnB;
      const uint32_t q0 = desc_lo(smem_addr(base), 0), r0 = desc_lo(smem_addr(ring), 0);
      constexpr uint32_t kBlockStep = kBlockBytes >> 4;
      const int per = nkb + a.v_blocks;
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
        mbar_arrive(&sm.unit_empty[un & 1]);
        if (u.h < 0) break;
        const int n0 = key_tiles<kRows>(a, u, 0), n1 = key_tiles<kRows>(a, u, 1), nt = max(n0, n1);
        if (nt == 0) continue;
        if (!(ok = bounded_wait(&sm.q_full, busy & 1u, wc))) break;
        ++busy;
        bool k_here = false, v_here = false;
        // S_q of the next K part; `last`: no other tile needs the part
        auto scores = [&](int q, bool last) {
          if (!k_here && !bounded_wait(&sm.full[kp % kParts], (kp / kParts) & 1u, wc)) return false;
          k_here = true;
          tc_fence_after();
          uint32_t da = q0 + q * nkb * kBlockStep;
          int s = kc;
          for (int j = 0; j < nkb; ++j, da += kBlockStep) {
            const uint32_t db = r0 + s * kBlockStep;
            if (++s == a.ring) s = 0;
            const int ks = j == a.nope_blocks - 1 ? a.nope_ksteps : (j == nkb - 1 ? a.rope_ksteps : 4);
            if (ks == 4) {
              umma_ss_steps<4, 2, 2>(tmem + q * 128, da, db, id_s, j > 0 ? 1u : 0u);
            } else {
              for (int k = 0; k < ks; ++k) umma_ss_steps<1, 2, 2>(tmem + q * 128, da + 2 * k, db + 2 * k, id_s, j + k > 0 ? 1u : 0u);
            }
          }
          if (last) {
            umma_commit(&sm.empty[kp % kParts]);
            advance(kc, kp);
            k_here = false;
          }
          umma_commit(&sm.s_full[q]);
          return true;
        };
        // O_q of the next V part
        auto values = [&](int q, bool first, bool final, bool last) {
          if (first && outs[q] > 0 && !bounded_wait(&sm.o_empty[q], (outs[q] - 1) & 1u, wc)) return false;
          if (!v_here && !bounded_wait(&sm.full[vp % kParts], (vp / kParts) & 1u, wc)) return false;
          v_here = true;
          if (!bounded_wait(&sm.p_full[q], ptile[q] & 1u, wc)) return false;
          ++ptile[q];
          tc_fence_after();
          int s = vc;
          for (int j = 0; j < a.v_blocks; ++j) {
            umma_ts_steps<8, 128>(tmem + 256 + q * 128 + j * 64, tmem + q * 128, r0 + s * kBlockStep, id_o, first ? 0u : 1u);
            if (++s == a.ring) s = 0;
          }
          if (last) {
            umma_commit(&sm.empty[vp % kParts]);
            advance(vc, vp);
            v_here = false;
          }
          if (final) {
            umma_commit(&sm.o_full[q]);
            ++outs[q];
          }
          return true;
        };
        if (n0 > 0) ok = scores(0, n1 == 0);
        if (ok && n1 > 0) ok = scores(1, true);
        if (ok && nt == 1) umma_commit(&sm.q_empty);
        for (int t = 0; t < nt && ok; ++t) {
          if (t < n0) ok = values(0, t == 0, t == n0 - 1, t >= n1);
          if (ok && t + 1 < n0) ok = scores(0, t + 1 >= n1);
          if (ok && t < n1) ok = values(1, t == 0, t == n1 - 1, true);
          if (ok && t + 1 < n1) ok = scores(1, true);
          if (ok && t + 2 == nt) umma_commit(&sm.q_empty);
        }
      }
      // nothing is in flight when the CTA ends, whichever role gave up
      umma_commit(&sm.drain);
      drain_wait(&sm.drain, 0, kDrainNs);
    }
    __syncwarp();
  } else if (warp == kLoadWarp) {
    // ------------------------------------------------ units and loads
    const int64_t total = all_units<kRows>(a, lane);
    int64_t next = blockIdx.x;
    uint32_t part = 0, tail = 0, busy = 0;       // parts loaded, parts known to be free again, units with keys
    int free_blocks = a.ring, slot = 0;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      const Unit u = find_unit<kRows>(a, next, total, lane);
      if (u.h >= 0 && lane == 0) next = static_cast<int64_t>(gridDim.x) + atomicAdd(a.next_unit, 1u);
      next = __shfl_sync(0xffffffffu, next, 0);
      if (un >= 2) ok = __all_sync(0xffffffffu, bounded_wait(&sm.unit_empty[un & 1], ((un >> 1) - 1) & 1u, wc));
      if (!ok) break;
      if (lane == 0) {
        sm.unit[un & 1] = u;
        mbar_arrive(&sm.unit_full[un & 1]);
      }
      if (u.h < 0) break;
      const int n0 = key_tiles<kRows>(a, u, 0), n1 = key_tiles<kRows>(a, u, 1), nt = max(n0, n1);
      if (nt == 0) continue;
      int good = 1;
      if (lane == 0) {
        // a part of `blocks` blocks of the ring, once they are free
        auto room = [&](int blocks) {
          while (free_blocks < blocks || part - tail >= kParts) {
            if (!bounded_wait(&sm.empty[tail % kParts], (tail / kParts) & 1u, wc)) return false;
            free_blocks += tail & 1 ? a.v_blocks : nkb;
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
          mbar_arrive_expect_tx(&sm.q_full, tiles * nkb * kBlockBytes);
          ++busy;
          for (int q = 0; q < tiles; ++q)
            for (int j = 0; j < nkb; ++j)
              tma_load_3d(base + (q * nkb + j) * kBlockBytes, &a.map_q, &sm.q_full,
                          j < a.nope_blocks ? 64 * j : a.d_nope + 64 * (j - a.nope_blocks), u.h, u.q0 + u.row0 + q * kTile);
          for (int t = 0; t < nt; ++t) {
            const int row = u.k0 + t * kTile;
            if (!(good = room(nkb))) break;
            uint64_t* bar = &sm.full[part % kParts];
            mbar_arrive_expect_tx(bar, nkb * kBlockBytes);
            for (int j = 0; j < nkb; ++j) {
              if (j < a.nope_blocks) tma_load_3d(next_slot(), &a.map_k, bar, 64 * j, u.h, row);
              else tma_load_2d(next_slot(), &a.map_kr, bar, 64 * (j - a.nope_blocks), row);
            }
            ++part;
            if (!(good = room(a.v_blocks))) break;
            // values past the sequence's end are zeroed before anyone reads them
            bar = (t + 1) * kTile > u.nk ? &sm.raw[part % kParts] : &sm.full[part % kParts];
            mbar_arrive_expect_tx(bar, a.v_blocks * kBlockBytes);
            for (int j = 0; j < a.v_blocks; ++j) tma_load_3d(next_slot(), &a.map_v, bar, 64 * j, u.h, row);
            ++part;
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, good, 0) != 0;
    }
    if (lane == 0) {
      // the copies that were issued land before the CTA ends, whichever role gave up
      for (uint32_t f = part > kParts ? part - kParts : 0; f < part; ++f)
        drain_wait(&sm.full[f % kParts], (f / kParts) & 1u, kDrainNs);
      if (busy > 0) drain_wait(&sm.q_full, (busy - 1) & 1u, kDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------ zeroes behind a sequence's last values
    int vc = nkb % a.ring;                       // ring position of the unit's first V part
    uint32_t vp = 1, raw_phase = 0;
    const int per = nkb + a.v_blocks;
    bool ok = true;
    for (uint32_t un = 0; ok; ++un) {
      ok = __all_sync(0xffffffffu, bounded_wait_sleep(&sm.unit_full[un & 1], (un >> 1) & 1u, wc));
      if (!ok) break;
      const Unit u = sm.unit[un & 1];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[un & 1]);
      if (u.h < 0) break;
      const int nt = max(key_tiles<kRows>(a, u, 0), key_tiles<kRows>(a, u, 1));
      if (nt > 0 && nt * kTile > u.nk) {
        const uint32_t p = vp + 2 * (nt - 1);
        const int keep = u.nk - (nt - 1) * kTile;
        int s = (vc + (nt - 1) * per) % a.ring;
        ok = __all_sync(0xffffffffu, bounded_wait_sleep(&sm.raw[p % kParts], (raw_phase >> (p % kParts)) & 1u, wc));
        if (!ok) break;
        raw_phase ^= 1u << (p % kParts);
        for (int j = 0; j < a.v_blocks; ++j) {
          uint4* rows = reinterpret_cast<uint4*>(ring + s * kBlockBytes);
          for (int x = keep * 8 + lane; x < kTile * 8; x += 32) rows[x] = make_uint4(0u, 0u, 0u, 0u);
          if (++s == a.ring) s = 0;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.full[p % kParts]);
      }
      vc = (vc + nt * per) % a.ring;
      vp += 2 * nt;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
  // the last CTA leaves the counters as it found them
  if (threadIdx.x == 0) {
    unsigned prev;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(prev) : "l"(a.done) : "memory");
    if (prev == gridDim.x - 1) {
      *a.next_unit = 0u;
      *a.done = 0u;
    }
  }
}

}  // namespace

bool prompt_mma_layout(PromptMmaArgs* a, int num_sms, int max_smem) {
  a->box_rows = kTile;
  a->nope_blocks = (a->d_nope + 63) / 64;
  a->rope_blocks = (a->d_rope + 63) / 64;
  a->v_blocks = (a->d_v + 63) / 64;
  a->nope_ksteps = (a->d_nope - 64 * (a->nope_blocks - 1) + 15) / 16;
  a->rope_ksteps = (a->d_rope + 15) / 16;
  const int64_t q = 2ll * (a->nope_blocks + a->rope_blocks) * kBlockBytes;
  const int64_t room = static_cast<int64_t>(max_smem) - 1024 - q - static_cast<int64_t>(sizeof(Smem));
  a->ring = static_cast<int>(std::min<int64_t>(kMaxRing, room / kBlockBytes));
  if (a->ring < a->nope_blocks + a->rope_blocks + a->v_blocks) return false;
  a->smem_bytes = static_cast<uint32_t>(1024 + q + a->ring * kBlockBytes + sizeof(Smem));
  const int64_t units = (static_cast<int64_t>(a->total_q) / kRows + a->batch) * a->H;
  a->grid = static_cast<int>(std::min<int64_t>(num_sms, units));
  return true;
}

cudaError_t launch_prompt_mma(const PromptMmaArgs& a, cudaStream_t st) {
  const cudaError_t e = raise_smem_limit(reinterpret_cast<const void*>(prompt_mma_kernel), static_cast<int>(a.smem_bytes));
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_mma_kernel, dim3(a.grid), dim3(kThreads), a.smem_bytes, st, 1, a);
}

}  // namespace li
