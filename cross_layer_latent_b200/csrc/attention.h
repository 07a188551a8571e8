// attention.h -- launch interfaces of the attention operators' kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/li.h"

namespace li {

// ---- row transforms (rows.cu)

constexpr int kMaxRowSets = 4;
constexpr int kMaxRowDim = 1024;

struct NormRopeArgs {
  li_head_rows set[kMaxRowSets];
  int n_sets;
  int tasks;               // of a token: a warp's worth of rows of one set each
  int per_block, blocks;   // tasks of a block, blocks of a token
  int tab_stride;          // slots of a set's table of angles (even)
  const int32_t* pos;
};

struct AppendPagedArgs {
  const void* x;
  int64_t tok_stride;
  void* data;
  const int32_t* page_table;
  int32_t* lengths;
  const int32_t* start;
  const int32_t* n_new;
  int batch, T, n_pages, page_size, max_pages, dim;
  li_row_transform tf;
  int lengths_last;        // rows take their numbers from the lengths: these advance when every row has
  unsigned int* done;
  int* status;
};

// How the rows are spread: lanes a row (0: a warp by way of shared memory) in
// chunks of 8 elements, rows of a warp's task, warps of a block.
struct NormRopePlan {
  int lanes, chunks, rows, warps;
  bool plain;              // RMS or no norm, no beta, rotary chunks in one register row
};
NormRopePlan plan_norm_rope(const li_head_rows* sets, int n_sets, bool chunked, int max_dim);
bool append_in_chunks(const li_row_transform& tf, int dim);
cudaError_t launch_norm_rope(const NormRopeArgs& a, li_dtype dtype, const NormRopePlan& p, int64_t grid, cudaStream_t st);
cudaError_t launch_append_paged(const AppendPagedArgs& a, li_dtype dtype, bool vec, int num_sms, cudaStream_t st);

// ---- attention

// What a row's sum of weights l makes of it: the factor of its output and its
// log-sum-exp, `log_sum` where there are weights.  l = 0: nothing attended, or
// only scores of -inf, so out = 0 and lse = -inf.  l is NaN where a score was NaN
// or +inf, and stays so.
#ifdef __CUDACC__
__device__ __forceinline__ float inverse_sum(float l) { return l > 0.f ? 1.f / l : l; }
__device__ __forceinline__ float row_lse(float l, float log_sum) { return l > 0.f ? log_sum : (l == 0.f ? -INFINITY : l); }
#endif

struct LatentAttnArgs {
  const float* q;
  const float* data;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* q_pos;
  const int32_t* sel;
  float* out;
  float* lse;
  int* status;
  int batch, T, H, k, dim, d_v;
  int n_pages, page_size, max_pages;
  float scale;
};

// bf16 on the tensor cores (latent_mma.cu).
struct alignas(64) LatentMmaArgs {
  CUtensorMap map_q;      // queries: dims {dim, rows, seqs}, box {64, N, 1}
  CUtensorMap map_box;    // pool rows: dims {dim, pool rows}, box {64, box}
  const void* data;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* q_pos;
  const int32_t* sel;
  void* out;
  float* lse;
  float* part_o;          // [2 grid][64][part_stride] sums of the parts, and
  float* part_ml;         // [2 grid][64][2] their maxima (log2) and weight sums
  int4* cuts;             // [n_cuts] groups that several CTAs work on: first row, rows (0: none), first and last CTA
  int* status;
  uint64_t wait_ns;
  float scale_log2;       // scale * log2(e)
  int seqs;               // work units with rows of their own: sequences, with sel (sequence, query) pairs
  int rows;               // query rows of a unit: T * H, with sel H
  int T, H, k, dim, d_v;
  int n_pages, page_size, max_pages;
  int box;                // rows of a box (a divisor of the page size), 0: rows one by one always
  int box_shift;          // log2 of box
  // filled by latent_mma_layout
  int N, groups;          // MMA columns, groups of N rows in a unit
  int nb, last_ksteps;    // 64-column blocks of a row, 16-element K steps of the last one
  int m_blocks;           // blocks of 128 values
  int slots, bufs;        // 8 KB slots of a tile, tiles held in shared memory
  int s_bufs;             // score buffers in tensor memory
  int part_stride;
  int n_cuts, cuts_by_group;
  int grid;
  uint32_t tmem_cols, smem_bytes;
};

constexpr int latent_part_stride(int d_v) { return (d_v + 3) / 4 * 4; }
size_t latent_part_bytes(int num_sms, int d_v);
bool latent_mma_layout(LatentMmaArgs* a, int num_sms, int max_smem);
cudaError_t launch_latent_mma(const LatentMmaArgs& a, cudaStream_t st);
cudaError_t launch_latent_join(const LatentMmaArgs& a, cudaStream_t st);

struct alignas(64) PromptMmaArgs {
  CUtensorMap map_q;      // dims {d_nope + d_rope, H, total_q}, box {64, 1, 128}
  CUtensorMap map_k;      // dims {d_nope, H, total_k}, box {64, 1, box_rows}
  CUtensorMap map_kr;     // dims {d_rope, total_k}, box {64, box_rows}
  CUtensorMap map_v;      // dims {d_v, H, total_k}, box {64, 1, box_rows}
  const int32_t* cu_q;
  const int32_t* cu_k;
  void* out;
  float* lse;
  unsigned int* next_unit;  // workspace counters, zero between calls
  unsigned int* done;
  int* status;
  uint64_t wait_ns;
  float scale_log2;       // |scale| * log2(e)
  int negate;             // scale < 0
  int causal;
  int wide_out;           // every output row is 32-byte aligned
  int batch, H, total_q, total_k, max_q;
  int d_nope, d_rope, d_v;
  // filled by prompt_mma_layout or prompt_pair_layout
  int box_rows;                             // rows of a block of keys or values
  int nope_blocks, rope_blocks, v_blocks;   // 64-column blocks
  int nope_ksteps, rope_ksteps;             // 16-element K steps of each part's last block
  int ring;                                 // blocks of the ring
  int grid;
  uint32_t smem_bytes;
};

bool prompt_mma_layout(PromptMmaArgs* a, int num_sms, int max_smem);     // one CTA a unit (prompt_mma.cu)
cudaError_t launch_prompt_mma(const PromptMmaArgs& a, cudaStream_t st);
bool prompt_pair_layout(PromptMmaArgs* a, int num_sms, int max_smem);    // two (prompt_pair.cu)
cudaError_t launch_prompt_pair(const PromptMmaArgs& a, cudaStream_t st);

// fp32 (attn_rows.cu).
cudaError_t launch_latent_attn_rows(const LatentAttnArgs& a, cudaStream_t st);
cudaError_t launch_prompt_attn_rows(const li_prompt& p, float* out, float* lse, cudaStream_t st);

}  // namespace li
