// attention.h -- launch interfaces of the attention operators' kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/li.h"

namespace li {

// ---- row transforms (rows.cu)

constexpr int kMaxRowSets = 4;
constexpr int kMaxRowDim = 1024;

struct NormRopeArgs {
  li_head_rows set[kMaxRowSets];
  int n_sets;
  int heads;               // heads of all sets together
  int heads_per_block;
  int64_t n_tok;
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
  unsigned int* done;
  int* status;
};

cudaError_t launch_norm_rope(const NormRopeArgs& a, li_dtype dtype, bool vec, int max_dim, int64_t grid, cudaStream_t st);
cudaError_t launch_append_paged(const AppendPagedArgs& a, li_dtype dtype, bool vec, int num_sms, cudaStream_t st);

// ---- attention

struct LatentAttnArgs {
  const void* q;
  const void* data;
  const int32_t* page_table;
  const int32_t* lengths;
  const int32_t* q_pos;
  const int32_t* sel;
  void* out;
  float* lse;
  int* status;
  int batch, T, H, k, dim, d_v;
  int n_pages, page_size, max_pages;
  float scale;
};

cudaError_t launch_latent_attn_rows(const LatentAttnArgs& a, li_dtype dtype, cudaStream_t st);
cudaError_t launch_prompt_attn_rows(const li_prompt& p, void* out, float* lse, cudaStream_t st);

}  // namespace li
