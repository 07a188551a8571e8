// ctx.h -- host state of a li_ctx and the small helpers that every entry point
// uses: error text, launch profile, workspace addressing, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <string>
#include <vector>

#include "internal.h"

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

struct ProfRec {
  std::string name;
  cudaEvent_t beg, end;
  int grid, block, smem;
};

struct ScanPlan {
  li::ScanArgs a;
  int kind;
  int grid;
};

// Everything a scan plan depends on (zero-filled, compared bytewise).
struct PlanKey {
  const void* data;
  const float* scale;
  const int32_t* lengths;
  const void* q;
  const float* q_scale;
  const float* beta;
  const float* w;
  const int32_t* q_pos;
  const uint64_t* trace;
  uint64_t wait_ns;
  int32_t batch, capacity, dim, dtype;
  int32_t q_dtype, T, H, gather;
  int32_t cand_stride, scale_split;
};

struct li_ctx {
  int device = 0;
  int num_sms = 0;
  int max_smem_optin = 0;
  // resident clusters of the single-launch selection, by cluster size 1..16
  int cluster_cap[17] = {};
  EncodeTiledFn encode = nullptr;
  std::string last_error;
  uint64_t wait_ns = 2000000000ull;
  bool profile = false;
  uint64_t* trace = nullptr;
  std::vector<ProfRec> prof;
  std::vector<cudaEvent_t> free_events;
  // Recently built scan plans (tensor maps included): a decode loop calls
  // the same entry points on the same buffers every step.
  static constexpr int kPlanCache = 16;
  PlanKey plan_key[kPlanCache] = {};
  ScanPlan plan_val[kPlanCache];
  bool plan_used[kPlanCache] = {};
  int plan_next = 0;
};

namespace li {

inline li_status fail(li_ctx* ctx, li_status s, const char* fmt, ...) {
  if (ctx) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    ctx->last_error = buf;
  }
  return s;
}

inline li_status cuda_fail(li_ctx* ctx, cudaError_t e, const char* what) {
  return fail(ctx, LI_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int elt_bytes(li_dtype d) { return d == LI_F32 ? 4 : (d == LI_BF16 ? 2 : 1); }

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<uint8_t*>(ws) + off); }

// ------------------------------------------------------------------ profiling

inline cudaEvent_t get_event(li_ctx* c) {
  if (!c->free_events.empty()) {
    cudaEvent_t e = c->free_events.back();
    c->free_events.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  cudaEventCreate(&e);
  return e;
}

struct Launch {
  li_ctx* c;
  cudaStream_t st;
  const char* name;
  int grid, block, smem;
  cudaEvent_t beg = nullptr;
  Launch(li_ctx* c_, cudaStream_t st_, const char* name_, int grid_, int block_, int smem_)
      : c(c_), st(st_), name(name_), grid(grid_), block(block_), smem(smem_) {
    if (c->profile) {
      beg = get_event(c);
      cudaEventRecord(beg, st);
    }
  }
  void done() {
    if (c->profile && beg) {
      cudaEvent_t end = get_event(c);
      cudaEventRecord(end, st);
      c->prof.push_back(ProfRec{name, beg, end, grid, block, smem});
    }
  }
};

// ------------------------------------------------------------------ tensor maps

// Tiled loads stream whole rows and use 256-byte L2 promotion; row gathers
// read scattered rows and ask for none (promotion would pull in neighbouring
// sectors of every gathered row).
inline li_status encode_map(li_ctx* ctx, CUtensorMap* m, li_dtype dt, int rank, void* base, const cuuint64_t* dims,
                     const cuuint64_t* strides, const cuuint32_t* box, int swz, bool promote = true) {
  const CUtensorMapDataType t = dt == LI_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dt == LI_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                : CU_TENSOR_MAP_DATA_TYPE_UINT8;
  const CUtensorMapSwizzle sw = swz == 128 ? CU_TENSOR_MAP_SWIZZLE_128B
                                : swz == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                            : CU_TENSOR_MAP_SWIZZLE_32B;
  const cuuint32_t es[3] = {1, 1, 1};
  const CUresult r = ctx->encode(m, t, rank, base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                                 promote ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ctx, LI_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return LI_OK;
}

}  // namespace li
