// Arguments and launchers of the page plan and the dense-layout page kernels
// (page_plan.cu, paged_store.cu, paged_attn.cu; entry checks in paged.cpp).
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "tq_internal.h"

namespace tq {

struct PlanArgs {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int batch;
  int ring;  // 0 or kRing
  int32_t* block_table;
  int max_blocks, num_blocks;
  int32_t* queue;
  int queue_cap;
  const int32_t* queue_state;
  int32_t* lengths;
  int32_t* n_paged;
  int32_t* n_ring;
  int32_t* token_start;
  int64_t* slots;
  int32_t* positions;
  int32_t* rows;
  int max_tokens;
  int32_t* queue_state_out;
  uint32_t* err;
};

struct StoreArgs {
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, v_stride;  // elements from token to token
  const int64_t* slots;
  int n_tokens;
  uint8_t* pool;
  int num_blocks;
  int hkv;
  uint32_t* err;
};

struct PagedArgs {
  const uint16_t* q;
  int64_t q_stride;  // elements from sequence to sequence
  int batch;
  const uint8_t* pool;
  int num_blocks;
  const int32_t* block_table;
  int max_blocks;
  const int32_t* lengths;
  int window;
  float scale;
  float* out;
  float* lse;
  int hq, hkv, n_rep;
  uint32_t* err;
};

// The pool as a TMA tensor: rows of `d` elements of `elem` bytes, 32 rows (keys, then values) per tile,
// `tiles` tiles `tile_bytes` apart; boxes of `box_rows` rows, `row_bytes` wide and swizzled (128 or 64).
struct PagedTensorMap {
  const void* pool;
  int elem, d;
  int64_t tiles;
  int tile_bytes, row_bytes, box_rows;
};
bool encode_paged_map(const PagedTensorMap& t, CUtensorMap* map);

// A launch that may begin before the kernel in front of it ends.  The kernel says griddepcontrol.wait before
// it touches memory, and griddepcontrol.launch_dependents for the next such launch; what that hides is
// the launch itself.  Inputs are read by ordinary loads: the kernel in front may write them while this one
// is resident, so they are not constant for its lifetime (no __ldg).
template <typename... Params, typename... Values>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, Values... values) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(values)...);
}

cudaError_t launch_plan(tq_ctx* ctx, const PlanArgs& a, cudaStream_t s);
cudaError_t launch_store(tq_ctx* ctx, const StoreArgs& a, cudaStream_t s);
size_t paged_workspace(const tq_ctx* ctx, int batch);
cudaError_t launch_paged(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s);

// one translation unit per element type
size_t paged_workspace_f16(const tq_ctx* ctx, int batch);
size_t paged_workspace_bf16(const tq_ctx* ctx, int batch);
size_t paged_workspace_e4m3(const tq_ctx* ctx, int batch);
cudaError_t launch_paged_f16(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_paged_bf16(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s);
cudaError_t launch_paged_e4m3(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s);

}  // namespace tq
