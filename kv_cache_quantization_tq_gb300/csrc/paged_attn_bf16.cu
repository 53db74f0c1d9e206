// Single-token attention over dense-layout pages, bf16 elements (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

size_t paged_workspace_bf16(const tq_ctx* ctx, int batch) { return workspace_kind<kBF16>(ctx, batch); }

cudaError_t launch_paged_bf16(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  return launch_kind<kBF16>(ctx, a, workspace, s);
}

}  // namespace tq
