// Single-token attention over dense-layout pages, f16 elements (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

size_t paged_workspace_f16(const tq_ctx* ctx, int batch) { return workspace_kind<kF16>(ctx, batch); }

cudaError_t launch_paged_f16(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  return launch_kind<kF16>(ctx, a, workspace, s);
}

}  // namespace tq
