// Single-token attention over dense-layout pages, e4m3 elements (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

size_t paged_workspace_e4m3(const tq_ctx* ctx, int batch) { return workspace_kind<kE4M3>(ctx, batch); }

cudaError_t launch_paged_e4m3(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  return launch_kind<kE4M3, kAttend>(ctx, a, ScoreArgs{}, workspace, s);
}

}  // namespace tq
