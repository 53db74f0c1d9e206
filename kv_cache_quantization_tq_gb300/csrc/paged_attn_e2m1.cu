// Single-token attention over dense-layout pages, e2m1 elements with block scales (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

size_t paged_workspace_e2m1(const tq_ctx* ctx, int batch) { return workspace_kind<kE2M1>(ctx, batch); }

cudaError_t launch_paged_e2m1(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  return launch_kind<kE2M1, kAttend>(ctx, a, ScoreArgs{}, workspace, s);
}

}  // namespace tq
