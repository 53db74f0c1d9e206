// Single-token attention with capped or biased scores over dense-layout pages, e2m1 elements with block scales (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

cudaError_t launch_scored_e2m1(tq_ctx* ctx, const PagedArgs& a, const ScoreArgs& sc, void* workspace, cudaStream_t s) {
  return launch_kind<kE2M1, kScored>(ctx, a, sc, workspace, s);
}

}  // namespace tq
