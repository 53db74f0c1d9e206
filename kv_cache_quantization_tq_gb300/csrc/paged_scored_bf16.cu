// Single-token attention with capped or biased scores over dense-layout pages, bf16 elements (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

cudaError_t launch_scored_bf16(tq_ctx* ctx, const PagedArgs& a, const ScoreArgs& sc, void* workspace, cudaStream_t s) {
  return launch_kind<kBF16, kScored>(ctx, a, sc, workspace, s);
}

}  // namespace tq
