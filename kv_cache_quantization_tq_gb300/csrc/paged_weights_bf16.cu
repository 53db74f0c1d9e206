// Attention weights added up per token of dense-layout pages, bf16 elements (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

cudaError_t launch_weights_bf16(tq_ctx* ctx, const PagedArgs& a, const ScoreArgs& sc, const WeightArgs& w, cudaStream_t s) {
  return launch_weights_kind<kBF16>(ctx, a, sc, w, s);
}

}  // namespace tq
