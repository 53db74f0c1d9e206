// Attention weights added up per token of dense-layout pages, e2m1 elements with block scales (see paged_attn.cuh).
#include "paged_attn.cuh"

namespace tq {

cudaError_t launch_weights_e2m1(tq_ctx* ctx, const PagedArgs& a, const ScoreArgs& sc, const WeightArgs& w, cudaStream_t s) {
  return launch_weights_kind<kE2M1>(ctx, a, sc, w, s);
}

}  // namespace tq
