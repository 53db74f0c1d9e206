// Weight sums of tokens in front of a sliding window: out = decay in.  The kernel that adds weights up (paged_attn.cuh)
// visits the window's pages; these are the others.  Memory traffic bounds it: 4 bytes read and 4 written per entry.
#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kFadeThreads = 256, kFadeEach = 4;

__global__ void __launch_bounds__(kFadeThreads) fade_kernel(const PagedArgs a, const WeightArgs w, int chunks, int64_t items) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    const int64_t row = item / chunks;  // of a sequence and KV head
    const int len = a.lengths[row / a.hkv];
    if (len < 0 || len > a.max_len || len <= a.window) continue;
    const int end = (len - a.window) / kPage * kPage;
    const int64_t first = (item - row * chunks) * (kFadeThreads * kFadeEach) + threadIdx.x;
#pragma unroll
    for (int k = 0; k < kFadeEach; ++k) {
      const int64_t p = first + k * kFadeThreads;
      if (p < end) w.out[row * w.stride + p] = w.in ? w.decay * w.in[row * w.stride + p] : 0.f;
    }
  }
}

}  // namespace

cudaError_t launch_fade(tq_ctx* ctx, const PagedArgs& a, const WeightArgs& w, cudaStream_t s) {
  const int64_t most = a.max_len - a.window;  // entries of a row that can lie in front of the window
  if (most < kPage) return cudaSuccess;
  const int64_t chunks = (most + kFadeThreads * kFadeEach - 1) / (kFadeThreads * kFadeEach), items = chunks * a.batch * a.hkv;
  const int64_t ctas = items < (int64_t)ctx->sm_count * 8 ? items : (int64_t)ctx->sm_count * 8;
  const cudaError_t e = launch_early(fade_kernel, dim3((unsigned)ctas), dim3(kFadeThreads), 0, s, a, w, (int)chunks, items);
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
