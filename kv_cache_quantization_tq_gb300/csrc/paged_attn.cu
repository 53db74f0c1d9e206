// Attention of one new token per sequence over dense-layout pages.
//
//   s_p = scale q . k_p,  out = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m),  m = max_p s_p
//
// One CTA per (sequence, query head), its warps on every fourth position: the simplest form, one pass
// with a running maximum and sum per warp, joined in shared memory.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kWarps = 4;

template <bool BF>
__device__ __forceinline__ float elem16(uint16_t x) {
  if (BF) return __uint_as_float((uint32_t)x << 16);
  return __half2float(__ushort_as_half(x));
}
__device__ __forceinline__ float elem8(uint8_t x) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(x, __NV_E4M3)));
}

template <int D, bool FP8, bool BF>
__global__ void __launch_bounds__(kWarps * 32) simple_kernel(const PagedArgs a) {
  constexpr int E = D / 32;
  const int h = blockIdx.x, b = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
  int64_t len = a.lengths[b];
  if (len < 0 || len > (int64_t)a.max_blocks * kPage) {
    if (threadIdx.x == 0) flag_error(a.err, TQ_DEVERR_POSITION);
    len = 0;
  }
  const int64_t first = a.window && len > a.window ? len - a.window : 0;
  float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = elem16<BF>(a.q[b * a.q_stride + (int64_t)h * D + e * 32 + lane]);
    o[e] = 0.f;
  }
  constexpr size_t tile_bytes = FP8 ? 32 * D + 32 : 64 * D;
  for (int64_t p = first + w; p < len; p += kWarps) {
    const int id = a.block_table[(int64_t)b * a.max_blocks + p / kPage];
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
      continue;
    }
    const uint8_t* tile = a.pool + ((size_t)id * a.hkv + h / a.n_rep) * tile_bytes;
    const int t = (int)(p % kPage);
    float s = 0.f, ev = 1.f;
    if (FP8) {
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], elem8(tile[t * D + e * 32 + lane]), s);
      s = warp_sum(s) * exp2f((float)(int8_t)tile[32 * D + t]);
      ev = exp2f((float)(int8_t)tile[32 * D + kPage + t]);
    } else {
      const uint16_t* k = reinterpret_cast<const uint16_t*>(tile) + t * D;
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(q[e], elem16<BF>(k[e * 32 + lane]), s);
      s = warp_sum(s);
    }
    s *= a.scale;
    const float mn = fmaxf(m, s);
    const float c = mn == -INFINITY ? 1.f : expf(m - mn), pr = mn == -INFINITY ? 0.f : expf(s - mn);
    m = mn;
    l = l * c + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = FP8 ? elem8(tile[(kPage + t) * D + e * 32 + lane]) * ev
                          : elem16<BF>(reinterpret_cast<const uint16_t*>(tile)[(kPage + t) * D + e * 32 + lane]);
      o[e] = fmaf(pr, v, o[e] * c);
    }
  }
  if (lane == 0) {
    sm_m[w] = m;
    sm_l[w] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_o[w][e * 32 + lane] = o[e];
  __syncthreads();
  float M = -INFINITY, L = 0.f;
  for (int i = 0; i < kWarps; ++i) M = fmaxf(M, sm_m[i]);
  float c[kWarps];
  for (int i = 0; i < kWarps; ++i) {
    c[i] = M == -INFINITY ? 0.f : expf(sm_m[i] - M);
    L += c[i] * sm_l[i];
  }
  const int64_t row = (int64_t)b * a.hq + h;
  for (int i = threadIdx.x; i < D; i += kWarps * 32) {
    float x = 0.f;
    for (int k = 0; k < kWarps; ++k) x += c[k] * sm_o[k][i];
    a.out[row * D + i] = L == 0.f ? 0.f : x / L;
  }
  if (a.lse && threadIdx.x == 0) a.lse[row] = M + logf(L);
}

template <int D>
cudaError_t launch_d(const tq_config& c, const PagedArgs& a, cudaStream_t s) {
  const dim3 grid(a.hq, a.batch);
  const bool bf = c.key_format == TQ_ELEM_BF16;
  if (c.key_bits == 16) {
    if (bf) simple_kernel<D, false, true><<<grid, kWarps * 32, 0, s>>>(a);
    else simple_kernel<D, false, false><<<grid, kWarps * 32, 0, s>>>(a);
  } else {
    if (bf) simple_kernel<D, true, true><<<grid, kWarps * 32, 0, s>>>(a);
    else simple_kernel<D, true, false><<<grid, kWarps * 32, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace

size_t paged_workspace(const tq_ctx*, int) { return 256; }

cudaError_t launch_paged(tq_ctx* ctx, const PagedArgs& a, void*, cudaStream_t s) {
  const tq_config& c = ctx->cfg;
  cudaError_t e = cudaErrorInvalidValue;
  prof_start(ctx, kProfDecode, s);
  switch (c.head_dim) {
    case 64: e = launch_d<64>(c, a, s); break;
    case 128: e = launch_d<128>(c, a, s); break;
    case 256: e = launch_d<256>(c, a, s); break;
    case 512: e = launch_d<512>(c, a, s); break;
  }
  prof_stop(ctx, kProfDecode, s);
  ctx->decode_kernel = "simple_kernel";
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
