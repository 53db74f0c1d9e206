// Writing keys and values into dense-layout pages (16-bit copies, or e4m3 codes with one power-of-two
// exponent per vector).
//
// What bounds it: memory traffic, each element read once and written once.  A thread moves 16
// bytes of a row; consecutive threads take consecutive pieces of one token's key heads, then of its value
// heads, so that reads are whole rows and writes whole vectors of d elements.  Four pieces per
// thread keep four loads in flight.
//
// The exponent of a vector is e = min { e : max|x| <= 448 2^e }, read off the float bits of max|x|: with
// max|x| = m 2^x, 1 <= m < 2, it is x - 8 for m <= 1.75 and x - 7 otherwise (448 = 1.75 2^8).  A power of two
// makes x 2^-e exact, so the only rounding is the one to e4m3 (3 fraction bits, relative 2^-4); e4m3 being a
// floating type, a scale that is no power of two would buy no precision.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kStoreThreads = 256;
constexpr int kPieces = 4;  // 16-byte pieces per thread

// fp32 values of a pair of 16-bit elements
template <bool BF>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Magnitude bits (15) of the larger finite entry of a pair and m.
template <bool BF>
__device__ __forceinline__ uint32_t max_bits(uint32_t w, uint32_t m) {
  constexpr uint32_t inf = BF ? 0x7f80u : 0x7c00u;
  const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
  if (lo < inf) m = max(m, lo);
  if (hi < inf) m = max(m, hi);
  return m;
}

__device__ __forceinline__ int exponent_of(float top) {
  const uint32_t u = __float_as_uint(top);
  const int x = (int)(u >> 23) - 127;
  const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
  return max(e, -120);
}

__device__ __forceinline__ float two_to(int e) { return __int_as_float((e + 127) << 23); }

// One piece: 8 elements of one row of one tile.
struct Piece {
  const uint16_t* src;
  uint8_t* tile;  // NULL: nothing to do
  int t, side, i;  // token of the page, 0 key / 1 value, piece of the row
};

template <int D, bool FP8>
__device__ __forceinline__ Piece piece_of(const StoreArgs& a, int64_t u, uint32_t per, bool& bad) {
  constexpr int P = D / 8;  // pieces of a row
  Piece p{nullptr, nullptr, 0, 0, 0};
  const int64_t n = (int64_t)a.n_tokens * per;
  if (u >= n) return p;
  const uint32_t tok = (uint32_t)((uint64_t)u / per), w = (uint32_t)(u - (int64_t)tok * per);
  const int64_t slot = a.slots[tok];
  if (slot < 0) return p;
  const int64_t block = slot / kPage;
  if (block >= a.num_blocks) {
    bad = true;
    return p;
  }
  const uint32_t half = per / 2;  // pieces of the token's keys
  p.side = w >= half;
  const uint32_t r = w - (p.side ? half : 0);
  const int h = r / P;
  p.i = r % P;
  p.t = (int)(slot % kPage);
  p.src = (p.side ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) + (size_t)r * 8;
  constexpr size_t tile = FP8 ? 32 * D + 32 : 64 * D;
  p.tile = a.pool + ((size_t)block * a.hkv + h) * tile;
  return p;
}

template <int D, bool FP8, bool BF>
__global__ void __launch_bounds__(kStoreThreads) store_kernel(const StoreArgs a) {
  constexpr int P = D / 8;
  constexpr int G = P < 32 ? P : 32;  // lanes that share a row (a row of 512 is two pieces a lane, see below)
  const uint32_t per = 2u * a.hkv * P;
  const int64_t base = (int64_t)blockIdx.x * (kStoreThreads * kPieces);
  bool bad = false;
  Piece p[kPieces];
  uint4 x[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    p[k] = piece_of<D, FP8>(a, base + k * kStoreThreads + threadIdx.x, per, bad);
    x[k] = make_uint4(0, 0, 0, 0);
    if (p[k].tile) x[k] = *reinterpret_cast<const uint4*>(p[k].src);
  }
#pragma unroll
  for (int k = 0; k < kPieces; ++k) {
    if constexpr (!FP8) {
      if (p[k].tile)
        *reinterpret_cast<uint4*>(p[k].tile + (size_t)(p[k].side * kPage + p[k].t) * D * 2 + p[k].i * 16) = x[k];
    } else {
      uint32_t m = max_bits<BF>(x[k].x, max_bits<BF>(x[k].y, max_bits<BF>(x[k].z, max_bits<BF>(x[k].w, 0u))));
#pragma unroll
      for (int o = 1; o < G; o <<= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
      if constexpr (P > 32) {
        // the row's other half is with the neighbouring warp
        __shared__ uint32_t half[kPieces][kStoreThreads / 32];
        if ((threadIdx.x & 31) == 0) half[k][threadIdx.x >> 5] = m;
        __syncthreads();
        m = max(m, half[k][(threadIdx.x >> 5) ^ 1]);
      }
      const float top = BF ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
      const int e = exponent_of(top);
      const float down = two_to(-e);
      uint32_t c[2];
      const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float2 f = pair_of<BF>(w[i]);
        f.x *= down;
        f.y *= down;
        const uint32_t two = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
        c[i >> 1] = i & 1 ? c[i >> 1] | two << 16 : two;
      }
      if (p[k].tile) {
        *reinterpret_cast<uint2*>(p[k].tile + (size_t)(p[k].side * kPage + p[k].t) * D + p[k].i * 8) = make_uint2(c[0], c[1]);
        if (p[k].i == 0) p[k].tile[32 * D + p[k].side * kPage + p[k].t] = (uint8_t)e;
      }
    }
  }
  if (bad) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
}

template <int D>
cudaError_t launch_d(const tq_config& c, const StoreArgs& a, int64_t grid, cudaStream_t s) {
  const bool bf = c.key_format == TQ_ELEM_BF16;
  if (c.key_bits == 16) store_kernel<D, false, false><<<(unsigned)grid, kStoreThreads, 0, s>>>(a);
  else if (bf) store_kernel<D, true, true><<<(unsigned)grid, kStoreThreads, 0, s>>>(a);
  else store_kernel<D, true, false><<<(unsigned)grid, kStoreThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_store(tq_ctx* ctx, const StoreArgs& a, cudaStream_t s) {
  const tq_config& c = ctx->cfg;
  const int64_t units = (int64_t)a.n_tokens * 2 * a.hkv * (c.head_dim / 8);
  const int64_t grid = (units + kStoreThreads * kPieces - 1) / (kStoreThreads * kPieces);
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = cudaErrorInvalidValue;
  switch (c.head_dim) {
    case 64: e = launch_d<64>(c, a, grid, s); break;
    case 128: e = launch_d<128>(c, a, grid, s); break;
    case 256: e = launch_d<256>(c, a, grid, s); break;
    case 512: e = launch_d<512>(c, a, grid, s); break;
  }
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
