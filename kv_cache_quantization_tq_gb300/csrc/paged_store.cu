// Writing keys and values into dense-layout pages (16-bit copies, or e4m3 codes with one power-of-two
// exponent per vector).
//
// What bounds it: memory traffic, each element read once and written once.  A thread moves 32 bytes of a row
// (16 elements: one 16-byte store of codes); the d / 16 lanes of a row are neighbours, so that a vector's
// largest entry is found by shuffles within a warp for every d.  Rows go token by token; by tiles (16 tokens of a
// head, neighbours in the pool) measured the same.  32768 tokens x 8 heads x 128, bf16: 41.1 us as 16-bit
// copies (6.5 TB/s, 96% of a plain copy), 33.3 us as e4m3 (6.1 TB/s, 89%, with the ALU pipe 67% and the issue slots 66%
// taken: the conversions and packed maxima beside the memory, neither of them alone).
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

// Division by a launch constant: n / d = umulhi(n, mul) >> shift for n < 2^31 (Granlund and Montgomery 1994).
struct Divisor {
  uint32_t d, mul, shift;
  explicit Divisor(uint32_t x) : d(x), shift(0) {
    while ((1ull << shift) < x) ++shift;  // ceil(log2 x)
    mul = (uint32_t)(((1ull << (31 + shift)) + x - 1) / x);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return __umulhi(n * 2u, mul) >> shift; }
};

// fp32 values of a pair of 16-bit elements
template <bool BF>
__device__ __forceinline__ float2 pair_of(uint32_t w) {
  if (BF) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// Magnitudes of a pair's entries with the ones that are not finite as 0.
template <bool BF>
__device__ __forceinline__ uint32_t finite_bits(uint32_t w) {
  constexpr uint32_t inf = BF ? 0x7f80u : 0x7c00u;
  const uint32_t lo = w & 0x7fffu, hi = w >> 16 & 0x7fffu;
  return (lo < inf ? lo : 0u) | (hi < inf ? hi << 16 : 0u);
}

__device__ __forceinline__ int exponent_of(float top) {
  const uint32_t u = __float_as_uint(top);
  const int x = (int)(u >> 23) - 127;
  const int e = (u & 0x7fffffu) <= 0x600000u ? x - 8 : x - 7;
  return max(e, -120);
}

// One thread's share of a row: 16 elements of one vector of one tile.
struct Share {
  const uint4* src;
  uint8_t* tile;  // NULL: nothing to do
  int at, i;      // row of the tile (token, values behind 16 keys), share of the row
};

template <int D, bool FP8>
__device__ __forceinline__ Share share_of(const StoreArgs& a, const Divisor& rows, uint32_t u, bool& bad) {
  constexpr int L = D / 16;  // lanes of a row
  Share p{nullptr, nullptr, 0, 0};
  const uint32_t row = u / L, tok = rows(row);  // a token's key heads, then its value heads
  if (tok >= (uint32_t)a.n_tokens) return p;
  const int64_t slot = a.slots[tok];
  if (slot < 0) return p;
  if (slot >= (int64_t)a.num_blocks * kPage) {
    bad = true;
    return p;
  }
  int h = row - tok * rows.d;
  const bool side = h >= a.hkv;
  h -= side ? a.hkv : 0;
  p.i = u % L;
  p.at = (int)(slot % kPage) + (side ? kPage : 0);
  p.src = reinterpret_cast<const uint4*>((side ? a.v + tok * a.v_stride : a.k + tok * a.k_stride) + h * D + p.i * 16);
  constexpr size_t tile = FP8 ? 32 * D + 32 : 64 * D;
  p.tile = a.pool + ((size_t)(slot / kPage) * a.hkv + h) * tile;
  return p;
}

template <int D, bool FP8, bool BF, int N>
__global__ void __launch_bounds__(kStoreThreads) store_kernel(const StoreArgs a, const Divisor rows) {
  constexpr int L = D / 16;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  bool bad = false;
  Share p[N];
  uint4 x[N][2];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    p[k] = share_of<D, FP8>(a, rows, (blockIdx.x * N + k) * kStoreThreads + threadIdx.x, bad);
    x[k][0] = x[k][1] = make_uint4(0, 0, 0, 0);
    if (p[k].tile) {
      x[k][0] = p[k].src[0];
      x[k][1] = p[k].src[1];
    }
  }
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if constexpr (!FP8) {
      if (p[k].tile) {
        uint4* dst = reinterpret_cast<uint4*>(p[k].tile + (size_t)p[k].at * D * 2) + p[k].i * 2;
        dst[0] = x[k][0];
        dst[1] = x[k][1];
      }
    } else {
      const uint32_t w[8] = {x[k][0].x, x[k][0].y, x[k][0].z, x[k][0].w, x[k][1].x, x[k][1].y, x[k][1].z, x[k][1].w};
      // the largest magnitude as 15-bit patterns, two at a time
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
#pragma unroll
      for (int o = 1; o < L; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFull, m, o));
      m = max(m & 0xffffu, m >> 16);
      constexpr uint32_t inf = BF ? 0x7f80u : 0x7c00u;
      if (__any_sync(kFull, m >= inf)) {  // rare: an entry that is not finite; without those
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, finite_bits<BF>(w[i]));
#pragma unroll
        for (int o = 1; o < L; o <<= 1) m = __vmaxu2(m, __shfl_xor_sync(kFull, m, o));
        m = max(m & 0xffffu, m >> 16);
      }
      const int e = exponent_of(BF ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m)));
      const float down = __int_as_float((127 - e) << 23);
      uint32_t c[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float2 f = pair_of<BF>(w[i]);
        f.x *= down;
        f.y *= down;
        const uint32_t two = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3);
        c[i >> 1] = i & 1 ? __byte_perm(c[i >> 1], two, 0x5410) : two;
      }
      if (p[k].tile) {
        reinterpret_cast<uint4*>(p[k].tile + (size_t)p[k].at * D)[p[k].i] = make_uint4(c[0], c[1], c[2], c[3]);
        if (p[k].i == 0) p[k].tile[32 * D + p[k].at] = (uint8_t)e;
      }
    }
  }
  if (bad) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
}

template <int D, bool FP8, bool BF>
cudaError_t launch_t(const StoreArgs& a, int sm_count, cudaStream_t s) {
  const int64_t units = (int64_t)a.n_tokens * 2 * a.hkv * (D / 16);
  const Divisor rows(2u * a.hkv);
  // two shares a thread once that still leaves every multiprocessor its full number of threads
  const int n = units >= (int64_t)sm_count * 4096 ? 2 : 1;
  const dim3 grid((unsigned)((units + n * kStoreThreads - 1) / (n * kStoreThreads)));
  return n == 2 ? launch_early(store_kernel<D, FP8, BF, 2>, grid, dim3(kStoreThreads), 0, s, a, rows)
                : launch_early(store_kernel<D, FP8, BF, 1>, grid, dim3(kStoreThreads), 0, s, a, rows);
}

template <int D>
cudaError_t launch_d(const tq_config& c, const StoreArgs& a, int sm_count, cudaStream_t s) {
  const bool bf = c.key_format == TQ_ELEM_BF16;
  if (c.key_bits == 16) return launch_t<D, false, false>(a, sm_count, s);
  return bf ? launch_t<D, true, true>(a, sm_count, s) : launch_t<D, true, false>(a, sm_count, s);
}

}  // namespace

cudaError_t launch_store(tq_ctx* ctx, const StoreArgs& args, cudaStream_t s) {
  const tq_config& c = ctx->cfg;
  // a launch counts its shares in 31 bits: more tokens than that take several
  const int64_t per = 2ll * args.hkv * (c.head_dim / 16);
  const int64_t most = (1ll << 30) / per;
  if (most < 1) return cudaErrorInvalidValue;
  StoreArgs a = args;
  for (int64_t at = 0; at < args.n_tokens; at += most) {
    a.k = args.k + at * args.k_stride;
    a.v = args.v + at * args.v_stride;
    a.slots = args.slots + at;
    a.n_tokens = (int)(args.n_tokens - at < most ? args.n_tokens - at : most);
    cudaError_t e = cudaErrorInvalidValue;
    switch (c.head_dim) {
      case 64: e = launch_d<64>(c, a, ctx->sm_count, s); break;
      case 128: e = launch_d<128>(c, a, ctx->sm_count, s); break;
      case 256: e = launch_d<256>(c, a, ctx->sm_count, s); break;
      case 512: e = launch_d<512>(c, a, ctx->sm_count, s); break;
    }
    if (e != cudaSuccess) return e;
    ctx->launches++;
  }
  return cudaSuccess;
}

}  // namespace tq
