// Eviction by accumulated attention weight, and the return of the pages that it empties.
//
//   kept = the first `lead` slots, the last `last` ones, and of those between them the m with the largest weights (the
//   lower slot of equal ones);  token kept[i] moves to slot i, kept ascending.
//
// One cluster of CTAs per (sequence, KV head).  Selection: the m-th largest weight by radix select, 8 bits of an order-
// preserving integer key at a time, the slice of a CTA held in shared memory where it fits; the clusters' histograms
// are added up through distributed shared memory.  Places: a count per warp of what lies above the threshold
// and on it, one scan over the warps, ballots within them.  Moving: in place, in rounds of as many tokens as the cluster's
// registers hold: load, barrier, store.  kept[i] >= i, so a round's stores touch no token that a later round loads, and the
// one barrier per round is all the order that is needed.
//
// What bounds it: the tokens that move, read once and written once; in front of that, and for a single sequence all in all,
// the chain of passes.  64 sequences of 8 heads from 4.2K to 4K tokens as replayed graphs, 3 us above the kernel's own time:
//   many equal sums, so that the newest of them go and a sixth of the tokens moves   e4m3 62 us (31.5 at the copy rate), 16 bits 89 (59), 4 bits 48 (19)
//   sums that are all different: nearly all tokens move                              e4m3 208 (162), 16 bits 364 (318), 4 bits 132 (94)
// The first of these by phases: 6 us to the weights, 10 to the threshold, 9 to the places, 29 of moves; 1 x 32K to 2K, fp16
// (23 us): 4.5, 7, 5.5 and 7.
#include <cooperative_groups.h>

#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMostWarps = 16;
constexpr int kHeld = 10 * 1024;   // weights of a CTA's slice that are kept in shared memory
constexpr int kInFlight = 8;       // 16-byte pieces of a thread and round
constexpr int kDigits = 256;

// Where a token comes from and goes to: byte offsets of the tiles in the pool with the slots in their low 4 bits; -1: no move.
struct __align__(16) Move {
  int64_t src, dst;
};
struct EvictSmem {
  union {
    float held[kHeld];
    Move move[2][1024];  // of a round and the next
  };
  uint32_t hist[2][kDigits];   // of this CTA; two passes' by turns
  uint32_t total[kDigits];     // of the cluster
  uint32_t above[kMostWarps], on[kMostWarps];  // per warp: keys above the threshold, and equal to it
  uint32_t cta_above, cta_on;
  int first_gone;  // lowest slot of the slice that does not stay
  uint32_t digit, left;
};

// Larger weights have larger keys; -0 counts as 0 and NaN as the largest.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Byte layout of a tile: rows of keys, rows of values, 4-bit scales of both, exponents of both.
template <int BITS, int D, int THREADS>
struct Tile {
  static constexpr int ROW = D * BITS / 8, PIECES = 2 * ROW / 16;  // 16-byte pieces of a token's key and value
  static constexpr int SCALE = BITS == 4 ? D / 16 : 0;             // bytes of a token's scales on a side
  static constexpr int AT_SCALE = 2 * kPage * ROW, AT_EXP = AT_SCALE + 2 * kPage * SCALE;
  static constexpr int BYTES = AT_EXP + (BITS < 16 ? 2 * kPage : 0);
  static constexpr int TOKENS = THREADS * kInFlight / PIECES;  // of a CTA and round
  static_assert(TOKENS <= 1024 && BYTES % 16 == 0, "the moves' list");
};

// A token's scales of one side as one value.
template <int N>
struct Scales {
  uint4 v[N / 16];
};
template <>
struct Scales<4> {
  uint32_t v;
};
template <>
struct Scales<8> {
  uint2 v;
};

template <int BITS, int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) evict_kernel(const EvictArgs a) {
  using T = Tile<BITS, D, THREADS>;
  constexpr int WARPS = THREADS / 32;
  extern __shared__ __align__(16) uint8_t raw[];
  EvictSmem& sm = *reinterpret_cast<EvictSmem*>(raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const unsigned row = blockIdx.x / ctas;
  const int b = row / a.hkv, h = row - b * a.hkv;
  auto meet = [&]() {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  int n = a.lengths[b];
  const int64_t most = min((int64_t)a.max_blocks * kPage, a.stride);
  if (n < 0 || n > most) {
    if (tid == 0 && rank == 0 && h == 0) flag_error(a.err, TQ_DEVERR_POSITION);
    n = 0;
  }
  const int keep = max(min(a.keep[b], n), 0), last = min(keep, a.recent), lead = min(keep - last, a.sinks);
  if (tid == 0 && rank == 0 && h == 0) a.lengths_out[b] = keep;
  if (n == 0) return;  // all of the cluster
  const int lo = lead, hi = n - last;  // the slots between
  int m = keep - last - lead;          // how many of them stay
  const float* w = a.weights + (int64_t)row * a.stride;

  // ---- this CTA's slice of them
  const int each = (hi - lo + ctas - 1) / ctas;
  const int s0 = (int)min((int64_t)hi, lo + (int64_t)rank * each), size = min(each, hi - s0);
  const bool held = size <= kHeld;
  if (held) {
#pragma unroll 1
    for (int i = tid; i < size; i += 8 * THREADS) {
      float x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = i + k * THREADS < size ? w[s0 + i + k * THREADS] : 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (i + k * THREADS < size) sm.held[i + k * THREADS] = x[k];
    }
  }
  auto weight_at = [&](int i) { return held ? sm.held[i] : w[s0 + i]; };
  auto key_at = [&](int i) { return key_of(weight_at(i)); };

  // ---- the threshold: `prefix` collects the digits of the m-th largest key, m what is still to be found below it
  uint32_t prefix = 0;
  const bool all = m >= hi - lo, none = m == 0;
  if (!all && !none) {
    for (int i = tid; i < 2 * kDigits; i += THREADS) sm.hist[i / kDigits][i % kDigits] = 0;
    __syncthreads();
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      uint32_t* hist = sm.hist[shift >> 3 & 1];
#pragma unroll 4
      for (int i = tid; i < size; i += THREADS) {
        const uint32_t k = key_at(i);
        if (shift == 24 || k >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[k >> shift & 255], 1u);
      }
      meet();
      for (int i = tid; i < kDigits; i += THREADS) {
        uint32_t t = 0;
        for (int c = 0; c < ctas; ++c) t += ctas > 1 ? cluster.map_shared_rank(hist, c)[i] : hist[i];
        sm.total[i] = t;
        // the pass before: everyone has read it, and the next one wants it clear
        sm.hist[~shift >> 3 & 1][i] = 0;
      }
      __syncthreads();
      if (wid == 0) {  // the digit with which the count from above reaches m: lane 0 has the top 8
        uint32_t c[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i] = sm.total[255 - 8 * lane - i];
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t up = __shfl_up_sync(kFull, inc, o);
          if (lane >= o) inc += up;
        }
        uint32_t before = inc - sum;
        if (before < (uint32_t)m && inc >= (uint32_t)m) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (before < (uint32_t)m && before + c[i] >= (uint32_t)m) {
              sm.digit = 255 - 8 * lane - i;
              sm.left = m - before;
              break;
            }
            before += c[i];
          }
        }
      }
      __syncthreads();
      prefix |= sm.digit << shift;
      m = sm.left;
    }
  }
  __syncthreads();  // the keys are there, also where no pass was needed
  // stays: above the threshold, or one of the first m equal to it
  auto above = [&](uint32_t k) { return all || (!none && k > prefix); };
  auto on = [&](uint32_t k) { return !all && !none && k == prefix; };

  // ---- places: a warp has a stretch of the slice
  const int stretch = (size + THREADS - 1) / THREADS * 32;  // stride <= 2^30: nothing here passes 31 bits
  const int i0 = min(wid * stretch, size), i1 = min(i0 + stretch, size);
  uint32_t ca = 0, co = 0;
#pragma unroll 4
  for (int i = i0 + lane; i < i1; i += 32) {
    const uint32_t k = key_at(i);
    ca += above(k);
    co += on(k);
  }
  ca = __reduce_add_sync(kFull, ca);
  co = __reduce_add_sync(kFull, co);
  if (lane == 0) {
    sm.above[wid] = ca;
    sm.on[wid] = co;
  }
  if (tid == 0) sm.first_gone = keep;
  __syncthreads();
  if (wid == 0) {
    const uint32_t x = __reduce_add_sync(kFull, lane < WARPS ? sm.above[lane] : 0u);
    const uint32_t y = __reduce_add_sync(kFull, lane < WARPS ? sm.on[lane] : 0u);
    if (lane == 0) {
      sm.cta_above = x;
      sm.cta_on = y;
    }
  }
  meet();
  uint32_t fa = 0, fo = 0;  // in front of this warp's stretch
  for (int c = 0; c < rank; ++c) {
    fa += *cluster.map_shared_rank(&sm.cta_above, c);
    fo += *cluster.map_shared_rank(&sm.cta_on, c);
  }
  for (int k = 0; k < wid; ++k) {
    fa += sm.above[k];
    fo += sm.on[k];
  }
  int32_t* kept = a.kept + (int64_t)row * a.stride;
  float* out = a.weights_out + (int64_t)row * a.stride;
  const uint32_t before = (1u << lane) - 1;
  int first = keep;  // the warp's first slot that does not stay
#pragma unroll 2
  for (int i = i0; i < i1; i += 32) {
    const float x = i + lane < i1 ? weight_at(i + lane) : 0.f;
    const uint32_t k = key_of(x);
    const uint32_t va = __ballot_sync(kFull, i + lane < i1 && above(k)), vo = __ballot_sync(kFull, i + lane < i1 && on(k));
    const uint32_t ra = fa + __popc(va & before), ro = fo + __popc(vo & before);
    const bool tie = vo >> lane & 1;
    const bool stays = (va >> lane & 1) || (tie && ro < (uint32_t)m);
    const uint32_t gone = __ballot_sync(kFull, i + lane < i1 && !stays);
    if (gone && first == keep) {
      first = min(first, s0 + i + __ffs(gone) - 1);
      if (lane == 0) atomicMin(&sm.first_gone, first);
    }
    if (stays) {
      const int at = lead + ra + min(ro, all || none ? 0u : (uint32_t)m);
      kept[at] = s0 + i + lane;
      out[at] = x;
    }
    fa += __popc(va);
    fo += __popc(vo);
  }
  const int self = rank * THREADS + tid, everyone = ctas * THREADS;
  for (int i = self; i < lead; i += everyone) {
    kept[i] = i;
    out[i] = w[i];
  }
  for (int i = self; i < last; i += everyone) {
    kept[keep - last + i] = hi + i;
    out[keep - last + i] = w[hi + i];
  }
  for (int i = keep + self; i < n; i += everyone) out[i] = 0.f;
  if (keep == n) {  // nothing moves; no CTA leaves while another reads its shared memory
    meet();
    return;
  }
  meet();  // the list is there, for all of the cluster

  // ---- moving, from the first token that does not stay where it is: the list is i below the first slot that goes
  int from = keep;
  for (int c = 0; c < ctas; ++c) from = min(from, *cluster.map_shared_rank(&sm.first_gone, c));
  if (from >= keep) {
    meet();  // before a CTA leaves
    return;
  }
  const int32_t* table = a.block_table + (int64_t)b * a.max_blocks;
  bool bad = false;
  // The moves of the round that begins at token `first`, listed by a thread per token; all loads of a step before the next.
  auto list = [&](int first, Move* to) {
    constexpr int EACH = (T::TOKENS + THREADS - 1) / THREADS;
    int p[EACH], from_id[EACH], to_id[EACH];
#pragma unroll
    for (int u = 0; u < EACH; ++u) p[u] = __ldcg(kept + min(first + u * THREADS + tid, keep - 1));
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
      from_id[u] = table[p[u] / kPage];
      to_id[u] = table[min(first + u * THREADS + tid, keep - 1) / kPage];
    }
#pragma unroll
    for (int u = 0; u < EACH; ++u) {
      const int k = u * THREADS + tid, i = first + k;
      const bool ok = (unsigned)from_id[u] < (unsigned)a.num_blocks && (unsigned)to_id[u] < (unsigned)a.num_blocks;
      bad |= i < keep && k < T::TOKENS && !ok;
      Move m{-1, -1};
      if (ok && i < keep) {
        m.src = ((int64_t)from_id[u] * a.hkv + h) * T::BYTES + p[u] % kPage;
        m.dst = ((int64_t)to_id[u] * a.hkv + h) * T::BYTES + i % kPage;
      }
      if (k < T::TOKENS) to[k] = m;
    }
  };
  int turn = 0;
  list(from + rank * T::TOKENS, sm.move[0]);
  __syncthreads();
#pragma unroll 1
  for (int first = from + rank * T::TOKENS; first - rank * T::TOKENS < keep; first += ctas * T::TOKENS, turn ^= 1) {
    const Move* moves = sm.move[turn];
    uint4 x[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int unit = u * THREADS + tid, piece = unit % T::PIECES, side = piece / (T::PIECES / 2);
      const int64_t src = moves[unit / T::PIECES].src;
      if (src >= 0)
        x[u] = *reinterpret_cast<const uint4*>(a.pool + (src & ~15ll) + (side * kPage + (src & 15)) * T::ROW + piece % (T::PIECES / 2) * 16);
    }
    // scales and exponents: a token per thread, TOKENS of them
    constexpr int SMALL = BITS == 16 ? 1 : (T::TOKENS + THREADS - 1) / THREADS;
    Scales<BITS == 4 ? T::SCALE : 4> sc[SMALL][2];
    uint8_t ex[SMALL][2];
    if constexpr (BITS < 16) {
#pragma unroll
      for (int u = 0; u < SMALL; ++u) {
        const int k = u * THREADS + tid;
        const int64_t src = k < T::TOKENS ? moves[k].src : -1;
        if (src >= 0) {
          const uint8_t* tile = a.pool + (src & ~15ll);
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const int row = side * kPage + (int)(src & 15);
            ex[u][side] = tile[T::AT_EXP + row];
            if constexpr (BITS == 4) sc[u][side] = *reinterpret_cast<const Scales<T::SCALE>*>(tile + T::AT_SCALE + row * T::SCALE);
          }
        }
      }
    }
    const int next = first + ctas * T::TOKENS;
    if (next < keep) list(next, sm.move[turn ^ 1]);
    else {  // this CTA is through, the cluster may not be
      for (int k = tid; k < T::TOKENS; k += THREADS) sm.move[turn ^ 1][k] = Move{-1, -1};
    }
    meet();
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
      const int unit = u * THREADS + tid, piece = unit % T::PIECES, side = piece / (T::PIECES / 2);
      const int64_t dst = moves[unit / T::PIECES].dst;
      if (dst >= 0)
        *reinterpret_cast<uint4*>(a.pool + (dst & ~15ll) + (side * kPage + (dst & 15)) * T::ROW + piece % (T::PIECES / 2) * 16) = x[u];
    }
    if constexpr (BITS < 16) {
#pragma unroll
      for (int u = 0; u < SMALL; ++u) {
        const int k = u * THREADS + tid;
        const int64_t dst = k < T::TOKENS ? moves[k].dst : -1;
        if (dst >= 0) {
          uint8_t* tile = a.pool + (dst & ~15ll);
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const int row = side * kPage + (int)(dst & 15);
            tile[T::AT_EXP + row] = ex[u][side];
            if constexpr (BITS == 4) *reinterpret_cast<Scales<T::SCALE>*>(tile + T::AT_SCALE + row * T::SCALE) = sc[u][side];
          }
        }
      }
    }
    __syncthreads();  // the list is read before the round after the next one writes it
  }
  if (bad) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
}

// Pages that hold no token any more, behind the queue's end in order.  A CTA has a stretch of the requests and adds up itself
// what those in front give back: a few bytes per request from L2, against a second launch or CTAs that wait for one another.
constexpr int kReleaseThreads = 1024;

__global__ void __launch_bounds__(kReleaseThreads) release_kernel(const ReleaseArgs a) {
  __shared__ int64_t part[kReleaseThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  uint32_t flags = 0;
  // pages [first, first + count) of request b go
  auto pages = [&](int b, int& first) -> int {
    const int old = a.lengths[b], now = a.new_lengths[b];
    first = 0;
    if (now < 0 || now > old || ((int64_t)old + kPage - 1) / kPage > a.max_blocks) return -1;
    first = (int)(((int64_t)now + kPage - 1) / kPage);
    return (int)(((int64_t)old + kPage - 1) / kPage) - first;
  };
  const int head = a.queue_state[0], count = a.queue_state[1];
  const bool sound = count >= 0 && count <= a.queue_cap && head >= 0 && (head < a.queue_cap || a.queue_cap == 0);
  const int each = (a.batch + gridDim.x - 1) / gridDim.x;
  const int b0 = min((int)blockIdx.x * each, a.batch), b1 = min(b0 + each, a.batch);
  const bool final = blockIdx.x == gridDim.x - 1;
  int64_t sum = 0;
  int first;
  for (int b = tid; b < b0; b += kReleaseThreads) sum += max(pages(b, first), 0);
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) part[wid] = sum;
  __syncthreads();
  int64_t at = 0;
#pragma unroll
  for (int k = 0; k < kReleaseThreads / 32; ++k) at += part[k];
  const int64_t room = sound ? a.queue_cap - count : 0;
  for (int b = b0; b < b1; ++b) {
    const int gone = pages(b, first);
    if (gone < 0) flags |= TQ_DEVERR_POSITION;
    for (int j = tid; j < gone; j += kReleaseThreads) {
      const int id = a.block_table[(int64_t)b * a.max_blocks + first + j];
      if (at + j >= room) {
        flags |= TQ_DEVERR_PAGES;
        break;
      }
      if (id < 0 || id >= a.num_blocks) flags |= TQ_DEVERR_BLOCK_ID;
      const int64_t to = (int64_t)head + count + at + j;  // below twice the capacity
      a.queue[to < a.queue_cap ? to : to - a.queue_cap] = id;
    }
    at += max(gone, 0);
  }
  if (final && tid == 0) {
    a.queue_state_out[0] = head;
    a.queue_state_out[1] = sound ? count + (int)min(at, room) : count;
  }
  if (!sound) flags |= TQ_DEVERR_PAGES;
  if (flags) flag_error(a.err, flags);
}

template <int BITS, int D, int THREADS>
cudaError_t launch_evict_t(tq_ctx* ctx, const EvictArgs& a, int ctas, cudaStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.hkv;
  auto kern = evict_kernel<BITS, D, THREADS>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(EvictSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(rows * ctas));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = sizeof(EvictSmem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a);
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

// Rows enough for every multiprocessor twice are CTAs of 256 threads, four resident on each (64 sequences of 8 heads from 4.2K
// to 4K tokens, e4m3: 67 us with the return of the pages, with 512 threads 74); fewer rows are clusters of CTAs of 512, enough
// for two on every multiprocessor, up to the portable cluster of 8 (1 x 32K to 2K, 8 heads, likewise: 26.6 us, with 256 threads 32, with
// 16 CTAs 29).  The rule looks at the number of rows alone: a CTA with more than kHeld weights reads them from memory in every pass
// (64 x 32K to 2K, e4m3: 343 us for 678 MB, 101 at the copy rate), and a long row among many short ones ends late.
template <int BITS, int D>
cudaError_t launch_evict_rows(tq_ctx* ctx, const EvictArgs& a, cudaStream_t s) {
  const int64_t rows = (int64_t)a.batch * a.hkv;
  if (rows >= 2 * ctx->sm_count) return launch_evict_t<BITS, D, 256>(ctx, a, 1, s);
  int ctas = 1;
  while (ctas < 8 && rows * ctas <= ctx->sm_count) ctas *= 2;
  return launch_evict_t<BITS, D, 512>(ctx, a, ctas, s);
}

template <int BITS>
cudaError_t launch_evict_d(tq_ctx* ctx, const EvictArgs& a, cudaStream_t s) {
  switch (ctx->cfg.head_dim) {
    case 64: return launch_evict_rows<BITS, 64>(ctx, a, s);
    case 128: return launch_evict_rows<BITS, 128>(ctx, a, s);
    case 256: return launch_evict_rows<BITS, 256>(ctx, a, s);
    case 512: return launch_evict_rows<BITS, 512>(ctx, a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_evict(tq_ctx* ctx, const EvictArgs& a, cudaStream_t s) {
  return ctx->cfg.key_bits == 16  ? launch_evict_d<16>(ctx, a, s)
         : ctx->cfg.key_bits == 8 ? launch_evict_d<8>(ctx, a, s)
                                  : launch_evict_d<4>(ctx, a, s);
}

cudaError_t launch_release(tq_ctx* ctx, const ReleaseArgs& a, cudaStream_t s) {
  const int ctas = a.batch < 1 ? 1 : a.batch < ctx->sm_count ? a.batch : ctx->sm_count;
  const cudaError_t e = launch_early(release_kernel, dim3(ctas), dim3(kReleaseThreads), 0, s, a);
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
