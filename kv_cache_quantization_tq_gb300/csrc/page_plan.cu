// Page plan of one serving step: block tables, slot maps and the queue of free pages from the
// requests' lengths, in one launch.
//
//   need_b = pages(c_b + n_b) - pages(c_b),  P = exclusive prefix sum of need, T = of n
//   table[b][pages(c_b) + j] = queue[head + P_b + j],  slot of token T_b + i = page of position c_b + i
//
// What bounds it: launch latency and a chain of dependent loads (lengths, then queue, then the
// stores); the data are a few bytes per request and 16 per token.  So nothing is handed from CTA
// to CTA: every CTA scans all lengths itself (one entry of `stride` requests per thread, at most 1024
// entries, kept in shared memory) and then writes its own share of the rows, pages and tokens, finding the
// request of an item by bisection in the scan.  A second launch for the scan, or CTAs that wait for one
// another, would cost more than the repeated reads (8 bytes per request, from L2).  A thread has one token while
// the grid has threads enough (the shortest chain), four with a shared search beyond that (fewer instructions).
//
// Sums are held at 2^31 - 1: every page handed out and every token written lies below that, so a held sum only
// says "behind everything", whatever the lengths on the device are.
#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kPlanThreads = 1024;
constexpr unsigned kHold = 0x7fffffffu;

__device__ __forceinline__ unsigned add_held(unsigned x, unsigned y) { return min(x + y, kHold); }

struct Req {
  int ctx;             // tokens held
  unsigned add;        // tokens added
  unsigned old, need;  // pages held and wanted
  unsigned back;       // pages given back
  bool ended, sound;   // sound: non-negative length, pages within the row
};

__device__ __forceinline__ unsigned pages_of(unsigned tokens, int ring) {
  if (ring) return tokens ? (tokens - 1) / kRing * (kRing / kPage) : 0;
  return (tokens + kPage - 1) / kPage;
}

__device__ __forceinline__ Req request(const PlanArgs& a, int ctx, int add) {
  Req r;
  r.ctx = ctx;
  r.ended = add < 0;
  r.add = add < 0 ? 0 : add;
  r.old = ctx < 0 ? 0 : pages_of(ctx, a.ring);
  const unsigned total = (unsigned)ctx + r.add;
  const unsigned all = pages_of(total, a.ring);
  r.sound = ctx >= 0 && total <= kHold && all <= (unsigned)a.max_blocks;
  r.need = r.sound && !r.ended ? all - r.old : 0;
  r.back = r.sound && r.ended ? r.old : 0;
  return r;
}

struct Sums {
  unsigned tok, need, back;
  __device__ __forceinline__ Sums& operator+=(const Sums& o) {
    tok = add_held(tok, o.tok);
    need = add_held(need, o.need);
    back = add_held(back, o.back);
    return *this;
  }
  __device__ __forceinline__ Sums& operator+=(const Req& r) { return *this += Sums{r.add, r.need, r.back}; }
};

__device__ __forceinline__ Sums of_lane(const Sums& s, int lane) {
  return Sums{__shfl_sync(kFull, s.tok, lane), __shfl_sync(kFull, s.need, lane), __shfl_sync(kFull, s.back, lane)};
}
// Inclusive sums over the lanes.
__device__ __forceinline__ Sums scan_warp(Sums s, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up{__shfl_up_sync(kFull, s.tok, o), __shfl_up_sync(kFull, s.need, o), __shfl_up_sync(kFull, s.back, o)};
    if (lane >= o) s += up;
  }
  return s;
}

struct PlanSmem {
  unsigned tok[kPlanThreads], need[kPlanThreads], back[kPlanThreads];  // sums in front of each entry
  int ctx[kPlanThreads], add[kPlanThreads];                           // the requests, where stride is 1
  Sums warp[32];
  unsigned taken[32];
};

// Free pages the step may hand out, and where they start; a state that is not one counts as empty.
struct Queue {
  unsigned head, count;
  bool sound;
};

// A request is served when it is sound, its tokens fit the buffer and its pages the queue.  `at` are the sums in
// front of it; they grow with b, so the pages of the served requests are the first ones of the queue
// without a gap.
__device__ __forceinline__ bool served(const PlanArgs& a, const Queue& q, const Req& r, const Sums& at) {
  return r.sound && (r.add == 0 || at.tok + r.add <= (unsigned)a.max_tokens) && (r.need == 0 || at.need + r.need <= q.count);
}

__device__ __forceinline__ unsigned wrap(unsigned i, unsigned cap) { return i >= cap ? i - cap : i; }

// A free page by its place in the queue; -1 for an id that is not a block.
__device__ __forceinline__ int free_page(const PlanArgs& a, const Queue& q, unsigned k) {
  const int id = a.queue[wrap(q.head + k, a.queue_cap)];
  return id >= 0 && id < a.num_blocks ? id : -1;
}

template <int T>  // tokens of a thread
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a, const int vec) {
  __shared__ PlanSmem sm;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wid = tid >> 5;
  const int stride = (a.batch + nt - 1) / nt;                   // requests per entry
  const int ne = stride ? (a.batch + stride - 1) / stride : 0;  // entries
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- scan of the entries' sums
  const int q_head = a.queue_state[0], q_count = a.queue_state[1];
  Sums own{0, 0, 0};
  const int b0 = tid < ne ? tid * stride : a.batch, b1 = min(b0 + stride, a.batch);
  for (int b = b0; b < b1; ++b) {
    sm.ctx[tid] = a.ctx_len[b];
    sm.add[tid] = a.new_len[b];
    own += request(a, sm.ctx[tid], sm.add[tid]);
  }
  Queue q;
  q.sound = q_count >= 0 && q_count <= a.queue_cap && q_head >= 0 && (q_head < a.queue_cap || a.queue_cap == 0);
  q.head = q.sound ? q_head : 0;
  q.count = q.sound ? q_count : 0;
  const Sums inc = scan_warp(own, lane);
  if (lane == 31) sm.warp[wid] = inc;
  __syncthreads();
  const Sums warps = scan_warp(lane < nt / 32 ? sm.warp[lane] : Sums{0, 0, 0}, lane), total = of_lane(warps, 31);
  // in front of this thread: the warps before, and the lanes before (held sums cannot be subtracted)
  Sums before = of_lane(warps, max(wid - 1, 0));
  if (wid == 0) before = Sums{0, 0, 0};
  const Sums lanes = of_lane(inc, max(lane - 1, 0));
  if (lane) before += lanes;
  sm.tok[tid] = before.tok;
  sm.need[tid] = before.need;
  sm.back[tid] = before.back;
  __syncthreads();
  auto get = [&](int b) {
    return stride == 1 ? request(a, sm.ctx[b], sm.add[b]) : request(a, a.ctx_len[b], a.new_len[b]);
  };
  // The request that item x of the given sums belongs to (x is below their total) and the sums in front of it.
  auto find = [&](const unsigned* sum, unsigned x, unsigned Sums::*which, unsigned Req::*size, Sums& at, Req& r) {
    int lo = 0, hi = ne - 1;  // the last entry that does not begin behind x
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sum[mid] <= x) lo = mid;
      else hi = mid - 1;
    }
    at = Sums{sm.tok[lo], sm.need[lo], sm.back[lo]};
    int b = lo * stride;
    r = get(b);
    while (x >= at.*which + r.*size && b + 1 < a.batch) {
      at += r;
      r = get(++b);
    }
    return b;
  };

  // ---- per-request outputs: this CTA's share of the entries (CTA 0 looks at all for the flags and the queue)
  const int per = (ne + gridDim.x - 1) / gridDim.x;
  const bool mine = tid < ne && tid >= per * (int)blockIdx.x && tid < per * ((int)blockIdx.x + 1);
  uint32_t flags = q.sound ? 0u : TQ_DEVERR_PAGES;
  unsigned taken = 0;
  if (mine || blockIdx.x == 0) {
    Sums at = before;
    for (int b = b0; b < b1; ++b) {
      const Req r = get(b);
      const bool ok = served(a, q, r, at);
      if (ok && r.need) taken = at.need + r.need;
      if (!r.sound) flags |= TQ_DEVERR_POSITION;
      else if (!ok) flags |= TQ_DEVERR_PAGES;
      if (mine) {
        const int len = r.ended ? 0 : ok ? r.ctx + (int)r.add : max(r.ctx, 0);
        const int paged = a.ring ? max(len - 1, 0) / kRing * kRing : len;
        a.lengths[b] = len;
        if (a.n_paged) a.n_paged[b] = paged;
        if (a.n_ring) a.n_ring[b] = len - paged;
        a.token_start[b] = at.tok;
      }
      at += r;
    }
  }
  // pages given back beyond the queue's room cannot be stored: they are dropped and flagged
  const unsigned room = q.sound ? a.queue_cap - q.count : 0, kept = min(total.back, room);
  if (blockIdx.x == 0) {
    taken = __reduce_max_sync(kFull, taken);
    if (lane == 0) sm.taken[wid] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < nt / 32; ++w) taken = max(taken, sm.taken[w]);
      if (kept < total.back) flags |= TQ_DEVERR_PAGES;
      a.token_start[a.batch] = total.tok;
      a.queue_state_out[0] = q.sound ? (a.queue_cap ? wrap(q.head + taken, a.queue_cap) : 0) : q_head;
      a.queue_state_out[1] = q.sound ? q.count - taken + kept : q_count;
    }
    if (flags) flag_error(a.err, flags);
  }

  // tokens from the first thread on, pages from the last: in a small step different warps have them
  const unsigned gn = gridDim.x * nt, gt = blockIdx.x * nt + tid, rt = gn - 1 - gt;
  bool bad = false;

  // ---- new table entries (pages beyond the queue's count go to nobody)
  for (uint64_t j = rt; j < min(total.need, q.count); j += gn) {
    Sums at;
    Req r;
    const int b = find(sm.need, j, &Sums::need, &Req::need, at, r);
    if (!served(a, q, r, at)) continue;
    const int id = free_page(a, q, j);
    bad |= id < 0;
    a.block_table[(int64_t)b * a.max_blocks + r.old + ((unsigned)j - at.need)] = id;
  }

  // ---- pages given back, behind the queue's end
  for (uint64_t j = rt; j < kept; j += gn) {
    Sums at;
    Req r;
    const int b = find(sm.back, j, &Sums::back, &Req::back, at, r);
    const int id = a.block_table[(int64_t)b * a.max_blocks + ((unsigned)j - at.back)];
    bad |= id < 0 || id >= a.num_blocks;  // leaving it out would move every page behind it: a scan over all pages
    a.queue[wrap(wrap(q.head + q.count, a.queue_cap) + (unsigned)j, a.queue_cap)] = id;
  }

  // ---- tokens
  for (uint64_t i0 = (uint64_t)T * gt; i0 < (unsigned)a.max_tokens; i0 += (uint64_t)T * gn) {
    int64_t slot[T];
    int pos[T], row[T];
    Sums at{0, 0, 0};
    Req r;
    int b = -1, id = -1;
    unsigned page = 0xffffffffu;  // the page of request b that id is
    bool ok = false;
    unsigned paged = 0;
    auto open = [&]() {
      ok = served(a, q, r, at);
      const unsigned len = r.ctx + r.add;
      paged = a.ring ? (len - 1) / kRing * kRing : len;  // len > 0: a token is at hand
      page = 0xffffffffu;
    };
#pragma unroll
    for (int k = 0; k < T; ++k) {
      const unsigned i = (unsigned)i0 + k;
      slot[k] = -1;
      pos[k] = row[k] = -1;
      if (i >= total.tok) continue;
      if (b < 0) {
        b = find(sm.tok, i, &Sums::tok, &Req::add, at, r);
        open();
      } else if (i >= at.tok + r.add) {
        do {
          at += r;
          r = get(++b);
        } while (i >= at.tok + r.add && b + 1 < a.batch);
        open();
      }
      const unsigned p = (unsigned)r.ctx + (i - at.tok);
      pos[k] = r.ctx < 0 || p > kHold ? -1 : (int)p;
      row[k] = b;
      if (!ok || p >= paged) continue;
      if (p / kPage != page) {
        page = p / kPage;
        if (page < r.old) {
          id = a.block_table[(int64_t)b * a.max_blocks + page];
          if (id < 0 || id >= a.num_blocks) id = -1;
        } else {
          id = free_page(a, q, at.need + (page - r.old));
        }
      }
      if (id >= 0) slot[k] = (int64_t)id * kPage + p % kPage;
      else bad = true;
    }
    if (T == 4 && vec && i0 + 4 <= (unsigned)a.max_tokens) {
      reinterpret_cast<longlong2*>(a.slots + i0)[0] = make_longlong2(slot[0], slot[T > 1]);
      reinterpret_cast<longlong2*>(a.slots + i0)[1] = make_longlong2(slot[T > 2 ? 2 : 0], slot[T - 1]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[T > 1], pos[T > 2 ? 2 : 0], pos[T - 1]);
      if (a.rows) *reinterpret_cast<int4*>(a.rows + i0) = make_int4(row[0], row[T > 1], row[T > 2 ? 2 : 0], row[T - 1]);
    } else {
#pragma unroll
      for (int k = 0; k < T; ++k) {
        if (i0 + k >= (unsigned)a.max_tokens) break;
        a.slots[i0 + k] = slot[k];
        if (a.positions) a.positions[i0 + k] = pos[k];
        if (a.rows) a.rows[i0 + k] = row[k];
      }
    }
  }
  if (bad) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
}

}  // namespace

cudaError_t launch_plan(tq_ctx* ctx, const PlanArgs& a, cudaStream_t s) {
  // one CTA for a decode step; more when tokens (or rows, whose pages may be many) ask for them
  const int threads = a.batch <= 128 ? 128 : a.batch <= 256 ? 256 : kPlanThreads;
  const int64_t most = 2ll * ctx->sm_count * (kPlanThreads / threads);
  const int tokens = a.max_tokens <= most * threads ? 1 : 4;
  const int64_t work = ((int64_t)a.max_tokens + tokens * threads - 1) / (tokens * threads);
  int64_t grid = work > (a.batch + 63) / 64 ? work : (a.batch + 63) / 64;
  if (grid < 1) grid = 1;
  if (grid > most) grid = most;
  const int vec = ((((uintptr_t)a.slots) | ((uintptr_t)a.positions) | ((uintptr_t)a.rows)) & 15) == 0;
  const cudaError_t e = launch_early(tokens == 1 ? plan_kernel<1> : plan_kernel<4>, dim3((unsigned)grid), dim3(threads), 0, s, a, vec);
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
