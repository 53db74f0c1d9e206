// Page plan of one serving step: block tables, slot maps and the queue of free pages from the
// requests' lengths, in one launch.
//
//   need_b = pages(c_b + n_b) - pages(c_b),  P = exclusive prefix sum of need, T = of n
//   table[b][pages(c_b) + j] = queue[head + P_b + j],  slot of token T_b + i = page of position c_b + i
//
// What bounds it: launch latency and a chain of dependent loads (lengths, then queue, then the
// stores); the data are a few bytes per request and 16 per token.  So nothing is handed from CTA
// to CTA: every CTA scans all lengths itself (one entry of `stride` requests per thread, at most 1024
// entries) and then writes its own share of the rows, pages and tokens, finding the request
// of an item by bisection in the scan.  A second launch for the scan, or CTAs that wait for one
// another, would cost more than the repeated reads (8 bytes per request, from L2).
#include "common.cuh"
#include "paged.cuh"

namespace tq {
namespace {

constexpr int kPlanThreads = 1024;

struct Req {
  int64_t ctx, add;    // tokens held and added
  int64_t old, need;   // pages held and wanted
  int64_t back;        // pages given back
  bool ended, sound;   // sound: non-negative length, pages within the row
};

__device__ __forceinline__ int64_t pages_of(int64_t tokens, int ring) {
  if (ring) return tokens > 0 ? (tokens - 1) / kRing * (kRing / kPage) : 0;
  return (tokens + kPage - 1) / kPage;
}

__device__ __forceinline__ Req request(const PlanArgs& a, int b) {
  Req r;
  r.ctx = a.ctx_len[b];
  const int64_t n = a.new_len[b];
  r.ended = n < 0;
  r.add = n < 0 ? 0 : n;
  r.old = r.ctx < 0 ? 0 : pages_of(r.ctx, a.ring);
  const int64_t all = pages_of(r.ctx + r.add, a.ring);
  r.sound = r.ctx >= 0 && all <= a.max_blocks && r.ctx + r.add <= 0x7fffffff;
  r.need = r.sound && !r.ended ? all - r.old : 0;
  r.back = r.sound && r.ended ? r.old : 0;
  return r;
}

struct Sums {
  int64_t tok, need, back;
  __device__ __forceinline__ Sums& operator+=(const Sums& o) {
    tok += o.tok;
    need += o.need;
    back += o.back;
    return *this;
  }
};

struct PlanSmem {
  int64_t tok[kPlanThreads + 1], need[kPlanThreads + 1], back[kPlanThreads + 1];  // exclusive sums per entry
  Sums warp[32];
  int64_t taken[32];
};

// Free pages the step may hand out, and where they start; a state that is not one counts as empty.
struct Queue {
  int head;
  int64_t count;
  bool sound;
};
__device__ __forceinline__ Queue queue_of(const PlanArgs& a) {
  Queue q;
  q.head = a.queue_state[0];
  q.count = a.queue_state[1];
  q.sound = q.count >= 0 && q.count <= a.queue_cap && q.head >= 0 && (q.head < a.queue_cap || a.queue_cap == 0);
  if (!q.sound) {
    q.head = 0;
    q.count = 0;
  }
  return q;
}

// A request is served when it is sound, its tokens fit the buffer and its pages the queue.  tok and need
// are the sums in front of it; both sums grow with b, so the pages of the served requests are
// the first ones of the queue without a gap.
__device__ __forceinline__ bool served(const PlanArgs& a, const Queue& q, const Req& r, int64_t tok, int64_t need) {
  return r.sound && (r.add == 0 || tok + r.add <= a.max_tokens) && (r.need == 0 || need + r.need <= q.count);
}

__device__ __forceinline__ int64_t wrap(int64_t i, int cap) { return i >= cap ? i - cap : i; }

// A free page by its place in the queue; -1 for an id that is not a block.
__device__ __forceinline__ int free_page(const PlanArgs& a, const Queue& q, int64_t k) {
  const int id = a.queue[wrap(q.head + k, a.queue_cap)];
  return id >= 0 && id < a.num_blocks ? id : -1;
}

// Last entry whose sum in front is <= x (sums ascend; n >= 1).
__device__ __forceinline__ int entry_of(const int64_t* sum, int n, int64_t x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sum[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanArgs a) {
  __shared__ PlanSmem sm;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, wid = tid >> 5;
  const int stride = (a.batch + nt - 1) / nt;                       // requests per entry
  const int ne = stride ? (a.batch + stride - 1) / stride : 0;      // entries
  const Queue q = queue_of(a);
  uint32_t flags = q.sound ? 0u : TQ_DEVERR_PAGES;

  // ---- scan of the entries' sums
  Sums own{0, 0, 0};
  const int b0 = tid < ne ? tid * stride : a.batch, b1 = min(b0 + stride, a.batch);
  for (int b = b0; b < b1; ++b) {
    const Req r = request(a, b);
    own += Sums{r.add, r.need, r.back};
  }
  Sums inc = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums up{__shfl_up_sync(kFull, inc.tok, o), __shfl_up_sync(kFull, inc.need, o),
                  __shfl_up_sync(kFull, inc.back, o)};
    if (lane >= o) inc += up;
  }
  if (lane == 31) sm.warp[wid] = inc;
  __syncthreads();
  Sums before{0, 0, 0}, total{0, 0, 0};
  for (int w = 0; w < nt / 32; ++w) {
    if (w == wid) before = total;
    total += sm.warp[w];
  }
  before += Sums{inc.tok - own.tok, inc.need - own.need, inc.back - own.back};
  sm.tok[tid] = before.tok;
  sm.need[tid] = before.need;
  sm.back[tid] = before.back;
  __syncthreads();

  // ---- per-request outputs: this CTA's share of the entries (CTA 0 looks at all for the flags and the queue)
  const int per = (ne + gridDim.x - 1) / gridDim.x;
  const bool mine = tid / max(per, 1) == (int)blockIdx.x && tid < ne;
  int64_t taken = 0;
  if (mine || blockIdx.x == 0) {
    Sums at = before;
    for (int b = b0; b < b1; ++b) {
      const Req r = request(a, b);
      const bool ok = served(a, q, r, at.tok, at.need);
      if (ok && r.need) taken = at.need + r.need;
      if (!r.sound) flags |= TQ_DEVERR_POSITION;
      else if (!ok) flags |= TQ_DEVERR_PAGES;
      if (mine) {
        const int64_t len = r.ended ? 0 : ok ? r.ctx + r.add : r.ctx < 0 ? 0 : r.ctx;
        const int64_t paged = a.ring ? (len > 0 ? (len - 1) / kRing * kRing : 0) : len;
        a.lengths[b] = (int)len;
        if (a.n_paged) a.n_paged[b] = (int)paged;
        if (a.n_ring) a.n_ring[b] = (int)(len - paged);
        a.token_start[b] = (int)at.tok;
      }
      at += Sums{r.add, r.need, r.back};
    }
  }
  if (blockIdx.x == 0) {
    for (int o = 16; o; o >>= 1) taken = max(taken, __shfl_xor_sync(kFull, taken, o));
    if (lane == 0) sm.taken[wid] = taken;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < nt / 32; ++w) taken = max(taken, sm.taken[w]);
      // pages given back beyond the queue's room cannot be stored: they are dropped and flagged
      const int64_t room = q.sound ? a.queue_cap - q.count : 0;
      const int64_t kept = total.back < room ? total.back : room;
      if (kept < total.back) flags |= TQ_DEVERR_PAGES;
      a.token_start[a.batch] = (int)total.tok;
      a.queue_state_out[0] = q.sound ? (a.queue_cap ? (int)wrap(q.head + taken, a.queue_cap) : 0) : a.queue_state[0];
      a.queue_state_out[1] = q.sound ? (int)(q.count - taken + kept) : a.queue_state[1];
    }
    if (flags) flag_error(a.err, flags);
  }

  // ---- new table entries
  const int64_t gt = (int64_t)blockIdx.x * nt + tid, gn = (int64_t)gridDim.x * nt;
  bool bad = false;
  const int64_t want = total.need < q.count ? total.need : q.count;  // no later page can be handed out
  for (int64_t j = gt; j < want; j += gn) {
    const int e = entry_of(sm.need, ne, j);
    Sums at{sm.tok[e], sm.need[e], 0};
    int b = e * stride;
    Req r = request(a, b);
    while (j >= at.need + r.need) {
      at += Sums{r.add, r.need, 0};
      r = request(a, ++b);
    }
    if (!served(a, q, r, at.tok, at.need)) continue;
    const int id = free_page(a, q, j);
    bad |= id < 0;
    a.block_table[(int64_t)b * a.max_blocks + r.old + (j - at.need)] = id;
  }

  // ---- pages given back, behind the queue's end
  const int64_t room = q.sound ? a.queue_cap - q.count : 0;
  const int64_t kept = total.back < room ? total.back : room;
  for (int64_t j = gt; j < kept; j += gn) {
    const int e = entry_of(sm.back, ne, j);
    int64_t at = sm.back[e];
    int b = e * stride;
    Req r = request(a, b);
    while (j >= at + r.back) {
      at += r.back;
      r = request(a, ++b);
    }
    a.queue[wrap(wrap(q.head + q.count, a.queue_cap) + j, a.queue_cap)] =
        a.block_table[(int64_t)b * a.max_blocks + (j - at)];
  }

  // ---- tokens
  for (int64_t i = gt; i < a.max_tokens; i += gn) {
    int64_t slot = -1;
    int pos = -1, row = -1;
    if (i < total.tok) {
      const int e = entry_of(sm.tok, ne, i);
      Sums at{sm.tok[e], sm.need[e], 0};
      int b = e * stride;
      Req r = request(a, b);
      while (i >= at.tok + r.add) {
        at += Sums{r.add, r.need, 0};
        r = request(a, ++b);
      }
      const int64_t p = r.ctx + (i - at.tok);
      pos = r.ctx < 0 || p > 0x7fffffff ? -1 : (int)p;
      row = b;
      const int64_t len = r.ctx + r.add;
      if (served(a, q, r, at.tok, at.need) && (!a.ring || p < (len - 1) / kRing * kRing)) {
        const int64_t pg = p / kPage;
        int id;
        if (pg < r.old) {
          id = a.block_table[(int64_t)b * a.max_blocks + pg];
          if (id < 0 || id >= a.num_blocks) id = -1;
        } else {
          id = free_page(a, q, at.need + (pg - r.old));
        }
        if (id >= 0) slot = (int64_t)id * kPage + p % kPage;
        else bad = true;
      }
    }
    a.slots[i] = slot;
    if (a.positions) a.positions[i] = pos;
    if (a.rows) a.rows[i] = row;
  }
  if (bad) flag_error(a.err, TQ_DEVERR_BLOCK_ID);
}

}  // namespace

cudaError_t launch_plan(tq_ctx* ctx, const PlanArgs& a, cudaStream_t s) {
  // one CTA for a decode step; more when tokens (or rows, whose pages may be many) ask for them
  const int threads = a.batch <= 256 ? 256 : kPlanThreads;
  const int64_t work = ((int64_t)a.max_tokens + threads - 1) / threads;
  int64_t grid = work > (a.batch + 63) / 64 ? work : (a.batch + 63) / 64;
  if (grid < 1) grid = 1;
  if (grid > ctx->sm_count) grid = ctx->sm_count;
  plan_kernel<<<(int)grid, threads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) ctx->launches++;
  return e;
}

}  // namespace tq
