// Argument checks of the page plan and of the dense-layout page calls, the choice of the attention's
// translation unit and the TMA descriptor of a pool.
#include <limits.h>
#include <math.h>

#include "paged.cuh"

namespace {

tq_status cuda_status(cudaError_t e) { return e == cudaSuccess ? TQ_OK : TQ_ERR_CUDA; }

// The context's error word and the caller's tensors live on the context's device: a launch from
// another current device would touch memory of the wrong one.
bool on_device(const tq_ctx* ctx) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == ctx->device;
}

bool aligned16(const void* p) { return (((uintptr_t)p) & 15) == 0; }

}  // namespace

namespace tq {

bool encode_paged_map(const PagedTensorMap& t, CUtensorMap* map) {
  // the driver's encoder, looked up once (the library is not linked against libcuda)
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<Encode>(f);
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)t.d, 2 * kPage, (cuuint64_t)t.tiles};
  const cuuint64_t strides[2] = {(cuuint64_t)t.d * t.elem, (cuuint64_t)t.tile_bytes};
  const cuuint32_t box[3] = {(cuuint32_t)(t.row_bytes / t.elem), (cuuint32_t)t.box_rows, 1}, step[3] = {1, 1, 1};
  return encode(map, t.elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_UINT16, 3,
                const_cast<void*>(t.pool), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                t.row_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

size_t paged_workspace(const tq_ctx* ctx, int batch) {
  const tq_config& c = ctx->cfg;
  return c.key_bits == 8 ? paged_workspace_e4m3(ctx, batch)
         : c.key_format == TQ_ELEM_BF16 ? paged_workspace_bf16(ctx, batch) : paged_workspace_f16(ctx, batch);
}

cudaError_t launch_paged(tq_ctx* ctx, const PagedArgs& a, void* workspace, cudaStream_t s) {
  const tq_config& c = ctx->cfg;
  return c.key_bits == 8 ? launch_paged_e4m3(ctx, a, workspace, s)
         : c.key_format == TQ_ELEM_BF16 ? launch_paged_bf16(ctx, a, workspace, s) : launch_paged_f16(ctx, a, workspace, s);
}

}  // namespace tq

extern "C" {

tq_status tq_plan_pages(tq_ctx* ctx, const int32_t* ctx_len, const int32_t* new_len, int batch, int ring_capacity,
                        int32_t* block_table, int max_blocks, int num_blocks, int32_t* queue, int queue_cap,
                        const int32_t* queue_state, int32_t* lengths, int32_t* n_paged, int32_t* n_ring,
                        int32_t* token_start, int64_t* slots, int32_t* positions, int32_t* rows, int max_tokens,
                        int32_t* queue_state_out, cudaStream_t stream) {
  if (!ctx || batch < 0 || max_blocks < 0 || num_blocks < 0 || queue_cap < 0 || max_tokens < 0)
    return TQ_ERR_INVALID_ARG;
  if (ring_capacity != 0 && ring_capacity != tq::kRing) return TQ_ERR_UNSUPPORTED;
  if (max_blocks > INT_MAX / tq::kPage) return TQ_ERR_INVALID_ARG;  // positions are int32
  if (!token_start || !queue_state || !queue_state_out || queue_state == queue_state_out) return TQ_ERR_INVALID_ARG;
  if (batch > 0 && (!ctx_len || !new_len || !lengths || lengths == ctx_len || lengths == new_len))
    return TQ_ERR_INVALID_ARG;
  if ((batch > 0 && max_blocks > 0 && !block_table) || (queue_cap > 0 && !queue) || (max_tokens > 0 && !slots))
    return TQ_ERR_INVALID_ARG;
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  tq::PlanArgs a;
  a.ctx_len = ctx_len;
  a.new_len = new_len;
  a.batch = batch;
  a.ring = ring_capacity;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.num_blocks = num_blocks;
  a.queue = queue;
  a.queue_cap = queue_cap;
  a.queue_state = queue_state;
  a.lengths = lengths;
  a.n_paged = n_paged;
  a.n_ring = n_ring;
  a.token_start = token_start;
  a.slots = slots;
  a.positions = positions;
  a.rows = rows;
  a.max_tokens = max_tokens;
  a.queue_state_out = queue_state_out;
  a.err = ctx->d_err;
  return cuda_status(tq::launch_plan(ctx, a, stream));
}

tq_status tq_paged_store(tq_ctx* ctx, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
                         const int64_t* slots, int n_tokens, void* pool, int num_blocks, cudaStream_t stream) {
  if (!ctx || n_tokens < 0 || num_blocks < 0) return TQ_ERR_INVALID_ARG;
  if (ctx->cfg.layout != TQ_LAYOUT_DENSE) return TQ_ERR_UNSUPPORTED;
  if (n_tokens == 0) return TQ_OK;
  const int64_t row = (int64_t)ctx->cfg.num_kv_heads * ctx->cfg.head_dim;
  if (!k || !v || !slots || (num_blocks > 0 && !pool) || !aligned16(k) || !aligned16(v) || !aligned16(pool)) return TQ_ERR_INVALID_ARG;
  if (k_stride < row || v_stride < row || (k_stride | v_stride) & 7) return TQ_ERR_INVALID_ARG;
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  tq::StoreArgs a;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.slots = slots;
  a.n_tokens = n_tokens;
  a.pool = static_cast<uint8_t*>(pool);
  a.num_blocks = num_blocks;
  a.hkv = ctx->cfg.num_kv_heads;
  a.err = ctx->d_err;
  return cuda_status(tq::launch_store(ctx, a, stream));
}

tq_status tq_paged_workspace_size(const tq_ctx* ctx, int batch, size_t* bytes) {
  if (!ctx || !bytes || batch < 0) return TQ_ERR_INVALID_ARG;
  if (ctx->cfg.layout != TQ_LAYOUT_DENSE) return TQ_ERR_UNSUPPORTED;
  *bytes = tq::paged_workspace(ctx, batch);
  return TQ_OK;
}

tq_status tq_set_wait_limit(tq_ctx* ctx, uint32_t nanoseconds) {
  if (!ctx) return TQ_ERR_INVALID_ARG;
  ctx->wait_limit = nanoseconds;
  return TQ_OK;
}

tq_status tq_paged_attention(tq_ctx* ctx, const void* q, int64_t q_stride, int batch, const void* pool, int num_blocks,
                             const int32_t* block_table, int max_blocks, const int32_t* lengths, int window,
                             float scale, float* out, float* lse, void* workspace, size_t ws_bytes,
                             cudaStream_t stream) {
  if (!ctx || batch < 0 || num_blocks < 0 || max_blocks < 0 || window < 0) return TQ_ERR_INVALID_ARG;
  if (ctx->cfg.layout != TQ_LAYOUT_DENSE) return TQ_ERR_UNSUPPORTED;
  if (!isfinite(scale)) return TQ_ERR_INVALID_ARG;
  if (batch == 0) return TQ_OK;
  const tq_config& c = ctx->cfg;
  if (!q || !out || !lengths || (max_blocks > 0 && !block_table) || (num_blocks > 0 && !pool))
    return TQ_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(out) || !aligned16(pool) || (q_stride & 7) ||
      q_stride < (int64_t)c.num_q_heads * c.head_dim)
    return TQ_ERR_INVALID_ARG;
  if (max_blocks > INT_MAX / tq::kPage || (int64_t)num_blocks * c.num_kv_heads > INT_MAX) return TQ_ERR_INVALID_ARG;
  if (!workspace || ws_bytes < tq::paged_workspace(ctx, batch)) return TQ_ERR_WORKSPACE;
  if (((uintptr_t)workspace) & 255) return TQ_ERR_INVALID_ARG;
  if (!on_device(ctx)) return TQ_ERR_INVALID_ARG;
  tq::PagedArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.batch = batch;
  a.pool = static_cast<const uint8_t*>(pool);
  a.num_blocks = num_blocks;
  a.block_table = block_table;
  a.max_blocks = max_blocks;
  a.lengths = lengths;
  a.window = window;
  a.scale = scale == 0.f ? (float)(1.0 / sqrt((double)c.head_dim)) : scale;
  a.out = out;
  a.lse = lse;
  a.hq = c.num_q_heads;
  a.hkv = c.num_kv_heads;
  a.n_rep = c.num_q_heads / c.num_kv_heads;
  a.err = ctx->d_err;
  return cuda_status(tq::launch_paged(ctx, a, workspace, stream));
}

}  // extern "C"
