// cache_api.cpp -- the C entry points around the decode: block tables and slots from
// lengths, rows appended to the cache, rows read back, drafts verified. Argument checks and launches
// only; nothing here allocates or synchronises.
#include <algorithm>
#include <cstring>

#include "cache_ops.h"

namespace da {
// (defined beside the context in api.cpp)
int ctx_device(const da_ctx *ctx);
int ctx_num_sms(const da_ctx *ctx);
bool ctx_planned(const da_ctx *ctx);
const da_problem &ctx_problem(const da_ctx *ctx);
}  // namespace da

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Checks that the calls share.
da_status check_call(const da_ctx *ctx, const void *args, const void *ws, size_t bytes) {
  if (!ctx || !args) return DA_ERR_INVALID_ARG;
  if (!da::ctx_planned(ctx)) return DA_ERR_NOT_PLANNED;
  if (!ws || !aligned(ws, 256) || (int64_t)bytes < da::kWorkspaceHeader) return DA_ERR_WORKSPACE;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return DA_ERR_CUDA;
  if (dev != da::ctx_device(ctx)) return DA_ERR_INVALID_ARG;  // the context's device must be current
  return DA_OK;
}

int kind_of(const da_problem &p) {
  if (p.is_mla) return 5;
  switch (p.kv_dtype) {
    case DA_DTYPE_FP8_E4M3: return 1;
    case DA_DTYPE_FP8_E4M3_TOKEN_SCALE: return 2;
    case DA_DTYPE_INT4_GROUPS: return 3;
    case DA_DTYPE_FP4_E2M1_BLOCKS: return 4;
    case DA_DTYPE_FP8_E4M3_BLOCKS: return 6;
    case DA_DTYPE_INT8_BLOCKS: return 7;
    default: return 0;
  }
}

// The cache's pointers and layout, for both directions.
da_status cache_params(const da_ctx *ctx, const void *k, const void *v, const float *k_scale, const float *v_scale,
                       const int32_t *kss, const int32_t *vss, void *ws, da::CacheRowParams *c) {
  const da_problem &p = da::ctx_problem(ctx);
  const int kind = kind_of(p);
  if (!k || !v || !aligned(k, 16) || !aligned(v, 16)) return DA_ERR_INVALID_ARG;
  if ((kind == 1 || kind == 4 || kind >= 6) && (!k_scale || !v_scale)) return DA_ERR_INVALID_ARG;
  if (kind == 2 && (!kss || !vss)) return DA_ERR_INVALID_ARG;
  c->k = const_cast<void *>(k);
  c->v = const_cast<void *>(v);
  c->k_scale = k_scale;
  c->v_scale = v_scale;
  if (kind >= 6) {
    if (!aligned(k_scale, 4) || !aligned(v_scale, 4)) return DA_ERR_INVALID_ARG;
    c->k_block_scale = const_cast<float *>(k_scale);
    c->v_block_scale = const_cast<float *>(v_scale);
  }
  c->k_scale_shift = const_cast<int32_t *>(kss);
  c->v_scale_shift = const_cast<int32_t *>(vss);
  const bool paged = p.kv_layout == DA_KV_PAGED;
  c->rows_per_page = paged ? p.page_size : p.max_seq_len;
  c->num_slots = (int64_t)(paged ? p.num_pages : p.batch) * c->rows_per_page;
  c->num_kv_heads = p.num_kv_heads;
  c->kv_groups = p.kv_groups;
  c->err = reinterpret_cast<uint32_t *>(ws);
  return DA_OK;
}

da_status append(da_ctx *ctx, const da_append_args *a, const da_norm_args *norm, void *workspace,
                 size_t workspace_bytes, da_stream_t stream) {
  da_status st = check_call(ctx, a, workspace, workspace_bytes);
  if (st != DA_OK) return st;
  const da_problem &p = da::ctx_problem(ctx);
  const bool mla = p.is_mla != 0, has_kv = a->k_new != nullptr;
  if (norm) {
    if (!(norm->eps >= 0.f) || norm->eps > 3.4e38f) return DA_ERR_INVALID_ARG;  // negative, NaN, infinite
    if (!aligned(norm->q_weight, 16) || !aligned(norm->k_weight, 16)) return DA_ERR_INVALID_ARG;
    if ((norm->q_weight && !a->q) || (norm->k_weight && !has_kv)) return DA_ERR_INVALID_ARG;
    if (norm->q_weight && mla) return DA_ERR_UNSUPPORTED;  // (q is the rope part of a query alone)
  }
  if (a->num_tokens < 0 || a->q_len < 0) return DA_ERR_INVALID_ARG;
  if (a->num_tokens == 0) return DA_OK;  // (empty tensors may have no address)
  if ((a->q != nullptr) != (a->q_out != nullptr) || has_kv != (a->v_new != nullptr)) return DA_ERR_INVALID_ARG;
  if (!a->q && !has_kv) return DA_ERR_INVALID_ARG;
  if (has_kv && !a->slot_map) return DA_ERR_INVALID_ARG;
  const int64_t head = mla ? 64 : 128;
  const int64_t need[3] = {p.num_q_heads * head, mla ? 512 : p.num_kv_heads * head, mla ? 64 : p.num_kv_heads * head};
  const void *src[3] = {a->q, a->k_new, a->v_new};
  const int64_t stride[3] = {a->q_stride, a->k_stride, a->v_stride};
  for (int i = 0; i < 3; ++i)
    if (src[i] && (!aligned(src[i], 16) || stride[i] % 8 != 0 || stride[i] < need[i])) return DA_ERR_INVALID_ARG;
  if (!aligned(a->q_out, 16)) return DA_ERR_INVALID_ARG;
  if (a->q_len > 1 && a->q) {
    if (a->q_len != p.q_len || (int64_t)p.batch * a->q_len != a->num_tokens) return DA_ERR_INVALID_ARG;
    if (a->q_out == a->q) return DA_ERR_INVALID_ARG;  // the layouts differ
  }
  if (a->q_out && a->q_out == a->q && a->q_stride != need[0]) return DA_ERR_INVALID_ARG;
  da::CacheRowParams c;
  std::memset(&c, 0, sizeof c);
  if (has_kv) {
    st = cache_params(ctx, a->k, a->v, a->k_scale, a->v_scale, a->k_scale_shift, a->v_scale_shift, workspace, &c);
    if (st != DA_OK) return st;
  } else {
    c.rows_per_page = 1;
    const bool paged = p.kv_layout == DA_KV_PAGED;
    c.num_slots = (int64_t)(paged ? p.num_pages : p.batch) * (paged ? p.page_size : p.max_seq_len);
    c.err = reinterpret_cast<uint32_t *>(workspace);
  }
  if (a->rope_dim < 0 || a->rope_dim > head) return DA_ERR_INVALID_ARG;
  if (a->rope_dim % 16 != 0) return DA_ERR_UNSUPPORTED;
  if (a->rope_adjacent != 0 && a->rope_adjacent != 1) return DA_ERR_INVALID_ARG;
  c.rope_pairs = a->rope_dim / 2;
  if (c.rope_pairs > 0) {
    if (!a->positions || !a->cos_sin || !aligned(a->cos_sin, 16) || a->max_position <= 0) return DA_ERR_INVALID_ARG;
    if (a->rope_axes < 1 || a->rope_axes > 255) return DA_ERR_INVALID_ARG;
    if (a->rope_axes > 1 && a->position_stride < a->num_tokens) return DA_ERR_INVALID_ARG;
    const int group = 8;  // pairs of a lane
    c.rope_whole = 1;
    for (int i = 0; i < c.rope_pairs; ++i) {
      const int ax = a->pair_axis ? a->pair_axis[i] : 0;
      if (ax >= a->rope_axes) return DA_ERR_INVALID_ARG;
      c.pair_axis[i] = (uint8_t)ax;
      if (ax != c.pair_axis[i / group * group]) c.rope_whole = 0;
    }
  }
  c.q = reinterpret_cast<const __nv_bfloat16 *>(a->q);
  c.k_new = reinterpret_cast<const __nv_bfloat16 *>(a->k_new);
  c.v_new = reinterpret_cast<const __nv_bfloat16 *>(a->v_new);
  c.q_stride = a->q_stride;
  c.k_stride = a->k_stride;
  c.v_stride = a->v_stride;
  c.q_out = reinterpret_cast<__nv_bfloat16 *>(a->q_out);
  c.slot_map = a->slot_map;
  c.positions = a->positions;
  c.position_stride = a->position_stride;
  c.cos_sin = a->cos_sin;
  c.max_position = a->max_position;
  c.rope_adjacent = a->rope_adjacent;
  c.num_tokens = a->num_tokens;
  c.num_q_heads = p.num_q_heads;
  c.q_len = a->q_len;
  if (norm) {
    c.q_weight = norm->q_weight;
    c.k_weight = norm->k_weight;
    c.norm_eps = norm->eps;
  }
  const auto s = reinterpret_cast<cudaStream_t>(stream);
  const int kind = kind_of(p), sms = da::ctx_num_sms(ctx);
  const cudaError_t e = kind >= 6 && has_kv ? da::launch_append_blocks(c, kind == 7, sms, s)
                                            : da::launch_append(c, kind >= 6 ? 0 : kind, sms, s);  // (queries alone)
  return e == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // namespace

extern "C" {

da_status decode_attn_build_tables(da_ctx *ctx, const da_table_args *a, void *workspace,
                                   size_t workspace_bytes, da_stream_t stream) {
  da_status st = check_call(ctx, a, workspace, workspace_bytes);
  if (st != DA_OK) return st;
  const da_problem &p = da::ctx_problem(ctx);
  const bool paged = p.kv_layout == DA_KV_PAGED;
  if (!a->seq_lens || !a->new_lens || !a->seq_lens_out || a->slot_capacity < 0) return DA_ERR_INVALID_ARG;
  if (a->slot_capacity > 0 && !a->slot_map) return DA_ERR_INVALID_ARG;
  if (paged != (a->block_table != nullptr)) return DA_ERR_INVALID_ARG;
  const bool alloc = a->free_pages != nullptr;
  if (alloc && (!paged || !a->num_free || !a->num_free_out || a->free_capacity < 0)) return DA_ERR_INVALID_ARG;
  if (!alloc && (a->num_free || a->num_free_out)) return DA_ERR_INVALID_ARG;
  const int64_t capacity = paged ? (int64_t)p.max_pages_per_seq * p.page_size : (int64_t)p.max_seq_len;
  if (capacity >= (1ll << 31)) return DA_ERR_UNSUPPORTED;
  da::TableParams t;
  std::memset(&t, 0, sizeof t);
  t.seq_lens = a->seq_lens;
  t.new_lens = a->new_lens;
  t.free_pages = a->free_pages;
  t.num_free = a->num_free;
  t.block_table = a->block_table;
  t.seq_lens_out = a->seq_lens_out;
  t.num_free_out = a->num_free_out;
  t.slot_map = a->slot_map;
  t.positions = a->positions;
  t.token_row = a->token_row;
  t.cu_new = a->cu_new;
  t.err = reinterpret_cast<uint32_t *>(workspace);
  t.ticket = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(workspace) + da::kTicketOffset);
  t.capacity = capacity;
  t.batch = p.batch;
  t.page_size = paged ? p.page_size : 1;
  t.max_pages = p.max_pages_per_seq;
  t.num_pages = p.num_pages;
  t.free_capacity = a->free_capacity;
  t.slot_capacity = a->slot_capacity;
  t.paged = paged ? 1 : 0;
  t.in_place = (a->seq_lens_out == a->seq_lens || (alloc && a->num_free_out == a->num_free)) ? 1 : 0;
  return da::launch_tables(t, da::ctx_num_sms(ctx), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

da_status decode_attn_append(da_ctx *ctx, const da_append_args *args, void *workspace, size_t workspace_bytes,
                             da_stream_t stream) {
  return append(ctx, args, nullptr, workspace, workspace_bytes, stream);
}

da_status decode_attn_append_normed(da_ctx *ctx, const da_append_args *args, const da_norm_args *norm,
                                    void *workspace, size_t workspace_bytes, da_stream_t stream) {
  if (!norm) return DA_ERR_INVALID_ARG;
  return append(ctx, args, norm, workspace, workspace_bytes, stream);
}

da_status decode_attn_gather(da_ctx *ctx, const da_gather_args *a, void *workspace, size_t workspace_bytes,
                             da_stream_t stream) {
  da_status st = check_call(ctx, a, workspace, workspace_bytes);
  if (st != DA_OK) return st;
  if (a->num_tokens < 0) return DA_ERR_INVALID_ARG;
  if (a->num_tokens == 0) return DA_OK;
  if (!a->slot_map || !a->k_out || !a->v_out) return DA_ERR_INVALID_ARG;
  if (!aligned(a->k_out, 16) || !aligned(a->v_out, 16)) return DA_ERR_INVALID_ARG;
  const da_problem &p = da::ctx_problem(ctx);
  da::CacheRowParams c;
  std::memset(&c, 0, sizeof c);
  st = cache_params(ctx, a->k, a->v, a->k_scale, a->v_scale, a->k_scale_shift, a->v_scale_shift, workspace, &c);
  if (st != DA_OK) return st;
  c.slot_map = a->slot_map;
  c.k_out = reinterpret_cast<__nv_bfloat16 *>(a->k_out);
  c.v_out = reinterpret_cast<__nv_bfloat16 *>(a->v_out);
  c.num_tokens = a->num_tokens;
  return da::launch_gather(c, kind_of(p), da::ctx_num_sms(ctx), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? DA_OK
             : DA_ERR_CUDA;
}

da_status decode_attn_verify(da_ctx *ctx, const da_verify_args *a, void *workspace, size_t workspace_bytes,
                             da_stream_t stream) {
  da_status st = check_call(ctx, a, workspace, workspace_bytes);
  if (st != DA_OK) return st;
  const da_problem &p = da::ctx_problem(ctx);
  const bool paged = p.kv_layout == DA_KV_PAGED, greedy = a->target_tokens != nullptr;
  if (a->q_len < 1 || a->vocab < 1 || !a->tokens_out || !a->num_accepted) return DA_ERR_INVALID_ARG;
  if (greedy == (a->target_probs != nullptr) || (greedy && (a->draft_probs || a->uniforms))) return DA_ERR_INVALID_ARG;
  if (a->q_len > 1 && !a->draft_tokens) return DA_ERR_INVALID_ARG;
  if (!aligned(a->target_probs, 4) || !aligned(a->draft_probs, 4) || !aligned(a->uniforms, 4)) return DA_ERR_INVALID_ARG;
  if (!greedy && (!a->uniforms || a->target_stride < a->vocab)) return DA_ERR_INVALID_ARG;
  if (a->draft_probs && a->q_len > 1 && a->draft_stride < a->vocab) return DA_ERR_INVALID_ARG;
  if ((a->seq_lens != nullptr) != (a->seq_lens_out != nullptr)) return DA_ERR_INVALID_ARG;
  if (a->seq_lens_before && !a->seq_lens) return DA_ERR_INVALID_ARG;
  const bool gives = a->free_pages != nullptr;
  if (gives && (!paged || !a->seq_lens || !a->block_table || !a->num_free || !a->num_free_out || a->free_capacity < 0))
    return DA_ERR_INVALID_ARG;
  if (!gives && (a->block_table || a->num_free || a->num_free_out)) return DA_ERR_INVALID_ARG;
  // (the segments' sums of a row are in shared memory; CTAs are counted in 31 bits)
  if (a->vocab > (1 << 21) || a->q_len > (1 << 20) || p.batch > (1 << 27)) return DA_ERR_UNSUPPORTED;
  const int64_t capacity = paged ? (int64_t)p.max_pages_per_seq * p.page_size : (int64_t)p.max_seq_len;
  if (capacity >= (1ll << 31)) return DA_ERR_UNSUPPORTED;
  da::VerifyParams v;
  std::memset(&v, 0, sizeof v);
  v.target = a->target_probs;
  v.draft = a->draft_probs;
  v.target_stride = a->target_stride;
  v.draft_stride = a->draft_stride;
  v.target_tokens = a->target_tokens;
  v.draft_tokens = a->draft_tokens;
  v.num_draft = a->num_draft;
  v.uniforms = a->uniforms;
  v.tokens_out = a->tokens_out;
  v.num_accepted = a->num_accepted;
  v.seq_lens = a->seq_lens;
  v.seq_lens_before = a->seq_lens_before;
  v.seq_lens_out = a->seq_lens_out;
  v.block_table = a->block_table;
  v.free_pages = a->free_pages;
  v.num_free = a->num_free;
  v.num_free_out = a->num_free_out;
  v.err = reinterpret_cast<uint32_t *>(workspace);
  v.ticket = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(workspace) + da::kVerifyTicketOffset);
  v.capacity = capacity;
  v.batch = p.batch;
  v.q_len = a->q_len;
  v.vocab = a->vocab;
  v.free_capacity = a->free_capacity;
  v.page_size = paged ? p.page_size : 1;
  v.max_pages = p.max_pages_per_seq;
  v.num_pages = p.num_pages;
  return da::launch_verify(v, da::ctx_num_sms(ctx), reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? DA_OK : DA_ERR_CUDA;
}

}  // extern "C"
