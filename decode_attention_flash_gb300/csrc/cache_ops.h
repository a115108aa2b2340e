// cache_ops.h -- host/device structures of the cache calls (cache_api.cpp, cache_rows.cu,
// cache_blocks.cu, tables.cu) and of the decode over caches in granules (stream_split.cuh).
#pragma once

#include "internal.h"

namespace da {

// The workspace's header (kWorkspaceHeader bytes) is the error word at byte 0 and, in what the
// decode kernels know as its padding, build_tables' block counter here, zero between calls.
constexpr int64_t kTicketOffset = 64;
constexpr int64_t kVerifyTicketOffset = 128;  // and that of decode_attn_verify

// Decode over a cache in granules of 16 rows, read through their addresses (stream_split.cuh):
// 4-bit floats (fp4_split.cu, 1152 bytes each) or 8-bit blocks (block8_split.cu, 2048 bytes);
// o_head holds, per CTA and warp, the piece of a unit that ended inside that warp's range.
struct StreamParams {
  GqaParams g;                 // (8-bit blocks: k_scale, v_scale are the blocks' scales)
  const uint8_t *k, *v;
  float *o_head;               // [ctas][warps][G][128]
  int32_t whole;               // CTA c has unit c, whole (the grid is the units)
  int32_t kv_shift;            // a kv head's queries are 2^kv_shift units (g.num_kv_heads counts those)
  int32_t few_tiles, few_ctas; // a call of at most few_tiles tiles takes at most few_ctas CTAs
  int32_t scale_shift;         // 8-bit blocks: a granule's byte offset to the index of its block's scale
};

// Which instantiation a call's score and mask modifications need: 0 none; 1
// several query tokens, a draft-tree mask, a soft cap; 2 the flex-style mods too.
inline int gqa_mod(const GqaParams &p) {
  return (p.mask_window != nullptr || p.alibi_slopes != nullptr)
             ? 2
             : (p.q_len > 1 || p.spec_mask != nullptr || p.softcap_l2 > 0.f) ? 1 : 0;
}

// Rows of the cache written (append) or read back (gather), cache_rows.cu and cache_blocks.cu. A
// slot is page * rows_per_page + offset (contiguous: batch row * cache length +
// position, rows_per_page the cache length).
struct CacheRowParams {
  const __nv_bfloat16 *q, *k_new, *v_new;  // rows of a token, strides in elements
  int64_t q_stride, k_stride, v_stride;
  __nv_bfloat16 *q_out;        // [T][HQ][D], or [B][HQ][q_len][D] when q_len > 1
  void *k, *v;                 // the cache
  const float *k_scale, *v_scale;
  int32_t *k_scale_shift, *v_scale_shift;
  const int64_t *slot_map;     // [T]; -1 is padding; null: queries only
  int64_t num_slots;
  const int32_t *positions;    // [axes][T], rows position_stride apart
  int64_t position_stride;
  const float *cos_sin;        // [max_position][2 * rope_pairs]: cosines, then sines
  __nv_bfloat16 *k_out, *v_out;  // gather: [T][HKV][D] each (latent: [T][512], [T][64])
  uint32_t *err;
  int32_t num_tokens, num_q_heads, num_kv_heads, rows_per_page, kv_groups, q_len;
  int32_t max_position, rope_pairs;
  int32_t rope_adjacent;       // pairs are elements 2i, 2i + 1 (else i, i + n)
  int32_t rope_whole;          // a lane's pairs share an axis (vector loads of the table)
  int32_t parts;               // warps a token's heads are spread over (the launcher's)
  const float *q_weight, *k_weight;  // the norm's weights of a head (latent: k_weight of 512); null: no norm
  float norm_eps;
  float *k_block_scale, *v_block_scale;  // 8-bit blocks: [pages][HKV][rows_per_page / kv_groups]
  uint8_t pair_axis[64];
};
// The append of 8-bit blocks: the launcher's choices.
struct BlockRowParams : CacheRowParams {
  int32_t warp_rows;           // rows of a block that a warp has
  int32_t window;              // tokens that one group of warps looks through
  int32_t num_axes;            // the distinct axes in pair_axis, and those
  uint8_t axes[64];
};

// decode_attn_build_tables, tables.cu.
struct TableParams {
  const int32_t *seq_lens, *new_lens;  // [B]
  const int32_t *free_pages, *num_free;  // null: the table already holds every page
  int32_t *block_table;        // [B][max_pages]
  int32_t *seq_lens_out, *num_free_out;
  int64_t *slot_map;           // [slot_capacity]
  int32_t *positions, *token_row, *cu_new;  // optional
  uint32_t *err, *ticket;
  int64_t capacity;            // positions a row can hold
  int32_t batch, page_size, max_pages, num_pages, free_capacity, slot_capacity;
  int32_t paged, in_place;     // in_place: an output overlaps an input that every block reads
};

// decode_attn_verify, verify.cu.
struct VerifyParams {
  const float *target, *draft;         // [B][Q][V], [B][Q - 1][V], rows *_stride on; draft null: certain drafts
  int64_t target_stride, draft_stride;
  const int32_t *target_tokens;        // [B][Q] instead of probabilities
  const int32_t *draft_tokens, *num_draft;
  const float *uniforms;               // [B][Q]
  int32_t *tokens_out, *num_accepted;
  const int32_t *seq_lens;             // optional
  const int32_t *seq_lens_before;      // optional: those before the step's tokens
  int32_t *seq_lens_out;
  const int32_t *block_table;          // with free_pages
  int32_t *free_pages;                 // optional
  const int32_t *num_free;
  int32_t *num_free_out;
  uint32_t *err, *ticket;
  int64_t capacity;                    // positions a row can hold
  int32_t batch, q_len, vocab, free_capacity, page_size, max_pages, num_pages;
};

// Launches a kernel that begins with wait_for_previous_kernel (cache_ptx.cuh), so that its
// blocks may take their places while the stream's previous kernel drains: a
// launch after another one of ours costs about 1.5 us less. Ordering is that of the
// stream, as for any launch, also in captured graphs.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), unsigned grid, unsigned block, size_t smem,
                             cudaStream_t stream, const Args &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Params(args)...);
}

// Kinds whose decode is stream_split.cuh.
inline bool is_block8(const da_problem &p) {
  return p.kv_dtype == DA_DTYPE_FP8_E4M3_BLOCKS || p.kv_dtype == DA_DTYPE_INT8_BLOCKS;
}
inline bool is_stream(const da_problem &p) { return p.kv_dtype == DA_DTYPE_FP4_E2M1_BLOCKS || is_block8(p); }
cudaError_t fp4_prepare();
cudaError_t block8_prepare();
int fp4_tile();                // tokens per stage
int block8_tile(int group);
int fp4_warps(int group);      // warps of a CTA for `group` rows per unit
int block8_warps(int group);
inline int stream_tile(const da_problem &p, int group) { return is_block8(p) ? block8_tile(group) : fp4_tile(); }
inline int stream_warps(const da_problem &p, int group) { return is_block8(p) ? block8_warps(group) : fp4_warps(group); }
// log2 of the units that a kv head's queries are split into, so that each has at most 16 rows
// (one query token, dense); -1: no such split.
int stream_kv_shift(const da_problem &p);
cudaError_t launch_fp4(const StreamParams &p, int ctas, cudaStream_t stream);
cudaError_t launch_block8(const StreamParams &p, bool integers, int ctas, cudaStream_t stream);
// Byte offset of StreamParams::o_head in the workspace (after the partial LSEs).
int64_t stream_head_offset(const da_plan_info &info);
void stream_few(const da_problem &p, const da_plan_info &info, const int32_t *seq_lens_host,
                int32_t num_splits_override, int32_t *few_tiles, int32_t *few_ctas);

cudaError_t launch_append(CacheRowParams p, int kind, int num_sms, cudaStream_t stream);
cudaError_t append_blocks_prepare();  // sets shared-memory attributes
cudaError_t launch_append_blocks(const CacheRowParams &p, bool integers, int num_sms, cudaStream_t stream);
cudaError_t launch_gather(CacheRowParams p, int kind, int num_sms, cudaStream_t stream);
cudaError_t launch_verify(const VerifyParams &p, int num_sms, cudaStream_t stream);
cudaError_t launch_tables(const TableParams &p, int num_sms, cudaStream_t stream);

}  // namespace da
