// cache_blocks.cu -- decode_attn_append into a cache of 8-bit codes with an fp32 scale for each
// block of positions and kv head (DA_DTYPE_FP8_E4M3_BLOCKS, DA_DTYPE_INT8_BLOCKS).
//
// The mathematics. A block of n positions of one head keeps codes x / s. Its scale s is the least
// power of two that brings the greatest |x| written to it into the codes' range, and it only grows
// until the block is started anew by its first row. Powers of two, because a block fills over many
// calls: rows that stay are rounded again when s grows, and a doubled scale costs an integer code at
// most half a step (of the new scale; the halves before it were of smaller steps, so all of them
// together stay below one) and an e4m3 code nothing but its subnormal bits. With scales amax / 127 each
// of n calls could add half a step. An e4m3 code keeps its precision under any scale; an integer
// loses half a bit on average.
//
// The layout. The tokens of one block (a run, neighbours in slot_map) are the work of a group of
// n / 16 warps, for one head and K or V: a warp holds 16 of their rows in registers (two rows of 16 lanes at a
// time, as in cache_rows.cu), normed and turned; the greatest |x| of the group's warps meets in shared
// memory; then the rows go out as codes. So a row is read once. Only where the scale grew the
// group reads the block's other rows, 16 a warp, and writes them rounded again. Runs are found by the warps
// themselves: a group looks through a window of tokens for those whose predecessor is in another block.
// Queries are the other blocks of the grid, as in cache_rows.cu.
#include <algorithm>

#include "cache_rows.cuh"

namespace da {
namespace {

constexpr int kRows = 16;      // rows of a run, and of a block, that a warp has
constexpr int kMinWarps = 4;   // of a CTA
constexpr int kMaxWarps = 16;

template <bool INT>
__device__ __forceinline__ float max_of(float a, float b) {
  return INT ? max_nan(a, b) : fmaxf(a, b);  // (an e4m3 code can be NaN by itself)
}

// The least power of two that brings |x| <= a into the codes' range: 448 = 1.75 2^8, 127 = 1.984375 2^6.
// 0 for 0; at least 2^-126, and for infinity that of the greatest bf16.
template <bool INT>
__device__ __forceinline__ float least_scale(float a) {
  if (!(a > 0.f)) return a == 0.f ? 0.f : a;  // (NaN stays)
  const uint32_t u = __float_as_uint(fminf(a, 3.3895313892515355e38f));
  const int e = (int)(u >> 23) - (INT ? 6 : 8) + ((u & 0x7FFFFFu) > (INT ? 0x7E0000u : 0x600000u) ? 1 : 0);
  return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// Four quotients as codes.
template <bool INT>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  if (INT) {
    auto code = [](float x) { return (uint32_t)(__float2int_rn(fminf(fmaxf(x, -127.f), 127.f)) & 0xFF); };
    return code(a) | (code(b) << 8) | (code(c) << 16) | (code(d) << 24);
  }
  return f32x2_to_e4m3x2(a, b) | (f32x2_to_e4m3x2(c, d) << 16);
}
// Four codes times `ratio`, as codes.
template <bool INT>
__device__ __forceinline__ uint32_t again4(uint32_t w, float ratio) {
  float x[4];
  if (INT) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)(w >> (8 * i));
  } else {
    const uint32_t h[2] = {e4m3x2_to_f16x2((uint16_t)w), e4m3x2_to_f16x2((uint16_t)(w >> 16))};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  return codes4<INT>(x[0] * ratio, x[1] * ratio, x[2] * ratio, x[3] * ratio);
}

// Whether every position that turns a pair of token t is in the table.
__device__ __forceinline__ bool positions_ok(const CacheRowParams &p, int64_t t) {
  bool ok = true;
  int last = -1;
  for (int i = 0; i < p.rope_pairs; ++i) {
    const int a = p.pair_axis[i];
    if (a == last) continue;
    last = a;
    const int pos = p.positions[(int64_t)a * p.position_stride + t];
    ok = ok && pos >= 0 && pos < p.max_position;
  }
  return ok;
}

// The first kv_blocks CTAs have the keys and values, the others the queries (a warp a part of a token).
template <bool INT, bool NORM>
__global__ void __launch_bounds__(kMaxWarps * 32) append_blocks_kernel(const __grid_constant__ CacheRowParams p,
                                                                       const int kv_blocks) {
  __shared__ uint32_t written_all[kMinWarps][8];  // rows of the block that the run writes, per group
  __shared__ float amax_all[kMaxWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  begin_dependent();
  if ((int)blockIdx.x >= kv_blocks) {
    const int64_t item = (int64_t)((int)blockIdx.x - kv_blocks) * warps + warp;
    const int64_t t = item / p.parts;
    const int part = (int)(item - t * p.parts);
    if (t >= p.num_tokens) return;
    const int nq = (p.num_q_heads + 3) / 4;
    const QueryLane<128> ql(p, lane);
    int64_t slot;
    float c[8], s[8];
    append_queries<128, NORM>(p, t, lane, ql, (int)((int64_t)part * nq / p.parts),
                              (int)((int64_t)(part + 1) * nq / p.parts), p.num_q_heads, slot, c, s);
    return;
  }
  const int n = p.kv_groups, shift = 31 - __clz(n), gw = n / kRows;  // a block's rows, a group's warps
  const int group = warp / gw, gwarp = warp - group * gw, HK = p.num_kv_heads;
  const int64_t windows = ((int64_t)p.num_tokens + p.window - 1) / p.window;
  const int64_t item = (int64_t)blockIdx.x * (warps / gw) + group;
  if (item >= windows * HK * 2) return;
  const int64_t w0 = item / (2 * HK) * p.window;
  const int h = (int)(item % (2 * HK)) >> 1, side = (int)(item & 1);  // side 0: K
  uint32_t *written = written_all[group];
  float *amax = amax_all + group * gw;
  auto meet = [&]() {
    if (gw == 1) __syncwarp();
    else named_barrier_sync(1 + group, gw * 32);
  };
  const bool tells = h == 0 && side == 0 && gwarp == 0;  // of bad slots and positions
  const uint4 *src = reinterpret_cast<const uint4 *>(side ? p.v_new : p.k_new) + h * 16;
  const int64_t stride = (side ? p.v_stride : p.k_stride) / 8;
  uint8_t *cache = reinterpret_cast<uint8_t *>(side ? p.v : p.k);
  float *scales = side ? p.v_block_scale : p.k_block_scale;

  // a row: 16 lanes of 8 elements, two rows a warp
  const int kl = lane & 15, sub = lane >> 4, r = side ? 0 : p.rope_pairs / 8;
  const bool turned = kl < 2 * r, second = turned && !p.rope_adjacent && kl >= r;
  const int partner = lane - kl + (turned && !p.rope_adjacent ? (second ? kl - r : kl + r) : kl);
  const bool norm = NORM && side == 0 && p.k_weight != nullptr;
  float wo[8], wp[8];
  if (norm) {
    load8(p.k_weight + 8 * kl, wo);
    load8(p.k_weight + 8 * (partner & 15), wp);
  }

  auto block_of = [&](int64_t t) -> int64_t {  // -1: padding or outside the cache
    const int64_t s = p.slot_map[t];
    return s < 0 || s >= p.num_slots ? -1 : s >> shift;
  };
  uint32_t err = 0;
  uint32_t leads;  // tokens of the window whose run starts there
  {
    const int64_t t = w0 + lane;
    const bool in = lane < p.window && t < p.num_tokens;
    const int64_t b = in ? block_of(t) : -1;
    if (in && b < 0 && p.slot_map[t] != -1) err |= DA_DEVERR_SLOT;
    leads = __ballot_sync(0xffffffffu, b >= 0 && (t == 0 || block_of(t - 1) != b));
  }
  for (; leads != 0; leads &= leads - 1) {
    const int64_t t0 = w0 + __ffs(leads) - 1, blk = block_of(t0);
    const int64_t unit = blk / (p.rows_per_page >> shift), j = blk - unit * (p.rows_per_page >> shift);  // page, block in it
    const int64_t row0 = (unit * HK + h) * p.rows_per_page + j * n;
    float *scale = scales + (unit * HK + h) * (p.rows_per_page >> shift) + j;
    const float was = *scale;
    // ---- which tokens, and which rows they write
    bool fresh = false;
    uint32_t mine = 0;  // of the warp's 16 tokens, those that are written
    int my_off = 0;     // lane i < 16: the row of the i-th
    for (int base = 0; base < n; base += 32) {
      const int64_t t = t0 + base + lane;
      const bool in = base + lane < n && t < p.num_tokens;
      const bool same = in && block_of(t) == blk;
      const uint32_t run = __ballot_sync(0xffffffffu, same);
      const int m = run == 0xffffffffu ? 32 : __ffs(~run) - 1;  // up to the first of another block
      bool use = lane < m;
      if (use && !positions_ok(p, t)) {
        err |= DA_DEVERR_POSITION;
        use = false;
      }
      const int off = use ? (int)(p.slot_map[t] & (n - 1)) : -1;
      fresh = fresh || __any_sync(0xffffffffu, off == 0);
      const uint32_t used = __ballot_sync(0xffffffffu, use);
      const int o16 = __shfl_sync(0xffffffffu, off, (gwarp & 1) * 16 + (lane & 15));
      if (base / 32 == gwarp / 2) {
        mine = (used >> ((gwarp & 1) * 16)) & 0xFFFFu;
        my_off = o16;
      }
      if (gwarp == 0) {  // (a run of one block: every row once)
        if (base == 0 && lane < 8) written[lane] = 0;
        __syncwarp();
        if (use) atomicOr(&written[off >> 5], 1u << (off & 31));
      }
      if (m < 32) break;
    }
    // ---- the warp's rows: read, normed, turned, in bf16
    uint4 x[kRows / 2];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((mine >> (2 * i + sub)) & 1u) x[i] = src[(t0 + gwarp * kRows + 2 * i + sub) * stride + kl];
    }
#pragma unroll 2
    for (int i = 0; i < kRows / 2; ++i) {
      if (((mine >> (2 * i)) & 3u) == 0) continue;
      const bool on = (mine >> (2 * i + sub)) & 1u;
      const int64_t t = t0 + gwarp * kRows + 2 * i + sub;
      if (r > 0 || norm) {
        float c[8], s[8];
        if (on && turned) {
          if (p.rope_adjacent) load_turn<4>(p, t, 4 * kl, c, s);
          else load_turn<8>(p, t, 8 * (second ? kl - r : kl), c, s);
          if (second)  // (b c + a s) is (x c - u s) with s of the other sign
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = -s[k];
        }
        if (norm) norm_key(p, x[i], kl, partner, turned, c, s, wo, wp);
        else turn_key(p, x[i], partner, turned, c, s);
      }
      float e[8];
      values8(x[i], e);
#pragma unroll
      for (int k = 0; k < 8; ++k) top = on ? max_of<INT>(top, fabsf(e[k])) : top;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = max_of<INT>(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) amax[gwarp] = top;
    meet();
    for (int i = 0; i < gw; ++i) top = max_of<INT>(top, amax[i]);
    // ---- the scale
    const float old = fresh ? 0.f : was, need = least_scale<INT>(top);
    const float now = old == old ? (need > old || need != need ? need : old) : old;
    const float inv = now != 0.f ? __frcp_rn(now) : 0.f;
#pragma unroll
    for (int i = 0; i < kRows / 2; ++i) {
      const int off = __shfl_sync(0xffffffffu, my_off, 2 * i + sub);
      if ((mine >> (2 * i + sub)) & 1u) {
        float e[8];
        values8(x[i], e);
        *reinterpret_cast<uint2 *>(cache + (row0 + off) * 128 + kl * 8) =
            make_uint2(codes4<INT>(e[0] * inv, e[1] * inv, e[2] * inv, e[3] * inv),
                       codes4<INT>(e[4] * inv, e[5] * inv, e[6] * inv, e[7] * inv));
      }
    }
    // ---- rows that stay, rounded again
    if (!fresh && now > old) {
      const float ratio = old * inv;
      const uint32_t keep = ~(written[gwarp >> 1] >> ((gwarp & 1) * 16));
      uint4 *rows = reinterpret_cast<uint4 *>(cache + (row0 + gwarp * kRows) * 128) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // four rows of 8 lanes
        if ((keep >> (4 * i + (lane >> 3))) & 1u) {
          const uint4 a = rows[32 * i];
          rows[32 * i] = make_uint4(again4<INT>(a.x, ratio), again4<INT>(a.y, ratio), again4<INT>(a.z, ratio),
                                    again4<INT>(a.w, ratio));
        }
    }
    if (gwarp == 0 && lane == 0 && (fresh || !(now == was))) *scale = now;
    meet();  // (the next run writes `amax` and `written`)
  }
  if (tells && err) atomicOr(p.err, err);
}

}  // namespace

cudaError_t launch_append_blocks(CacheRowParams p, bool integers, int num_sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int gw = p.kv_groups / kRows, warps = std::max(kMinWarps, gw);
  // Windows of one token while that makes few warps (a decode step: every token a run of its own), else
  // wider ones, up to half a block: most groups then find no run and end, or one.
  const int64_t one = (int64_t)p.num_tokens * p.num_kv_heads * 2 * gw;
  int window = 1;
  while (window < 32 && window * 2 <= p.kv_groups && one / window > (int64_t)num_sms * 64) window *= 2;
  p.window = window;
  const int64_t items = ((int64_t)p.num_tokens + window - 1) / window * p.num_kv_heads * 2;
  const int64_t kv_blocks = (items + warps / gw - 1) / (warps / gw);
  int64_t q_blocks = 0;
  p.parts = 1;
  if (p.q) {
    const int64_t groups = (p.num_q_heads + 3) / 4;
    p.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)num_sms * 32 / p.num_tokens));
    q_blocks = ((int64_t)p.num_tokens * p.parts + warps - 1) / warps;
  }
  if (kv_blocks + q_blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(kv_blocks + q_blocks), threads = (unsigned)warps * 32;
  const bool norm = p.q_weight || p.k_weight;
  const int kv = (int)kv_blocks;
#define DA_BLOCKS(I, N) return launch_dependent(append_blocks_kernel<I, N>, grid, threads, 0, stream, p, kv)
  if (integers) {
    if (norm) DA_BLOCKS(true, true);
    else DA_BLOCKS(true, false);
  } else {
    if (norm) DA_BLOCKS(false, true);
    else DA_BLOCKS(false, false);
  }
#undef DA_BLOCKS
}

}  // namespace da
