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
// The layout. The tokens of one block (a run, neighbours in slot_map but for tokens without a place) are the work of
// a group of n / 16 warps, for one head and K or V: a warp stages 16 of their rows in shared memory by asynchronous
// copies and turns them in place (two rows of 16 lanes at a time, as in cache_rows.cu); the greatest |x| of
// the group's warps meets in shared memory; then the rows go out as codes. So a row is read once. Only where
// the scale grew the group reads the block's other rows, 16 a warp, and writes them rounded again. Runs are
// found by the warps themselves: a group looks through a window of tokens for those whose predecessor is in
// another block. Padding and slots outside the cache have no block: both that predecessor and the run's next token are
// looked for past them, so no two groups have the same block (4096 tokens of padding behind a prefill of 4096: 2 us
// with blocks of 16, 8 with blocks of 256). Queries are the other blocks of the grid, as in cache_rows.cu.
//
// What bounds it. A decode step is latency: 64 tokens of 32 + 16 heads, blocks of 64: 4.7 us (queries alone
// 2.5); four warps a group there, most with nothing to do, made two waves of blocks: 7.3. A prefill of 4096 such
// tokens into blocks of 32 takes 27 us against a floor of 13.6: keys wait for their angles (5 of the 10 us that a
// group takes, now loaded a step ahead), rows of one head and one block are little work for the slots,
// positions and scales that have to be looked up first, and a scheduler has four warps at most. Measured and not
// kept: rows in registers (32 us then); eight rows a warp (the same); more blocks an SM with spills (32 -> 38);
// the rows' angles copied to shared memory along with them (27.6 -> 29.7, with three axes 48).
// Past 256 tokens a group takes the runs of its window one after another, which suits a prefill's long ones. A decode
// step's short ones wait for each other: one token each of 256, 257, 512 and 1024 rows, 8 heads: 10.9, 20.5, 36.1 and
// 67.6 us in blocks of 64, 31, 73, 134 and 262 in blocks of 256, 8.8, 8.8, 13.0 and 21.0 in blocks of 16.
#include <algorithm>
#include <cstring>

#include "cache_rows.cuh"

namespace da {
namespace {

constexpr int kRows = 16;      // rows of a run, and of a block, that a warp has (of few tokens up to kFewRows)
constexpr int kFewRows = 64;
constexpr int kLook = 30;      // tokens that a group looks at together for runs that start there (at most)
constexpr int kMinWarps = 4;   // of a CTA
constexpr int kMaxWarps = 16;
constexpr int kPerSm = 4;      // CTAs of kMinWarps an SM

// The greater of two; NaN wins for integers (an e4m3 code can be NaN by itself).
template <bool INT>
__device__ __forceinline__ float max_of(float a, float b) {
  return INT ? max_nan(a, b) : fmaxf(a, b);
}
template <bool INT>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t w) {  // of bf16 pairs; a is not negative
  w &= 0x7FFF7FFFu;
  const __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162 *>(&a), y = *reinterpret_cast<__nv_bfloat162 *>(&w);
  const __nv_bfloat162 r = INT ? __hmax2_nan(x, y) : __hmax2(x, y);
  return *reinterpret_cast<const uint32_t *>(&r);
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
// A row's eight elements over the scale, as codes. Integers of finite rows (nothing past 127) by adding
// 1.5 2^23, after which the low byte of a float is its nearest integer, ties to even.
template <bool INT>
__device__ __forceinline__ uint2 codes8(const uint4 &row, float inv, bool finite) {
  Eight x = times(values8(row), inv);
  float e[8];
  if (INT && finite) {
    const Pair m = pack(12582912.f, 12582912.f);
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) unpack(add2(x.v[i], m), e[2 * i], e[2 * i + 1]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[i] = prmt(prmt(__float_as_uint(e[4 * i]), __float_as_uint(e[4 * i + 1]), 0x0040),
                  prmt(__float_as_uint(e[4 * i + 2]), __float_as_uint(e[4 * i + 3]), 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack(x.v[i], e[2 * i], e[2 * i + 1]);
  return make_uint2(codes4<INT>(e[0], e[1], e[2], e[3]), codes4<INT>(e[4], e[5], e[6], e[7]));
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

// The slots of a call, and the block of one: -1 for padding, and outside the cache.
struct Slots {
  const int64_t *map;
  int64_t end;
  int tokens, shift;
  __device__ __forceinline__ int64_t block_of(int64_t slot) const { return slot < 0 || slot >= end ? -1 : slot >> shift; }
  __device__ __forceinline__ int64_t at(int64_t t) const { return t >= 0 && t < tokens ? map[t] : -1; }
};
// Past tokens without a block, by a warp: the first that has one of t, t + step, .. (step 1 or -1), -1: none has, and
// its block. 256 tokens a trip to memory. (A function that is called: inlined, its instructions stand in the way of
// those that every call needs, 0.2 to 0.6 us; of 512 tokens a trip, its registers spill the caller's.)
constexpr int kFar = 8;
__device__ __noinline__ int64_t next_block(const int64_t *map, int64_t end, int tokens, int shift, int64_t t, int step, int64_t &blk) {
  const Slots s = {map, end, tokens, shift};
  const int lane = threadIdx.x & 31;
  for (; t >= 0 && t < tokens; t += 32 * kFar * step) {
    int64_t slot[kFar];
#pragma unroll
    for (int k = 0; k < kFar; ++k) slot[k] = s.at(t + (32 * k + lane) * step);
#pragma unroll
    for (int k = 0; k < kFar; ++k) {
      blk = s.block_of(slot[k]);
      const uint32_t some = __ballot_sync(0xffffffffu, blk >= 0);
      if (some) {
        blk = __shfl_sync(0xffffffffu, blk, __ffs(some) - 1);
        return t + (32 * k + __ffs(some) - 1) * step;
      }
    }
  }
  blk = -1;
  return -1;
}

// Whether every position that turns a pair of token t is in the table.
__device__ __forceinline__ bool positions_ok(const BlockRowParams &p, int64_t t) {
  bool ok = true;
  for (int i = 0; i < p.num_axes; ++i) {
    const int pos = p.positions[(int64_t)p.axes[i] * p.position_stride + t];
    ok = ok && pos >= 0 && pos < p.max_position;
  }
  return ok;
}

// kv_blocks CTAs have the keys and values, the others the queries (a warp a part of a token).
// WARPS: of a CTA, at most.
template <bool INT, bool NORM, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == kMinWarps ? kPerSm : 1) append_blocks_kernel(const __grid_constant__ BlockRowParams p,
                                                                       const int kv_blocks) {
  extern __shared__ uint4 staged_all[];  // [warp][row][16]
  __shared__ uint32_t written_all[kMinWarps][256 / 32];  // rows of the block that the run writes, per group
  __shared__ int2 place_all[kMaxWarps * kRows];  // a row's token (past the run's first) and position in the block
  __shared__ float amax_all[kMaxWarps];
  __shared__ uint32_t leads_all[kMinWarps][2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  begin_dependent();
  // Keys first, which take longest, then values and queries in turn as long as there are both (the one waits
  // for memory, the other streams).
  const int half = kv_blocks / 2, q_blocks = (int)gridDim.x - kv_blocks, b = (int)blockIdx.x - half;
  const int both = 2 * min(half, q_blocks);
  const bool queries = b >= 0 && (b < both ? (b & 1) != 0 : half < q_blocks);
  const uint32_t block = b < 0 ? b + half : (b < both ? b >> 1 : b - both / 2) + (queries ? 0 : half);  // of its kind
  if (queries) {
    const uint32_t item = block * warps + warp;
    const uint32_t t = item / (uint32_t)p.parts;
    const int part = (int)(item - t * p.parts);
    if (t >= (uint32_t)p.num_tokens) return;
    const int nq = (p.num_q_heads + 3) / 4;
    const QueryLane<128> ql(p, lane);
    int64_t slot;
    float c[8], s[8];
    append_queries<128, NORM>(p, t, lane, ql, (int)((uint32_t)(part * nq) / (uint32_t)p.parts),
                              (int)((uint32_t)((part + 1) * nq) / (uint32_t)p.parts), p.num_q_heads, slot, c, s);
    return;
  }
  const int n = p.kv_groups, shift = 31 - __clz(n), R = p.warp_rows, gw = n / R;  // a block's rows, a warp's, a group's warps
  const int group = warp / gw, gwarp = warp - group * gw, HK = p.num_kv_heads;
  const int side = (int)block >= half ? 1 : 0;  // 0: K
  const uint32_t item = (block - side * half) * (uint32_t)(warps / gw) + group, at = item / (uint32_t)HK;
  const int64_t w0 = (int64_t)at * p.window;
  if (w0 >= p.num_tokens) return;
  const int h = (int)(item - at * HK);
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
  uint4 *mine_at = staged_all + (warp * R + sub) * 16 + kl;  // this lane's part of every second row
  int2 *place = place_all + warp * R;
  const Slots slots = {p.slot_map, p.num_slots, p.num_tokens, shift};

  uint32_t err = 0;
  const int64_t w1 = min(w0 + p.window, (int64_t)p.num_tokens);
  uint32_t leads = 0, alone = 0;  // of kLook tokens, those whose run starts there, and those whose run is one token
  int64_t from = w0 - kLook;
  const int ahead = (32 - min(p.window, kLook)) / 2;  // tokens before those, to see whose run they are in
  while (true) {
    while (leads == 0 && (from += kLook) < w1) {
      // lane i: the slot of token from - ahead + i
      const int64_t t = from - ahead + lane;
      const bool mine = lane >= ahead && lane < ahead + kLook && t < w1;
      const int64_t slot = slots.at(t), blk = slots.block_of(slot);
      if (mine && blk < 0 && slot != -1) err |= DA_DEVERR_SLOT;
      // the blocks of the tokens before and after this one that have one
      const uint32_t some = __ballot_sync(0xffffffffu, blk >= 0);
      const uint32_t down = some & ((1u << lane) - 1u), up = some & ~((2u << lane) - 1u);
      int64_t before = __shfl_sync(0xffffffffu, blk, 31 - __clz(down));  // (any lane's, if there is none)
      const int64_t after = __shfl_sync(0xffffffffu, blk, __ffs(up) - 1);
      if (!down) before = -1;
      if (from > ahead && gwarp == 0 && __any_sync(0xffffffffu, mine && blk >= 0 && !down)) {
        int64_t far;
        next_block(slots.map, slots.end, slots.tokens, shift, from - ahead - 1, -1, far);
        if (!down) before = far;
      }
      leads = __ballot_sync(0xffffffffu, mine && blk >= 0 && before != blk) >> ahead;
      alone = __ballot_sync(0xffffffffu, up ? after != blk : from - ahead + 32 >= p.num_tokens) >> ahead;
      if (gw > 1) {  // (the group's warps meet below: what its first one saw holds for all)
        if (gwarp == 0 && lane == 0) leads_all[group][0] = leads, leads_all[group][1] = alone;
        meet();
        leads = leads_all[group][0];
        alone = leads_all[group][1];
        meet();
      }
    }
    if (leads == 0) break;
    const int first = __ffs(leads) - 1;
    leads &= leads - 1;
    const int64_t t0 = from + first, blk = slots.block_of(slots.map[t0]);
    const bool single = (alone >> first) & 1u;  // (a decode step: the tokens after it are not looked at)
    const uint32_t per = (uint32_t)p.rows_per_page >> shift;  // blocks of a page
    const int64_t page = (blk >> 32) == 0 ? (int64_t)((uint32_t)blk / per) : blk / per, j = blk - page * per;
    const int64_t row0 = (page * HK + h) * p.rows_per_page + j * n;
    float *scale = scales + (page * HK + h) * per + j;
    const float was = *scale;
    // ---- which tokens, and which rows they write; the k-th of them is row k % R of the group's warp k / R
    bool fresh = false;
    int count = 0;
    if (gwarp == 0 && lane < 8) written[lane] = 0;
    __syncwarp();
    for (int64_t t = t0;;) {
      const int64_t i = t + lane;
      const int64_t slot = lane == 0 || !single ? slots.at(i) : -1, b = slots.block_of(slot);
      const uint32_t others = __ballot_sync(0xffffffffu, b >= 0 && b != blk);
      bool use = b == blk && (others == 0 || lane < __ffs(others) - 1);  // up to the first of another block
      if (use && !positions_ok(p, i)) {
        err |= DA_DEVERR_POSITION;
        use = false;
      }
      const int off = (int)(slot & (n - 1));
      fresh = fresh || __any_sync(0xffffffffu, use && off == 0);
      const uint32_t used = __ballot_sync(0xffffffffu, use);
      const uint32_t k = count + __popc(used & ((1u << lane) - 1u)) - gwarp * R;
      if (use && k < (uint32_t)R) place[k] = make_int2((int)(i - t0), off);
      if (use && gwarp == 0) atomicOr(&written[off >> 5], 1u << (off & 31));
      count += __popc(used);
      t += 32;
      if (others || single || count >= n || t >= p.num_tokens) break;
      if (__shfl_sync(0xffffffffu, b, 31) < 0) {
        int64_t found;
        t = next_block(slots.map, slots.end, slots.tokens, shift, t, 1, found);
        if (found != blk) break;
      }
    }
    __syncwarp();
    // ---- the warp's rows: read, normed, turned, in bf16
    const int have = min(max(count - gwarp * R, 0), R), pairs = (have + 1) / 2;
#pragma unroll 4
    for (int i = 0; i < pairs; ++i)
      if (2 * i + sub < have) cp_async_16(smem_u32(mine_at + 32 * i), src + (t0 + place[2 * i + sub].x) * stride + kl);
    cp_async_commit();
    uint32_t top2 = 0;
    const int pair0 = p.rope_adjacent ? 4 * kl : 8 * (second ? kl - r : kl);
    cp_async_wait_group<0>();  // (a lane reads what it copied itself)
    // (the next rows' angles are in flight while these are turned)
    auto angles = [&](int i, float (&c)[8], float (&s)[8]) {
      if (!turned || 2 * i + sub >= have) return;
      const int64_t t = t0 + place[2 * i + sub].x;
      if (p.rope_adjacent) load_turn<4>(p, t, pair0, c, s);
      else load_turn<8>(p, t, pair0, c, s);
    };
    auto turn_rows = [&](int i, float (&c)[8], float (&s)[8]) {
      if (i >= pairs) return;
      const bool on = 2 * i + sub < have;
      uint4 x = on ? mine_at[32 * i] : make_uint4(0u, 0u, 0u, 0u);
      if (r > 0 || norm) {
        if (norm) {
          norm_key(p, x, kl, partner, turned, second, c, s);
        } else {
          if (second)  // (b c + a s) is (x c - u s) with s of the other sign
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = -s[k];
          turn_key(p, x, partner, turned, c, s);
        }
        if (on) mine_at[32 * i] = x;
        else x = make_uint4(0u, 0u, 0u, 0u);
      }
      top2 = max_abs2<INT>(max_abs2<INT>(top2, x.x), x.y);
      top2 = max_abs2<INT>(max_abs2<INT>(top2, x.z), x.w);
    };
    if (side == 0) {
      float c[8], s[8], c2[8], s2[8];
      angles(0, c, s);
#pragma unroll 1
      for (int i = 0; i < pairs; i += 2) {
        angles(i + 1, c2, s2);
        turn_rows(i, c, s);
        angles(i + 2, c, s);
        turn_rows(i + 1, c2, s2);
      }
    } else {
#pragma unroll 2
      for (int i = 0; i < pairs; ++i) {
        const uint4 x = 2 * i + sub < have ? mine_at[32 * i] : make_uint4(0u, 0u, 0u, 0u);
        top2 = max_abs2<INT>(max_abs2<INT>(top2, x.x), x.y);
        top2 = max_abs2<INT>(max_abs2<INT>(top2, x.z), x.w);
      }
    }
    float top = max_of<INT>(bf_lo(top2), bf_hi(top2));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) top = max_of<INT>(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0) amax[gwarp] = top;
    meet();
    for (int i = 0; i < gw; ++i) top = max_of<INT>(top, amax[i]);
    // ---- the scale
    const float old = fresh ? 0.f : was, need = least_scale<INT>(top);
    const float now = old == old ? (need > old || need != need ? need : old) : old;
    const float inv = now != 0.f ? __frcp_rn(now) : 0.f;
    const bool finite = top < __int_as_float(0x7f800000);
    uint8_t *out = cache + row0 * 128 + kl * 8;
#pragma unroll 2
    for (int i = 0; i < pairs; ++i)
      if (2 * i + sub < have)
        *reinterpret_cast<uint2 *>(out + place[2 * i + sub].y * 128) = codes8<INT>(mine_at[32 * i], inv, finite);
    // ---- rows that stay, rounded again
    if (!fresh && now > old) {
      const float ratio = old * inv;
      uint4 *rows = reinterpret_cast<uint4 *>(cache + (row0 + gwarp * R) * 128) + lane;
#pragma unroll 4
      for (int i = 0; i < R / 4; ++i)  // four rows of 8 lanes
        if (!((written[(gwarp * R + 4 * i) >> 5] >> ((gwarp * R + 4 * i + (lane >> 3)) & 31)) & 1u)) {
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

template <bool INT, bool NORM>
static cudaError_t prepare_blocks() {
  const cudaFuncAttribute a = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const cudaError_t e = cudaFuncSetAttribute(append_blocks_kernel<INT, NORM, kMinWarps>, a, kMinWarps * kFewRows * 256);
  return e != cudaSuccess ? e : cudaFuncSetAttribute(append_blocks_kernel<INT, NORM, kMaxWarps>, a, kMaxWarps * kRows * 256);
}
cudaError_t append_blocks_prepare() {
  cudaError_t e = prepare_blocks<false, false>();
  if (e == cudaSuccess) e = prepare_blocks<false, true>();
  if (e == cudaSuccess) e = prepare_blocks<true, false>();
  return e != cudaSuccess ? e : prepare_blocks<true, true>();
}

cudaError_t launch_append_blocks(const CacheRowParams &rows, bool integers, int num_sms, cudaStream_t stream) {
  if (rows.num_tokens == 0) return cudaSuccess;
  BlockRowParams p;
  std::memset(&p, 0, sizeof p);
  static_cast<CacheRowParams &>(p) = rows;
  for (int i = 0; i < p.rope_pairs; ++i) {
    const int a = p.pair_axis[i];
    if (std::memchr(p.axes, a, (size_t)p.num_axes) == nullptr) p.axes[p.num_axes++] = (uint8_t)a;
  }
  // Few tokens (a decode step: every token, or every few, a run of its own) take a warp for up to 64 rows of
  // a block, most of which have nothing to write: 64 tokens of 8 heads, blocks of 64: 7.3 -> 4.7 us.
  const bool few = p.num_tokens <= 256;
  p.warp_rows = std::min<int>(p.kv_groups, few ? kFewRows : kRows);
  const int gw = p.kv_groups / p.warp_rows, warps = std::max(kMinWarps, gw);
  // Windows of one token while that makes few warps, else wider ones, up to a block (less a sixteenth): few groups
  // then find no run. Up to 32 warps an SM, twice what it holds: narrower windows seldom have the ends of two
  // runs, which one group would take in turn (16: 300 tokens into blocks of 256 25.7 us, now 17.2, 2000 into
  // blocks of 128 23.3 and 17.6; 300 and 2000 into blocks of 32 10.2 and 17.6, now 10.5 and 18.5; 64: 4096 into
  // blocks of 32 27.6 -> 28.5).
  const int64_t one = (int64_t)p.num_tokens * p.num_kv_heads * 2 * gw;
  int window = 1;
  while (!few && window < p.kv_groups * 15 / 16 && one / window > (int64_t)num_sms * 32)
    window = window < 16 ? 2 * window : window < kLook ? kLook : 2 * window;
  p.window = window;
  const int64_t items = ((int64_t)p.num_tokens + window - 1) / window * p.num_kv_heads;  // of K, and of V
  const int64_t kv_blocks = 2 * ((items + warps / gw - 1) / (warps / gw));
  int64_t q_blocks = 0;
  p.parts = 1;
  if (p.q) {
    const int64_t groups = (p.num_q_heads + 3) / 4;
    p.parts = (int32_t)std::max<int64_t>(1, std::min<int64_t>(groups, (int64_t)num_sms * 32 / p.num_tokens));
    q_blocks = ((int64_t)p.num_tokens * p.parts + warps - 1) / warps;
  }
  if (kv_blocks + q_blocks > INT32_MAX / kMaxWarps) return cudaErrorInvalidConfiguration;  // (items in 32 bits)
  const unsigned grid = (unsigned)(kv_blocks + q_blocks), threads = (unsigned)warps * 32;
  const bool norm = p.q_weight || p.k_weight;
  const int kv = (int)kv_blocks;
  const size_t smem = (size_t)warps * p.warp_rows * 256;
#define DA_BLOCKS(I, N)                                                                                               \
  return warps == kMinWarps ? launch_dependent(append_blocks_kernel<I, N, kMinWarps>, grid, threads, smem, stream, p, kv) \
                            : launch_dependent(append_blocks_kernel<I, N, kMaxWarps>, grid, threads, smem, stream, p, kv)
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
