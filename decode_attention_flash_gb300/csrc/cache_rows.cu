// cache_rows.cu -- rows of the K/V cache written and read back: decode_attn_append (rotary
// positions, then the element kind's quantisation, at a slot) and decode_attn_gather.
//
// The mathematics. Pair i of a rotated head (elements i and i + n of its first
// 2n, or 2i and 2i + 1) is turned by the angle of its token's position on the
// pair's axis, whose cosine and sine are a row of a table that the caller
// keeps: (a, b) -> (a c - b s, b c + a s), products and sums each rounded to
// fp32, the result to bf16. Keys and values then take the cache's element kind
// (the rules stand at put_row); a quantised cache holds the quantised bf16 key.
//
// What bounds it. Every byte is read and written once, so HBM does for a prefill
// and latency for a decode step; the arithmetic has to stay out of the way (a first
// form with every head as 16 lanes of 8 elements, partners exchanged by shuffles, was
// bound by instruction issue). A warp owns a token, or a part of its heads when there
// are fewer tokens than the SMs take warps. Queries: a lane takes both halves of
// eight pairs (two 16-byte loads), so a head is 8 lanes (4 for the 64-element rope
// heads of the latent cache), nothing is exchanged, and the cosines and sines of its
// pairs stay in registers for all heads of the token. Keys and values: 16 lanes of 8
// elements a head, as the element kinds want them (block maxima are shuffles of 2, 4
// or 16 lanes), a key's halves exchanged by shuffles, K and V side by side, pointers that
// advance by a head's stride; kAhead or 2 kSide loads are in flight. (A token staged in
// shared memory by bulk copies instead kept fewer warps on an SM: 33.9 -> 43.5 us for the
// e4m3 rows below; its first keys and values loaded before its queries are stored: 30.4
// -> 32.8.)
// Blocks of four warps leave an SM sooner than blocks of eight, so a last wave ends sooner
// (eight: 62.7, 30.4 and 56.3 us for the three below, two: 62.7, 31.3 and 55.3).
// At eight blocks an SM the append has 64 registers a thread; every form of it spills a little
// (4 to 28 bytes). 96 registers and fewer warps took longer: 30.4 -> 33.8 for the e4m3 rows.
// Measured: 16381 tokens of 32 + 16 heads, three axes, bf16 cache: 62.3 us, 97 % of the
// copy rate; 4099 tokens of 64 + 16 heads into e4m3 with token scales: 29.7 us (79 %, two
// thirds of a wave short of two); 65537 4-bit rows of 8 heads read back: 54.8 us (93 %); 2048
// latent rows with 128 heads: 13.7 us (78 %; the rope key loaded after the latent row is
// stored: 14.0).
// K first and then V, with a head's address worked out for each row: 65.2, 31.4 and
// 61.3 us, bound by instruction issue; one row in flight of K and of V instead of two:
// 65.2, 31.0 and 70.7.
// The read-back gives half a warp to a token (two tokens of one head a warp: 65537 of
// them 21.7 -> 12.4 us, of two heads 23.4 -> 16.5, of eight 54.7 either way).
#include <algorithm>

#include <cuda_fp16.h>

#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace da {
namespace {

constexpr int kWarps = 4;
constexpr int kAhead = 4;  // loads of queries in flight a lane
constexpr int kSide = 2;   // rows of K, and as many of V, in flight

enum Kind { kBf16 = 0, kE4m3 = 1, kE4m3Token = 2, kInt4 = 3, kFp4 = 4, kLatent = 5 };

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// e2m1 codes of (lo, hi), to nearest even, in the low and high nibble of a byte.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
      "cvt.u32.u8 %0, t;\n\t}"
      : "=r"(r)
      : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t f16_bits(float x) { return (uint32_t)__half_as_ushort(__float2half_rn(x)); }
__device__ __forceinline__ float f16_value(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)b));
}

// Where the rows of one slot are: lane l of 16 of kv head 0 in K and in V, the next
// head `head` bytes on; the scale words (or, 4-bit float, the block scales) likewise.
struct RowAt {
  uint8_t *k, *v, *ks, *vs;
  int64_t head, shead;
};
template <int KIND>
__device__ __forceinline__ RowAt row_at(const CacheRowParams &p, int64_t slot, int l) {
  const uint32_t P = (uint32_t)p.rows_per_page;
  const int64_t page = (slot >> 32) == 0 ? (int64_t)((uint32_t)slot / P) : slot / P;
  const int off = (int)(slot - page * P);
  RowAt a;
  a.ks = a.vs = nullptr;
  a.shead = 0;
  int64_t at;
  if (KIND == kFp4) {
    const int64_t gran = P / 16;
    const int64_t g0 = (page * p.num_kv_heads * gran + off / 16) * 1152;
    at = g0 + off % 16 * 64 + l * 4;
    a.head = a.shead = gran * 1152;
    const int64_t sc = g0 + 1024 + off % 16 * 8 + (l >> 1);
    a.ks = reinterpret_cast<uint8_t *>(p.k) + sc;
    a.vs = reinterpret_cast<uint8_t *>(p.v) + sc;
  } else {
    const int64_t row0 = page * p.num_kv_heads * P + off;
    const int row_bytes = KIND == kBf16 ? 256 : KIND == kInt4 ? 4 * (p.kv_groups + 16) : 128;
    at = row0 * row_bytes + (KIND == kBf16 ? l * 16 : KIND == kInt4 ? (p.kv_groups + l) * 4 : l * 8);
    a.head = (int64_t)P * row_bytes;
    if (KIND == kInt4) {  // the coefficient word of the lane's group
      const int64_t sc = row0 * row_bytes + l * p.kv_groups / 16 * 4;
      a.ks = reinterpret_cast<uint8_t *>(p.k) + sc;
      a.vs = reinterpret_cast<uint8_t *>(p.v) + sc;
      a.shead = a.head;
    }
    if (KIND == kE4m3Token) {
      a.ks = reinterpret_cast<uint8_t *>(p.k_scale_shift + row0);
      a.vs = reinterpret_cast<uint8_t *>(p.v_scale_shift + row0);
      a.shead = (int64_t)P * 4;
    }
  }
  a.k = reinterpret_cast<uint8_t *>(p.k) + at;
  a.v = reinterpret_cast<uint8_t *>(p.v) + at;
  return a;
}

// One row of 128 elements, 8 per lane (lane l of 16: elements 8l .. 8l + 7, as bf16
// pairs in `raw`), to `dst` (and its scale to `sdst`) in the cache's element kind:
// (quotients as products with one fp32 reciprocal: eight divisions a lane took
// longer than the copies)
//   e4m3        code = e4m3(x / scale[h]), to nearest even, saturating
//   e4m3, token shift = f16((max + min) / 2), scale = f16((max - min) / 2 / 448) (1
//               when that is 0), code = e4m3((x - shift) / scale)
//   int4        per group: shift = f16(min), scale = f16((max - min) / 15) (1 when
//               that is 0), code = round((x - shift) / scale) within 0..15
//   4-bit float per block of 16: block scale = e4m3(max |x| / (6 scale[h])), code =
//               e2m1(x * (1 / (block scale * scale[h]))), zeros when that product is 0
// Every lane of the warp calls it (shuffles); lanes with !on store nothing.
template <int KIND>
__device__ __forceinline__ void put_row(const CacheRowParams &p, bool on, uint8_t *dst, uint8_t *sdst, float head_scale,
                                        int l, const uint4 &raw) {
  if (KIND == kBf16) {
    if (on) *reinterpret_cast<uint4 *>(dst) = raw;
    return;
  }
  const float x[8] = {bf_lo(raw.x), bf_hi(raw.x), bf_lo(raw.y), bf_hi(raw.y),
                      bf_lo(raw.z), bf_hi(raw.z), bf_lo(raw.w), bf_hi(raw.w)};
  if (KIND == kE4m3) {
    const float inv = __frcp_rn(head_scale);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_e4m3x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv));
    if (on) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    return;
  }
  if (KIND == kFp4) {
    float a = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(x[i]));
    a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const float g = head_scale;
    const uint32_t sb = f32x2_to_e4m3x2(__fdiv_rn(a, __fmul_rn(6.f, g)), 0.f) & 0xFFu;
    const uint32_t half2 = e4m3x2_to_f16x2((uint16_t)sb);
    const float eff = __fmul_rn(f16_value(half2 & 0xFFFFu), g);
    const float inv = eff >= 0x1p-126f ? __frcp_rn(eff) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= e2m1x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)) << (8 * i);
    if (on) {
      *reinterpret_cast<uint32_t *>(dst) = w;
      if ((l & 1) == 0) *sdst = (uint8_t)sb;
    }
    return;
  }
  // a minimum and a maximum over the row, or over the lanes of a group
  float hi = x[0], lo = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    hi = max_nan(hi, x[i]);
    lo = min_nan(lo, x[i]);
  }
  const int lanes = KIND == kInt4 ? 16 / p.kv_groups : 16;
  for (int o = 1; o < lanes; o <<= 1) {
    hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  const float span = __fsub_rn(hi, lo);
  const uint32_t shift = f16_bits(KIND == kInt4 ? lo : __fmul_rn(__fadd_rn(hi, lo), 0.5f));
  uint32_t scale = f16_bits(KIND == kInt4 ? __fdiv_rn(span, 15.f) : __fdiv_rn(__fmul_rn(span, 0.5f), 448.f));
  if (scale == 0) scale = 0x3C00u;
  const float inv = __frcp_rn(f16_value(scale)), sh = f16_value(shift);
  const int32_t word = (int32_t)(scale | (shift << 16));
  if (KIND == kE4m3Token) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32x2_to_e4m3x2(__fmul_rn(__fsub_rn(x[2 * i], sh), inv), __fmul_rn(__fsub_rn(x[2 * i + 1], sh), inv));
    if (on) {
      *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      if (l == 0) *reinterpret_cast<int32_t *>(sdst) = word;
    }
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf(__fmul_rn(__fsub_rn(x[i], sh), inv));
      w |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
    }
    if (on) {
      *reinterpret_cast<uint32_t *>(dst) = w;
      if (l % lanes == 0) *reinterpret_cast<int32_t *>(sdst) = word;
    }
  }
}

// Slot of token t, checked: -1 for padding (and, with the error bit, for a slot outside the cache).
__device__ __forceinline__ int64_t load_slot(const CacheRowParams &p, int64_t t, uint32_t &err) {
  if (!p.slot_map) return -1;
  const int64_t s = p.slot_map[t];
  if (s >= p.num_slots || s < -1) {
    err |= DA_DEVERR_SLOT;
    return -2;
  }
  return s;
}

// The cosines and sines of pairs pair0 .. pair0 + 7 (or + 3: kPairs) of token t;
// false when a position is outside the table.
template <int kPairs>
__device__ __forceinline__ bool load_turn(const CacheRowParams &p, int64_t t, int pair0, float (&c)[8], float (&s)[8]) {
  const int n = p.rope_pairs;
  if (p.rope_whole) {  // they share an axis: vector loads
    const int pos = p.positions[(int64_t)p.pair_axis[pair0] * p.position_stride + t];
    if (pos < 0 || pos >= p.max_position) return false;
    const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + pair0);
    const float4 *row2 = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + n + pair0);
#pragma unroll
    for (int j = 0; j < kPairs / 4; ++j) {
      const float4 a = __ldg(row + j), b = __ldg(row2 + j);
      c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
      s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
    }
    return true;
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    const int pos = p.positions[(int64_t)p.pair_axis[pair0 + i] * p.position_stride + t];
    const bool in = pos >= 0 && pos < p.max_position;
    ok = ok && in;
    c[i] = in ? __ldg(p.cos_sin + (int64_t)pos * 2 * n + pair0 + i) : 1.f;
    s[i] = in ? __ldg(p.cos_sin + (int64_t)pos * 2 * n + n + pair0 + i) : 0.f;
  }
  return ok;
}

// (a c - b s, b c + a s), every product and sum rounded to fp32
__device__ __forceinline__ void turn(float a, float b, float c, float s, float &x, float &y) {
  x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  y = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
}
// Pairs (element i of `lo`, element i of `hi`), i < 8.
__device__ __forceinline__ void turn_halves(uint4 &lo, uint4 &hi, const float (&c)[8], const float (&s)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x0, y0, x1, y1;
    turn(bf_lo(a[i]), bf_lo(b[i]), c[2 * i], s[2 * i], x0, y0);
    turn(bf_hi(a[i]), bf_hi(b[i]), c[2 * i + 1], s[2 * i + 1], x1, y1);
    a[i] = pack_bf16(x0, x1);
    b[i] = pack_bf16(y0, y1);
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}
// Pairs of neighbours: elements 2i, 2i + 1 of `v`, i < 4, with cosines c[at + i].
__device__ __forceinline__ void turn_adjacent(uint4 &v, const float (&c)[8], const float (&s)[8], int at) {
  uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x, y;
    turn(bf_lo(a[i]), bf_hi(a[i]), c[at + i], s[at + i], x, y);
    a[i] = pack_bf16(x, y);
  }
  v = make_uint4(a[0], a[1], a[2], a[3]);
}

// HEAD: elements of a rotated head, 128 (the latent cache: 64).
template <int KIND, int HEAD>
__global__ void __launch_bounds__(kWarps * 32, 8) append_kernel(const __grid_constant__ CacheRowParams p) {
  constexpr int kChunks = HEAD / 8;        // 16-byte chunks of a head
  constexpr int kLanes = kChunks / 2;      // lanes of a head with both halves of its pairs
  constexpr int kHeads = 32 / kLanes;      // query heads a warp takes at once
  constexpr int kDeep = kAhead / 2;        // groups of them in flight
  const int lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  let_next_kernel_start();
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = p.parts == 1 ? item : (int64_t)((uint32_t)item / (uint32_t)p.parts);
  const int part = (int)(item - t * p.parts);
  if (t >= p.num_tokens) return;
  const int HQ = p.q ? p.num_q_heads : 0, HK = p.k_new ? p.num_kv_heads : 0;
  // groups: queries kHeads at a time, then (not the latent cache) keys and values of two heads
  const int nq = (HQ + kHeads - 1) / kHeads, nk = KIND == kLatent ? 0 : (HK + 1) / 2;
  const int groups = nq + nk;
  const int g0 = (int)((uint32_t)(part * groups) / (uint32_t)p.parts);
  const int g1 = (int)((uint32_t)((part + 1) * groups) / (uint32_t)p.parts);

  // ---- queries: this lane's chunks of a head. Half-split pairs of r chunks: lane i < r
  // has chunks i and i + r; neighbours as pairs: chunks 2i and 2i + 1; elements past
  // the rotated ones stay, two chunks a lane.
  const int l = lane % kLanes, sub = lane / kLanes, r = p.rope_pairs / 8;
  const bool turned = l < r;
  const bool split = turned && !p.rope_adjacent;
  const int ca = split ? l : 2 * l, cb = split ? l + r : 2 * l + 1;
  const int gq1 = min(g1, nq);
  const uint4 *qsrc = reinterpret_cast<const uint4 *>(p.q + t * p.q_stride);
  uint4 a[kDeep], b[kDeep];
  auto load_q = [&](int g) {
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int hd = (g + k) * kHeads + sub;
      if (g + k < gq1 && hd < HQ) {
        a[k] = qsrc[hd * kChunks + ca];
        b[k] = qsrc[hd * kChunks + cb];
      }
    }
  };
  load_q(g0);  // in flight while the slot and the positions are looked up
  uint32_t err = 0;
  const int64_t slot = load_slot(p, t, err);
  const bool padding = p.slot_map != nullptr && slot < 0;
  float c[8], s[8];
  bool bad = false;
  if (turned) bad = !load_turn<8>(p, t, 8 * l, c, s);
  bad = __any_sync(0xffffffffu, bad);
  if (bad && !padding) err |= DA_DEVERR_POSITION;
  if (err && lane == 0) atomicOr(p.err, err);
  if (bad || padding) return;
  {
    const bool many = p.q_len > 1;
    const int64_t row0 = many ? (t / p.q_len * p.num_q_heads) * p.q_len + t % p.q_len : t * p.num_q_heads;
    const int step = (many ? p.q_len : 1) * kChunks;
    uint4 *dst = reinterpret_cast<uint4 *>(p.q_out) + row0 * kChunks;
    for (int g = g0; g < gq1; g += kDeep) {
      if (g > g0) load_q(g);
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int hd = (g + k) * kHeads + sub;
        if (g + k >= gq1 || hd >= HQ) continue;
        if (split) {
          turn_halves(a[k], b[k], c, s);
        } else if (turned) {
          turn_adjacent(a[k], c, s, 0);
          turn_adjacent(b[k], c, s, 4);
        }
        dst[(int64_t)hd * step + ca] = a[k];
        dst[(int64_t)hd * step + cb] = b[k];
      }
    }
  }
  if (HK == 0) return;
  if constexpr (KIND == kLatent) {
    // the row of the latent cache: 512 elements as they are, 64 turned, by the last part
    if (part != p.parts - 1) return;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.k_new + t * p.k_stride) + lane;
    uint4 *dst = reinterpret_cast<uint4 *>(p.k) + slot * 64 + lane;
    const uint4 x = src[0], y = src[32];
    const uint4 *rope = reinterpret_cast<const uint4 *>(p.v_new + t * p.v_stride);
    uint4 u, v;
    if (lane < kLanes) u = rope[ca], v = rope[cb];
    dst[0] = x;
    dst[32] = y;
    if (lane < kLanes) {
      if (split) {
        turn_halves(u, v, c, s);
      } else if (turned) {
        turn_adjacent(u, c, s, 0);
        turn_adjacent(v, c, s, 4);
      }
      uint4 *out = reinterpret_cast<uint4 *>(p.v) + slot * 8;
      out[ca] = u;
      out[cb] = v;
    }
    return;
  } else {
    if (g1 <= nq) return;
    // ---- keys and values: 16 lanes a head, two heads at once
    const int kl = lane & 15, ksub = lane >> 4;
    const bool kturned = kl < 2 * r, second = kturned && !p.rope_adjacent && kl >= r;
    const int partner = lane - kl + (kturned && !p.rope_adjacent ? (second ? kl - r : kl + r) : kl);
    const RowAt at = row_at<KIND>(p, slot, kl);
    const int first = max(g0, nq);
    if (r > 0) {
      if (kturned) {
        if (p.rope_adjacent) load_turn<4>(p, t, 4 * kl, c, s);
        else load_turn<8>(p, t, 8 * (second ? kl - r : kl), c, s);
      }
      if (second)  // (b c + a s) is (x c - u s) with s of the other sign
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = -s[i];
    }
    int h = 2 * (first - nq) + ksub;
    const uint4 *ksrc = reinterpret_cast<const uint4 *>(p.k_new + t * p.k_stride) + h * 16 + kl;
    const uint4 *vsrc = reinterpret_cast<const uint4 *>(p.v_new + t * p.v_stride) + h * 16 + kl;
    uint8_t *kd = at.k + h * at.head, *vd = at.v + h * at.head;
    uint8_t *ks = at.ks + h * at.shead, *vs = at.vs + h * at.shead;
    for (int g = first; g < g1; g += kSide) {
      uint4 w[kSide], u[kSide];
      float sk[kSide], sv[kSide];
#pragma unroll
      for (int i = 0; i < kSide; ++i) {
        w[i] = u[i] = make_uint4(0u, 0u, 0u, 0u);
        sk[i] = sv[i] = 1.f;
        if (g + i < g1 && h + 2 * i < HK) {
          w[i] = ksrc[32 * i];
          u[i] = vsrc[32 * i];
          if (KIND == kE4m3 || KIND == kFp4) {
            sk[i] = __ldg(p.k_scale + h + 2 * i);
            sv[i] = __ldg(p.v_scale + h + 2 * i);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < kSide; ++i) {
        if (g + i >= g1) break;
        if (r > 0) {
          if (p.rope_adjacent) {
            if (kturned) turn_adjacent(w[i], c, s, 0);
          } else {
            const uint4 z = make_uint4(__shfl_sync(0xffffffffu, w[i].x, partner), __shfl_sync(0xffffffffu, w[i].y, partner),
                                       __shfl_sync(0xffffffffu, w[i].z, partner), __shfl_sync(0xffffffffu, w[i].w, partner));
            if (kturned) {
              uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
              const uint32_t y[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[j] = pack_bf16(__fsub_rn(__fmul_rn(bf_lo(x[j]), c[2 * j]), __fmul_rn(bf_lo(y[j]), s[2 * j])),
                                 __fsub_rn(__fmul_rn(bf_hi(x[j]), c[2 * j + 1]), __fmul_rn(bf_hi(y[j]), s[2 * j + 1])));
              w[i] = make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
        }
        const bool mine = h + 2 * i < HK;
        put_row<KIND>(p, mine, kd, ks, sk[i], kl, w[i]);
        put_row<KIND>(p, mine, vd, vs, sv[i], kl, u[i]);
        kd += 2 * at.head;
        vd += 2 * at.head;
        ks += 2 * at.shead;
        vs += 2 * at.shead;
      }
      h += 2 * kSide;
      ksrc += 32 * kSide;
      vsrc += 32 * kSide;
    }
  }
}

// Eight elements (lane l of 16) of a row as bf16 pairs: each value is the fp32
// product (and sum) of its parts, rounded once more to bf16.
struct RowBits {
  uint4 a;      // the lane's codes (bf16: its values)
  uint32_t s;   // block scale byte, or scale and shift halves
};
template <int KIND>
__device__ __forceinline__ RowBits get_row(const uint8_t *src, const uint8_t *ssrc) {
  RowBits r;
  r.a = make_uint4(0u, 0u, 0u, 0u);
  r.s = 0;
  if (KIND == kBf16) r.a = *reinterpret_cast<const uint4 *>(src);
  if (KIND == kE4m3 || KIND == kE4m3Token) {
    const uint2 v = *reinterpret_cast<const uint2 *>(src);
    r.a.x = v.x;
    r.a.y = v.y;
  }
  if (KIND == kInt4 || KIND == kFp4) r.a.x = *reinterpret_cast<const uint32_t *>(src);
  if (KIND == kInt4 || KIND == kE4m3Token) r.s = *reinterpret_cast<const uint32_t *>(ssrc);
  if (KIND == kFp4) r.s = *ssrc;
  return r;
}
template <int KIND>
__device__ __forceinline__ uint4 row_values(const RowBits &r, float head_scale) {
  if (KIND == kBf16) return r.a;
  float x[8];
  if (KIND == kE4m3 || KIND == kE4m3Token) {
    const uint32_t h[4] = {e4m3x2_to_f16x2((uint16_t)r.a.x), e4m3x2_to_f16x2((uint16_t)(r.a.x >> 16)),
                           e4m3x2_to_f16x2((uint16_t)r.a.y), e4m3x2_to_f16x2((uint16_t)(r.a.y >> 16))};
    const float sc = KIND == kE4m3 ? head_scale : f16_value(r.s & 0xFFFFu);
    const float sh = KIND == kE4m3 ? 0.f : f16_value(r.s >> 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = f16_value((h[i >> 1] >> (16 * (i & 1))) & 0xFFFFu);
      x[i] = KIND == kE4m3 ? __fmul_rn(c, sc) : fmaf(c, sc, sh);
    }
  } else if (KIND == kInt4) {
    const float sc = f16_value(r.s & 0xFFFFu), sh = f16_value(r.s >> 16);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = fmaf((float)((r.a.x >> (4 * i)) & 15u), sc, sh);
  } else {
    const uint32_t s2 = e4m3x2_to_f16x2((uint16_t)(r.s | (r.s << 8)));
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(r.a.x));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&h[i]), *reinterpret_cast<const __half2 *>(&s2));
      const float2 f = __half22float2(v);  // exact
      x[2 * i] = __fmul_rn(f.x, head_scale);
      x[2 * i + 1] = __fmul_rn(f.y, head_scale);
    }
  }
  return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

template <int KIND>
__global__ void __launch_bounds__(kWarps * 32) gather_kernel(const __grid_constant__ CacheRowParams p) {
  const int lane = threadIdx.x & 31;
  wait_for_previous_kernel();
  let_next_kernel_start();
  constexpr int kTeam = KIND == kLatent ? 32 : 16;  // lanes of a token
  const int64_t item = (int64_t)blockIdx.x * (kWarps * 32 / kTeam) + threadIdx.x / kTeam;
  const int64_t t = p.parts == 1 ? item : (int64_t)((uint32_t)item / (uint32_t)p.parts);
  const int part = (int)(item - t * p.parts);
  if (t >= p.num_tokens) return;
  uint32_t err = 0;
  const int64_t slot = load_slot(p, t, err);
  if (err && lane % kTeam == 0) atomicOr(p.err, err);
  if (slot < 0) return;
  if (KIND == kLatent) {  // 512 + 64 elements: 72 chunks of 16 bytes
    const uint4 *ck = reinterpret_cast<const uint4 *>(p.k) + slot * 64;
    uint4 *ok = reinterpret_cast<uint4 *>(p.k_out) + t * 64;
    const uint4 a = ck[lane], b = ck[32 + lane];
    if (lane < 8) {
      const uint4 c = reinterpret_cast<const uint4 *>(p.v)[slot * 8 + lane];
      *(reinterpret_cast<uint4 *>(p.v_out) + t * 8 + lane) = c;
    }
    ok[lane] = a;
    ok[32 + lane] = b;
    return;
  }
  const int l = lane & 15;
  const RowAt at = row_at<KIND>(p, slot, l);
  // head by head, of K and of V side by side, pointers a stride on; kSide rows of each in
  // flight
  const int HK = p.num_kv_heads;
  const int h0 = (int)((uint32_t)(part * HK) / (uint32_t)p.parts);
  const int h1 = (int)((uint32_t)((part + 1) * HK) / (uint32_t)p.parts);
  const uint8_t *k = at.k + h0 * at.head, *v = at.v + h0 * at.head;
  const uint8_t *ks = at.ks + h0 * at.shead, *vs = at.vs + h0 * at.shead;
  uint4 *ko = reinterpret_cast<uint4 *>(p.k_out) + (t * HK + h0) * 16 + l;
  uint4 *vo = reinterpret_cast<uint4 *>(p.v_out) + (t * HK + h0) * 16 + l;
  for (int h = h0; h < h1; h += kSide) {
    RowBits rk[kSide], rv[kSide];
    float sk[kSide], sv[kSide];
#pragma unroll
    for (int i = 0; i < kSide; ++i)
      if (h + i < h1) {
        rk[i] = get_row<KIND>(k, ks);
        rv[i] = get_row<KIND>(v, vs);
        if (KIND == kE4m3 || KIND == kFp4) {
          sk[i] = __ldg(p.k_scale + h + i);
          sv[i] = __ldg(p.v_scale + h + i);
        }
        k += at.head;
        v += at.head;
        ks += at.shead;
        vs += at.shead;
      }
#pragma unroll
    for (int i = 0; i < kSide; ++i)
      if (h + i < h1) {
        ko[16 * i] = row_values<KIND>(rk[i], sk[i]);
        vo[16 * i] = row_values<KIND>(rv[i], sv[i]);
      }
    ko += 16 * kSide;
    vo += 16 * kSide;
  }
}

int64_t blocks_for(int64_t items) { return (items + kWarps - 1) / kWarps; }

// Parts a token's heads are cut into by the read-back: about 48 warps for every SM.
int parts_for(int64_t tokens, int groups, int num_sms) {
  const int64_t want = (int64_t)num_sms * 48;
  const int64_t parts = (want + tokens - 1) / tokens;
  return (int)std::max<int64_t>(1, std::min<int64_t>({parts, groups, INT32_MAX / groups}));
}

// The append, whose parts look slot and angles up again: as many as one wave holds (32
// warps an SM), and two where that is none or one, the heads are many and the waves few.
// 1100 tokens, 32 query heads, latent rows of 128: 6.8 -> 6.0, 11.5 -> 9.3 us against 48 warps
// an SM; 4099 tokens of 8 + 16 heads in one part 12.3, in two 14.8; of 64 + 16 31.8, 29.2.
int append_parts(int64_t tokens, int groups, int num_sms) {
  const int64_t wave = (int64_t)num_sms * 32;
  int64_t parts = wave / tokens;
  if (parts < 2) parts = groups >= 12 && tokens < 2 * wave ? 2 : 1;
  return (int)std::min<int64_t>({parts, groups, INT32_MAX / groups});
}

}  // namespace

cudaError_t launch_append(CacheRowParams p, int kind, int num_sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  if (!p.q && !p.k_new) return cudaSuccess;
  const int per = kind == kLatent ? 8 : 4;
  const int groups = (p.q ? (p.num_q_heads + per - 1) / per : 0) +
                     (p.k_new && kind != kLatent ? (p.num_kv_heads + 1) / 2 : 0);
  p.parts = append_parts(p.num_tokens, groups < 1 ? 1 : groups, num_sms);
  const int64_t blocks = blocks_for((int64_t)p.num_tokens * p.parts);
  const unsigned grid = (unsigned)blocks;
  switch (kind) {
    case kBf16: return launch_dependent(append_kernel<kBf16, 128>, grid, kWarps * 32, 0, stream, p);
    case kE4m3: return launch_dependent(append_kernel<kE4m3, 128>, grid, kWarps * 32, 0, stream, p);
    case kE4m3Token: return launch_dependent(append_kernel<kE4m3Token, 128>, grid, kWarps * 32, 0, stream, p);
    case kInt4: return launch_dependent(append_kernel<kInt4, 128>, grid, kWarps * 32, 0, stream, p);
    case kFp4: return launch_dependent(append_kernel<kFp4, 128>, grid, kWarps * 32, 0, stream, p);
    default: return launch_dependent(append_kernel<kLatent, 64>, grid, kWarps * 32, 0, stream, p);
  }
}

cudaError_t launch_gather(CacheRowParams p, int kind, int num_sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  p.parts = kind == kLatent ? 1 : parts_for(((int64_t)p.num_tokens + 1) / 2, p.num_kv_heads, num_sms);
  const int64_t items = (int64_t)p.num_tokens * p.parts;  // half a warp each, but the latent rows
  const unsigned grid = (unsigned)blocks_for(kind == kLatent ? items : (items + 1) / 2);
  switch (kind) {
    case kBf16: return launch_dependent(gather_kernel<kBf16>, grid, kWarps * 32, 0, stream, p);
    case kE4m3: return launch_dependent(gather_kernel<kE4m3>, grid, kWarps * 32, 0, stream, p);
    case kE4m3Token: return launch_dependent(gather_kernel<kE4m3Token>, grid, kWarps * 32, 0, stream, p);
    case kInt4: return launch_dependent(gather_kernel<kInt4>, grid, kWarps * 32, 0, stream, p);
    case kFp4: return launch_dependent(gather_kernel<kFp4>, grid, kWarps * 32, 0, stream, p);
    default: return launch_dependent(gather_kernel<kLatent>, grid, kWarps * 32, 0, stream, p);
  }
}

}  // namespace da
