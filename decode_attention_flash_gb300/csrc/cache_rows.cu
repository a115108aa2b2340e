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
// What bounds it. Every byte is read and written once, so HBM does for a
// prefill and latency for a decode step. A warp owns a token (or, when there are
// fewer tokens than the SMs take warps, a part of its heads): it loads the
// token's cosines and sines once into registers and walks the heads, 16 lanes of
// 8 elements a head (8 lanes for the 64-element rope heads of the latent cache),
// kAhead loads in flight. A half-split pair sits in two lanes of the head and is
// exchanged by shuffles; block maxima are shuffles of 2, 4 or 16 lanes.
#include <cuda_fp16.h>

#include "internal.h"
#include "ptx.cuh"

namespace da {
namespace {

constexpr int kWarps = 8;
constexpr int kAhead = 4;

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

// The cache row (in rows of one head) of slot `s`, kv head h: slots count the
// positions of all pages (or of all batch rows of a contiguous cache).
__device__ __forceinline__ int64_t cache_row(const CacheRowParams &p, int64_t page, int off, int h) {
  return (page * p.num_kv_heads + h) * p.rows_per_page + off;
}

// One row of 128 elements, 8 per lane (lane l of 16: elements 8l .. 8l + 7, bf16
// values in fp32), into row `row` of the cache in its element kind:
//   e4m3        code = e4m3(x / scale[h]), to nearest even, saturating
//   e4m3, token shift = f16((max + min) / 2), scale = f16((max - min) / 2 / 448) (1
//               when that is 0), code = e4m3((x - shift) / scale)
//   int4        per group: shift = f16(min), scale = f16((max - min) / 15) (1 when
//               that is 0), code = round((x - shift) / scale) within 0..15
//   4-bit float per block of 16: block scale = e4m3(max |x| / (6 scale[h])), code =
//               e2m1(x * (1 / (block scale * scale[h]))), zeros when that product is 0
// Every lane of the warp calls it (shuffles); lanes with !on store nothing.
template <int KIND>
__device__ __forceinline__ void put_row(const CacheRowParams &p, bool is_v, bool on, int64_t row, int h,
                                        int l, const float (&x)[8], const uint4 &raw) {
  void *cache = is_v ? p.v : p.k;
  if (KIND == kBf16) {
    if (on) *(reinterpret_cast<uint4 *>(cache) + row * 16 + l) = raw;
    return;
  }
  if (KIND == kE4m3) {
    const float s = on ? __ldg((is_v ? p.v_scale : p.k_scale) + h) : 1.f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
    if (on)
      *(reinterpret_cast<uint2 *>(cache) + row * 16 + l) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
    return;
  }
  if (KIND == kFp4) {
    float a = fabsf(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) a = max_nan(a, fabsf(x[i]));
    a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
    const float g = on ? __ldg((is_v ? p.v_scale : p.k_scale) + h) : 1.f;
    const uint32_t sb = f32x2_to_e4m3x2(__fdiv_rn(a, __fmul_rn(6.f, g)), 0.f) & 0xFFu;
    const uint32_t half2 = e4m3x2_to_f16x2((uint16_t)sb);
    const float eff = __fmul_rn(f16_value(half2 & 0xFFFFu), g);
    const float inv = eff >= 0x1p-126f ? __frcp_rn(eff) : 0.f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) w |= e2m1x2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)) << (8 * i);
    if (on) {
      uint8_t *gran = reinterpret_cast<uint8_t *>(cache) + (row >> 4) * 1152;
      const int r = (int)(row & 15);
      *reinterpret_cast<uint32_t *>(gran + r * 64 + l * 4) = w;
      if ((l & 1) == 0) gran[1024 + r * 8 + (l >> 1)] = (uint8_t)sb;
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
  const float sc = f16_value(scale), sh = f16_value(shift);
  const int32_t word = (int32_t)(scale | (shift << 16));
  if (KIND == kE4m3Token) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32x2_to_e4m3x2(__fdiv_rn(__fsub_rn(x[2 * i], sh), sc), __fdiv_rn(__fsub_rn(x[2 * i + 1], sh), sc));
    if (on) {
      *(reinterpret_cast<uint2 *>(cache) + row * 16 + l) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
      if (l == 0) (is_v ? p.v_scale_shift : p.k_scale_shift)[row] = word;
    }
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float c = rintf(__fdiv_rn(__fsub_rn(x[i], sh), sc));
      w |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * i);
    }
    if (on) {
      int32_t *dst = reinterpret_cast<int32_t *>(cache) + row * (p.kv_groups + 16);
      dst[p.kv_groups + l] = (int32_t)w;
      if (l % lanes == 0) dst[l / lanes] = word;
    }
  }
}

// Slot of token t, checked: -1 for padding (and, with the error bit, for a slot outside the cache).
__device__ __forceinline__ int64_t load_slot(const CacheRowParams &p, int64_t t, uint32_t &err) {
  if (!p.slot_map) return -1;
  const int64_t s = __ldg(p.slot_map + t);
  if (s >= p.num_slots || s < -1) {
    err |= DA_DEVERR_SLOT;
    return -2;
  }
  return s;
}

// LPH lanes of 8 elements a rotated head: 16 (heads of 128) or 8 (the latent cache's 64).
template <int KIND, int LPH>
__global__ void __launch_bounds__(kWarps * 32) append_kernel(const __grid_constant__ CacheRowParams p) {
  constexpr int kPer = 32 / LPH;  // heads a warp takes at once
  constexpr int kHead = LPH * 8;
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = item / p.parts;
  const int part = (int)(item - t * p.parts);
  if (t >= p.num_tokens) return;
  const int l = lane % LPH, sub = lane / LPH;
  const int HQ = p.q ? p.num_q_heads : 0;
  const int HK = p.k_new ? (KIND == kLatent ? 1 : p.num_kv_heads) : 0;
  const int heads = HQ + (KIND == kLatent ? HK : 2 * HK);  // rotated q, rotated k, then v
  const int groups = (heads + kPer - 1) / kPer;
  const int g0 = (int)((int64_t)part * groups / p.parts), g1 = (int)((int64_t)(part + 1) * groups / p.parts);
  const __nv_bfloat16 *qrow = p.q + t * p.q_stride, *krow = p.k_new + t * p.k_stride, *vrow = p.v_new + t * p.v_stride;
  auto src_of = [&](int hd) -> const uint4 * {
    const __nv_bfloat16 *s = hd < HQ ? qrow + (int64_t)hd * kHead
                             : KIND == kLatent ? vrow  // the rope part of the latent row
                             : hd < HQ + HK ? krow + (hd - HQ) * kHead
                                            : vrow + (hd - HQ - HK) * kHead;
    return reinterpret_cast<const uint4 *>(s) + l;
  };
  uint4 w[kAhead];
  auto load = [&](int g) {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int hd = (g + k) * kPer + sub;
      w[k] = make_uint4(0u, 0u, 0u, 0u);
      if (g + k < g1 && hd < heads) w[k] = __ldg(src_of(hd));
    }
  };
  load(g0);  // in flight while the slot and the position are looked up
  uint32_t err = 0;
  const int64_t slot = load_slot(p, t, err);
  const bool padding = p.slot_map != nullptr && slot < 0;
  // this lane's pairs: half-split lanes l and l + n / 8 hold elements i and i + n
  const int n = p.rope_pairs;
  const int nl = n / 8;                       // lanes of a half (half-split)
  const bool turned = n > 0 && l < 2 * nl;
  const bool second = !p.rope_adjacent && l >= nl;
  const int pair0 = p.rope_adjacent ? 4 * l : 8 * (second ? l - nl : l);
  const int npairs = p.rope_adjacent ? 4 : 8;
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  bool bad = false;
  if (turned) {
    if (p.rope_whole) {  // one axis per aligned group of this lane's pairs: vector loads
      const int pos = __ldg(p.positions + (int64_t)p.pair_axis[pair0] * p.position_stride + t);
      bad = pos < 0 || pos >= p.max_position;
      if (!bad) {
        const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + pair0);
        const float4 *row2 = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + n + pair0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (4 * j < npairs) {
            const float4 a = __ldg(row + j), b = __ldg(row2 + j);
            c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
            s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
          }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < npairs) {
          const int pos = __ldg(p.positions + (int64_t)p.pair_axis[pair0 + i] * p.position_stride + t);
          const bool b = pos < 0 || pos >= p.max_position;
          bad = bad || b;
          if (!b) {
            c[i] = __ldg(p.cos_sin + (int64_t)pos * 2 * n + pair0 + i);
            s[i] = __ldg(p.cos_sin + (int64_t)pos * 2 * n + n + pair0 + i);
          }
        }
    }
  }
  bad = __any_sync(0xffffffffu, bad);
  if (bad && !padding) err |= DA_DEVERR_POSITION;
  if (err && lane == 0) atomicOr(p.err, err);
  if (bad || padding) return;
  const int64_t page = p.slot_map ? slot / p.rows_per_page : 0;
  const int off = p.slot_map ? (int)(slot - page * p.rows_per_page) : 0;
  const int64_t qbase = p.q_len > 1 ? (t / p.q_len * p.num_q_heads) * p.q_len + t % p.q_len : t * p.num_q_heads;
  const int partner = lane - l + (second ? l - nl : l + nl);

  for (int g = g0; g < g1; g += kAhead) {
    if (g > g0) load(g);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (g + k >= g1) break;
      const int hd = (g + k) * kPer + sub;
      const bool on = hd < heads;
      const bool is_q = hd < HQ, is_v = KIND != kLatent && hd >= HQ + HK;
      float x[8] = {bf_lo(w[k].x), bf_hi(w[k].x), bf_lo(w[k].y), bf_hi(w[k].y),
                    bf_lo(w[k].z), bf_hi(w[k].z), bf_lo(w[k].w), bf_hi(w[k].w)};
      if (n > 0 && __any_sync(0xffffffffu, !is_v)) {
        uint4 o = w[k];
        if (p.rope_adjacent) {
          float y[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            y[2 * i] = __fsub_rn(__fmul_rn(x[2 * i], c[i]), __fmul_rn(x[2 * i + 1], s[i]));
            y[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], c[i]), __fmul_rn(x[2 * i], s[i]));
          }
          o = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        } else {
          uint4 z;
          z.x = __shfl_sync(0xffffffffu, w[k].x, partner);
          z.y = __shfl_sync(0xffffffffu, w[k].y, partner);
          z.z = __shfl_sync(0xffffffffu, w[k].z, partner);
          z.w = __shfl_sync(0xffffffffu, w[k].w, partner);
          const float u[8] = {bf_lo(z.x), bf_hi(z.x), bf_lo(z.y), bf_hi(z.y),
                              bf_lo(z.z), bf_hi(z.z), bf_lo(z.w), bf_hi(z.w)};
          float y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float a = __fmul_rn(x[i], c[i]), b = __fmul_rn(u[i], s[i]);
            y[i] = second ? __fadd_rn(a, b) : __fsub_rn(a, b);
          }
          o = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        }
        if (turned && !is_v) {
          w[k] = o;
          x[0] = bf_lo(o.x), x[1] = bf_hi(o.x), x[2] = bf_lo(o.y), x[3] = bf_hi(o.y);
          x[4] = bf_lo(o.z), x[5] = bf_hi(o.z), x[6] = bf_lo(o.w), x[7] = bf_hi(o.w);
        }
      }
      if (on && is_q) {
        const int64_t row = p.q_len > 1 ? qbase + (int64_t)hd * p.q_len : qbase + hd;
        *(reinterpret_cast<uint4 *>(p.q_out) + row * LPH + l) = w[k];
      }
      if (KIND == kLatent) {
        if (on && !is_q) *(reinterpret_cast<uint4 *>(p.v) + slot * 8 + l) = w[k];
      } else if (__any_sync(0xffffffffu, on && !is_q)) {
        const int h = hd - HQ - (is_v ? HK : 0);
        put_row<KIND>(p, is_v, on && !is_q, cache_row(p, page, off, h), h, l, x, w[k]);
      }
    }
  }
  if (KIND == kLatent && HK && part == p.parts - 1) {  // the 512 latent elements, as they are
    const uint4 *src = reinterpret_cast<const uint4 *>(krow) + lane;
    uint4 *dst = reinterpret_cast<uint4 *>(p.k) + slot * 64 + lane;
    const uint4 a = __ldg(src), b = __ldg(src + 32);
    dst[0] = a;
    dst[32] = b;
  }
}

// Eight elements (lane l of 16) of row `row` as bf16 pairs: each value is the
// fp32 product (and sum) of its parts, rounded once more to bf16.
struct RowBits {
  uint4 a;      // the lane's codes (bf16: its values)
  uint32_t s;   // block scale byte, or scale and shift halves
};
template <int KIND>
__device__ __forceinline__ RowBits get_row(const CacheRowParams &p, bool is_v, int64_t row, int l) {
  const void *cache = is_v ? p.v : p.k;
  RowBits r;
  r.a = make_uint4(0u, 0u, 0u, 0u);
  r.s = 0;
  if (KIND == kBf16) r.a = __ldg(reinterpret_cast<const uint4 *>(cache) + row * 16 + l);
  if (KIND == kE4m3 || KIND == kE4m3Token) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(cache) + row * 16 + l);
    r.a.x = v.x;
    r.a.y = v.y;
    if (KIND == kE4m3Token) r.s = (uint32_t)__ldg((is_v ? p.v_scale_shift : p.k_scale_shift) + row);
  }
  if (KIND == kInt4) {
    const uint32_t *src = reinterpret_cast<const uint32_t *>(cache) + row * (p.kv_groups + 16);
    r.a.x = __ldg(src + p.kv_groups + l);
    r.s = __ldg(src + l * p.kv_groups / 16);
  }
  if (KIND == kFp4) {
    const uint8_t *gran = reinterpret_cast<const uint8_t *>(cache) + (row >> 4) * 1152;
    const int i = (int)(row & 15);
    r.a.x = __ldg(reinterpret_cast<const uint32_t *>(gran + i * 64 + l * 4));
    r.s = __ldg(gran + 1024 + i * 8 + (l >> 1));
  }
  return r;
}
template <int KIND>
__device__ __forceinline__ uint4 row_values(const CacheRowParams &p, const RowBits &r, float head_scale) {
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
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = item / p.parts;
  const int part = (int)(item - t * p.parts);
  if (t >= p.num_tokens) return;
  uint32_t err = 0;
  const int64_t slot = load_slot(p, t, err);
  if (err && lane == 0) atomicOr(p.err, err);
  if (slot < 0) return;
  if (KIND == kLatent) {  // 512 + 64 elements: 72 chunks of 16 bytes
    const uint4 *ck = reinterpret_cast<const uint4 *>(p.k) + slot * 64;
    uint4 *ok = reinterpret_cast<uint4 *>(p.k_out) + t * 64;
    const uint4 a = __ldg(ck + lane), b = __ldg(ck + 32 + lane);
    if (lane < 8) {
      const uint4 c = __ldg(reinterpret_cast<const uint4 *>(p.v) + slot * 8 + lane);
      *(reinterpret_cast<uint4 *>(p.v_out) + t * 8 + lane) = c;
    }
    ok[lane] = a;
    ok[32 + lane] = b;
    return;
  }
  const int l = lane & 15, sub = lane >> 4;
  const int64_t page = slot / p.rows_per_page;
  const int off = (int)(slot - page * p.rows_per_page);
  const int rows = 2 * p.num_kv_heads;  // K then V; two rows at once
  const int groups = p.num_kv_heads;
  const int g0 = (int)((int64_t)part * groups / p.parts), g1 = (int)((int64_t)(part + 1) * groups / p.parts);
  for (int g = g0; g < g1; g += kAhead) {
    RowBits r[kAhead];
    float hs[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = (g + k) * 2 + sub;
      if (g + k < g1 && i < rows) {
        const bool is_v = i >= p.num_kv_heads;
        const int h = is_v ? i - p.num_kv_heads : i;
        r[k] = get_row<KIND>(p, is_v, cache_row(p, page, off, h), l);
        if (KIND == kE4m3 || KIND == kFp4) hs[k] = __ldg((is_v ? p.v_scale : p.k_scale) + h);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = (g + k) * 2 + sub;
      if (g + k < g1 && i < rows) {
        const bool is_v = i >= p.num_kv_heads;
        const int h = is_v ? i - p.num_kv_heads : i;
        *(reinterpret_cast<uint4 *>(is_v ? p.v_out : p.k_out) + (t * p.num_kv_heads + h) * 16 + l) =
            row_values<KIND>(p, r[k], hs[k]);
      }
    }
  }
}

int64_t blocks_for(int64_t items) { return (items + kWarps - 1) / kWarps; }

// Parts a token's heads are cut into: about 48 warps for every SM, when there are
// fewer tokens than that.
int parts_for(int64_t tokens, int groups, int num_sms) {
  const int64_t want = (int64_t)num_sms * 48;
  const int64_t parts = (want + tokens - 1) / tokens;
  return (int)(parts < 1 ? 1 : parts > groups ? groups : parts);
}

}  // namespace

cudaError_t launch_append(CacheRowParams p, int kind, int num_sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  const int per = kind == kLatent ? 4 : 2;
  const int heads = (p.q ? p.num_q_heads : 0) + (p.k_new ? (kind == kLatent ? 1 : 2 * p.num_kv_heads) : 0);
  if (heads == 0) return cudaSuccess;
  p.parts = parts_for(p.num_tokens, (heads + per - 1) / per, num_sms);
  const int64_t blocks = blocks_for((int64_t)p.num_tokens * p.parts);
  const unsigned grid = (unsigned)blocks;
  switch (kind) {
    case kBf16: append_kernel<kBf16, 16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kE4m3: append_kernel<kE4m3, 16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kE4m3Token: append_kernel<kE4m3Token, 16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kInt4: append_kernel<kInt4, 16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kFp4: append_kernel<kFp4, 16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    default: append_kernel<kLatent, 8><<<grid, kWarps * 32, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_gather(CacheRowParams p, int kind, int num_sms, cudaStream_t stream) {
  if (p.num_tokens == 0) return cudaSuccess;
  p.parts = kind == kLatent ? 1 : parts_for(p.num_tokens, p.num_kv_heads, num_sms);
  const unsigned grid = (unsigned)blocks_for((int64_t)p.num_tokens * p.parts);
  switch (kind) {
    case kBf16: gather_kernel<kBf16><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kE4m3: gather_kernel<kE4m3><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kE4m3Token: gather_kernel<kE4m3Token><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kInt4: gather_kernel<kInt4><<<grid, kWarps * 32, 0, stream>>>(p); break;
    case kFp4: gather_kernel<kFp4><<<grid, kWarps * 32, 0, stream>>>(p); break;
    default: gather_kernel<kLatent><<<grid, kWarps * 32, 0, stream>>>(p); break;
  }
  return cudaGetLastError();
}

}  // namespace da
