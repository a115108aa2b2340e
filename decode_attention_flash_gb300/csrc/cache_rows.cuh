// cache_rows.cuh -- what the append of any element kind shares (cache_rows.cu, cache_blocks.cu):
// slots, positions, the norm over a head, the turn by its positions, and the queries' part.
#pragma once

#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace da {
namespace {

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

// The cosines and sines of pairs pair0 .. pair0 + 7 (or + 3: kPairs) at a position of the table.
template <int kPairs>
__device__ __forceinline__ void load_angles(const CacheRowParams &p, int pos, int pair0, float (&c)[8], float (&s)[8]) {
  const int n = p.rope_pairs;
  const float4 *row = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + pair0);
  const float4 *row2 = reinterpret_cast<const float4 *>(p.cos_sin + (int64_t)pos * 2 * n + n + pair0);
#pragma unroll
  for (int j = 0; j < kPairs / 4; ++j) {
    const float4 a = __ldg(row + j), b = __ldg(row2 + j);
    c[4 * j] = a.x, c[4 * j + 1] = a.y, c[4 * j + 2] = a.z, c[4 * j + 3] = a.w;
    s[4 * j] = b.x, s[4 * j + 1] = b.y, s[4 * j + 2] = b.z, s[4 * j + 3] = b.w;
  }
}
// The cosines and sines of pairs pair0 .. pair0 + 7 (or + 3: kPairs) of token t;
// false when a position is outside the table.
template <int kPairs>
__device__ __forceinline__ bool load_turn(const CacheRowParams &p, int64_t t, int pair0, float (&c)[8], float (&s)[8]) {
  const int n = p.rope_pairs;
  if (p.rope_whole) {  // they share an axis: vector loads
    const int pos = p.positions[(int64_t)p.pair_axis[pair0] * p.position_stride + t];
    if (pos < 0 || pos >= p.max_position) return false;
    load_angles<kPairs>(p, pos, pair0, c, s);
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

// A key of 16 lanes, 8 elements each, turned (lanes with `turned`); the partner of a half-split pair is
// in lane `partner`, c and s are signed for the lane's half. Every lane of the warp calls it.
__device__ __forceinline__ void turn_key(const CacheRowParams &p, uint4 &v, int partner, bool turned, const float (&c)[8],
                                         const float (&s)[8]) {
  if (p.rope_adjacent) {
    if (turned) turn_adjacent(v, c, s, 0);
    return;
  }
  const uint4 z = make_uint4(__shfl_sync(0xffffffffu, v.x, partner), __shfl_sync(0xffffffffu, v.y, partner),
                             __shfl_sync(0xffffffffu, v.z, partner), __shfl_sync(0xffffffffu, v.w, partner));
  if (turned) {
    uint32_t x[4] = {v.x, v.y, v.z, v.w};
    const uint32_t y[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = pack_bf16(__fsub_rn(__fmul_rn(bf_lo(x[j]), c[2 * j]), __fmul_rn(bf_lo(y[j]), s[2 * j])),
                       __fsub_rn(__fmul_rn(bf_hi(x[j]), c[2 * j + 1]), __fmul_rn(bf_hi(y[j]), s[2 * j + 1])));
    v = make_uint4(x[0], x[1], x[2], x[3]);
  }
}

// ---------------------------------------------------------------- the norm of a head

// Eight bf16 elements, or eight consecutive floats (ordinary loads; 16-byte aligned), as pairs.
struct Eight {
  Pair v[4];
};
__device__ __forceinline__ Eight values8(const uint4 &w) {
  return {{pack(bf_lo(w.x), bf_hi(w.x)), pack(bf_lo(w.y), bf_hi(w.y)), pack(bf_lo(w.z), bf_hi(w.z)),
           pack(bf_lo(w.w), bf_hi(w.w))}};
}
__device__ __forceinline__ Eight load8(const float *src) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2 *>(src)[0], b = reinterpret_cast<const ulonglong2 *>(src)[1];
  return {{a.x, a.y, b.x, b.y}};
}
__device__ __forceinline__ uint32_t bf16x2_of(Pair v) {
  float a, b;
  unpack(v, a, b);
  return pack_bf16(a, b);
}
__device__ __forceinline__ uint4 pack8(const Eight &x) {
  return make_uint4(bf16x2_of(x.v[0]), bf16x2_of(x.v[1]), bf16x2_of(x.v[2]), bf16x2_of(x.v[3]));
}
__device__ __forceinline__ Eight times(const Eight &x, const Eight &y) {
  return {{mul2(x.v[0], y.v[0]), mul2(x.v[1], y.v[1]), mul2(x.v[2], y.v[2]), mul2(x.v[3], y.v[3])}};
}
__device__ __forceinline__ Eight times(const Eight &x, float n) {
  const Pair m = pack(n, n);
  return {{mul2(x.v[0], m), mul2(x.v[1], m), mul2(x.v[2], m), mul2(x.v[3], m)}};
}
__device__ __forceinline__ Eight plus(const Eight &x, const Eight &y) {
  return {{add2(x.v[0], y.v[0]), add2(x.v[1], y.v[1]), add2(x.v[2], y.v[2]), add2(x.v[3], y.v[3])}};
}
__device__ __forceinline__ Eight minus(const Eight &x, const Eight &y) {
  return {{sub2(x.v[0], y.v[0]), sub2(x.v[1], y.v[1]), sub2(x.v[2], y.v[2]), sub2(x.v[3], y.v[3])}};
}
__device__ __forceinline__ Eight pairs8(const float (&x)[8]) {
  return {{pack(x[0], x[1]), pack(x[2], x[3]), pack(x[4], x[5]), pack(x[6], x[7])}};
}
__device__ __forceinline__ float squares(const Eight &x) {
  Pair sum = mul2(x.v[0], x.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) sum = fma2(x.v[i], x.v[i], sum);
  float a, b;
  unpack(sum, a, b);
  return a + b;
}
// 1 / sqrt(mean x^2 + eps) of a head of LANES lanes with ELEMENTS each and these sums of squares; every
// lane of the warp calls it.
template <int LANES, int ELEMENTS>
__device__ __forceinline__ float head_rsqrt(float sum, float eps) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return rsqrtf(fmaf(sum, 1.f / (LANES * ELEMENTS), eps));
}
// Neighbours as pairs: elements 2i, 2i + 1 with cosines c[at + i].
__device__ __forceinline__ void turn_neighbours(Eight &x, const float (&c)[8], const float (&s)[8], int at) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b, u, v;
    unpack(x.v[i], a, b);
    turn(a, b, c[at + i], s[at + i], u, v);
    x.v[i] = pack(u, v);
  }
}

// A key of 16 lanes, 8 elements each: normed, then turned (lanes with `turned`); the partner of a
// half-split pair is in lane `partner`, c and s are its angle's (`second`: the lane has the pair's second
// elements). Every lane of the warp calls it. (The weights come from L1 for each key: 32 registers held
// for them cost more warps than they save.)
__device__ __forceinline__ void norm_key(const CacheRowParams &p, uint4 &v, int kl, int partner, bool turned, bool second,
                                         const float (&c)[8], const float (&s)[8]) {
  Eight x = values8(v);
  const float n = head_rsqrt<16, 8>(squares(x), p.norm_eps);
  const uint4 z = make_uint4(__shfl_sync(0xffffffffu, v.x, partner), __shfl_sync(0xffffffffu, v.y, partner),
                             __shfl_sync(0xffffffffu, v.z, partner), __shfl_sync(0xffffffffu, v.w, partner));
  x = times(times(x, n), load8(p.k_weight + 8 * kl));
  if (turned) {
    if (p.rope_adjacent) {
      turn_neighbours(x, c, s, 0);
    } else {
      // (b c + a s) is (x c - y s) with y of the other sign
      const Eight y = times(times(values8(z), second ? -n : n), load8(p.k_weight + 8 * (partner & 15)));
      x = minus(times(x, pairs8(c)), times(y, pairs8(s)));
    }
  }
  v = pack8(x);
}

// ---------------------------------------------------------------- the queries of a token

constexpr int kAhead = 4;  // loads of queries in flight a lane

// This lane's chunks of a head. Half-split pairs of r chunks: lane i < r
// has chunks i and i + r; neighbours as pairs: chunks 2i and 2i + 1; elements past
// the rotated ones stay, two chunks a lane.
template <int HEAD>
struct QueryLane {
  bool turned, split;
  int ca, cb, sub;
  __device__ __forceinline__ QueryLane(const CacheRowParams &p, int lane) {
    constexpr int kLanes = HEAD / 16;
    const int l = lane % kLanes, r = p.rope_pairs / 8;
    sub = lane / kLanes;
    turned = l < r;
    split = turned && !p.rope_adjacent;
    ca = split ? l : 2 * l, cb = split ? l + r : 2 * l + 1;
  }
};

// Query heads of groups g0 .. gq1 - 1 (32 / kLanes heads each) of token t, and the token's slot and
// this lane's cosines and sines for whoever comes next. False: nothing more is to be done for
// the token (padding, or a slot or position that is out of range).
template <int HEAD, bool NORM>
__device__ __forceinline__ bool append_queries(const CacheRowParams &p, int64_t t, int lane, const QueryLane<HEAD> &ql,
                                               int g0, int gq1, int HQ, int64_t &slot, float (&c)[8], float (&s)[8]) {
  constexpr int kChunks = HEAD / 8;        // 16-byte chunks of a head
  constexpr int kLanes = kChunks / 2;      // lanes of a head with both halves of its pairs
  constexpr int kHeads = 32 / kLanes;      // query heads a warp takes at once
  constexpr int kDeep = kAhead / 2;        // groups of them in flight
  const int l = lane % kLanes, sub = ql.sub, ca = ql.ca, cb = ql.cb;
  const bool turned = ql.turned, split = ql.split;
  const uint4 *qsrc = reinterpret_cast<const uint4 *>(p.q + t * p.q_stride);
  uint4 a[kDeep], b[kDeep];
  auto load_q = [&](int g) {
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int hd = (g + k) * kHeads + sub;
      if (NORM) a[k] = b[k] = make_uint4(0u, 0u, 0u, 0u);
      if (g + k < gq1 && hd < HQ) {
        a[k] = qsrc[hd * kChunks + ca];
        b[k] = qsrc[hd * kChunks + cb];
      }
    }
  };
  load_q(g0);  // in flight while the slot and the positions are looked up
  uint32_t err = 0;
  slot = load_slot(p, t, err);
  const bool padding = p.slot_map != nullptr && slot < 0;
  bool bad = false;
  if (turned) bad = !load_turn<8>(p, t, 8 * l, c, s);
  bad = __any_sync(0xffffffffu, bad);
  if (bad && !padding) err |= DA_DEVERR_POSITION;
  if (err && lane == 0) atomicOr(p.err, err);
  if (bad || padding) return false;
  const bool norm = NORM && p.q_weight != nullptr;
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
        if (g + k >= gq1 || (!NORM && hd >= HQ)) continue;
        if (norm) {
          Eight x = values8(a[k]), y = values8(b[k]);
          const float n = head_rsqrt<kLanes, 16>(squares(x) + squares(y), p.norm_eps);
          x = times(times(x, n), load8(p.q_weight + 8 * ca));
          y = times(times(y, n), load8(p.q_weight + 8 * cb));
          if (split) {
            const Eight cc = pairs8(c), ss = pairs8(s), u = minus(times(x, cc), times(y, ss));
            y = plus(times(y, cc), times(x, ss));
            x = u;
          } else if (turned) {
            turn_neighbours(x, c, s, 0);
            turn_neighbours(y, c, s, 4);
          }
          a[k] = pack8(x);
          b[k] = pack8(y);
        } else if (split) {
          turn_halves(a[k], b[k], c, s);
        } else if (turned) {
          turn_adjacent(a[k], c, s, 0);
          turn_adjacent(b[k], c, s, 4);
        }
        if (NORM && hd >= HQ) continue;
        dst[(int64_t)hd * step + ca] = a[k];
        dst[(int64_t)hd * step + cb] = b[k];
      }
    }
  }
  return true;
}

}  // namespace
}  // namespace da
