// block8_split.cu -- persistent split-KV GQA decode over a cache of 8-bit codes with an fp32 scale
// for each block of 16 to 256 positions and kv head, for sm_103a.
//
// The mathematics. A cached key or value element is code * scale[block]: an e4m3 or a signed
// integer code, exact in f16. A granule of 16 positions lies in one block, so
//   S^T = (K codes) Q^T * kscale,   O^T += vscale * (V codes)^T P^T
// with the products on f16 operands with fp32 sums and the scales applied to them in fp32: any
// fp32 scale serves. With sixteen rows a unit, where the scheduler's issue is what bounds the kernel, the V
// scale joins the weights instead, over a power of two that O is in units of (but where it is far below
// that, or not finite). With eight rows, which HBM bounds, that costs more than it saves. Roundings: the weights
// meet V as f16 (11 bits, as the codes' products with them need no more for a bf16 output: 2^-11 of a weight; the
// smallest step is 2^-29 of the greatest weight, or 2^-25 where a V scale is joined that is 2^-4 of its reference),
// everything else is fp32. (Integers as code plus 128, whose bits are an f16 as they stand, with 128 sum q taken off
// the score: a subtraction less for two codes, no time, 95.6 us either way, and scores that are differences of two
// great sums: off by 1.7e-3 where these are by 3e-6.)
//
// What bounds it. 16 positions of one kv head are 4096 bytes, 732 cycles of a scheduler at the
// measured copy bandwidth; their conversions, products and weights take about 250. So HBM does.
// How tiles are walked, cut and merged stands in stream_split.cuh.
// Measured: 32 rows of 1024..8192 tokens, 8 kv heads of 4 rows: 56.3 us (floor 40.4); one row of 131072, 8 heads of 8
// rows: 56.7 (39.6). While it streams it takes 97 to 106 % of the copy rate (rows of 16384 tokens against rows of 8192);
// the first tile is there after 5 us, the last block's warps end 5 us after the median one's, pieces and units
// that blocks share take 7. Sixteen rows a unit: 16 rows of 1000..20000 tokens, 4 query tokens, 95.3 us (51.4);
// e4m3 streams at 84 % of the copy rate there, integers at 74 % (936 instructions for 32 tokens, issue 47 %).
// Measured and not kept for eight rows: 9, 11, 13 or 15 warps, one or two stages, tiles of 16 tokens (55 to 61 us).
//
// The stage. Rows of 128 bytes land with their eight 16-byte chunks turned by the row: chunk c of
// row r at c ^ (r & 7). A quad reads chunks 2 q, 2 q + 1 of a K row (its dims 32 q .. 32 q + 31: the
// contraction's order is free and Q is read in the same), a lane chunk r of its V rows, both
// without bank conflicts.
#include "stream_split.cuh"

namespace da {
namespace {

// Two pairs of codes (bytes 0, 1 and 2, 3 of w) as f16 pairs, exact. Integers come with 128 added,
// as bytes below 0x64: 1024 + byte, less 1152.
template <bool INT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (INT) {
    const __half2 off = __half2half2(__ushort_as_half(0x6480));
    const uint32_t a = prmt(w, 0x64646464u, 0x4140), b = prmt(w, 0x64646464u, 0x4342);
    const __half2 x = __hsub2(*reinterpret_cast<const __half2 *>(&a), off);
    const __half2 y = __hsub2(*reinterpret_cast<const __half2 *>(&b), off);
    lo = *reinterpret_cast<const uint32_t *>(&x);
    hi = *reinterpret_cast<const uint32_t *>(&y);
  } else {
    lo = e4m3x2_to_f16x2((uint16_t)w);
    hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  }
}
template <bool INT>
__device__ __forceinline__ uint32_t biased(uint32_t w) {
  return INT ? w ^ 0x80808080u : w;
}
__device__ __forceinline__ uint32_t word(const uint4 &v, int c) {
  return c == 0 ? v.x : c == 1 ? v.y : c == 2 ? v.z : v.w;
}

// Up to eight rows a unit: 32 tokens a stage, seven streaming warps, Q in registers. Sixteen, whose O takes
// 64 registers: 16 tokens a stage, eleven warps in 168 registers, Q in shared memory (16 rows of 1000..20000
// tokens, 4 query tokens: 95.3 us, with 8 to 42 bytes of spills a thread; as for eight rows, in 255 registers, 102;
// fifteen warps in 128: 106).
template <bool INT, int ROWS>
struct Block8Format {
  static constexpr int kT = ROWS == 1 ? 32 : 16;
  static constexpr int kH = kT / 16;
  static constexpr int kGranBytes = 2048;
  static constexpr int kSideBytes = 16;  // K's scales, then V's
  static constexpr bool kHeadScales = false;
  static constexpr bool kCareful = true;
  static constexpr bool kBlockScales = true;
  static constexpr bool kFoldsV = ROWS == 2;
  static constexpr int kWarps(int nt) { return nt == 1 ? 7 : 11; }
  static constexpr int kStages(int) { return 3; }
  static constexpr bool kQShared(int nt) { return nt == 2; }

  const uint8_t *k_lane, *v_lane;
  const float *scale;  // lane 0: K's, lane 1: V's
  int lane, shift, k0, k1, v0, v1;
  uint32_t even, turn;  // where the lane's 16 bytes of rows 0 .. 3 go, and how much further those of rows 4 .. 7
  __device__ __forceinline__ Block8Format(const StreamParams &fp, int l)
      : k_lane(fp.k + l * 16), v_lane(fp.v + l * 16), scale(l == 0 ? fp.g.k_scale : fp.g.v_scale), lane(l),
        shift(fp.scale_shift) {
    const int q4 = l & 3, r8 = l >> 2;
    even = (l >> 3) * 128 + (((l & 7) ^ (l >> 3)) << 4);
    turn = (even ^ 64) - even;
    k0 = r8 * 128 + (((2 * q4) ^ r8) << 4);
    k1 = r8 * 128 + (((2 * q4 + 1) ^ r8) << 4);
    v0 = 2 * q4 * 128 + ((r8 ^ (2 * q4)) << 4);
    v1 = (2 * q4 + 1) * 128 + ((r8 ^ (2 * q4 + 1)) << 4);
  }
  __device__ __forceinline__ uint32_t lane_at() const { return even; }
  __device__ __forceinline__ void copy(uint32_t k, uint32_t v, int64_t off, uint8_t *scales, int gi) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      cp_async_16(k + j * 512 + (j & 1 ? turn : 0u), k_lane + off + j * 512);
      cp_async_16(v + j * 512 + (j & 1 ? turn : 0u), v_lane + off + j * 512);
    }
    if (lane < 2) cp_async_4(scales + 4 * (lane * kH + gi), scale + (off >> shift));
  }
  __device__ static __forceinline__ float v_scale(const uint8_t *scales, int gi) {
    return reinterpret_cast<const float *>(scales)[kH + gi];
  }
  template <int NT>
  __device__ __forceinline__ void scores(const uint8_t *stage, const uint8_t *scales, const uint32_t (&qf)[NT][8][2],
                                         const uint4 *qs, float (&s)[NT][kH][4]) const {
    const float *ks = reinterpret_cast<const float *>(scales);
#pragma unroll
    for (int gi = 0; gi < kH; ++gi) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][gi][0] = s[nt][gi][1] = s[nt][gi][2] = s[nt][gi][3] = 0.f;
      const uint8_t *gk = stage + gi * kGranBytes;
      uint4 a[2], b[2];  // rows r8 and r8 + 8
      a[0] = *reinterpret_cast<const uint4 *>(gk + k0);
      a[1] = *reinterpret_cast<const uint4 *>(gk + k1);
      b[0] = *reinterpret_cast<const uint4 *>(gk + k0 + 1024);
      b[1] = *reinterpret_cast<const uint4 *>(gk + k1 + 1024);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        uint32_t a0, a1, a2, a3;
        codes_to_f16<INT>(biased<INT>(word(a[c >> 2], c & 3)), a0, a2);
        codes_to_f16<INT>(biased<INT>(word(b[c >> 2], c & 3)), a1, a3);
        if constexpr (kQShared(NT)) {
          const uint4 q = qs[c * 32];
          mma_f16_16816(s[0][gi], a0, a1, a2, a3, q.x, q.y);
          mma_f16_16816(s[NT - 1][gi], a0, a1, a2, a3, q.z, q.w);
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt][gi], a0, a1, a2, a3, qf[nt][c][0], qf[nt][c][1]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][gi][e] *= ks[gi];
    }
  }
  // Masked tokens weigh 0: their rows must not hold NaN codes, nor a granule that was not copied
  // any scale.
  __device__ __forceinline__ void drop(uint8_t *stage, uint8_t *scales, uint32_t valid) const {
    if (!INT && lane < kT && !((valid >> lane) & 1u)) {
      uint4 *row = reinterpret_cast<uint4 *>(stage + kH * kGranBytes + lane * 128);
#pragma unroll
      for (int j = 0; j < 8; ++j) row[j ^ (lane & 7)] = make_uint4(0u, 0u, 0u, 0u);
    }
    if (lane < kH && ((valid >> (16 * lane)) & 0xFFFFu) == 0) reinterpret_cast<float *>(scales)[kH + lane] = 0.f;
  }
  template <int NT>
  __device__ __forceinline__ void values(const uint8_t *v, const float (&vmul)[kH], bool fold,
                                         const uint32_t (&pb)[NT][kH][2], float (&oacc)[NT][8][4]) const {
    if (kFoldsV && fold) products<NT, true>(v, vmul, pb, oacc);
    else products<NT, false>(v, vmul, pb, oacc);
  }
  template <int NT, bool FOLD>
  __device__ __forceinline__ void products(const uint8_t *v, const float (&vmul)[kH], const uint32_t (&pb)[NT][kH][2],
                                           float (&oacc)[NT][8][4]) const {
#pragma unroll
    for (int gi = 0; gi < kH; ++gi) {
      const uint8_t *gv = v + gi * kGranBytes;
      // tokens 2 q4, 2 q4 + 1 and the same + 8, dims 16 r8 .. 16 r8 + 15 of each
      const uint4 w0 = *reinterpret_cast<const uint4 *>(gv + v0), w1 = *reinterpret_cast<const uint4 *>(gv + v1);
      const uint4 w8 = *reinterpret_cast<const uint4 *>(gv + v0 + 1024);
      const uint4 w9 = *reinterpret_cast<const uint4 *>(gv + v1 + 1024);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t x0 = biased<INT>(word(w0, c)), x1 = biased<INT>(word(w1, c));
        const uint32_t x8 = biased<INT>(word(w8, c)), x9 = biased<INT>(word(w9, c));
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // dims 16 r8 + 4 c + 2 k and the next
          uint32_t a0, a1, a2, a3;
          codes_to_f16<INT>(prmt(x0, x1, k ? 0x7362 : 0x5140), a0, a1);
          codes_to_f16<INT>(prmt(x8, x9, k ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (FOLD) {
              mma_f16_16816(oacc[nt][2 * c + k], a0, a1, a2, a3, pb[nt][gi][0], pb[nt][gi][1]);
            } else {
              float o[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16_16816(o, a0, a1, a2, a3, pb[nt][gi][0], pb[nt][gi][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) oacc[nt][2 * c + k][e] = fmaf(o[e], vmul[gi], oacc[nt][2 * c + k][e]);
            }
          }
        }
      }
    }
  }
  // Whether a valid token of the stage has a NaN value code, or a V scale is not finite.
  __device__ __forceinline__ bool not_finite(const uint8_t *v, const uint8_t *scales, uint32_t valid) const {
    bool odd = false;
    if (!INT && lane < kT && ((valid >> lane) & 1u)) {
      const uint4 *row = reinterpret_cast<const uint4 *>(v + lane * 128);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint4 x = row[j ^ (lane & 7)];
#pragma unroll
        for (int c = 0; c < 4; ++c) odd = odd || (((word(x, c) & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
      }
    }
    if (lane < kH) odd = odd || !(fabsf(reinterpret_cast<const float *>(scales)[kH + lane]) < __int_as_float(0x7f800000));
    return __any_sync(0xffffffffu, odd);
  }
  // values() token by token, leaving out what a row's mask leaves out.
  template <int NT>
  __device__ __forceinline__ void values_kept(const uint8_t *v, const float (&vmul)[kH], uint32_t valid,
                                              const float (&s)[NT][kH][4], const float (&y)[NT][2][2 * kH],
                                              float (&oacc)[NT][8][4]) const {
    const int q4 = lane & 3, r8 = lane >> 2;
    const float ninf = -__int_as_float(0x7f800000);
#pragma unroll
    for (int k = 0; k < 2 * kH; ++k) {
      const float vs = vmul[k >> 1];
      for (int r = 0; r < 8; ++r) {  // token 8 k + r, whose weights lane (r, q4) has
        float w[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // (-1: not kept; a masked score is -inf)
            const bool kept = ((valid >> (8 * k + r8)) & 1u) && s[nt][k >> 1][(k & 1) * 2 + e] != ninf;
            w[nt][e] = __shfl_sync(0xffffffffu, kept ? y[nt][e][k] : -1.f, r * 4 + q4);
          }
        const uint4 x = *reinterpret_cast<const uint4 *>(v + (8 * k + r) * 128 + ((r8 ^ r) << 4));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t h[2];
          codes_to_f16<INT>(biased<INT>(word(x, c)), h[0], h[1]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 d = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (w[nt][e] < 0.f) continue;  // (NaN weights go through)
                oacc[nt][2 * c + j][e] = fmaf(w[nt][e], d.x * vs, oacc[nt][2 * c + j][e]);
                oacc[nt][2 * c + j][2 + e] = fmaf(w[nt][e], d.y * vs, oacc[nt][2 * c + j][2 + e]);
              }
          }
        }
      }
    }
  }
};

template <bool INT, int NT, int MOD>
__global__ void __launch_bounds__(StreamLayout<Block8Format<INT, NT>, NT>::kThreads, 1)
    block8_split_kernel(const StreamParams fp) {
  begin_dependent();
  stream_split<Block8Format<INT, NT>, NT, MOD>(fp);
}

template <bool INT, int NT, int MOD>
cudaError_t block8_attr() {
  return cudaFuncSetAttribute(block8_split_kernel<INT, NT, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              StreamLayout<Block8Format<INT, NT>, NT>::kTotal);
}
template <bool INT>
cudaError_t block8_attrs() {
  cudaError_t e;
  if ((e = block8_attr<INT, 1, 0>()) != cudaSuccess) return e;
  if ((e = block8_attr<INT, 1, 1>()) != cudaSuccess) return e;
  if ((e = block8_attr<INT, 1, 2>()) != cudaSuccess) return e;
  if ((e = block8_attr<INT, 2, 0>()) != cudaSuccess) return e;
  if ((e = block8_attr<INT, 2, 1>()) != cudaSuccess) return e;
  return block8_attr<INT, 2, 2>();
}

template <bool INT>
cudaError_t launch(const StreamParams &p, int ctas, cudaStream_t stream) {
  const int mod = gqa_mod(p.g);
#define DA_B8(NT, M)                                                                                          \
  return launch_dependent(block8_split_kernel<INT, NT, M>, (unsigned)ctas,                                     \
                          StreamLayout<Block8Format<INT, NT>, NT>::kThreads, StreamLayout<Block8Format<INT, NT>, NT>::kTotal, \
                          stream, p)
  if (p.g.group <= 8) {
    if (mod == 0) DA_B8(1, 0);
    else if (mod == 1) DA_B8(1, 1);
    else DA_B8(1, 2);
  } else {
    if (mod == 0) DA_B8(2, 0);
    else if (mod == 1) DA_B8(2, 1);
    else DA_B8(2, 2);
  }
#undef DA_B8
}

}  // namespace

int block8_tile(int group) { return group <= 8 ? Block8Format<false, 1>::kT : Block8Format<false, 2>::kT; }
int block8_warps(int group) { return Block8Format<false, 1>::kWarps(group <= 8 ? 1 : 2); }

cudaError_t block8_prepare() {
  cudaError_t e = append_blocks_prepare();
  if (e == cudaSuccess) e = block8_attrs<false>();
  return e != cudaSuccess ? e : block8_attrs<true>();
}

cudaError_t launch_block8(const StreamParams &p, bool integers, int ctas, cudaStream_t stream) {
  return integers ? launch<true>(p, ctas, stream) : launch<false>(p, ctas, stream);
}

}  // namespace da
