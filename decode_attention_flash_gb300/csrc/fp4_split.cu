// fp4_split.cu -- persistent split-KV GQA decode over a 4-bit floating-point cache, for sm_103a.
//
// The mathematics. A cached key or value element is code * block_scale *
// head_scale: an e2m1 code (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), an
// e4m3 scale shared by 16 consecutive elements of the row, and one fp32 scale
// per kv head. code * block_scale has at most six significant bits between 2^-10
// and 2688, so it is exact in f16; the head scale of K joins the score factor and
// that of V the epilogue. The rest is the online softmax of gqa_split.cuh:
//   S^T = K Q^T,  O^T += V^T P^T   (mma.sync m16n8k16, f16 operands, fp32 sums)
// with the query group as the MMA's N dimension.
//
// What bounds it. 16 tokens of one kv head are 2304 bytes and 4096 elements to
// turn into f16. Measured per scheduler: an e2m1 conversion (a pair a lane) takes 2
// cycles of the ALU, a multiply by the block's scale 2 of the FMA pipe, an m16n8k16
// 8.2; 64 + 64 + 16 of them, with what they hold up of each other, take 322 cycles for
// 16 tokens, against 412 that the measured copy bandwidth leaves. So the kernel is
// laid out to add as little as possible to that (291 instructions for 16 tokens in
// all, 211 of them the above):
//  - every warp streams alone: its own ring of 32-token stages, filled by its own
//    16-byte asynchronous copies of whole granules (16 rows, 1152 bytes), and no
//    barrier between warps until the end. (Bulk copies, one lane each, cost about 12
//    instructions a copy: their operands are warp-uniform.) What a tile is -- its pages,
//    its valid tokens, its addresses -- one further warp, the walker, works out for all
//    of them, a lane for each (every warp walking for itself, with bulk copies: 146 us
//    for 32 rows of 16384 tokens, against 131 then);
//  - K: lane (r, q) of a quad takes bytes 16q..16q+15 of row r as one 16-byte load:
//    the contraction's order is free, so these are its A fragments of all eight
//    k-steps (Q is read in the same order), within two blocks, two scales;
//  - V: a lane takes bytes 8r..8r+7 (one block) of its four tokens; two shifts and
//    two bit selects interleave the nibbles of a token pair so that one
//    conversion gives the (token, token + 1) pair of a V^T fragment;
//  - the weights' reference, set 5 octaves below the greatest score, is raised only when a
//    sum of weights passes 2^15 (one warp vote per stage; the weights, at most 2^15, meet V
//    as f16, which keeps 11 bits of each where V has 6 and 2^-24 of the reference, 2^-29 of
//    the greatest weight, as its smallest step; their sums are fp32), so a stage usually
//    needs no shuffle and no rescaling of O;
//  - no branch inside a stage: both granules are always computed, word by word in
//    turn, and what a half that was not copied holds is masked (131 -> 119 us for 32
//    rows of 16384 tokens).
// Long rows stream at 90 % of the copy rate (32 rows of 16384 tokens, 8 kv heads:
// 117 us, floor 89). A call of 32 rows of 1024..8192 takes 42 us, floor 22.7: 2 us
// until the schedule stands, 2 until the first tile, 28 of stream, 4 in which the
// warps end one after another, 2 for the pieces of a CTA and 4 for units that CTAs
// share. Measured and not kept: 16 streaming warps with a register split (more
// instructions: 42.0 -> 45.4 us), shares weighted by scheduler (115 -> 124 us), the walk
// and the end as functions of their own (42.1 -> 45.5 us). Not built: tiles handed to
// whichever warp has room, against the 4 us in which warps end one after another.
// 9 to 16 rows a unit (three warps a scheduler, 168 registers, 16 to 18 bytes of spill) are
// bound by latency, no pipe being full: 16 rows of 1000..20000, 4 query tokens: 74.7 us,
// floor 28.9, issue 42 %, ALU 32 %.
// How tiles are walked, cut and merged stands in stream_split.cuh.
#include "stream_split.cuh"

namespace da {
namespace {

// Four bytes of e2m1 pairs (low nibble first) as four f16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t f4_mul2(uint32_t x, uint32_t y) {
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&y));
  return *reinterpret_cast<const uint32_t *>(&r);
}
// A pair times the low or the high half of `s`.
__device__ __forceinline__ uint32_t f4_scale(uint32_t x, uint32_t s, int high) {
  const __half2 h = *reinterpret_cast<const __half2 *>(&s);
  const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&x), high ? __high2half2(h) : __low2half2(h));
  return *reinterpret_cast<const uint32_t *>(&r);
}

struct Fp4Format {
  static constexpr int kT = 32;
  static constexpr int kGranBytes = 1152;  // 16 x 64 code bytes, then 16 x 8 scale bytes
  static constexpr int kScaleOff = 1024;
  static constexpr int kSideBytes = 0;
  static constexpr bool kHeadScales = true;
  static constexpr bool kCareful = false;
  static constexpr bool kBlockScales = false;
  static constexpr bool kFoldsV = false;
  static constexpr int kWarps(int nt) { return nt == 1 ? 15 : 11; }  // with the walker four (three) a scheduler
  static constexpr int kStages(int) { return 3; }
  // Q^T fragments: registers for up to eight rows; for sixteen, whose O takes 64
  // registers a thread, shared memory (16 bytes a lane and k-step): 16 rows x 4 query
  // tokens 89.6 -> 80.9 us (four warps a scheduler instead, in 128 registers: 118 us)
  static constexpr bool kQShared(int nt) { return nt == 2; }

  const uint8_t *k_lane, *v_lane;
  int lane, k_off, ks_off, v_off, vs_off;  // this lane in a granule of K, and of V
  __device__ __forceinline__ Fp4Format(const StreamParams &fp, int l) : lane(l) {
    const int q4 = l & 3, r8 = l >> 2;
    k_lane = fp.k + l * 16;
    v_lane = fp.v + l * 16;
    k_off = r8 * 64 + q4 * 16, ks_off = kScaleOff + r8 * 8 + q4 * 2;
    v_off = q4 * 128 + r8 * 8, vs_off = kScaleOff + q4 * 16 + r8;
  }
  // 16 bytes a lane, 72 lanes' worth a granule
  __device__ __forceinline__ void copy_one(uint32_t dst, const uint8_t *src) const {
    cp_async_16(dst, src);
    cp_async_16(dst + 512, src + 512);
    if (lane < 8) cp_async_16(dst + 1024, src + 1024);
  }
  __device__ __forceinline__ uint32_t lane_at() const { return lane * 16; }
  __device__ __forceinline__ void copy(uint32_t k, uint32_t v, int64_t off, uint8_t *, int) const {
    copy_one(k, k_lane + off);
    copy_one(v, v_lane + off);
  }
  template <int NT>
  __device__ __forceinline__ void scores(const uint8_t *stage, const uint8_t *, const uint32_t (&qf)[NT][8][2],
                                         const uint4 *qs, float (&s)[NT][2][4]) const {
    uint4 ra[2], rb[2];
    uint32_t sa[2], sb[2];
#pragma unroll
    for (int gi = 0; gi < 2; ++gi) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) s[nt][gi][0] = s[nt][gi][1] = s[nt][gi][2] = s[nt][gi][3] = 0.f;
      const uint8_t *gk = stage + gi * kGranBytes;
      ra[gi] = *reinterpret_cast<const uint4 *>(gk + k_off);
      rb[gi] = *reinterpret_cast<const uint4 *>(gk + k_off + 512);
      sa[gi] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(gk + ks_off));
      sb[gi] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(gk + ks_off + 64));
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // word c: k-steps 2c and 2c + 1, block c / 2 of the lane's two
      uint32_t q[2][NT][2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (kQShared(NT)) {
          const uint4 v = qs[(2 * c + k) * 32];
          q[k][0][0] = v.x;
          q[k][0][1] = v.y;
          q[k][NT - 1][0] = v.z;
          q[k][NT - 1][1] = v.w;
        } else {
          q[k][0][0] = qf[0][2 * c + k][0];
          q[k][0][1] = qf[0][2 * c + k][1];
        }
      }
#pragma unroll
      for (int gi = 0; gi < 2; ++gi) {
        uint32_t fa[4], fb[4];
        e2m1x8_to_f16(c == 0 ? ra[gi].x : c == 1 ? ra[gi].y : c == 2 ? ra[gi].z : ra[gi].w, fa);
        e2m1x8_to_f16(c == 0 ? rb[gi].x : c == 1 ? rb[gi].y : c == 2 ? rb[gi].z : rb[gi].w, fb);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t a0 = f4_scale(fa[2 * k], sa[gi], c >> 1), a2 = f4_scale(fa[2 * k + 1], sa[gi], c >> 1);
          const uint32_t a1 = f4_scale(fb[2 * k], sb[gi], c >> 1), a3 = f4_scale(fb[2 * k + 1], sb[gi], c >> 1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_f16_16816(s[nt][gi], a0, a1, a2, a3, q[k][nt][0], q[k][nt][1]);
        }
      }
    }
  }
  // a masked token's value row may hold any scale (NaN; its codes are finite): zero them
  __device__ __forceinline__ void drop(uint8_t *stage, uint8_t *, uint32_t valid) const {
    if (!((valid >> lane) & 1u))
      *reinterpret_cast<uint2 *>(stage + (2 + (lane >> 4)) * kGranBytes + kScaleOff + (lane & 15) * 8) =
          make_uint2(0u, 0u);
  }
  template <int NT>
  __device__ __forceinline__ void values(const uint8_t *v, const float (&)[2], bool, const uint32_t (&pb)[NT][2][2],
                                         float (&oacc)[NT][8][4]) const {
#pragma unroll
    for (int gi = 0; gi < 2; ++gi) {
      const uint8_t *gv = v + gi * kGranBytes;
      // tokens 2 q4, 2 q4 + 1 and the same + 8: one block (8 bytes) of each, and its scale
      uint2 w[4];
      uint32_t sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = (k & 1) + 8 * (k >> 1);
        w[k] = *reinterpret_cast<const uint2 *>(gv + v_off + t * 64);
        sc[k] = gv[vs_off + t * 8];
      }
      const uint32_t s01 = e4m3x2_to_f16x2((uint16_t)prmt(sc[0], sc[1], 0x0040));
      const uint32_t s89 = e4m3x2_to_f16x2((uint16_t)prmt(sc[2], sc[3], 0x0040));
      constexpr uint32_t kLow = 0x0F0F0F0Fu;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t a = c ? w[0].y : w[0].x, bq = c ? w[1].y : w[1].x;
        const uint32_t d = c ? w[2].y : w[2].x, e = c ? w[3].y : w[3].x;
        uint32_t e01[4], o01[4], e89[4], o89[4];  // even and odd dims of the two token pairs
        e2m1x8_to_f16((a & kLow) | ((bq << 4) & ~kLow), e01);
        e2m1x8_to_f16(((a >> 4) & kLow) | (bq & ~kLow), o01);
        e2m1x8_to_f16((d & kLow) | ((e << 4) & ~kLow), e89);
        e2m1x8_to_f16(((d >> 4) & kLow) | (e & ~kLow), o89);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t a0 = f4_mul2(e01[k], s01), a1 = f4_mul2(o01[k], s01);
          const uint32_t a2 = f4_mul2(e89[k], s89), a3 = f4_mul2(o89[k], s89);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16_16816(oacc[nt][4 * c + k], a0, a1, a2, a3, pb[nt][gi][0], pb[nt][gi][1]);
        }
      }
    }
  }
};

template <int NT, int MOD>
__global__ void __launch_bounds__(StreamLayout<Fp4Format, NT>::kThreads, 1)
    fp4_split_kernel(const StreamParams fp) {
  wait_for_previous_kernel();
  let_next_kernel_start();
  stream_split<Fp4Format, NT, MOD>(fp);
}

template <int NT, int MOD>
cudaError_t f4_attr() {
  return cudaFuncSetAttribute(fp4_split_kernel<NT, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              StreamLayout<Fp4Format, NT>::kTotal);
}

}  // namespace

int fp4_tile() { return Fp4Format::kT; }
int fp4_warps(int group) { return group <= 8 ? Fp4Format::kWarps(1) : Fp4Format::kWarps(2); }

cudaError_t fp4_prepare() {
  cudaError_t e;
  if ((e = f4_attr<1, 0>()) != cudaSuccess) return e;
  if ((e = f4_attr<1, 1>()) != cudaSuccess) return e;
  if ((e = f4_attr<1, 2>()) != cudaSuccess) return e;
  if ((e = f4_attr<2, 0>()) != cudaSuccess) return e;
  if ((e = f4_attr<2, 1>()) != cudaSuccess) return e;
  return f4_attr<2, 2>();
}

cudaError_t launch_fp4(const StreamParams &p, int ctas, cudaStream_t stream) {
  const int mod = gqa_mod(p.g);
#define DA_F4(NT, M) \
  return launch_dependent(fp4_split_kernel<NT, M>, (unsigned)ctas, StreamLayout<Fp4Format, NT>::kThreads, StreamLayout<Fp4Format, NT>::kTotal, stream, p)
  if (p.g.group <= 8) {
    if (mod == 0) DA_F4(1, 0);
    else if (mod == 1) DA_F4(1, 1);
    else DA_F4(1, 2);
  } else {
    if (mod == 0) DA_F4(2, 0);
    else if (mod == 1) DA_F4(2, 1);
    else DA_F4(2, 2);
  }
#undef DA_F4
}

}  // namespace da
