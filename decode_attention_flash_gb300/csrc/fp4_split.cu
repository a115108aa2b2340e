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
// turn into f16. The e2m1 conversion runs at half rate (2 cycles a warp for a
// pair per lane, measured), an m16n8k16 takes 8.5 cycles of a scheduler, and every
// pair takes a multiply by its block's scale: about 320 issue cycles per 16
// tokens and scheduler, against 392 that the measured copy bandwidth leaves. So
// the kernel is laid out to add as little as possible to that:
//  - every warp streams alone: its own ring of 32-token stages, filled by
//    untiled bulk copies of whole granules (16 rows, 1152 bytes; no tensor map),
//    its own barriers, no producer warp and no barrier between warps until the end;
//  - K: lane (r, q) of a quad takes bytes 16q..16q+15 of row r as one 16-byte load:
//    the contraction's order is free, so these are its A fragments of all eight
//    k-steps (Q is read in the same order), within two blocks, two scales;
//  - V: a lane takes bytes 8r..8r+7 (one block) of its four tokens; two shifts and
//    two bit selects interleave the nibbles of a token pair so that one
//    conversion gives the (token, token + 1) pair of a V^T fragment;
//  - the running maximum is only raised when a score passes it by 2^8 (one
//    warp vote per stage; P <= 2^8 in f16, sums in fp32), so a stage usually
//    needs no shuffle and no rescaling of O.
//
// The split. As in gqa_split.cuh the tiles of all (row, kv head) units are laid
// end to end and cut into equal ranges, one per CTA; a CTA's range is cut again
// into one range per warp. A unit inside one warp's range is written from its
// registers; pieces of a unit shared by warps meet in shared memory after the
// stream, and pieces shared by CTAs in global memory (counted and merged as in
// gqa_split.cuh, without any CTA waiting for another).
#include "gqa_split.cuh"

namespace da {
namespace {

constexpr int kT = 32;               // tokens per stage
constexpr int kGran = 16;            // rows of a granule
constexpr int kGranBytes = 1152;     // 16 x 64 code bytes, then 16 x 8 scale bytes
constexpr int kScaleOff = 1024;
constexpr int kStageBytes = 2 * (kT / kGran) * kGranBytes;  // K granules, then V granules
constexpr float kRaise = 8.f;        // log2 headroom of the running maximum

template <int NT>
struct F4 {
  static constexpr int kWarps = NT == 1 ? 16 : 12;
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kStages = NT == 1 ? 3 : 4;
  static constexpr int kRingBytes = kStages * kStageBytes;       // one warp's ring
  static constexpr int oFull = kWarps * kRingBytes;
  static constexpr int oMeta = oFull + 8 * kWarps * kStages + 16;  // + the test stall's barrier
  static constexpr int oStat = oMeta + 32 * kWarps * kStages;    // [warp][tail|head][m|l][16]
  static constexpr int oScan = oStat + kWarps * 64 * 4;
  static constexpr int oFlags = oScan + 16 * 4;                  // 40 ints, as in gqa_split.cuh
  static constexpr int oStart = oFlags + 40 * 4;                 // [warp] int64 first tile of the start unit
  static constexpr int oStartU = oStart + kWarps * 8;            // [warp] start unit
  static constexpr int oLead = oStartU + kWarps * 4;             // [warp + 1] groups (see below)
  static constexpr int kTotal = oLead + (kWarps + 1) * 16 + 128;
  static_assert(kRingBytes >= NT * 8 * kD * 4, "a warp's ring holds its piece after the stream");
  static_assert(kRingBytes % 128 == 0 && oFull % 16 == 0 && oMeta % 16 == 0 && oStart % 8 == 0, "alignment");
};

struct __align__(16) F4Meta {
  uint32_t valid;   // bit t: token t of the stage is a valid position
  int32_t unit;
  int32_t flags;    // kFirst, kLast, kFull; kUnitStart / kUnitEnd: the unit's first / last tile
  int32_t nval;     // the row's length minus the stage's first position
  int32_t pos0;     // the stage's first position in the row
  int32_t warps;    // first and last warp of this CTA holding the unit (bits 0-7, 8-15),
                    // whether the last one goes on to another unit (bit 16), and
                    // whether the unit reaches other CTAs (bit 17)
  int32_t c_first, n_seg;
};
static_assert(sizeof(F4Meta) == 32, "layout");
constexpr int32_t kUnitStart = 8, kUnitEnd = 16;

__device__ __forceinline__ UnitInfo f4_unit_info(const GqaParams &p, int u, uint32_t &err) {
  UnitInfo x = unit_info(p, u, err);
  x.tiles = p.sparse_block_size > 0 ? x.tiles * (kTile / kT) : (x.n_valid + kT - 1) / kT;
  return x;
}

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

template <int NT, int MOD>
__global__ void __launch_bounds__(F4<NT>::kThreads, 1)
    fp4_split_kernel(const Fp4Params fp) {
  using C = F4<NT>;
  constexpr int W = C::kWarps, S = C::kStages;
  const GqaParams &p = fp.g;
  extern __shared__ uint8_t f4_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(f4_smem) + 127) & ~uintptr_t(127));
  float *stat_all = reinterpret_cast<float *>(smem + C::oStat);
  int *scan = reinterpret_cast<int *>(smem + C::oScan);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + C::oFlags);
  // flags: [0] a wait gave up; [12] merges owed, [13] scratch, [24..31] those
  // merges (record_merge of gqa_split.cuh)
  int64_t *wstart = reinterpret_cast<int64_t *>(smem + C::oStart);
  int *wunit = reinterpret_cast<int *>(smem + C::oStartU);
  // Groups: the pieces of one unit inside this CTA, warps a..b. Entry a, written
  // by warp a (entry W when the piece is warp 0's head alone): unit (-1: none); b,
  // with bit 8 when warp b goes on to another unit; c_first; n_seg (0: the whole
  // unit is in this CTA).
  int4 *lead = reinterpret_cast<int4 *>(smem + C::oLead);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  const int U = p.batch * p.num_kv_heads;
  const int cta = blockIdx.x;
  uint32_t dev_err = 0;

  if (threadIdx.x == 0) {
    if (p.paged) prefetch_share_l2(p.block_table, (int64_t)p.batch * p.max_pages * 4);
    flags[0] = 0;
    flags[12] = 0;
  }
  if (threadIdx.x <= W) lead[threadIdx.x] = make_int4(-1, 0, 0, 0);

  // ---- the schedule (see gqa_split.cuh): this CTA's range, then this warp's
  const int per = (U + C::kThreads - 1) / C::kThreads;
  const int u_beg = min(U, (int)threadIdx.x * per), u_end = min(U, u_beg + per);
  int local = 0;
  for (int u = u_beg; u < u_end; ++u) local += f4_unit_info(p, u, dev_err).tiles;
  int T32 = 0;
  const int incl = block_inclusive_scan(local, scan, &T32);
  const int64_t T = T32;
  const int CTAS = (int)(T < (int64_t)gridDim.x ? T : (int64_t)gridDim.x);
  const int64_t lo = cta < CTAS ? (int64_t)cta * T / CTAS : 0;
  const int64_t hi = cta < CTAS ? (int64_t)(cta + 1) * T / CTAS : 0;
  const int n_cta = (int)(hi - lo);
  const int owner_of_tail = CTAS > 0 ? CTAS - 1 : 0;
  {
    int64_t Pu = incl - local;
    uint32_t ignored = 0;
    for (int u = u_beg; u < u_end; ++u) {
      const UnitInfo x = f4_unit_info(p, u, ignored);
      const int t_u = x.tiles;
      if (t_u > 0 && Pu < hi && Pu + t_u > lo) {
        // warps whose range starts in this unit
        const int w0 = Pu <= lo ? 0 : cta_of(Pu - lo, n_cta, W);
        for (int w = w0; w < W; ++w) {
          const int64_t s = lo + (int64_t)w * n_cta / W;
          if (s >= Pu + t_u) break;
          if (s >= Pu) {
            wstart[w] = Pu;
            wunit[w] = u;
          }
        }
      }
      if (t_u == 0 && ((Pu >= lo && Pu < hi) || (Pu >= T && cta == owner_of_tail))) {
        const int64_t row0 = (int64_t)x.b * p.num_q_heads + x.h * G;
        for (int e = 0; e < G * kD; ++e) p.out[row0 * kD + e] = __float2bfloat16(0.f);
        if (p.lse)
          for (int g = 0; g < G; ++g) p.lse[row0 + g] = neg_inf();
      }
      Pu += t_u;
    }
  }
  if (n_cta <= 0) {
    if (dev_err) atomicOr(p.err, dev_err);
    return;
  }
  uint8_t *ring = smem + (size_t)warp * C::kRingBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::oFull) + warp * S;
  uint64_t *stall_bar = reinterpret_cast<uint64_t *>(smem + C::oFull) + W * S;  // nothing arrives on it
  F4Meta *meta = reinterpret_cast<F4Meta *>(smem + C::oMeta) + warp * S;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
    if (warp == 0) mbar_init(stall_bar, 1);
    fence_mbar_init();
  }
  __syncthreads();

  const int64_t wlo = lo + (int64_t)warp * n_cta / W, whi = lo + (int64_t)(warp + 1) * n_cta / W;
  const int ntiles = (int)(whi - wlo);
  bool ok = true;
  int issued = 0;

  if (ntiles == 0) stat_all[warp * 64 + lane] = 0.f;  // no piece: weight 0 in the sums below
  if (ntiles > 0) {
    // ------------------------------------------------------------ the walker of this warp's tiles
    const int q4 = lane & 3, r8 = lane >> 2;
    const int P = p.page_size;
    const bool sparse = p.sparse_block_size > 0;
    // entries (pages or listed blocks) of `tpe` tiles each; pages of 16 tokens: two per tile
    const int tpe = sparse ? p.sparse_block_size / kT : (p.paged ? (P >= kT ? P / kT : 1) : 1);
    const bool two_pages = p.paged && P < kT;
    const bool has_ids = p.paged || sparse;
    const int64_t gran_unit = p.paged ? P / kGran : p.cache_len / kGran;  // granules per (page | row, head)
    int u = wunit[warp], j = (int)(wlo - wstart[warp]);
    int64_t Pu = wstart[warp];
    UnitInfo x;
    int ent = 0, sub = 0, nent = 0;     // current entry, tile inside it, entries of the unit
    int wbase = 0, wid = -1, wnext = -1;  // 32 entry ids from wbase (one per lane), and the next 32
    int winfo = 0, c_first = 0, n_seg = 0;
    auto load_id = [&](int e) -> int {
      if (e >= nent) return -1;
      if (sparse)
        return e < x.nbp ? __ldg(p.kv_idx + (int64_t)x.trow * p.max_sparse_blocks + e)
                         : __ldg(p.kv_full_idx + (int64_t)x.trow * p.max_sparse_blocks + e - x.nbp);
      return __ldg(p.block_table + (int64_t)x.b * p.max_pages + e);
    };
    auto enter_unit = [&]() {  // x holds unit u's info; tile j of it comes next
      if (has_ids) {
        if (two_pages) {
          ent = 2 * j;
          sub = 0;
        } else {
          ent = j / tpe;
          sub = j - ent * tpe;
        }
        nent = sparse ? x.tiles / tpe : (x.n_valid + P - 1) / P;
        wbase = ent;
        wid = load_id(ent + lane);
        wnext = load_id(ent + 32 + lane);
      }
      const int64_t a = Pu < lo ? lo : Pu, b = Pu + x.tiles > hi ? hi : Pu + x.tiles;
      const bool outside = Pu < lo || Pu + x.tiles > hi;
      const int bw = cta_of(b - 1 - lo, n_cta, W);
      const bool goes_on = b < lo + (int64_t)(bw + 1) * n_cta / W;
      winfo = cta_of(a - lo, n_cta, W) | (bw << 8) | (goes_on ? 1 << 16 : 0) | (outside ? 1 << 17 : 0);
      c_first = outside ? cta_of(Pu, T, CTAS) : cta;
      n_seg = outside ? cta_of(Pu + x.tiles - 1, T, CTAS) - c_first + 1 : 0;
    };
    x = f4_unit_info(p, u, dev_err);
    enter_unit();

    auto issue = [&](int i) {
      const int st = i % S;
      const int tok0 = j * kT;
      int pos0 = tok0;
      int64_t gr0 = -1, gr1 = -1;  // granules of the stage's two halves
      uint32_t valid = 0;
      bool full_blk = false;
      if (!has_ids) {
        gr0 = (int64_t)u * gran_unit + tok0 / kGran;
        gr1 = gr0 + 1;
        valid = (uint32_t)low_bits(min(x.n_valid - tok0, kT));
      } else {
        if (ent >= wbase + 32) {
          wid = wnext;
          wbase += 32;
          wnext = load_id(wbase + 32 + lane);
        }
        if (two_pages) {
          const int id0 = __shfl_sync(0xffffffffu, wid, ent - wbase);
          const int id1 = __shfl_sync(0xffffffffu, wid, ent + 1 - wbase);  // wbase is even: same window
          const bool in1 = tok0 + kGran < x.n_valid;
          const bool ok0 = id0 >= 0 && id0 < p.num_pages, ok1 = in1 && id1 >= 0 && id1 < p.num_pages;
          if (!ok0 || (in1 && !ok1)) dev_err |= DA_DEVERR_PAGE_INDEX;
          const uint32_t v = (uint32_t)low_bits(min(x.n_valid - tok0, kT));
          if (ok0) {
            gr0 = (int64_t)id0 * p.num_kv_heads + x.h;
            valid |= v & 0xFFFFu;
          }
          if (ok1) {
            gr1 = (int64_t)id1 * p.num_kv_heads + x.h;
            valid |= v & 0xFFFF0000u;
          }
          ent += 2;
        } else {
          const int id = __shfl_sync(0xffffffffu, wid, ent - wbase);
          if (sparse) {
            full_blk = ent >= x.nbp;
            if (id < 0 || (int64_t)id * p.sparse_block_size >= p.cache_len) {
              dev_err |= DA_DEVERR_SPARSE_INDEX;
            } else {
              pos0 = id * p.sparse_block_size + sub * kT;
              valid = (uint32_t)low_bits(min(min(x.n_valid - pos0, kT), p.cache_len - pos0));
              gr0 = (int64_t)u * gran_unit + pos0 / kGran;
            }
          } else if (id < 0 || id >= p.num_pages) {
            dev_err |= DA_DEVERR_PAGE_INDEX;
          } else {
            valid = (uint32_t)low_bits(min(x.n_valid - tok0, kT));
            gr0 = ((int64_t)id * p.num_kv_heads + x.h) * gran_unit + sub * (kT / kGran);
          }
          gr1 = gr0 >= 0 ? gr0 + 1 : -1;
          if (++sub == tpe) {
            sub = 0;
            ++ent;
          }
        }
      }
      const bool v0 = (valid & 0xFFFFu) != 0, v1 = (valid >> 16) != 0;  // halves with no token are not read
      if (lane == 0) {
        F4Meta m;
        m.valid = valid;
        m.unit = u;
        m.flags = (i == 0 || j == 0 ? kFirst : 0) | (i + 1 == ntiles || j + 1 == x.tiles ? kLast : 0) |
                  (full_blk ? kFull : 0) | (j == 0 ? kUnitStart : 0) | (j + 1 == x.tiles ? kUnitEnd : 0);
        m.nval = x.n_valid - pos0;
        m.pos0 = pos0;
        m.warps = winfo;
        m.c_first = c_first;
        m.n_seg = n_seg;
        meta[st] = m;
        mbar_arrive_expect_tx(&full[st], (v0 ? 2u * kGranBytes : 0u) + (v1 ? 2u * kGranBytes : 0u));
      }
      __syncwarp();
      // lane 0, 1: K and V of the first half; 2, 3: of the second
      if (lane < 4) {
        const int64_t gr = lane < 2 ? gr0 : gr1;
        if (lane < 2 ? v0 : v1)
          bulk_copy_g2s(ring + st * kStageBytes + ((lane & 1) * 2 + (lane >> 1)) * kGranBytes,
                        (lane & 1 ? fp.v : fp.k) + gr * kGranBytes, kGranBytes, &full[st]);
      }
      issued = i + 1;
      if (++j == x.tiles && i + 1 < ntiles) {
        Pu += x.tiles;
        do {
          ++u;
          x = f4_unit_info(p, u < U ? u : U - 1, dev_err);
        } while (u < U && x.tiles == 0);
        j = 0;
        enter_unit();
      }
    };
    for (int i = 0; i < S && i < ntiles; ++i) issue(i);

    // ------------------------------------------------------------ the stream
    uint32_t qf[NT][8][2];
    float oacc[NT][8][4];
    float m_run[NT][2], l_part[NT][2];
    float sscale = p.score_scale, vmul = 1.f;
    const bool softcap = MOD >= 1 && p.softcap_l2 > 0.f;
    const bool mods = MOD == 2 && (p.mask_window != nullptr || p.alibi_slopes != nullptr);
    int trow[NT][2];
    uint32_t mword[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        trow[nt][e] = (nt * 8 + 2 * q4 + e) % p.q_len;
        mword[nt][e] = (2u << trow[nt][e]) - 1u;
      }
    bool from_start = false;  // the segment holds its unit's first tile
    // (the test stall of GqaParams, in the warp that always has a tile: the timeout path
    // runs as after a real failure)
    if (p.test_stall_ns != 0 && warp == W - 1) ok = warp_wait(stall_bar, 0u, p.test_stall_ns);
    for (int i = 0; ok && i < ntiles; ++i) {
      const int st = i % S;
      if (!warp_wait(&full[st], (i / S) & 1, kWaitLimitNs)) {
        ok = false;
        break;
      }
      const F4Meta m = meta[st];
      const uint8_t *stage = ring + st * kStageBytes;
      if (m.flags & kFirst) {
        from_start = (m.flags & kUnitStart) != 0;
        const int b = m.unit / p.num_kv_heads, h = m.unit - b * p.num_kv_heads;
        // Q^T fragments straight from global memory: k-step s of lane (r8, q4) is
        // dims 32 q4 + 4s .. + 3 of row r8 (the bytes a lane has of a K row). The
        // rows are scaled by one power of two into f16's range (gqa_split.cuh).
        uint2 qw[NT][8];
        float amax = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int g = nt * 8 + r8;
          const uint4 *src = reinterpret_cast<const uint4 *>(
              p.q + ((int64_t)b * p.num_q_heads + h * G + (g < G ? g : 0)) * kD + 32 * q4);
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint4 v = __ldg(src + s);
            qw[nt][2 * s] = make_uint2(v.x, v.y);
            qw[nt][2 * s + 1] = make_uint2(v.z, v.w);
          }
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            if (g >= G) qw[nt][s] = make_uint2(0u, 0u);
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qw[nt][s].x << 16)),
                                     fabsf(__uint_as_float(qw[nt][s].x & 0xFFFF0000u))));
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(qw[nt][s].y << 16)),
                                     fabsf(__uint_as_float(qw[nt][s].y & 0xFFFF0000u))));
          }
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int qexp = q_exponent(amax);
        const float q2 = pow2f(qexp);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            qf[nt][s][0] = bf16x2_to_f16x2(qw[nt][s].x, q2);
            qf[nt][s][1] = bf16x2_to_f16x2(qw[nt][s].y, q2);
          }
        sscale = p.score_scale * p.k_scale[h] * pow2f(-qexp);
        vmul = p.v_scale[h];
        if (MOD >= 1 && p.spec_mask != nullptr) {
          const uint32_t *mrow = p.spec_mask + (size_t)b * p.q_len;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) mword[nt][e] = mrow[trow[nt][e]];
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e) oacc[nt][mt][e] = 0.f;
          m_run[nt][0] = m_run[nt][1] = neg_inf();
          l_part[nt][0] = l_part[nt][1] = 0.f;
        }
      }
      if (m.valid != 0) {
        // ---------------- S^T = K Q^T, two granules of 16 tokens
        float s[NT][2][4];
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][gi][0] = s[nt][gi][1] = s[nt][gi][2] = s[nt][gi][3] = 0.f;
          if (((m.valid >> (16 * gi)) & 0xFFFFu) == 0) continue;
          const uint8_t *gk = stage + gi * kGranBytes;
          const uint4 ra = *reinterpret_cast<const uint4 *>(gk + r8 * 64 + q4 * 16);
          const uint4 rb = *reinterpret_cast<const uint4 *>(gk + (r8 + 8) * 64 + q4 * 16);
          const uint32_t sa = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(gk + kScaleOff + r8 * 8 + q4 * 2));
          const uint32_t sb =
              e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(gk + kScaleOff + (r8 + 8) * 8 + q4 * 2));
          const uint32_t wa[4] = {ra.x, ra.y, ra.z, ra.w}, wb[4] = {rb.x, rb.y, rb.z, rb.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {  // word c: k-steps 2c and 2c + 1, block c / 2 of the lane's two
            uint32_t fa[4], fb[4];
            e2m1x8_to_f16(wa[c], fa);
            e2m1x8_to_f16(wb[c], fb);
            const uint32_t xa = prmt(sa, 0, c < 2 ? 0x1010 : 0x3232), xb = prmt(sb, 0, c < 2 ? 0x1010 : 0x3232);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t a0 = f4_mul2(fa[2 * k], xa), a2 = f4_mul2(fa[2 * k + 1], xa);
              const uint32_t a1 = f4_mul2(fb[2 * k], xb), a3 = f4_mul2(fb[2 * k + 1], xb);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(s[nt][gi], a0, a1, a2, a3, qf[nt][2 * c + k][0], qf[nt][2 * c + k][1]);
            }
          }
        }
        // ---------------- masks and the online softmax (log2 units)
        const bool part = m.valid != 0xFFFFFFFFu;
        if (MOD >= 1) {  // scores become x = score * log2 e here; masked ones -inf
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int t = r8 + 8 * k;  // token of the stage
                float v = s[nt][k >> 1][(k & 1) * 2 + e] * sscale;
                if (softcap) v = cap_tanh(v, p.softcap_l2, p.softcap_k);
                const int jnew = t - (m.nval - p.q_len);
                bool keep = (m.valid >> t) & 1u;
                keep = keep && (jnew < 0 || ((mword[nt][e] >> min(jnew, 31)) & 1u));
                if (mods) {
                  const int row = min(nt * 8 + 2 * q4 + e, G - 1);
                  const int hq = (m.unit % p.num_kv_heads) * (G / p.q_len) + row / p.q_len;
                  const int kv = m.pos0 + t, qpos = m.nval + m.pos0 - p.q_len + trow[nt][e];
                  if (p.mask_window && !(m.flags & kFull)) {
                    const int w = __ldg(p.mask_window + hq), sk = p.mask_sink ? __ldg(p.mask_sink + hq) : 0;
                    keep = keep && (kv < sk || w < 0 || kv > qpos - w);
                  }
                  if (p.alibi_slopes)
                    v += __ldg(p.alibi_slopes + hq) * 1.4426950408889634f * (float)(kv - qpos);
                }
                s[nt][k >> 1][(k & 1) * 2 + e] = keep ? v : neg_inf();
              }
        }
        const float f = MOD >= 1 ? 1.f : sscale;
        float y[NT][2][4];
        bool raise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mu = m_run[nt][e] == neg_inf() ? 0.f : m_run[nt][e];
            raise = raise || m_run[nt][e] == neg_inf();
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float v = MOD >= 1 ? s[nt][k >> 1][(k & 1) * 2 + e] - mu
                                 : fmaf(s[nt][k >> 1][(k & 1) * 2 + e], f, -mu);
              if (MOD == 0 && part) v = (m.valid >> (r8 + 8 * k)) & 1u ? v : neg_inf();
              y[nt][e][k] = v;
              raise = raise || v > kRaise;
            }
          }
        if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float mu = m_run[nt][e] == neg_inf() ? 0.f : m_run[nt][e];
              float t = fmaxf(fmaxf(y[nt][e][0], y[nt][e][1]), fmaxf(y[nt][e][2], y[nt][e][3])) + mu;
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              const float m_new = fmaxf(m_run[nt][e], t);
              const float mn = m_new == neg_inf() ? 0.f : m_new;
              alpha[e] = ex2(m_run[nt][e] - mn);
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // (masked scores stay -inf)
                const float v = s[nt][k >> 1][(k & 1) * 2 + e];
                y[nt][e][k] = y[nt][e][k] == neg_inf() ? neg_inf() : MOD >= 1 ? v - mn : fmaf(v, f, -mn);
              }
              l_part[nt][e] *= alpha[e];
              m_run[nt][e] = m_new;
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              oacc[nt][mt][0] *= alpha[0];
              oacc[nt][mt][1] *= alpha[1];
              oacc[nt][mt][2] *= alpha[0];
              oacc[nt][mt][3] *= alpha[1];
            }
          }
        }
        // P^T fragments: weights as f16 (at most 2^8), the row sum from the fp32 ones
        uint32_t pb[NT][2][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int k = 0; k < 4; ++k) y[nt][e][k] = ex2(y[nt][e][k]);
            l_part[nt][e] += (y[nt][e][0] + y[nt][e][1]) + (y[nt][e][2] + y[nt][e][3]);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
            pb[nt][k >> 1][k & 1] = movmatrix_trans(pack_f16(y[nt][0][k], y[nt][1][k]));
        }
        // ---------------- O^T += V^T P^T
#pragma unroll
        for (int gi = 0; gi < 2; ++gi) {
          const uint32_t vb = (m.valid >> (16 * gi)) & 0xFFFFu;
          if (vb == 0) continue;
          const uint8_t *gv = stage + (2 + gi) * kGranBytes;
          // tokens 2 q4, 2 q4 + 1 and the same + 8: one block (8 bytes) of each, and its scale
          uint2 w[4];
          uint32_t sc[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int t = 2 * q4 + (k & 1) + 8 * (k >> 1);
            w[k] = *reinterpret_cast<const uint2 *>(gv + t * 64 + r8 * 8);
            sc[k] = gv[kScaleOff + t * 8 + r8];
          }
          uint32_t s01 = e4m3x2_to_f16x2((uint16_t)(sc[0] | (sc[1] << 8)));
          uint32_t s89 = e4m3x2_to_f16x2((uint16_t)(sc[2] | (sc[3] << 8)));
          if (vb != 0xFFFFu) {  // a masked token's row may hold any scale (codes are finite)
            s01 &= lo16_mask((vb >> (2 * q4)) & 1u, (vb >> (2 * q4 + 1)) & 1u);
            s89 &= lo16_mask((vb >> (2 * q4 + 8)) & 1u, (vb >> (2 * q4 + 9)) & 1u);
          }
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
      __syncwarp();  // every lane has read the stage
      if (i + S < ntiles) issue(i + S);
      if (!(m.flags & kLast)) continue;
      // ---------------- the segment ends. Row sums, then: a unit held by this
      // segment alone goes out from the registers; another segment's (m, l, O) to
      // this warp's ring when it is the warp's last, else to its global slot
      const bool whole = from_start && (m.flags & kUnitEnd);
      const bool tail = i + 1 == ntiles;
      const int b = m.unit / p.num_kv_heads, h = m.unit - b * p.num_kv_heads;
      float *piece = nullptr;
      if (!whole) {
        float *stat = stat_all + (warp * 2 + (tail ? 0 : 1)) * 32;
        piece = tail ? reinterpret_cast<float *>(ring)
                     : fp.o_head + ((int64_t)cta * W + warp) * G * kD;
        // the unit's first warp here names the group (a head alone is warp 0's)
        if (lane == 0 && (m.warps & 255) == warp)
          lead[tail ? warp : W] = make_int4(m.unit, (m.warps >> 8) & 0x1FF, m.c_first, (m.warps >> 17) ? m.n_seg : 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = l_part[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (r8 == 0) {
              stat[nt * 8 + 2 * q4 + e] = m_run[nt][e] == neg_inf() ? 0.f : m_run[nt][e];
              stat[16 + nt * 8 + 2 * q4 + e] = l;
            }
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int g = nt * 8 + 2 * q4 + e;
            if (g < G) {
              float4 *dst = reinterpret_cast<float4 *>(piece + g * kD + 16 * r8);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k] = make_float4(oacc[nt][2 * k][e], oacc[nt][2 * k][2 + e], oacc[nt][2 * k + 1][e],
                                     oacc[nt][2 * k + 1][2 + e]);
            }
          }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = l_part[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            const int g = nt * 8 + 2 * q4 + e;
            if (g < G) {
              const int64_t row = (int64_t)b * p.num_q_heads + h * G + g;
              const float mul = l == 0.f ? 0.f : vmul / l;  // no valid token: 0; NaN goes through
              uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kD + 16 * r8);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                dst[k] = make_uint4(pack_bf16(oacc[nt][4 * k][e] * mul, oacc[nt][4 * k][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 1][e] * mul, oacc[nt][4 * k + 1][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 2][e] * mul, oacc[nt][4 * k + 2][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 3][e] * mul, oacc[nt][4 * k + 3][2 + e] * mul));
              if (r8 == 0 && p.lse) {
                const float mu = m_run[nt][e] == neg_inf() ? 0.f : m_run[nt][e];
                p.lse[row] = l == 0.f ? neg_inf() : (mu + __log2f(l)) * 0.69314718055994531f;
              }
            }
          }
      }
    }
    if (!ok) {
      // a wait gave up: wait (bounded) for the copies in flight before leaving
      for (int st = 0; st < S && st < issued; ++st) {
        const int last = (issued - 1) - ((issued - 1 - st) % S);
        mbar_wait_bounded(&full[st], (last / S) & 1, kWaitLimitNs);
      }
      dev_err |= DA_DEVERR_TIMEOUT;
      flags[0] = 1;
    }
  }
  __syncthreads();
  if (flags[0]) {
    if (dev_err) atomicOr(p.err, dev_err);
    return;
  }
  // ---------------------------------------------------------------- pieces of this CTA, unit by unit
  const int nout = G * (kD / 4);
  int ngroups = 0;
  for (int k = 0; k <= W; ++k) ngroups += lead[k].x >= 0 ? 1 : 0;
  for (int item = threadIdx.x; item < ngroups * nout; item += C::kThreads) {
    int k = 0;
    for (int skip = item / nout;; ++k) {
      if (lead[k].x < 0) continue;
      if (skip-- == 0) break;
    }
    const int4 grp = lead[k];
    const int o = item % nout, g = o / (kD / 4);
    const int a = k == W ? 0 : k, bw = grp.y & 255;
    // the last warp's piece is its head when that warp went on to another unit
    auto stat_of = [&](int w) { return stat_all + (w * 2 + (w == bw && (grp.y & 256) ? 1 : 0)) * 32; };
    float M = neg_inf();
    for (int w = a; w <= bw; ++w) {
      const float *st = stat_of(w);
      if (st[16 + g] != 0.f) M = fmaxf(M, st[g]);
    }
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int w = a; w <= bw; ++w) {
      const float *st = stat_of(w);
      const float l = st[16 + g];
      if (l == 0.f) continue;
      const float e = ex2(st[g] - M);
      const bool head = w == bw && (grp.y & 256);
      const float4 v = head ? __ldcg(reinterpret_cast<const float4 *>(fp.o_head + ((int64_t)cta * W + w) * G * kD) + o)
                            : reinterpret_cast<const float4 *>(smem + (size_t)w * C::kRingBytes)[o];
      L += e * l;
      acc.x += e * v.x;
      acc.y += e * v.y;
      acc.z += e * v.z;
      acc.w += e * v.w;
    }
    const int b = grp.x / p.num_kv_heads, h = grp.x - b * p.num_kv_heads;
    const float mul = L == 0.f ? 0.f : p.v_scale[h] / L;
    acc.x *= mul;
    acc.y *= mul;
    acc.z *= mul;
    acc.w *= mul;
    const float lse = L == 0.f ? neg_inf() : (M + __log2f(L)) * 0.69314718055994531f;
    if (grp.w == 0) {
      const int64_t row0 = (int64_t)b * p.num_q_heads + h * G;
      *reinterpret_cast<uint2 *>(p.out + row0 * kD + 4 * o) =
          make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
      if (o % (kD / 4) == 0 && p.lse) p.lse[row0 + g] = lse;
    } else {
      const int64_t slot = (int64_t)grp.x + cta;
      reinterpret_cast<float4 *>(p.o_part + slot * G * kD)[o] = acc;
      if (o % (kD / 4) == 0) p.lse_part[slot * G + g] = lse;
    }
  }
  __syncthreads();
  // ---------------------------------------------------------------- units shared with other CTAs
  if (threadIdx.x == 0)
    for (int k = 0; k <= W; ++k) {
      const int4 grp = lead[k];
      if (grp.x >= 0 && grp.w > 0) count_piece(p, flags, grp.x, grp.z, grp.w, false);
    }
  __syncthreads();
  const int npending = flags[12];
  float *scr = reinterpret_cast<float *>(smem);
  volatile int *last_group = flags + 13;
  for (int k = 0; k < npending; ++k) {
    const int unit = flags[24 + 4 * k], cf = flags[25 + 4 * k], ns = flags[26 + 4 * k];
    const int q = flags[27 + 4 * k];
    const int64_t slot0 = (int64_t)unit + cf;
    if (q < 0) {
      merge_slots_small(p, unit, G, slot0, 1, ns, true, 0, scr);  // at most kOneLevelSegs = kSmallMerge pieces
      if (threadIdx.x == 0) p.counters[unit] = 0u;
      __syncthreads();
      continue;
    }
    const int K = merge_group_size(ns), ng = (ns + K - 1) / K, gs = min(K, ns - q * K);
    if (gs <= kSmallMerge)
      merge_slots_small(p, unit, G, slot0 + (int64_t)q * K, 1, gs, false, slot0 + (int64_t)q * K, scr);
    else
      merge_slots_cta(p, unit, G, slot0 + (int64_t)q * K, 1, gs, false, slot0 + (int64_t)q * K, scr);
    if (threadIdx.x == 0)
      *last_group = atomic_add_acq_rel_gpu(p.counters + unit, 1u) == (unsigned)(ng - 1) ? 1 : 0;
    __syncthreads();
    if (*last_group) {
      if (ng <= kSmallMerge) merge_slots_small(p, unit, G, slot0, K, ng, true, 0, scr);
      else merge_slots_cta(p, unit, G, slot0, K, ng, true, 0, scr);
      uint32_t *gc = p.counters + p.batch * p.num_kv_heads + (int64_t)unit * max_merge_groups(gridDim.x);
      for (int i = threadIdx.x; i < ng; i += C::kThreads) gc[i] = 0u;
      if (threadIdx.x == 0) p.counters[unit] = 0u;
    }
    __syncthreads();
  }
  if (dev_err) atomicOr(p.err, dev_err);
}

template <int NT, int MOD>
cudaError_t f4_attr() {
  return cudaFuncSetAttribute(fp4_split_kernel<NT, MOD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              F4<NT>::kTotal);
}

}  // namespace

int fp4_tile() { return kT; }
int fp4_warps(int group) { return group <= 8 ? F4<1>::kWarps : F4<2>::kWarps; }

cudaError_t fp4_prepare() {
  cudaError_t e;
  if ((e = f4_attr<1, 0>()) != cudaSuccess) return e;
  if ((e = f4_attr<1, 1>()) != cudaSuccess) return e;
  if ((e = f4_attr<1, 2>()) != cudaSuccess) return e;
  if ((e = f4_attr<2, 0>()) != cudaSuccess) return e;
  if ((e = f4_attr<2, 1>()) != cudaSuccess) return e;
  return f4_attr<2, 2>();
}

cudaError_t launch_fp4(const Fp4Params &p, int ctas, cudaStream_t stream) {
  const int mod = gqa_mod(p.g);
#define DA_F4(NT, M) fp4_split_kernel<NT, M><<<ctas, F4<NT>::kThreads, F4<NT>::kTotal, stream>>>(p)
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
  return cudaGetLastError();
}

}  // namespace da
