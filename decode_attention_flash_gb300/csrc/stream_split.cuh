// stream_split.cuh -- persistent split-KV GQA decode whose warps stream alone, over the formats
// of a cache in granules of 16 rows (fp4_split.cu, block8_split.cu).
//
// The mathematics is the online softmax of gqa_split.cuh with the query group as the MMA's N
// dimension (mma.sync m16n8k16, f16 operands, fp32 sums):
//   S^T = K Q^T,  O^T += V^T P^T
//
// The layout. Every warp has a range of tiles and a ring of stages, filled by its own 16-byte
// asynchronous copies of whole granules, and no barrier with other warps until the end. What a
// tile is -- its pages, its valid tokens, its addresses -- one further warp, the walker, works
// out for all of them, a lane for each. The weights' reference, 5 octaves below the greatest
// score, is raised only when a sum of weights passes 2^15, so a stage usually needs no shuffle
// and no rescaling of O.
//
// The split. As in gqa_split.cuh the tiles of all (row, kv head) units are laid
// end to end and cut into equal ranges, one per CTA; a CTA's range is cut again
// into one range per warp. A unit inside one warp's range is written from its
// registers; pieces of a unit shared by warps meet in shared memory after the
// stream, and pieces shared by CTAs in global memory (counted and merged as in
// gqa_split.cuh, without any CTA waiting for another). Small calls give a CTA to every
// unit instead (plan.cpp): no scan, no merge between CTAs.
// More than 16 query heads a kv head are units of up to 16 that read the same cache
// (num_kv_heads counts them, shifted right by kv_shift it counts the cache's).
#pragma once

#include <type_traits>

#include "cache_ops.h"
#include "cache_ptx.cuh"
#include "gqa_split.cuh"

namespace da {
namespace {

constexpr int kGran = 16;             // rows of a granule
constexpr int kQueue = 8;             // described tiles a warp may have waiting or in its ring
constexpr float kRoom = 5.f;         // octaves from the weights' reference up to the greatest score so far
constexpr float kRaise = 32768.f;    // a sum of weights past this raises the reference

// A format F of the cache is a struct of constants (tokens of a stage, granule bytes, streaming
// warps, stages of a ring, bytes of scales beside a stage) and of what a lane does: copy a half
// of a stage, S^T = K Q^T, drop what masked tokens hold, O^T += V^T P^T. kHeadScales: K and V have
// a scale a head; kBlockScales: a scale a granule, which kFoldsV joins to the weights.
template <class F, int NT>
struct StreamLayout {
  static constexpr int kT = F::kT;                               // tokens per stage
  static constexpr int kHalves = kT / kGran;                     // granules of K, and of V, in a stage
  static constexpr int kStageBytes = 2 * kHalves * F::kGranBytes;  // K granules, then V granules
  static constexpr int kWarps = F::kWarps(NT);                   // consumers (an odd number: with the walker an even one)
  static constexpr int kThreads = (kWarps + 1) * 32;             // and the walker
  static constexpr int kStages = F::kStages(NT);
  static constexpr bool kQShared = F::kQShared(NT);              // Q^T fragments in shared memory, not in registers
  static constexpr int kQBytes = kQShared ? 8 * 32 * 16 : 0;
  static constexpr int kRingBytes = kStages * kStageBytes;       // one warp's ring
  static constexpr int kSideBytes = kStages * F::kSideBytes;     // and its stages' scales
  static constexpr int oQ = kWarps * kRingBytes;                 // [warp][k-step][lane]
  static constexpr int oSide = oQ + kWarps * kQBytes;            // [warp][stage]
  static constexpr int oStall = oSide + kWarps * kSideBytes;     // the test stall's barrier
  static constexpr int oCount = oStall + 16;                     // [16] tiles described, [16] tiles read, per warp
  static constexpr int oDesc = oCount + 128;                     // [warp][kQueue] StreamTile
  static constexpr int oStat = oDesc + kWarps * kQueue * 48;     // [warp][tail|head][m|l][16]
  static constexpr int oScan = oStat + kWarps * 64 * 4;
  static constexpr int oPre = oScan + 16 * 4;                    // [thread] tiles up to a thread's items
  static constexpr int oFlags = oPre + kThreads * 4;             // 40 ints, as in gqa_split.cuh
  static constexpr int oLead = oFlags + 40 * 4;                  // [warp + 1] groups (see below)
  static constexpr int oSum = oLead + (kWarps + 1) * 16;         // [warp + 1][16] 1 / L, [..][16] LSE
  static constexpr int kTotal = oSum + (kWarps + 1) * 32 * 4 + 128;
  static_assert(kWarps % 2 == 1 && kWarps <= 15, "two halves of a block merge, sixteen lanes a group");
  static_assert(kRingBytes >= NT * 8 * kD * 4, "a warp's ring holds its piece after the stream");
  static_assert(kRingBytes % 128 == 0 && oSide % 16 == 0 && oDesc % 16 == 0 && oScan % 16 == 0 && oLead % 16 == 0,
                "alignment");
  // (both one-level merges of a block have 16 KB of scratch, the larger group's takes 10.3 KB)
  static_assert(kWarps * kRingBytes >= 32768, "scratch of the merges");
  static_assert(kTotal <= 232448, "shared memory of a CTA");
};

// A tile as the walker describes it to the warp that reads it: the valid tokens
// (bit t: token t of the stage), flags (kFirst, kLast, kFull; kUnitStart / kUnitEnd:
// the unit's first / last tile), for the masks the row's length minus the tile's
// first position and that position; the byte offsets of its two halves' granules (in
// K and V alike; a half without a valid token is not read); the unit, its number of
// tiles and its first tile.
struct __align__(16) StreamTile {
  uint32_t valid;
  int32_t flags, nval, pos0;
  int64_t off0, off1;
  int32_t unit, tiles, P, pad;
};
constexpr int32_t kUnitStart = 8, kUnitEnd = 16;
static_assert(sizeof(StreamTile) == 48, "layout");

// n tiles cut into c consecutive ranges whose lengths differ by at most one (the
// first n % c are the longer ones).
struct Cut {
  uint32_t base, rem;
  __device__ __forceinline__ Cut(uint32_t n, uint32_t c) : base(n / c), rem(n % c) {}
  __device__ __forceinline__ int start(uint32_t i) const { return (int)(i * base + min(i, rem)); }
  __device__ __forceinline__ int owner(uint32_t t) const {
    const uint32_t split = rem * (base + 1);
    return (int)(t < split ? t / (base + 1) : rem + (t - split) / base);
  }
};

template <int kT>
__device__ __forceinline__ UnitInfo stream_unit_info(const GqaParams &p, int u, uint32_t &err) {
  UnitInfo x = unit_info(p, u, err);
  x.tiles = p.sparse_block_size > 0 ? x.tiles * (kTile / kT) : (x.n_valid + kT - 1) / kT;
  return x;
}

// `threads` threads (a whole number of warps, this one the `tid`-th, meeting at named
// barrier `bar`) merge the n <= 32 pieces of `unit` in slots slot0, slot0 + stride, .. into
// the output (to < 0) or one piece in slot `to`, which may be the first of them: a warp
// takes a row's LSEs, or four rows' of few pieces, one piece a lane, for the weights; the threads' loads of the
// pieces' O, kLoads at a time, are in flight meanwhile. `scr`: shared memory, free.
template <class F, int NT>
__device__ __noinline__ void stream_merge(const GqaParams &p, int unit, int64_t slot0, int stride, int n, int64_t to,
                                      int G, float *scr, int tid, int threads, int bar) {
  constexpr int kLoads = 8;
  const int lane = tid & 31, warp = tid >> 5;
  const int nout = G * (kD / 4);
  float *w = scr;                                          // [G][32] weights over their sum
  float *lse_to = scr + G * 32;                            // [16] of the piece (its slot is still read)
  float4 *acc = reinterpret_cast<float4 *>(scr + G * 32 + 16);  // [parts][nout]
  // sums of every parts-th piece that an output is the sum of: as many as the whole block has
  // threads for, also where half of it merges (a half then takes two rounds). The order of the
  // sum must not follow from whether this block came last for one unit or for two.
  const int parts = max(1, min(StreamLayout<F, NT>::kThreads / nout, n));
  const float4 *src = reinterpret_cast<const float4 *>(p.o_part + slot0 * G * kD);
  const int64_t step = (int64_t)stride * nout;
  const int b = unit / p.num_kv_heads, h = unit - b * p.num_kv_heads;
  const int64_t row0 = (int64_t)b * p.num_q_heads + h * G;
  auto weights = [&](auto lanes) {  // `lanes` lanes a row
    constexpr int kLanes = decltype(lanes)::value;
    const int sub = lane & (kLanes - 1), rows = threads / kLanes;
    auto lse_of = [&](int g) {
      return sub < n && g < G ? __ldcg(p.lse_part + (slot0 + sub * stride) * G + g) : neg_inf();
    };
    float ahead = lse_of(tid / kLanes);
    for (int g0 = 0; g0 < G; g0 += rows) {
      const int g = g0 + tid / kLanes;
      if (kLanes == 32 && g >= G) break;
      const float l = ahead;
      ahead = lse_of(g + rows);
      float M = l;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
      const float e = l == neg_inf() ? 0.f : ex2((l - M) * 1.4426950408889634f);
      float sum = e;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (kLanes < 32 && g >= G) continue;
      w[g * 32 + sub] = sum == 0.f ? 0.f : e / sum;
      if (sub == 0) {
        const float lse = sum == 0.f ? neg_inf() : M + __log2f(sum) * 0.69314718055994531f;
        if (to >= 0) lse_to[g] = lse;
        else if (p.lse) p.lse[row0 + g] = lse;
      }
    }
  };
  // (more rows than a pass of warps takes, 16 rows of 1000..20000 tokens: 75.4 -> 74.4 us)
  if (NT == 2 && n <= 8) weights(std::integral_constant<int, 8>());
  else weights(std::integral_constant<int, 32>());
  // (items are warp-uniform in number: nout * parts is a multiple of 32)
  bool met = false;
  for (int item = tid; item < nout * parts; item += threads) {
    const int o = item % nout, s0 = item / nout, g = o / (kD / 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = s0; s < n; s += parts * kLoads) {
      float4 v[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        v[k] = s + k * parts < n ? __ldcg(src + (int64_t)(s + k * parts) * step + o) : make_float4(0.f, 0.f, 0.f, 0.f);
      if (!met) named_barrier_sync(bar, threads);  // the weights are in w
      met = true;
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const float e = s + k * parts < n ? w[g * 32 + s + k * parts] : 0.f;
        if (e != 0.f) {  // a piece of weight 0 may hold anything
          a.x += e * v[k].x;
          a.y += e * v[k].y;
          a.z += e * v[k].z;
          a.w += e * v[k].w;
        }
      }
    }
    acc[item] = a;
  }
  if (!met) named_barrier_sync(bar, threads);  // (a warp without an item)
  named_barrier_sync(bar, threads);
  for (int o = tid; o < nout; o += threads) {
    float4 a = acc[o];
    for (int k = 1; k < parts; ++k) {
      const float4 v = acc[k * nout + o];
      a.x += v.x;
      a.y += v.y;
      a.z += v.z;
      a.w += v.w;
    }
    if (to >= 0) reinterpret_cast<float4 *>(p.o_part + to * G * kD)[o] = a;
    else *reinterpret_cast<uint2 *>(p.out + row0 * kD + 4 * o) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
  }
  if (to >= 0 && tid < G) p.lse_part[to * G + tid] = lse_to[tid];
  if (to < 0 && tid == 0) p.counters[unit] = 0u;  // ready for the next call
}
constexpr int kOneLevel = 32;  // pieces that stream_merge takes (a lane's worth); a unit of more is merged in
                               // two levels, groups as in gqa_split.cuh (by its own merge: 2.3 us more)

// The kernel's body, for a kernel of StreamLayout<F, NT>::kThreads threads that has waited for
// the stream's previous kernel. MOD: which score and mask modifications (gqa_mod).
template <class F, int NT, int MOD>
__device__ __forceinline__ void stream_split(const StreamParams &fp) {
  using C = StreamLayout<F, NT>;
  constexpr int W = C::kWarps, S = C::kStages, kT = C::kT, H = C::kHalves, kStageBytes = C::kStageBytes;
  constexpr int kGranBytes = F::kGranBytes;
  constexpr uint32_t kAll = kT == 32 ? 0xFFFFFFFFu : (1u << kT) - 1u;  // every token of a stage
  const GqaParams &p = fp.g;
  extern __shared__ uint8_t stream_smem[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(stream_smem) + 127) & ~uintptr_t(127));
  float *stat_all = reinterpret_cast<float *>(smem + C::oStat);
  int *scan = reinterpret_cast<int *>(smem + C::oScan);
  volatile int *flags = reinterpret_cast<volatile int *>(smem + C::oFlags);
  // flags: [0] a wait gave up; [13] scratch, [24..31] the merges owed (two: unit,
  // c_first, n_seg, group; unit -1: none)
  int *pre = reinterpret_cast<int *>(smem + C::oPre);
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

  if (threadIdx.x == W * 32 && p.paged)  // (a warp that has no lengths to wait for)
    prefetch_share_l2(p.block_table, (int64_t)p.batch * p.max_pages * 4);
  if (threadIdx.x == 0) {
    flags[0] = 0;
    flags[24] = flags[28] = -1;
  }
  if (threadIdx.x <= W) lead[threadIdx.x] = make_int4(-1, 0, 0, 0);

  // ---- the schedule. fp.whole: CTA c has unit c, whole (nothing to scan, no piece
  // leaves the CTA). Else the tiles of all units, end to end, one range per CTA. Thread t
  // counts the items [t * per, t * per + per): rows (all heads of a dense row are alike)
  // or, for listed blocks, units. The prefix sums stay in shared memory, where the
  // walker finds the unit that each warp's range starts in.
  const bool sparse = p.sparse_block_size > 0;
  const int items = sparse ? U : p.batch, heads = sparse ? 1 : p.num_kv_heads;
  const int per = (items + C::kThreads - 1) / C::kThreads;
  auto item_tiles = [&](int it, uint32_t &err) -> int {  // of one unit of item `it`
    return stream_unit_info<kT>(p, sparse ? it : it * heads, err).tiles;
  };
  // rows without a tile: zeros and -inf from the warp of the CTA that the item falls to
  auto write_empty = [&](int64_t row0, int rows) {
    for (int i = lane; i < rows * (kD / 8); i += 32)
      reinterpret_cast<uint4 *>(p.out + row0 * kD)[i] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse)
      for (int i = lane; i < rows; i += 32) p.lse[row0 + i] = neg_inf();
  };
  int T = 0, CTAS = 1;
  if (fp.whole) {
    const UnitInfo x = stream_unit_info<kT>(p, cta, dev_err);
    T = x.tiles;
    if (T == 0) {
      if (warp == 0) write_empty((int64_t)x.b * p.num_q_heads + x.h * G, G);
      if (dev_err) atomicOr(p.err, dev_err);
      return;
    }
  }
  int local = 0;
  for (int k = 0; !fp.whole && k < per; ++k) {
    const int it = (int)threadIdx.x * per + k;
    const int t = it < items ? item_tiles(it, dev_err) : 1;
    if (it < items) local += t * heads;
    uint32_t none = __ballot_sync(0xffffffffu, t == 0 && it % (int)gridDim.x == cta);
    for (; none != 0; none &= none - 1) {
      const int e = __shfl_sync(0xffffffffu, it, __ffs(none) - 1);
      write_empty(sparse ? (int64_t)(e / p.num_kv_heads) * p.num_q_heads + e % p.num_kv_heads * G
                         : (int64_t)e * p.num_q_heads,
                  heads * G);
    }
  }
  if (!fp.whole) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, local, o);
      if (lane >= o) local += v;
    }
    if (lane == 31) scan[warp] = local;
    if (threadIdx.x < 16 && threadIdx.x > W) scan[threadIdx.x] = 0;  // (a vector of 16 sums is read)
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int4 v = reinterpret_cast<const int4 *>(scan)[k];
      before += (4 * k < warp ? v.x : 0) + (4 * k + 1 < warp ? v.y : 0) + (4 * k + 2 < warp ? v.z : 0) +
                (4 * k + 3 < warp ? v.w : 0);
      T += v.x + v.y + v.z + v.w;
    }
    pre[threadIdx.x] = before + local;
    CTAS = min(T, (int)gridDim.x);  // never more ranges than tiles
    // of few tiles so few that a unit is merged in one level (ranges of 1 and 2 tiles side
    // by side would be twice as many for a unit of the short ones: none is short of the
    // mean, rounded up; of 8 tiles and more one matters little)
    if (T > 0 && T <= fp.few_tiles) {
      const uint32_t n = (uint32_t)T, few = (uint32_t)fp.few_ctas;
      CTAS = min(CTAS, (int)(n / 8 >= few ? few : n / ((n + few - 1) / few)));
    }
    if (cta >= CTAS) {
      if (dev_err) atomicOr(p.err, dev_err);
      return;
    }
  }
  const Cut cut((uint32_t)T, (uint32_t)CTAS);
  const int lo = fp.whole ? 0 : cut.start(cta), n_cta = fp.whole ? T : cut.start(cta + 1) - lo, hi = lo + n_cta;
  const Cut wcut((uint32_t)n_cta, W);
  uint64_t *stall_bar = reinterpret_cast<uint64_t *>(smem + C::oStall);  // nothing arrives on it
  uint32_t *ready_all = reinterpret_cast<uint32_t *>(smem + C::oCount);  // tiles described, per warp
  uint32_t *done_all = ready_all + 16;                                   // and tiles read
  StreamTile *tiles_all = reinterpret_cast<StreamTile *>(smem + C::oDesc);
  if (threadIdx.x == 0) {
    mbar_init(stall_bar, 1);
    fence_mbar_init();
  }
  if (threadIdx.x < 32) ready_all[threadIdx.x] = 0u;
  __syncthreads();

  bool ok = true;
  if (warp == W) {
    // ============================================================ the walker
    // Lane w walks the tiles of warp w's range, a few tiles ahead of it: which pages or
    // blocks, which tokens are valid, where the bytes are. One pass of the loop serves
    // every warp, so the walk costs a fraction of what it would in each of them.
    const int w = lane < W ? lane : 0;
    const int wlo = lo + wcut.start(w);
    const int ntiles = lane < W ? lo + wcut.start(w + 1) - wlo : 0;
    StreamTile *queue = tiles_all + w * kQueue;
    const int P = p.page_size;
    // entries (pages or listed blocks) of `tpe` tiles each; pages of 16 tokens: two per tile
    const int tpe = sparse ? p.sparse_block_size / kT : (p.paged ? (P >= kT ? P / kT : 1) : 1);
    const bool two_pages = p.paged && P < kT;
    const bool has_ids = p.paged || sparse;
    const int gran_unit = p.paged ? P / kGran : p.cache_len / kGran;  // granules per (page | row, head)
    const int kv_heads = p.num_kv_heads >> fp.kv_shift;                // of the cache
    int u = 0, j = 0, ent = 0, sub = 0, nent = 0;  // unit, its tile, current entry, tile inside it, entries
    int id0 = -1, id1 = -1;                        // the current tile's ids
    int Pu = 0;                                    // the unit's first tile
    UnitInfo x;
    x.b = x.h = x.n_valid = x.nbp = x.trow = 0;
    x.tiles = 1;
    auto load_id = [&](int e) -> int {
      if (e >= nent) return -1;
      if (sparse)
        return e < x.nbp ? p.kv_idx[(int64_t)x.trow * p.max_sparse_blocks + e]
                         : p.kv_full_idx[(int64_t)x.trow * p.max_sparse_blocks + e - x.nbp];
      return p.block_table[(int64_t)x.b * p.max_pages + e];
    };
    auto load_ids = [&]() {
      id0 = load_id(ent);
      if (two_pages) id1 = load_id(ent + 1);
    };
    auto enter_unit = [&]() {  // x holds unit u's info; tile j of it comes next
      if (has_ids) {
        ent = two_pages ? 2 * j : j / tpe;
        sub = two_pages ? 0 : j - ent * tpe;
        nent = sparse ? x.tiles / tpe : (x.n_valid + P - 1) / P;
        load_ids();
      }
      prefetch_l2(p.q + ((int64_t)x.b * p.num_q_heads + x.h * G) * kD, (uint32_t)(G * kD * 2));
    };
    if (ntiles > 0) {
      uint32_t ignored = 0;
      if (fp.whole) {
        u = cta;
        x = stream_unit_info<kT>(p, u, ignored);
      } else {
        // the thread whose items hold tile wlo, then the item, then the head
        int first = 0;
        for (int n = C::kThreads; n > 0;) {  // the number of threads whose sum is at most wlo
          const int half = n >> 1;
          if (pre[first + half] <= wlo) {
            first += half + 1;
            n -= half + 1;
          } else {
            n = half;
          }
        }
        Pu = first > 0 ? pre[first - 1] : 0;
        int it = first * per;
        x = stream_unit_info<kT>(p, it * heads, ignored);
        while (wlo >= Pu + x.tiles * heads) {
          Pu += x.tiles * heads;
          ++it;
          x = stream_unit_info<kT>(p, it * heads, ignored);
        }
        const int h = sparse ? 0 : (wlo - Pu) / x.tiles;
        u = it * heads + h;
        x.h += h;
        Pu += h * x.tiles;
      }
      j = wlo - Pu;
      enter_unit();
    }
    int i = 0;
    uint64_t since = 0;
    while (true) {
      const bool go = i < ntiles && i < (int)ld_acquire_cta(&done_all[w]) + kQueue;
      if (go) {
        int pos0 = j * kT;
        uint32_t valid = 0;
        int64_t gr0, gr1;
        bool full_blk = false;
        if (sparse) {
          full_blk = ent >= x.nbp;
          if (id0 < 0 || (int64_t)id0 * p.sparse_block_size >= p.cache_len) {
            dev_err |= DA_DEVERR_SPARSE_INDEX;
          } else {
            pos0 = id0 * p.sparse_block_size + sub * kT;
            valid = (uint32_t)low_bits(min(min(x.n_valid - pos0, kT), p.cache_len - pos0));
          }
          gr0 = (int64_t)u * gran_unit + pos0 / kGran;
          gr1 = gr0 + 1;
        } else {
          const int left = x.n_valid - pos0;  // at least 1
          valid = left >= kT ? kAll : (1u << left) - 1u;
          if (!p.paged) {
            gr0 = (int64_t)(u >> fp.kv_shift) * gran_unit + j * (kT / kGran);
            gr1 = gr0 + 1;
          } else if (two_pages) {
            const bool ok0 = (uint32_t)id0 < (uint32_t)p.num_pages, ok1 = (uint32_t)id1 < (uint32_t)p.num_pages;
            if (!ok0 || (left > kGran && !ok1)) dev_err |= DA_DEVERR_PAGE_INDEX;
            valid &= (ok0 ? 0xFFFFu : 0u) | (ok1 ? 0xFFFF0000u : 0u);
            gr0 = (int64_t)id0 * kv_heads + (x.h >> fp.kv_shift);
            gr1 = (int64_t)id1 * kv_heads + (x.h >> fp.kv_shift);
          } else {
            if ((uint32_t)id0 >= (uint32_t)p.num_pages) {
              dev_err |= DA_DEVERR_PAGE_INDEX;
              valid = 0;
            }
            gr0 = ((int64_t)id0 * kv_heads + (x.h >> fp.kv_shift)) * gran_unit + sub * (kT / kGran);
            gr1 = gr0 + 1;
          }
        }
        const int fl = (i == 0 || j == 0 ? kFirst : 0) | (i + 1 == ntiles || j + 1 == x.tiles ? kLast : 0) |
                       (full_blk ? kFull : 0) | (j == 0 ? kUnitStart : 0) | (j + 1 == x.tiles ? kUnitEnd : 0);
        StreamTile t;
        t.valid = valid;
        t.flags = fl;
        t.nval = x.n_valid - pos0;
        t.pos0 = pos0;
        t.off0 = gr0 * kGranBytes;
        t.off1 = gr1 * kGranBytes;
        t.unit = u;
        t.tiles = x.tiles;
        t.P = Pu;
        queue[i % kQueue] = t;
        ++i;
        st_release_cta(&ready_all[w], (uint32_t)i);
        // the next tile, its ids in flight until there is room for it
        if (++j < x.tiles) {
          if (two_pages) {
            ent += 2;
            load_ids();
          } else if (has_ids && ++sub == tpe) {
            sub = 0;
            ++ent;
            load_ids();
          }
        } else if (i < ntiles) {
          Pu += x.tiles;
          ++u;
          if (!sparse && x.h + 1 < p.num_kv_heads) {
            ++x.h;  // the next head of the row: the same lengths and pages
          } else {
            x = stream_unit_info<kT>(p, u < U ? u : U - 1, dev_err);
            while (x.tiles == 0 && u + heads < U) {  // (rows without a tile were written above)
              u += heads;
              x = stream_unit_info<kT>(p, u, dev_err);
            }
          }
          j = 0;
          enter_unit();
        }
      }
      if (!__any_sync(0xffffffffu, i < ntiles)) break;
      if (__any_sync(0xffffffffu, go)) {
        since = 0;
      } else {
        // every queue is full: wait a little (bounded, like every wait)
        const uint64_t now = global_timer_ns();
        if (since == 0) since = now;
        if (flags[0] || now - since > kWaitLimitNs) {
          ok = false;
          break;
        }
        __nanosleep(100);
      }
    }
    if (!__all_sync(0xffffffffu, ok)) {
      dev_err |= DA_DEVERR_TIMEOUT;
      flags[0] = 1;
    }
    __syncthreads();
    if (flags[0]) {
      if (dev_err) atomicOr(p.err, dev_err);
      return;
    }
  } else {
    // ============================================================ consumers
    const int q4 = lane & 3, r8 = lane >> 2;
    const int ntiles = wcut.start(warp + 1) - wcut.start(warp);
    uint8_t *ring = smem + (size_t)warp * C::kRingBytes;
    const StreamTile *queue = tiles_all + warp * kQueue;
    if (ntiles == 0) stat_all[warp * 64 + lane] = 0.f;  // no piece: weight 0 in the sums below
    // Tile i's copies into stage `to`: 16 bytes a lane, 72 lanes' worth a granule, one
    // commit group. False when the walker stays away.
    uint32_t ready = 0;
    const F fmt(fp, lane);
    const uint32_t ring_at = smem_u32(ring) + fmt.lane_at();
    uint8_t *side = smem + C::oSide + warp * C::kSideBytes;
    auto issue = [&](int i, int to) -> bool {
      if ((int)ready <= i) {
        ready = ld_acquire_cta(&ready_all[warp]);
        if ((int)ready <= i) {
          const uint64_t t0 = global_timer_ns();
          while ((int)(ready = ld_acquire_cta(&ready_all[warp])) <= i)
            if (flags[0] || global_timer_ns() - t0 > kWaitLimitNs) break;
        }
        ready = __reduce_min_sync(0xffffffffu, ready);
        if ((int)ready <= i) return false;
      }
      const StreamTile *t = &queue[i % kQueue];
      const uint32_t valid = t->valid;
      const longlong2 off = *reinterpret_cast<const longlong2 *>(&t->off0);
      const uint32_t dst = ring_at + to * kStageBytes;
      uint8_t *scales = side + to * F::kSideBytes;
#pragma unroll
      for (int gi = 0; gi < H; ++gi)
        if ((valid >> (kGran * gi)) & 0xFFFFu)
          fmt.copy(dst + gi * kGranBytes, dst + (H + gi) * kGranBytes, gi == 0 ? off.x : off.y, scales, gi);
      return true;
    };
    // The first tile alone, so that no warp's first tile queues behind the others' second
    // and third; those follow when the first has landed.
    if (ntiles > 0) ok = issue(0, 0);
    cp_async_commit();
    // ------------------------------------------------------------ the stream
    uint32_t qf[NT][8][2];
    uint4 *qs = reinterpret_cast<uint4 *>(smem + C::oQ + warp * C::kQBytes) + lane;  // kQShared
    float oacc[NT][8][4];
    float m_neg[NT][2], l_part[NT][2];  // minus the weights' reference (log2 units), and their sums
    bool no_ref[NT][2];                 // (MOD > 0) no kept token of the row so far
    float sscale = p.score_scale;
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
    // (kFoldsV) O is in units of vref, a power of two not below any V scale of the segment so far
    float vref = 0x1p-126f;
    bool from_start = false;  // the segment holds its unit's first tile
    bool fresh = false;       // no reference for the segment's weights yet
    int unit = 0;
    // (the test stall of GqaParams, in the warp that always has a tile: the timeout path
    // runs as after a real failure)
    if (p.test_stall_ns != 0 && warp == W - 1) ok = warp_wait(stall_bar, 0u, p.test_stall_ns);
    int st = -1;
    for (int i = 0; ok && i < ntiles; ++i) {
      st = st + 1 == S ? 0 : st + 1;
      const StreamTile *tile = &queue[i % kQueue];
      uint32_t valid;
      int fl, nval = 0, pos0 = 0;
      if (MOD == 0) {
        const uint2 m = *reinterpret_cast<const uint2 *>(tile);
        valid = m.x;
        fl = (int)m.y;
      } else {
        const uint4 m = *reinterpret_cast<const uint4 *>(tile);
        valid = m.x;
        fl = (int)m.y;
        nval = (int)m.z;
        pos0 = (int)m.w;
      }
      uint8_t *stage = ring + st * kStageBytes;
      if (__builtin_expect(fl & kFirst, 0)) {
        from_start = (fl & kUnitStart) != 0;
        fresh = true;
        unit = tile->unit;
        const int b = unit / p.num_kv_heads, h = unit - b * p.num_kv_heads;
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
            const uint4 v = src[s];
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
        for (int s = 0; s < 8; ++s) {
          if constexpr (C::kQShared) {  // (each lane reads back what it wrote)
            qs[s * 32] = make_uint4(bf16x2_to_f16x2(qw[0][s].x, q2), bf16x2_to_f16x2(qw[0][s].y, q2),
                                    bf16x2_to_f16x2(qw[NT - 1][s].x, q2), bf16x2_to_f16x2(qw[NT - 1][s].y, q2));
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              qf[nt][s][0] = bf16x2_to_f16x2(qw[nt][s].x, q2);
              qf[nt][s][1] = bf16x2_to_f16x2(qw[nt][s].y, q2);
            }
          }
        }
        sscale = p.score_scale * (F::kHeadScales ? p.k_scale[h >> fp.kv_shift] : 1.f) * pow2f(-qexp);
        // a zero factor (uniform weights) as 2^-100: a finite score still weighs 1, and
        // an infinite one (a masked token's) 0
        if (sscale == 0.f) sscale = 0x1p-100f;
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
          if (F::kFoldsV) vref = 0x1p-126f;
          m_neg[nt][0] = m_neg[nt][1] = 0.f;
          no_ref[nt][0] = no_ref[nt][1] = true;
          l_part[nt][0] = l_part[nt][1] = 0.f;
        }
      }
      if (__builtin_expect(i == 0, 0)) {
        cp_async_wait_group<0>();
#pragma unroll
        for (int k = 1; k < S; ++k) {
          if (ok && k < ntiles) ok = issue(k, k);
          cp_async_commit();
        }
      }
      cp_async_wait_group<S - 1>();  // this lane's copies of tile i have landed,
      __syncwarp();                  // and so have the other lanes'
      if (__builtin_expect(valid != 0, 1)) {
        // ---------------- S^T = K Q^T (every granule of the stage: a branch between them would
        // keep their instructions apart; what a half that was not copied holds is masked below)
        float s[NT][H][4];
        const uint8_t *scales = side + st * F::kSideBytes;
        fmt.template scores<NT>(stage, scales, qf, qs, s);
        // ---------------- masks and the online softmax (log2 units)
        const bool part = valid != kAll;
        float f = sscale;  // log2 units of a score in s
        // several query tokens: a stage of older positions only has nothing to mask
        const bool masks = MOD == 2 || (MOD == 1 && (softcap || nval - p.q_len < kT));
        if (MOD >= 1 && masks) {  // scores become x = score * log2 e here; masked ones -inf
          f = 1.f;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int k = 0; k < 2 * H; ++k) {
                const int t = r8 + 8 * k;  // token of the stage
                float v = s[nt][k >> 1][(k & 1) * 2 + e] * sscale;
                if (softcap) v = cap_tanh(v, p.softcap_l2, p.softcap_k);
                const int jnew = t - (nval - p.q_len);
                bool keep = (valid >> t) & 1u;
                keep = keep && (jnew < 0 || ((mword[nt][e] >> min(jnew, 31)) & 1u));
                if (mods) {
                  const int row = min(nt * 8 + 2 * q4 + e, G - 1);
                  const int hq = (unit % p.num_kv_heads) * (G / p.q_len) + row / p.q_len;
                  const int kv = pos0 + t, qpos = nval + pos0 - p.q_len + trow[nt][e];
                  if (p.mask_window && !(fl & kFull)) {
                    const int w = __ldg(p.mask_window + hq), sk = p.mask_sink ? __ldg(p.mask_sink + hq) : 0;
                    keep = keep && (kv < sk || w < 0 || kv > qpos - w);
                  }
                  if (p.alibi_slopes)
                    v += __ldg(p.alibi_slopes + hq) * 1.4426950408889634f * (float)(kv - qpos);
                }
                s[nt][k >> 1][(k & 1) * 2 + e] = keep ? v : neg_inf();
              }
        }
        if (__builtin_expect(part, 0)) {  // the row's end, or a page that was not there
          if (MOD == 0 || !masks) {
            // a masked score takes the value whose weight is 0 whatever the scale's sign
            const float none = sscale < 0.f ? -neg_inf() : neg_inf();
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2 * H; ++k)
                if (!((valid >> (r8 + 8 * k)) & 1u)) s[nt][k >> 1][(k & 1) * 2] = s[nt][k >> 1][(k & 1) * 2 + 1] = none;
          }
          fmt.drop(stage, side + st * F::kSideBytes, valid);  // what masked tokens' value rows hold
          __syncwarp();
        }
        // The weights 2^(x - m) against the held reference m, and their sums. The
        // reference is raised only when a sum passes 2^15 (so no weight does, and
        // f16 holds them all; the sums are fp32), or when there is none yet.
        float y[NT][2][2 * H], sum[NT][2];
        bool raise = fresh;
        auto weights = [&]() {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
              for (int k = 0; k < 2 * H; ++k) {
                const float v = s[nt][k >> 1][(k & 1) * 2 + e];
                y[nt][e][k] = ex2(fmaf(v, f, m_neg[nt][e]));
              }
              sum[nt][e] = y[nt][e][0] + y[nt][e][1];
              if constexpr (H == 2) sum[nt][e] += y[nt][e][2] + y[nt][e][3];
            }
        };
        weights();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) raise = raise || sum[nt][0] > kRaise || sum[nt][1] > kRaise;
        if (MOD >= 1)  // (a row may have had no kept token so far)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) raise = raise || no_ref[nt][0] || no_ref[nt][1];
        if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
          const bool first = fresh;
          fresh = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float t = neg_inf();
#pragma unroll
              for (int k = 0; k < 2 * H; ++k) {
                const float v = s[nt][k >> 1][(k & 1) * 2 + e];
                t = fmaxf(t, v * f);
              }
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 4));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 8));
              t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 16));
              // while no score of the row is valid the reference is 0, with nothing to rescale
              const bool none = MOD == 0 ? first : no_ref[nt][e];
              const float m_new = none ? t - kRoom : fmaxf(-m_neg[nt][e], t - kRoom);
              const float mn = m_new == neg_inf() ? 0.f : m_new;
              alpha[e] = none ? 1.f : ex2(-m_neg[nt][e] - mn);
              if (MOD >= 1) no_ref[nt][e] = m_new == neg_inf();
              m_neg[nt][e] = -mn;
              l_part[nt][e] *= alpha[e];
            }
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              oacc[nt][mt][0] *= alpha[0];
              oacc[nt][mt][1] *= alpha[1];
              oacc[nt][mt][2] *= alpha[0];
              oacc[nt][mt][3] *= alpha[1];
            }
          }
          weights();
        }
        // The V scales over vref join the weights (16 multiplies, not 128, for 32 tokens of 16 rows). One below
        // 2^-4 of it would cost small weights their bits in f16, one that is not finite is no factor of f16:
        // such a stage's products are scaled in fp32.
        float vmul[H];
        bool fold = true;
        if constexpr (F::kFoldsV) {
          float most = 0.f;
#pragma unroll
          for (int gi = 0; gi < H; ++gi) {
            vmul[gi] = F::v_scale(scales, gi);
            if (fabsf(vmul[gi]) < __int_as_float(0x7f800000)) most = fmaxf(most, fabsf(vmul[gi]));
          }
          if (__builtin_expect(most > vref && vref < 0x1p126f, 0)) {  // (the same in every lane)
            const float up = fminf(__uint_as_float((__float_as_uint(most) + 0x7FFFFFu) & 0x7F800000u), 0x1p126f);
            const float alpha = vref / up;
            vref = up;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) oacc[nt][mt][e] *= alpha;
          }
          const float vinv = __uint_as_float(0x7F000000u - __float_as_uint(vref));
#pragma unroll
          for (int gi = 0; gi < H; ++gi) {
            vmul[gi] *= vinv;
            fold = fold && (vmul[gi] == 0.f || (vmul[gi] >= 0x1p-4f && vmul[gi] <= 1.f));
          }
        } else if constexpr (F::kBlockScales) {
#pragma unroll
          for (int gi = 0; gi < H; ++gi) vmul[gi] = F::v_scale(scales, gi);
        }
        // P^T fragments: weights as f16, the row sums from the fp32 ones
        uint32_t pb[NT][H][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          l_part[nt][0] += sum[nt][0];
          l_part[nt][1] += sum[nt][1];
#pragma unroll
          for (int k = 0; k < 2 * H; ++k)
            pb[nt][k >> 1][k & 1] = movmatrix_trans(
                F::kFoldsV ? pack_f16(y[nt][0][k] * (fold ? vmul[k >> 1] : 1.f), y[nt][1][k] * (fold ? vmul[k >> 1] : 1.f))
                           : pack_f16(y[nt][0][k], y[nt][1][k]));
        }
        // ---------------- O^T += V^T P^T
        // (a weight of 0 times NaN is no 0: a token that some query rows see and others do not
        // may hold one)
        bool careful = false;
        if constexpr (MOD >= 1 && F::kCareful) {
          if (masks) {
            bool some = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int k = 0; k < 2 * H; ++k)
                  some = some || (((valid >> (r8 + 8 * k)) & 1u) && s[nt][k >> 1][(k & 1) * 2 + e] == neg_inf());
            if (__any_sync(0xffffffffu, some)) careful = fmt.not_finite(stage + H * kGranBytes, scales, valid);
          }
        }
        if constexpr (MOD >= 1 && F::kCareful) {
          if (__builtin_expect(careful, 0)) fmt.template values_kept<NT>(stage + H * kGranBytes, vmul, valid, s, y, oacc);
        }
        if (!careful) fmt.template values<NT>(stage + H * kGranBytes, vmul, fold, pb, oacc);
      }
      int seg_P = 0, seg_tiles = 0;
      if (fl & kLast) {
        seg_P = tile->P;
        seg_tiles = tile->tiles;
      }
      __syncwarp();  // every lane has read the stage and its description
      if (lane == 0) st_release_cta(&done_all[warp], (uint32_t)(i + 1));
      if (i + S < ntiles) ok = issue(i + S, st);
      cp_async_commit();  // (a group a tile, empty ones at the end)
      if (__builtin_expect(!(fl & kLast), 1)) continue;
      // ---------------- the segment ends. Row sums, then: a unit held by this
      // segment alone goes out from the registers; another segment's (m, l, O) to
      // this warp's ring when it is the warp's last, else to its global slot
      const bool whole = from_start && (fl & kUnitEnd);
      const bool tail = i + 1 == ntiles;
      const int b = unit / p.num_kv_heads, h = unit - b * p.num_kv_heads;
      float *piece = nullptr;
      if (!whole) {
        float *stat = stat_all + (warp * 2 + (tail ? 0 : 1)) * 32;
        if constexpr (F::kFoldsV) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int mt = 0; mt < 8; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) oacc[nt][mt][e] *= vref;
        }
        piece = tail ? reinterpret_cast<float *>(ring)
                     : fp.o_head + ((int64_t)cta * W + warp) * G * kD;
        // the unit's first warp here names the group (a head alone is warp 0's)
        if (lane == 0) {
          const int first = max(seg_P, lo), end = min(seg_P + seg_tiles, hi);
          if (wcut.owner(first - lo) == warp) {
            const int bw = wcut.owner(end - 1 - lo);
            const bool goes_on = end < lo + wcut.start(bw + 1);
            int c_first = 0, n_seg = 0;
            if (seg_P < lo || seg_P + seg_tiles > hi) {
              c_first = cut.owner(seg_P);
              n_seg = cut.owner(seg_P + seg_tiles - 1) - c_first + 1;
            }
            lead[tail ? warp : W] = make_int4(unit, bw | (goes_on ? 256 : 0), c_first, n_seg);
            reinterpret_cast<float *>(smem + C::oSum)[(tail ? warp : W) * 32 + 16] =
                F::kHeadScales ? p.v_scale[h >> fp.kv_shift] : 1.f;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = l_part[nt][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (r8 == 0) {
              stat[nt * 8 + 2 * q4 + e] = -m_neg[nt][e];
              stat[16 + nt * 8 + 2 * q4 + e] = l;
            }
          }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int g = nt * 8 + 2 * q4 + e;
            if (g < G) {
              // (float4 f of a row stands at f ^ (f >> 3 & 3): no bank conflicts either way)
              float4 *dst = reinterpret_cast<float4 *>(piece + g * kD + 16 * r8);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                dst[k ^ (r8 >> 1)] = make_float4(oacc[nt][2 * k][e], oacc[nt][2 * k][2 + e], oacc[nt][2 * k + 1][e],
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
              const float mul = l == 0.f ? 0.f : (F::kHeadScales ? p.v_scale[h >> fp.kv_shift] : F::kFoldsV ? vref : 1.f) / l;  // no valid token: 0; NaN goes through
              uint4 *dst = reinterpret_cast<uint4 *>(p.out + row * kD + 16 * r8);
#pragma unroll
              for (int k = 0; k < 2; ++k)
                dst[k] = make_uint4(pack_bf16(oacc[nt][4 * k][e] * mul, oacc[nt][4 * k][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 1][e] * mul, oacc[nt][4 * k + 1][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 2][e] * mul, oacc[nt][4 * k + 2][2 + e] * mul),
                                    pack_bf16(oacc[nt][4 * k + 3][e] * mul, oacc[nt][4 * k + 3][2 + e] * mul));
              if (r8 == 0 && p.lse) {
                p.lse[row] = l == 0.f ? neg_inf() : (__log2f(l) - m_neg[nt][e]) * 0.69314718055994531f;
              }
            }
          }
      }
    }
    cp_async_wait_group<0>();  // no copy outlives the loop (one that gave up leaves early)
    if (!ok) {
      dev_err |= DA_DEVERR_TIMEOUT;
      flags[0] = 1;
    }
    __syncthreads();
    if (flags[0]) {
      if (dev_err) atomicOr(p.err, dev_err);
      return;
    }
  }
  // ---------------------------------------------------------------- pieces of this CTA, unit by unit
  // First the weights: per group and row the reference M of its pieces, each piece's
  // 2^(m - M) (in place of its m) and 1 / L; then the weighted sums.
  const int nout = G * (kD / 4);
  float *sums = reinterpret_cast<float *>(smem + C::oSum);
  // the piece of group (k, b) in warp w: its head when w is the last and went on
  auto stat_of = [&](const int4 &grp, int w) {
    return stat_all + (w * 2 + (w == (grp.y & 255) && (grp.y & 256) ? 1 : 0)) * 32;
  };
  const uint32_t groups = __ballot_sync(0xffffffffu, lane <= W && lead[min(lane, W)].x >= 0);
  const int ngroups = __popc(groups);
  auto group_at = [&](int i) {  // the i-th group
    uint32_t rest = groups;
    for (; i > 0; --i) rest &= rest - 1;
    return __ffs(rest) - 1;
  };
  // sixteen lanes a (group, row), one piece each
  for (int t0 = warp * 2; t0 < ngroups * G; t0 += C::kThreads / 16) {
    const int task = t0 + (lane >> 4), sub = lane & 15;
    const bool on = task < ngroups * G;
    const int gi = on ? task / G : 0, g = on ? task - gi * G : 0;
    const int k = group_at(gi);
    const int4 grp = lead[k];
    const int w = (k == W ? 0 : k) + sub;
    float *st = stat_of(grp, min(w, W - 1));
    const float l = on && w <= (grp.y & 255) ? st[16 + g] : 0.f;
    const float m = l != 0.f ? st[g] : neg_inf();
    float M = m;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float e = l == 0.f ? 0.f : ex2(m - M);
    float L = l == 0.f ? 0.f : e * l;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (on && w <= (grp.y & 255)) st[g] = e;
    if (on && sub == 0) {
      const int b = grp.x / p.num_kv_heads, h = grp.x - b * p.num_kv_heads;
      sums[k * 32 + g] = L == 0.f ? 0.f : sums[k * 32 + 16] / L;
      const float lse = L == 0.f ? neg_inf() : (M + __log2f(L)) * 0.69314718055994531f;
      if (grp.w > 0) p.lse_part[((int64_t)grp.x + cta) * G + g] = lse;
      else if (p.lse) p.lse[(int64_t)b * p.num_q_heads + h * G + g] = lse;
    }
  }
  __syncthreads();
  // items (group, float4 o of its rows), thread by thread
  uint32_t rest = groups;
  for (int o = threadIdx.x;; o += C::kThreads) {
    for (; rest != 0 && o >= nout; o -= nout) rest &= rest - 1;
    if (rest == 0) break;
    const int k = __ffs(rest) - 1;
    const int4 grp = lead[k];
    const int g = o / (kD / 4), f = o % (kD / 4), at = g * (kD / 4) + (f ^ ((f >> 3) & 3));
    const int a = k == W ? 0 : k, bw = grp.y & 255;
    const bool head = (grp.y & 256) != 0;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f), last = acc;
    if (head) last = __ldcg(reinterpret_cast<const float4 *>(fp.o_head + ((int64_t)cta * W + bw) * G * kD) + at);
    auto add = [&](const float4 &v, float e) {
      if (e != 0.f) {  // a piece of weight 0 may hold anything
        acc.x += e * v.x;
        acc.y += e * v.y;
        acc.z += e * v.z;
        acc.w += e * v.w;
      }
    };
#pragma unroll 4
    for (int w = a; w <= bw - (head ? 1 : 0); ++w)
      add(reinterpret_cast<const float4 *>(smem + (size_t)w * C::kRingBytes)[at], stat_all[w * 64 + g]);
    if (head) add(last, stat_all[bw * 64 + 32 + g]);
    const float mul = sums[k * 32 + g];
    acc.x *= mul;
    acc.y *= mul;
    acc.z *= mul;
    acc.w *= mul;
    if (grp.w == 0) {
      const int b = grp.x / p.num_kv_heads, h = grp.x - b * p.num_kv_heads;
      *reinterpret_cast<uint2 *>(p.out + ((int64_t)b * p.num_q_heads + h * G) * kD + 4 * o) =
          make_uint2(pack_bf16(acc.x, acc.y), pack_bf16(acc.z, acc.w));
    } else {
      reinterpret_cast<float4 *>(p.o_part + ((int64_t)grp.x + cta) * G * kD)[o] = acc;
    }
  }
  __syncthreads();
  // ---------------------------------------------------------------- units shared with other CTAs
  // (at most two: the one that the range starts in and the one that it ends in),
  // each counted by a thread of its own; the count that completes a unit, or a group
  // of one merged in two levels, makes its merge this CTA's
  if (threadIdx.x <= W && lead[threadIdx.x].x >= 0 && lead[threadIdx.x].w > 0) {
    const int4 grp = lead[threadIdx.x];
    const int unit = grp.x, cf = grp.z, ns = grp.w;
    int q = -1, of = ns;
    uint32_t *counter = p.counters + unit;
    if (ns > kOneLevel) {
      const int K = merge_group_size(ns);
      q = (cta - cf) / K;
      of = min(K, ns - q * K);
      counter = p.counters + U + (int64_t)unit * max_merge_groups(gridDim.x) + q;
    }
    if (atomic_add_acq_rel_gpu(counter, 1u) == (unsigned)(of - 1)) {
      const int slot = cf < cta ? 24 : 28;  // the unit that the range starts in, or ends in
      flags[slot + 1] = cf;
      flags[slot + 2] = ns;
      flags[slot + 3] = q;
      flags[slot] = unit;
    }
  }
  __syncthreads();
  float *scr = reinterpret_cast<float *>(smem);
  volatile int *last_group = flags + 13;
  // one-level merges: the whole block for one, a half each for two
  const bool one0 = flags[24] >= 0 && flags[27] < 0, one1 = flags[28] >= 0 && flags[31] < 0;
  if (one0 || one1) {
    constexpr int kHalf = (W + 1) / 2 * 32;
    const bool both = one0 && one1;
    const int mine = both ? (int)threadIdx.x / kHalf : 0, slot = (both ? mine : one0 ? 0 : 1) ? 28 : 24;
    stream_merge<F, NT>(p, flags[slot], (int64_t)flags[slot] + flags[slot + 1], 1, flags[slot + 2], -1, G, scr + mine * 4096,
             (int)threadIdx.x - mine * kHalf, both ? kHalf : C::kThreads, 1 + mine);
    __syncthreads();
  }
  for (int slot = 24; slot <= 28; slot += 4) {
    const int unit = flags[slot], cf = flags[slot + 1], ns = flags[slot + 2], q = flags[slot + 3];
    if (unit < 0 || q < 0) continue;
    const int64_t slot0 = (int64_t)unit + cf;
    const int K = merge_group_size(ns), ng = (ns + K - 1) / K, gs = min(K, ns - q * K);
    const int64_t first = slot0 + (int64_t)q * K;
    stream_merge<F, NT>(p, unit, first, 1, gs, first, G, scr, (int)threadIdx.x, C::kThreads, 1);
    __syncthreads();
    if (threadIdx.x == 0)
      *last_group = atomic_add_acq_rel_gpu(p.counters + unit, 1u) == (unsigned)(ng - 1) ? 1 : 0;
    __syncthreads();
    if (*last_group) {
      uint32_t *gc = p.counters + U + (int64_t)unit * max_merge_groups(gridDim.x);
      for (int i = threadIdx.x; i < ng; i += C::kThreads) gc[i] = 0u;
      stream_merge<F, NT>(p, unit, slot0, K, ng, -1, G, scr, (int)threadIdx.x, C::kThreads, 1);
    }
    __syncthreads();
  }
  if (dev_err) atomicOr(p.err, dev_err);
}

}  // namespace
}  // namespace da
