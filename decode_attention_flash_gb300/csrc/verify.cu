// verify.cu -- drafted tokens verified against the target's probabilities (decode_attn_verify).
//
// The mathematics. Row b has n drafted tokens x_0 .. x_{n-1} with the draft's probabilities q_i and
// the target's p_0 .. p_n. Token i is accepted while u_i q_i(x_i) < p_i(x_i). At the first that is not,
// the next token is drawn from max(p_i - q_i, 0) (rejection sampling: the tokens are then distributed
// as the target's own), else from p_n. A draw takes the first token whose running sum of weights passes
// r times their sum. Running sums meet borders, so they are kept far beyond fp32, as unevaluated pairs of
// floats: the rounding error of every difference, sum and product is computed exactly (Knuth's two-sum,
// the product's by a fused multiply) and carried along in the second float. That is an fp32 sum itself: weights
// that each round away beside a great one all land in it, and after hundreds of additions it would be off by
// 2^-36 of the sum. So it passes what it can on to the first float after the few additions of a segment, and in
// a lane's sum over its segments a third float has its rounding errors. With u = 2^-24 (a float's rounding) what is
// left is at most 100 u^2 of a segment's sum (ten additions, the second float at most ten u by then), 3 u^2 for each
// addition of two such sums, about fifteen in a row, and 40 u^2 inside the segment that is drawn from: 2^-40 of the
// sum, however the weights lie; 2^-50 of a softmax. (Doubles instead, for every token: 16 cycles of an SM for a warp's
// one addition; 82.7, 33.0 and 16.0 us for the three below; for the sums of segments alone 44.1, 15.2 and 9.9.) Two
// such sums side by side take the packed adds.
// A drafted token's product is compared exactly, in 64 bits.
//
// What bounds it. One row of p and one of q a batch row, read once: HBM, and latency for few rows.
// A cluster of CTAs takes a batch row. Every CTA finds the row's first rejection itself (a lane a
// drafted token), sums its share of the vocabulary in segments of 256, and reads the other
// CTAs' sums through the cluster; the one whose share holds the border finds its segment and looks at
// that again, from L2.
// Measured: 256 rows of 128000, four drafts each: 42 us. A row that keeps all its drafts reads no draft's
// distribution, so 175 MB there, 4.2 TB/s (floor 25.8): rows of one distribution and of two lie side by side, and an
// SM that has more of the second ends later (CTAs of 256 threads, half as many: 43 where these took 41). 64 rows of
// 151937, no draft's: 14 us from L2 (floor 5.8): 7 us a row has beside its stream (drafts, then their probabilities,
// then the sums' way through the cluster and back). 4 rows of 32000: 9.2 us, latency, 2.4 of them the pages' return (a
// count of the rows, then lengths, then table entries). Segments of 512 instead of 256: 9.5, 15.2 and 44.1 us where
// these took 8.5, 15.3 and 43.4; of 128: 8.2, 15.5 and 51.2. A warp's reduction for each segment's sum alone, not four at
// once: 16.9 and 45.
#include <algorithm>

#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;           // tokens of a segment a lane
constexpr int kTogether = 4;      // segments that a warp loads at once (of two rows half as many)
constexpr int kSeg = 32 * kPer;
constexpr int kMaxCtas = 8;       // of a cluster
constexpr int kGive = 2;          // rows of a thread that takes pages back

__device__ __forceinline__ uint32_t cta_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// An unevaluated sum of two floats.
struct Two {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void join(const Two &x) {  // (lo grows by a rounding of the sum)
    add(x.hi);
    lo = __fadd_rn(lo, x.lo);
  }
  // lo to at most half a step of hi again (it is less than hi: both are of sums without a negative term)
  __device__ __forceinline__ void tidy() {
    const float s = __fadd_rn(hi, lo);
    lo = __fsub_rn(lo, __fsub_rn(s, hi));
    hi = s;
  }
  __device__ __forceinline__ void add(const Two &x) {
    join(x);
    tidy();
  }
  // max(p - q, 0), with its rounding error; NaN counts as 0
  __device__ __forceinline__ void add_rest(float p, float q) {
    const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
    const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b));
    const bool on = p > q;
    lo = __fadd_rn(lo, on ? e : 0.f);
    add(on ? d : 0.f);
  }
  __device__ __forceinline__ bool above(const Two &x) const {
    return __fadd_rn(__fsub_rn(hi, x.hi), __fsub_rn(lo, x.lo)) > 0.f;
  }
  __device__ __forceinline__ bool positive() const { return __fadd_rn(hi, lo) > 0.f; }
  __device__ __forceinline__ bool negative() const { return __fadd_rn(hi, lo) < 0.f; }
  __device__ __forceinline__ Two minus(const Two &x) const {
    Two r = *this;
    r.add(-x.hi);
    r.lo = __fsub_rn(r.lo, x.lo);
    return r;
  }
  __device__ __forceinline__ Two times(float x) const {
    Two r;
    r.hi = __fmul_rn(hi, x);
    r.lo = fmaf(lo, x, fmaf(hi, x, -r.hi));
    return r;
  }
};
__device__ __forceinline__ Two load_remote(const float2 *p, uint32_t rank) {
  uint32_t at;
  Two v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.hi), "=f"(v.lo) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ Two shuffle(const Two &v, int lane) {
  Two r;
  r.hi = __shfl_sync(0xffffffffu, v.hi, lane);
  r.lo = __shfl_sync(0xffffffffu, v.lo, lane);
  return r;
}
__device__ __forceinline__ Two swap(const Two &v, int bit) {
  Two r;
  r.hi = __shfl_xor_sync(0xffffffffu, v.hi, bit);
  r.lo = __shfl_xor_sync(0xffffffffu, v.lo, bit);
  return r;
}
// 0 in the first `o` lanes: adding that changes nothing (a branch around the additions instead: 0.6 us)
__device__ __forceinline__ Two shuffle_up(const Two &v, int o, int lane) {
  Two r;
  r.hi = __shfl_up_sync(0xffffffffu, v.hi, o);
  r.lo = __shfl_up_sync(0xffffffffu, v.lo, o);
  r.hi = lane >= o ? r.hi : 0.f;
  r.lo = lane >= o ? r.lo : 0.f;
  return r;
}
// Sums up to this lane, itself included, of the first LANES lanes.
template <int LANES>
__device__ __forceinline__ Two inclusive(Two v, int lane) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v.add(shuffle_up(v, o, lane));
  return v;
}
// The first lane whose sum passes `border`, else the last with a weight; -1: none has one.
__device__ __forceinline__ int pick_lane(const Two &sum, const Two &own, const Two &border) {
  const uint32_t some = __ballot_sync(0xffffffffu, own.positive());
  const uint32_t past = __ballot_sync(0xffffffffu, sum.above(border)) & some;
  return past ? __ffs(past) - 1 : some ? 31 - __clz(some) : -1;
}

// Two such sums side by side.
struct TwoPairs {
  Pair hi = 0, lo = 0;
  __device__ __forceinline__ void add(Pair x) {
    const Pair s = add2(hi, x), b = sub2(s, hi);
    lo = add2(lo, add2(sub2(hi, sub2(s, b)), sub2(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void add_rest(float p0, float p1, float q0, float q1) {  // as Two::add_rest
    const Pair p = pack(p0, p1), q = pack(q0, q1);
    const Pair d = sub2(p, q), b = sub2(d, p), e = sub2(sub2(p, sub2(d, b)), add2(q, b));
    float d0, d1, e0, e1;
    unpack(d, d0, d1);
    unpack(e, e0, e1);
    lo = add2(lo, pack(d0 > 0.f ? e0 : 0.f, d1 > 0.f ? e1 : 0.f));
    add(pack(fmaxf(d0, 0.f), fmaxf(d1, 0.f)));
  }
  __device__ __forceinline__ Two both() const {
    Two a, b;
    unpack(hi, a.hi, b.hi);
    unpack(lo, a.lo, b.lo);
    a.join(b);
    return a;
  }
};

// A vocabulary's weights max(p - q, 0): q is a row of the draft's, or (null) 1 for token `only` and else 0.
// Segments begin `shift` elements before the row, where p is 16-byte aligned.
struct Rows {
  const float *p, *q;
  int only, vocab, shift;
};
// Tokens 128 k + 4 lane + j (VEC: 16-byte loads) or 128 k + 32 j + lane of a row's segment: in any order, for
// sums; outside the vocabulary 0.
template <bool VEC>
__device__ __forceinline__ void load_segment(const float *row, int first, int vocab, int lane, float (&x)[kPer]) {
  if (first >= 0 && first + kSeg <= vocab) {
#pragma unroll
    for (int k = 0; k < kPer / 4; ++k) {
      if (VEC) {
        const float4 a = reinterpret_cast<const float4 *>(row + first)[32 * k + lane];
        x[4 * k] = a.x, x[4 * k + 1] = a.y, x[4 * k + 2] = a.z, x[4 * k + 3] = a.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * k + j] = row[first + 128 * k + 32 * j + lane];
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = first + 128 * (k >> 2) + (VEC ? 4 * lane + (k & 3) : 32 * (k & 3) + lane);
      x[k] = i >= 0 && i < vocab ? row[i] : 0.f;
    }
  }
}
// The certain draft's token, where a segment that begins at `first` has it: 1 less (above 0 only past 1,
// where it is exact).
__device__ __forceinline__ void less_certain(const Rows &w, int first, int lane, float (&x)[kPer]) {
  const int i = w.only - first;
  if (w.only < 0 || i < 0 || i >= kSeg) return;  // (the same for every lane)
  const int at = (i >> 2 & 31) == lane ? (i >> 7) * 4 + (i & 3) : -1;
#pragma unroll
  for (int k = 0; k < kPer; ++k) x[k] = k == at ? x[k] - 1.f : x[k];
}
// A CTA's segments, a warp each in turn: their sums, kAt segments at a time. DRAFT: q is a row; VEC: and
// aligned where p is.
template <bool DRAFT, bool VEC>
__device__ __forceinline__ void sum_segments(const Rows &w, int g0, int ng, int warp, int lane, float2 *sums) {
  constexpr int kAt = DRAFT ? kTogether / 2 : kTogether;
#pragma unroll 1
  for (int g = warp; g < ng; g += kAt * kWarps) {
    float x[kAt][kPer], y[kAt][kPer];
#pragma unroll
    for (int a = 0; a < kAt; ++a) {
      // (past the CTA's share: loaded as a segment past the vocabulary, zeros)
      const int first = g + a * kWarps < ng ? (g0 + g + a * kWarps) * kSeg - w.shift : w.vocab;
      load_segment<VEC>(w.p, first, w.vocab, lane, x[a]);
      if (DRAFT) load_segment<VEC>(w.q, first, w.vocab, lane, y[a]);
    }
    Two s[kAt];
#pragma unroll
    for (int a = 0; a < kAt; ++a) {
      TwoPairs s2;
      if (!DRAFT) less_certain(w, (g0 + g + a * kWarps) * kSeg - w.shift, lane, x[a]);
#pragma unroll
      for (int k = 0; k < kPer; k += 2) {
        if (DRAFT) s2.add_rest(x[a][k], x[a][k + 1], y[a][k], y[a][k + 1]);
        else s2.add(pack(fmaxf(x[a][k], 0.f), fmaxf(x[a][k + 1], 0.f)));  // (NaN counts as 0)
      }
      s[a] = s2.both();
    }
    // The segments' sums over the lanes: half of the sums go to the neighbour in each of the first steps, so
    // that lane i (of the first kAt) ends with segment `mine`: 6 additions for four sums, not 20.
    int mine = 0;
    if constexpr (kAt == 4) {
      const bool odd = lane & 1;
      const Two u = swap(odd ? s[0] : s[2], 1), v = swap(odd ? s[1] : s[3], 1);
      s[0] = odd ? s[2] : s[0];
      s[1] = odd ? s[3] : s[1];
      s[0].join(u);
      s[1].join(v);
      mine = 2 * (lane & 1);
    }
    constexpr int kHalve = kAt / 2;  // the lane bit that parts the last two sums
    {
      const bool up = lane & kHalve;
      const Two u = swap(up ? s[0] : s[1], kHalve);
      s[0] = up ? s[1] : s[0];
      s[0].join(u);
      mine += up ? 1 : 0;
    }
#pragma unroll
    for (int o = kAt; o < 32; o <<= 1) s[0].join(swap(s[0], o));
    s[0].tidy();
    if (lane < kAt && g + mine * kWarps < ng) sums[g + mine * kWarps] = make_float2(s[0].hi, s[0].lo);
  }
}

// The token of a segment, by one warp: the first whose running sum passes `border`, else the last that
// has a weight; -1: none has. Lane by lane four tokens of each 128.
__device__ __forceinline__ int pick_token(const Rows &w, int seg, Two border, int lane) {
  const int first = seg * kSeg - w.shift;
  float x[kPer], y[kPer];
  load_segment<true>(w.p, first, w.vocab, lane, x);
  if (!w.q) {
    less_certain(w, first, lane, x);
#pragma unroll
    for (int k = 0; k < kPer; ++k) y[k] = 0.f;
  } else {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int i = first + 128 * (k >> 2) + 4 * lane + (k & 3);
      y[k] = i >= 0 && i < w.vocab ? w.q[i] : 0.f;
    }
  }
  constexpr int kGroups = kPer / 4;
  Two own[kGroups], sum[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
#pragma unroll
    for (int j = 0; j < 4; ++j) own[g].add_rest(x[4 * g + j], y[4 * g + j]);
    sum[g] = own[g];
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int g = 0; g < kGroups; ++g) sum[g].add(shuffle_up(sum[g], o, lane));
  // the group: the last with a weight whose tokens begin at or below the border
  int token = -1;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const Two all = shuffle(sum[g], 31);
    if (all.positive() && (token < 0 || !border.negative())) {
      const int l = pick_lane(sum[g], own[g], border);
      Two at = sum[g].minus(own[g]);
      int mine = -1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (x[4 * g + j] > y[4 * g + j] && (mine < 0 || !at.above(border))) mine = first + 128 * g + 4 * lane + j;
        at.add_rest(x[4 * g + j], y[4 * g + j]);
      }
      token = __shfl_sync(0xffffffffu, mine, l);
    }
    border = border.minus(all);
  }
  return token;
}

// A row's drafted tokens, -1 if it takes no part: its caller says so, or it got fewer tokens in this step than its
// known one and the drafts (those that it got stood where other query tokens' masks apply, or nowhere). That test
// gives the same again after the row's length has been written over either of the two that it compares.
__device__ __forceinline__ int drafts_of(const VerifyParams &p, int b) {
  const int n = min(p.num_draft ? p.num_draft[b] : p.q_len - 1, p.q_len - 1);
  if (!p.seq_lens_before) return n;
  const int len = p.seq_lens[b], before = p.seq_lens_before[b];
  return before < 0 || before > len || len - before <= n ? -1 : n;
}
// A row's length after the step, and its length `len` with the step's tokens in; n and kept of its drafts. A row that
// takes no part because it got fewer tokens goes back to what it had. False: a length out of range, left as it is.
__device__ __forceinline__ bool length_after(const VerifyParams &p, int b, int n, int kept, int &len, int &after) {
  int before = len = p.seq_lens[b];
  const bool asked = !p.num_draft || p.num_draft[b] >= 0;
  if (p.seq_lens_before && asked) before = p.seq_lens_before[b];
  after = n >= 0 ? len - (n - kept) : before;
  const bool ok = before >= 0 && before <= len && after >= 0 && len <= p.capacity;
  if (!ok) after = len;
  return ok;
}

// Rows' lengths without their rejected tokens, and the pages that only those had back on the stack: the
// last row's first, each row's from its end. By the threads of one CTA.
__device__ __forceinline__ void release(const VerifyParams &p, int *scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t err = 0;
  int64_t top = p.num_free[0];
  if (top < 0 || top > p.free_capacity) {
    err |= DA_DEVERR_NO_PAGES;
    top = top < 0 ? 0 : p.free_capacity;
  }
  // a thread has up to kGive rows that follow one another, whose loads are in flight together
  const int per = min((p.batch + kThreads - 1) / kThreads, kGive);
  for (int base = 0; base < p.batch; base += kThreads * per) {
    int give = 0, before[kGive], after[kGive], row[kGive];  // pages of a row with and without its rejected tokens
#pragma unroll
    for (int j = 0; j < kGive; ++j) {
      const int b = p.batch - 1 - base - (int)threadIdx.x * per - j;
      row[j] = j < per && b >= 0 ? b : -1;
      before[j] = after[j] = 0;
      if (row[j] < 0) continue;
      int len, left;
      if (!length_after(p, b, drafts_of(p, b), __ldcg(p.num_accepted + b), len, left)) {
        err |= DA_DEVERR_SEQ_LEN;
      } else {
        before[j] = (int)(((int64_t)len + p.page_size - 1) / p.page_size);
        after[j] = (int)(((int64_t)left + p.page_size - 1) / p.page_size);
      }
      p.seq_lens_out[b] = left;
    }
#pragma unroll
    for (int j = 0; j < kGive; ++j)
      for (int c = after[j]; c < before[j]; ++c) {
        if ((uint32_t)p.block_table[(int64_t)row[j] * p.max_pages + c] < (uint32_t)p.num_pages) ++give;
        else err |= DA_DEVERR_PAGE_INDEX;
      }
    int sum = give;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    int all = 0;
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) sum += scan[k];
      all += scan[k];
    }
    int64_t at = top + sum - give;
#pragma unroll
    for (int j = 0; j < kGive; ++j)
      for (int c = before[j] - 1; c >= after[j]; --c) {
        const int32_t id = p.block_table[(int64_t)row[j] * p.max_pages + c];
        if ((uint32_t)id >= (uint32_t)p.num_pages) continue;
        if (at < p.free_capacity) p.free_pages[at] = id;
        else err |= DA_DEVERR_NO_PAGES;
        ++at;
      }
    top += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) p.num_free_out[0] = (int32_t)min(top, (int64_t)p.free_capacity);
  if (err) atomicOr(p.err, err);
}

__global__ void __launch_bounds__(kThreads, 8) verify_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ float2 seg_sum[];  // of this CTA's segments
  __shared__ float2 s_total;
  __shared__ int s_accepted, s_rejected, s_token, s_home, s_last, s_scan[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cta_rank(), ctas = (int)cluster_ctas();
  const int b = blockIdx.x / ctas, Q = p.q_len;
  begin_dependent();
  const int32_t *draft = p.draft_tokens + (int64_t)b * (Q - 1);
  const int n = drafts_of(p, b);
  uint32_t err = 0;

  // ---- the first drafted token that is not accepted, a lane each (the lanes do not wait for n to load
  // their token's probabilities)
  if (warp == 0) {
    int kept = max(n, 0);
    bool rejected = false;
    for (int base = 0; base < Q - 1; base += 32) {
      const int i = base + lane;
      bool ok = false, real = false, past = false;
      if (i < Q - 1) {
        const int x = draft[i];
        past = x >= p.vocab;
        real = x >= 0 && !past;
        if (real && p.target_tokens) {
          ok = p.target_tokens[(int64_t)b * Q + i] == x;
        } else if (real) {
          const float t = p.target[((int64_t)b * Q + i) * p.target_stride + x];
          const float d = p.draft ? p.draft[((int64_t)b * (Q - 1) + i) * p.draft_stride + x] : 1.f;
          ok = (double)p.uniforms[(int64_t)b * Q + i] * (double)d < (double)t;
        }
      }
      const uint32_t no = __ballot_sync(0xffffffffu, i < n && !ok);
      if (no) {
        const int l = __ffs(no) - 1;
        kept = base + l;
        rejected = __shfl_sync(0xffffffffu, (int)real, l) != 0;  // (padding ends the drafts, rejecting none)
        if (lane == l && past) err |= DA_DEVERR_TOKEN;
        break;
      }
      if (base + 32 >= n) break;
    }
    if (lane == 0) {
      s_accepted = kept;
      s_rejected = rejected;
      s_token = -1;
    }
  }
  __syncthreads();
  const int a = s_accepted;
  bool winner = rank == 0;
  if (n >= 0 && p.target_tokens) {
    if (threadIdx.x == 0) s_token = p.target_tokens[(int64_t)b * Q + a];
  } else if (n >= 0) {
    // ---- the next token
    Rows w;
    w.vocab = p.vocab;
    w.p = p.target + ((int64_t)b * Q + a) * p.target_stride;
    w.q = s_rejected && p.draft ? p.draft + ((int64_t)b * (Q - 1) + a) * p.draft_stride : nullptr;
    w.only = s_rejected && !p.draft ? draft[a] : -1;
    w.shift = (int)(reinterpret_cast<uintptr_t>(w.p) >> 2) & 3;
    const int segs = (p.vocab + w.shift + kSeg - 1) / kSeg;
    const int g0 = (int)((int64_t)segs * rank / ctas), ng = (int)((int64_t)segs * (rank + 1) / ctas) - g0;
    const float r = p.uniforms[(int64_t)b * Q + Q - 1];
    while (true) {
      if (!w.q) sum_segments<false, true>(w, g0, ng, warp, lane, seg_sum);
      else if ((((reinterpret_cast<uintptr_t>(w.p) ^ reinterpret_cast<uintptr_t>(w.q)) >> 2) & 3) == 0)
        sum_segments<true, true>(w, g0, ng, warp, lane, seg_sum);
      else sum_segments<true, false>(w, g0, ng, warp, lane, seg_sum);
      __syncthreads();
      // a lane's segments of the CTA's, and the CTA's of the cluster's
      const int per = (ng + 31) / 32, s0 = min(lane * per, ng), s1 = min(s0 + per, ng);
      Two own, sum;
      if (warp == 0) {
        Two low;  // own's second float, kept as a sum of its own
        for (int g = s0; g < s1; ++g) {
          own.lo = 0.f;
          own.add(seg_sum[g].x);
          low.add(own.lo);
          low.add(seg_sum[g].y);
        }
        own.lo = __fadd_rn(low.hi, low.lo);
        own.tidy();
        sum = inclusive<32>(own, lane);
        if (lane == 31) s_total = make_float2(sum.hi, sum.lo);
      }
      cluster_arrive();
      cluster_wait();
      if (warp == 0) {
        Two part;
        if (lane < ctas) part = load_remote(&s_total, (uint32_t)lane);
        const Two upto = inclusive<kMaxCtas>(part, lane), total = shuffle(upto, ctas - 1);
        const Two border = total.times(r > 0.f ? r : 0.f);
        const bool some = total.hi > 0.f && total.hi < __int_as_float(0x7f800000);
        const int home = some ? pick_lane(upto, part, border) : -1;
        if (home == rank) {
          const Two rest = border.minus(shuffle(upto.minus(part), home));
          const int l = pick_lane(sum, own, rest), a1 = min(l * per + per, ng);
          Two at = shuffle(sum.minus(own), l), before;
          int seg = -1;
          for (int a = l * per; a < a1; a += 32) {  // that lane's segments, a lane each
            Two x;
            if (a + lane < a1) x.hi = seg_sum[a + lane].x, x.lo = seg_sum[a + lane].y;
            Two upto_it = x;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              if (o >= per) break;
              upto_it.add(shuffle_up(upto_it, o, lane));
            }
            upto_it.add(at);
            const int j = pick_lane(upto_it, x, rest);
            if (j >= 0) {
              seg = a + j;
              before = shuffle(upto_it.minus(x), j);
              if (shuffle(upto_it, j).above(rest)) break;
            }
            at = shuffle(upto_it, 31);
          }
          const int token = pick_token(w, g0 + seg, rest.minus(before), lane);
          if (lane == 0) s_token = token;
        }
        if (lane == 0) s_home = home;
      }
      cluster_arrive();  // (nobody's sum is written again, and nobody leaves, before all have read)
      cluster_wait();
      const int home = s_home;
      winner = rank == max(home, 0);
      if (home < 0 && (w.q || w.only >= 0)) {  // target and draft alike everywhere, up to rounding: the target's own
        w.q = nullptr;
        w.only = -1;
        continue;
      }
      if (home < 0) err |= DA_DEVERR_PROBS;  // no token has a probability
      break;
    }
  }
  __syncthreads();
  // ---- outputs, by the CTA that has the token
  if (winner) {
    for (int j = threadIdx.x; j < Q; j += kThreads)
      p.tokens_out[(int64_t)b * Q + j] = n < 0 || j > a ? -1 : j < a ? draft[j] : s_token;
    if (threadIdx.x == 0) {
      p.num_accepted[b] = a;
      if (p.seq_lens && !p.free_pages) {
        int len, left;
        if (!length_after(p, b, n, a, len, left)) err |= DA_DEVERR_SEQ_LEN;
        p.seq_lens_out[b] = left;
      }
    }
    if (err && warp == 0) atomicOr(p.err, err);
    if (!p.free_pages) return;
    if (threadIdx.x == 0) {
      s_last = atomic_add_acq_rel_gpu(p.ticket, 1u) == (unsigned)p.batch - 1;
      if (s_last) *p.ticket = 0u;
    }
    __syncthreads();
    if (s_last) release(p, s_scan);
  }
}

}  // namespace

// CTAs of a cluster: as many as the SMs hold at once (eight each) and as leave each half a segment a warp.
// 256 rows of 128000: four CTAs a row 42 us; with the sums before these 41, two 52, eight 44. The sums of a CTA's segments fit 40 KB.
static int verify_ctas(const VerifyParams &p, int num_sms) {
  if (p.target_tokens) return 1;
  int c = kMaxCtas;
  const int segs = (p.vocab + 3 + kSeg - 1) / kSeg;
  while (c > 1 && segs / (c / 2) < 5000 && ((int64_t)p.batch * c > num_sms * 8 || (int64_t)p.vocab < (int64_t)c * kSeg * kWarps / 2)) c /= 2;
  return c;
}

cudaError_t launch_verify(const VerifyParams &p, int num_sms, cudaStream_t stream) {
  const int ctas = verify_ctas(p, num_sms);
  const int segs = (p.vocab + 3 + kSeg - 1) / kSeg;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.target_tokens ? 0 : (size_t)((segs + ctas - 1) / ctas) * sizeof(float2);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_kernel, p);
}

}  // namespace da
