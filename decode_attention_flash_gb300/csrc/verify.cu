// verify.cu -- drafted tokens verified against the target's probabilities (decode_attn_verify).
//
// The mathematics. Row b has n drafted tokens x_0 .. x_{n-1} with the draft's probabilities q_i and
// the target's p_0 .. p_n. Token i is accepted while u_i q_i(x_i) < p_i(x_i). At the first that is not,
// the next token is drawn from max(p_i - q_i, 0) (rejection sampling: the tokens are then distributed
// as the target's own), else from p_n. A draw takes the first token whose running sum of weights passes
// r times their sum. Running sums meet borders, so they are kept far beyond fp32: a lane adds its
// weights as pairs of floats (the rounding error of every difference and sum is carried along: 2^-45
// or so of the sum after some hundred terms), and pairs meet as doubles. Comparisons of a draft are of
// exact products of two floats in 64 bits.
//
// What bounds it. One row of p and one of q a batch row, read once: HBM, and latency for few rows.
// A cluster of CTAs takes a batch row. Every CTA finds the row's first rejection itself (a lane a
// drafted token), sums its share of the vocabulary in segments of 512, and reads the other
// CTAs' sums through the cluster; the one whose share holds the border finds its segment and looks at
// that again, from L2.
#include <algorithm>

#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 16;          // elements of a segment a lane
constexpr int kSeg = 32 * kPer;

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
__device__ __forceinline__ double load_remote(const double *p, uint32_t rank) {
  uint32_t at;
  double v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(at) : "memory");
  return v;
}

// A sum as a pair of floats.
struct Two {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  // max(p - q, 0), its rounding error with it; NaN counts as 0
  __device__ __forceinline__ void add_rest(float p, float q) {
    if (!(p > q)) return;
    const float d = __fsub_rn(p, q), b = __fsub_rn(d, p);
    lo = __fadd_rn(lo, __fsub_rn(__fsub_rn(p, __fsub_rn(d, b)), __fadd_rn(q, b)));
    add(d);
  }
};

// The rest of one token: `q` is the draft's row, or null, and then 1 for token `only` (-1: none).
struct Weights {
  const float *p, *q;
  int only, vocab;
  __device__ __forceinline__ float less(int i) const { return q ? q[i] : i == only ? 1.f : 0.f; }
};

__device__ __forceinline__ double inclusive(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// The first lane whose sum passes `border`, else the last with a weight; -1: none has one.
__device__ __forceinline__ int pick_lane(double sum, double own, double border) {
  const uint32_t past = __ballot_sync(0xffffffffu, sum > border && own > 0.0);
  if (past) return __ffs(past) - 1;
  const uint32_t some = __ballot_sync(0xffffffffu, own > 0.0);
  return some ? 31 - __clz(some) : -1;
}

// The token of a segment, by one warp: the first whose running sum passes `border`, else the last that
// has a weight.
__device__ int pick_token(const Weights &w, int seg, double border, int lane) {
  const int first = seg * kSeg + lane * kPer;
  double x[kPer], own = 0.0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int i = first + k;
    x[k] = 0.0;
    if (i < w.vocab) {
      const float a = w.p[i], b = w.less(i);
      if (a > b) x[k] = (double)a - (double)b;
    }
    own += x[k];
  }
  const double sum = inclusive(own, lane);
  const int l = pick_lane(sum, own, border);
  if (l < 0) return -1;
  int token = -1;
  double at = sum - own;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    if (x[k] > 0.0 && (token < 0 || at <= border)) token = first + k;
    at += x[k];
  }
  return __shfl_sync(0xffffffffu, token, l);
}

__device__ __forceinline__ int drafts_of(const VerifyParams &p, int b) {
  const int n = p.num_draft ? p.num_draft[b] : p.q_len - 1;
  return min(n, p.q_len - 1);
}

// Rows' lengths without their rejected tokens, and the pages that only those had back on the stack: the
// last row's first, each row's from its end. By the threads of one CTA.
__device__ void release(const VerifyParams &p, int *scan) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t err = 0;
  int64_t top = p.num_free[0];
  if (top < 0 || top > p.free_capacity) {
    err |= DA_DEVERR_NO_PAGES;
    top = top < 0 ? 0 : p.free_capacity;
  }
  for (int base = 0; base < p.batch; base += kThreads) {
    const int b = p.batch - 1 - base - (int)threadIdx.x;
    int give = 0;
    int64_t old_pages = 0, new_pages = 0;
    const int32_t *table = nullptr;
    if (b >= 0) {
      const int n = drafts_of(p, b);
      int64_t len = p.seq_lens[b];
      int64_t less = n < 0 ? 0 : n - __ldcg(p.num_accepted + b);
      if (len < less || len > p.capacity) {
        err |= DA_DEVERR_SEQ_LEN;
        less = 0;
        old_pages = new_pages = 0;
      } else {
        old_pages = (len + p.page_size - 1) / p.page_size;
        new_pages = (len - less + p.page_size - 1) / p.page_size;
      }
      p.seq_lens_out[b] = (int32_t)(len - less);
      table = p.block_table + (int64_t)b * p.max_pages;
      for (int64_t c = new_pages; c < old_pages; ++c) {
        if ((uint32_t)table[c] < (uint32_t)p.num_pages) ++give;
        else err |= DA_DEVERR_PAGE_INDEX;
      }
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
    for (int64_t c = old_pages - 1; c >= new_pages; --c) {
      const int32_t id = table[c];
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

__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
  extern __shared__ double seg_sum[];  // of this CTA's segments
  __shared__ double s_total;
  __shared__ int s_accepted, s_rejected, s_token, s_last, s_scan[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cta_rank(), ctas = (int)cluster_ctas();
  const int b = blockIdx.x / ctas, Q = p.q_len;
  begin_dependent();
  const int n = drafts_of(p, b);
  const int32_t *draft = p.draft_tokens + (int64_t)b * (Q - 1);
  uint32_t err = 0;

  // ---- the first drafted token that is not accepted, a lane each
  if (warp == 0) {
    int kept = max(n, 0);
    bool rejected = false;
    for (int base = 0; base < n; base += 32) {
      const int i = base + lane;
      bool ok = false, real = false;
      if (i < n) {
        const int x = draft[i];
        real = x >= 0 && x < p.vocab;
        if (x >= p.vocab) err |= DA_DEVERR_TOKEN;
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
        if (lane > l) err = 0;  // (tokens behind it do not matter)
        break;
      }
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
    Weights w;
    w.vocab = p.vocab;
    w.p = p.target + ((int64_t)b * Q + a) * p.target_stride;
    w.q = s_rejected && p.draft ? p.draft + ((int64_t)b * (Q - 1) + a) * p.draft_stride : nullptr;
    w.only = s_rejected && !p.draft ? draft[a] : -1;
    const int segs = (p.vocab + kSeg - 1) / kSeg;
    const int g0 = (int)((int64_t)segs * rank / ctas), ng = (int)((int64_t)segs * (rank + 1) / ctas) - g0;
    const float r = p.uniforms[(int64_t)b * Q + Q - 1];
    while (true) {
      for (int g = warp; g < ng; g += kWarps) {
        const int first = (g0 + g) * kSeg + lane;
        float x[kPer], y[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int i = first + 32 * k;
          x[k] = i < p.vocab ? w.p[i] : 0.f;
          y[k] = i < p.vocab ? w.less(i) : 0.f;
        }
        Two s;
#pragma unroll
        for (int k = 0; k < kPer; ++k) s.add_rest(x[k], y[k]);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const float hi = __shfl_xor_sync(0xffffffffu, s.hi, o), lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
          s.add(hi);
          s.lo = __fadd_rn(s.lo, lo);
        }
        if (lane == 0) seg_sum[g] = (double)s.hi + (double)s.lo;
      }
      __syncthreads();
      // a lane's segments of the CTA's, and the CTA's of the cluster's
      const int per = (ng + 31) / 32, s0 = min(lane * per, ng), s1 = min(s0 + per, ng);
      double own = 0.0, sum = 0.0;
      if (warp == 0) {
        for (int g = s0; g < s1; ++g) own += seg_sum[g];
        sum = inclusive(own, lane);
        if (lane == 31) s_total = sum;
      }
      cluster_arrive();
      cluster_wait();
      const double part = lane < ctas ? load_remote(&s_total, (uint32_t)lane) : 0.0;
      cluster_arrive();  // (nobody's sum is written again, and nobody leaves, before all have read)
      const double upto = inclusive(part, lane);
      const double total = __shfl_sync(0xffffffffu, upto, 31);
      if (!(total > 0.0 && total < 1e300)) {
        cluster_wait();
        if (w.q || w.only >= 0) {  // target and draft alike everywhere, up to rounding: the target's own
          w.q = nullptr;
          w.only = -1;
          continue;
        }
        err |= DA_DEVERR_PROBS;  // no token has a probability
        break;
      }
      const double border = (double)(r > 0.f ? r : 0.f) * total;
      const int home = pick_lane(upto, part, border);
      winner = rank == home;
      if (winner && warp == 0) {
        const double rest = border - __shfl_sync(0xffffffffu, upto - part, home);
        const int l = pick_lane(sum, own, rest);
        double at = sum - own;
        int seg = -1;
        double before = 0.0;
        for (int g = s0; g < s1; ++g) {
          if (seg_sum[g] > 0.0 && (seg < 0 || at <= rest)) {
            seg = g;
            before = at;
          }
          at += seg_sum[g];
        }
        seg = __shfl_sync(0xffffffffu, seg, l);
        before = __shfl_sync(0xffffffffu, before, l);
        const int token = pick_token(w, g0 + seg, rest - before, lane);
        if (lane == 0) s_token = token;
      }
      cluster_wait();
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
        int len = p.seq_lens[b];
        const int less = n < 0 ? 0 : n - a;
        if (len < less || len > p.capacity) err |= DA_DEVERR_SEQ_LEN;
        else len -= less;
        p.seq_lens_out[b] = len;
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

// CTAs of a cluster: as many as leave each a segment a warp.
static int verify_ctas(const VerifyParams &p) {
  if (p.target_tokens) return 1;
  int c = 8;
  while (c > 1 && (int64_t)p.vocab < (int64_t)c * kSeg * kWarps) c /= 2;
  return c;
}

cudaError_t launch_verify(const VerifyParams &p, cudaStream_t stream) {
  const int ctas = verify_ctas(p);
  const int segs = (p.vocab + kSeg - 1) / kSeg;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.batch * ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.target_tokens ? 0 : (size_t)((segs + ctas - 1) / ctas) * sizeof(double);
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
