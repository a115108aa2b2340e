// tables.cu -- block tables and slot maps from request lengths (decode_attn_build_tables).
//
// The mathematics. Row b holds old tokens and takes nw new ones: it needs
// need_b = ceil((old + nw) / P) - ceil(old / P) pages, the ones after the
// a_b = sum_{b' < b} need_b' pages that earlier rows take from the top of the
// free stack F[0 .. n): its k-th new page is F[n - 1 - (a_b + k)]. New token i of
// row b stands at position old + i, in slot page(pos / P) * P + pos % P, where the
// page is the table's for the pages that the row had and the stack's for the others
// (so no token waits for the table to be written). An id outside the pool ends the stack
// (every block looks all ids over that the rows ask for, the first kThreads of them while the
// scan runs), so a row has all of its new pages or none, and its length says which.
//
// What bounds it. A decode step moves a few KB: latency. So it is one launch,
// and no block waits for another: every block scans all rows' lengths again (two
// block scans of a few thousand integers from L2) and then writes its own share of
// the tokens, of the new table entries and (block 0) of the per-row results;
// a token finds its row by bisecting the scan, kept per thread in shared memory.
// 256 rows of one token: 5.0 us, a launch and three dependent loads (4.85 before the ids
// were looked over); 125 000 tokens of 61 rows: 8.1 us (7.5 before; four tokens a thread in fewer
// blocks took 1.9 more).
// Results written over the lengths they came from wait for the block that is last
// to have read them (a counter in the workspace, back at zero afterwards).
#include "cache_ops.h"
#include "cache_ptx.cuh"

namespace da {
namespace {

constexpr int kThreads = 512;

struct Row {
  int64_t old, nw, asked;   // cached positions, new ones that fit, new tokens asked for
  int64_t first, need;      // pages it has, pages it needs
};

// Row b, `at` tokens behind the first: those that neither its capacity nor the slot map holds
// are not among the ones that fit, so no length counts a position that nothing was written to.
__device__ __forceinline__ Row row_of(const TableParams &p, int b, int64_t at, uint32_t &err) {
  Row r;
  int64_t o = p.seq_lens[b], a = p.new_lens[b];
  if (o < 0 || o > p.capacity) {
    err |= DA_DEVERR_SEQ_LEN;
    o = o < 0 ? 0 : p.capacity;
  }
  if (a < 0) {
    err |= DA_DEVERR_SEQ_LEN;
    a = 0;
  }
  r.old = o;
  r.asked = a;
  r.nw = a;
  if (o + a > p.capacity) {
    err |= DA_DEVERR_SEQ_LEN;
    r.nw = p.capacity - o;
  }
  r.nw = max((int64_t)0, min(r.nw, p.slot_capacity - at));
  r.first = r.need = 0;
  if (p.paged) {
    const uint32_t P = (uint32_t)p.page_size;
    r.first = (uint32_t)(o + P - 1) / P;
    r.need = p.free_pages ? (uint32_t)(o + r.nw + P - 1) / P - r.first : 0;
  }
  return r;
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TableParams p) {
  __shared__ int64_t s_tok[kThreads + 1], s_pg[kThreads + 1];
  __shared__ int64_t w_tok[kThreads / 32], w_pg[kThreads / 32];
  __shared__ int64_t s_used;
  __shared__ int s_last, s_bad;  // s_bad: depth in the stack of the first id outside the pool
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.batch + kThreads - 1) / kThreads;
  const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
  uint32_t err = 0;
  wait_for_previous_kernel();
  let_next_kernel_start();
  int64_t nf = 0;
  if (p.free_pages) {
    nf = *p.num_free;
    if (nf < 0 || nf > p.free_capacity) {
      err |= DA_DEVERR_NO_PAGES;
      nf = nf < 0 ? 0 : p.free_capacity;
    }
  }
  const int top = tid < nf ? p.free_pages[nf - 1 - tid] : 0;
  if (tid == 0) {
    s_used = 0;
    s_last = 1;
    s_bad = INT32_MAX;
  }
  int64_t tok = 0, pg = 0;
  for (int b = b0; b < b1; ++b) {
    const Row r = row_of(p, b, 0, err);
    tok += r.asked;
    pg += r.need;
  }
  int64_t it = tok, ip = pg;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, it, o), y = __shfl_up_sync(0xffffffffu, ip, o);
    if (lane >= o) {
      it += x;
      ip += y;
    }
  }
  if (lane == 31) {
    w_tok[warp] = it;
    w_pg[warp] = ip;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    it += w_tok[w];
    ip += w_pg[w];
  }
  s_tok[tid + 1] = it;
  s_pg[tid + 1] = ip;
  if (tid == 0) s_tok[0] = s_pg[0] = 0;
  if ((uint32_t)top >= (uint32_t)p.num_pages && tid < nf) atomicMin(&s_bad, tid);
  __syncthreads();
  const int64_t total = s_tok[kThreads];
  if (total > p.slot_capacity) {  // fewer pages than counted: the scan again, tokens cut off
    uint32_t ignored = 0;
    int64_t at = s_tok[tid];
    ip = 0;
    for (int b = b0; b < b1; ++b) {
      const Row r = row_of(p, b, at, ignored);
      at += r.asked;
      ip += r.need;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, ip, o);
      if (lane >= o) ip += y;
    }
    if (lane == 31) w_pg[warp] = ip;
    __syncthreads();
    for (int w = 0; w < warp; ++w) ip += w_pg[w];
    s_pg[tid + 1] = ip;
    __syncthreads();
  }
  const int64_t pages = s_pg[kThreads];
  const int64_t deep = min(pages, nf);
  if (deep > kThreads) {
    constexpr int kLoads = 8;
    const int32_t *f = p.free_pages + (nf - 1);
    for (int64_t a = kThreads + tid; a < deep; a += kLoads * kThreads) {
      int id[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) id[k] = a + k * kThreads < deep ? f[-(a + k * kThreads)] : 0;
#pragma unroll
      for (int k = 0; k < kLoads; ++k)
        if ((uint32_t)id[k] >= (uint32_t)p.num_pages) atomicMin(&s_bad, (int)a + k * kThreads);
    }
    __syncthreads();
  }
  const int64_t usable = min(nf, (int64_t)s_bad);
  if (s_bad < deep) err |= DA_DEVERR_PAGE_INDEX;

  auto served = [&](int64_t ahead, int64_t need) { return need == 0 || ahead + need <= usable; };
  auto free_id = [&](int64_t a) { return p.free_pages[nf - 1 - a]; };  // the a-th page taken (of a row that is served)
  // the thread whose rows hold item i of a prefix array
  auto find = [&](const int64_t *s, int64_t i) {
    int lo = 0, hi = kThreads;
    while (hi - lo > 1) {
      const int m = (lo + hi) >> 1;
      if (s[m] <= i) lo = m;
      else hi = m;
    }
    return lo;
  };

  const int64_t stride = (int64_t)gridDim.x * kThreads, start = (int64_t)blockIdx.x * kThreads + tid;
  // ---- tokens
  for (int64_t i = start; i < p.slot_capacity; i += stride) {
    int64_t slot = -1, pos = 0;
    int row = -1;
    if (i < total) {
      const int c = find(s_tok, i);
      int64_t at = s_tok[c], ahead = s_pg[c];
      int b = c * per;
      uint32_t ignored = 0;
      Row r = row_of(p, b, at, ignored);
      while (i >= at + r.asked) {
        at += r.asked;
        ahead += r.need;
        r = row_of(p, ++b, at, ignored);
      }
      row = b;
      const int64_t k = i - at;
      pos = r.old + k;
      if (k < r.nw && served(ahead, r.need)) {
        if (!p.paged) {
          slot = (int64_t)b * p.capacity + pos;
        } else {
          const uint32_t P = (uint32_t)p.page_size, pi = (uint32_t)pos / P;
          int id;
          if (pi < r.first || !p.free_pages) {
            id = p.block_table[(int64_t)b * p.max_pages + pi];
            if (id < 0 || id >= p.num_pages) {
              err |= DA_DEVERR_PAGE_INDEX;
              id = -1;
            }
          } else {
            id = free_id(ahead + pi - r.first);
          }
          if (id >= 0) slot = (int64_t)id * P + ((uint32_t)pos - pi * P);
        }
      }
    }
    p.slot_map[i] = slot;
    if (p.positions) p.positions[i] = (int32_t)min(pos, (int64_t)INT32_MAX);
    if (p.token_row) p.token_row[i] = row;
  }
  // ---- new table entries
  for (int64_t a = start; a < pages; a += stride) {
    const int c = find(s_pg, a);
    int64_t at = s_tok[c], ahead = s_pg[c];
    int b = c * per;
    uint32_t ignored = 0;
    Row r = row_of(p, b, at, ignored);
    while (a >= ahead + r.need) {
      at += r.asked;
      ahead += r.need;
      r = row_of(p, ++b, at, ignored);
    }
    if (served(ahead, r.need)) p.block_table[(int64_t)b * p.max_pages + r.first + (a - ahead)] = free_id(a);
  }
  // ---- per-row results: block 0, or the last block to have read the lengths
  bool mine = blockIdx.x == 0;
  if (p.in_place && gridDim.x > 1) {
    __syncthreads();
    if (tid == 0) {
      s_last = atomic_add_acq_rel_gpu(p.ticket, 1u) == gridDim.x - 1;
      if (s_last) *p.ticket = 0u;
    }
    __syncthreads();
    mine = s_last != 0;
  } else {
    __syncthreads();  // this block's reads of the lengths
  }
  if (mine) {
    int64_t at = s_tok[tid], ahead = s_pg[tid], used = 0;
    for (int b = b0; b < b1; ++b) {
      const Row r = row_of(p, b, at, err);
      const bool ok = served(ahead, r.need);
      if (!ok && ahead + r.need > nf) err |= DA_DEVERR_NO_PAGES;
      if (ok && r.need > 0) used = ahead + r.need;  // (rows served without a page may stand after one refused)
      if (p.cu_new) p.cu_new[b] = (int32_t)min(at, (int64_t)INT32_MAX);
      p.seq_lens_out[b] = (int32_t)(ok ? r.old + r.nw : r.old);
      at += r.asked;
      ahead += r.need;
    }
    if (p.free_pages) atomicMax(reinterpret_cast<unsigned long long *>(&s_used), (unsigned long long)used);
    __syncthreads();
    if (tid == 0) {
      if (p.cu_new) p.cu_new[p.batch] = (int32_t)min(total, (int64_t)INT32_MAX);
      if (p.free_pages) *p.num_free_out = (int32_t)(nf - s_used);
      if (total > p.slot_capacity) err |= DA_DEVERR_SLOT;
    }
  }
  if (err) atomicOr(p.err, err);
}

}  // namespace

cudaError_t launch_tables(const TableParams &p, int num_sms, cudaStream_t stream) {
  // a token a thread, at most one block for each SM
  int64_t blocks = (p.slot_capacity + kThreads - 1) / kThreads;
  if (blocks < 1) blocks = 1;
  if (blocks > num_sms) blocks = num_sms;
  return launch_dependent(tables_kernel, (unsigned)blocks, kThreads, 0, stream, p);
}

}  // namespace da
