// pages.cu -- page bookkeeping on the GPU: block tables, slot maps and prefix
// sums of a step built from its requests' lengths (hb_pages_assign), and the
// pages of finished requests put back (hb_pages_release).
//
// "In-flight Batching", §KV Cache 管理的协同优化: fixed-size pages that a block
// table maps, handed out as a sequence grows and freed when it finishes.  The
// host builder (builder.cpp) keeps that list on the host; here it is a ring
// of page ids in device memory, so that tables and appends need no trip to the
// host, in a captured graph either (an attention's plan takes the lengths there).
//
// The mathematics is two prefix sums over the sequences: cu[s], the new
// tokens before s, and pg[s], the new pages before s, where s takes pages
// first .. last-1 with first = ceil((ctx - q) / 16), last = ceil(ctx / 16).
// Then everything is a direct lookup: logical page lp >= first of s is ring
// entry head + pg[s] + lp - first, and token t of s sits at position
// ctx - q + t - cu[s].  So no CTA reads what another one writes: each CTA
// stages the lengths in shared memory, takes both sums for itself (a few
// microseconds at thousands of sequences, far less than a second launch or a
// grid-wide wait) and then writes its share of the tokens and of the pages.
//
// The ring's head and tail may be read and written in place: every CTA reads
// them first, then counts itself in (in the state's third entry); the last one
// to do so writes them back.  Into another array the first CTA writes them.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>

#include "hb.h"
#include "hb_internal.h"
#include "ptx.cuh"

namespace hb {

hb_status internal_fail(hb_status s, const char* msg);
hb_status internal_ok();
hb_status internal_device(int** err, int* num_sms);
void internal_count_launch();
void internal_note_other_launch(void* stream);

namespace {

constexpr int kPagesThreads = 512;
constexpr int kSeg = 8;                   // released pages per thread and pass
constexpr int kPagesMaxSeqs = 16384;      // three int32 per sequence in shared memory

struct PagesParams {
  const int32_t* q_len;
  const int32_t* ctx;                     // context lengths, or lengths to release
  int32_t num_seqs, max_tokens, max_pages_per_seq, num_pages;
  const int64_t* state_in;
  int64_t* state_out;
  int32_t* ring;
  int32_t* block_table;
  int32_t* cu_q_len;
  int64_t* slot_map;
  int* dev_error;
};

// What the sums need and give: s_q[s] becomes cu[s], s_pg[s] becomes pg[s]
// (both with the total at [S]); s_off[s] = ctx - q.  Returns 0, or the error
// for lengths outside 0 <= q <= ctx <= table room (which every CTA finds
// alike, so that nothing is written then).
struct Sums {
  int32_t *s_q, *s_pg, *s_off;
  int64_t tokens, pages;
};

__device__ int prefix_sums(const PagesParams& p, Sums& a, int64_t* s_state) {
  __shared__ int64_t w_q[kPagesThreads / 32], w_pg[kPagesThreads / 32];
  const int S = p.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t room = (int64_t)p.max_pages_per_seq * kPageSize;
  int bad = 0;
  // (the ring's state arrives with the lengths)
  longlong2 state = make_longlong2(0, 0);
  if (tid == 0) state = make_longlong2(__ldcg(p.state_in), __ldcg(p.state_in + 1));
  for (int s = tid; s < S; s += kPagesThreads) {
    const int ctx = __ldcg(p.ctx + s);
    const int q = __ldcg(p.q_len + s);
    if (q < 0 || ctx < q || ctx > room) {
      bad = 1;
      continue;
    }
    const int off = ctx - q;
    a.s_q[s] = q;
    // (in 64 bits: a length near 2^31 must not wrap)
    a.s_pg[s] = (int32_t)(((int64_t)ctx + kPageSize - 1) / kPageSize -
                          ((int64_t)off + kPageSize - 1) / kPageSize);
    a.s_off[s] = off;
  }
  if (tid == 0) {
    s_state[0] = state.x;
    s_state[1] = state.y;
    s_state[2] = state.x % p.num_pages;   // where the ring's next page to take stands
  }
  if (__syncthreads_or(bad)) return HB_DEVERR_LENGTHS;
  // each thread sums a run of sequences, the block scans the runs
  const int per = (S + kPagesThreads - 1) / kPagesThreads;
  const int s0 = min(S, tid * per), s1 = min(S, s0 + per);
  int64_t q = 0, pg = 0;
  for (int s = s0; s < s1; ++s) {
    q += a.s_q[s];
    pg += a.s_pg[s];
  }
  int64_t iq = q, ipg = pg;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, iq, d), y = __shfl_up_sync(0xffffffffu, ipg, d);
    if (lane >= d) {
      iq += x;
      ipg += y;
    }
  }
  if (lane == 31) {
    w_q[warp] = iq;
    w_pg[warp] = ipg;
  }
  __syncthreads();
  int64_t bq = 0, bpg = 0, tq = 0, tpg = 0;
#pragma unroll
  for (int w = 0; w < kPagesThreads / 32; ++w) {
    if (w < warp) {
      bq += w_q[w];
      bpg += w_pg[w];
    }
    tq += w_q[w];
    tpg += w_pg[w];
  }
  a.tokens = tq;
  a.pages = tpg;
  // sums past 32 bits are refused by the caller, so what is stored fits
  if (tq > INT_MAX || tpg > INT_MAX) return HB_DEVERR_LENGTHS;
  int32_t rq = (int32_t)(bq + iq - q), rpg = (int32_t)(bpg + ipg - pg);
  for (int s = s0; s < s1; ++s) {
    const int32_t x = a.s_q[s], y = a.s_pg[s];
    a.s_q[s] = rq;
    a.s_pg[s] = rpg;
    rq += x;
    rpg += y;
  }
  if (tid == 0) {
    a.s_q[S] = (int32_t)tq;
    a.s_pg[S] = (int32_t)tpg;
  }
  __syncthreads();
  return 0;
}

// the largest s in 0 .. S-1 with sums[s] <= x (x below the total: the
// sequence that owns x, empty ones skipped)
__device__ __forceinline__ int owner(const int32_t* sums, int S, int x) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (sums[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Head and tail as the launch found them (s_state) moved by `dh` / `dt`,
// written by the last CTA to have read them, or to another array by the first.
// Called by one thread of each CTA.
__device__ void write_state(const PagesParams& p, const int64_t* s_state, int64_t dh, int64_t dt) {
  bool last = blockIdx.x == 0;
  if (gridDim.x > 1 && p.state_out == p.state_in) {
    __threadfence();
    last = atomicAdd(reinterpret_cast<unsigned long long*>(p.state_out + 2), 1ull) + 1ull == gridDim.x;
    __threadfence();
  }
  if (last) {
    p.state_out[0] = s_state[0] + dh;
    p.state_out[1] = s_state[1] + dt;
    p.state_out[2] = 0;
    p.state_out[3] = 0;
  }
}

// kRun: tokens per thread and pass (slots).  One where a thread per token is
// at hand (256 decodes: 4.3 us, with four 5.6), four for more (129053 tokens
// of 1053 rows: 8.0 us, with one 8.3; both 0.2 to 0.9 less since the state
// needs no count where it is written elsewhere).
template <int kRun>
__global__ void __launch_bounds__(kPagesThreads) pages_assign_kernel(const PagesParams p) {
  extern __shared__ int32_t s_dyn[];
  __shared__ int64_t s_state[3];
  griddep_wait();
  griddep_launch_dependents();
  const int S = p.num_seqs;
  Sums a{s_dyn, s_dyn + S + 1, s_dyn + 2 * (S + 1), 0, 0};
  int err = prefix_sums(p, a, s_state);
  const int64_t head = s_state[0], tail = s_state[1];
  if (!err && (head < 0 || tail < head || tail - head > p.num_pages || a.tokens > p.max_tokens))
    err = HB_DEVERR_LENGTHS;
  const bool lengths_ok = !err;
  if (!err && a.pages > tail - head) err = HB_DEVERR_PAGES;
  if (threadIdx.x == 0) write_state(p, s_state, err ? 0 : a.pages, 0);
  if (err && blockIdx.x == 0 && threadIdx.x == 0) report_error(p.dev_error, err);

  const int lane = threadIdx.x & 31;
  const int64_t first_thread = (int64_t)blockIdx.x * kPagesThreads + threadIdx.x;
  const int64_t step = (int64_t)gridDim.x * kPagesThreads;
  if (!lengths_ok) {
    // a batch without tokens: the sums and slots of the step before, with this
    // step's lengths, would send an append behind this call to other places
    // (entry 0 is only read, so the CTAs need not agree on when)
    const int c0 = __ldcg(p.cu_q_len);
    for (int64_t s = first_thread + 1; s <= S; s += step) p.cu_q_len[s] = c0;
    if (p.slot_map)
      for (int64_t t = first_thread; t < p.max_tokens; t += step)
        if (__ldcg(p.slot_map + t) >= 0) p.slot_map[t] = -1;
    return;
  }
  const int64_t first_warp = first_thread >> 5, warps = step / 32;
  for (int64_t s = first_thread; s <= S; s += step) p.cu_q_len[s] = S > 0 ? a.s_q[s] : 0;
  if (S == 0) return;
  const int32_t* cu = a.s_q;
  // the entry of the k-th page to take
  auto entry = [&](int64_t k) -> int32_t* {
    const int s = owner(a.s_pg, S, (int)k);
    const int lp = (a.s_off[s] + kPageSize - 1) / kPageSize + (int)k - a.s_pg[s];
    return p.block_table + (size_t)s * p.max_pages_per_seq + lp;
  };
  if (err) {
    // too few pages: no token has a slot, and no entry that was to be filled
    // may name a page -- what a finished request left there can be another
    // sequence's by now, and an append behind this call would write to it
    for (int64_t k = first_thread; k < a.pages; k += step) {
      int32_t* at = entry(k);
      if ((unsigned)__ldcg(at) < (unsigned)p.num_pages) *at = -1;
    }
    if (p.slot_map)
      for (int64_t t = first_thread; t < a.tokens; t += step) p.slot_map[t] = -1;
    return;
  }
  const int64_t at0 = s_state[2];
  // ring entry k past the head (k below the pages taken, so at most one wrap)
  auto fresh_page = [&](int64_t k) -> int {
    int64_t i = at0 + k;
    if (i >= p.num_pages) i -= p.num_pages;
    const int page = __ldcg(p.ring + i);
    return (unsigned)page < (unsigned)p.num_pages ? page : -1;
  };
  // table entries of the pages taken
  for (int64_t k = first_thread; k < a.pages; k += step) {
    const int page = fresh_page(k);
    if (page < 0) report_error(p.dev_error, HB_DEVERR_INDEX);
    *entry(k) = page;
  }
  if (!p.slot_map) return;
  // slots: a warp takes 32 kRun consecutive tokens, 32 at a time so that what
  // it reads and writes lies together; a lane searches again only where its
  // next token has left the sequence.  Where each page id stands is found
  // first, so that a lane's loads are in flight together.
  const int32_t tokens = (int32_t)a.tokens, h0 = (int32_t)at0;
  for (int64_t tt = first_warp * 32 * kRun + lane; tt < tokens; tt += warps * 32 * kRun) {
    const int32_t* src[kRun];
    int in_page[kRun], page[kRun];
    int s = owner(cu, S, (int)tt);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const int t = (int)min(tt + 32 * j, (int64_t)tokens - 1);
      if (cu[s + 1] <= t) s = owner(cu, S, t);
      const int off = a.s_off[s];
      const int pos = off + t - cu[s];
      const int lp = pos / kPageSize, first = (off + kPageSize - 1) / kPageSize;
      int64_t k = (int64_t)h0 + a.s_pg[s] + lp - first;
      if (k >= p.num_pages) k -= p.num_pages;
      src[j] = lp >= first ? p.ring + k : p.block_table + (size_t)s * p.max_pages_per_seq + lp;
      in_page[j] = pos % kPageSize;
    }
#pragma unroll
    for (int j = 0; j < kRun; ++j) page[j] = __ldcg(src[j]);
    bool bad = false;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool in = (unsigned)page[j] < (unsigned)p.num_pages;
      bad |= !in;
      if (tt + 32 * j < tokens)
        p.slot_map[tt + 32 * j] = in ? (int64_t)page[j] * kPageSize + in_page[j] : -1;
    }
    if (bad) report_error(p.dev_error, HB_DEVERR_INDEX);
  }
}

// A CTA takes a group of rows (all of them in `groups` groups; where rows are
// few, `slices` CTAs share one) and needs of the sums only the pages of the
// rows before, so it adds those up and keeps no more than its own rows'.
// 2047 rows of up to 1024 pages: 6.9 us a call, with the sums of all rows in
// every CTA 11.2; 5 rows: 3 us of device time, the call's own 6 us.
__global__ void __launch_bounds__(kPagesThreads) pages_release_kernel(const PagesParams p,
                                                                      const int groups, const int slices) {
  extern __shared__ int32_t s_n[];      // pages of the group's rows
  __shared__ int64_t s_state[3];
  __shared__ int64_t w_before[kPagesThreads / 32], w_all[kPagesThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int S = p.num_seqs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int group = (int)blockIdx.x % groups, slice = (int)blockIdx.x / groups;
  const int r0 = (int)((int64_t)S * group / groups), r1 = (int)((int64_t)S * (group + 1) / groups);
  const int64_t room = (int64_t)p.max_pages_per_seq * kPageSize;
  int bad = 0;
  // (the ring's state arrives with the lengths)
  longlong2 state = make_longlong2(0, 0);
  if (tid == 0) state = make_longlong2(__ldcg(p.state_in), __ldcg(p.state_in + 1));
  int64_t before = 0, all = 0;
  for (int s = tid; s < S; s += kPagesThreads) {
    const int len = __ldcg(p.ctx + s);
    if (len < 0 || len > room) {
      bad = 1;
      continue;
    }
    // (without adding to a length near 2^31)
    const int n = len / kPageSize + (len % kPageSize ? 1 : 0);
    all += n;
    if (s < r0) before += n;
    else if (s < r1) s_n[s - r0] = n;
  }
  // (below 2^32: at most 32 lengths a thread, 2^27 pages each; the sum of a
  // warp is taken of 16 bits at a time)
  const auto warp_sum = [](int64_t v) {
    return (int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(v & 0xffff)) +
           ((int64_t)__reduce_add_sync(0xffffffffu, (uint32_t)(v >> 16)) << 16);
  };
  before = warp_sum(before);
  all = warp_sum(all);
  if (lane == 0) {
    w_before[warp] = before;
    w_all[warp] = all;
  }
  if (tid == 0) {
    s_state[0] = state.x;
    s_state[1] = state.y;
    s_state[2] = state.y % p.num_pages;   // where the ring's next page to put in stands
  }
  int err = __syncthreads_or(bad) ? HB_DEVERR_LENGTHS : 0;
  before = all = 0;
#pragma unroll
  for (int w = 0; w < kPagesThreads / 32; ++w) {
    before += w_before[w];
    all += w_all[w];
  }
  const int64_t head = s_state[0], tail = s_state[1];
  if (!err && (head < 0 || tail < head || tail - head > p.num_pages || all > p.num_pages - (tail - head)))
    err = HB_DEVERR_LENGTHS;
  if (err && blockIdx.x == 0 && tid == 0) report_error(p.dev_error, err);
  // (by a thread of the warp that has the fewest rows to move)
  if (tid == kPagesThreads - 32) write_state(p, s_state, 0, err ? 0 : all);
  if (err) return;
  const int64_t at0 = s_state[2] + before;
  // a warp takes up to 32 kSeg pages of one row at a time: what it reads and
  // what it writes are runs, and its loads are in flight together
  const int segs = (p.max_pages_per_seq + 32 * kSeg - 1) / (32 * kSeg);
  const int mine = (segs - slice + slices - 1) / slices;   // segments slice, slice + slices, ..
  const int rows = r1 - r0;
  for (int t = warp; t < rows * mine; t += kPagesThreads / 32) {
    // (segment-major: rows of one length fill the warps evenly)
    const int i = t % rows, seg = slice + t / rows * slices, n = s_n[i];
    const int lp0 = seg * 32 * kSeg + lane;
    if (seg * 32 * kSeg >= n) continue;
    const int32_t* row = p.block_table + (size_t)(r0 + i) * p.max_pages_per_seq;
    int page[kSeg];
#pragma unroll
    for (int j = 0; j < kSeg; ++j) page[j] = lp0 + 32 * j < n ? __ldcg(row + lp0 + 32 * j) : 0;
    int k0 = 0;   // pages of the group's rows before this one (all of them fit the ring)
    for (int x = lane; x < i; x += 32) k0 += s_n[x];
    k0 = __reduce_add_sync(0xffffffffu, k0);
    bool out = false;
#pragma unroll
    for (int j = 0; j < kSeg; ++j) {
      const bool there = lp0 + 32 * j < n;
      if ((unsigned)page[j] >= (unsigned)p.num_pages) {
        out = true;
        page[j] = -1;   // found again by the call that would hand it out
      }
      int64_t at = at0 + k0 + lp0 + 32 * j;
      if (at >= p.num_pages) at -= p.num_pages;
      if (there) p.ring[at] = page[j];
    }
    if (out) report_error(p.dev_error, HB_DEVERR_INDEX);
  }
}

hb_status check_common(int32_t num_seqs, int32_t max_pages_per_seq, int32_t num_pages, int32_t page_size,
                       const void* lens, const void* ring, const void* state_in, const void* state_out,
                       const void* block_table) {
  if (num_seqs < 0) return internal_fail(HB_ERR_SHAPE, "num_seqs must be >= 0");
  if (num_seqs > kPagesMaxSeqs) return internal_fail(HB_ERR_UNSUPPORTED, "num_seqs above 16384");
  if (page_size != kPageSize) return internal_fail(HB_ERR_UNSUPPORTED, "only page_size 16 is built");
  if (max_pages_per_seq <= 0 || num_pages <= 0)
    return internal_fail(HB_ERR_SHAPE, "max_pages_per_seq and num_pages must be > 0");
  if ((int64_t)max_pages_per_seq * kPageSize > INT_MAX || (int64_t)num_pages * kPageSize > INT_MAX)
    return internal_fail(HB_ERR_UNSUPPORTED, "max_pages_per_seq or num_pages too large");
  if (num_seqs > 0 && (!lens || !block_table))
    return internal_fail(HB_ERR_INVALID_ARG, "the length arrays and block_table must be non-NULL");
  if (!ring || !state_in || !state_out)
    return internal_fail(HB_ERR_INVALID_ARG, "free_pages, state_in and state_out must be non-NULL");
  if ((reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(ring) |
       reinterpret_cast<uintptr_t>(block_table)) & 3u)
    return internal_fail(HB_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(state_in) | reinterpret_cast<uintptr_t>(state_out)) & 7u)
    return internal_fail(HB_ERR_INVALID_ARG, "state_in and state_out must be 8-byte aligned");
  const uintptr_t a = reinterpret_cast<uintptr_t>(state_in), b = reinterpret_cast<uintptr_t>(state_out);
  if (a != b && a < b + 32 && b < a + 32)
    return internal_fail(HB_ERR_INVALID_ARG, "state_in and state_out overlap without being one");
  return HB_OK;
}

template <typename... Params, typename... Args>
hb_status launch(void (*kernel)(Params...), int64_t grid, size_t smem, void* stream, const char* what,
                 const Args&... args) {
  cudaError_t e = cudaSuccess;
  if (smem > 32 * 1024)   // (more than a launch gets unasked, next to the static part)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024);
  if (e == cudaSuccess)
    e = launch_serialized(kernel, (unsigned)grid, kPagesThreads, smem, static_cast<cudaStream_t>(stream),
                          args...);
  if (e != cudaSuccess) return internal_fail(HB_ERR_CUDA, what);
  internal_note_other_launch(stream);
  internal_count_launch();
  return internal_ok();
}

}  // namespace
}  // namespace hb

using namespace hb;

extern "C" hb_status hb_pages_assign(int32_t num_seqs, int32_t max_tokens, int32_t max_pages_per_seq,
                                     int32_t num_pages, int32_t page_size, const int32_t* q_len,
                                     const int32_t* context_len, const int32_t* free_pages,
                                     const int64_t* state_in, int64_t* state_out,
                                     int32_t* block_table, int32_t* cu_q_len, int64_t* slot_map,
                                     void* stream) {
  try {
    hb_status s = check_common(num_seqs, max_pages_per_seq, num_pages, page_size, context_len,
                               free_pages, state_in, state_out, block_table);
    if (s != HB_OK) return s;
    if (max_tokens < 0) return internal_fail(HB_ERR_SHAPE, "max_tokens must be >= 0");
    if (!cu_q_len || (num_seqs > 0 && !q_len))
      return internal_fail(HB_ERR_INVALID_ARG, "q_len and cu_q_len must be non-NULL");
    if ((reinterpret_cast<uintptr_t>(q_len) | reinterpret_cast<uintptr_t>(cu_q_len)) & 3u)
      return internal_fail(HB_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
    if (reinterpret_cast<uintptr_t>(slot_map) & 7u)
      return internal_fail(HB_ERR_INVALID_ARG, "slot_map must be 8-byte aligned");
    PagesParams p{};
    p.q_len = q_len;
    p.ctx = context_len;
    p.num_seqs = num_seqs;
    p.max_tokens = max_tokens;
    p.max_pages_per_seq = max_pages_per_seq;
    p.num_pages = num_pages;
    p.state_in = state_in;
    p.state_out = state_out;
    p.ring = const_cast<int32_t*>(free_pages);
    p.block_table = block_table;
    p.cu_q_len = cu_q_len;
    p.slot_map = slot_map;
    int num_sms = 0;
    if ((s = internal_device(&p.dev_error, &num_sms)) != HB_OK) return s;
    // a thread per run of slots, or per table entry (at most one per 16 tokens
    // and one more per sequence, and the table's); at most two CTAs per SM
    const bool few = max_tokens <= kPagesThreads * num_sms;
    const int64_t entries = std::min((int64_t)max_tokens / kPageSize + num_seqs,
                                     (int64_t)num_seqs * max_pages_per_seq);
    const int64_t runs = slot_map ? (int64_t)max_tokens / (few ? 1 : 4) + num_seqs : entries;
    const int64_t grid =
        std::max<int64_t>(1, std::min<int64_t>((runs + kPagesThreads - 1) / kPagesThreads, 2LL * num_sms));
    const size_t smem = 3 * ((size_t)num_seqs + 1) * sizeof(int32_t);
    return launch(few ? pages_assign_kernel<1> : pages_assign_kernel<4>, grid, smem, stream,
                  "pages_assign launch failed", p);
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_pages_assign");
  }
}

extern "C" hb_status hb_pages_release(int32_t num_seqs, int32_t max_pages_per_seq, int32_t num_pages,
                                      int32_t page_size, const int32_t* lengths,
                                      const int32_t* block_table, int32_t* free_pages,
                                      const int64_t* state_in, int64_t* state_out, void* stream) {
  try {
    hb_status s = check_common(num_seqs, max_pages_per_seq, num_pages, page_size, lengths,
                               free_pages, state_in, state_out, block_table);
    if (s != HB_OK) return s;
    PagesParams p{};
    p.ctx = lengths;
    p.num_seqs = num_seqs;
    p.max_pages_per_seq = max_pages_per_seq;
    p.num_pages = num_pages;
    p.state_in = state_in;
    p.state_out = state_out;
    p.ring = free_pages;
    p.block_table = const_cast<int32_t*>(block_table);
    int num_sms = 0;
    if ((s = internal_device(&p.dev_error, &num_sms)) != HB_OK) return s;
    // three CTAs per SM (two 7.5 us, four 9.0); more than one for a row only
    // where its segments are more than a CTA's warps
    const int ctas = 3 * num_sms, warps = kPagesThreads / 32;
    const int segs = (max_pages_per_seq + 32 * kSeg - 1) / (32 * kSeg);
    const int groups = std::max(1, std::min(num_seqs, ctas));
    const int slices = std::max(1, std::min((segs + warps - 1) / warps, ctas / groups));
    const size_t smem = (size_t)((num_seqs + groups - 1) / groups) * sizeof(int32_t);
    return launch(pages_release_kernel, (int64_t)groups * slices, smem, stream,
                  "pages_release launch failed", p, groups, slices);
  } catch (...) {
    return internal_fail(HB_ERR_CUDA, "unexpected exception in hb_pages_release");
  }
}
