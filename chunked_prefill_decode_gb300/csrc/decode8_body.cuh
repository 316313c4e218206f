// decode8_body.cuh -- attention of decode rows over the 8-bit cache (kv8.cuh):
// the per-CTA body that the 8-bit attention kernel (attention8.cu) runs for
// decode CTAs.
//
// "Sarathi-Serve：以 chunked-prefills 与 stall-free batching 驯服 LLM 推理的吞吐—
// 延迟权衡", §GPU / 系统数据路径 ⑤: a decode reads all earlier KV of its
// sequence every step.  Half the bytes of the bf16 cache, so the same stream
// leaves half the time per page for the work on it.
//
// The mathematics, for one q head over keys t whose page has the exponents
// ke, ve (values k, v):
//     x_t = (q . k_t) scale log2(e) 2^ke             M = max x_t
//     P_t = 2^(x_t - M)      l = sum P_t      o = sum P_t 2^ve v_t / l
// P goes to the products in fp16 (11 significant bits, against bf16's 8), times
// 2^kDec8PShift and the page's 2^(ve - R).  R is a reference exponent of the
// warp, o's unit: it stays while the pages' ve lie within kDec8Spread of it
// (those of one head mostly differ by a bit or two) and else moves to the next
// page's ve, o being multiplied by 2^(old R - new R), which is exact.  So the
// scales cost a weight nothing: the largest error of a far key's weight, half
// of fp16's smallest step, is 2^-32 of the row's largest weight (ve - R = -2).
// R is held within 2^64 of the largest one before it in the item, so that o
// stays inside fp32; a page whose V scale lies further below counts as zeros.
// (With ve inside the maximum, as x_t + ve, a page with a large V scale pushes
// the other pages' weights out of fp16: one scale 2^24 above the others' made
// their part of o wrong by up to 150 times what the roundings allow.)
// GB300: 256 decodes 346 us, with ve inside the maximum 345; 64 decodes and a
// 448-token chunk 78.8 and 78.6; 4 rows of 8192 16.4 and 16.1.  V scales anywhere
// within 2^60 cost 1 % more.  A stage's body stands there twice, for windows of
// 32 pages that lie near R and for others: one body with the branch for a move
// takes 350 and 12 rows on one kv head 15.3 instead of 14.8.
// q is scaled by a power of two per head so that its largest element is near
// 2^12 and every element keeps its bits in fp16; e4m3 is exact in fp16.
//
// Layout of the work, and why:
//  * the host plan gives each CTA an equal contiguous range of the decode
//    rows' pages, cut into items at row boundaries, or, where rows are few, a
//    piece of one row (decode_plan.h);
//  * a stage of the ring is as many pages as make sixteen (kv head, page)
//    pairs, K and V, at D 128 and 32 at D 64: two (four) pages of 8 heads, or
//    16 (32) pages of one head, so a warp has the same work per stage whatever
//    the head count.  Four producer
//    warps fill it with one TMA box per page and pool ([kv head][slot][D bytes],
//    swizzled by the row width);
//  * eight consumer warps, each with one head and two pages of the stage (four
//    at D 64), so that as many chains of products, softmax and products run
//    side by side: a
//    page alone is a chain of latencies (1390 cycles at D 128, hardly less at
//    D 64), and filling a stage costs the producer about 750 cycles whatever it
//    holds;
//  * the products are taken transposed as in decode_body.cuh.  The MMA's k
//    index may run over the head dims in any order that q shares, so a lane
//    takes its K operand as 16 contiguous bytes of a key (two LDS.128 per key
//    at D 128; neighbouring rows' chunks fall into different banks under the
//    swizzle), and each 4-byte word is one k step: no ldmatrix, no shuffles.
//    V^T comes by ldmatrix.trans of byte pairs (two dims of one key): one byte
//    permutation turns two keys' pairs into two rows of the A operand, so the
//    operand's rows r and r + 8 are dims 2r and 2r + 1 of a 16-dim block and
//    a lane's outputs are neighbours.  cvt.f16x2.e4m3x2 does two elements per
//    instruction;
//  * producer and consumers walk the same items, so a stage carries no
//    header; each warp keeps the exponents of 32 of its pages in a lane each
//    (table entry, then both exponents, a window ahead, the next item's first
//    window while the current item runs), one shuffle per page;
//  * warps that share a head merge their states pairwise in shared memory at
//    the end of an item; a row that straddles CTAs is merged by its last piece
//    through the workspace, as in decode_body.cuh;
//  * the consumers hold 224 registers (the producer's warpgroup gives up 112).
//
// Bytes per decode row: 2 * context * Hkv * D.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "hb_internal.h"
#include "kv8.cuh"
#include "ptx.cuh"

namespace hb {

constexpr int kDec8Consumers = 8;     // warps 0-7
constexpr int kDec8Producers = 4;     // warps 8-11
// pages of a stage per consumer warp: 256 head dims' worth
inline __host__ __device__ constexpr int decode8_pages(int head_dim) { return 256 / head_dim; }
// stages that fit at most: the smallest stage is that of 5 kv heads
constexpr int kDec8MaxStages = 5;
static_assert(227 * 1024 / (2 * 5 * kPageSize * 256) == kDec8MaxStages, "ring of the smallest stage");
constexpr float kDec8RescaleThreshold = 4.0f;   // log2 units
constexpr int kDec8Spread = 2;                  // of a page's ve about the reference
constexpr float kDec8PShift = 9.0f;             // P <= 2^(4 + 9 + 2) in fp16
constexpr int kDec8Drop = 64;                   // the reference falls no further, see above
constexpr int kDec8Regs = 224;        // per thread, warps 0-7
constexpr int kDec8LightRegs = 56;    // per thread, warps 8-11
static_assert(256 * kDec8Regs + 128 * kDec8LightRegs <= 384 * 168,
              "register split exceeds the launch allocation");

struct Decode8Layout {
  int32_t n_stages;
  int32_t parts;         // warps that share a head
  int32_t half_bytes;    // K (or V) of one page
  int32_t stage_bytes;
  int32_t qslot_bytes;
  int32_t merge_bytes;   // states of the warps that share a head
  int32_t smem_bytes;
};

// floats that one warp leaves for the merge of the warps that share its head
inline __host__ __device__ int decode8_state_floats(int head_dim, int group) {
  const int nq = group <= 8 ? 1 : 2;
  return (head_dim / 16 * nq * 4 + 2 * nq * 2) * 32;
}

inline __host__ Decode8Layout decode8_layout(int head_dim, int kvh_block, int group) {
  Decode8Layout L{};
  L.parts = kDec8Consumers / kvh_block;   // 8, 4, 2, 2, 1 ..: a power of two
  L.half_bytes = kvh_block * kPageSize * head_dim;
  L.stage_bytes = 2 * L.half_bytes * L.parts * decode8_pages(head_dim);
  L.qslot_bytes = ((kvh_block * group * head_dim * 2) + 1023) / 1024 * 1024;
  L.merge_bytes = L.parts / 2 * kvh_block * decode8_state_floats(head_dim, group) * 4;
  const int fixed = 1024 /*align*/ + 2 * L.qslot_bytes + L.merge_bytes +
                    (2 * kDec8MaxStages + 5) * 8 + 64;
  int s = (227 * 1024 - fixed) / L.stage_bytes;
  if (s > kDec8MaxStages) s = kDec8MaxStages;
  L.n_stages = s;
  L.smem_bytes = fixed + s * L.stage_bytes;
  return L;
}

// The last piece of a row (and block of kv heads) merges all of them: o = sum
// 2^(m_i - M) o_i / sum 2^(m_i - M) l_i.  A warp takes kMh of the block's nh q
// heads at a time and kUnroll pieces of each, their loads in flight together;
// each lane owns D / 32 dims.  (A block of few heads has many pieces.)
template <int D, int kMh, int kUnroll>
__device__ __forceinline__ void merge_rows8(const DecodeParams& p, const DecodeItem& it, int nh,
                                            int warp) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, Hq = p.num_q_heads;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
  for (int h0 = warp; h0 < nh; h0 += kMh * kDec8Consumers) {
    float mmax[kMh], lsum[kMh], acc[kMh][E];
    size_t hh[kMh];
#pragma unroll
    for (int h = 0; h < kMh; ++h) {
      // (past the block's heads: the first one again, not stored)
      hh[h] = (size_t)(it.kvh0 * p.group + (h0 + h * kDec8Consumers < nh ? h0 + h * kDec8Consumers : h0));
      mmax[h] = -INFINITY;
      lsum[h] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[h][e] = 0.f;
    }
    // the pieces' (m, l), 32 at a time, a lane each; the first 32 (as good as
    // always all) stay in registers
    float2 st0[kMh];
#pragma unroll
    for (int h = 0; h < kMh; ++h) {
      st0[h] = make_float2(-INFINITY, 0.f);
      if (lane < it.n_splits) st0[h] = __ldcg(&ml[(size_t)(it.slot + lane) * Hq + hh[h]]);
    }
#pragma unroll
    for (int h = 0; h < kMh; ++h) mmax[h] = st0[h].x;
    for (int i2 = lane + 32; i2 < it.n_splits; i2 += 32)
#pragma unroll
      for (int h = 0; h < kMh; ++h)
        mmax[h] = fmaxf(mmax[h], __ldcg(&ml[(size_t)(it.slot + i2) * Hq + hh[h]]).x);
#pragma unroll
    for (int h = 0; h < kMh; ++h)
#pragma unroll
      for (int d = 16; d > 0; d >>= 1)
        mmax[h] = fmaxf(mmax[h], __shfl_xor_sync(0xffffffffu, mmax[h], d));
    for (int base = 0; base < it.n_splits; base += 32) {
      float wgt[kMh];
#pragma unroll
      for (int h = 0; h < kMh; ++h) {
        float2 st2 = st0[h];
        if (base > 0) {
          st2 = make_float2(-INFINITY, 0.f);
          if (base + lane < it.n_splits) st2 = __ldcg(&ml[(size_t)(it.slot + base + lane) * Hq + hh[h]]);
        }
        wgt[h] = fast_exp2(st2.x - mmax[h]);   // 0 past the pieces
        lsum[h] += wgt[h] * st2.y;
      }
      const int m = min(32, it.n_splits - base);
#pragma unroll kUnroll
      for (int i2 = 0; i2 < m; ++i2)
#pragma unroll
        for (int h = 0; h < kMh; ++h) {
          const float wi = __shfl_sync(0xffffffffu, wgt[h], i2);
          const float* po = p.part_o + ((size_t)(it.slot + base + i2) * Hq + hh[h]) * D + lane * E;
          if constexpr (E == 4) {
            const float4 v = __ldcg(reinterpret_cast<const float4*>(po));
            acc[h][0] += wi * v.x; acc[h][1] += wi * v.y;
            acc[h][2] += wi * v.z; acc[h][3] += wi * v.w;
          } else {
            const float2 v = __ldcg(reinterpret_cast<const float2*>(po));
            acc[h][0] += wi * v.x; acc[h][1] += wi * v.y;
          }
        }
    }
#pragma unroll
    for (int h = 0; h < kMh; ++h) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) lsum[h] += __shfl_xor_sync(0xffffffffu, lsum[h], d);
      if (h0 + h * kDec8Consumers >= nh) continue;
      const float inv = 1.f / lsum[h];
      uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((size_t)it.tok * Hq + hh[h]) * D + lane * E);
#pragma unroll
      for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[h][e] * inv, acc[h][e + 1] * inv);
    }
  }
}

// Body of one decode CTA (index `cta` among the decode CTAs); `smem` is the
// 1024-byte-aligned dynamic shared memory.
template <int D>
__device__ __forceinline__ void decode8_cta(const DecodeParams& p, const Decode8Params& p8,
                                            const Decode8Layout& L, const CUtensorMap& kmap,
                                            const CUtensorMap& vmap, uint8_t* smem, int cta) {
  const int S = L.n_stages;
  uint8_t* stages = smem;
  uint8_t* qbuf = smem + S * L.stage_bytes;
  float* mbuf = reinterpret_cast<float*>(qbuf + 2 * L.qslot_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(mbuf) + L.merge_bytes);
  uint64_t* empty = full + kDec8MaxStages;
  uint64_t* qfull = empty + kDec8MaxStages;
  uint64_t* qempty = qfull + 2;
  uint64_t* together = qempty + 2;                  // the consumers among themselves
  int* flags = reinterpret_cast<int*>(together + 1);  // [0] abort, [1] merge
  volatile int* abort_flag = flags;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g = p.group;
  const int kvhb = p.kvh_block;
  const int parts = L.parts;
  constexpr int U = decode8_pages(D);
  const int pps = parts * U;            // pages per stage; divides 32

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], kDec8Producers);
      mbar_init(&empty[s], kDec8Consumers);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 1);
      mbar_init(&qempty[i], kDec8Consumers);
    }
    mbar_init(together, kDec8Consumers);
    flags[0] = 0;
    flags[1] = 0;
    fence_mbar_init();
  }
  __syncthreads();

  const int item0 = p.cta_offsets[cta], item1 = p.cta_offsets[cta + 1];

  // (each role sets its registers inside its own branch: code that both
  // could reach would be held to the smaller number)
  if (warp >= kDec8Consumers) {
    setmaxnreg_dec<kDec8LightRegs>();
    // ------------------------------------------------------------ producer
    // Four warps walk the stages side by side and issue every fourth box of
    // each (K and V of page i are boxes 2i and 2i + 1): a box takes a warp
    // about 110 cycles to issue, and a stage of 16 pages of one head has 32.
    // In each warp a lane holds one block-table entry of a 32-page window
    // (fetched a window ahead) and lane 0 works the barriers.
    const int me = warp - kDec8Consumers;
    if (lane == 0) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    int st = 0;
    uint32_t ph = 0;
    int qslot = 0;
    uint32_t qph[2] = {0u, 0u};
    uint32_t issued_mask = 0, last_par_mask = 0;
    bool dep_done = false;   // griddep_wait done (before the first page with a new token)
    // (complete already, Decode8Params: what it wrote with plain stores is read
    // by copies of the async proxy)
    if (!p8.wait_new) fence_proxy_async_global();
    const uint32_t qbytes = (uint32_t)(kvhb * g * D * 2);
    // lane l: block-table entry of page base + l of item x, checked where used
    auto window = [&](const DecodeItem& x, int base) -> int {
      const int lp = base + lane;
      if (lp >= x.page_end || lp >= p.max_pages_per_seq) return -1;
      return __ldcg(&p.block_table[(size_t)x.seq * p.max_pages_per_seq + lp]);
    };
    bool ok = true;
    DecodeItem it{}, nxt{};
    int win = 0, win_next = 0, nxt_win = 0;
    if (item0 < item1) {
      it = p.items[item0];
      win = window(it, it.page_begin);
      win_next = window(it, it.page_begin + 32);
    }
    for (int i = item0; ok && i < item1; ++i) {
      if (me == 0 && lane == 0) {
        ok = mbar_wait(&qempty[qslot], qph[qslot] ^ 1u, abort_flag);
        if (ok) {
          mbar_arrive_expect_tx(&qfull[qslot], qbytes);
          bulk_load(qbuf + qslot * L.qslot_bytes,
                    p.q + ((size_t)it.tok * p.num_q_heads + (size_t)it.kvh0 * g) * D, qbytes,
                    &qfull[qslot]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      qph[qslot] ^= 1u;
      const int new_page = (it.ctx - 1) / kPageSize;   // holds the row's new token
      for (int lp = it.page_begin; ok && lp < it.page_end; lp += pps) {
        const int k = (lp - it.page_begin) & 31;
        if (k == 0 && lp != it.page_begin) {
          win = win_next;
          win_next = window(it, lp + 32);
        }
        const int np = min(pps, it.page_end - lp);
        const int box = 4 * lane + me;   // this lane's box of the stage, if there are so many
        int phys = __shfl_sync(0xffffffffu, win, k + min(box >> 1, pps - 1));
        const bool issuer = box < 2 * np;
        if (issuer && (unsigned)phys >= (unsigned)p.num_pages) {
          // out of range: reported, and fetched out of bounds (zeros)
          report_error(p.dev_error, HB_DEVERR_INDEX);
          phys = p.num_pages;
        }
        // the append before this launch wrote the new token's page
        if (p8.wait_new && !dep_done && lp + np > new_page) {
          griddep_wait();
          fence_proxy_async_global();
          dep_done = true;
        }
        if (lane == 0) {
          ok = mbar_wait(&empty[st], ph ^ 1u, abort_flag);
          // (the boxes of this warp)
          if (ok) mbar_arrive_expect_tx(&full[st], (uint32_t)((2 * np - me + 3) / 4 * L.half_bytes));
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok) {
          if (issuer)
            tma_load_4d(stages + st * L.stage_bytes + box * L.half_bytes, (box & 1) ? &vmap : &kmap,
                        &full[st], 0, 0, it.kvh0, phys);
          issued_mask |= 1u << st;
          last_par_mask = (last_par_mask & ~(1u << st)) | (ph << st);
        }
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
        if (lp == it.page_begin && i + 1 < item1) {
          // with the item's first pages in flight: the next item's first window
          nxt = p.items[i + 1];
          nxt_win = window(nxt, nxt.page_begin);
        }
      }
      qslot ^= 1;
      it = nxt;
      win = nxt_win;
      if (i + 1 < item1) win_next = window(it, it.page_begin + 32);
    }
    if (lane == 0)   // copies in flight must land before the CTA exits
      for (int s2 = 0; s2 < S; ++s2)
        if (issued_mask & (1u << s2)) drain_wait(&full[s2], (last_par_mask >> s2) & 1u, abort_flag);
  } else {
    setmaxnreg_inc<kDec8Regs>();
    // ------------------------------------------------------------ consumers
    auto consume = [&](auto nq_const) {
      constexpr int NQ = decltype(nq_const)::value;   // 8-head column tiles
      constexpr int KC = D / 64;                      // 16-byte K chunks per lane and key
      const int w = warp % kvhb;                      // local kv head of this warp
      const int part = warp / kvhb;                   // its pages of a stage: part + u * parts
      const bool active = part < parts;
      const int r = lane >> 2, c = lane & 3;
      const int mi = lane >> 3, r8 = lane & 7;        // ldmatrix: matrix, row
      uint32_t qb[D / 16][NQ][2];          // B operand Q^T
      float o[D / 16][NQ][4];              // O^T: dims 16 jj + 2 r (+ 1 in [2], [3]), heads 2c, 2c + 1
      float m_run[NQ][2], l_part[NQ][2];   // head 8 nq + 2c + e; l over this lane's keys
      float qs[NQ][2];                     // softmax scale * log2(e) * 2^(q's exponent)
      // All consumers get here, and see what the others wrote before; false
      // if one of them has given up.  (A bounded wait: a hardware barrier
      // would wait for a warp that left.)
      uint32_t tph = 0;
      auto all_here = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(together);
        const bool ok = __all_sync(0xffffffffu, mbar_wait(together, tph, abort_flag));
        tph ^= 1u;
        return ok;
      };
      // One page per lane, the (base + lane)-th of this warp in item x: its
      // table entry (raw), then its exponents (ke | ve << 8).
      auto entry = [&](const DecodeItem& x, int base) -> int {
        const int lp = x.page_begin + part + (base + lane) * parts;
        return (active && lp < x.page_end && lp < p.max_pages_per_seq)
                   ? __ldcg(&p.block_table[(size_t)x.seq * p.max_pages_per_seq + lp])
                   : -1;
      };
      auto exponents = [&](const DecodeItem& x, int raw) -> int {
        if ((unsigned)raw >= (unsigned)p.num_pages) return 0;
        const size_t at = (size_t)raw * p.num_kv_heads + x.kvh0 + w;
        return (kv8_exp(ldcg_s8(p8.k_exp + at)) & 0xff) | (kv8_exp(ldcg_s8(p8.v_exp + at)) << 8);
      };
      // what the append wrote (the exponents of the last pages) is complete
      if (p8.wait_new) griddep_wait();

      int st = 0;
      uint32_t ph = 0;
      int qslot = 0;
      uint32_t qph[2] = {0u, 0u};
      bool ok = true;
      DecodeItem it{}, nxt{};
      // ahead: of the next item nothing (0), its description (1), its first
      // table entries (2) or their exponents (3) are here
      int ahead = 0, nxt_raw = -1, nxt_e = 0;
      if (item0 < item1) {
        nxt = p.items[item0];
        ahead = 1;
      }
      for (int i = item0; ok && i < item1; ++i) {
        it = nxt;
        if (ahead < 2) nxt_raw = entry(it, 0);
        if (ahead < 3) nxt_e = exponents(it, nxt_raw);
        int e_cur = nxt_e, e_next = 0, raw_next = entry(it, 32);
        ahead = 0;
        if (i + 1 < item1) {
          nxt = p.items[i + 1];
          ahead = 1;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&qfull[qslot], qph[qslot], abort_flag));
        if (!ok) break;
        qph[qslot] ^= 1u;
        if (active) {
          const uint16_t* q0 = reinterpret_cast<const uint16_t*>(qbuf + qslot * L.qslot_bytes) +
                               (size_t)w * g * D;
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            const int head = nq * 8 + r;
            uint32_t mx = 0;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              // k step kk: word kk % 4 of chunk KC c + kk / 4
              const int d0 = (KC * c + kk / 4) * 16 + (kk & 3) * 4;
              uint2 v = make_uint2(0u, 0u);
              if (head < g) v = *reinterpret_cast<const uint2*>(q0 + head * D + d0);
              qb[kk][nq][0] = v.x;
              qb[kk][nq][1] = v.y;
              mx = max(max(mx, max(v.x & 0x7fffu, (v.x >> 16) & 0x7fffu)),
                       max(v.y & 0x7fffu, (v.y >> 16) & 0x7fffu));
            }
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // largest element 2^(E - 127) .. 2^(E - 126): to 2^12 .. 2^13
            const int qe = min(max((int)(mx >> 7) - 127 - 12, -100), 115);
            const float mul = pow2i(-qe);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t v = qb[kk][nq][x];
                qb[kk][nq][x] = pack_f16x2(bf16lo_to_f32(v) * mul, bf16hi_to_f32(v) * mul);
              }
#pragma unroll
            for (int e = 0; e < 2; ++e)   // the head of accumulator column 2c + e
              qs[nq][e] = p.scale_log2 * pow2i(__shfl_sync(0xffffffffu, qe, (2 * c + e) * 4));
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&qempty[qslot]);
        qslot ^= 1;
#pragma unroll
        for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) o[jj][nq][0] = o[jj][nq][1] = o[jj][nq][2] = o[jj][nq][3] = 0.f;
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
          m_run[nq][0] = m_run[nq][1] = -INFINITY;
          l_part[nq][0] = l_part[nq][1] = 0.f;
        }

        int tl = 0;   // this warp's page of the window of 32
        // o's unit and the largest one so far (alike in the warp)
        int ref = __shfl_sync(0xffffffffu, e_cur, 0) >> 8, ref_max = ref;
        // the pages of the window of 32 that begins with page `first` all lie near it
        const auto near = [&](int first) -> bool {
          return __all_sync(0xffffffffu, first + lane * parts >= it.page_end ||
                                             (unsigned)((e_cur >> 8) - ref + kDec8Spread) <= 2u * kDec8Spread);
        };
        bool calm = near(it.page_begin + part);
        // The warp's pages lp0, lp0 + parts, .. of the stage at hand.  (Twice, so
        // that the usual one has no branch for a unit that moves.)
        const auto stage = [&](int lp0, auto calm_const) {
          constexpr bool kCalm = decltype(calm_const)::value;
          const uint32_t sbase = smem_u32(stages + st * L.stage_bytes) + (uint32_t)(w * kPageSize * D);
          // byte address of 16-byte chunk x of key row `row`
          auto chunk = [&](uint32_t base, int row, int x) -> uint32_t {
            if constexpr (D == 128) return base + (uint32_t)(row * 128 + ((x ^ (row & 7)) << 4));
            return base + (uint32_t)(row * 64 + ((x ^ ((row >> 1) & 3)) << 4));
          };
          uint4 kr[U][2][KC];            // keys r and r + 8
          uint32_t vr[U][D / 32][4];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t kbase = sbase + (uint32_t)(2 * (part + u * parts) * L.half_bytes);
#pragma unroll
            for (int x = 0; x < KC; ++x) {
              kr[u][0][x] = lds128(chunk(kbase, r, KC * c + x));
              kr[u][1][x] = lds128(chunk(kbase, r + 8, KC * c + x));
            }
          }
          // V byte pairs, transposed: matrices (keys 0-7, 8-15) of chunks 2 j, 2 j + 1
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t vbase = sbase + (uint32_t)((2 * (part + u * parts) + 1) * L.half_bytes);
#pragma unroll
            for (int j = 0; j < D / 32; ++j)
              ldsm_x4_trans(chunk(vbase, ((mi & 1) << 3) + r8, 2 * j + (mi >> 1)), vr[u][j][0],
                            vr[u][j][1], vr[u][j][2], vr[u][j][3]);
          }
          // K and V of the pages are in registers: the stage goes back
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
          float fk[U], fv[U];
          int valid[U], lo_valid[U], ves[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int ex = __shfl_sync(0xffffffffu, e_cur, (tl + u) & 31);
            const int ke = (int)(int8_t)(ex & 0xff), ve = ex >> 8;
            fk[u] = pow2i(ke);
            const int lp = lp0 + u * parts;
            // (a page past the item's end: the stage holds none, no key is seen)
            valid[u] = lp < it.page_end ? min(kPageSize, it.ctx - lp * kPageSize) : 0;
            ves[u] = ve;
            fv[u] = pow2i(ve - ref);
            // with a sliding window the row sees keys ctx - W .. ctx - 1 only
            lo_valid[u] = p.window > 0 ? it.ctx - p.window - lp * kPageSize : 0;
          }
          [[maybe_unused]] int move[U];   // 2^move times o before the products of a page
          if constexpr (!kCalm) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
              move[u] = 0;
              if (valid[u] > 0 && (unsigned)(ves[u] - ref + kDec8Spread) > 2u * kDec8Spread) {
                const int to = max(ves[u], ref_max - kDec8Drop);
                move[u] = ref - to;
                ref = to;
                ref_max = max(ref_max, to);
              }
              fv[u] = pow2i(ves[u] - ref);
            }
          }
          // independent accumulators, so that the chains of MMAs are short
          constexpr int kQk = NQ * U <= 2 ? 2 : 1;
          float s[U][kQk][NQ][4];
#pragma unroll
          for (int u = 0; u < U; ++u)
#pragma unroll
            for (int x = 0; x < kQk; ++x)
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq)
                s[u][x][nq][0] = s[u][x][nq][1] = s[u][x][nq][2] = s[u][x][nq][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const uint4 k0 = kr[u][0][kk / 4], k1 = kr[u][1][kk / 4];
              const uint32_t w0 = (kk & 3) == 0 ? k0.x : (kk & 3) == 1 ? k0.y : (kk & 3) == 2 ? k0.z : k0.w;
              const uint32_t w1 = (kk & 3) == 0 ? k1.x : (kk & 3) == 1 ? k1.y : (kk & 3) == 2 ? k1.z : k1.w;
              const uint32_t ka[4] = {f16x2_of_e4m3x2(w0), f16x2_of_e4m3x2(w1),
                                      f16x2_of_e4m3x2(w0 >> 16), f16x2_of_e4m3x2(w1 >> 16)};
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq)
                mma_f16_16816(s[u][kk % kQk][nq], ka, qb[kk][nq][0], qb[kk][nq][1]);
            }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (valid[u] < kPageSize || lo_valid[u] > 0) {
              // values of keys that the row does not see may be anything,
              // NaN included: cleared, since P = 0 would not stop it
              const auto seen = [&](int key) { return key < valid[u] && key >= lo_valid[u]; };
              const uint32_t m0 = (seen(2 * c) ? 0xffffu : 0u) | (seen(2 * c + 1) ? 0xffff0000u : 0u);
              const uint32_t m1 = (seen(2 * c + 8) ? 0xffffu : 0u) | (seen(2 * c + 9) ? 0xffff0000u : 0u);
#pragma unroll
              for (int j = 0; j < D / 32; ++j) {
                vr[u][j][0] &= m0;
                vr[u][j][1] &= m1;
                vr[u][j][2] &= m0;
                vr[u][j][3] &= m1;
              }
            }
          float x0[U][NQ][2], x1[U][NQ][2], alpha[NQ][2];
          bool need = false;
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              alpha[nq][e] = 1.f;
#pragma unroll
              for (int u = 0; u < U; ++u) {
                float a0 = s[u][0][nq][e], a1 = s[u][0][nq][2 + e];
#pragma unroll
                for (int x = 1; x < kQk; ++x) {
                  a0 += s[u][x][nq][e];
                  a1 += s[u][x][nq][2 + e];
                }
                const float cs = qs[nq][e] * fk[u];
                x0[u][nq][e] = r < valid[u] && r >= lo_valid[u] ? a0 * cs : -INFINITY;
                x1[u][nq][e] = r + 8 < valid[u] && r + 8 >= lo_valid[u] ? a1 * cs : -INFINITY;
                need |= fmaxf(x0[u][nq][e], x1[u][nq][e]) > m_run[nq][e] + kDec8RescaleThreshold;
              }
            }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(x0[0][nq][e], x1[0][nq][e]);
#pragma unroll
                for (int u = 1; u < U; ++u) mx = fmaxf(mx, fmaxf(x0[u][nq][e], x1[u][nq][e]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                if (mx > m_run[nq][e] + kDec8RescaleThreshold) {
                  alpha[nq][e] = fast_exp2(m_run[nq][e] - mx);
                  m_run[nq][e] = mx;
                }
              }
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int x = 0; x < 4; ++x) o[jj][nq][x] *= alpha[nq][x & 1];
          }
          uint32_t pb[U][NQ][2];
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
#pragma unroll
            for (int e = 0; e < 2; ++e) l_part[nq][e] *= alpha[nq][e];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              float p0[2], p1[2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // no key seen yet: every x is -inf and so is P's exponent
                const float mu = (m_run[nq][e] == -INFINITY ? 0.f : m_run[nq][e]) - kDec8PShift;
                p0[e] = fast_exp2(x0[u][nq][e] - mu);
                p1[e] = fast_exp2(x1[u][nq][e] - mu);
                l_part[nq][e] += p0[e] + p1[e];
              }
              const uint64_t f = pack_f32x2(fv[u], fv[u]);
              unpack_f32x2(mul_f32x2(pack_f32x2(p0[0], p0[1]), f), p0[0], p0[1]);
              unpack_f32x2(mul_f32x2(pack_f32x2(p1[0], p1[1]), f), p1[0], p1[1]);
              pb[u][nq][0] = movmatrix_trans(pack_f16x2(p0[0], p0[1]));   // B: keys 2c, 2c + 1 of head r
              pb[u][nq][1] = movmatrix_trans(pack_f16x2(p1[0], p1[1]));   // keys 8 + 2c ..
            }
          }
          // O^T += V^T P^T
          const auto products = [&](int u) {
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj) {
              // bytes (key 0: dims 0, 1; key 1: dims 0, 1) -> (dim 0: keys 0, 1; dim 1: ..)
              const uint32_t v0 = __byte_perm(vr[u][jj / 2][2 * (jj & 1)], 0u, 0x3120);
              const uint32_t v1 = __byte_perm(vr[u][jj / 2][2 * (jj & 1) + 1], 0u, 0x3120);
              const uint32_t va[4] = {f16x2_of_e4m3x2(v0), f16x2_of_e4m3x2(v0 >> 16),
                                      f16x2_of_e4m3x2(v1), f16x2_of_e4m3x2(v1 >> 16)};
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq) mma_f16_16816(o[jj][nq], va, pb[u][nq][0], pb[u][nq][1]);
            }
          };
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if constexpr (!kCalm) {
              if (move[u] != 0) {
                const float f = pow2i(move[u]);
#pragma unroll
                for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
                  for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                    for (int x = 0; x < 4; ++x) o[jj][nq][x] *= f;
              }
            }
            products(u);
          }
        };
        for (int lp0 = it.page_begin + part; lp0 - part < it.page_end; lp0 += pps) {
          ok = __all_sync(0xffffffffu, mbar_wait(&full[st], ph, abort_flag));
          if (!ok) break;
          if (active && lp0 < it.page_end) {
            if (calm) stage(lp0, std::true_type{});
            else stage(lp0, std::false_type{});
          } else {
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[st]);
          }
          if (++st == S) {
            st = 0;
            ph ^= 1u;
          }
          // exponents: the next window's entries are here since this window
          // began, their exponents are asked for in its middle
          tl += U;
          if (tl == 16) {
            e_next = exponents(it, raw_next);
          } else if (tl == 32) {
            tl = 0;
            e_cur = e_next;
            calm = near(lp0 + pps);
            raw_next = entry(it, (lp0 + pps - it.page_begin - part) / parts + 32);
          }
          if (ahead == 1) {
            nxt_raw = entry(nxt, 0);
            ahead = 2;
          } else if (ahead == 2) {
            nxt_e = exponents(nxt, nxt_raw);
            ahead = 3;
          }
        }
        if (!ok) break;

        // ---------------------------------------------------------- the item's end
        const int Hq = p.num_q_heads;
        float unit = pow2i(ref);   // times o is the sum itself
        float l_tot[NQ][2];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = l_part[nq][e];
            x += __shfl_xor_sync(0xffffffffu, x, 4);
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            l_tot[nq][e] = x;
          }
        // warps of one head: the upper half of the parts leave their state,
        // lane by lane (the fragments have the same owners), the lower half
        // take it in, until part 0 has everything
        const int n_state = decode8_state_floats(D, g);
#pragma unroll 1
        for (int half = parts / 2; half > 0; half >>= 1) {
          if (active && part >= half && part < 2 * half) {
            float* dst = mbuf + (size_t)((part - half) * kvhb + w) * n_state + lane;
            int k = 0;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                dst[32 * k++] = m_run[nq][e];
                dst[32 * k++] = l_tot[nq][e];
              }
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int x = 0; x < 4; ++x) dst[32 * k++] = o[jj][nq][x] * unit;
          }
          if (!(ok = all_here())) break;
          if (part < half) {
            const float* src = mbuf + (size_t)(part * kvhb + w) * n_state + lane;
            float wa[NQ][2], wb[NQ][2];
            int k = 0;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float m2 = src[32 * k++], l2 = src[32 * k++];
                const float mm = fmaxf(m_run[nq][e], m2);
                wa[nq][e] = m_run[nq][e] == -INFINITY ? 0.f : fast_exp2(m_run[nq][e] - mm);
                wb[nq][e] = m2 == -INFINITY ? 0.f : fast_exp2(m2 - mm);
                m_run[nq][e] = mm;
                l_tot[nq][e] = l_tot[nq][e] * wa[nq][e] + l2 * wb[nq][e];
                wa[nq][e] *= unit;
              }
            unit = 1.f;
#pragma unroll
            for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
              for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  o[jj][nq][x] = o[jj][nq][x] * wa[nq][x & 1] + src[32 * k++] * wb[nq][x & 1];
          }
          if (!(ok = all_here())) break;   // the buffer may be written again
        }
        if (!ok) break;
        if (part == 0) {
          const int head0 = (it.kvh0 + w) * g;
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int head = nq * 8 + 2 * c + e;
              if (head >= g) continue;
              if (it.n_splits == 1) {
                const float inv = unit / l_tot[nq][e];
                uint32_t* dst = reinterpret_cast<uint32_t*>(
                    p.out + ((size_t)it.tok * Hq + head0 + head) * D + 2 * r);
#pragma unroll
                for (int jj = 0; jj < D / 16; ++jj)
                  dst[jj * 8] = pack_bf16x2(o[jj][nq][e] * inv, o[jj][nq][2 + e] * inv);
              } else {
                const size_t slot = (size_t)(it.slot + it.split);
                float* dst = p.part_o + (slot * Hq + head0 + head) * D + 2 * r;
#pragma unroll
                for (int jj = 0; jj < D / 16; ++jj)
                  *reinterpret_cast<float2*>(dst + jj * 16) =
                      make_float2(o[jj][nq][e] * unit, o[jj][nq][2 + e] * unit);
                if (r == 0)
                  reinterpret_cast<float2*>(p.part_ml)[slot * Hq + head0 + head] =
                      make_float2(m_run[nq][e], l_tot[nq][e]);
              }
            }
        }
        if (it.n_splits > 1) {
          // publish this piece's state: every consumer's stores come before
          // its arrival, and those before thread 0's device-scope release
          if (!(ok = all_here())) break;
          if (threadIdx.x == 0) {
            // release this piece's state, acquire the others'
            const int old = atom_add_acq_rel(&p.counters[kCounterMerge0 + it.merge_id], 1);
            flags[1] = (old == it.n_splits - 1) ? 1 : 0;
          }
          if (!(ok = all_here())) break;
          if (flags[1]) {
            if (kvhb * g <= kDec8Consumers) merge_rows8<D, 1, 16>(p, it, kvhb * g, warp);
            else merge_rows8<D, 4, 4>(p, it, kvhb * g, warp);
            if (threadIdx.x == 0) p.counters[kCounterMerge0 + it.merge_id] = 0;
          }
        }
      }
    };
    if (g <= 8) consume(std::integral_constant<int, 1>{});
    else consume(std::integral_constant<int, 2>{});
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) report_error(p.dev_error, HB_DEVERR_TIMEOUT);
}

}  // namespace hb
