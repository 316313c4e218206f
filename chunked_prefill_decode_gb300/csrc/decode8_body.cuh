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
//     x_t = (q . k_t) scale log2(e) 2^ke + ve        M = max x_t
//     P_t = 2^(x_t - M)      l = sum P_t 2^-ve       o = sum P_t v_t / l
// The V scale goes through the exponent, not onto P or v: P_t <= 1 whatever
// the scales, and a page whose values are tiny next to another's weighs as
// little in o as it should, so P fits fp16 (11 significant bits, against
// bf16's 8) for any spread of scales.  P carries a factor 2^7 that cancels in
// o, which puts fp16's smallest step at 2^-31 of the largest weight.
// q is scaled by a power of two per head so that its largest element is near
// 2^12 and every element keeps its bits in fp16; e4m3 is exact in fp16.
//
// Layout of the work, and why:
//  * the host plan gives each CTA an equal contiguous range of the decode
//    rows' pages (decode_plan.h), cut into items at row boundaries;
//  * a stage of the ring is as many pages as make eight (kv head, page)
//    pairs, K and V: one page of 8 heads, or 8 pages of one head, so a warp
//    has the same work per stage whatever the head count.  One producer warp
//    fills it with one TMA box per page and pool ([kv head][slot][D bytes],
//    swizzled by the row width);
//  * eight consumer warps, one per (head, page) pair of the stage, the
//    products taken transposed as in decode_body.cuh.  The MMA's k index may
//    run over the head dims in any order that q shares, so a lane takes its K
//    operand as 16 contiguous bytes of a key (two LDS.128 per key at D 128;
//    neighbouring rows' chunks fall into different banks under the swizzle),
//    and each 4-byte word is one k step: no ldmatrix, no shuffles.  V^T comes
//    by ldmatrix.trans of byte pairs (two dims of one key): one byte
//    permutation turns two keys' pairs into two rows of the A operand, so the
//    operand's rows r and r + 8 are dims 2r and 2r + 1 of a 16-dim block and
//    a lane's outputs are neighbours.  cvt.f16x2.e4m3x2 does two elements per
//    instruction;
//  * each warp keeps the exponents of 32 of its pages in a lane each (table
//    entry, then both exponents, a window ahead), one shuffle per page;
//  * warps that share a head (several pages per stage) merge their states in
//    shared memory at the end of an item; a row that straddles CTAs is merged
//    by its last piece through the workspace, as in decode_body.cuh.
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

constexpr int kDec8Consumers = 8;     // warps 0-7; warp 8 is the producer
constexpr int kDec8MaxStages = 14;
constexpr float kDec8RescaleThreshold = 8.0f;   // log2 units
constexpr float kDec8PShift = 7.0f;             // P <= 2^(8 + 7) in fp16

struct Stage8Header {
  DecodeItem item;
  int32_t lpage;      // first page of the stage
  int32_t first, last, end;
};
static_assert(sizeof(Stage8Header) == 64, "stage header size");

struct Decode8Layout {
  int32_t n_stages;
  int32_t pages_per_stage;
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
  L.pages_per_stage = kDec8Consumers / kvh_block;   // 8, 4, 2, 2, 1 ..: divides 32
  L.half_bytes = kvh_block * kPageSize * head_dim;
  L.stage_bytes = 2 * L.half_bytes * L.pages_per_stage;
  L.qslot_bytes = ((kvh_block * group * head_dim * 2) + 1023) / 1024 * 1024;
  L.merge_bytes = (L.pages_per_stage - 1) * kvh_block * decode8_state_floats(head_dim, group) * 4;
  const int fixed = 1024 /*align*/ + 2 * L.qslot_bytes + L.merge_bytes +
                    kDec8MaxStages * (int)sizeof(Stage8Header) + (2 * kDec8MaxStages + 5) * 8 + 64;
  int s = (227 * 1024 - fixed) / L.stage_bytes;
  if (s > kDec8MaxStages) s = kDec8MaxStages;
  L.n_stages = s;
  L.smem_bytes = fixed + s * L.stage_bytes;
  return L;
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
  Stage8Header* hdr = reinterpret_cast<Stage8Header*>(reinterpret_cast<uint8_t*>(mbuf) + L.merge_bytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(hdr + kDec8MaxStages);
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
  const int pps = L.pages_per_stage;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
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

  if (warp == kDec8Consumers) {
    // ------------------------------------------------------------ producer
    // The whole warp runs the loop: each lane holds one block-table entry of
    // a 32-page window (fetched a window ahead), lane 0 works the barriers,
    // lanes 2i and 2i + 1 issue K and V of the stage's page i.
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
      if (lane == 0) {
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
      for (int lp = it.page_begin; ok && lp < it.page_end; lp += pps) {
        const int k = (lp - it.page_begin) & 31;
        if (k == 0 && lp != it.page_begin) {
          win = win_next;
          win_next = window(it, lp + 32);
        }
        const int np = min(pps, it.page_end - lp);
        // (pps divides 32: a stage's pages lie in one window)
        int phys = __shfl_sync(0xffffffffu, win, k + (lane >> 1 < pps ? lane >> 1 : 0));
        const bool issuer = lane < 2 * np;
        if (issuer && (phys < 0 || phys >= p.num_pages)) {
          // out of range: reported, and fetched out of bounds (zeros)
          report_error(p.dev_error, HB_DEVERR_INDEX);
          phys = p.num_pages;
        }
        // a decode row's new token (position ctx - 1, written by the append
        // before this launch) is on its last page
        if (!dep_done && lp + np - 1 >= (it.ctx - 1) / kPageSize) {
          griddep_wait();
          fence_proxy_async_global();
          dep_done = true;
        }
        if (lane == 0) {
          ok = mbar_wait(&empty[st], ph ^ 1u, abort_flag);
          if (ok) {
            Stage8Header& h = hdr[st];
            h.item = it;
            h.lpage = lp;
            h.first = lp == it.page_begin;
            h.last = lp + pps >= it.page_end;
            h.end = 0;
            mbar_arrive_expect_tx(&full[st], 2u * (uint32_t)(np * L.half_bytes));
            issued_mask |= 1u << st;
            last_par_mask = (last_par_mask & ~(1u << st)) | (ph << st);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (ok && issuer)
          tma_load_4d(stages + st * L.stage_bytes + lane * L.half_bytes, (lane & 1) ? &vmap : &kmap,
                      &full[st], 0, 0, it.kvh0, phys);
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
    if (lane == 0) {
      if (ok && mbar_wait(&empty[st], ph ^ 1u, abort_flag)) {
        hdr[st].end = 1;
        issued_mask &= ~(1u << st);  // its earlier copy was consumed
        mbar_arrive(&full[st]);
      }
      for (int s2 = 0; s2 < S; ++s2)
        if (issued_mask & (1u << s2)) drain_wait(&full[s2], (last_par_mask >> s2) & 1u, abort_flag);
    }
  } else if (warp < kDec8Consumers) {
    // ------------------------------------------------------------ consumers
    auto consume = [&](auto nq_const) {
      constexpr int NQ = decltype(nq_const)::value;   // 8-head column tiles
      constexpr int KC = D / 64;                      // 16-byte K chunks per lane and key
      const int w = warp % kvhb;                      // local kv head of this warp
      const int part = warp / kvhb;                   // its page of a stage
      const bool active = part < pps;
      const int r = lane >> 2, c = lane & 3;
      const int mi = lane >> 3, r8 = lane & 7;        // ldmatrix: matrix, row
      uint32_t qb[D / 16][NQ][2];          // B operand Q^T
      float o[D / 16][NQ][4];              // O^T: dims 16 jj + 2 r (+ 1 in [2], [3]), heads 2c, 2c + 1
      float m_run[NQ][2], l_part[NQ][2];   // head 8 nq + 2c + e; l over this lane's keys
      float qs[NQ][2];                     // softmax scale * log2(e) * 2^(q's exponent)
      int e_cur = 0, e_next = 0, raw_next = -1;   // exponents ke | ve << 8 of one page per lane
      int t = 0;                           // stage of the item
      // All consumers get here, and see what the others wrote before; false
      // if one of them has given up.  (A bounded wait: a hardware barrier
      // would wait for a warp that left.)
      uint32_t tph = 0;
      auto all_here = [&]() -> bool {
        __syncwarp();
        if (lane == 0) mbar_arrive(together);
        const bool ok = mbar_wait(together, tph, abort_flag);
        tph ^= 1u;
        return ok;
      };
      // what the append wrote (the exponents of the last pages) is complete
      griddep_wait();

      int st = 0;
      uint32_t ph = 0;
      int qslot = 0;
      uint32_t qph[2] = {0u, 0u};
      while (true) {
        if (!mbar_wait(&full[st], ph, abort_flag)) break;
        const Stage8Header& h = hdr[st];
        if (h.end) break;
        // (the stage, and with it the header, goes back to the producer
        // before the end of the page: what is needed later is read here)
        const int ctx = h.item.ctx, page_end = h.item.page_end, kvh0 = h.item.kvh0;
        const int lp = h.lpage + part;
        const bool first = h.first, last = h.last;
        const int it_tok = h.item.tok, it_splits = h.item.n_splits, it_split = h.item.split;
        const int it_slot = h.item.slot, it_merge = h.item.merge_id;
        // one page per lane: table entry (raw), then its exponents
        const int32_t* bt = p.block_table + (size_t)h.item.seq * p.max_pages_per_seq;
        auto entry = [&](int wbase) -> int {
          const int x = lp + (wbase + lane) * pps;
          return (x < page_end && x < p.max_pages_per_seq) ? __ldcg(&bt[x]) : -1;
        };
        auto exponents = [&](int raw) -> int {
          if ((unsigned)raw >= (unsigned)p.num_pages) return 0;
          const size_t at = (size_t)raw * p.num_kv_heads + kvh0 + w;
          return (kv8_exp(ldcg_s8(p8.k_exp + at)) & 0xff) | (kv8_exp(ldcg_s8(p8.v_exp + at)) << 8);
        };
        if (first) {
          t = 0;
          if (active) e_cur = exponents(entry(0));
          if (!mbar_wait(&qfull[qslot], qph[qslot], abort_flag)) break;
          qph[qslot] ^= 1u;
          if (active) {
            const uint16_t* q0 = reinterpret_cast<const uint16_t*>(qbuf + qslot * L.qslot_bytes) +
                                 (size_t)w * g * D;
            float mul[NQ];
            int qe[NQ];
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
              qe[nq] = min(max((int)(mx >> 7) - 127 - 12, -100), 115);
              mul[nq] = pow2i(-qe[nq]);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                  const uint32_t v = qb[kk][nq][x];
                  qb[kk][nq][x] = pack_f16x2(bf16lo_to_f32(v) * mul[nq], bf16hi_to_f32(v) * mul[nq]);
                }
#pragma unroll
              for (int e = 0; e < 2; ++e)   // the head of accumulator column 2c + e
                qs[nq][e] = p.scale_log2 * pow2i(__shfl_sync(0xffffffffu, qe[nq], (2 * c + e) * 4));
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
        }
        const int tl = t & 31;
        if (active) {
          if (tl == 0) {
            if (t > 0) e_cur = e_next;
            raw_next = entry(32);
          } else if (tl == 8) {
            e_next = exponents(raw_next);
          }
        }
        const int ex = __shfl_sync(0xffffffffu, e_cur, tl);
        ++t;

        if (active && lp < page_end) {
          const uint8_t* kst = stages + st * L.stage_bytes + 2 * part * L.half_bytes;
          const uint32_t kbase = smem_u32(kst) + (uint32_t)(w * kPageSize * D);
          const uint32_t vbase = kbase + (uint32_t)L.half_bytes;
          const int valid = min(kPageSize, ctx - lp * kPageSize);
          // with a sliding window the row sees keys ctx - W .. ctx - 1 only
          const int lo_valid = p.window > 0 ? ctx - p.window - lp * kPageSize : 0;
          // byte address of 16-byte chunk u of key row `row`
          auto chunk = [&](uint32_t base, int row, int u) -> uint32_t {
            if constexpr (D == 128) return base + (uint32_t)(row * 128 + ((u ^ (row & 7)) << 4));
            return base + (uint32_t)(row * 64 + ((u ^ ((row >> 1) & 3)) << 4));
          };
          uint4 kr[2][KC];                 // keys r and r + 8
#pragma unroll
          for (int i = 0; i < KC; ++i) {
            kr[0][i] = lds128(chunk(kbase, r, KC * c + i));
            kr[1][i] = lds128(chunk(kbase, r + 8, KC * c + i));
          }
          // V byte pairs, transposed: matrices (keys 0-7, 8-15) of chunks 2 j, 2 j + 1
          uint32_t vr[D / 32][4];
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            ldsm_x4_trans(chunk(vbase, ((mi & 1) << 3) + r8, 2 * j + (mi >> 1)), vr[j][0], vr[j][1],
                          vr[j][2], vr[j][3]);
          // K and V of the page are in registers: the stage goes back
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
          constexpr int kQk = NQ == 1 ? 4 : 2;
          float s[kQk][NQ][4];
#pragma unroll
          for (int x = 0; x < kQk; ++x)
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) s[x][nq][0] = s[x][nq][1] = s[x][nq][2] = s[x][nq][3] = 0.f;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint4 k0 = kr[0][kk / 4], k1 = kr[1][kk / 4];
            const uint32_t w0 = (kk & 3) == 0 ? k0.x : (kk & 3) == 1 ? k0.y : (kk & 3) == 2 ? k0.z : k0.w;
            const uint32_t w1 = (kk & 3) == 0 ? k1.x : (kk & 3) == 1 ? k1.y : (kk & 3) == 2 ? k1.z : k1.w;
            const uint32_t ka[4] = {f16x2_of_e4m3x2(w0), f16x2_of_e4m3x2(w1), f16x2_of_e4m3x2(w0 >> 16),
                                    f16x2_of_e4m3x2(w1 >> 16)};
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
              mma_f16_16816(s[kk % kQk][nq], ka, qb[kk][nq][0], qb[kk][nq][1]);
          }
          if (valid < kPageSize || lo_valid > 0) {
            // values of keys that the row does not see may be anything, NaN
            // included: cleared, since P = 0 would not stop it
            const auto seen = [&](int key) { return key < valid && key >= lo_valid; };
            uint32_t m0 = (seen(2 * c) ? 0xffffu : 0u) | (seen(2 * c + 1) ? 0xffff0000u : 0u);
            uint32_t m1 = (seen(2 * c + 8) ? 0xffffu : 0u) | (seen(2 * c + 9) ? 0xffff0000u : 0u);
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
              vr[j][0] &= m0;
              vr[j][1] &= m1;
              vr[j][2] &= m0;
              vr[j][3] &= m1;
            }
          }
          const int ke = (int)(int8_t)(ex & 0xff), ve = ex >> 8;
          const float fk = pow2i(ke), fv = (float)ve, inv_v = pow2i(-ve);
          const bool ok0 = r < valid && r >= lo_valid;
          const bool ok1 = r + 8 < valid && r + 8 >= lo_valid;
          float x0[NQ][2], x1[NQ][2], alpha[NQ][2];
          bool need = false;
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float a0 = s[0][nq][e], a1 = s[0][nq][2 + e];
#pragma unroll
              for (int x = 1; x < kQk; ++x) {
                a0 += s[x][nq][e];
                a1 += s[x][nq][2 + e];
              }
              const float cs = qs[nq][e] * fk;
              x0[nq][e] = ok0 ? fmaf(a0, cs, fv) : -INFINITY;
              x1[nq][e] = ok1 ? fmaf(a1, cs, fv) : -INFINITY;
              need |= fmaxf(x0[nq][e], x1[nq][e]) > m_run[nq][e] + kDec8RescaleThreshold;
              alpha[nq][e] = 1.f;
            }
          if (__any_sync(0xffffffffu, need)) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(x0[nq][e], x1[nq][e]);
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
          uint32_t pb[NQ][2];
#pragma unroll
          for (int nq = 0; nq < NQ; ++nq) {
            float p0[2], p1[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // no key seen yet: every x is -inf and so is P's exponent
              const float mu = (m_run[nq][e] == -INFINITY ? 0.f : m_run[nq][e]) - kDec8PShift;
              p0[e] = fast_exp2(x0[nq][e] - mu);
              p1[e] = fast_exp2(x1[nq][e] - mu);
              l_part[nq][e] = fmaf(p0[e] + p1[e], inv_v, l_part[nq][e] * alpha[nq][e]);
            }
            pb[nq][0] = movmatrix_trans(pack_f16x2(p0[0], p0[1]));   // B: keys 2c, 2c + 1 of head r
            pb[nq][1] = movmatrix_trans(pack_f16x2(p1[0], p1[1]));   // keys 8 + 2c ..
          }
          // O^T += V^T P^T
#pragma unroll
          for (int jj = 0; jj < D / 16; ++jj) {
            // bytes (key 0: dims 0, 1; key 1: dims 0, 1) -> (dim 0: keys 0, 1; dim 1: ..)
            const uint32_t v0 = __byte_perm(vr[jj / 2][2 * (jj & 1)], 0u, 0x3120);
            const uint32_t v1 = __byte_perm(vr[jj / 2][2 * (jj & 1) + 1], 0u, 0x3120);
            const uint32_t va[4] = {f16x2_of_e4m3x2(v0), f16x2_of_e4m3x2(v0 >> 16), f16x2_of_e4m3x2(v1),
                                    f16x2_of_e4m3x2(v1 >> 16)};
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) mma_f16_16816(o[jj][nq], va, pb[nq][0], pb[nq][1]);
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[st]);
        }

        if (last) {
          const int Hq = p.num_q_heads;
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
          if (pps > 1) {
            // warps of one head: parts 1 .. leave their state, lane by lane
            // (the fragments have the same owners), part 0 takes them in
            const int n = decode8_state_floats(D, g);
            if (active && part > 0) {
              float* dst = mbuf + (size_t)((part - 1) * kvhb + w) * n + lane;
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
                  for (int x = 0; x < 4; ++x) dst[32 * k++] = o[jj][nq][x];
            }
            if (!all_here()) break;
            if (part == 0) {
#pragma unroll 1
              for (int i = 1; i < pps; ++i) {
                const float* src = mbuf + (size_t)((i - 1) * kvhb + w) * n + lane;
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
                  }
#pragma unroll
                for (int jj = 0; jj < D / 16; ++jj)
#pragma unroll
                  for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                      o[jj][nq][x] = o[jj][nq][x] * wa[nq][x & 1] + src[32 * k++] * wb[nq][x & 1];
              }
            }
            if (!all_here()) break;   // the buffer may be written again
          }
          if (part == 0) {
            const int head0 = (kvh0 + w) * g;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int head = nq * 8 + 2 * c + e;
                if (head >= g) continue;
                if (it_splits == 1) {
                  const float inv = 1.f / l_tot[nq][e];
                  uint32_t* dst = reinterpret_cast<uint32_t*>(
                      p.out + ((size_t)it_tok * Hq + head0 + head) * D + 2 * r);
#pragma unroll
                  for (int jj = 0; jj < D / 16; ++jj)
                    dst[jj * 8] = pack_bf16x2(o[jj][nq][e] * inv, o[jj][nq][2 + e] * inv);
                } else {
                  const size_t slot = (size_t)(it_slot + it_split);
                  float* dst = p.part_o + (slot * Hq + head0 + head) * D + 2 * r;
#pragma unroll
                  for (int jj = 0; jj < D / 16; ++jj)
                    *reinterpret_cast<float2*>(dst + jj * 16) = make_float2(o[jj][nq][e], o[jj][nq][2 + e]);
                  if (r == 0)
                    reinterpret_cast<float2*>(p.part_ml)[slot * Hq + head0 + head] =
                        make_float2(m_run[nq][e], l_tot[nq][e]);
                }
              }
          }
          if (it_splits > 1) {
            // publish this piece's state: the barrier orders every consumer's
            // stores before thread 0's device-scope fence + atomic
            if (!all_here()) break;
            if (threadIdx.x == 0) {
              __threadfence();
              const int old = atomicAdd(&p.counters[kCounterMerge0 + it_merge], 1);
              __threadfence();  // acquire: the other pieces' states are visible
              flags[1] = (old == it_splits - 1) ? 1 : 0;
            }
            if (!all_here()) break;
            if (flags[1]) {
              __threadfence();
              // one warp per q head of the block; each lane owns D / 32 dims
              constexpr int E = D / 32;
              const float2* ml = reinterpret_cast<const float2*>(p.part_ml);
              for (int hl = warp; hl < kvhb * g; hl += kDec8Consumers) {
                const int hh = kvh0 * g + hl;
                float mmax = -INFINITY;
                for (int i = 0; i < it_splits; ++i)
                  mmax = fmaxf(mmax, __ldcg(&ml[(size_t)(it_slot + i) * Hq + hh]).x);
                float acc[E];
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] = 0.f;
                float lsum = 0.f;
#pragma unroll 4
                for (int i = 0; i < it_splits; ++i) {
                  const size_t slot = (size_t)(it_slot + i);
                  const float2 st2 = __ldcg(&ml[slot * Hq + hh]);
                  const float wgt = fast_exp2(st2.x - mmax);
                  lsum += wgt * st2.y;
                  const float* po = p.part_o + (slot * Hq + hh) * D + lane * E;
                  if constexpr (E == 4) {
                    const float4 v = __ldcg(reinterpret_cast<const float4*>(po));
                    acc[0] += wgt * v.x; acc[1] += wgt * v.y;
                    acc[2] += wgt * v.z; acc[3] += wgt * v.w;
                  } else {
                    const float2 v = __ldcg(reinterpret_cast<const float2*>(po));
                    acc[0] += wgt * v.x; acc[1] += wgt * v.y;
                  }
                }
                const float inv = 1.f / lsum;
                uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((size_t)it_tok * Hq + hh) * D + lane * E);
#pragma unroll
                for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
              }
              if (threadIdx.x == 0) p.counters[kCounterMerge0 + it_merge] = 0;
            }
          }
        }
        if (++st == S) {
          st = 0;
          ph ^= 1u;
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
