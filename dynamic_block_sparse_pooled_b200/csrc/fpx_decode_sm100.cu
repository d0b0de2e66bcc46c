// fpx_decode_sm100.cu -- the shared prompts of fpx_decode on the tensor cores of the fifth
// generation (bf16 caches, head dim 128): the rows of all requests of a group, times the query heads
// of a KV head, against the prompt's keys.
//
// With r rows per KV head each cached byte is used for r multiply-adds, so from about 200 rows on
// the work is bound by the tensor cores, not by HBM (a 32768-token prompt behind 128 requests of 4
// heads per KV head: 69 GFLOP, 134 MB; 88 us, 780 TFLOP/s, the tensor pipe 38 % busy: the softmax
// chain of 2.5 us per pair of tiles sets the pace, and 10 us go into starting and the partials; an L2
// prefetch four tiles ahead made it slower).  At 208 registers the softmax threads spill 96 words without
// cap and bias, 59 to 79 with them (-Xptxas -v).  P is in bf16, as V is; its sum is of the weights
// before that rounding.  The pipeline is that of the prefill attention
// (fpx_attn_sm100.cuh): two 128-row tiles per CTA, S and O in TMEM, P over S, one warp that issues
// every MMA in a fixed order, one that loads by TMA, two softmax warpgroups; K / V rings of two
// 128-key slots.  A CTA's work is a stretch of the line of tiles (fpx_decode.cuh) instead of a unit.
//   Two row tiles (more than 128 rows): both use every key tile, loaded once.
//   One row tile: the two softmax warpgroups take the key tiles in turn with the same Q, so that the
//   one's softmax still overlaps the other's MMAs; each leaves a partial of its own.
// Rows of a tile are tokens x heads of one KV head, token-major: one 3-D TMA box of Q.  Pages are
// whole (the shared range ends on a page border); a page of fewer than 128 keys takes several
// boxes, the part of a tile behind the range's end is filled with zeros by a box outside the cache.
#include <cuda.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include <climits>

#include "fpx_decode.cuh"
#include "fpx_internal.h"
#include "fpx_softmax.cuh"

namespace fpx {
namespace decode {

using namespace sm100;

namespace {

constexpr int kTileKeys = 128;
constexpr int kDim = 128;
constexpr int kTcThreads = 384;
// 256 softmax threads x 208 + 128 others x 88 registers <= 384 x 168
constexpr int kSoftmaxRegs = 208, kOtherRegs = 88;
constexpr int kMmaWarp = 8, kLoadWarp = 10;
constexpr uint32_t kBox = 128 * 128;       // 128 rows x 128 bytes
constexpr uint32_t kSlot = 2 * kBox;       // 128 x 128 bf16
constexpr uint32_t kOffQ = 0, kOffK = 2 * kSlot, kOffV = 4 * kSlot, kOffBar = 6 * kSlot;
constexpr size_t kTcSmem = 6 * kSlot + 512 + 1024;
constexpr int kSteps = kDim / 16;
constexpr uint32_t kIdescQK = make_idesc(1, 1, false, 128, 128);
constexpr uint32_t kIdescPV = make_idesc(1, 1, true, 128, 128);

enum Bar {
  kBarQ = 0, kBarQEmpty = 1,
  kBarKFull = 2, kBarKEmpty = 4, kBarVFull = 6, kBarVEmpty = 8,  // + slot
  kBarSFull = 10, kBarPReady = 12, kBarODone = 14,               // + tile
  kBarDrain = 16,
  kBarUFull = 17, kBarUEmpty = 19,                               // + slot of the piece ring
  kNumBars = 21
};
constexpr int kReaders = 9;  // the MMA warp and the eight softmax warps

// A stretch of key tiles of one segment, as the load warp hands it to the other roles through a
// two-slot ring in shared memory (they would each spend registers on the walk along the line).
struct Piece {
  int cnt;         // key tiles; 0 ends the CTA's work
  int key0, k1;    // first key, end of the segment's range
  int kvh;
  int ntiles;      // row tiles of the pair
  int tok, tok1;   // first query token of the pair, end of the group's
  int slot;        // partial slot
};
__device__ __forceinline__ Piece piece_of(const Walk& c, int tpt, int worker) {
  Piece p;
  p.kvh = c.j / c.w.nrt;
  const int pair = c.j - p.kvh * c.w.nrt;
  p.cnt = c.cnt;
  p.key0 = c.w.k0 + c.t0 * kTileKeys;
  p.k1 = c.w.k1;
  p.ntiles = c.w.ntok - pair * 2 * tpt > tpt ? 2 : 1;
  p.tok = c.w.tok0 + pair * 2 * tpt;
  p.tok1 = c.w.tok0 + c.w.ntok;
  p.slot = c.w.seg + c.j + worker;
  return p;
}
template <bool kCap, bool kBias>
__global__ void __launch_bounds__(kTcThreads, 1)
decode_tc_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                 const __grid_constant__ CUtensorMap tmV, const __grid_constant__ DecodeDesc p,
                 const __grid_constant__ Line line, StatusBlock* st) {
  constexpr unsigned kFull = 0xffffffffu;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t sbase = (raw_u32 + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - raw_u32);
  const uint32_t bar0 = sbase + kOffBar;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + kOffBar + 8 * kNumBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + kOffBar + 8 * kNumBars + 4);
  Piece* ring = reinterpret_cast<Piece*>(gbase + kOffBar + 256);
  static_assert(8 * kNumBars + 8 <= 256 && 2 * sizeof(Piece) <= 256, "shared memory layout");
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(bar(kBarQ), 1);
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarKFull + i), 1);
      mbar_init(bar(kBarKEmpty + i), 1);
      mbar_init(bar(kBarVFull + i), 1);
      mbar_init(bar(kBarVEmpty + i), 1);
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPReady + i), 4);  // one arrival per softmax warp
      mbar_init(bar(kBarODone + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarUFull + i), 1);
      mbar_init(bar(kBarUEmpty + i), kReaders);
    }
    mbar_init(bar(kBarDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_enter();  // after the previous kernel on the stream, which the set-up above overlaps
  // Piece k of this CTA; false on a timeout.  Warp-uniform.
  auto take_piece = [&](int k, Piece& w) -> bool {
    if (!__all_sync(kFull, mbar_wait(bar(kBarUFull + (k & 1)), (k >> 1) & 1, abort_flag)))
      return false;
    w = ring[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(kBarUEmpty + (k & 1)));
    return true;
  };

  if (warp >= 8) {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kLoadWarp) {
      // ---------------------------------------------------------------- TMA producer ----
      const int rows = min(p.page, kTileKeys);  // keys of a box
      const int pieces = kTileKeys / rows;      // boxes of a tile along the keys
      int n = 0, k = 0;                         // ring entries, pieces of the line
      bool ok = true;
      const int64_t total = line.owners[line.n].line;
      const int64_t nw = active_workers(line, total);
      const int worker = blockIdx.x;
      Walk cur;
      if (worker < nw)
        cur.enter(line, static_cast<int>(line_begin(worker, total, nw)),
                  static_cast<int>(line_begin(worker + 1, total, nw)));
      else
        cur.left = 0;
      int u = 0;  // pieces published
      while (true) {
        Piece w = {};
        if (cur.next(p.hkv)) w = piece_of(cur, line.tpt, worker);
        if (!__all_sync(kFull, mbar_wait(bar(kBarUEmpty + (u & 1)), ((u >> 1) & 1) ^ 1, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          ring[u & 1] = w;
          mbar_arrive(bar(kBarUFull + (u & 1)));  // release: the slot's write is visible first
        }
        __syncwarp();
        ++u;
        if (w.cnt == 0) break;
        if (k > 0 && !__all_sync(kFull, mbar_wait(bar(kBarQEmpty), (k - 1) & 1, abort_flag))) {
          ok = false;
          break;
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(bar(kBarQ), w.ntiles * line.tpt * p.group * 256);
          for (int t = 0; t < w.ntiles; ++t)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tma_load_3d(sbase + kOffQ + t * kSlot + b * kBox, &tmQ, bar(kBarQ), b * 64,
                          w.kvh * p.group, w.tok + t * line.tpt);
        }
        __syncwarp();
        ++k;
        for (int e = 0; e < w.cnt; ++e) {
          const int slot = n & 1;
          const uint32_t ph = (n >> 1) & 1;
          // cache row of box `lane`; behind the range's end or outside the cache: zeros
          int row = p.num_pages << p.log2_page;
          const int key = w.key0 + e * kTileKeys + lane * rows;
          if (lane < pieces && key < w.k1) {
            const int pg = p.table[static_cast<int64_t>(cur.w.row) * p.pages_per_seq + (key >> p.log2_page)];
            if (pg < 0 || pg >= p.num_pages)
              record_error(st, FPX_ERR_DEVICE_INPUT, 70, cur.w.row, key >> p.log2_page);
            else
              row = (pg << p.log2_page) + (key & (p.page - 1));
          }
          if (!__all_sync(kFull, mbar_wait(bar(kBarKEmpty + slot), ph ^ 1, abort_flag))) {
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarKFull + slot), kSlot);
          __syncwarp();
          if (lane < pieces)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tma_load_3d(sbase + kOffK + slot * kSlot + b * kBox + lane * rows * 128, &tmK,
                          bar(kBarKFull + slot), b * 64, w.kvh, row);
          if (!__all_sync(kFull, mbar_wait(bar(kBarVEmpty + slot), ph ^ 1, abort_flag))) {
            volatile int never = 0;  // K of this entry is in flight
            mbar_wait(bar(kBarKFull + slot), ph, &never);
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(bar(kBarVFull + slot), kSlot);
          __syncwarp();
          if (lane < pieces)
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tma_load_3d(sbase + kOffV + slot * kSlot + b * kBox + lane * rows * 128, &tmV,
                          bar(kBarVFull + slot), b * 64, w.kvh, row);
          ++n;
        }
        if (!ok) break;
      }
      if (!ok) *abort_flag = 1;
      // every load in flight lands before shared memory is given up
      volatile int never = 0;
      if (k > 0) mbar_wait(bar(kBarQ), (k - 1) & 1, &never);
      for (int e = max(0, n - 2); e < n; ++e) {
        mbar_wait(bar(kBarKFull + (e & 1)), (e >> 1) & 1, &never);
        mbar_wait(bar(kBarVFull + (e & 1)), (e >> 1) & 1, &never);
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- MMA issuer -------
      const uint64_t dq0 = smem_desc_sw128(sbase + kOffQ, 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(sbase + kOffK, 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(sbase + kOffV, 16384, 1024);
      constexpr uint64_t kSlotDesc = kSlot >> 4;
      const uint32_t tS0 = tmem, tS1 = tmem + 128, tO0 = tmem + 256, tO1 = tmem + 384;
      auto issue_s = [&](uint32_t tS, uint64_t dq, int slot) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const uint64_t off = ((kk / 4) * kBox + (kk % 4) * 32) >> 4;
          mma_f16_ss(tS, dq + off, dk0 + slot * kSlotDesc + off, kIdescQK, kk > 0);
        }
      };
      auto issue_pv = [&](uint32_t tO, uint32_t tS, int slot, bool started) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk)
          mma_f16_ts(tO, tS + kk * 8, dv0 + slot * kSlotDesc + ((kk * 16 * 128) >> 4), kIdescPV,
                     (started || kk > 0) ? 1u : 0u);
      };
      int n = 0, k = 0;
      uint32_t ph_p0 = 0, ph_p1 = 0;
      bool ok = true;
      auto wait = [&](int b, uint32_t ph) {
        ok = __all_sync(kFull, mbar_wait(bar(b), ph, abort_flag));
        return ok;
      };
      while (true) {
        Piece w;
        if (!take_piece(k, w)) {
          ok = false;
          break;
        }
        if (w.cnt == 0) break;
        if (!wait(kBarQ, k & 1)) break;
        ++k;
        bool o1 = false;
        if (!wait(kBarKFull + (n & 1), (n >> 1) & 1)) break;
        if (elect_one()) {  // S_0 of the first entry
          tc_fence_after();
          issue_s(tS0, dq0, n & 1);
          mma_commit(bar(kBarSFull + 0));
          if (w.ntiles == 1) mma_commit(bar(kBarKEmpty + (n & 1)));
        }
        __syncwarp();
        if (w.ntiles == 2) {
          // per entry: O_1 += P_1 V of the previous one, S_1 | O_0 += P_0 V, S_0 of the next one
          for (int e = 0; e < w.cnt; ++e, ++n) {
            const int slot = n & 1, ps = slot ^ 1;
            if (e > 0) {
              if (!wait(kBarPReady + 1, ph_p1)) break;
              ph_p1 ^= 1;
            }
            if (elect_one()) {
              tc_fence_after();
              if (e > 0) {
                issue_pv(tO1, tS1, ps, o1);
                mma_commit(bar(kBarVEmpty + ps));
              }
              issue_s(tS1, dq0 + kSlotDesc, slot);
              mma_commit(bar(kBarSFull + 1));
              mma_commit(bar(kBarKEmpty + slot));
            }
            __syncwarp();
            o1 = e > 0;
            const bool next = e + 1 < w.cnt;
            if (next && !wait(kBarKFull + ps, ((n + 1) >> 1) & 1)) break;
            if (!wait(kBarPReady + 0, ph_p0)) break;
            ph_p0 ^= 1;
            if (!wait(kBarVFull + slot, (n >> 1) & 1)) break;
            if (elect_one()) {
              tc_fence_after();
              issue_pv(tO0, tS0, slot, e > 0);
              if (next) {
                issue_s(tS0, dq0, ps);
                mma_commit(bar(kBarSFull + 0));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) mma_commit(bar(kBarQEmpty));  // every S of the piece is issued
          __syncwarp();
          if (!wait(kBarPReady + 1, ph_p1)) break;
          ph_p1 ^= 1;
          if (elect_one()) {
            tc_fence_after();
            issue_pv(tO1, tS1, (n - 1) & 1, o1);
            mma_commit(bar(kBarVEmpty + ((n - 1) & 1)));
            mma_commit(bar(kBarODone + 0));
            mma_commit(bar(kBarODone + 1));
          }
          __syncwarp();
        } else {
          // entries in turn: O_t += P_t V, S_t of the entry after next
          if (w.cnt > 1) {
            const int slot = (n + 1) & 1;
            if (!wait(kBarKFull + slot, ((n + 1) >> 1) & 1)) break;
            if (elect_one()) {
              tc_fence_after();
              issue_s(tS1, dq0, slot);
              mma_commit(bar(kBarSFull + 1));
              mma_commit(bar(kBarKEmpty + slot));
            }
            __syncwarp();
          }
          for (int e = 0; e < w.cnt; ++e, ++n) {
            const int slot = n & 1;
            const bool next = e + 2 < w.cnt;
            if (next && !wait(kBarKFull + slot, ((n + 2) >> 1) & 1)) break;
            if ((e & 1) == 0) {
              if (!wait(kBarPReady + 0, ph_p0)) break;
              ph_p0 ^= 1;
            } else {
              if (!wait(kBarPReady + 1, ph_p1)) break;
              ph_p1 ^= 1;
            }
            if (!wait(kBarVFull + slot, (n >> 1) & 1)) break;
            const uint32_t tS = (e & 1) ? tS1 : tS0, tO = (e & 1) ? tO1 : tO0;
            if (elect_one()) {
              tc_fence_after();
              issue_pv(tO, tS, slot, e > 1);
              mma_commit(bar(kBarVEmpty + slot));
              if (next) {
                issue_s(tS, dq0, slot);
                mma_commit(bar(kBarSFull + (e & 1)));
                mma_commit(bar(kBarKEmpty + slot));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) {
            mma_commit(bar(kBarQEmpty));
            mma_commit(bar(kBarODone + 0));
            if (w.cnt > 1) mma_commit(bar(kBarODone + 1));
          }
          __syncwarp();
        }
      }
      if (!ok) *abort_flag = 1;
      if (elect_one()) mma_commit(bar(kBarDrain));
      volatile int never = 0;
      mbar_wait(bar(kBarDrain), 0, &never);
    }
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    // ------------------------------------------------------------------ softmax ----------
    const int t = warp >> 2;  // softmax warpgroup
    const int row = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + t * 128 + lane_base;
    const uint32_t tO = tmem + 256 + t * 128 + lane_base;
    uint32_t s_phase = 0, od_phase = 0;
    bool ok = true;
    int it = 0;
    for (int k = 0;; ++k) {
      Piece w;
      if (!take_piece(k, w)) {
        ok = false;
        break;
      }
      if (w.cnt == 0) break;
      const int rt = w.ntiles == 2 ? t : 0;  // row tile that this warpgroup works on
      const int tk = w.tok + rt * line.tpt + row / p.group;
      const bool valid = row < line.tpt * p.group && tk < w.tok1;
      const int head = w.kvh * p.group + row % p.group;
      RowPos rp = row_pos(p, valid ? tk : w.tok);
      // rows of no query hold leftovers of shared memory: masked, they decide nothing for their warp
      if (!valid) rp.span = {0, -1};
      rp.span.hi = min(rp.span.hi, w.k1 - 1);
      const ScoreMap map = score_map(p.rule, p.scale, head);
      TanhPoly poly = {};
      if (kCap) poly.set(map.cap2);
      const float sl2 = kCap || kBias ? 1.f : map.k;
      float m_ref = -CUDART_INF_F, l_run = 0.f;
      it = 0;
      // with one row tile the two warpgroups take the key tiles in turn
      const int stride = w.ntiles == 2 ? 1 : 2;
      for (int e = w.ntiles == 2 ? 0 : t; e < w.cnt; e += stride) {
        const int kb = w.key0 + e * kTileKeys;
        const int c_lo = rp.span.lo - kb, c_hi = rp.span.hi - kb;
        const int partial = (__any_sync(kFull, c_lo > 0) ? 1 : 0) |
                            (__any_sync(kFull, c_hi < kTileKeys - 1) ? 2 : 0);
        const float rel = static_cast<float>(rp.i - kb);
        if (!__all_sync(kFull, mbar_wait(bar(kBarSFull + t), s_phase, abort_flag))) {
          ok = false;
          break;
        }
        s_phase ^= 1;
        tc_fence_after();
        uint32_t r[128];
        tmem_ld32(tS, r);
        tmem_ld32(tS + 32, r + 32);
        tmem_wait_ld(r);
        tmem_wait_ld(r + 32);
        tmem_ld32(tS + 64, r + 64);
        tmem_ld32(tS + 96, r + 96);
        rule_half<kCap, kBias>(r, 0, map, poly, rel, c_lo, c_hi, partial);
        const float mx_lo = row_max64(r);
        tmem_wait_ld(r + 64);
        tmem_wait_ld(r + 96);
        rule_half<kCap, kBias>(r + 64, 64, map, poly, rel, c_lo, c_hi, partial);
        const float mx = fmaxf(mx_lo, row_max64(r + 64)) * sl2;
        float corr = 1.f;
        if (mx > m_ref + kRescaleLog2) {
          corr = ex2_approx(m_ref - mx);  // 0 for the first keys
          l_run *= corr;
          m_ref = mx;
        }
        if (it > 0 && __any_sync(kFull, corr != 1.f)) {
          // O_t is stable: the previous P V into it completed before S_t was written
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t ov[32];
            tmem_ld32(tO + c * 32, ov);
            tmem_wait_ld(ov);
#pragma unroll
            for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * corr);
            tmem_st32(tO + c * 32, ov);
          }
        }
        const float neg_m = m_ref == -CUDART_INF_F ? 0.f : -m_ref;
        float rs = softmax_part_to_p<false, false, 0, 64>(r, sl2, neg_m);
        tmem_st32(tS, r);
        rs += softmax_part_to_p<false, false, 64, 64>(r, sl2, neg_m);
        tmem_st32(tS + 32, r + 32);
        l_run += rs;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarPReady + t));
        ++it;
      }
      if (!ok) break;
      // the piece's partial: tile t's rows are 128 t .. 128 t + 127 of the slot
      const int64_t at = static_cast<int64_t>(w.slot) * line.rps + t * 128 + row;
      if (valid) line.part_ml[at] = make_float2(m_ref, l_run);
      if (it > 0) {
        if (!__all_sync(kFull, mbar_wait(bar(kBarODone + t), od_phase, abort_flag))) {
          ok = false;
          break;
        }
        od_phase ^= 1;
        tc_fence_after();
        float4* dst = reinterpret_cast<float4*>(line.part_o + at * kDim);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(tO + c * 32, r);
          tmem_wait_ld(r);
          if (valid) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              dst[c * 8 + i] =
                  make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]),
                              __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
          }
        }
        // read before the next piece's first P V into these columns, which waits for this
        // warp's first P of that piece
        tc_fence_before();
      }
    }
    if (!ok) {
      *abort_flag = 1;
      if (row == 0) record_error(st, FPX_ERR_TIMEOUT, 71, static_cast<int>(blockIdx.x), it);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

bool tc_supported(const DecodeDesc& p, fpx_dtype dt) {
  return dt == FPX_BF16 && p.d == kDim && p.group <= 128;
}

void tc_line(const DecodeDesc& p, Line* l) {
  l->tpt = 128 / p.group;
  l->rt = 2 * l->tpt * p.group;
  l->tile = kTileKeys;
  l->rps = 256;
}

template <bool kCap, bool kBias>
static cudaError_t launch_tc_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                               const DecodeDesc& p, const Line& line, StatusBlock* st,
                               cudaStream_t s) {
  const cudaError_t e = allow_smem<decode_tc_kernel<kCap, kBias>>(kTcSmem);
  if (e != cudaSuccess) return e;
  FPX_CHAIN((decode_tc_kernel<kCap, kBias>), line.nw, kTcThreads, kTcSmem, s, mq, mk, mv, p, line,
            st);
  return cudaGetLastError();
}

cudaError_t launch_tc(const DecodeDesc& p, const Line& line, const void* q, const void* kc,
                      const void* vc, StatusBlock* st, cudaStream_t s, bool* encode_failed) {
  CUtensorMap mq, mk, mv;
  const int rows = p.num_pages << p.log2_page;
  const int box = p.page < kTileKeys ? p.page : kTileKeys;
  if (!make_tmap_heads(&mq, q, p.tokens, p.hq, p.d, p.group, line.tpt) ||
      !make_tmap_rows(&mk, kc, rows, p.hkv, p.d, 2, 64, box) ||
      !make_tmap_rows(&mv, vc, rows, p.hkv, p.d, 2, 64, box)) {
    *encode_failed = true;
    return cudaErrorInvalidValue;
  }
  const bool cap = p.rule.softcap > 0.f, bias = p.rule.slopes != nullptr;
  return cap ? (bias ? launch_tc_t<true, true>(mq, mk, mv, p, line, st, s)
                     : launch_tc_t<true, false>(mq, mk, mv, p, line, st, s))
             : (bias ? launch_tc_t<false, true>(mq, mk, mv, p, line, st, s)
                     : launch_tc_t<false, false>(mq, mk, mv, p, line, st, s));
}

}  // namespace decode
}  // namespace fpx
