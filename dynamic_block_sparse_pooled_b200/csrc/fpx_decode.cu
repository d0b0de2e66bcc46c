// fpx_decode.cu -- attention of a batch's last tokens against a paged K / V cache, with prompts
// shared by groups of requests read once per group.
//
// Bound by HBM: each cached K / V row is read once per (request or group) and used for q_len x
// group rows (one request of 131072 tokens, 8 KV heads, bf16: 537 MB in 87 us, 6.1 TB/s).  A worker
// (one warp; for bf16 and more than 16 rows 2, 4 or 8) owns a ring in shared memory that it fills
// itself with TMA, K and V half-stages of 32 keys alternating, so it never waits for another worker;
// the eight warps of a CTA keep up to 192 KB in flight per SM.
// The products run on mma.sync m16n8k16: 16 rows is the least a tensor instruction takes and
// most batches fill only group x q_len of them, so the tensor pipe is far from the limit and a
// 128-row tcgen05 tile would only add latency.
//   bf16 cache  Q, P in bf16, ldmatrix from a 128-byte swizzled tile.  (P takes V's type, as both
//               operands of a product have one: a rounding of 2^-8 a weight, that of the output.  The
//               sum that divides O is of the weights before it, in 32 bits.)
//   e4m3 cache  codes are widened to f16 in registers (exact); Q in f16 after a power-of-two scale
//               per row that puts its largest value in [1, 2) (bf16 values stay exact down to
//               2^-14 of it), P in f16 (2^-11 a weight; those below 2^-25 of the piece's first
//               maximum vanish from O, at most 2^-25 of the row's sum each), the head's scales
//               in 32 bits outside the products.  K^T and V
//               fragments are read by plain 16-byte shared loads: the order of the D dimension
//               (for K) and of the keys in eights is permuted alike on both operands, so that each
//               lane's bytes are contiguous and free of bank conflicts.  Bound by instruction issue
//               (128 conversions, 64 permutes, 64 products per 32 keys): 138 MB in 42 us, 3.3 TB/s;
//               widening by integer operations was 20 % slower, 64 keys a tile the same.
//   fp32 cache  CUDA cores, all 32-bit: a lane per key for the scores, a lane per four
//               dimensions for P V.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math_constants.h>

#include <cfloat>
#include <climits>
#include <cstdint>

#include "fpx_decode.cuh"
#include "fpx_internal.h"
#include "fpx_sm100.cuh"

namespace fpx {
namespace decode {

using sm100::smem_u32;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtas = 148;                     // one CTA per SM
constexpr uint32_t kRingBytes = 24 * 1024;     // per warp
constexpr uint32_t kRing = kWarps * kRingBytes;  // 192 KB
constexpr uint32_t kBarPitch = 16;             // a slot's full barrier, then its empty one
constexpr float kRescaleLog2 = 8.0f;           // the running maximum moves in steps above this

// ---- plan ---------------------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;

__device__ __forceinline__ int2 block_scan(int2 v, int2* warp_sum, int2& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
    if (lane >= o) {
      x.x += a;
      x.y += b;
    }
  }
  __syncthreads();
  if (lane == 31) warp_sum[w] = x;
  __syncthreads();
  if (w == 0) {
    int2 y = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int a = __shfl_up_sync(0xffffffffu, y.x, o), b = __shfl_up_sync(0xffffffffu, y.y, o);
      if (lane >= o) {
        y.x += a;
        y.y += b;
      }
    }
    warp_sum[lane] = y;
  }
  __syncthreads();
  total = warp_sum[31];
  if (w > 0) {
    x.x += warp_sum[w - 1].x;
    x.y += warp_sum[w - 1].y;
  }
  return make_int2(x.x - v.x, x.y - v.y);  // exclusive
}

// (units, segments) before each owner, in place.
__device__ __forceinline__ void scan_line(const Line& l, int hkv, int2* warp_sum) {
  const int per = (l.n + kPlanThreads - 1) / kPlanThreads;
  const int a = min(l.n, static_cast<int>(threadIdx.x) * per), b = min(l.n, a + per);
  int2 sum = make_int2(0, 0);
  for (int i = a; i < b; ++i) {
    const Owner w = load_owner(l.owners + i);
    sum.x += units_of(w, l) * w.nrt * hkv;
    sum.y += w.nrt * hkv;
  }
  int2 total;
  int2 at = block_scan(sum, warp_sum, total);
  for (int i = a; i < b; ++i) {
    const Owner w = load_owner(l.owners + i);
    l.owners[i].line = at.x;
    l.owners[i].seg = at.y;
    at.x += units_of(w, l) * w.nrt * hkv;
    at.y += w.nrt * hkv;
  }
  if (threadIdx.x == 0) {
    Owner end = {0, 0, 0, 0, 0, total.x, total.y, 0};
    l.owners[l.n] = end;
  }
}

// One CTA: the owners of both lines from the lengths and groups.
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(DecodeDesc p, Line own, Line shared,
                                                            int32_t* __restrict__ group_of,
                                                            StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  __shared__ int2 warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int most = p.pages_per_seq << p.log2_page;
  bool good = true;
  for (int g = tid; g < p.num_groups; g += kPlanThreads) {
    const int a = p.group_ptr[g], b = p.group_ptr[g + 1];
    if (a < 0 || b < a || b > p.num_seqs || p.prefix_pages[g] < 0) {
      record_error(st, FPX_ERR_DEVICE_INPUT, 60, g, a);
      good = false;
    }
  }
  good = __syncthreads_and(good);
  for (int s = tid; s < p.num_seqs; s += kPlanThreads) group_of[s] = -1;
  __syncthreads();
  // shared parts: a warp per group
  for (int g = warp; g < p.num_groups; g += kPlanThreads / 32) {
    Owner w = {0, 0, 0, 0, 0, 0, 0, 0};
    if (good) {
      const int a = p.group_ptr[g], b = p.group_ptr[g + 1];
      const int prefix = min(p.prefix_pages[g], p.pages_per_seq) << p.log2_page;
      int first = INT_MAX, last = 0;  // keys that some request of the group can see
      for (int s = a + lane; s < b; s += 32) {
        group_of[s] = g;
        const int ctx = min(max(p.ctx[s], 0), most);
        if (ctx == 0) continue;
        last = max(last, ctx);
        const int lo = p.rule.window > 0 ? max(ctx - p.q_len, 0) - min(p.rule.window - 1, most) : 0;
        first = min(first, max(lo, 0));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
        last = max(last, __shfl_xor_sync(0xffffffffu, last, o));
      }
      // whole pages that some request's context covers: rows behind a context may hold anything
      w.k1 = min(prefix, last & ~(p.page - 1));
      w.k0 = min(first / shared.tile * shared.tile, w.k1);
      w.tok0 = a * p.q_len;
      w.ntok = (b - a) * p.q_len;
      w.row = a;
      w.nrt = shared.tpt ? (w.ntok + 2 * shared.tpt - 1) / (2 * shared.tpt)
                         : (w.ntok * p.group + shared.rt - 1) / shared.rt;
    }
    if (lane == 0) shared.owners[g] = w;
  }
  __syncthreads();
  for (int s = tid; s < p.num_seqs; s += kPlanThreads) {
    int ctx = p.ctx[s];
    if (ctx < 0 || ctx > most) {
      record_error(st, FPX_ERR_DEVICE_INPUT, 61, s, ctx);
      ctx = min(max(ctx, 0), most);
    }
    Owner w = {0, 0, s * p.q_len, p.q_len, s, 0, 0, 0};
    w.nrt = (p.q_len * p.group + own.rt - 1) / own.rt;
    if (good) {
      const int g = group_of[s];
      const int prefix = g >= 0 ? load_owner(shared.owners + g).k1 : 0;  // what the group covers
      const int lo = p.rule.window > 0 ? max(ctx - p.q_len, 0) - min(p.rule.window - 1, most) : 0;
      w.k0 = prefix + (lo > prefix ? (lo - prefix) / 32 * 32 : 0);
      w.k1 = max(ctx, w.k0);
    }
    own.owners[s] = w;
  }
  __syncthreads();
  scan_line(own, p.hkv, warp_sum);
  if (p.num_groups > 0) scan_line(shared, p.hkv, warp_sum);
}

// Few requests and nothing shared: every CTA lays the line out for itself in shared memory instead of
// waiting for a launch that does (one warp; replayed from a graph, 1 / 16 / 64 requests of 500 tokens: 14 /
// 17 / 39 us instead of 16 / 21 / 49).
constexpr int kLocalSeqs = 64;

__device__ __forceinline__ void plan_local(const DecodeDesc& p, Line& l, Owner* owners,
                                           StatusBlock* st) {
  l.owners = owners;
  const int lane = threadIdx.x;
  if (lane < 32) {
    const int most = p.pages_per_seq << p.log2_page;
    const int nrt = (p.q_len * p.group + l.rt - 1) / l.rt;
    int line = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
      const int s = s0 + lane;
      Owner w = {0, 0, s * p.q_len, p.q_len, s, 0, s * nrt * p.hkv, nrt};
      if (s < p.num_seqs) {
        int ctx = p.ctx[s];
        if (ctx < 0 || ctx > most) {
          record_error(st, FPX_ERR_DEVICE_INPUT, 61, s, ctx);
          ctx = min(max(ctx, 0), most);
        }
        const int lo = p.rule.window > 0 ? max(ctx - p.q_len, 0) - min(p.rule.window - 1, most) : 0;
        w.k0 = lo > 0 ? lo / 32 * 32 : 0;
        w.k1 = max(ctx, w.k0);
      }
      const int mine = units_of(w, l) * nrt * p.hkv;
      int x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      w.line = line + x - mine;
      if (s < p.num_seqs) owners[s] = w;
      line += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      Owner end = {0, 0, 0, 0, 0, line, p.num_seqs * nrt * p.hkv, 0};
      owners[p.num_seqs] = end;
    }
  }
  __syncthreads();
}

// ---- the ring -----------------------------------------------------------------------------------

// Layout of a half-stage: kTile keys x D elements as boxes of kRowB bytes per key.
template <int kEs, int D, int kTileKeys>
struct Half {
  static constexpr int kRowB = D * kEs < 128 ? D * kEs : 128;
  static constexpr int kBoxes = D * kEs / kRowB;
  static constexpr uint32_t kBoxBytes = kTileKeys * kRowB;
  static constexpr uint32_t kBytes = kBoxes * kBoxBytes;
  static constexpr int kSlots1 = kRingBytes / kBytes;  // slots of one warp's ring
};

// The loads of one worker: half-stages K, V, K, V, ... of its tiles, in order, into its ring.
template <int kEs, int D, int kTileKeys>
struct Loader {
  using H = Half<kEs, D, kTileKeys>;
  Walk c;
  int t;      // next tile of the piece
  bool more;  // there is one
  int row[2];  // first cache row of the next tile's one or two page pieces; -1: not loaded
  uint32_t slot, slots, ring, full;

  __device__ __forceinline__ void lookup(const DecodeDesc& p, StatusBlock* st) {
    const int kb = c.w.k0 + t * kTileKeys;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      row[i] = -1;
      const int key = kb + i * p.page;  // i = 1 only for pages smaller than the tile
      if (i == 1 && p.page >= kTileKeys) continue;
      if (key >= c.w.k1) continue;
      const int pg = p.table[static_cast<int64_t>(c.w.row) * p.pages_per_seq + (key >> p.log2_page)];
      if (pg < 0 || pg >= p.num_pages) {
        record_error(st, FPX_ERR_DEVICE_INPUT, 62, c.w.row, key >> p.log2_page);
        row[i] = p.num_pages << p.log2_page;  // past the cache: TMA fills zeros
      } else {
        row[i] = (pg << p.log2_page) + (key & (p.page - 1));
      }
    }
  }
  __device__ __forceinline__ void start(const DecodeDesc& p, const Line& l, int x0, int x1,
                                        StatusBlock* st) {
    slot = 0;
    c.enter(l, x0, x1);
    more = c.next(p.hkv);
    t = c.t0;
    if (more) lookup(p, st);
  }
  // Requests the next half-stage (K first, then V of the same tile); the whole warp calls it.
  __device__ __forceinline__ void request(const DecodeDesc& p, const CUtensorMap* map, bool is_v,
                                          StatusBlock* st) {
    const int rows = p.page < kTileKeys ? p.page : kTileKeys;
    if (sm100::elect_one()) {
      const uint32_t dst = ring + slot * H::kBytes, bar = full + slot * kBarPitch;
      const int pieces = row[1] >= 0 ? 2 : 1;
      sm100::mbar_arrive_expect_tx(bar, pieces * rows * H::kRowB * H::kBoxes);
      const int kvh = c.j / c.w.nrt;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row[i] < 0) continue;
#pragma unroll
        for (int b = 0; b < H::kBoxes; ++b)
          sm100::tma_load_3d(dst + b * H::kBoxBytes + i * rows * H::kRowB, map, bar,
                             b * (H::kRowB / kEs), kvh, row[i]);
      }
    }
    __syncwarp();
    if (++slot == slots) slot = 0;
    if (!is_v) return;
    if (++t == c.t0 + c.cnt) {
      more = c.next(p.hkv);
      t = c.t0;
    }
    if (more) lookup(p, st);
  }
};

// ---- tensor-core helpers --------------------------------------------------------------------------

template <bool kF16>
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
        " {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void sts128_zero(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0) : "memory");
}
// Four e4m3 codes to two f16x2 (codes 0, 1 and codes 2, 3); exact.
__device__ __forceinline__ void f16x2_of_e4m3(uint32_t x, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Swizzled byte offset of 16-byte chunk `ch` of key `key` inside a box of kRowB-byte rows (TMA's
// 128-byte swizzle XORs the chunk with address bits 7-9, the 64-byte one with bits 7-8).
template <int kRowB>
__device__ __forceinline__ uint32_t swz(int key, int ch) {
  return kRowB == 128 ? key * 128 + ((ch ^ (key & 7)) << 4)
                      : key * 64 + ((ch ^ ((key >> 1) & 3)) << 4);
}

// Place in a group of eight keys that column n of an S tile holds (e4m3; bf16 keeps the order).
// Even columns 2c hold key 2c, odd columns 2c + 1 key 2c + 5 (mod 8): neighbouring lanes' 16-byte
// reads then fall into different banks for K (columns n, n + 1) as for V (columns 2c, c = 0..3).
__device__ __forceinline__ int key_of_col(int n) { return (n & 1) ? ((n + 4) & 7) : n; }

// ---- tensor-core kernel ----------------------------------------------------------------------------

constexpr int kTile = 32;  // keys

template <bool kFp8, int D, int RW>
__global__ void __launch_bounds__(kThreads, 1)
decode_mma_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ DecodeDesc p, const __grid_constant__ Line line_,
                  const __nv_bfloat16* __restrict__ q, StatusBlock* st) {
  using H = Half<kFp8 ? 1 : 2, D, kTile>;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int kGroups = kWarps / RW;
  constexpr int kSlots = H::kSlots1 * RW;
  // half-stages between the one consumed and the one whose slot is refilled: a worker of several
  // warps refills one behind, so that its first warp rarely waits for the others
  constexpr int kLag = RW == 1 ? 0 : 2;
  constexpr int kSteps = D / 16;  // k-steps of Q K^T, and pairs of n-tiles of P V
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bars = base + kRing;
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int grp = warp / RW, wr = warp % RW;
  const int g4 = lane >> 2, c4 = lane & 3;
  if (tid == 0) abort_flag_s = 0;
  if (tid < kGroups * kSlots) {
    sm100::mbar_init(bars + tid * kBarPitch, 1);       // full
    sm100::mbar_init(bars + tid * kBarPitch + 8, RW);  // empty
    sm100::fence_mbar_init();
  }
  static_assert(kGroups * kSlots <= kThreads, "one thread per slot");
  __syncthreads();
  pdl_enter();  // after the previous kernel on the stream, which the set-up above overlaps
  __shared__ Owner local[kLocalSeqs + 1];
  Line line = line_;
  if (!line.owners) plan_local(p, line, local, st);
  const int worker = blockIdx.x * kGroups + grp;
  const int64_t total = line.owners[line.n].line;
  const int64_t nw = active_workers(line, total);
  if (worker >= nw) return;  // no later CTA-wide barrier
  const int x0 = static_cast<int>(line_begin(worker, total, nw));
  const int x1 = static_cast<int>(line_begin(worker + 1, total, nw));
  const uint32_t ring = base + grp * RW * kRingBytes;
  const uint32_t full0 = bars + grp * kSlots * kBarPitch;

  Loader<kFp8 ? 1 : 2, D, kTile> load;
  int requested = 0;  // half-stages (first warp of the worker)
  auto request = [&]() {
    load.request(p, (requested & 1) ? &tmV : &tmK, requested & 1, st);
    ++requested;
  };
  if (wr == 0) {
    load.ring = ring;
    load.full = full0;
    load.slots = kSlots;
    load.start(p, line, x0, x1, st);
    while ((load.more || (requested & 1)) && requested < kSlots - kLag) request();
  }
  bool ok = true;
  int e = 0;            // half-stages consumed
  uint32_t slot = 0, phase = 0;
  auto wait_full = [&]() {
    ok = __all_sync(kFull, sm100::mbar_wait(full0 + slot * kBarPitch, phase, abort_flag));
    return ok;
  };
  // This warp is done with the current half-stage: hand its slot back and refill.
  auto release = [&]() -> bool {
    __syncwarp();
    if (RW > 1 && lane == 0) sm100::mbar_arrive(full0 + slot * kBarPitch + 8);
    ++e;
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
    if (wr == 0 && (load.more || (requested & 1)) && requested < e + kSlots - kLag) {
      if (RW > 1 && requested >= kSlots) {
        const int f = requested - kSlots;  // the half-stage that used the slot before
        ok = __all_sync(kFull, sm100::mbar_wait(full0 + (f % kSlots) * kBarPitch + 8, (f / kSlots) & 1,
                                                abort_flag));
        if (!ok) return false;
      }
      request();
    }
    return true;
  };

  const bool capped = p.rule.softcap > 0.f, biased = p.rule.slopes != nullptr;
  // The rows of a piece that this thread has, g4 and g4 + 8 of its warp's sixteen.  They are looked
  // up one piece ahead, so that the loads they depend on are hidden behind the tiles before.
  struct Rows {
    int kvh, tok[2], head[2], pos[2];
    KeySpan span[2];
    bool valid[2], active;
  };
  auto rows_of = [&](const Walk& c) {
    Rows R;
    R.kvh = c.j / c.w.nrt;
    const int nrows = c.w.ntok * p.group;
    const int r0 = (c.j - R.kvh * c.w.nrt) * line.rt + wr * 16;
    R.active = r0 < nrows;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + g4 + 8 * h;
      R.valid[h] = r < nrows;
      const int rr = R.valid[h] ? r : 0;
      R.tok[h] = c.w.tok0 + rr / p.group;
      R.head[h] = R.kvh * p.group + rr % p.group;
      const RowPos rp = row_pos(p, R.tok[h]);
      R.pos[h] = rp.i;
      R.span[h] = rp.span;
      R.span[h].hi = min(R.span[h].hi, c.w.k1 - 1);  // the range may end inside a tile
      if (!R.valid[h]) R.span[h] = {0, INT_MAX};     // discarded: no reason to mask
    }
    return R;
  };
  uint32_t qf[kSteps][4];
  ScoreMap map[2];
  float mul[2];
  auto load_q = [&](const Rows& R) {
    float kscale = p.scale;
    if (kFp8) kscale *= p.k_scale[R.kvh];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat16* qrow = q + (static_cast<int64_t>(R.tok[h]) * p.hq + R.head[h]) * D;
      float row_scale = 1.f;
      if (kFp8) {
        float v[D / 4];
        float top = 0.f;
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {  // 4 elements at (b / 4) * 64 + c4 * 16 + (b % 4) * 4
          const uint2 u = R.valid[h] ? *reinterpret_cast<const uint2*>(
                                           qrow + (b / 4) * 64 + c4 * 16 + (b % 4) * 4)
                                     : make_uint2(0, 0);
          v[4 * b] = __uint_as_float(u.x << 16);
          v[4 * b + 1] = __uint_as_float(u.x & 0xffff0000u);
          v[4 * b + 2] = __uint_as_float(u.y << 16);
          v[4 * b + 3] = __uint_as_float(u.y & 0xffff0000u);
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, fabsf(v[4 * b + i]));
        }
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // 2^-e with e the exponent of the largest value, kept inside the normal range
        int ex = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        ex = top > 0.f && top < CUDART_INF_F ? min(max(ex, -126), 126) : 0;
        const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
        row_scale = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
#pragma unroll
        for (int b = 0; b < D / 16; ++b) {
          qf[b][h] = pack_f16x2(v[4 * b] * down, v[4 * b + 1] * down);
          qf[b][h + 2] = pack_f16x2(v[4 * b + 2] * down, v[4 * b + 3] * down);
        }
      } else {
#pragma unroll
        for (int b = 0; b < kSteps; ++b) {
          qf[b][h] = R.valid[h] ? *reinterpret_cast<const uint32_t*>(qrow + b * 16 + c4 * 2) : 0u;
          qf[b][h + 2] =
              R.valid[h] ? *reinterpret_cast<const uint32_t*>(qrow + b * 16 + c4 * 2 + 8) : 0u;
        }
      }
      map[h] = score_map(p.rule, kscale * row_scale, R.head[h]);
      // without cap and bias the scale stays in the exponent (kept above 0: -inf * 0 is NaN)
      mul[h] = capped || biased ? 1.f : fmaxf(map[h].k, FLT_MIN);
    }
  };
  Walk cur;
  cur.enter(line, x0, x1);
  bool have = cur.next(p.hkv);
  Rows R = {};
  if (have) {
    R = rows_of(cur);
    load_q(R);
  }
  while (have) {
    const int k0 = cur.w.k0, k1 = cur.w.k1, t0 = cur.t0, cnt = cur.cnt;
    const int64_t slot_id = static_cast<int64_t>(cur.w.seg) + cur.j + worker;
    have = cur.next(p.hkv);
    Rows next = {};
    if (have) next = rows_of(cur);
    float acc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
    float m[2] = {-CUDART_INF_F, -CUDART_INF_F}, l[2] = {0.f, 0.f};

    for (int t = 0; t < cnt; ++t) {
      const int kb = k0 + (t0 + t) * kTile;
      // ---- S = Q K^T
      if (!wait_full()) break;
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) s[i][k] = 0.f;
      const uint32_t kt = ring + slot * H::kBytes;
      if (R.active) {
        if (kFp8) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) {
            const int key = nt * 8 + key_of_col(g4);
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf) {
              // 16 codes of this lane's key: k-steps 4 hf .. 4 hf + 3
              const uint4 u = lds128(kt + swz<H::kRowB>(key, hf * 4 + c4));
              const uint32_t w4[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                f16x2_of_e4m3(w4[i], b0, b1);
                mma16816<true>(s[nt], qf[hf * 4 + i], b0, b1);
              }
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < kSteps; ++ks) {
#pragma unroll
            for (int np = 0; np < 2; ++np) {
              // matrices: keys 16 np .. +7 / +8 .. +15, dimensions 16 ks .. +7 / +8 .. +15
              const int key = np * 16 + (lane >> 4) * 8 + (lane & 7);
              const int ch = ks * 2 + ((lane >> 3) & 1);
              uint32_t b[4];
              ldsm4(b, kt + (ch >> 3) * H::kBoxBytes + swz<128>(key, ch & 7));
              mma16816<false>(s[2 * np], qf[ks], b[0], b[1]);
              mma16816<false>(s[2 * np + 1], qf[ks], b[2], b[3]);
            }
          }
        }
      }
      if (!release()) break;
      // ---- softmax
      uint32_t pf[2][4];  // P as A fragments of the two 16-key steps
      if (R.active) {
        const bool partial = __any_sync(kFull, R.span[0].lo > kb || R.span[0].hi < kb + kTile - 1 ||
                                                   R.span[1].lo > kb || R.span[1].hi < kb + kTile - 1);
        if (capped) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              s[nt][k] = map[k >> 1].cap2 * tanh_any(s[nt][k] * map[k >> 1].k);
        }
        if (biased) {
          const float rel[2] = {static_cast<float>(R.pos[0] - kb - (kFp8 ? 0 : c4 * 2)),
                                static_cast<float>(R.pos[1] - kb - (kFp8 ? 0 : c4 * 2))};
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float col = kFp8 ? static_cast<float>(nt * 8 + key_of_col(c4 * 2 + (k & 1)))
                                     : static_cast<float>(nt * 8 + (k & 1));
              s[nt][k] = fmaf(-map[k >> 1].slope2, fabsf(rel[k >> 1] - col),
                              capped ? s[nt][k] : s[nt][k] * map[k >> 1].k);
            }
        }
        if (partial) {
#pragma unroll
          for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int col = c4 * 2 + (k & 1);
              const int key = kb + nt * 8 + (kFp8 ? key_of_col(col) : col);
              if (key < R.span[k >> 1].lo || key > R.span[k >> 1].hi) s[nt][k] = -CUDART_INF_F;
            }
        }
        float corr[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int nt = 0; nt < 4; ++nt) mx = fmaxf(mx, fmaxf(s[nt][2 * h], s[nt][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2)) * mul[h];
          corr[h] = 1.f;
          if (mx > m[h] + kRescaleLog2) {
            corr[h] = ex2_approx(m[h] - mx);  // 0 for the first keys
            m[h] = mx;
            l[h] *= corr[h];
          }
        }
        if (__any_sync(kFull, corr[0] != 1.f || corr[1] != 1.f)) {
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][0] *= corr[0];
            acc[i][1] *= corr[0];
            acc[i][2] *= corr[1];
            acc[i][3] *= corr[1];
          }
        }
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float ref = m[h] == -CUDART_INF_F ? 0.f : -m[h];
            const float p0 = ex2_approx(fmaf(s[nt][2 * h], mul[h], ref));
            const float p1 = ex2_approx(fmaf(s[nt][2 * h + 1], mul[h], ref));
            l[h] += p0 + p1;
            pf[nt >> 1][h + 2 * (nt & 1)] = kFp8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
          }
        }
      }
      // ---- O += P V
      if (!wait_full()) break;
      const uint32_t vt = ring + slot * H::kBytes;
      if (R.active) {
        const int keys = k1 - kb;
        if (keys < kTile) {
          // rows past the last key may hold anything (NaN too): zero them, every warp for itself
          // (all write the same zeros), ordered before the slot's next TMA write
          constexpr int kChunks = H::kRowB / 16;
          for (int i = lane; i < (kTile - keys) * kChunks * H::kBoxes; i += 32) {
            const int ch = i % kChunks, rest = i / kChunks;
            const int b = rest % H::kBoxes, key = keys + rest / H::kBoxes;
            sts128_zero(vt + b * H::kBoxBytes + key * H::kRowB + ch * 16);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
        }
        if (kFp8) {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            // lane (n = g4, c4): the codes V[key][n * D / 8 ..] of the keys of columns 2 c4,
            // 2 c4 + 1 of the step's two S tiles; code i goes to n-tile i
            uint32_t u[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = ks * 16 + (k >> 1) * 8 + key_of_col(c4 * 2 + (k & 1));
              if (D == 128) {
                const uint4 x = lds128(vt + swz<H::kRowB>(key, g4));
                u[k][0] = x.x;
                u[k][1] = x.y;
                u[k][D / 32 - 2] = x.z;
                u[k][D / 32 - 1] = x.w;
              } else {
                const uint2 x = lds64(vt + swz<H::kRowB>(key, g4 >> 1) + (g4 & 1) * 8);
                u[k][0] = x.x;
                u[k][1] = x.y;
              }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t f[4][2];  // f16x2 of codes 4 i, + 1 and 4 i + 2, + 3 of the four keys
#pragma unroll
              for (int k = 0; k < 4; ++k) f16x2_of_e4m3(u[k][i], f[k][0], f[k][1]);
#pragma unroll
              for (int hw = 0; hw < 2; ++hw) {
                const int nt = 4 * i + 2 * hw;
                mma16816<true>(acc[nt], pf[ks], __byte_perm(f[0][hw], f[1][hw], 0x5410),
                               __byte_perm(f[2][hw], f[3][hw], 0x5410));
                mma16816<true>(acc[nt + 1], pf[ks], __byte_perm(f[0][hw], f[1][hw], 0x7632),
                               __byte_perm(f[2][hw], f[3][hw], 0x7632));
              }
            }
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int np = 0; np < kSteps; ++np) {
              // matrices: keys 16 ks .. +7 / +8 .. +15, dimensions 16 np .. +7 / +8 .. +15
              const int key = ks * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
              const int ch = np * 2 + (lane >> 4);
              uint32_t b[4];
              ldsm4t(b, vt + (ch >> 3) * H::kBoxBytes + swz<128>(key, ch & 7));
              mma16816<false>(acc[2 * np], pf[ks], b[0], b[1]);
              mma16816<false>(acc[2 * np + 1], pf[ks], b[2], b[3]);
            }
          }
        }
      }
      if (!release()) break;
    }
    if (!ok) break;
    // ---- the piece's partial
    if (R.active) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = l[h];
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        if (!R.valid[h]) continue;
        const int64_t at = slot_id * line.rps + wr * 16 + g4 + 8 * h;
        if (c4 == 0) line.part_ml[at] = make_float2(m[h], sum);
        float* dst = line.part_o + at * D;
        if (kFp8) {
          // columns 2 c4 and 2 c4 + 1 of n-tile i: dimensions (2 c4) D / 8 + i, (2 c4 + 1) D / 8 + i
#pragma unroll
          for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int i = 0; i < D / 8; i += 4)
              *reinterpret_cast<float4*>(dst + (2 * c4 + half) * (D / 8) + i) =
                  make_float4(acc[i][2 * h + half], acc[i + 1][2 * h + half],
                              acc[i + 2][2 * h + half], acc[i + 3][2 * h + half]);
        } else {
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            *reinterpret_cast<float2*>(dst + i * 8 + c4 * 2) =
                make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
        }
      }
    }
    R = next;
    if (have) load_q(R);
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) record_error(st, FPX_ERR_TIMEOUT, 63, worker, e);
    // every load in flight lands before the CTA's shared memory is given up
    if (wr == 0) {
      volatile int never = 0;
      for (int f = max(0, requested - kSlots); f < requested; ++f)
        sm100::mbar_wait(full0 + (f % kSlots) * kBarPitch, (f / kSlots) & 1, &never);
    }
  }
}

// ---- fp32 kernel ------------------------------------------------------------------------------------

constexpr int kTileF32 = 16;  // keys
constexpr int kRowsF32 = 8;   // query rows of a worker (one warp)
constexpr int kWarpsF32 = 7;  // an eighth ring would not leave room for the Q rows and weights

template <int D>
__global__ void __launch_bounds__(kWarpsF32 * 32, 1)
decode_f32_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                  const __grid_constant__ DecodeDesc p, const __grid_constant__ Line line_,
                  const float* __restrict__ q, StatusBlock* st) {
  using H = Half<4, D, kTileF32>;
  constexpr unsigned kFull = 0xffffffffu;
  constexpr int kSlots = H::kSlots1;
  constexpr int kHalfD = D / 2;          // dimensions of a lane's part of a dot product
  constexpr int kQPitch = kHalfD + 4;    // the two halves of a Q row fall into different banks
  constexpr int kVd = D / 32;            // dimensions of a lane's part of O
  extern __shared__ uint8_t smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - smem_u32(smem_raw));
  const uint32_t bars = base + kWarpsF32 * kRingBytes;
  __shared__ int abort_flag_s;
  volatile int* abort_flag = &abort_flag_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) abort_flag_s = 0;
  if (tid < kWarpsF32 * kSlots) {
    sm100::mbar_init(bars + tid * kBarPitch, 1);
    sm100::fence_mbar_init();
  }
  __syncthreads();
  pdl_enter();  // after the previous kernel on the stream, which the set-up above overlaps
  __shared__ Owner local[kLocalSeqs + 1];
  Line line = line_;
  if (!line.owners) plan_local(p, line, local, st);
  // Q rows [kRowsF32][2][kQPitch] and weights [kTileF32][kRowsF32] of this warp
  float* sq = reinterpret_cast<float*>(gbase + kWarpsF32 * kRingBytes + 1024) +
              warp * (kRowsF32 * 2 * kQPitch + kTileF32 * kRowsF32);
  float* sp = sq + kRowsF32 * 2 * kQPitch;
  const int worker = blockIdx.x * kWarpsF32 + warp;
  const int64_t total = line.owners[line.n].line;
  const int64_t nw = active_workers(line, total);
  if (worker >= nw) return;  // no later CTA-wide barrier
  const int x0 = static_cast<int>(line_begin(worker, total, nw));
  const int x1 = static_cast<int>(line_begin(worker + 1, total, nw));
  const uint32_t full0 = bars + warp * kSlots * kBarPitch;
  Loader<4, D, kTileF32> load;
  load.ring = base + warp * kRingBytes;
  load.full = full0;
  load.slots = kSlots;
  int requested = 0;
  auto request = [&]() {
    load.request(p, (requested & 1) ? &tmV : &tmK, requested & 1, st);
    ++requested;
  };
  load.start(p, line, x0, x1, st);
  while ((load.more || (requested & 1)) && requested < kSlots) request();
  bool ok = true;
  uint32_t slot = 0, phase = 0;
  int e = 0;
  auto wait_full = [&]() {
    ok = __all_sync(kFull, sm100::mbar_wait(full0 + slot * kBarPitch, phase, abort_flag));
    return ok;
  };
  auto release = [&]() {
    __syncwarp();
    ++e;
    if (++slot == kSlots) {
      slot = 0;
      phase ^= 1;
    }
    if (load.more || (requested & 1)) request();
  };
  const int kl = lane & 15, dh = lane >> 4;  // key and half of D in the dot products

  Walk cur;
  cur.enter(line, x0, x1);
  while (cur.next(p.hkv)) {
    const Owner w = cur.w;
    const int j = cur.j, t0 = cur.t0, cnt = cur.cnt;
    const int kvh = j / w.nrt, rt = j - kvh * w.nrt;
    const int nrows = w.ntok * p.group;
    const int r0 = rt * kRowsF32;
    const int rows = min(kRowsF32, nrows - r0);
    __syncwarp();
    for (int i = lane; i < kRowsF32 * D; i += 32) {
      const int r = i / D, dd = i % D;
      float x = 0.f;
      if (r < rows) {
        const int tok = w.tok0 + (r0 + r) / p.group, head = kvh * p.group + (r0 + r) % p.group;
        x = q[(static_cast<int64_t>(tok) * p.hq + head) * D + dd];
      }
      sq[(r * 2 + dd / kHalfD) * kQPitch + dd % kHalfD] = x;
    }
    // lane r keeps row r's position, span and score map; the loop below broadcasts them
    int my_pos = 0, my_lo = 0, my_hi = -1;
    ScoreMap my_map = score_map(p.rule, p.scale, kvh * p.group);
    if (lane < rows) {
      const int tok = w.tok0 + (r0 + lane) / p.group;
      const RowPos rp = row_pos(p, tok);
      my_pos = rp.i;
      my_lo = rp.span.lo;
      my_hi = min(rp.span.hi, w.k1 - 1);  // the range may end inside a tile
      my_map = score_map(p.rule, p.scale, kvh * p.group + (r0 + lane) % p.group);
    }
    __syncwarp();
    float acc[kRowsF32][kVd];
    float m[kRowsF32], l[kRowsF32];
#pragma unroll
    for (int r = 0; r < kRowsF32; ++r) {
      m[r] = -CUDART_INF_F;
      l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < kVd; ++i) acc[r][i] = 0.f;
    }
    for (int t = 0; t < cnt; ++t) {
      const int kb = w.k0 + (t0 + t) * kTileF32;
      if (!wait_full()) break;
      const uint32_t kt = load.ring + slot * H::kBytes;
      float s[kRowsF32];
#pragma unroll
      for (int r = 0; r < kRowsF32; ++r) s[r] = 0.f;
#pragma unroll 4
      for (int c = 0; c < kHalfD / 4; ++c) {
        const int ch = dh * (kHalfD / 4) + c;
        const uint4 u = lds128(kt + (ch >> 3) * H::kBoxBytes + swz<128>(kl, ch & 7));
        const float k0 = __uint_as_float(u.x), k1 = __uint_as_float(u.y);
        const float k2 = __uint_as_float(u.z), k3 = __uint_as_float(u.w);
#pragma unroll
        for (int r = 0; r < kRowsF32; ++r) {
          const float4 x = *reinterpret_cast<const float4*>(sq + (r * 2 + dh) * kQPitch + c * 4);
          s[r] = fmaf(x.x, k0, fmaf(x.y, k1, fmaf(x.z, k2, fmaf(x.w, k3, s[r]))));
        }
      }
      release();
      const int key = kb + kl;
#pragma unroll
      for (int r = 0; r < kRowsF32; ++r) {
        const float dot = s[r] + __shfl_xor_sync(kFull, s[r], 16);
        ScoreMap map;
        map.k = my_map.k;  // the same for every row
        map.cap2 = my_map.cap2;
        map.slope2 = __shfl_sync(kFull, my_map.slope2, r);
        const int pos = __shfl_sync(kFull, my_pos, r);
        const int lo = __shfl_sync(kFull, my_lo, r), hi = __shfl_sync(kFull, my_hi, r);
        float y = map(dot, fabsf(static_cast<float>(pos - key)));
        if (key < lo || key > hi) y = -CUDART_INF_F;
        float mx = y;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
        float corr = 1.f;
        if (mx > m[r]) {
          corr = ex2_approx(m[r] - mx);
          m[r] = mx;
        }
        const float pr = m[r] == -CUDART_INF_F ? 0.f : ex2_approx(y - m[r]);
        l[r] = l[r] * corr + pr;  // this lane's key column (both halves of the warp hold it)
#pragma unroll
        for (int i = 0; i < kVd; ++i) acc[r][i] *= corr;
        if (dh == 0) sp[kl * kRowsF32 + r] = pr;
      }
      __syncwarp();
      if (!wait_full()) break;
      const uint32_t vt = load.ring + slot * H::kBytes;
      const int have = min(kTileF32, w.k1 - kb);  // rows past the last key may hold anything
      for (int kk = 0; kk < have; ++kk) {
        float v[kVd];
        if (D == 128) {
          const uint4 u = lds128(vt + (lane >> 3) * H::kBoxBytes + swz<128>(kk, lane & 7));
          v[0] = __uint_as_float(u.x);
          v[1] = __uint_as_float(u.y);
          v[kVd - 2] = __uint_as_float(u.z);
          v[kVd - 1] = __uint_as_float(u.w);
        } else {
          const uint2 u = lds64(vt + (lane >> 4) * H::kBoxBytes + swz<128>(kk, (lane >> 1) & 7) +
                                (lane & 1) * 8);
          v[0] = __uint_as_float(u.x);
          v[1] = __uint_as_float(u.y);
        }
        const float4 pa = *reinterpret_cast<const float4*>(sp + kk * kRowsF32);
        const float4 pb = *reinterpret_cast<const float4*>(sp + kk * kRowsF32 + 4);
        const float pr[8] = {pa.x, pa.y, pa.z, pa.w, pb.x, pb.y, pb.z, pb.w};
#pragma unroll
        for (int r = 0; r < kRowsF32; ++r)
#pragma unroll
          for (int i = 0; i < kVd; ++i) acc[r][i] = fmaf(pr[r], v[i], acc[r][i]);
      }
      release();
    }
    if (!ok) break;
    const int64_t slot_id = w.seg + j + worker;
#pragma unroll
    for (int r = 0; r < kRowsF32; ++r) {
      float sum = l[r];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (r >= rows) continue;
      const int64_t at = slot_id * line.rps + r;
      if (lane == 0) line.part_ml[at] = make_float2(m[r], sum);
#pragma unroll
      for (int i = 0; i < kVd; ++i) line.part_o[at * D + lane * kVd + i] = acc[r][i];
    }
  }
  if (!ok) {
    *abort_flag = 1;
    if (lane == 0) record_error(st, FPX_ERR_TIMEOUT, 64, worker, e);
    volatile int never = 0;
    for (int f = max(0, requested - kSlots); f < requested; ++f)
      sm100::mbar_wait(full0 + (f % kSlots) * kBarPitch, (f / kSlots) & 1, &never);
  }
}

// ---- join -----------------------------------------------------------------------------------------

// The partials of one row on a line: `count` of them, i at slot first + i / per, row in + i % per *
// 128 of the slot.
struct Pieces {
  int64_t first;
  int count, per, in;
};
__device__ __forceinline__ Pieces pieces_of(const Line& l, int owner, int kvh, int tok, int hg,
                                            int group) {
  Pieces r = {0, 0, 1, 0};
  if (owner < 0) return r;
  const Owner w = load_owner(l.owners + owner);
  const int n = tiles_of(w, l.tile);
  if (n == 0) return r;
  const int64_t total = l.owners[l.n].line;
  tok -= w.tok0;
  int rt;
  if (l.tpt) {
    const int tile = tok / l.tpt;
    rt = tile >> 1;
    r.per = w.ntok - rt * 2 * l.tpt > l.tpt ? 1 : 2;
    r.in = (tile & 1) * 128 + (tok - tile * l.tpt) * group + hg;
  } else {
    const int row = tok * group + hg;
    rt = row / l.rt;
    r.in = row - rt * l.rt;
  }
  const int j = kvh * w.nrt + rt;
  const int64_t x = w.line + static_cast<int64_t>(j) * (n + l.pad) + l.pad;
  const int64_t nw = active_workers(l, total);
  const int w0 = worker_of(x, total, nw), w1 = worker_of(x + n - 1, total, nw);
  r.first = w.seg + j + w0;
  r.count = (w1 - w0 + 1) * r.per;
  return r;
}

// kWpr warps per row (token, head): each joins every kWpr-th partial, then the warps are joined.
// Several warps per row shorten the chain of loads when there are few rows and many partials.
template <typename OT, int D, int kWpr>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ DecodeDesc p,
                                                   const __grid_constant__ Line own_,
                                                   const __grid_constant__ Line shared,
                                                   const int32_t* __restrict__ group_of,
                                                   OT* __restrict__ o, float* __restrict__ lse,
                                                   StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  __shared__ Owner local[kLocalSeqs + 1];
  Line own = own_;
  if (!own.owners) plan_local(p, own, local, st);
  constexpr int kVd = D / 32;
  __shared__ float sm[8], sl[8], so[8][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / kWpr) + warp / kWpr;
  const int sub = warp % kWpr;
  const bool valid = row < static_cast<int64_t>(p.tokens) * p.hq;
  float m = -CUDART_INF_F, l = 0.f, acc[kVd];
#pragma unroll
  for (int i = 0; i < kVd; ++i) acc[i] = 0.f;
  const int tok = valid ? static_cast<int>(row / p.hq) : 0;
  const int h = valid ? static_cast<int>(row - static_cast<int64_t>(tok) * p.hq) : 0;
  if (valid) {
    const int kvh = h / p.group, hg = h - kvh * p.group;
    const int s = tok / p.q_len;
    Pieces pc[2];
    const int g = p.num_groups > 0 ? group_of[s] : -1;
    pc[0] = pieces_of(shared, g, kvh, tok, hg, p.group);
    pc[1] = pieces_of(own, s, kvh, tok, hg, p.group);
    // 32 partials at a time: a lane reads the statistics of one each, the weights follow from their
    // maximum, and then the loads of O depend on nothing but their index
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const Line& ln = k == 0 ? shared : own;
      for (int i0 = sub; i0 < pc[k].count; i0 += 32 * kWpr) {
        const int mine = i0 + lane * kWpr;
        int64_t at = 0;
        float2 ml = make_float2(-CUDART_INF_F, 0.f);
        if (mine < pc[k].count) {
          at = pc[k].per == 2 ? (pc[k].first + (mine >> 1)) * ln.rps + pc[k].in + (mine & 1) * 128
                              : (pc[k].first + mine) * ln.rps + pc[k].in;
          ml = ln.part_ml[at];
        }
        float mn = ml.x;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
        mn = fmaxf(mn, m);
        if (mn == -CUDART_INF_F) continue;  // no key seen so far
        const float w = ex2_approx(ml.x - mn), a = ex2_approx(m - mn);
        float sum = w * ml.y;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
        l = l * a + sum;
        m = mn;
#pragma unroll
        for (int c = 0; c < kVd; ++c) acc[c] *= a;
        const int cnt = min(32, (pc[k].count - i0 + kWpr - 1) / kWpr);
#pragma unroll 8
        for (int i = 0; i < cnt; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
          const float* src = ln.part_o + __shfl_sync(0xffffffffu, at, i) * D + lane * kVd;
          float x[kVd];
          if (kVd == 4) {
            const float4 u = *reinterpret_cast<const float4*>(src);
            x[0] = u.x;
            x[1] = u.y;
            x[kVd - 2] = u.z;
            x[kVd - 1] = u.w;
          } else {
            const float2 u = *reinterpret_cast<const float2*>(src);
            x[0] = u.x;
            x[1] = u.y;
          }
          // a partial that saw no key may hold anything in O
#pragma unroll
          for (int c = 0; c < kVd; ++c) acc[c] += wi == 0.f ? 0.f : x[c] * wi;
        }
      }
    }
  }
  if (kWpr > 1) {
    if (lane == 0) {
      sm[warp] = m;
      sl[warp] = l;
    }
#pragma unroll
    for (int i = 0; i < kVd; ++i) so[warp][lane * kVd + i] = acc[i];
    __syncthreads();
    if (sub != 0) return;
#pragma unroll
    for (int k = 1; k < kWpr; ++k) {
      const float m2 = sm[warp + k], mn = fmaxf(m, m2);
      if (mn == -CUDART_INF_F) continue;
      const float a = ex2_approx(m - mn), b = ex2_approx(m2 - mn);
      l = l * a + sl[warp + k] * b;
#pragma unroll
      for (int i = 0; i < kVd; ++i) acc[i] = acc[i] * a + so[warp + k][lane * kVd + i] * b;
      m = mn;
    }
  }
  if (!valid) return;
  const bool none = m == -CUDART_INF_F;
  float inv = none ? 0.f : 1.f / l;
  if (p.v_scale) inv *= p.v_scale[h / p.group];
  OT* dst = o + row * D + lane * kVd;
#pragma unroll
  for (int i = 0; i < kVd; ++i) {
    const float x = none ? 0.f : acc[i] * inv;
    if (sizeof(OT) == 4) *reinterpret_cast<float*>(dst + i) = x;
    else *reinterpret_cast<__nv_bfloat16*>(dst + i) = __float2bfloat16_rn(x);
  }
  if (lse && lane == 0)
    lse[static_cast<int64_t>(h) * p.tokens + tok] =
        none ? -CUDART_INF_F : (m + __log2f(l)) * 0.6931471805599453f;
}

// ---- host side --------------------------------------------------------------------------------------

// Warps of a worker.  bf16: enough 16-row tiles for the rows that share keys, so that these are read
// from one copy in shared memory; up to a whole CTA (8 requests at 8192 tokens, 32 / 64 / 128 / 256
// rows per KV head: 74 / 125 / 217 / 421 us; with one warp 99 / 173 / 289 / 632, with eight 203 / 203
// / 217 / 420).  e4m3: one.  There the conversions and products set the pace, not the reads, and a
// worker of several warps pads its rows to more (same sizes: 75 / 127 / 237 / 453 us with one warp,
// 80 / 139 / 242 / 476 by the bf16 rule).
static int warps_for(int64_t rows, fpx_dtype dt) {
  if (dt == FPX_E4M3) return 1;
  return rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= 64 ? 4 : 8;
}

// What a segment costs a worker in itself, in key tiles.  Measured with 0 / 1 / 2 / 4 / 6: 48 requests
// of 53 to 4220 keys on an e4m3 cache 129 / 105 / 102 / 106 / 106 us, 128 requests of 1 to 601 keys
// behind a prompt 160 / 149 / 148 / 149 / 150 us; long contexts do not change.
constexpr int kPad = 2, kPadTc = 2;
// Rows (per group and KV head, on average) from which the shared part takes 128-row tiles: behind a
// prompt of 18944 tokens 32 / 48 / 64 / 128 / 256 rows take 57 / 58 / 60 / 73 / 78 us with them and
// 51 / 67 / 68 / 99 / 162 us with 16-row tiles.
constexpr int kTcRows = 48;


struct Layout {
  int rw_own, rw_shared;  // warps per worker (fp32: 1)
  bool tc_shared;
  Line own, shared;       // offsets instead of pointers in owners / part_o / part_ml
  size_t owners_own, owners_shared, group_of, ml_own, o_own, ml_shared, o_shared, end;
};

static Layout layout_of(const DecodeDesc& p, fpx_dtype dt) {
  Layout L = {};
  const int64_t own_rows = static_cast<int64_t>(p.q_len) * p.group;
  const int64_t all_rows = own_rows * p.num_seqs;
  if (dt == FPX_F32) {
    L.rw_own = L.rw_shared = 1;
    L.own.rt = L.shared.rt = kRowsF32;
    L.own.tile = L.shared.tile = kTileF32;
  } else {
    L.rw_own = warps_for(own_rows, dt);
    L.rw_shared = warps_for(p.num_groups > 0 ? (all_rows + p.num_groups - 1) / p.num_groups : 1, dt);
    L.own.rt = 16 * L.rw_own;
    L.shared.rt = 16 * L.rw_shared;
    L.own.tile = L.shared.tile = kTile;
  }
  // Many rows behind a prompt: 128-row tiles on the tensor cores of the fifth generation.
  L.tc_shared = p.num_groups > 0 && tc_supported(p, dt) && all_rows >= kTcRows * p.num_groups;
  if (L.tc_shared) tc_line(p, &L.shared);
  L.own.n = p.num_seqs;
  L.shared.n = p.num_groups;
  L.own.nw = kCtas * (dt == FPX_F32 ? kWarpsF32 : kWarps / L.rw_own);
  L.shared.nw = L.tc_shared ? kCtas : kCtas * (dt == FPX_F32 ? kWarpsF32 : kWarps / L.rw_shared);
  L.own.pad = dt == FPX_F32 ? 1 : kPad;
  L.shared.pad = L.tc_shared ? kPadTc : L.own.pad;
  L.own.rps = static_cast<int>(own_rows < L.own.rt ? own_rows : L.own.rt);
  if (!L.tc_shared) L.shared.rps = L.shared.rt;
  const size_t own_slots =
      static_cast<size_t>(p.num_seqs) * ((own_rows + L.own.rt - 1) / L.own.rt) * p.hkv + L.own.nw;
  const size_t shared_slots =
      p.num_groups > 0
          ? static_cast<size_t>(all_rows / L.shared.rt + p.num_groups) * p.hkv + L.shared.nw
          : 0;
  size_t at = kStatusBytes;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 256);
    return a;
  };
  L.owners_own = take(sizeof(Owner) * (p.num_seqs + 1));
  L.owners_shared = take(sizeof(Owner) * (p.num_groups + 1));
  L.group_of = take(sizeof(int32_t) * p.num_seqs);
  L.ml_own = take(sizeof(float2) * own_slots * L.own.rps);
  L.o_own = take(sizeof(float) * own_slots * L.own.rps * p.d);
  L.ml_shared = take(sizeof(float2) * shared_slots * L.shared.rps);
  L.o_shared = take(sizeof(float) * shared_slots * L.shared.rps * p.d);
  L.end = at;
  return L;
}

// [rows, hkv, d] cache -> 3-D map with boxes of one head, `box_rows` keys and at most 128 bytes.
static bool make_cache_map(CUtensorMap* map, const void* base, int rows, int hkv, int d, int es,
                           int box_rows) {
  const int inner = d * es < 128 ? d : 128 / es;
  return make_tmap_rows(map, base, rows, hkv, d, es, inner, box_rows);
}

template <bool kFp8, int D, int RW>
static cudaError_t launch_mma_t(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeDesc& p,
                                const Line& line, const void* q, StatusBlock* st, cudaStream_t s) {
  constexpr size_t smem =
      1024 + kRing + kBarPitch * kWarps * Half<kFp8 ? 1 : 2, D, kTile>::kSlots1;
  const cudaError_t e = allow_smem<decode_mma_kernel<kFp8, D, RW>>(smem);
  if (e != cudaSuccess) return e;
  FPX_CHAIN((decode_mma_kernel<kFp8, D, RW>), kCtas, kThreads, smem, s, mk, mv, p, line,
            static_cast<const __nv_bfloat16*>(q), st);
  return cudaGetLastError();
}

template <int D>
static cudaError_t launch_bf16(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeDesc& p,
                               const Line& line, int rw, const void* q, StatusBlock* st,
                               cudaStream_t s) {
  switch (rw) {
    case 1: return launch_mma_t<false, D, 1>(mk, mv, p, line, q, st, s);
    case 2: return launch_mma_t<false, D, 2>(mk, mv, p, line, q, st, s);
    case 4: return launch_mma_t<false, D, 4>(mk, mv, p, line, q, st, s);
    default: return launch_mma_t<false, D, 8>(mk, mv, p, line, q, st, s);
  }
}

template <int D>
static cudaError_t launch_f32(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeDesc& p,
                              const Line& line, const void* q, StatusBlock* st, cudaStream_t s) {
  constexpr size_t smem =
      1024 + kWarpsF32 * kRingBytes + 1024 +
      kWarpsF32 * sizeof(float) * (kRowsF32 * 2 * (D / 2 + 4) + kTileF32 * kRowsF32);
  static_assert(kBarPitch * kWarpsF32 * Half<4, D, kTileF32>::kSlots1 <= 1024, "barriers");
  const cudaError_t e = allow_smem<decode_f32_kernel<D>>(smem);
  if (e != cudaSuccess) return e;
  FPX_CHAIN(decode_f32_kernel<D>, kCtas, kWarpsF32 * 32, smem, s, mk, mv, p, line,
            static_cast<const float*>(q), st);
  return cudaGetLastError();
}

static cudaError_t launch_line(const CUtensorMap& mk, const CUtensorMap& mv, const DecodeDesc& p,
                               fpx_dtype dt, const Line& line, int rw, const void* q,
                               StatusBlock* st, cudaStream_t s) {
  if (dt == FPX_F32)
    return p.d == 128 ? launch_f32<128>(mk, mv, p, line, q, st, s)
                      : launch_f32<64>(mk, mv, p, line, q, st, s);
  if (dt == FPX_BF16)
    return p.d == 128 ? launch_bf16<128>(mk, mv, p, line, rw, q, st, s)
                      : launch_bf16<64>(mk, mv, p, line, rw, q, st, s);
  return p.d == 128 ? launch_mma_t<true, 128, 1>(mk, mv, p, line, q, st, s)
                    : launch_mma_t<true, 64, 1>(mk, mv, p, line, q, st, s);
}

template <typename OT, int D>
static cudaError_t launch_join(const DecodeDesc& p, const Line& own, const Line& shared,
                               const int32_t* group_of, void* o, float* lse, StatusBlock* st, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.hq;
  // With as many rows as warps on the GPU one warp per row keeps enough loads in flight (2048 / 8192
  // rows: 183 / 208 us a call with one, 190 / 237 with eight); with fewer, the chain over a row's
  // partials counts (32 / 128 rows: 126 / 64 us with one, 101 / 57 with eight).
  if (rows >= kCtas * kWarps)
    FPX_CHAIN((join_kernel<OT, D, 1>), static_cast<unsigned>((rows + 7) / 8), 256, 0, s, p, own,
              shared, group_of, static_cast<OT*>(o), lse, st);
  else
    FPX_CHAIN((join_kernel<OT, D, 8>), static_cast<unsigned>(rows), 256, 0, s, p, own, shared,
              group_of, static_cast<OT*>(o), lse, st);
  return cudaGetLastError();
}

}  // namespace decode

size_t decode_workspace(const decode::DecodeDesc& p, fpx_dtype dt) {
  return decode::layout_of(p, dt).end;
}

bool decode_fits(const decode::DecodeDesc& p, fpx_dtype dt) {
  const decode::Layout L = decode::layout_of(p, dt);
  const double keys = static_cast<double>(p.pages_per_seq) * p.page;
  const double rows = static_cast<double>(p.q_len) * p.group;
  const double own = (keys / L.own.tile + 1 + L.own.pad) * p.num_seqs * p.hkv * (rows / L.own.rt + 1);
  const double shared = (keys / L.shared.tile + 1 + L.shared.pad) * p.hkv *
                        (rows * p.num_seqs / L.shared.rt + p.num_groups + 1);
  return own < INT32_MAX && shared < INT32_MAX;
}

cudaError_t launch_decode(const decode::DecodeDesc& p, fpx_dtype dt, const void* q, const void* kc,
                          const void* vc, void* o, float* lse, void* ws, StatusBlock* st,
                          cudaStream_t s, bool* encode_failed) {
  using namespace decode;
  *encode_failed = false;
  Layout L = layout_of(p, dt);
  char* base = static_cast<char*>(ws);
  L.own.owners = reinterpret_cast<Owner*>(base + L.owners_own);
  L.shared.owners = reinterpret_cast<Owner*>(base + L.owners_shared);
  L.own.part_ml = reinterpret_cast<float2*>(base + L.ml_own);
  L.own.part_o = reinterpret_cast<float*>(base + L.o_own);
  L.shared.part_ml = reinterpret_cast<float2*>(base + L.ml_shared);
  L.shared.part_o = reinterpret_cast<float*>(base + L.o_shared);
  int32_t* group_of = reinterpret_cast<int32_t*>(base + L.group_of);
  const int es = dt == FPX_F32 ? 4 : dt == FPX_BF16 ? 2 : 1;
  const int box = p.page < L.own.tile ? p.page : L.own.tile;
  CUtensorMap mk, mv;
  const int rows = p.num_pages << p.log2_page;
  if (!make_cache_map(&mk, kc, rows, p.hkv, p.d, es, box) ||
      !make_cache_map(&mv, vc, rows, p.hkv, p.d, es, box)) {
    *encode_failed = true;
    return cudaErrorInvalidValue;
  }
  if (p.num_groups == 0 && p.num_seqs <= kLocalSeqs)
    L.own.owners = nullptr;  // laid out by each CTA
  else
    FPX_CHAIN(plan_kernel, 1, kPlanThreads, 0, s, p, L.own, L.shared, group_of, st);
  cudaError_t e;
  if (p.num_groups > 0) {
    e = L.tc_shared ? launch_tc(p, L.shared, q, kc, vc, st, s, encode_failed)
                    : launch_line(mk, mv, p, dt, L.shared, L.rw_shared, q, st, s);
    if (e != cudaSuccess) return e;
  }
  if ((e = launch_line(mk, mv, p, dt, L.own, L.rw_own, q, st, s)) != cudaSuccess) return e;
  if (dt == FPX_F32)
    return p.d == 128 ? launch_join<float, 128>(p, L.own, L.shared, group_of, o, lse, st, s)
                      : launch_join<float, 64>(p, L.own, L.shared, group_of, o, lse, st, s);
  return p.d == 128 ? launch_join<__nv_bfloat16, 128>(p, L.own, L.shared, group_of, o, lse, st, s)
                    : launch_join<__nv_bfloat16, 64>(p, L.own, L.shared, group_of, o, lse, st, s);
}

}  // namespace fpx
