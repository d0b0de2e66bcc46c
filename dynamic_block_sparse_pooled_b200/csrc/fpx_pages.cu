// fpx_pages.cu -- the paged cache's bookkeeping on the device: block tables, the stack of free
// pages and the slot map from request lengths (fpx_page_resize), and the write of new K / V rows
// into the cache (fpx_kv_append).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "fpx_internal.h"

namespace fpx {
namespace pages {

constexpr int kThreads = 1024;
// Tokens up to which the planning CTA moves the pages and writes the slot map itself; above, a second
// launch does both with the whole GPU.  Replayed from a graph, prompts of 256 tokens on pages of 16, 256 /
// 2048 / 4096 / 8192 / 16384 tokens in all: 3.3 / 4.3 / 5.7 / 8.6 / 15.0 us in one launch, 4.9 / 5.1 / 5.5
// / 5.7 / 6.1 in two.  Pages given back are work too, but the host does not know how many they are, and
// a step in which many come is rare: one request of 8192 pages 8.2 us in one launch and 7.0 in two, 64
// requests of 512 pages 21 and 10, 1024 requests of 188 pages 161 and 52.
constexpr int kInlineTokens = 4096;

// Pages given and taken before each request; for the second launch in [num_seqs] their totals.
struct Plan {
  int32_t* give;
  int32_t* take;
  int32_t* ok;  // second launch: 1 where the call goes through, then the stack's height
};

// Requests and tokens of a call: a thread's next index, one stride of the largest grid (303104) or one
// CTA's round of requests further, has to stay within 32 bits.
constexpr int kMostItems = INT32_MAX - (1 << 20);
constexpr int kPushes = 4;  // pages that a thread gives back at a time: their loads overlap

struct ResizeArgs {
  int num_seqs, page, log2_page, num_pages, pages_per_seq, token_capacity;
  const int32_t* lens;
  const int32_t* new_lens;
  const int32_t* keep;
  int32_t* table;
  int32_t* free_pages;
  const int32_t* free_count;
  int32_t* free_count_out;
  int32_t* cu_new;
  int32_t* slots;
  int32_t* positions;
};

__device__ __forceinline__ int pages_of(const ResizeArgs& a, int len) {
  return (len + a.page - 1) >> a.log2_page;  // len <= INT32_MAX - page (checked)
}

// Pages that request s gives back (`give`), takes (`take`) and tokens it adds; false where its
// lengths are malformed.
struct Change {
  int have, want, give, take, tokens, first_give;
};
__device__ __forceinline__ bool change_of(const ResizeArgs& a, int s, Change& c) {
  const int n = a.lens[s], m = a.new_lens[s], keep = a.keep ? a.keep[s] : 0;
  const int64_t most = static_cast<int64_t>(a.pages_per_seq) << a.log2_page;
  if (n < 0 || m < 0 || n > most || m > most || keep < 0) {
    c = {0, 0, 0, 0, 0, 0};
    return false;
  }
  c.have = pages_of(a, n);
  c.want = pages_of(a, m);
  c.first_give = max(c.want, keep);
  c.give = max(c.have - c.first_give, 0);
  c.take = max(c.want - c.have, 0);
  c.tokens = max(m - n, 0);
  return true;
}

// The last request s in [0, n) with off[s] <= i (off non-decreasing, off[0] = 0, i < off[n]): the one
// that item i belongs to.
__device__ __forceinline__ int owner_of(const int32_t* off, int n, int i) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = lo + ((hi - lo + 1) >> 1);
    if (off[mid] <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Cache row of the token at position `pos` of request s, whose page is `pg`; -1 for a bad page.
__device__ __forceinline__ int slot_at(const ResizeArgs& a, int pg, int s, int pos,
                                       StatusBlock* st) {
  if (pg < 0 || pg >= a.num_pages) {
    record_error(st, FPX_ERR_DEVICE_INPUT, 51, s, pg);
    return -1;
  }
  return (pg << a.log2_page) + (pos & (a.page - 1));
}

struct Sums {
  int64_t give, take, tokens;
};
__device__ __forceinline__ Sums operator+(const Sums& x, const Sums& y) {
  return {x.give + y.give, x.take + y.take, x.tokens + y.tokens};
}
__device__ __forceinline__ Sums shfl_up(const Sums& x, int o) {
  return {__shfl_up_sync(0xffffffffu, x.give, o), __shfl_up_sync(0xffffffffu, x.take, o),
          __shfl_up_sync(0xffffffffu, x.tokens, o)};
}

// The i-th page given back by this call.
__device__ __forceinline__ int given_at(const ResizeArgs& a, const Plan& plan, int i) {
  const int s = owner_of(plan.give, a.num_seqs, i);
  const int first = max(pages_of(a, a.new_lens[s]), a.keep ? a.keep[s] : 0);
  return a.table[static_cast<int64_t>(s) * a.pages_per_seq + first + i - plan.give[s]];
}
// The page at place x of the stack after the pushes.  A page pushed by this call is looked up where
// it comes from, so that no thread waits for another one's push.
__device__ __forceinline__ int stack_at(const ResizeArgs& a, const Plan& plan, int count, int x) {
  return x < count ? a.free_pages[x] : given_at(a, plan, x - count);
}

// Pushes, pops and the slot map, an item each for the threads first, first + step, .. (a request gives
// or takes, so no row of the table is both read here and written; pushes go above the height that
// pops read below).
__device__ __forceinline__ void make_moves(const ResizeArgs& a, const Plan& plan, int count,
                                           int gives, int takes, int total, int first, int step,
                                           StatusBlock* st) {
  const int top = count + gives;
  if (first == 0) *a.free_count_out = top - takes;
  for (int i0 = first; i0 < gives; i0 += kPushes * step) {
    int pg[kPushes];
#pragma unroll
    for (int b = 0; b < kPushes; ++b)
      if (i0 + b * step < gives) pg[b] = given_at(a, plan, i0 + b * step);
#pragma unroll
    for (int b = 0; b < kPushes; ++b) {
      if (i0 + b * step >= gives) continue;
      if (pg[b] < 0 || pg[b] >= a.num_pages)
        record_error(st, FPX_ERR_DEVICE_INPUT, 55, i0 + b * step, pg[b]);
      a.free_pages[count + i0 + b * step] = pg[b];
    }
  }
  for (int i = first; i < takes; i += step) {
    const int s = owner_of(plan.take, a.num_seqs, i);
    const int pg = stack_at(a, plan, count, top - 1 - i);
    if (pg < 0 || pg >= a.num_pages) record_error(st, FPX_ERR_DEVICE_INPUT, 53, s, pg);
    a.table[static_cast<int64_t>(s) * a.pages_per_seq + pages_of(a, a.lens[s]) + i - plan.take[s]] = pg;
  }
  for (int t = first; t < a.token_capacity; t += step) {
    int slot = -1, pos = -1;
    if (t < total) {
      const int s = owner_of(a.cu_new, a.num_seqs, t);
      const int len = a.lens[s], have = pages_of(a, len);
      pos = len + t - a.cu_new[s];
      const int j = pos >> a.log2_page;
      const int pg = j < have ? a.table[static_cast<int64_t>(s) * a.pages_per_seq + j]
                              : stack_at(a, plan, count, top - 1 - (plan.take[s] + j - have));
      slot = slot_at(a, pg, s, pos, st);
    }
    a.slots[t] = slot;
    a.positions[t] = pos;
  }
}

// One CTA: thread t owns a run of consecutive requests.  Pass 1 sums what they give, take and add;
// a scan over the threads gives each its first place on the stack and among the tokens; the
// totals are checked before anything is written.  Then cu_new and the plan, and from it the moves,
// spread over this CTA's threads for few tokens, else over the second launch's.
// (The stack needs the requests' order, so the scan is the operator; it is latency-bound: two
// reads of the lengths and the scan.)
template <bool kInline>
__global__ void __launch_bounds__(kThreads) resize_kernel(ResizeArgs a, Plan plan, StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  __shared__ Sums warp_sum[32];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int per = (a.num_seqs + kThreads - 1) / kThreads;
  const int s0 = min(a.num_seqs, tid * per), s1 = min(a.num_seqs, s0 + per);
  const int count = *a.free_count;
  Sums sum = {0, 0, 0};
  Change c;
  bool good = true;
  for (int s = s0; s < s1; ++s) {
    if (!change_of(a, s, c)) {
      record_error(st, FPX_ERR_DEVICE_INPUT, 50, s, a.new_lens[s]);
      good = false;
    }
    sum = sum + Sums{c.give, c.take, c.tokens};
  }
  Sums x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums y = shfl_up(x, o);
    if (lane >= o) x = x + y;
  }
  if (lane == 31) warp_sum[w] = x;
  good = __syncthreads_and(good);
  if (w == 0) {
    Sums v = warp_sum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums y = shfl_up(v, o);
      if (lane >= o) v = v + y;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  const Sums all = warp_sum[31];
  Sums at = x;  // exclusive prefix of this thread's requests
  if (w > 0) at = at + warp_sum[w - 1];
  at = {at.give - sum.give, at.take - sum.take, at.tokens - sum.tokens};

  const bool fits = count >= 0 && count <= a.num_pages && count + all.give <= a.num_pages &&
                    all.take <= count + all.give && all.tokens <= a.token_capacity;
  if (!good || !fits) {
    if (tid == 0) {
      if (good) record_error(st, FPX_ERR_CAPACITY, 52, count, static_cast<int>(all.take));
      *a.free_count_out = count;
      if (!kInline) *plan.ok = 0;
    }
    for (int s = tid; s <= a.num_seqs; s += kThreads) a.cu_new[s] = 0;
    if (kInline)
      for (int t = tid; t < a.token_capacity; t += kThreads) a.slots[t] = a.positions[t] = -1;
    return;
  }
  const int gives = static_cast<int>(all.give), takes = static_cast<int>(all.take);
  const int total = static_cast<int>(all.tokens);
  for (int s = s0; s < s1; ++s) {
    change_of(a, s, c);
    a.cu_new[s] = static_cast<int>(at.tokens);
    plan.give[s] = static_cast<int>(at.give);
    plan.take[s] = static_cast<int>(at.take);
    at = at + Sums{c.give, c.take, c.tokens};
  }
  if (tid == 0) {
    a.cu_new[a.num_seqs] = total;
    if (!kInline) {
      plan.give[a.num_seqs] = gives;
      plan.take[a.num_seqs] = takes;
      plan.ok[0] = 1;
      plan.ok[1] = count;  // the second launch writes the new height, which may lie over it
    }
  }
  if (!kInline) return;
  __syncthreads();  // cu_new and the plan are written
  make_moves(a, plan, count, gives, takes, total, tid, kThreads, st);
}

__global__ void __launch_bounds__(256) moves_kernel(ResizeArgs a, Plan plan, StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  const int first = blockIdx.x * blockDim.x + threadIdx.x, step = gridDim.x * blockDim.x;
  if (plan.ok[0] != 0) {
    make_moves(a, plan, plan.ok[1], plan.give[a.num_seqs], plan.take[a.num_seqs],
               a.cu_new[a.num_seqs], first, step, st);
  } else {
    for (int t = first; t < a.token_capacity; t += step) a.slots[t] = a.positions[t] = -1;
  }
}

// ---- append -------------------------------------------------------------------------------------

// x / scale rounded to fp32 as by IEEE division, where that matters for an e4m3 code: the quotient by
// the reciprocal, corrected once by its remainder (Markstein's step: exact to the last bit when the
// reciprocal is correctly rounded).  Beyond 1024 the code saturates whatever the last bits are, and
// the remainder could overflow.  Scales near the ends of fp32's range, whose reciprocal is not a
// normal number, are divided by.  (Three multiply-adds instead of a division: with the walk of append_kernel
// 16384 rows of 8 x 128 took 27 us instead of 35.)
struct Divisor {
  float s, r;
  bool plain;
  __device__ __forceinline__ void set(float scale) {
    s = scale;
    r = __fdiv_rn(1.f, scale);
    plain = !(scale > 1e-30f && scale < 1e30f);
  }
  __device__ __forceinline__ float operator()(float x) const {
    if (plain) return __fdiv_rn(x, s);
    const float q = x * r;
    return fabsf(q) < 1024.f ? fmaf(fmaf(-q, s, x), r, q) : q;
  }
};
// Two values as e4m3, round to nearest even, saturating (NaN stays NaN).
__device__ __forceinline__ uint32_t quant2(float x, float y, const Divisor& d) {
  return __nv_cvt_float2_to_fp8x2(make_float2(d(x), d(y)), __NV_SATFINITE, __NV_E4M3);
}

constexpr int kBatch = 4;  // rows of a thread in flight

// A thread keeps one 16-byte chunk c of the row [hkv, d] (so its head's scale too) and walks over the
// tokens, kBatch at a time; neighbouring threads have neighbouring chunks, so both sides are
// contiguous per row.  blockIdx.y: K or V.  16384 rows of 8 x 128 from bf16 to e4m3: 101 MB in 27 us, 3.7
// TB/s; four rows in flight and no division of an index per chunk were worth 35 -> 27.  What bounds that
// case is its waves: the e4m3 form takes 72 registers, so 444 of its 1184 CTAs are resident, 2.7 waves.
template <bool kQuant>
__global__ void __launch_bounds__(256) append_kernel(
    int tokens, int row_chunks, int chunks_per_head, const char* __restrict__ k, int64_t k_stride,
    const char* __restrict__ v, int64_t v_stride, const int32_t* __restrict__ slots,
    char* __restrict__ k_cache, char* __restrict__ v_cache, int num_slots,
    const float* __restrict__ k_scale, const float* __restrict__ v_scale, StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  const bool is_v = blockIdx.y != 0;
  const char* src = is_v ? v : k;
  const int64_t stride = is_v ? v_stride : k_stride;
  char* dst = is_v ? v_cache : k_cache;
  const float* scale = is_v ? v_scale : k_scale;
  const int span = min(row_chunks, 256), rows = 256 / span;  // chunks and tokens of a block
  const int sub = threadIdx.x / span;
  if (sub >= rows) return;
  const int step = gridDim.x * rows;
  for (int c = threadIdx.x - sub * span; c < row_chunks; c += span) {
    Divisor div = {};
    if (kQuant) div.set(scale[c / chunks_per_head]);
    for (int64_t t0 = blockIdx.x * rows + sub; t0 < tokens; t0 += kBatch * static_cast<int64_t>(step)) {
      int slot[kBatch];
      uint4 x[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int64_t t = t0 + b * static_cast<int64_t>(step);
        slot[b] = -1;
        if (t < tokens) {
          slot[b] = slots[t];
          x[b] = __ldcs(reinterpret_cast<const uint4*>(src + t * stride + c * 16));
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        if (slot[b] < 0) continue;
        if (slot[b] >= num_slots) {
          if (c == 0)
            record_error(st, FPX_ERR_DEVICE_INPUT, 54, static_cast<int>(t0) + b * step, slot[b]);
          continue;
        }
        const int64_t at = static_cast<int64_t>(slot[b]) * row_chunks + c;
        if (kQuant) {
          const uint32_t u[4] = {x[b].x, x[b].y, x[b].z, x[b].w};
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            q[j] = quant2(__uint_as_float(u[j] << 16), __uint_as_float(u[j] & 0xffff0000u), div);
          *reinterpret_cast<uint2*>(dst + at * 8) =
              make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
        } else {
          *reinterpret_cast<uint4*>(dst + at * 16) = x[b];
        }
      }
    }
  }
}

bool is_aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

Plan plan_at(void* ws, int num_seqs) {
  int32_t* base = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kStatusBytes);
  return {base + 64, base + 64 + num_seqs + 1, base};
}

cudaError_t launch_resize(const ResizeArgs& a, void* ws, cudaStream_t s) {
  StatusBlock* st = static_cast<StatusBlock*>(ws);
  const Plan plan = plan_at(ws, a.num_seqs);
  if (a.token_capacity <= kInlineTokens) {
    FPX_CHAIN((resize_kernel<true>), 1, kThreads, 0, s, a, plan, st);
    return cudaGetLastError();
  }
  FPX_CHAIN((resize_kernel<false>), 1, kThreads, 0, s, a, plan, st);
  const int want = (a.token_capacity - 1) / 256 + 1;
  constexpr int kMoveCtas = 148 * 8;
  static_assert(kMoveCtas * 256 <= (1 << 20), "kMostItems");
  FPX_CHAIN(moves_kernel, want < kMoveCtas ? want : kMoveCtas, 256, 0, s, a, plan, st);
  return cudaGetLastError();
}

template <bool kQuant>
cudaError_t launch_append(int tokens, int row_chunks, int chunks_per_head, const void* k,
                          int64_t k_stride, const void* v, int64_t v_stride, const int32_t* slots,
                          void* kc, void* vc, int num_slots, const float* ks, const float* vs,
                          StatusBlock* st, cudaStream_t s) {
  const int rows = 256 / (row_chunks < 256 ? row_chunks : 256);
  const int want = (tokens - 1) / rows + 1;
  const unsigned grid = static_cast<unsigned>(want < 148 * 4 ? want : 148 * 4);
  FPX_CHAIN((append_kernel<kQuant>), dim3(grid, 2), 256, 0, s, tokens, row_chunks, chunks_per_head,
            static_cast<const char*>(k), k_stride, static_cast<const char*>(v), v_stride, slots,
            static_cast<char*>(kc), static_cast<char*>(vc), num_slots, ks, vs, st);
  return cudaGetLastError();
}

}  // namespace pages
}  // namespace fpx

using namespace fpx;
using fpx::pages::is_aligned;

extern "C" {

size_t fpx_page_workspace_bytes(int32_t num_seqs) {
  if (num_seqs < 1) return 0;
  return kStatusBytes + 256 + align_up(sizeof(int32_t) * 2 * (static_cast<size_t>(num_seqs) + 1), 256);
}

fpx_status fpx_page_resize(int32_t num_seqs, int32_t page, int32_t num_pages,
                           const int32_t* lens_d, const int32_t* new_lens_d,
                           const int32_t* keep_pages_d, int32_t* block_table_d,
                           int32_t pages_per_seq, int32_t* free_pages_d,
                           const int32_t* free_count_d, int32_t* free_count_out_d,
                           int32_t* cu_new_d, int32_t* slots_d, int32_t* positions_d,
                           int32_t token_capacity, void* ws, size_t ws_bytes,
                           fpx_stream_t stream) {
  if (num_seqs < 1 || num_pages < 1 || pages_per_seq < 1 || token_capacity < 0)
    return FPX_ERR_INVALID_ARG;
  if (page < 16 || page > 128 || (page & (page - 1)) != 0) return FPX_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(num_pages) * page > INT32_MAX ||
      static_cast<int64_t>(pages_per_seq) * page > INT32_MAX - page ||
      static_cast<int64_t>(pages_per_seq) * num_seqs > INT32_MAX ||
      num_seqs > pages::kMostItems || token_capacity > pages::kMostItems)
    return FPX_ERR_UNSUPPORTED;
  if (!lens_d || !new_lens_d || !block_table_d || !free_pages_d || !free_count_d ||
      !free_count_out_d || !cu_new_d || !ws)
    return FPX_ERR_INVALID_ARG;
  if (token_capacity > 0 && (!slots_d || !positions_d)) return FPX_ERR_INVALID_ARG;
  const void* words[] = {lens_d,           new_lens_d, keep_pages_d, block_table_d, free_pages_d,
                         free_count_d, free_count_out_d, cu_new_d,   slots_d,      positions_d};
  for (const void* x : words)
    if (!is_aligned(x, 4)) return FPX_ERR_ALIGNMENT;
  if (!is_aligned(ws, 256)) return FPX_ERR_ALIGNMENT;
  if (ws_bytes < fpx_page_workspace_bytes(num_seqs)) return FPX_ERR_CAPACITY;
  pages::ResizeArgs a;
  a.num_seqs = num_seqs;
  a.page = page;
  a.log2_page = 0;
  while ((1 << a.log2_page) < page) ++a.log2_page;
  a.num_pages = num_pages;
  a.pages_per_seq = pages_per_seq;
  a.token_capacity = token_capacity;
  a.lens = lens_d;
  a.new_lens = new_lens_d;
  a.keep = keep_pages_d;
  a.table = block_table_d;
  a.free_pages = free_pages_d;
  a.free_count = free_count_d;
  a.free_count_out = free_count_out_d;
  a.cu_new = cu_new_d;
  a.slots = slots_d;
  a.positions = positions_d;
  return pages::launch_resize(a, ws, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FPX_OK
             : FPX_ERR_CUDA;
}

fpx_status fpx_kv_append(fpx_dtype dtype, int32_t hkv, int32_t d, int32_t num_tokens,
                         const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const int32_t* slots_d, void* k_cache, void* v_cache, int32_t num_slots,
                         const float* k_scale_d, const float* v_scale_d, void* ws,
                         size_t ws_bytes, fpx_stream_t stream) {
  if (dtype != FPX_F32 && dtype != FPX_BF16 && dtype != FPX_E4M3) return FPX_ERR_UNSUPPORTED;
  if (d != 64 && d != 128) return FPX_ERR_UNSUPPORTED;
  if (hkv < 1 || num_tokens < 0 || num_slots < 1) return FPX_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(hkv) * d;
  if (row > INT32_MAX / 4) return FPX_ERR_UNSUPPORTED;
  const bool quant = dtype == FPX_E4M3;
  if (quant != (k_scale_d != nullptr) || quant != (v_scale_d != nullptr))
    return FPX_ERR_INVALID_ARG;
  if (!ws || (num_tokens > 0 && (!k || !v || !slots_d || !k_cache || !v_cache)))
    return FPX_ERR_INVALID_ARG;
  const int64_t es = dtype == FPX_F32 ? 4 : 2;
  const int64_t most = INT64_MAX / 4 / (static_cast<int64_t>(num_tokens) + 1);  // bytes fit int64
  if (k_stride < row || v_stride < row || k_stride > most || v_stride > most)
    return FPX_ERR_INVALID_ARG;
  if (!is_aligned(k, 16) || !is_aligned(v, 16) || (k_stride * es) % 16 != 0 ||
      (v_stride * es) % 16 != 0 || !is_aligned(slots_d, 4) || !is_aligned(k_cache, 16) ||
      !is_aligned(v_cache, 16) || !is_aligned(k_scale_d, 4) || !is_aligned(v_scale_d, 4) ||
      !is_aligned(ws, 256))
    return FPX_ERR_ALIGNMENT;
  if (ws_bytes < kStatusBytes) return FPX_ERR_CAPACITY;
  if (num_tokens == 0) return FPX_OK;
  const int row_chunks = static_cast<int>(row * es / 16), per_head = static_cast<int>(d * es / 16);
  StatusBlock* st = static_cast<StatusBlock*>(ws);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      quant ? pages::launch_append<true>(num_tokens, row_chunks, per_head, k, k_stride * es, v,
                                         v_stride * es, slots_d, k_cache, v_cache, num_slots,
                                         k_scale_d, v_scale_d, st, s)
            : pages::launch_append<false>(num_tokens, row_chunks, per_head, k, k_stride * es, v,
                                          v_stride * es, slots_d, k_cache, v_cache, num_slots,
                                          nullptr, nullptr, st, s);
  return e == cudaSuccess ? FPX_OK : FPX_ERR_CUDA;
}

}  // extern "C"
