// fpx_span.cu -- key spans of packed documents, and the key blocks that spans reach (CSR rows for
// the attention under a score rule).
#include <cuda_runtime.h>

#include "fpx_internal.h"

namespace fpx {
namespace span {

// Largest index d in [0, n) with off[d] <= t (off non-decreasing, off[0] <= t).
__device__ __forceinline__ int owner_of(const int32_t* __restrict__ off, int n, int t) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = lo + ((hi - lo + 1) >> 1);
    if (__ldg(off + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// One thread per token; 8 bytes written per token, the offsets come from cache.
__global__ void __launch_bounds__(256) spans_kernel(ProblemDesc p, int num_docs,
                                                    const int32_t* __restrict__ doc_cu,
                                                    const int32_t* __restrict__ prefix,
                                                    int32_t* __restrict__ key_lo,
                                                    int32_t* __restrict__ key_hi) {
  pdl_enter();  // after the previous kernel on the stream
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= p.total_tokens) return;
  const int s = p.cu ? owner_of(p.cu, p.num_seqs, t) : 0;
  const int a = seq_start(p, s), n = seq_len(p, s);
  int doc = s, d0 = a;
  int64_t d1 = static_cast<int64_t>(a) + n;
  bool inside = true;
  if (doc_cu) {
    inside = num_docs > 0 && t >= doc_cu[0] && t < doc_cu[num_docs];
    if (inside) {
      doc = owner_of(doc_cu, num_docs, t);
      d0 = max(d0, doc_cu[doc]);
      d1 = min(d1, static_cast<int64_t>(doc_cu[doc + 1]));
    }
  }
  int lo = 0, hi = -1;
  if (inside) {
    lo = d0 - a;
    hi = t - a;
    if (prefix) {
      const int64_t end = min(d1, static_cast<int64_t>(d0) + max(prefix[doc], 0)) - 1 - a;
      if (end > hi) hi = static_cast<int>(end);
    }
  }
  key_lo[t] = lo;
  key_hi[t] = hi;
}

constexpr int kWarps = 8;  // rows per CTA, as the select stage's kernels expect

// Row r = (h, s, I), a warp each: the blocks [lo / B, hi / B] of every query of block I, OR-ed into
// a bitmask in shared memory (a lane skips a range that the lane before it has: the queries of a
// block mostly share theirs), then written with its count in the select stage's layout.
__global__ void __launch_bounds__(kWarps * 32) span_count_kernel(
    ProblemDesc p, RuleDesc rule, SeqTables tab, int32_t* __restrict__ counts,
    int64_t* __restrict__ cta_tot, uint32_t* __restrict__ mask, int mask_words) {
  pdl_enter();  // after the previous kernel on the stream
  extern __shared__ uint32_t bits[];  // [kWarps][mask_words]
  __shared__ int w_tot[kWarps];
  if (!*tab.valid) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int R = p.hq * p.nb_total;
  const int r = blockIdx.x * kWarps + warp;
  uint32_t* mine = bits + warp * mask_words;
  int cnt = 0;
  if (r < R) {
    for (int w = lane; w < mask_words; w += 32) mine[w] = 0;
    __syncwarp();
    const int b = r % p.nb_total;
    const int s = seq_of_block(tab.blk_base, p.num_seqs, b);
    const int I = b - tab.blk_base[s];
    const int n = seq_len(p, s);
    const int64_t tok0 = seq_start(p, s);
    for (int c0 = 0; c0 < p.block; c0 += 32) {
      const int i = I * p.block + c0 + lane;
      int ja = 1, jb = 0;
      if (c0 + lane < p.block && i < n) {
        const KeySpan ks = rule_span(rule, tok0 + i, i, n);
        if (ks.lo <= ks.hi) {
          ja = ks.lo / p.block;
          jb = ks.hi / p.block;
        }
      }
      const int pa = __shfl_up_sync(0xffffffffu, ja, 1), pb = __shfl_up_sync(0xffffffffu, jb, 1);
      if (ja <= jb && (lane == 0 || pa != ja || pb != jb)) {
        for (int w = ja >> 5; w <= (jb >> 5); ++w) {
          const int x = max(ja - w * 32, 0), y = min(jb - w * 32, 31);
          atomicOr(&mine[w], (0xffffffffu >> (31 - y)) & (0xffffffffu << x));
        }
      }
    }
    __syncwarp();
    for (int w = lane; w < mask_words; w += 32) {
      mask[static_cast<int64_t>(r) * mask_words + w] = mine[w];
      cnt += __popc(mine[w]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
    if (lane == 0) counts[r] = cnt;
  }
  if (lane == 0) w_tot[warp] = cnt;
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t t = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += w_tot[i];
    cta_tot[blockIdx.x] = t;
  }
}

}  // namespace span

cudaError_t launch_spans(const ProblemDesc& p, int num_docs, const int32_t* doc_cu,
                         const int32_t* prefix, int32_t* key_lo, int32_t* key_hi, cudaStream_t s) {
  if (p.total_tokens == 0) return cudaSuccess;
  FPX_CHAIN(span::spans_kernel, static_cast<unsigned>((p.total_tokens - 1) / 256 + 1), 256, 0, s, p,
            num_docs, doc_cu, prefix, key_lo, key_hi);
  return cudaGetLastError();
}

cudaError_t launch_span_count(const ProblemDesc& p, const RuleDesc& rule, SeqTables t,
                              int32_t* counts, int64_t* cta_tot, uint32_t* mask, int mask_words,
                              cudaStream_t s) {
  const int64_t R = static_cast<int64_t>(p.hq) * p.nb_total;
  if (R == 0) return cudaSuccess;
  // nb_max <= 65535 (the worst-case CSR fits int32), so at most 64 KB
  const size_t smem = sizeof(uint32_t) * span::kWarps * static_cast<size_t>(mask_words);
  const cudaError_t e = allow_smem<span::span_count_kernel>(64 * 1024);
  if (e != cudaSuccess) return e;
  FPX_CHAIN(span::span_count_kernel, static_cast<unsigned>((R + span::kWarps - 1) / span::kWarps),
            span::kWarps * 32, smem, s, p, rule, t, counts, cta_tot, mask, mask_words);
  return cudaGetLastError();
}

}  // namespace fpx
