// fpx_span_simt.cu -- attention under a score rule on the CUDA cores, all arithmetic in 32 bits: fp32
// inputs and the shapes the tensor-core kernel does not take (blocks below 128, head dim 64).
//
// A CTA of 128 threads owns kRows query rows of one CSR row (h, s, I) and walks the row's key blocks
// kKeys at a time.  S = Q K^T: a thread has 2 rows x 4 keys (float4 along D: 6 shared loads for 32
// multiply-adds); the row statistics are reduced over the 8 lanes of a row pair; P goes through
// shared memory, transposed, so that P V has a thread at 4 rows x 4 or 8 columns (3 loads for 32
// multiply-adds).  The next keys are loaded into registers while the present ones are used.  Small
// row tiles, because what runs here is short: a 1000-token layer of 2 heads has 64 CTAs.
// 1000 tokens, 2 heads, D 64, window 200, the pass with spans and selection: 46 us, 175 us with a thread
// per query row.  What bounds it is the chain of short launches and, inside, latency.
#include <cuda_runtime.h>
#include <math_constants.h>

#include "fpx_internal.h"

namespace fpx {
namespace span {

constexpr int kSimtThreads = 128;

__device__ __forceinline__ void unpack16(const uint4& u, float* f, const float*) {
  f[0] = __uint_as_float(u.x);
  f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z);
  f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack16(const uint4& u, float* f, const __nv_bfloat16*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const uint4& u, float* f, const __nv_fp8_e4m3*) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    __nv_fp8_e4m3 c;
    c.__x = static_cast<__nv_fp8_storage_t>(w[i / 4] >> (8 * (i % 4)));
    f[i] = static_cast<float>(c);
  }
}

__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }
__device__ __forceinline__ void store_out(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// kRows rows and kRows keys per step (16 for blocks of 16, else 32).
template <typename T, typename OT, int D, int kRows>
__global__ void __launch_bounds__(kSimtThreads) span_simt_kernel(
    ProblemDesc p, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
    const int32_t* __restrict__ row_ptr, const int32_t* __restrict__ col_idx, OT* __restrict__ o,
    float* __restrict__ lse, SeqTables tab, const int32_t* __restrict__ order, RuleDesc rule,
    StatusBlock* st) {
  pdl_enter();  // after the previous kernel on the stream
  constexpr int kKeys = kRows;
  constexpr int kPitch = D + 4;                          // floats; 16-byte rows in other banks
  constexpr int kPerRow = D * static_cast<int>(sizeof(T)) / 16;  // 16-byte loads of a row
  constexpr int kElems = 16 / sizeof(T);
  constexpr int kLoads = (kKeys * kPerRow + kSimtThreads - 1) / kSimtThreads;
  constexpr int kTx = kKeys / 4;                         // threads along the keys (S)
  constexpr int kTy = kRows / 2;                         // row pairs
  static_assert(kTx * kTy <= kSimtThreads && 32 % kTx == 0, "S tile");
  constexpr int kCg = kSimtThreads / (kRows / 4);        // threads along D (P V)
  constexpr int kCols = D / kCg;                         // columns of a thread
  static_assert(kCols % 2 == 0, "columns");
  extern __shared__ float smem[];
  float* sq = smem;                       // [kRows][kPitch]
  float* sk = sq + kRows * kPitch;        // [kKeys][kPitch]
  float* sv = sk + kKeys * kPitch;        // [kKeys][kPitch]
  float* sp = sv + kKeys * kPitch;        // [kKeys][kRows + 4]: P transposed
  float* sc = sp + kKeys * (kRows + 4);   // [kRows] rescale of the accumulators, then 1 / sum
  if (!*tab.valid) return;

  const int subs = p.block / kRows;
  const int r = order[blockIdx.x / subs];
  const int h = r / p.nb_total;
  const int b = r - h * p.nb_total;
  const int s = seq_of_block(tab.blk_base, p.num_seqs, b);
  const int I = b - tab.blk_base[s];
  const int n = seq_len(p, s);
  const int64_t tok0 = seq_start(p, s);
  const int kvh = h / p.group;
  const int row0 = I * p.block + (blockIdx.x % subs) * kRows;
  if (row0 >= n) return;
  const int tid = threadIdx.x;

  for (int i = tid; i < kRows * kPerRow; i += kSimtThreads) {
    const int rr = i / kPerRow, c = i % kPerRow;
    float f[kElems];
    uint4 u = make_uint4(0, 0, 0, 0);
    if (row0 + rr < n)
      u = *reinterpret_cast<const uint4*>(q + ((tok0 + row0 + rr) * p.hq + h) * D + c * kElems);
    unpack16(u, f, static_cast<const T*>(nullptr));
#pragma unroll
    for (int e = 0; e < kElems; ++e) sq[rr * kPitch + c * kElems + e] = f[e];
  }

  // this thread's rows in S (two) and what they see
  const bool in_s = tid < kTx * kTy;
  const int tx = tid % kTx, ty = (tid / kTx) % kTy;
  float scale = p.scale;
  if (p.q_scale) scale *= p.q_scale[h] * p.k_scale[kvh];
  const ScoreMap map = score_map(rule, scale, h);
  int pos[2];
  KeySpan span[2];
  float m[2], l[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    pos[i] = row0 + 2 * ty + i;
    span[i] = {0, -1};
    if (pos[i] < n) span[i] = rule_span(rule, tok0 + pos[i], pos[i], n);
    m[i] = -CUDART_INF_F;
    l[i] = 0.f;
  }
  const int rg = tid / kCg, cg = tid % kCg;  // four rows, kCols columns of O
  float acc[4][kCols];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < kCols; ++c) acc[i][c] = 0.f;

  const int beg = row_ptr[r], end = row_ptr[r + 1];
  const int last = (n - 1) / p.block;
  // steps of kKeys keys over the listed blocks; entries outside the sequence are skipped
  int e = beg, sub = 0, key0 = 0;
  auto seek = [&]() -> bool {
    for (; e < end; ++e, sub = 0) {
      const int J = col_idx[e];
      if (J < 0 || J > last) {
        if (tid == 0 && blockIdx.x % subs == 0) record_error(st, FPX_ERR_DEVICE_INPUT, 21, r, J);
        continue;
      }
      key0 = J * p.block + sub * kKeys;
      if (sub < subs && key0 < n) {
        ++sub;
        return true;
      }
    }
    return false;
  };
  uint4 uk[kLoads], uv[kLoads];
  auto fetch = [&](int k0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = tid + i * kSimtThreads, kr = at / kPerRow, c = at % kPerRow;
      uk[i] = uv[i] = make_uint4(0, 0, 0, 0);
      if (kr < kKeys && k0 + kr < n) {
        const int64_t off = ((tok0 + k0 + kr) * p.hkv + kvh) * D + c * kElems;
        uk[i] = *reinterpret_cast<const uint4*>(k + off);
        uv[i] = *reinterpret_cast<const uint4*>(v + off);
      }
    }
  };
  bool more = seek();
  if (more) fetch(key0);
  while (more) {
    const int kb = key0;
    __syncthreads();  // the previous step's tiles are read
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = tid + i * kSimtThreads, kr = at / kPerRow, c = at % kPerRow;
      if (kr >= kKeys) continue;
      float f[kElems];
      unpack16(uk[i], f, static_cast<const T*>(nullptr));
#pragma unroll
      for (int x = 0; x < kElems; ++x) sk[kr * kPitch + c * kElems + x] = f[x];
      unpack16(uv[i], f, static_cast<const T*>(nullptr));
#pragma unroll
      for (int x = 0; x < kElems; ++x) sv[kr * kPitch + c * kElems + x] = f[x];
    }
    more = seek();
    if (more) fetch(key0);
    __syncthreads();
    if (in_s) {
      // keys tx, tx + kTx, ..: neighbouring lanes read neighbouring rows (pitch D + 4: other banks)
      float d[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll 8
      for (int c = 0; c < D; c += 4) {
        float4 a[2], w[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
          a[i] = *reinterpret_cast<const float4*>(sq + (2 * ty + i) * kPitch + c);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          w[j] = *reinterpret_cast<const float4*>(sk + (tx + j * kTx) * kPitch + c);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            d[i][j] = fmaf(a[i].x, w[j].x,
                           fmaf(a[i].y, w[j].y, fmaf(a[i].z, w[j].z, fmaf(a[i].w, w[j].w, d[i][j]))));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = kb + tx + j * kTx;
          const float y = map(d[i][j], fabsf(static_cast<float>(pos[i] - key)));
          d[i][j] = key >= span[i].lo && key <= span[i].hi ? y : -CUDART_INF_F;
          mx = fmaxf(mx, d[i][j]);
        }
#pragma unroll
        for (int x = kTx / 2; x > 0; x >>= 1)
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x, kTx));
        const float mn = fmaxf(m[i], mx);
        const float ref = mn == -CUDART_INF_F ? 0.f : mn;
        const float corr = m[i] == -CUDART_INF_F ? 0.f : ex2_approx(m[i] - mn);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float pr = ex2_approx(d[i][j] - ref);
          sum += pr;
          sp[(tx + j * kTx) * (kRows + 4) + 2 * ty + i] = pr;
        }
        l[i] = l[i] * corr + sum;  // this lane's keys
        m[i] = mn;
        if (tx == 0) sc[2 * ty + i] = corr;
      }
    }
    __syncthreads();
    const float4 c4 = *reinterpret_cast<const float4*>(sc + 4 * rg);
    const float cr[4] = {c4.x, c4.y, c4.z, c4.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[i][c] *= cr[i];
    const int have = min(kKeys, n - kb);
#pragma unroll 4
    for (int kk = 0; kk < have; ++kk) {
      const float4 p4 = *reinterpret_cast<const float4*>(sp + kk * (kRows + 4) + 4 * rg);
      const float pr[4] = {p4.x, p4.y, p4.z, p4.w};
      float w[kCols];
#pragma unroll
      for (int c = 0; c < kCols; c += 2) {
        const float2 x = *reinterpret_cast<const float2*>(sv + kk * kPitch + c * kCg + 2 * cg);
        w[c] = x.x;
        w[c + 1] = x.y;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < kCols; ++c) acc[i][c] = fmaf(pr[i], w[c], acc[i][c]);
    }
  }
  __syncthreads();
  if (in_s) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float sum = l[i];
#pragma unroll
      for (int x = kTx / 2; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x, kTx);
      if (tx != 0) continue;
      const bool none = m[i] == -CUDART_INF_F;
      sc[2 * ty + i] = none ? 0.f : 1.f / sum;
      if (lse && pos[i] < n)
        lse[static_cast<int64_t>(h) * p.total_tokens + tok0 + pos[i]] =
            none ? -CUDART_INF_F : (m[i] + __log2f(sum)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const float vs = p.v_scale ? p.v_scale[kvh] : 1.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 4 * rg + i;
    if (row >= n) continue;
    const float inv = sc[4 * rg + i] * vs;
    OT* dst = o + ((tok0 + row) * p.hq + h) * D + 2 * cg;
#pragma unroll
    for (int c = 0; c < kCols; c += 2) {
      store_out(dst + c * kCg, acc[i][c] * inv);
      store_out(dst + c * kCg + 1, acc[i][c + 1] * inv);
    }
  }
}

template <typename T, typename OT, int D, int kRows>
static cudaError_t launch_t(const ProblemDesc& p, const void* q, const void* k, const void* v,
                            const int32_t* row_ptr, const int32_t* col_idx, void* o, float* lse,
                            SeqTables t, const int32_t* order, const RuleDesc& rule,
                            StatusBlock* st, cudaStream_t s) {
  constexpr size_t smem =
      sizeof(float) * (3 * kRows * (D + 4) + kRows * (kRows + 4) + kRows);
  const cudaError_t e = allow_smem<span_simt_kernel<T, OT, D, kRows>>(smem);
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>(p.hq) * p.nb_total * (p.block / kRows);
  FPX_CHAIN((span_simt_kernel<T, OT, D, kRows>), static_cast<unsigned>(grid), kSimtThreads, smem, s, p,
            static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), row_ptr,
            col_idx, static_cast<OT*>(o), lse, t, order, rule, st);
  return cudaGetLastError();
}

template <typename T, typename OT>
static cudaError_t launch_d(const ProblemDesc& p, const void* q, const void* k, const void* v,
                            const int32_t* row_ptr, const int32_t* col_idx, void* o, float* lse,
                            SeqTables t, const int32_t* order, const RuleDesc& rule,
                            StatusBlock* st, cudaStream_t s) {
  if (p.block == 16)
    return p.d == 128
               ? launch_t<T, OT, 128, 16>(p, q, k, v, row_ptr, col_idx, o, lse, t, order, rule, st, s)
               : launch_t<T, OT, 64, 16>(p, q, k, v, row_ptr, col_idx, o, lse, t, order, rule, st, s);
  return p.d == 128
             ? launch_t<T, OT, 128, 32>(p, q, k, v, row_ptr, col_idx, o, lse, t, order, rule, st, s)
             : launch_t<T, OT, 64, 32>(p, q, k, v, row_ptr, col_idx, o, lse, t, order, rule, st, s);
}

}  // namespace span

cudaError_t launch_span_simt(const ProblemDesc& p, fpx_dtype dt, const void* q, const void* k,
                             const void* v, const int32_t* row_ptr, const int32_t* col_idx, void* o,
                             float* lse, SeqTables t, const int32_t* order, const RuleDesc& rule,
                             StatusBlock* st, cudaStream_t s) {
  if (p.hq * p.nb_total == 0) return cudaSuccess;
  switch (dt) {
    case FPX_F32:
      return span::launch_d<float, float>(p, q, k, v, row_ptr, col_idx, o, lse, t, order, rule, st, s);
    case FPX_BF16:
      return span::launch_d<__nv_bfloat16, __nv_bfloat16>(p, q, k, v, row_ptr, col_idx, o, lse, t,
                                                          order, rule, st, s);
    default:
      return span::launch_d<__nv_fp8_e4m3, __nv_bfloat16>(p, q, k, v, row_ptr, col_idx, o, lse, t,
                                                          order, rule, st, s);
  }
}

}  // namespace fpx
