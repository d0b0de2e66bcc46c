// fpx_attn_sm100.cu -- host side of the tensor-core attention (the kernel is in fpx_attn_sm100.cuh):
// tensor maps, the choice of the kernel and its launch.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <mutex>

#include "fpx_attn_sm100.cuh"
#include "fpx_internal.h"

namespace fpx {

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qr) ==
            cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

bool make_tmap_rows(CUtensorMap* map, const void* base, int T, int H, int D, int elem_bytes,
                    int box_elems, int box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t es = static_cast<cuuint64_t>(elem_bytes);
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(T)};
  cuuint64_t strides[2] = {D * es, static_cast<cuuint64_t>(H) * D * es};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(box_elems), 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = elem_bytes == 1   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : elem_bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT32;
  CUresult rc = fn(map, dt, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE,
                   box_elems * elem_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return rc == CUDA_SUCCESS;
}

bool make_tmap_heads(CUtensorMap* map, const void* base, int T, int H, int D, int heads,
                     int tokens) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(T)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(H) * D * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_tmap_rows128(CUtensorMap* map, const void* base, int T, int H, int D, int elem_bytes) {
  return make_tmap_rows(map, base, T, H, D, elem_bytes, 128 / elem_bytes, 128);
}

namespace sm100 {
static bool make_map(CUtensorMap* map, const void* base, int T, int H, int D, bool fp8) {
  return make_tmap_rows128(map, base, T, H, D, fp8 ? 1 : 2);
}

}  // namespace sm100

bool attn_tc_supported(const ProblemDesc& p, fpx_dtype dt) {
  return (dt == FPX_BF16 || dt == FPX_E4M3) && p.d == 128 && p.block == 128;
}

int64_t attn_tc_units(const ProblemDesc& p) {
  return static_cast<int64_t>(p.hkv) * p.nb_total * ((p.group + 1) / 2);
}

// Streaming multiprocessors of the current device (one resident CTA each: the kernel's shared
// memory admits no second one), looked up once per device.
static int sm_count() {
  static int counts[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (counts[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
      return 148;
    counts[dev] = n;
  }
  return counts[dev];
}

cudaError_t launch_attn_tc(const ProblemDesc& p, fpx_dtype dt, const void* q, const void* k,
                           const void* v, const int32_t* row_ptr, const int32_t* col_idx,
                           void* o, float* lse, SeqTables t, const int32_t* order,
                           int* queue_head, const uint32_t* vbits, const uint32_t* sbits,
                           int words, const RuleDesc* rule, StatusBlock* st, cudaStream_t s,
                           bool* encode_failed) {
  using namespace sm100;
  *encode_failed = false;
  const int64_t units = attn_tc_units(p);
  if (units == 0) return cudaSuccess;
  const bool fp8 = dt == FPX_E4M3;
  CUtensorMap mq, mk, mv;
  const int kv_rows = p.page_table ? p.num_pages * p.block : p.total_tokens;
  if (!make_map(&mq, q, p.total_tokens, p.hq, p.d, fp8) ||
      !make_map(&mk, k, kv_rows, p.hkv, p.d, fp8) ||
      !make_map(&mv, v, kv_rows, p.hkv, p.d, fp8)) {
    *encode_failed = true;
    return cudaErrorInvalidValue;
  }
  const bool mask = vbits != nullptr;
  const int rules = rule ? 1 | (rule->softcap > 0.f ? 2 : 0) | (rule->slopes ? 4 : 0) : 0;
  AttnKernel kern = rules ? (fp8 ? rule_kernel_e4m3(rules) : rule_kernel_bf16(rules))
                    : fp8 ? (mask ? attn_tc_kernel<true, true, 0> : attn_tc_kernel<true, false, 0>)
                          : (mask ? attn_tc_kernel<false, true, 0> : attn_tc_kernel<false, false, 0>);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(kSmemBytes));
  if (e != cudaSuccess) return e;
  // persistent: one CTA per SM takes units from the queue (heaviest first) until it is empty
  const int64_t grid = units < sm_count() ? units : sm_count();
  FPX_CHAIN(kern, static_cast<unsigned>(grid), kThreads, kSmemBytes, s, mq, mk, mv, p, row_ptr,
            col_idx, static_cast<__nv_bfloat16*>(o), lse, t, order, queue_head,
            static_cast<int>(units), vbits, sbits, words, rule ? *rule : RuleDesc{}, st);
  return cudaGetLastError();
}

}  // namespace fpx
