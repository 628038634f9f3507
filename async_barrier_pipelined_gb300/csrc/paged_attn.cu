// Attention of a serving step's new tokens over a paged key/value cache
// (attn_f16_paged_fwd): argument checks, kernels and entry point.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdio>

#include "host.h"
#include "ptx.cuh"
#include "schedule.h"
#include "common.cuh"
#include "paged_schedule.h"

#include "paged_small.cuh"
#include "paged_large.cuh"

using namespace gf16;
using namespace gf16::host;

namespace gf16 {
namespace host {

int paged_plan_init(gemm_f16_plan_s* p, const cudaDeviceProp& prop) {
  GF16_CUDA(cudaFuncSetAttribute(paged::small::paged_small_kernel<16>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::small::Cfg<16>::SMEM),
            "cudaFuncSetAttribute(paged attention kernel smem)");
  GF16_CUDA(cudaFuncSetAttribute(paged::small::paged_small_kernel<32>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::small::Cfg<32>::SMEM),
            "cudaFuncSetAttribute(paged attention kernel smem)");
  GF16_CUDA(cudaFuncSetAttribute(paged::small::paged_small_kernel<64>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::small::Cfg<64>::SMEM),
            "cudaFuncSetAttribute(paged attention kernel smem)");
  GF16_CUDA(cudaFuncSetAttribute(paged::large::paged_large_kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)paged::large::SMEM_BYTES),
            "cudaFuncSetAttribute(paged attention kernel smem)");
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(prop.multiProcessorCount / 2 * 2), 1, 1);
  cfg.blockDim = dim3(paged::large::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = paged::large::SMEM_BYTES;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  GF16_CUDA(cudaOccupancyMaxActiveClusters(&clusters, paged::large::paged_large_kernel, &cfg),
            "cudaOccupancyMaxActiveClusters(paged attention kernel)");
  p->paged_pairs = std::min(std::max(clusters, 1), paged::large::MAX_CLUSTERS);
  return GEMM_F16_OK;
}

void paged_plan_release(gemm_f16_plan_s* p) {
  if (p->paged_ws) cudaFree(p->paged_ws);
}

}  // namespace host
}  // namespace gf16

namespace {

constexpr int HEAD_DIM = 256;

// Workspace of the attention over a paged cache: the cut tiles, the partials'
// offsets and sums, and their FP32 O; of the two kernels' needs the larger.
// Its size depends on the device alone: allocated by the plan's first call and
// kept.  Not on the call's stream: an allocation that the stream records while
// it is captured into a graph belongs to the graph's replays, and a call outside
// them would use memory that is not there.
constexpr int SMALL_ROWS = 64;   // most rows of a request for the small kernel

int ensure_workspace(gemm_f16_plan_s* p, paged::Params* prm) {
  const size_t small_slots = 2 * (size_t)p->num_sms, large_slots = 2 * (size_t)p->paged_pairs;
  const size_t rows = std::max(small_slots * SMALL_ROWS, large_slots * paged::large::PART_ROWS);
  const size_t cut = (size_t)p->num_sms * sizeof(paged::CutTile);
  const size_t ml = rows * sizeof(float2);
  if (!p->paged_ws) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;   // this thread may be capturing
    GF16_CUDA(cudaThreadExchangeStreamCaptureMode(&mode), "cudaThreadExchangeStreamCaptureMode");
    const cudaError_t e = cudaMalloc(&p->paged_ws, cut + ml + rows * HEAD_DIM * sizeof(float));
    cudaThreadExchangeStreamCaptureMode(&mode);
    if (e != cudaSuccess) p->paged_ws = nullptr;
    GF16_CUDA(e, "paged attention workspace allocation");
  }
  char* ws = static_cast<char*>(p->paged_ws);
  prm->cut = reinterpret_cast<paged::CutTile*>(ws);
  prm->part_ml = reinterpret_cast<float2*>(ws + cut);
  prm->part = reinterpret_cast<float*>(ws + cut + ml);
  return GEMM_F16_OK;
}

// Tensor maps through the plan's cache (keys tagged apart from the others).
int encode(gemm_f16_plan_s* p, const uint64_t (&key)[8], CUtensorMap* map, int rank,
           const void* ptr, const cuuint64_t* dims, const cuuint64_t* strides,
           const cuuint32_t* box) {
  if (tmap_lookup(p, key, map)) return GEMM_F16_OK;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail_msg("cuTensorMapEncodeTiled entry point not available");
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r =
      fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims,
         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error),
                  "cuTensorMapEncodeTiled (paged attention operand) failed (CUresult %d)", (int)r);
    return GEMM_F16_ERR_CUDA;
  }
  tmap_remember(p, key, *map);
  return GEMM_F16_OK;
}

// A stride of an extent-1 dimension is not used; the map gets a valid one.
cuuint64_t stride_bytes(int64_t st, int64_t extent, int64_t other) {
  return (cuuint64_t)(extent > 1 ? st : other) * 2;
}

// Cache as a 4-D map: numbers, rows of a page, heads, pages; boxes of 64
// numbers by `rows` rows.
int encode_cache(gemm_f16_plan_s* p, CUtensorMap* map, const void* ptr, int num_pages,
                 int page_size, int kv_heads, const int64_t st[3], int rows) {
  const uint64_t key[8] = {(uint64_t)(uintptr_t)ptr,
                           ((uint64_t)(uint32_t)num_pages << 32) | (uint32_t)page_size,
                           ((uint64_t)(uint32_t)kv_heads << 32) | (uint32_t)rows,
                           (uint64_t)st[0], (uint64_t)st[1], (uint64_t)st[2], 0,
                           0x5043000000000000ull};
  const cuuint64_t dims[4] = {HEAD_DIM, (cuuint64_t)page_size, (cuuint64_t)kv_heads,
                              (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {stride_bytes(st[1], page_size, HEAD_DIM),
                                 stride_bytes(st[2], kv_heads, HEAD_DIM),
                                 stride_bytes(st[0], num_pages, HEAD_DIM)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1};
  return encode(p, key, map, 4, ptr, dims, strides, box);
}

// Queries as a 3-D map: numbers, heads, tokens; boxes of 64 numbers by the
// heads of one key/value head by `tokens`, which lie in shared memory as
// consecutive rows.
int encode_q(gemm_f16_plan_s* p, CUtensorMap* map, const void* ptr, int total_q, int q_heads,
             const int64_t st[2], int group, int tokens) {
  const uint64_t key[8] = {(uint64_t)(uintptr_t)ptr,
                           ((uint64_t)(uint32_t)total_q << 32) | (uint32_t)q_heads,
                           (uint64_t)st[0], (uint64_t)st[1],
                           ((uint64_t)(uint32_t)group << 32) | (uint32_t)tokens, 0, 0,
                           0x5051000000000000ull};
  const cuuint64_t dims[3] = {HEAD_DIM, (cuuint64_t)q_heads, (cuuint64_t)total_q};
  const cuuint64_t strides[2] = {stride_bytes(st[1], q_heads, HEAD_DIM),
                                 stride_bytes(st[0], total_q, HEAD_DIM)};
  const cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)tokens};
  return encode(p, key, map, 3, ptr, dims, strides, box);
}

// The merge of the tiles that `workers` cut.
int launch_merge(void (*kernel)(const paged::Params), const char* what, int workers, int parts,
                 int threads, cudaStream_t stream, const paged::Params& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)workers, (unsigned)parts, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, kernel, prm), what);
  return GEMM_F16_OK;
}

template <int N>
auto merge_kernel(int rows) {
  return rows == 2 ? paged::small::paged_small_merge_kernel<N, 2>
                   : paged::small::paged_small_merge_kernel<N, 4>;
}

using Kernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap,
                        const paged::Params);

int launch(gemm_f16_plan_s* p, Kernel kernel, const char* what, int ctas, int threads,
           size_t smem, cudaStream_t stream, const CUtensorMap& tmQ, const CUtensorMap& tmK,
           const CUtensorMap& tmV, const paged::Params& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  cudaEvent_t t0;
  int rc = timing_begin(p, stream, &t0);
  if (rc) return rc;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, tmQ, tmK, tmV, prm);
  rc = timing_end(p, stream, t0, le == cudaSuccess);
  GF16_CUDA(le, what);
  return rc;
}

bool off(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }

// Strides of a dimension of extent 1 are not used.
int check_strides(const int64_t* st, const int* extent, int n) {
  if (!st) return GEMM_F16_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && (st[i] < HEAD_DIM || st[i] >= ((int64_t)1 << 38)))
      return GEMM_F16_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && (st[i] & 7)) return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

}  // namespace

extern "C" {

int attn_f16_paged_validate(int batch, int total_q, int max_q, int q_heads, int kv_heads,
                            int head_dim, const void* Q, const int64_t q_strides[2],
                            const void* Kc, const int64_t kc_strides[3], const void* Vc,
                            const int64_t vc_strides[3], int num_pages, int page_size,
                            const int32_t* block_table, int64_t table_stride, int max_pages,
                            const int32_t* starts, const int32_t* kv_lens, const void* O,
                            const int64_t o_strides[2], float scale, int window, int sinks) {
  if (batch < 1 || batch > 65535 || total_q < 0 || max_q < 0) return GEMM_F16_ERR_INVALID_ARG;
  if (head_dim != HEAD_DIM || kv_heads < 1 || kv_heads > 1024 || q_heads < kv_heads ||
      q_heads % kv_heads || q_heads / kv_heads > 64)
    return GEMM_F16_ERR_INVALID_ARG;
  if (num_pages < 1 || page_size < 8 || page_size > 32768 || page_size % 8 || max_pages < 1 ||
      max_pages > (1 << 24) || table_stride < max_pages || window < 0 || sinks < 0)
    return GEMM_F16_ERR_INVALID_ARG;
  if (!(std::fabs(scale) <= 3.0e38f)) return GEMM_F16_ERR_INVALID_ARG;
  if (!Kc || !Vc || !block_table || !starts || !kv_lens) return GEMM_F16_ERR_INVALID_ARG;
  if (total_q > 0 && (!Q || !O)) return GEMM_F16_ERR_INVALID_ARG;
  int rc;
  const int e[2] = {total_q, q_heads}, ce[3] = {num_pages, page_size, kv_heads};
  if ((rc = check_strides(q_strides, e, 2)) || (rc = check_strides(o_strides, e, 2)) ||
      (rc = check_strides(kc_strides, ce, 3)) || (rc = check_strides(vc_strides, ce, 3)))
    return rc;
  if (off(Q, 15) || off(O, 15) || off(Kc, 15) || off(Vc, 15) || off(block_table, 3) ||
      off(starts, 3) || off(kv_lens, 3))
    return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

int attn_f16_paged_fwd(gemm_f16_plan_t p, int batch, int total_q, int max_q, int q_heads,
                       int kv_heads, int head_dim, const void* Q, const int64_t q_strides[2],
                       const void* Kc, const int64_t kc_strides[3], const void* Vc,
                       const int64_t vc_strides[3], int num_pages, int page_size,
                       const int32_t* block_table, int64_t table_stride, int max_pages,
                       const int32_t* starts, const int32_t* kv_lens, void* O,
                       const int64_t o_strides[2], float scale, int window, int sinks,
                       gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  int rc = attn_f16_paged_validate(batch, total_q, max_q, q_heads, kv_heads, head_dim, Q,
                                         q_strides, Kc, kc_strides, Vc, vc_strides, num_pages,
                                         page_size, block_table, table_stride, max_pages, starts,
                                         kv_lens, O, o_strides, scale, window, sinks);
  if (rc) return rc;
  if (total_q == 0) return GEMM_F16_OK;
  DeviceGuard g(p->device);
  const cudaStream_t st = (cudaStream_t)stream;
  paged::Params prm = {};
  prm.batch = batch;
  prm.total_q = total_q;
  prm.max_q = max_q;
  prm.q_heads = q_heads;
  prm.kv_heads = kv_heads;
  prm.group = q_heads / kv_heads;
  prm.num_pages = num_pages;
  prm.page_size = page_size;
  prm.max_pages = max_pages;
  prm.table = block_table;
  prm.starts = starts;
  prm.kv_lens = kv_lens;
  prm.table_stride = table_stride;
  prm.O = static_cast<__half*>(O);
  prm.o_tok = o_strides[0];
  prm.o_head = o_strides[1];
  // In base 2, and finite: an infinity would make a score of 0 a NaN.  A scale
  // of 0 becomes one whose products with any binary16 scores vanish beside 1,
  // so that a masked score may be an infinity.
  prm.scale_log2 = scale == 0.f ? 1e-30f
                                : std::clamp(scale * 1.4426950408889634f, -FLT_MAX, FLT_MAX);
  prm.masks.window = window;
  prm.masks.sinks = sinks;
  prm.status = p->status_dev;
  prm.timeout_ns = p->timeout_ns;
  prm.fault_unit = p->fault_unit;
  if ((rc = ensure_workspace(p, &prm))) return rc;
  CUtensorMap tmQ, tmK, tmV;
  const int page_rows = page_size & -page_size;   // the largest power of two in it
  const int64_t rows = std::max<int64_t>(1, max_q) * prm.group;   // room for a token at least
  // Requests of up to SMALL_ROWS rows (new tokens x group) are bound by
  // reading the cache and go to the small kernel, with room for the rows
  // that the step's largest has (16, 32 or 64).  Where some may be larger,
  // the small kernel takes those that fit the narrowest form a single token
  // fits, and the large one the others; a step of one request that may be
  // large launches that alone, which takes a request of any size.
  const bool any_large = rows > SMALL_ROWS, any_small = !any_large || batch > 1;
  if (any_small) {
    const int64_t fit = any_large ? prm.group : rows;
    const int n = fit <= 16 ? 16 : (fit <= 32 ? 32 : 64);
    prm.rows = std::min(page_rows, paged::BLOCK_KEYS);
    prm.tile_tokens = n / prm.group;
    prm.zero_rows = 1;
    if ((rc = encode_q(p, &tmQ, Q, total_q, q_heads, q_strides, prm.group, prm.tile_tokens)) ||
        (rc = encode_cache(p, &tmK, Kc, num_pages, page_size, kv_heads, kc_strides, prm.rows)) ||
        (rc = encode_cache(p, &tmV, Vc, num_pages, page_size, kv_heads, vc_strides, prm.rows)))
      return rc;
    const int ctas = p->sm_limit > 0 ? std::min(p->sm_limit, p->num_sms) : p->num_sms;
    using namespace paged::small;
    const Kernel kernel = n == 16 ? paged_small_kernel<16>
                                  : (n == 32 ? paged_small_kernel<32> : paged_small_kernel<64>);
    const int threads = n == 16 ? Cfg<16>::THREADS : (n == 32 ? Cfg<32>::THREADS : Cfg<64>::THREADS);
    const size_t smem = n == 16 ? Cfg<16>::SMEM : (n == 32 ? Cfg<32>::SMEM : Cfg<64>::SMEM);
    const int per_block = merge_rows((int64_t)batch * kv_heads, ctas);
    if ((rc = launch(p, kernel, "launch paged_small_kernel", ctas, threads, smem, st, tmQ, tmK,
                     tmV, prm)) ||
        (rc = launch_merge(n == 16 ? merge_kernel<16>(per_block)
                                   : (n == 32 ? merge_kernel<32>(per_block) : merge_kernel<64>(per_block)),
                           "launch paged_small_merge_kernel", ctas,
                           (int)ceil_div(std::min<int64_t>(n, rows), per_block), MERGE_THREADS, st,
                           prm)))
      return rc;
    prm.skip_tokens = prm.tile_tokens;
  }
  if (any_large) {
    using namespace paged::large;
    const int cta_tokens = CQ / prm.group;
    prm.rows = std::min(page_rows, MAX_ROWS);
    prm.tile_tokens = 2 * cta_tokens;
    prm.zero_rows = !any_small;
    if ((rc = encode_q(p, &tmQ, Q, total_q, q_heads, q_strides, prm.group, cta_tokens)) ||
        (rc = encode_cache(p, &tmK, Kc, num_pages, page_size, kv_heads, kc_strides, prm.rows)) ||
        (rc = encode_cache(p, &tmV, Vc, num_pages, page_size, kv_heads, vc_strides, prm.rows)))
      return rc;
    int pairs = p->paged_pairs;
    if (p->sm_limit > 0) pairs = std::max(1, std::min(pairs, p->sm_limit / 2));
    if ((rc = launch(p, paged_large_kernel, "launch paged_large_kernel", 2 * pairs, NUM_THREADS,
                     SMEM_BYTES, st, tmQ, tmK, tmV, prm)) ||
        (rc = launch_merge(paged_large_merge_kernel, "launch paged_large_merge_kernel", pairs,
                           PART_ROWS / 32, MERGE_THREADS, st, prm)))
      return rc;
  }
  return GEMM_F16_OK;
}

}  // extern "C"
