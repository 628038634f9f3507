// Attention of a serving step's new tokens over a paged key/value cache
// (attn_f16_paged_fwd): argument checks, kernels and entry point.

#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>

#include "host.h"
#include "ptx.cuh"
#include "schedule.h"
#include "common.cuh"
#include "paged_schedule.h"

#include "paged_small.cuh"

using namespace gf16;
using namespace gf16::host;

namespace gf16 {
namespace host {

int paged_plan_init(gemm_f16_plan_s*, const cudaDeviceProp&) {
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
  return GEMM_F16_OK;
}

void paged_plan_release(gemm_f16_plan_s* p) {
  if (p->paged_ws) cudaFree(p->paged_ws);
}

}  // namespace host
}  // namespace gf16

namespace {

constexpr int HEAD_DIM = 256;
constexpr int WARPS = 4;

struct Params {
  int batch, total_q, max_q, q_heads, kv_heads;
  const __half *Q, *Kc, *Vc;
  __half* O;
  int64_t q_st[2], o_st[2], k_st[3], v_st[3];
  int num_pages, page_size, max_pages;
  const int32_t *table, *starts, *kv_lens;
  int64_t table_stride;
  float scale_log2;
  int window, sinks;
  int* status;
  int skip;   // requests with at most this many new tokens are another kernel's
};

__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

// One warp per (token, query head), eight numbers of the head per lane; one
// pass over the visible keys with the running maximum and sum.
__global__ void __launch_bounds__(WARPS * 32) paged_attn_kernel(const Params p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  if (w >= (int64_t)p.total_q * p.q_heads) return;
  const int t = (int)(w / p.q_heads), h = (int)(w - (int64_t)t * p.q_heads);
  __half* out = p.O + t * p.o_st[0] + h * p.o_st[1] + lane * 8;
  // The last request whose first token is not after t.
  int lo = 0, hi = p.batch + 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.starts[mid] <= t) lo = mid; else hi = mid;
  }
  if (lo == p.batch) {
    *reinterpret_cast<uint4*>(out) = make_uint4(0, 0, 0, 0);
    return;
  }
  const int b = lo;
  const int s0 = p.starts[b], s1 = p.starts[b + 1];
  int64_t n = (int64_t)s1 - s0, len = p.kv_lens[b];
  const int64_t room = (int64_t)p.max_pages * p.page_size;
  if (s0 < 0 || n < 0 || n > p.max_q || s1 > p.total_q || len < 0 || len > room) {
    *(volatile int*)p.status = GEMM_F16_ERR_BAD_INDEX;
    len = len < 0 ? 0 : min(len, room);
  }
  if (n <= p.skip) return;
  const int64_t pos = min(len - n + (t - s0), len - 1);
  const int kvh = h / (p.q_heads / p.kv_heads);
  float q[8];
  unpack8(*reinterpret_cast<const uint4*>(p.Q + t * p.q_st[0] + h * p.q_st[1] + lane * 8), q);
  float m = -INFINITY, l = 0.f, acc[8] = {};
  const int64_t first = p.window > 0 ? max((int64_t)0, pos - p.window + 1) : 0;
  for (int64_t j = 0; j <= pos; ++j) {
    if (j < first && j >= p.sinks) j = first;
    const int page = p.table[b * p.table_stride + j / p.page_size];
    const int64_t row = j % p.page_size;
    float k[8] = {}, v[8] = {};
    if (page < 0 || page >= p.num_pages) {
      *(volatile int*)p.status = GEMM_F16_ERR_BAD_INDEX;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(p.Kc + page * p.k_st[0] + row * p.k_st[1] +
                                              kvh * p.k_st[2] + lane * 8), k);
      unpack8(*reinterpret_cast<const uint4*>(p.Vc + page * p.v_st[0] + row * p.v_st[1] +
                                              kvh * p.v_st[2] + lane * 8), v);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s = fmaf(q[i], k[i], s);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale_log2;
    const float mn = fmaxf(m, s);
    const float at = mn == -INFINITY ? 0.f : mn;  // only scores of -inf so far: no weight
    const float a = exp2f(m - at), e = exp2f(s - at);
    m = mn;
    l = l * a + e;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = fmaf(acc[i], a, e * v[i]);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint4 o;
  __half2 r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __floats2half2_rn(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  o.x = *reinterpret_cast<uint32_t*>(&r[0]);
  o.y = *reinterpret_cast<uint32_t*>(&r[1]);
  o.z = *reinterpret_cast<uint32_t*>(&r[2]);
  o.w = *reinterpret_cast<uint32_t*>(&r[3]);
  *reinterpret_cast<uint4*>(out) = o;
}

// Workspace of the attention over a paged cache: a counter per partial slot,
// zero between calls, then the partials' offsets and sums, then their FP32 O.
constexpr int SMALL_ROWS = 64;   // most rows of a request for the small kernel

int ensure_workspace(gemm_f16_plan_s* p, cudaStream_t stream, paged::Params* prm) {
  const size_t slots = 2 * (size_t)p->num_sms;
  const size_t counters = (slots * sizeof(int) + 255) / 256 * 256;
  const size_t ml = slots * SMALL_ROWS * sizeof(float2);
  const size_t bytes = counters + ml + slots * SMALL_ROWS * HEAD_DIM * sizeof(float);
  if (p->paged_ws_bytes < bytes) {
    const int rc = ensure_buffer(&p->paged_ws, &p->paged_ws_bytes, bytes, stream,
                                 "paged attention workspace allocation");
    if (rc) return rc;
    const cudaError_t e = cudaMemsetAsync(p->paged_ws, 0, counters, stream);
    if (e != cudaSuccess) {
      p->paged_ws_bytes = 0;   // set up again by the next call
      return cuda_fail(e, "clear paged attention counters");
    }
  }
  char* ws = static_cast<char*>(p->paged_ws);
  prm->counters = reinterpret_cast<int*>(ws);
  prm->part_ml = reinterpret_cast<float2*>(ws + counters);
  prm->part = reinterpret_cast<float*>(ws + counters + ml);
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

template <int N>
cudaError_t launch_small(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                         const paged::Params& prm, int ctas, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3(paged::small::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = paged::small::Cfg<N>::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged::small::paged_small_kernel<N>, tmQ, tmK, tmV, prm);
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
  const int rc = attn_f16_paged_validate(batch, total_q, max_q, q_heads, kv_heads, head_dim, Q,
                                         q_strides, Kc, kc_strides, Vc, vc_strides, num_pages,
                                         page_size, block_table, table_stride, max_pages, starts,
                                         kv_lens, O, o_strides, scale, window, sinks);
  if (rc) return rc;
  if (total_q == 0) return GEMM_F16_OK;
  DeviceGuard g(p->device);
  Params prm = {};
  prm.batch = batch;
  prm.total_q = total_q;
  prm.max_q = max_q;
  prm.q_heads = q_heads;
  prm.kv_heads = kv_heads;
  prm.Q = static_cast<const __half*>(Q);
  prm.Kc = static_cast<const __half*>(Kc);
  prm.Vc = static_cast<const __half*>(Vc);
  prm.O = static_cast<__half*>(O);
  for (int i = 0; i < 2; ++i) {
    prm.q_st[i] = q_strides[i];
    prm.o_st[i] = o_strides[i];
  }
  for (int i = 0; i < 3; ++i) {
    prm.k_st[i] = kc_strides[i];
    prm.v_st[i] = vc_strides[i];
  }
  prm.num_pages = num_pages;
  prm.page_size = page_size;
  prm.max_pages = max_pages;
  prm.table = block_table;
  prm.table_stride = table_stride;
  prm.starts = starts;
  prm.kv_lens = kv_lens;
  prm.scale_log2 = scale * 1.4426950408889634f;
  prm.window = window;
  prm.sinks = sinks;
  prm.status = p->status_dev;
  const int group = q_heads / kv_heads;
  int sk = 0;   // requests of up to this many tokens go to the small kernel
  {
    const int64_t rows = (int64_t)max_q * group;
    const int N = rows <= 16 ? 16 : (rows <= 32 ? 32 : 64);
    paged::Params sp = {};
    sp.batch = batch;
    sp.total_q = total_q;
    sp.max_q = max_q;
    sp.q_heads = q_heads;
    sp.kv_heads = kv_heads;
    sp.group = group;
    sp.num_pages = num_pages;
    sp.page_size = page_size;
    sp.max_pages = max_pages;
    sp.rows = std::min(page_size & -page_size, paged::BLOCK_KEYS);
    sp.table = block_table;
    sp.starts = starts;
    sp.kv_lens = kv_lens;
    sp.table_stride = table_stride;
    sp.O = static_cast<__half*>(O);
    sp.o_tok = o_strides[0];
    sp.o_head = o_strides[1];
    sp.scale_log2 = prm.scale_log2;
    sp.masks.window = window;
    sp.masks.sinks = sinks;
    sp.tile_tokens = N / group;
    sp.status = p->status_dev;
    sp.timeout_ns = p->timeout_ns;
    sp.fault_unit = p->fault_unit;
    int rc2 = ensure_workspace(p, (cudaStream_t)stream, &sp);
    CUtensorMap tmQ, tmK, tmV;
    if (rc2 || (rc2 = encode_q(p, &tmQ, Q, total_q, q_heads, q_strides, group, sp.tile_tokens)) ||
        (rc2 = encode_cache(p, &tmK, Kc, num_pages, page_size, kv_heads, kc_strides, sp.rows)) ||
        (rc2 = encode_cache(p, &tmV, Vc, num_pages, page_size, kv_heads, vc_strides, sp.rows)))
      return rc2;
    const int ctas = p->sm_limit > 0 ? std::min(p->sm_limit, p->num_sms) : p->num_sms;
    cudaEvent_t t0;
    if ((rc2 = timing_begin(p, (cudaStream_t)stream, &t0))) return rc2;
    const auto fn = N == 16 ? launch_small<16> : (N == 32 ? launch_small<32> : launch_small<64>);
    const cudaError_t le = fn(tmQ, tmK, tmV, sp, ctas, (cudaStream_t)stream);
    rc2 = timing_end(p, (cudaStream_t)stream, t0, le == cudaSuccess);
    GF16_CUDA(le, "launch paged_small_kernel");
    if (rc2) return rc2;
    sk = sp.tile_tokens;
    if (rows <= N) return GEMM_F16_OK;
  }
  prm.skip = sk;
  cudaLaunchConfig_t cfg = {};
  const int64_t blocks = ceil_div((int64_t)total_q * q_heads, WARPS);
  if (blocks > INT32_MAX) return GEMM_F16_ERR_INVALID_ARG;
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3(WARPS * 32, 1, 1);
  cfg.stream = (cudaStream_t)stream;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, paged_attn_kernel, prm), "launch paged_attn_kernel");
  return GEMM_F16_OK;
}

}  // extern "C"
