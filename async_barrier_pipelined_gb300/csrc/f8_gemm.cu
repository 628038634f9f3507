// Products of 8-bit floating-point matrices with block scales (gemm_f8_run):
// argument checks, the choice of kernel, tensor maps and launches.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdio>

#include "host.h"

#include "f8_large.cuh"
#include "f8_small.cuh"

using namespace gf16;
using namespace gf16::host;

namespace {

using LargeKernel = void (*)(const CUtensorMap, const CUtensorMap, const f8::Params);

struct SmallKernel {
  LargeKernel fn;
  uint32_t smem, smem_experts;
  int ctas;      // per SM
};
template <int NT>
SmallKernel small_kernel() {
  using C = f8::small::Cfg<NT>;
  return {f8::small::f8_small_kernel<NT>, C::SMEM, C::SMEM_EXPERTS, C::CTAS};
}
SmallKernel small_kernel(int nt) {
  return nt == 16 ? small_kernel<16>() : nt == 32 ? small_kernel<32>() : small_kernel<64>();
}

constexpr int MAX_SIZE = 0x7fffffff - 1023;   // coordinates of a last tile stay in 31 bits

// What a call launches.
struct Choice {
  bool small;
  int nt, split;          // small: rows of a tile, CTAs that share its K blocks
  int tail_tiles, parts;  // large: cut tiles and ranges of K blocks
};

int pairs_of(const gemm_f16_plan_s* p) {
  return p->sm_limit > 0 ? std::max(1, std::min(p->f8_pairs, p->sm_limit / 2)) : p->f8_pairs;
}
// CTAs of the small kernel at once.  Nothing places two of them on one SM, so
// that with a limit there is one for each SM that may be used.
int64_t small_room(const gemm_f16_plan_s* p, int ctas_per_sm) {
  return p->sm_limit > 0 ? std::min(p->sm_limit, p->num_sms) : (int64_t)p->num_sms * ctas_per_sm;
}

Choice choose(const gemm_f16_plan_s* p, int form, int M, int N, int K, int experts,
              bool a_transposed) {
  Choice c = {};
  c.parts = 1;
  const int kblocks = (int)ceil_div(K, f8::BLOCK);
  // Rows of a tile of the small kernel: those of the call, or of an expert on
  // the average if all of M, the room, is filled.  (How many rows there are is
  // known on the device alone: maps that fill experts up to a multiple of 128 come
  // here with 128 rows an expert, however few of them are tokens'.)  Up to 64 of
  // them: 64 x 4096 x 4096 takes 12.8 us there and 14.1
  // in the large kernel, 64 experts of 64 rows (1024 x 2048) 40.6 and 44.1; with a
  // tile of 128 rows 128 x 4096 x 4096 took 18.8 and 16 experts of 96 rows (4096 x
  // 2048) 102, in the large kernel 16.4 and 43.
  const int64_t rows = form == GEMM_F8_BY_ROWS ? ceil_div(M, experts) : M;
  if (form != GEMM_F8_BY_INNER && !a_transposed && rows <= 64) {
    c.small = true;
    c.nt = rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    // As many CTAs for a tile as keep all resident (CTAs per SM) and leave each
    // two K blocks or more.
    const int64_t tiles_n = ceil_div(N, f8::small::CN);
    const int64_t units = form == GEMM_F8_BY_ROWS
                              ? std::min<int64_t>(M, experts) * tiles_n
                              : ceil_div(M, c.nt) * tiles_n;
    const int64_t room = small_room(p, small_kernel(c.nt).ctas);
    c.split = 1;
    while (c.split < f8::small::MAX_SPLIT && 2 * c.split * units <= room && 4 * c.split <= kblocks)
      c.split *= 2;
    return c;
  }
  if (form == GEMM_F8_DENSE) {
    const int64_t tiles = ceil_div(M, f8::large::PM) * ceil_div(N, f8::large::PN);
    const int pairs = pairs_of(p);
    const int rem = (int)(tiles % pairs);
    // Parts for a last wave of at most half the pairs, each of four K blocks or
    // more, where they save sixteen blocks (0.4 to 0.65 us each): the parts' 256 KB,
    // written and read, and a launch cost 7 us.  129 x 4096 x 4096: 16.5 us with
    // four parts, 19.1 without; 1000 x 1024 x 2048 (12 blocks saved) 14.2 and 12.5.
    if (rem > 0) {
      const int parts = std::min({pairs / rem, kblocks / 4, f8::large::MAX_PARTS});
      if (parts > 1 && kblocks - ceil_div(kblocks, parts) >= 16) {
        c.tail_tiles = rem;
        c.parts = parts;
      }
    }
  }
  return c;
}

// CTAs of a call's kernel and of the one that joins cut tiles (0: none).
struct Grids {
  int product, join;
};
Grids grids(const gemm_f16_plan_s* p, const Choice& c, int form, int M, int N, int experts) {
  Grids g = {};
  if (c.small) {
    const int64_t tiles_n = ceil_div(N, f8::small::CN);
    const int64_t most = form == GEMM_F8_BY_ROWS ? (ceil_div(M, c.nt) + std::min(M, experts)) * tiles_n
                                                 : ceil_div(M, c.nt) * tiles_n;
    const int64_t room = std::max<int64_t>(1, small_room(p, small_kernel(c.nt).ctas) / c.split);
    g.product = (int)std::min(most, room) * c.split;
    return g;
  }
  const int64_t tiles_n = ceil_div(N, f8::large::PN), tiles = ceil_div(M, f8::large::PM) * tiles_n;
  const int64_t most = form == GEMM_F8_BY_ROWS
                           ? (ceil_div(M, f8::large::PM) + std::min(M, experts)) * tiles_n
                       : form == GEMM_F8_BY_INNER ? tiles * experts
                                                  : tiles + (int64_t)c.tail_tiles * (c.parts - 1);
  g.product = 2 * (int)std::min<int64_t>(most, pairs_of(p));
  g.join = c.tail_tiles * 2 * f8::large::PROMOTE_WARPS;
  if (p->sm_limit > 0) g.join = std::min(g.join, p->sm_limit);
  return g;
}

size_t workspace_bytes(const Choice& c) {
  if (c.small || c.parts == 1) return 0;
  return (size_t)c.tail_tiles * c.parts * f8::large::PART_FLOATS * 4;
}

bool off(const void* p, uintptr_t mask) { return ((uintptr_t)p & mask) != 0; }

// Tensor map of an operand: `outer` x `inner` numbers (outer: M or N; inner: K),
// boxes of 128 bytes by `rows`.
int encode_operand(gemm_f16_plan_s* p, CUtensorMap* map, const gemm_f8_operand& x, bool mn_major,
                   int outer, int inner, int matrices, int rows) {
  const uint64_t key[8] = {(uint64_t)(uintptr_t)x.data,
                           ((uint64_t)(uint32_t)outer << 32) | (uint32_t)inner,
                           (uint64_t)x.ld, (uint64_t)x.batch, (uint64_t)(uint32_t)matrices,
                           ((uint64_t)mn_major << 32) | (uint32_t)rows, 0, 0x4638000000000000ull};
  if (tmap_lookup(p, key, map)) return GEMM_F16_OK;
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail_msg("cuTensorMapEncodeTiled entry point not available");
  const cuuint64_t dims[3] = {(cuuint64_t)(mn_major ? outer : inner),
                              (cuuint64_t)(mn_major ? inner : outer), (cuuint64_t)matrices};
  const cuuint64_t ld = dims[1] > 1 ? (cuuint64_t)x.ld : (cuuint64_t)ceil_div(dims[0], 16) * 16;
  const cuuint64_t strides[2] = {ld, matrices > 1 ? (cuuint64_t)x.batch : ld * dims[1]};
  const cuuint32_t box[3] = {128, (cuuint32_t)(mn_major ? 128 : rows), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(x.data), dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    std::snprintf(g_last_cuda_error, sizeof(g_last_cuda_error),
                  "cuTensorMapEncodeTiled (8-bit operand) failed (CUresult %d)", (int)r);
    return GEMM_F16_ERR_CUDA;
  }
  tmap_remember(p, key, *map);
  return GEMM_F16_OK;
}

int launch(gemm_f16_plan_s* p, LargeKernel kernel, const char* what, int ctas, int cluster,
           int threads, size_t smem, cudaStream_t stream, const CUtensorMap& tmA,
           const CUtensorMap& tmB, const f8::Params& prm) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;   // 0: the kernel's own
  cudaEvent_t t0;
  int rc = timing_begin(p, stream, &t0);
  if (rc) return rc;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, prm);
  rc = timing_end(p, stream, t0, le == cudaSuccess);
  GF16_CUDA(le, what);
  return rc;
}

int check_operand(const gemm_f8_operand* x, int rows, int cols, int matrices) {
  if (!x) return GEMM_F16_ERR_INVALID_ARG;
  if (x->format != GEMM_F8_E4M3 && x->format != GEMM_F8_E5M2) return GEMM_F16_ERR_INVALID_ARG;
  if ((x->transposed | x->tiles) & ~1) return GEMM_F16_ERR_INVALID_ARG;
  const int64_t stored = x->transposed ? rows : cols, lines = x->transposed ? cols : rows;
  if (rows > 0 && cols > 0 && (!x->data || !x->scales)) return GEMM_F16_ERR_INVALID_ARG;
  if (lines > 1 && (x->ld < stored || x->ld >= ((int64_t)1 << 38))) return GEMM_F16_ERR_INVALID_ARG;
  if (matrices > 1 && (x->batch < 0 || x->batch >= ((int64_t)1 << 39))) return GEMM_F16_ERR_INVALID_ARG;
  if (x->s_outer < 0 || x->s_inner < 0 || x->s_batch < 0) return GEMM_F16_ERR_INVALID_ARG;
  if (off(x->data, 15) || (lines > 1 && (x->ld & 15)) || (matrices > 1 && (x->batch & 15)) ||
      off(x->scales, 3))
    return GEMM_F16_ERR_MISALIGNED;
  return GEMM_F16_OK;
}

}  // namespace

namespace gf16 {
namespace host {

int f8_plan_init(gemm_f16_plan_s* p, const cudaDeviceProp& prop) {
  const LargeKernel large[2] = {f8::large::f8_large_kernel<false>, f8::large::f8_large_kernel<true>};
  for (LargeKernel k : large)
    GF16_CUDA(cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)f8::large::SMEM_BYTES),
              "cudaFuncSetAttribute(8-bit product smem)");
  for (int nt = 16; nt <= 64; nt *= 2) {
    const SmallKernel k = small_kernel(nt);
    GF16_CUDA(cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (int)k.smem_experts),
              "cudaFuncSetAttribute(8-bit product smem)");
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(prop.multiProcessorCount / 2 * 2), 1, 1);
  cfg.blockDim = dim3(f8::large::NUM_THREADS, 1, 1);
  cfg.dynamicSmemBytes = f8::large::SMEM_BYTES;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  GF16_CUDA(cudaOccupancyMaxActiveClusters(&clusters, large[0], &cfg),
            "cudaOccupancyMaxActiveClusters(8-bit product)");
  p->f8_pairs = std::max(clusters, 1);
  return GEMM_F16_OK;
}

}  // namespace host
}  // namespace gf16

extern "C" {

int gemm_f8_validate(int form, int M, int N, int K, int experts, const int32_t* starts,
                     const gemm_f8_operand* A, const gemm_f8_operand* B, const void* C,
                     int64_t ldc, int64_t c_batch, int type, int accumulate) {
  if (form < GEMM_F8_DENSE || form > GEMM_F8_BY_INNER) return GEMM_F16_ERR_INVALID_ARG;
  if (M < 0 || N < 0 || K < 0 || M > MAX_SIZE || N > MAX_SIZE || K > MAX_SIZE)
    return GEMM_F16_ERR_INVALID_ARG;
  if (type < GEMM_F8_F16 || type > GEMM_F8_F32) return GEMM_F16_ERR_INVALID_ARG;
  if (accumulate != 0 && (accumulate != 1 || type != GEMM_F8_F32)) return GEMM_F16_ERR_INVALID_ARG;
  const bool by = form != GEMM_F8_DENSE;
  if (by && (experts < 1 || experts > f8::MAX_EXPERTS || !starts)) return GEMM_F16_ERR_INVALID_ARG;
  int rc = check_operand(A, M, K, 1);
  if (!rc) rc = check_operand(B, K, N, form == GEMM_F8_BY_ROWS ? experts : 1);
  if (rc) return rc;
  if (form == GEMM_F8_BY_ROWS && A->transposed) return GEMM_F16_ERR_INVALID_ARG;
  if (M > 0 && N > 0) {
    if (!C || (M > 1 && ldc < N) || ldc >= ((int64_t)1 << 38)) return GEMM_F16_ERR_INVALID_ARG;
    if (form == GEMM_F8_BY_INNER && (c_batch < 0 || c_batch >= ((int64_t)1 << 39)))
      return GEMM_F16_ERR_INVALID_ARG;
    if (off(C, type == GEMM_F8_F32 ? 3 : 1) || (by && off(starts, 3))) return GEMM_F16_ERR_MISALIGNED;
  }
  // Work units are counted in 31 bits.
  const int64_t tiles_n = ceil_div(N, 128);
  const int64_t tiles = form == GEMM_F8_BY_ROWS
                            ? (ceil_div(M, 16) + experts) * tiles_n
                            : ceil_div(M, 128) * tiles_n * (by ? experts : 1);
  if (tiles > MAX_SIZE / 8) return GEMM_F16_ERR_INVALID_ARG;
  return GEMM_F16_OK;
}

size_t gemm_f8_workspace(gemm_f16_plan_t p, int form, int M, int N, int K, int experts,
                         int a_transposed) {
  if (!p || M < 1 || N < 1 || K < 1 || (form != GEMM_F8_DENSE && experts < 1)) return 0;
  return workspace_bytes(choose(p, form, M, N, K, experts, a_transposed != 0));
}

int gemm_f8_run_choice(int form, int M, int N, int K, int experts, int a_transposed, int num_sms,
                       int max_pairs, int sm_limit, int info[4]) {
  if (!info || form < GEMM_F8_DENSE || form > GEMM_F8_BY_INNER || M < 1 || N < 1 || K < 1 ||
      M > MAX_SIZE || N > MAX_SIZE || K > MAX_SIZE || num_sms < 1 || max_pairs < 1 || sm_limit < 0 ||
      (form != GEMM_F8_DENSE && (experts < 1 || experts > f8::MAX_EXPERTS)))
    return GEMM_F16_ERR_INVALID_ARG;
  gemm_f16_plan_s p;
  p.num_sms = num_sms;
  p.f8_pairs = max_pairs;
  p.sm_limit = sm_limit;
  const Choice c = choose(&p, form, M, N, K, experts, a_transposed != 0);
  const Grids g = grids(&p, c, form, M, N, experts);
  info[0] = c.small ? 1 : 2;
  info[1] = c.small ? c.split : c.parts;
  info[2] = g.product;
  info[3] = g.join;
  return GEMM_F16_OK;
}

int gemm_f8_run(gemm_f16_plan_t p, int form, int M, int N, int K, int experts,
                const int32_t* starts, const gemm_f8_operand* A, const gemm_f8_operand* B, void* C,
                int64_t ldc, int64_t c_batch, int type, int accumulate, void* workspace,
                size_t workspace_size, gemm_f16_stream_t stream) {
  if (!p) return GEMM_F16_ERR_INVALID_ARG;
  int rc = gemm_f8_validate(form, M, N, K, experts, starts, A, B, C, ldc, c_batch, type, accumulate);
  if (rc) return rc;
  if (M == 0 || N == 0) return GEMM_F16_OK;
  DeviceGuard g(p->device);
  const cudaStream_t st = (cudaStream_t)stream;
  const bool by = form != GEMM_F8_DENSE;
  const int size = type == GEMM_F8_F32 ? 4 : 2;
  if (K == 0) {   // nothing to add up: every matrix of C is 0
    if (accumulate) return GEMM_F16_OK;
    for (int e = 0; e < (form == GEMM_F8_BY_INNER ? experts : 1); ++e)
      GF16_CUDA(cudaMemset2DAsync(static_cast<char*>(C) + (int64_t)e * c_batch * size,
                                  (size_t)(M > 1 ? ldc : N) * size, 0, (size_t)N * size, (size_t)M, st),
                "cudaMemset2DAsync");
    return GEMM_F16_OK;
  }
  const Choice c = choose(p, form, M, N, K, experts, A->transposed != 0);
  const size_t need = workspace_bytes(c);
  if (need > 0) {
    if (!workspace || workspace_size < need) return GEMM_F16_ERR_SCRATCH_TOO_SMALL;
    if (off(workspace, 15)) return GEMM_F16_ERR_MISALIGNED;
  }
  f8::Params prm = {};
  prm.form = form;
  prm.M = M;
  prm.N = N;
  prm.K = K;
  prm.experts = by ? experts : 1;
  prm.starts = starts;
  prm.a_mn = A->transposed;
  prm.b_mn = !B->transposed;
  prm.sa = A->scales;
  prm.sa_outer = A->s_outer;
  prm.sa_inner = A->s_inner;
  prm.sa_shift = A->tiles ? 7 : 0;
  prm.sb = B->scales;
  prm.sb_outer = B->s_outer;
  prm.sb_inner = B->s_inner;
  prm.sb_batch = B->s_batch;
  prm.sb_shift = B->tiles ? 7 : 0;
  prm.C = C;
  prm.ldc = M > 1 ? ldc : N;
  prm.c_batch = c_batch;
  prm.type = type;
  prm.accumulate = accumulate;
  prm.vec = !off(C, 15) && (M == 1 || ldc * size % 16 == 0) &&
            (form != GEMM_F8_BY_INNER || experts == 1 || c_batch * size % 16 == 0);
  prm.kblocks = (int)ceil_div(K, f8::BLOCK);
  prm.parts = c.parts;
  prm.status = p->status_dev;
  prm.timeout_ns = p->timeout_ns;
  prm.fault_unit = p->fault_unit;
  const int b_matrices = form == GEMM_F8_BY_ROWS ? experts : 1;
  const Grids grid = grids(p, c, form, M, N, experts);
  CUtensorMap tmA, tmB;
  if (c.small) {
    using namespace f8::small;
    const SmallKernel k = small_kernel(c.nt);
    if ((rc = encode_operand(p, &tmA, *A, false, M, K, 1, c.nt)) ||
        (rc = encode_operand(p, &tmB, *B, prm.b_mn, N, K, b_matrices, CN)))
      return rc;
    prm.tiles_m = (int)ceil_div(M, c.nt);
    prm.tiles_n = (int)ceil_div(N, CN);
    prm.units = prm.tiles_m * prm.tiles_n;
    // The MMA's rows are B's: formats and majors change places.
    prm.idesc = f8::idesc_f8(B->format, A->format, prm.b_mn, false, CN, c.nt);
    return launch(p, k.fn, "launch f8_small_kernel", grid.product, c.split, NUM_THREADS,
                  by ? k.smem_experts : k.smem, st, tmA, tmB, prm);
  }
  using namespace f8::large;
  if ((rc = encode_operand(p, &tmA, *A, prm.a_mn, M, K, 1, CM)) ||
      (rc = encode_operand(p, &tmB, *B, prm.b_mn, N, K, b_matrices, PN / 2)))
    return rc;
  prm.tiles_m = (int)ceil_div(M, PM);
  prm.tiles_n = (int)ceil_div(N, PN);
  prm.idesc = f8::idesc_f8(A->format, B->format, prm.a_mn, prm.b_mn, PM, PN);
  const int64_t tiles = (int64_t)prm.tiles_m * prm.tiles_n;
  prm.full_units = (int)tiles - c.tail_tiles;
  prm.units = form == GEMM_F8_BY_INNER ? (int)tiles * experts
                                       : prm.full_units + c.tail_tiles * c.parts;
  prm.cut_units = c.tail_tiles * c.parts;
  prm.ws = static_cast<float*>(workspace);
  rc = launch(p, prm.sb_shift ? f8_large_kernel<false> : f8_large_kernel<true>,
              "launch f8_large_kernel", grid.product, 0, NUM_THREADS, SMEM_BYTES, st, tmA, tmB, prm);
  if (rc || c.tail_tiles == 0) return rc;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid.join, 1, 1);
  prm.join_pieces = c.tail_tiles * 2 * PROMOTE_WARPS;
  cfg.blockDim = dim3(JOIN_THREADS, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute pdl;
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &pdl;
  cfg.numAttrs = 1;
  GF16_CUDA(cudaLaunchKernelEx(&cfg, prm.sb_shift ? f8_join_kernel<false> : f8_join_kernel<true>, prm),
            "launch f8_join_kernel");
  return GEMM_F16_OK;
}

}  // extern "C"
