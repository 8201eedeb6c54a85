// Product of two matrices of the microscaled 4-bit format on the block-scaled
// tcgen05 tensor cores:
//   y[m][n] = fp16(f sum_k a[m][k] w[n][k]),   f = a.factor * w.factor.
//
// A CTA computes 128 rows x 256 columns of y, 256 k at a time:
//   warp 0     TMA producer: the codes of both operands (128-byte rows,
//              128-byte swizzle) and their scale tiles, as they lie in memory
//              (512 bytes for 128 rows x 4 blocks: the tensor memory's order).
//   warp 1     one lane copies the scale tiles to tensor memory (tcgen05.cp)
//              and issues tcgen05.mma.block_scale, K = 64, in that order: the
//              two run in the order of issue, so that one place in tensor
//              memory serves every stage. fp32 sums in tensor memory.
//   warps 2-5  epilogue: a lane is a row, 32 columns at a time.
// With few output tiles K is split over CTAs; fp32 partial sums go to the
// workspace and a second kernel adds them in order.
#include <algorithm>
#include <cstring>

#include "exq_fp4.cuh"

namespace exq {
namespace {

__device__ unsigned g_fp4_gemm_err;

constexpr int BM = 128;
constexpr int BN = 256;
constexpr int BK = 256;  // k of a stage: four MMAs
constexpr int kStages = 4;
constexpr int kThreads = 6 * 32;

constexpr int kABytes = BM * BK / 2;
constexpr int kBBytes = BN * BK / 2;
constexpr int kScaleTiles = 2048;  // the scale tiles of 128 rows x 256 k: 4 (E4M3) or 2 (E8M0)
constexpr int kOffB = kABytes;
constexpr int kOffSA = kOffB + kBBytes;
constexpr int kOffSB = kOffSA + kScaleTiles;
constexpr int kStageBytes = kOffSB + 2 * kScaleTiles;
static_assert(kStageBytes % 1024 == 0, "stage alignment");
constexpr int kSmemBytes = kStages * kStageBytes + 1024 + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory budget");

constexpr uint32_t kTmemSA = BN;        // 4 columns a tile
constexpr uint32_t kTmemSB = BN + 16;   // 8 columns a tile of 256 rows
constexpr uint32_t kTmemCols = 512;

constexpr int kMaxSplit = 8;
constexpr int kMinUnits = 4;  // units of 256 k in a split, at least

struct Args {
  const uint8_t *sa, *sb;
  uint16_t* y;
  float* part;      // [split, M, N] where split > 1
  float factor;
  int M, N, K;
  int a_tiles, b_tiles;  // tiles of 128 rows
  int k_tiles;           // scale tiles along K
  int k_units, units_per;
  int split;
  int wait_limit, starve;
};

// shared-memory descriptor: K-major, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t codes_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

// of a scale tile: no swizzle, 16-byte rows, 8-row groups 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFF) >> 4) | (static_cast<uint64_t>(128 >> 4) << 32) | (1ull << 46);
}

// instruction descriptor of the block-scaled kinds: e2m1 operands, K-major
__device__ __forceinline__ uint32_t idesc_for(int fmt, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         ((fmt == EXQ_FP4_E8M0 ? 1u : 0u) << 23) | (static_cast<uint32_t>(BM >> 4) << 24);
}

template <int FMT>
__device__ __forceinline__ void mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                           uint32_t accumulate) {
  if constexpr (FMT == EXQ_FP4_E4M3)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(accumulate) : "memory");
}

// a scale tile (32 rows of 16 bytes) to 4 columns of tensor memory, in all four lane quarters
__device__ __forceinline__ void copy_scales(uint32_t tmem, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(desc) : "memory");
}

__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int FMT>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_kernel(const __grid_constant__ CUtensorMap ma, const __grid_constant__ CUtensorMap mb,
                const __grid_constant__ Args p) {
  constexpr int kTilesUnit = BK / fp4_tile_k(FMT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* done = empty + kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tile = blockIdx.x, n_tile = blockIdx.y;
  const int m0 = m_tile * BM, n0 = n_tile * BN;
  const int u0 = blockIdx.z * p.units_per, n_iter = min(p.k_units, u0 + p.units_per) - u0;  // >= 1
  const int n_mma = min(BN, (p.N - n0 + 15) & ~15);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(done), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && !p.starve) {
      int issued = 0;
      for (int i = 0; i < n_iter; ++i) {
        const int s = i % kStages, u = u0 + i;
        if (!mbar_wait(smem_u32(&empty[s]), ((i / kStages) & 1) ^ 1, abort_flag, p.wait_limit, &g_fp4_gemm_err)) break;
        uint8_t* st = smem + s * kStageBytes;
        const uint32_t bar = smem_u32(&full[s]);
        const int b_parts = min(2, p.b_tiles - 2 * n_tile);
        const uint32_t sbytes = min(kTilesUnit, p.k_tiles - u * kTilesUnit) * 512;
        mbar_expect_tx(bar, kABytes + kBBytes + (1 + b_parts) * sbytes);
        tma_load_2d(smem_u32(st), &ma, u * (BK / 2), m0, bar);
        tma_load_2d(smem_u32(st + kOffB), &mb, u * (BK / 2), n0, bar);
        const size_t along = static_cast<size_t>(u) * kTilesUnit;
        bulk_load(smem_u32(st + kOffSA), p.sa + (static_cast<size_t>(m_tile) * p.k_tiles + along) * 512, sbytes, bar);
        for (int h = 0; h < b_parts; ++h)
          bulk_load(smem_u32(st + kOffSB + h * kScaleTiles),
                    p.sb + (static_cast<size_t>(2 * n_tile + h) * p.k_tiles + along) * 512, sbytes, bar);
        issued = i + 1;
      }
      // every issued stage's copies land before the CTA may exit
      for (int i = max(0, issued - kStages); i < issued; ++i)
        for (int r = 0; r < p.wait_limit; ++r)
          if (mbar_try_wait(smem_u32(&full[i % kStages]), (i / kStages) & 1)) break;
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one();
    const uint32_t idesc = idesc_for(FMT, n_mma);
    for (int i = 0; i < n_iter; ++i) {
      const int s = i % kStages;
      if (!mbar_wait_warp(smem_u32(&full[s]), (i / kStages) & 1, abort_flag, p.wait_limit, &g_fp4_gemm_err)) break;
      tc_fence_after();
      const uint32_t st = smem_u32(smem) + s * kStageBytes;
      const int n_k = min(4, (p.K - (u0 + i) * BK + 63) / 64);  // MMAs with k of the matrices
      if (leader) {
#pragma unroll
        for (int j = 0; j < kTilesUnit; ++j) {
          copy_scales(tmem + kTmemSA + 4 * j, scale_desc(st + kOffSA + j * 512));
          copy_scales(tmem + kTmemSB + 8 * j, scale_desc(st + kOffSB + j * 512));
          copy_scales(tmem + kTmemSB + 8 * j + 4, scale_desc(st + kOffSB + kScaleTiles + j * 512));
        }
        const uint64_t ad = codes_desc(st), bd = codes_desc(st + kOffB);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 64 k: 32 bytes of a row
          if (j >= n_k) break;
          if constexpr (FMT == EXQ_FP4_E4M3) {
            mma_scaled<FMT>(tmem, ad + 2 * j, bd + 2 * j, idesc, tmem + kTmemSA + 4 * j, tmem + kTmemSB + 8 * j,
                            (i | j) != 0);
          } else {  // two scales of the tile's four: byte 0 or 2 of each word
            const uint32_t id = (j & 1) ? idesc | (2u << 4) | (2u << 29) : idesc;
            mma_scaled<FMT>(tmem, ad + 2 * j, bd + 2 * j, id, tmem + kTmemSA + 4 * (j >> 1), tmem + kTmemSB + 8 * (j >> 1),
                            (i | j) != 0);
          }
        }
        commit(smem_u32(&empty[s]));
      }
      __syncwarp();
    }
    if (leader) commit(smem_u32(done));
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue
    if (mbar_wait_warp(smem_u32(done), 0, abort_flag, p.wait_limit, &g_fp4_gemm_err) && !*abort_flag) {
      tc_fence_after();
      const int quarter = warp & 3;
      const int m = m0 + quarter * 32 + lane;
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        if (n0 + c >= p.N) break;
        uint32_t r[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + c, r);
        if (m >= p.M) continue;
        if (p.split == 1) {
          uint16_t* dst = p.y + static_cast<size_t>(m) * p.N + n0 + c;
#pragma unroll
          for (int j = 0; j < 32; j += 8) {
            if (n0 + c + j >= p.N) break;
            uint4 o;
            o.x = pack_half2(__uint_as_float(r[j]) * p.factor, __uint_as_float(r[j + 1]) * p.factor);
            o.y = pack_half2(__uint_as_float(r[j + 2]) * p.factor, __uint_as_float(r[j + 3]) * p.factor);
            o.z = pack_half2(__uint_as_float(r[j + 4]) * p.factor, __uint_as_float(r[j + 5]) * p.factor);
            o.w = pack_half2(__uint_as_float(r[j + 6]) * p.factor, __uint_as_float(r[j + 7]) * p.factor);
            *reinterpret_cast<uint4*>(dst + j) = o;
          }
        } else {
          float* dst = p.part + (static_cast<size_t>(blockIdx.z) * p.M + m) * p.N + n0 + c;
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            if (n0 + c + j >= p.N) break;
            *reinterpret_cast<uint4*>(dst + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// y = fp16(f * sum over the splits of K, in order)
__global__ void __launch_bounds__(256) join_kernel(const float* __restrict__ part, uint16_t* __restrict__ y, long long mn,
                                                   int split, float factor) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x * 8;
  for (long long e = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) * 8; e < mn; e += stride) {
    float acc[8] = {};
    for (int z = 0; z < split; ++z) {
      const float4* q = reinterpret_cast<const float4*>(part + z * mn + e);
      const float4 u = __ldcg(q), v = __ldcg(q + 1);
      acc[0] += u.x; acc[1] += u.y; acc[2] += u.z; acc[3] += u.w;
      acc[4] += v.x; acc[5] += v.y; acc[6] += v.z; acc[7] += v.w;
    }
    *reinterpret_cast<uint4*>(y + e) =
        make_uint4(pack_half2(acc[0] * factor, acc[1] * factor), pack_half2(acc[2] * factor, acc[3] * factor),
                   pack_half2(acc[4] * factor, acc[5] * factor), pack_half2(acc[6] * factor, acc[7] * factor));
  }
}

int div_up(int a, int b) { return (a + b - 1) / b; }

struct Plan {
  int split, units_per;
};

// Fewer output tiles than half the SMs: K is split over as many CTAs as fill
// them, at most kMaxSplit, each of at least kMinUnits units; none is empty.
Plan plan_for(int M, int N, int K, int sms) {
  const long long tiles = static_cast<long long>(div_up(M, BM)) * div_up(N, BN);
  const int units = div_up(K, BK);
  int s = 1;
  if (tiles * 2 <= sms) s = std::min(std::min(kMaxSplit, static_cast<int>(sms / tiles)), units / kMinUnits);
  if (s < 1) s = 1;
  const int per = div_up(units, s);
  return {div_up(units, per), per};
}

}  // namespace

size_t fp4_gemm_workspace_bytes(const exq_fp4_matrix& a, const exq_fp4_matrix& w, int sms) {
  const Plan plan = plan_for(a.rows, w.rows, a.K, sms);
  return plan.split > 1 ? static_cast<size_t>(plan.split) * a.rows * w.rows * 4 : 0;
}

exq_status launch_fp4_gemm(const exq_fp4_matrix& a, const exq_fp4_matrix& w, uint16_t* y, void* workspace, size_t,
                           int sms, int device, cudaStream_t stream) {
  CUtensorMap ma, mb;
  if (!encode_2d(&ma, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, a.K / 2, a.rows, a.K / 2, BK / 2, BM,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&mb, CU_TENSOR_MAP_DATA_TYPE_UINT8, w.codes, w.K / 2, w.rows, w.K / 2, BK / 2, BN,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_SWIZZLE_128B))
    return EXQ_ERR_CUDA;
  const Plan plan = plan_for(a.rows, w.rows, a.K, sms);
  Args p{};
  p.sa = a.scales;
  p.sb = w.scales;
  p.y = y;
  p.part = static_cast<float*>(workspace);
  p.factor = a.factor * w.factor;
  p.M = a.rows;
  p.N = w.rows;
  p.K = a.K;
  p.a_tiles = div_up(a.rows, 128);
  p.b_tiles = div_up(w.rows, 128);
  p.k_tiles = div_up(a.K, fp4_tile_k(a.format));
  p.k_units = div_up(a.K, BK);
  p.units_per = plan.units_per;
  p.split = plan.split;
  const int starve = testing_starve_rounds();
  p.wait_limit = starve > 0 ? starve : kFp4WaitLimit;
  p.starve = starve > 0 ? 1 : 0;

  auto fn = a.format == EXQ_FP4_E4M3 ? gemm_kernel<EXQ_FP4_E4M3> : gemm_kernel<EXQ_FP4_E8M0>;
  static PerDevice attr[2];
  if (!attr[a.format == EXQ_FP4_E4M3].once(device, [&] {
        return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) == cudaSuccess;
      }))
    return EXQ_ERR_CUDA;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(div_up(p.M, BM), div_up(p.N, BN), plan.split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  if (cudaLaunchKernelEx(&cfg, fn, ma, mb, p) != cudaSuccess) return EXQ_ERR_CUDA;
  if (plan.split == 1) return EXQ_OK;

  const long long mn = static_cast<long long>(p.M) * p.N;
  cudaLaunchConfig_t join{};
  join.gridDim = dim3(static_cast<unsigned>(std::min<long long>((mn / 8 + 255) / 256, 8LL * sms)));
  join.blockDim = dim3(256);
  join.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  join.attrs = at;
  join.numAttrs = 1;
  return cudaLaunchKernelEx(&join, join_kernel, static_cast<const float*>(p.part), y, mn, plan.split, p.factor) == cudaSuccess
             ? EXQ_OK
             : EXQ_ERR_CUDA;
}

unsigned take_fp4_gemm_errors(cudaStream_t stream) {
  unsigned v = 0, zero = 0;
  if (cudaMemcpyFromSymbolAsync(&v, g_fp4_gemm_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream) != cudaSuccess) return ~0u;
  if (cudaMemcpyToSymbolAsync(g_fp4_gemm_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream) != cudaSuccess) return ~0u;
  if (cudaStreamSynchronize(stream) != cudaSuccess) return ~0u;
  return v;
}

}  // namespace exq
