// Products of a few fp16 rows with matrices of the microscaled 4-bit format:
// the decode product (one matrix) and the two products of an expert layer.
//
//   out[t][n] = sum_k x[t][k] w[n][k],   t < 16
//
// Every code is read once, so the floor is the codes' and scales' bytes; the
// kernel is a stream through shared memory with just enough arithmetic behind
// it. Work is cut into units of 128 rows x 256 k of one matrix (16 KB of
// codes, 2 or 1 KB of scales). The units of a call, in an order in which those
// of one output tile follow one another, are divided evenly over the CTAs, one
// CTA an SM: no wave is left part-filled, whatever the shape.
//
//   warp 16     producer: for each unit the codes as one 2-D box (128-byte
//               rows, 128-byte swizzle), the scale tiles as one copy (they are
//               contiguous along K) and 512 bytes of each x row, all
//               completing on the stage's mbarrier.
//   warps 0-15  eight groups of 16 rows times the two halves of the unit's k.
//               Per 32 k: one word of codes a lane and row (8 codes of its
//               row), 16 bytes of x, two mma.sync.m16n8k16 with the weights
//               as A (16 rows) and x as B (8 tokens). The k within 32 go to
//               the MMA's places in an order of our own, the same for both
//               operands: lane t of a quad holds k 8t .. 8t + 7.
//               E4M3: code times scale is exact in fp16 (6 bits) and is what
//               the MMA sees. E8M0: the scale's range is beyond fp16, so the
//               codes go in as they are and the block's sum (the two MMAs
//               cover just one block of 32) is scaled in fp32.
//   end of tile the halves of k meet in shared memory. A tile whose units lie
//               in several CTAs goes through the workspace: each writes its
//               part, the last to arrive (a counter) adds them in CTA order,
//               so that the result does not depend on who it is.
//
// mma.sync and not tcgen05: with 8 or 16 tokens the arithmetic is far below
// either's rate, and registers take the dequantised A operand without a trip
// through tensor memory.
#pragma once

#include "exq_fp4.cuh"

namespace exq {
namespace fp4s {

static __device__ unsigned g_stream_err;

enum Mode { kGemv = 0, kUp = 1, kDown = 2 };

constexpr int kRows = 128;           // rows of a unit
constexpr int kUnitK = 256;          // k of a unit: 128 bytes of codes a row
constexpr int kConsumers = 16;       // warps
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr int kCodeBytes = kRows * kUnitK / 2;
constexpr int kScaleRoom = 2048;     // 4 tiles (E4M3) or 2 (E8M0)
constexpr int kXStride = kUnitK * 2 + 64;  // x rows 64 bytes apart modulo 128: two rows' quads hit all banks
constexpr int kMaxTokens = 16;
constexpr int kMaxPairs = 256;       // tokens x experts of each
constexpr int kMaxExperts = 512;
constexpr int kSmemMost = 227 * 1024;

// What lies between the two products of an expert, h, as up leaves and down
// reads it: for each (token, expert) and 256 values a piece of the first fp16
// parts, the second ones and the factors of the two halves of 128 (times which
// the sums of the parts are h).
constexpr int kHPiece = kUnitK * 4 + 16;
constexpr int kHStride = kHPiece + 48;     // in shared memory: 64 bytes apart modulo 128, as the x rows

__host__ __device__ constexpr int x_stride(int mode) { return mode == kDown ? kHStride : kXStride; }
__host__ __device__ constexpr int stage_bytes(int mode, int nt) {
  return (kCodeBytes + kScaleRoom + 8 * nt * x_stride(mode) + 1023) / 1024 * 1024;
}
// accumulators of a lane: 4 for each 8 tokens (and matrix)
__host__ __device__ constexpr int accs(int mode, int nt) { return 4 * nt * (mode == kUp ? 2 : 1); }
__host__ __device__ constexpr int meet_bytes(int mode, int nt) { return 2 * 8 * 32 * accs(mode, nt) * 4; }
constexpr int kRest = 10240 + 1024;  // barriers, the experts' tables, alignment
__host__ __device__ constexpr int stages(int mode, int nt) {
  const int n = (kSmemMost - kRest - meet_bytes(mode, nt)) / stage_bytes(mode, nt);
  return n < 8 ? n : 8;
}
__host__ __device__ constexpr int smem_bytes(int mode, int nt) {
  return stages(mode, nt) * stage_bytes(mode, nt) + meet_bytes(mode, nt) + kRest;
}
// floats of one CTA's part of a tile
__host__ __device__ constexpr int part_floats(int mode, int nt) { return 8 * 32 * accs(mode, nt); }

struct Args {
  const uint8_t* sc0;      // scale tiles of the matrix, or of expert 0's gate or down
  const uint8_t* sc1;      // of expert 0's up
  size_t sc_stride;        // from expert to expert
  const uint16_t* x;       // [M, K]; down: h, [pairs, k_units] pieces
  uint16_t* out;           // [M, rows]; up: h, [pairs, h_units] pieces
  const float *f0, *f1, *f2;  // experts' factors of gate, up and down, or NULL
  const int32_t* ids;      // [M, top_k]
  const float* weights;
  unsigned* counters;
  float* part;             // [CTAs][2][part_floats]
  float factor;
  int rows, K, M;
  int row_tiles, k_units, k_tiles, h_units;
  int top_k, n_experts, act;
  int wait_limit, starve;
};

// The experts of a call, the same in every CTA: those that some token chose,
// ascending, with the tokens of each and the place of (expert, token) in ids.
struct Experts {
  int n, pad[3];
  int expert[kMaxPairs];
  unsigned tokens[kMaxPairs];                 // a bit each
  uint8_t place[kMaxPairs][kMaxTokens];       // the first, where an id repeats
  int ids[kMaxPairs];
  float weight[kMaxPairs];                    // by that place: those of an id that repeats are added up
  float most[8][kMaxTokens];                  // up: the groups' largest h
};
static_assert(sizeof(Experts) + 256 <= 10240, "shared memory budget");

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// One warp's 16 rows times 128 k (half kh) of a stage, added to acc.
template <int FMT, int MODE, int NT>
__device__ __forceinline__ void consume(const uint8_t* st, int chunks, unsigned tokens, int rg, int kh, int lane,
                                        float (*acc)[4]) {
  const int g = lane >> 2, t = lane & 3;
  const int r0 = rg * 16 + g;  // and r0 + 8: both are g modulo 8
  const uint8_t* row0 = st + r0 * 128 + 4 * t;
  const uint8_t* sc = st + kCodeBytes;
  const uint8_t* x0 = st + kCodeBytes + kScaleRoom + g * x_stride(MODE) + 16 * t;
  constexpr int kTilesHalf = FMT == EXQ_FP4_E4M3 ? 2 : 1;  // scale tiles of 128 k
  uint32_t sw[2][kTilesHalf];
#pragma unroll
  for (int i = 0; i < kTilesHalf; ++i) {
    const uint8_t* tile = sc + (kh * kTilesHalf + i) * 512;
    sw[0][i] = *reinterpret_cast<const uint32_t*>(tile + fp4_tile_byte(r0));
    sw[1][i] = *reinterpret_cast<const uint32_t*>(tile + fp4_tile_byte(r0 + 8));
  }
  const uint32_t pick = t & 2 ? 0x3232u : 0x1010u;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int cc = 4 * kh + c;
    if (cc >= chunks) break;
    uint32_t w[2], b[NT * (MODE == kDown ? 2 : 1)][4];
    w[0] = *reinterpret_cast<const uint32_t*>(row0 + ((cc ^ g) << 4));
    w[1] = *reinterpret_cast<const uint32_t*>(row0 + 8 * 128 + ((cc ^ g) << 4));
#pragma unroll
    for (int n = 0; n < NT * (MODE == kDown ? 2 : 1); ++n) {
      const int token = 8 * (n % NT) + g;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if ((tokens >> token) & 1u)
        v = *reinterpret_cast<const uint4*>(x0 + n % NT * 8 * x_stride(MODE) + n / NT * kUnitK * 2 + cc * 64);
      b[n][0] = v.x; b[n][1] = v.y; b[n][2] = v.z; b[n][3] = v.w;
    }
    uint32_t a[2][4];  // of the two MMAs: (row g, row g + 8) x (first, second pair of k)
    a[0][0] = e2m1x2_f16<0>(w[0]); a[0][1] = e2m1x2_f16<0>(w[1]);
    a[0][2] = e2m1x2_f16<1>(w[0]); a[0][3] = e2m1x2_f16<1>(w[1]);
    a[1][0] = e2m1x2_f16<2>(w[0]); a[1][1] = e2m1x2_f16<2>(w[1]);
    a[1][2] = e2m1x2_f16<3>(w[0]); a[1][3] = e2m1x2_f16<3>(w[1]);
    if constexpr (FMT == EXQ_FP4_E4M3) {
      // the lane's 8 k lie in one block of 16: quads' first two lanes in the chunk's first, the others in its second
      const uint32_t s0 = __byte_perm(e4m3x2_f16(sw[0][c >> 1] >> (16 * (c & 1))), 0u, pick);
      const uint32_t s1 = __byte_perm(e4m3x2_f16(sw[1][c >> 1] >> (16 * (c & 1))), 0u, pick);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        a[j][0] = hmul2(a[j][0], s0); a[j][1] = hmul2(a[j][1], s1);
        a[j][2] = hmul2(a[j][2], s0); a[j][3] = hmul2(a[j][3], s1);
      }
#pragma unroll
      for (int n = 0; n < NT * (MODE == kDown ? 2 : 1); ++n) {
        mma16816(acc[n % NT], a[0], b[n][0], b[n][1]);
        mma16816(acc[n % NT], a[1], b[n][2], b[n][3]);
      }
    } else {
      const float s0 = e8m0_f32((sw[0][0] >> (8 * c)) & 0xFFu), s1 = e8m0_f32((sw[1][0] >> (8 * c)) & 0xFFu);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816(d, a[0], b[n][0], b[n][1]);
        mma16816(d, a[1], b[n][2], b[n][3]);
        if constexpr (MODE == kDown) {
          mma16816(d, a[0], b[NT + n][0], b[NT + n][1]);
          mma16816(d, a[1], b[NT + n][2], b[NT + n][3]);
        }
        acc[n][0] = fmaf(d[0], s0, acc[n][0]);
        acc[n][1] = fmaf(d[1], s0, acc[n][1]);
        acc[n][2] = fmaf(d[2], s1, acc[n][2]);
        acc[n][3] = fmaf(d[3], s1, acc[n][3]);
      }
    }
  }
}

// The experts' tables, by all threads of the CTA.
__device__ __forceinline__ void find_experts(const Args& a, Experts* e, unsigned* used, bool report) {
  const int tid = threadIdx.x, pairs = a.M * a.top_k;
  if (tid < kMaxExperts / 32) used[tid] = 0u;
  if (tid < kMaxPairs) e->tokens[tid] = 0u;
  const int id = tid < pairs ? __ldcg(a.ids + tid) : -1;
  const float w = tid < pairs ? __ldcg(a.weights + tid) : 0.f;
  if (tid < kMaxPairs) e->ids[tid] = id;
  __syncthreads();
  const bool good = static_cast<unsigned>(id) < static_cast<unsigned>(a.n_experts);
  if (good) atomicOr(&used[id >> 5], 1u << (id & 31));
  if (report && id != -1 && !good) atomicOr(&g_stream_err, kDevErrBadExpert);
  if (tid < kMaxPairs) e->weight[tid] = w;
  __syncthreads();
  if (tid == 0) {
    int n = 0;
    for (int i = 0; i < kMaxExperts / 32; ++i) n += __popc(used[i]);
    e->n = n;
  }
  bool first = good;
  float sum = 0.f;
  if (good) {
    int slot = __popc(used[id >> 5] & ((1u << (id & 31)) - 1u));
    for (int i = 0; i < (id >> 5); ++i) slot += __popc(used[i]);
    e->expert[slot] = id;
    const int t = tid / a.top_k;
    for (int p = t * a.top_k; p < (t + 1) * a.top_k; ++p)
      if (e->ids[p] == id) {
        first = first && p >= tid;
        sum += e->weight[p];
      }
    if (first) {
      e->place[slot][t] = static_cast<uint8_t>(tid);
      atomicOr(&e->tokens[slot], 1u << t);
    }
  }
  __syncthreads();
  if (first) e->weight[tid] = sum;
  __syncthreads();
}

__device__ __forceinline__ float activate(float v, int act) {
  if (act == EXQ_ACT_SILU) return v / (1.f + __expf(-v));
  const float u = 0.7978845608028654f * (v + 0.044715f * v * v * v);
  return 0.5f * v * (1.f + tanhf(u));
}

// The unit list of a call: n units, those of one tile consecutive.
struct Units {
  int tile_units;   // of a tile
  long long n;
};

template <int MODE>
__device__ __forceinline__ Units units_of(const Args& a, int experts) {
  if constexpr (MODE == kGemv) return {a.k_units, static_cast<long long>(a.row_tiles) * a.k_units};
  if constexpr (MODE == kUp) return {a.k_units, static_cast<long long>(experts) * a.row_tiles * a.k_units};
  return {experts * a.k_units, static_cast<long long>(a.row_tiles) * experts * a.k_units};
}

// The CTA that has unit u, of `ctas` that divide n units: CTA b has units
// [b n / ctas, (b + 1) n / ctas).
__device__ __forceinline__ int owner(long long u, long long n, int ctas) {
  return static_cast<int>(((u + 1) * ctas - 1) / n);
}

template <int FMT, int MODE, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    stream_kernel(const __grid_constant__ CUtensorMap m0, const __grid_constant__ CUtensorMap m1,
                  const __grid_constant__ Args a) {
  constexpr int kStages = stages(MODE, NT);
  constexpr int kStageBytes = stage_bytes(MODE, NT);
  constexpr int kParts = MODE == kUp ? 2 : 1;  // matrices of a unit, a stage each
  constexpr int kTilesUnit = kUnitK / fp4_tile_k(FMT);
  constexpr int kAccs = accs(MODE, NT) / 4;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* meet = reinterpret_cast<float4*>(smem + kStages * kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes + meet_bytes(MODE, NT));
  uint64_t* empty = full + kStages;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(empty + kStages);
  volatile int* last = abort_flag + 1;
  unsigned* used = reinterpret_cast<unsigned*>(empty + kStages) + 4;
  Experts* ex = reinterpret_cast<Experts*>(used + kMaxExperts / 32);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), kConsumers);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if constexpr (MODE == kUp) {
    // ids and weights may come from the launch before; the down product may start its own set-up from here
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  }
  int n_experts = 0;
  if constexpr (MODE != kGemv) {
    find_experts(a, ex, used, MODE == kUp && blockIdx.x == 0);
    n_experts = ex->n;
  } else {
    __syncthreads();
  }

  const Units un = units_of<MODE>(a, n_experts);
  if constexpr (MODE == kDown) {
    if (un.n == 0) {  // no token has an expert
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const long long n = static_cast<long long>(a.M) * a.rows;
      for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < n;
           i += static_cast<long long>(gridDim.x) * kThreads)
        a.out[i] = 0;
    }
  }
  const int ctas = static_cast<int>(un.n < gridDim.x ? un.n : gridDim.x);
  if (static_cast<int>(blockIdx.x) >= ctas) return;
  const long long u0 = blockIdx.x * un.n / ctas, u1 = (blockIdx.x + 1) * un.n / ctas;
  const unsigned everyone = (1u << a.M) - 1u;

  if (warp == kConsumers) {
    // ------------------------------------------------------------ producer
    if (a.starve) {  // test hook: a starved producer issues nothing
      if constexpr (MODE == kDown) asm volatile("griddepcontrol.wait;" ::: "memory");
    } else {
      const int n_stages = static_cast<int>(u1 - u0) * kParts;
      int x_from = 0;  // stages whose x rows are still to be issued (down: after the wait)
      bool waited = MODE != kDown;
      int issued = 0;
      auto place = [&](int i, int& kc, int& slot, int& row, int& id) {
        const long long u = u0 + i / kParts;
        const long long q = u / a.k_units;
        kc = static_cast<int>(u - q * a.k_units);
        slot = 0;
        id = 0;
        if constexpr (MODE == kGemv) {
          row = static_cast<int>(q);
        } else if constexpr (MODE == kUp) {
          slot = static_cast<int>(q / a.row_tiles);
          row = static_cast<int>(q) - slot * a.row_tiles;
          id = ex->expert[slot];
        } else {
          row = static_cast<int>(q / n_experts);
          slot = static_cast<int>(q) - row * n_experts;
          id = ex->expert[slot];
        }
      };
      auto issue_x = [&](int i) {
        int kc, slot, row, id;
        place(i, kc, slot, row, id);
        const unsigned tokens = MODE == kGemv ? everyone : ex->tokens[slot];
        if (lane < 8 * NT && ((tokens >> lane) & 1u)) {  // lane: the token
          const uint32_t dst = smem_u32(smem + (i % kStages) * kStageBytes + kCodeBytes + kScaleRoom + lane * x_stride(MODE));
          if constexpr (MODE == kDown)
            bulk_load(dst, a.x + (static_cast<size_t>(ex->place[slot][lane]) * a.k_units + kc) * (kHPiece / 2), kHPiece,
                      smem_u32(&full[i % kStages]));
          else
            bulk_load(dst, a.x + static_cast<size_t>(lane) * a.K + static_cast<size_t>(kc) * kUnitK,
                      min(kUnitK, a.K - kc * kUnitK) * 2, smem_u32(&full[i % kStages]));
        }
      };
      for (int i = 0; i < n_stages; ++i) {
        const int s = i % kStages;
        if (!waited && i == kStages) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          waited = true;
          for (; x_from < i; ++x_from) issue_x(x_from);
        }
        if (!mbar_wait_warp(smem_u32(&empty[s]), ((i / kStages) & 1) ^ 1, abort_flag, a.wait_limit, &g_stream_err)) break;
        int kc, slot, row, id;
        place(i, kc, slot, row, id);
        const int part = i % kParts;
        uint8_t* st = smem + s * kStageBytes;
        const uint32_t bar = smem_u32(&full[s]);
        if (lane == 0) {
          const unsigned tokens = MODE == kGemv ? everyone : ex->tokens[slot];
          const uint32_t xb = __popc(tokens) * (MODE == kDown ? kHPiece : min(kUnitK, a.K - kc * kUnitK) * 2);
          const uint32_t sb = min(kTilesUnit, a.k_tiles - kc * kTilesUnit) * 512;
          mbar_expect_tx(bar, kCodeBytes + sb + xb);
          tma_load_2d(smem_u32(st), part == 0 ? &m0 : &m1, kc * (kUnitK / 2), id * a.rows + row * kRows, bar);
          bulk_load(smem_u32(st + kCodeBytes),
                    (part == 0 ? a.sc0 : a.sc1) + id * a.sc_stride +
                        (static_cast<size_t>(row) * a.k_tiles + kc * kTilesUnit) * 512,
                    sb, bar);
        }
        __syncwarp();
        if (waited) {
          issue_x(i);
          x_from = i + 1;
        }
        issued = i + 1;
      }
      if (!waited) {
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (; x_from < issued; ++x_from) issue_x(x_from);
      }
      // every issued stage's copies land before the CTA may exit
      for (int i = max(0, issued - kStages); i < issued; ++i)
        for (int r = 0; r < a.wait_limit; ++r)
          if (mbar_try_wait(smem_u32(&full[i % kStages]), (i / kStages) & 1)) break;
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int rg = warp & 7, kh = warp >> 3;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  float acc[kAccs][4];       // of the tile
  float run[NT][4];          // down: of the unit, before the factors
  float share[NT][2];        // down: weight and factor of the expert for the lane's tokens
  int slot_of_share = -1;
#pragma unroll
  for (int i = 0; i < kAccs; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) run[i][j] = 0.f;

  int i = 0, tiles_done = 0;
  for (long long u = u0; u < u1; ++u) {
    const long long q = u / a.k_units;
    const int kc = static_cast<int>(u - q * a.k_units);
    int slot = 0, row;
    if constexpr (MODE == kGemv) {
      row = static_cast<int>(q);
    } else if constexpr (MODE == kUp) {
      slot = static_cast<int>(q / a.row_tiles);
      row = static_cast<int>(q) - slot * a.row_tiles;
    } else {
      row = static_cast<int>(q / n_experts);
      slot = static_cast<int>(q) - row * n_experts;
    }
    const unsigned tokens = MODE == kGemv ? everyone : ex->tokens[slot];
    const int chunks = min(8, (a.K - kc * kUnitK) / 32);
#pragma unroll
    for (int part = 0; part < kParts; ++part, ++i) {
      const int s = i % kStages;
      if (mbar_wait_warp(smem_u32(&full[s]), (i / kStages) & 1, abort_flag, a.wait_limit, &g_stream_err))
        consume<FMT, MODE, NT>(smem + s * kStageBytes, chunks, tokens, rg, kh, lane,
                               MODE == kDown ? run : acc + part * NT);
      if constexpr (MODE == kDown) {
        // weight, down's factor and that of h's half, all after the sum of products; an expert's sums go to its own
        // tokens only: a NaN of its weights reaches no other
        if (slot != slot_of_share) {
          slot_of_share = slot;
          const float fd = a.f2 ? __ldg(a.f2 + ex->expert[slot]) : 1.f;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const int token = 8 * n + t2 + c;
              share[n][c] = (tokens >> token) & 1u ? ex->weight[ex->place[slot][token]] * fd : 0.f;
            }
        }
        const uint8_t* x = smem + s * kStageBytes + kCodeBytes + kScaleRoom + kUnitK * 4 + 4 * kh;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int token = 8 * n + t2 + c;
            if (4 * kh < chunks && ((tokens >> token) & 1u)) {
              const float f = share[n][c] * *reinterpret_cast<const float*>(x + token * kHStride);
              acc[n][c] = fmaf(run[n][c], f, acc[n][c]);
              acc[n][2 + c] = fmaf(run[n][2 + c], f, acc[n][2 + c]);
            }
            run[n][c] = run[n][2 + c] = 0.f;
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&empty[s]));
    }
    const bool tile_ends = (u + 1) % un.tile_units == 0 || u + 1 == u1;
    if (!tile_ends) continue;

    // the two halves of k: the second's sums through shared memory (two areas in turn, one barrier a tile)
    float4* area = meet + (tiles_done & 1) * 8 * 32 * kAccs;
    ++tiles_done;
    if (kh == 1) {
#pragma unroll
      for (int n = 0; n < kAccs; ++n)
        area[(rg * kAccs + n) * 32 + lane] = make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
    if (kh == 0) {
#pragma unroll
      for (int n = 0; n < kAccs; ++n) {
        const float4 v = area[(rg * kAccs + n) * 32 + lane];
        acc[n][0] += v.x; acc[n][1] += v.y; acc[n][2] += v.z; acc[n][3] += v.w;
      }
      const long long tile = u / un.tile_units;
      const long long first = tile * un.tile_units, end = first + un.tile_units;
      const int b0 = owner(first, un.n, ctas), b1 = owner(end - 1, un.n, ctas);
      bool mine = true;  // this CTA writes the result
      if (b0 != b1) {
        auto part_of = [&](int b) {  // a CTA's tile that began before it is its part 0
          return reinterpret_cast<float4*>(a.part) +
                 (static_cast<size_t>(b) * 2 + (first < b * un.n / ctas ? 0 : 1)) * (part_floats(MODE, NT) / 4);
        };
        float4* p = part_of(blockIdx.x);
#pragma unroll
        for (int n = 0; n < kAccs; ++n)
          __stcg(p + (rg * kAccs + n) * 32 + lane, make_float4(acc[n][0], acc[n][1], acc[n][2], acc[n][3]));
        __threadfence();
        asm volatile("bar.sync 2, 256;" ::: "memory");
        if (threadIdx.x == 0) {
          int is_last = 0;
          if (!*abort_flag) {
            const unsigned before = atomicAdd(a.counters + tile, 1u);
            is_last = before == static_cast<unsigned>(b1 - b0);
            if (is_last) a.counters[tile] = 0u;
          }
          __threadfence();
          *last = is_last;
        }
        asm volatile("bar.sync 2, 256;" ::: "memory");
        mine = *last != 0;
        if (mine) {
#pragma unroll
          for (int n = 0; n < kAccs; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
          for (int b = b0; b <= b1; ++b) {
            const float4* o = part_of(b);
#pragma unroll
            for (int n = 0; n < kAccs; ++n) {
              const float4 v = __ldcg(o + (rg * kAccs + n) * 32 + lane);
              acc[n][0] += v.x; acc[n][1] += v.y; acc[n][2] += v.z; acc[n][3] += v.w;
            }
          }
        }
      }
      // lane's results: rows r and r + 8, tokens t2 and t2 + 1 of each eight
      const int r = row * kRows + rg * 16 + g;
      if constexpr (MODE == kUp) {
        if (mine) {
          const int id = ex->expert[slot];
          const float fg = a.f0 ? __ldg(a.f0 + id) : 1.f, fu = a.f1 ? __ldg(a.f1 + id) : 1.f;
          // h of the lane's two rows, and the largest of the tile for each token
          float most[NT][2];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                acc[n][2 * j + c] = activate(acc[n][2 * j + c] * fg, a.act) * (acc[NT + n][2 * j + c] * fu);
              float m = fmaxf(r < a.rows ? fabsf(acc[n][c]) : 0.f, r + 8 < a.rows ? fabsf(acc[n][2 + c]) : 0.f);
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
              if (g == 0) ex->most[rg][8 * n + t2 + c] = m;
            }
          asm volatile("bar.sync 2, 256;" ::: "memory");
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              most[n][c] = 0.f;
#pragma unroll
              for (int w = 0; w < 8; ++w) most[n][c] = fmaxf(most[n][c], ex->most[w][8 * n + t2 + c]);
            }
          if (!*abort_flag) {
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const int token = 8 * n + t2 + c;
                if (!((tokens >> token) & 1u)) continue;
                // a power of two that brings the tile's largest to 1 .. 2 (exact; what is not finite stays)
                const int e = min(max(static_cast<int>(__float_as_uint(most[n][c]) >> 23), 1), 253);
                const float up = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
                uint16_t* h = a.out + (static_cast<size_t>(ex->place[slot][token]) * a.h_units + (row >> 1)) * (kHPiece / 2);
                if (g == 0 && rg == 0) reinterpret_cast<float*>(h + kUnitK * 2)[row & 1] = __uint_as_float(static_cast<uint32_t>(e) << 23);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  if (r + 8 * j >= a.rows) continue;
                  const float v = acc[n][2 * j + c] * up;
                  const __half hi = __float2half_rn(v);
                  const float rest = v - __half2float(hi);
                  const int at = (row & 1) * kRows + rg * 16 + g + 8 * j;
                  h[at] = __half_as_ushort(hi);
                  h[kUnitK + at] = __half_as_ushort(__float2half_rn(isfinite(rest) ? rest : 0.f));
                }
              }
          }
        }
      } else if (mine && !*abort_flag) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int token = 8 * n + t2 + c;
            if (token >= a.M) continue;
            uint16_t* y = a.out + static_cast<size_t>(token) * a.rows;
            if (r < a.rows) y[r] = __half_as_ushort(__float2half_rn(acc[n][c] * a.factor));
            if (r + 8 < a.rows) y[r + 8] = __half_as_ushort(__float2half_rn(acc[n][2 + c] * a.factor));
          }
      }
    }
#pragma unroll
    for (int n = 0; n < kAccs; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;
  }
}

}  // namespace fp4s
}  // namespace exq
