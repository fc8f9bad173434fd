// The weight gradient of a linear layer from the 8-bit checkpoint of its input:
//
//   dW[o][i] = sum_t dy[t][o] x[t][i]     (+ dW)
//
// on the tcgen05 tensor cores.  A checkpoint's values are bf16 numbers, so that the tensor
// cores take them as they are; products are exact in fp32 and sums are fp32.
//
// x is first loaded into the workspace in bf16, where L2 mostly keeps it.  (Converting it in the
// product's own pipeline reads fewer bytes, but every 256 columns of dy convert all of x
// again: 8192 x 9728 x 2560 took 327 us so, of which 300 us remained without any MMA; it takes
// 236 us as it is, 1.73 PFLOP/s, of which the load is 11 us.  Called without a pause it meets the
// power limit: 264 us at 1770 MHz instead of 2070, and a library's bf16 product 239 instead of 203.  For 2560
// columns of dy and 9728 of x, whose 159 MB L2 does not hold, it takes 275 us, of which the load is 39.)
//
// Bound by the tensor cores and what feeds them: with static operands, no waits and no stores
// the same MMAs take 171 us, the loads without MMAs 214 us (15 TB/s from L2), and both 225 us.
//
// Both operands have the sum's index t outside (their rows are tokens) and are read MN-major.
// A pair of CTAs on two SMs computes a 256 x 256 tile of dW with one
// tcgen05.mma.cta_group::2 (M = N = 256); each CTA holds 128 rows of the tile (dy's columns)
// and one 128-wide half of x.  A stage is 64 tokens.  Warps of a CTA:
//   0      TMA producer, onto the leader's barrier
//   1      tcgen05.mma issuer (the leader's)
//   4-11   sums: TMEM to fp32 registers and, after a tile's last stage, to dW
// The tensor cores cut off what an accumulation cannot hold, always towards zero: 512 of them
// (8192 tokens) leave terms of one sign 2.1e-5 of their sum low in the mean, and terms of both
// signs 4.3e-6 of the mean |dW| off.  So an accumulator takes kChunkSteps stages only (64
// accumulations), and is then added to registers, rounding to nearest, while the next stages
// are summed into the other accumulator: 1.06e-6 and 2.5e-7.
//
// fp32 gradients are split into three bf16 parts (8 bits of the significand each) by a pass of
// its own, and the sum runs over the parts, the smallest first.  The parts add up to the value,
// but for what lies under bf16's smallest number, 2^-133: below 2^-110 the third part is cut there.
// The same pass copies bf16 gradients whose rows a TMA cannot read (16-byte boundaries).
//
// Where a matrix has at most half as many tiles as there are pairs, the tokens are divided among
// several pairs, whose fp32 sums are added in a fixed order by a last pass (plan_of).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "checkpoint.h"
#include "device.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "muon.h"
#include "rows.cuh"
#include "tensor_map.h"

namespace muon {
namespace {

constexpr int kTile = 256;          // rows and columns of a tile of dW
constexpr int kTokens = 64;         // tokens of a stage
constexpr int kGradThreads = 384;
constexpr int kGradStages = 6;
constexpr int kChunkSteps = 16;     // stages that one accumulator takes
constexpr uint32_t kChunk = kTokens * 128;          // 64 tokens of 64 bf16 columns
constexpr uint32_t kOperand = 2 * kChunk;           // a CTA's half of an operand
constexpr int kSummers = 8;                         // warps
constexpr int kTurn = 32 * 33;                      // floats of a warp's 32 x 32 block, to be turned
constexpr size_t kGradSmem = kGradStages * 2 * kOperand + kSummers * kTurn * 4 + 1024;
static_assert(kGradSmem <= 232448 - 512, "shared memory of one CTA");
constexpr uint32_t kGradTmem = 512;

struct GradArgs {
  CUtensorMap dy;         // [parts][tokens][outs] bf16, box 64 x 64
  CUtensorMap x;          // [tokens][cols] bf16, the same box
  int32_t cols, outs;
  int32_t parts, steps;   // bf16 parts of dy, 64-token steps of one
  int32_t tiles_n, tiles, splits, split_steps;
  void* out;              // dW, or the splits' sums [splits][outs][stride] fp32
  int64_t stride, split_stride;
  int32_t bf16, accumulate;
};

// Adds 32 lanes x 8 consecutive columns of Tensor Memory to the lanes' registers.
__device__ __forceinline__ void tmem_add8(uint32_t taddr, float (&v)[128], int at) {
  uint32_t r[8];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int j = 0; j < 8; ++j) v[at + j] += __uint_as_float(r[j]);
}

struct Unit {
  int m0, n0, split, kb0, kb1;
};
__device__ __forceinline__ Unit unit_of(const GradArgs& a, int u) {
  Unit r;
  r.split = u / a.tiles;
  const int t = u - r.split * a.tiles;
  r.m0 = t / a.tiles_n * kTile;
  r.n0 = t % a.tiles_n * kTile;
  r.kb0 = r.split * a.split_steps;
  r.kb1 = min(r.kb0 + a.split_steps, a.parts * a.steps);
  return r;
}

// A column of a turned block, `rows` elements, to dW: 16 rows' loads before their stores.
template <typename T>
__device__ __forceinline__ void add_rows(T* p, int64_t stride, int accumulate, const float* turn, int rows) {
#pragma unroll 1
  for (int r = 0; r < rows; r += 16) {
    float y[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = accumulate && r + i < rows ? Vec<T>::load(p + (r + i) * stride) : 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (r + i < rows) Vec<T>::store(p + (r + i) * stride, y[i] + turn[(r + i) * 33]);
  }
}

// A warp's 32 rows x 128 columns of dW from (row0, col), of which lane l has row l; poison, 0 or
// NaN, is added.
//
// Rows of fp32 on 32-byte boundaries that are only written go out as they are, whole sectors
// a lane.  Others are turned in shared memory, 32 columns at a time, so that a warp's accesses
// are to one row (2005 x 1537 fp32, added to: 91 us row by lane, 30 us so).
__device__ __forceinline__ void store_block(const GradArgs& a, int split, int64_t row0, int col, const float (&s)[128],
                                            float poison, float* turn, int lane) {
  const int64_t at = split * a.split_stride + row0 * a.stride + col;
  float* const out = reinterpret_cast<float*>(a.out) + at;
  if (!a.bf16 && !a.accumulate && (reinterpret_cast<uint64_t>(out) & 31) == 0 && a.stride % 8 == 0 && col + 128 <= a.cols) {
    float* const p = out + lane * a.stride;
    if (row0 + lane < a.outs) {
#pragma unroll
      for (int k = 0; k < 128; k += 8)
        asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + k), "f"(s[k] + poison),
                     "f"(s[k + 1] + poison), "f"(s[k + 2] + poison), "f"(s[k + 3] + poison), "f"(s[k + 4] + poison),
                     "f"(s[k + 5] + poison), "f"(s[k + 6] + poison), "f"(s[k + 7] + poison)
                     : "memory");
    }
    return;
  }
  const int rows = (int)min((int64_t)32, a.outs - row0);
#pragma unroll
  for (int c = 0; c < 128; c += 32) {
    if (col + c >= a.cols) break;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 32; ++j) turn[lane * 33 + j] = s[c + j] + poison;
    __syncwarp();
    if (col + c + lane >= a.cols) continue;
    if (a.bf16) add_rows(reinterpret_cast<__nv_bfloat16*>(a.out) + at + c + lane, a.stride, a.accumulate, turn + lane, rows);
    else add_rows(out + c + lane, a.stride, a.accumulate, turn + lane, rows);
  }
  __syncwarp();
}

__global__ void __launch_bounds__(kGradThreads, 1) weight_grad_kernel(const __grid_constant__ GradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ __align__(8) uint64_t full_bar[kGradStages], empty_bar[kGradStages];
  __shared__ __align__(8) uint64_t tfull_bar[2], tempty_bar[2], drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, units = a.tiles * a.splits;
  volatile int* abort_p = &abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kGradStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull_bar[i], 1);
      mbar_init(&tempty_bar[i], 2 * kSummers);
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&a.dy);
    tma_prefetch_desc(&a.x);
  }
  if (warp == 1) {
    tmem_alloc<2>(&tmem_slot, kGradTmem);
    tmem_relinquish<2>();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // barriers of both CTAs exist before any remote signal
  tc_fence_after();
  griddep_launch_dependents();
  griddep_wait();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    // ---- operands ----
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    const uint32_t lead = mapa_shared(&full_bar[0], 0);
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit t = unit_of(a, u);
      int part = a.parts - 1 - t.kb0 / a.steps, step = t.kb0 % a.steps;  // the smallest part first
      for (int kb = t.kb0; kb < t.kb1; ++kb) {
        const bool got = mbar_wait(&empty_bar[stage], phase ^ 1u, abort_p, nullptr);
        if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
        if (lane == 0) {
          uint8_t* sa = smem + (size_t)stage * 2 * kOperand;
          if (leader) mbar_arrive_expect_tx(&full_bar[stage], 4 * kOperand);
          const uint32_t bar = lead + stage * 8;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            tma_load_3d_pair(sa + h * kChunk, &a.dy, bar, t.m0 + rank * 128 + h * 64, step * kTokens, part);
            tma_load_3d_pair(sa + kOperand + h * kChunk, &a.x, bar, t.n0 + rank * 128 + h * 64, step * kTokens, 0);
          }
        }
        __syncwarp();
        if (++step == a.steps) {
          step = 0;
          --part;
        }
        if (++stage == kGradStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (*abort_p && leader && lane == 0) {
      // loads already issued land before the CTA exits (bounded)
      for (int s = 0; s < kGradStages; ++s)
        (void)mbar_wait(&full_bar[s], phase ^ (s < stage ? 0u : 1u), nullptr, nullptr, 100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      // ---- tensor cores ----
      const uint32_t idesc = make_idesc(1u, kTile, kTile, 1u, 1u);
      // 64-column chunks kChunk bytes apart, 8-token groups 1024; the address field counts 16 bytes
      const uint64_t operand0 = smem_desc_sw128(smem_u32(smem), kChunk, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true, ready = false;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit t = unit_of(a, u);
        for (int c0 = t.kb0; c0 < t.kb1; c0 += kChunkSteps) {
          const int c1 = min(c0 + kChunkSteps, t.kb1);
          const bool free_acc = mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_p, nullptr);
          if (!__all_sync(0xffffffffu, free_acc)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * kTile);
          for (int kb = c0; kb < c1; ++kb) {
            if (!ready) {
              const bool got = mbar_wait(&full_bar[stage], phase, abort_p, nullptr);
              if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
            }
            const uint64_t at = operand0 + (uint32_t)stage * (2 * kOperand >> 4);
            uint64_t* const empty = &empty_bar[stage];
            if (++stage == kGradStages) { stage = 0; phase ^= 1u; }
            // whether the next stage has landed is asked before this one's MMAs are issued: the
            // tensor core's queue is too short to cover the answer's latency (8192 x 9728 x 2560:
            // 245 us without, 237 us with it)
            ready = __all_sync(0xffffffffu, mbar_test_wait(&full_bar[stage], phase));
            if (lane == 0) {
#pragma unroll
              for (int kk = 0; kk < kTokens / 16; ++kk)
                mma<false, 2>(d, at + kk * (16 * 128 >> 4), at + ((kOperand >> 4) + kk * (16 * 128 >> 4)), idesc,
                              (kb > c0 || kk > 0) ? 1u : 0u);
              mma_commit_multicast<2>(empty, 3);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (lane == 0) mma_commit_multicast<2>(&tfull_bar[acc], 3);
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      if (lane == 0) {  // every MMA has completed before TMEM is freed
        mma_commit<2>(&drain_bar);
        (void)mbar_wait(&drain_bar, 0u, nullptr, nullptr);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---- sums ----
    const int quad = warp & 3, half = (warp - 4) >> 2;
    float* const turn = reinterpret_cast<float*>(smem + kGradStages * 2 * kOperand) + (warp - 4) * kTurn;
    const uint32_t lead = mapa_shared(&tempty_bar[0], 0);
    const uint32_t from = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)(half * (kTile / 2));
    int acc = 0;
    uint32_t acc_phase = 0;
    for (int u = pair; u < units; u += pairs) {
      const Unit t = unit_of(a, u);
      float sum[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.f;
      bool ok = true;
      for (int c0 = t.kb0; c0 < t.kb1; c0 += kChunkSteps) {
        const bool got = mbar_wait(&tfull_bar[acc], acc_phase, abort_p, nullptr);
        ok = __all_sync(0xffffffffu, got) && ok;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 16; ++c) tmem_add8(from + (uint32_t)(acc * kTile + c * 8), sum, c * 8);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(lead + acc * 8);
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
      }
      // where a wait ran out, no stale values pass for a gradient
      const float poison = ok ? 0.f : NAN;
      const int64_t row0 = (int64_t)t.m0 + rank * 128 + quad * 32;
      const int col = t.n0 + half * (kTile / 2);
      if (row0 < a.outs && col < a.cols) store_block(a, t.split, row0, col, sum, poison, turn, lane);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA frees Tensor Memory or exits while the pair's signals may still reach it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<2>(tmem, kGradTmem);
  }
}

// dy as `parts` bf16 matrices [parts][tokens][ld]: a copy, or the three parts of fp32 values,
// each cut off at 8 bits of what the ones before it leave (cutting cannot overflow), and at
// 2^-133.  It runs
// beside the load of x before it, and ends after it, so that the product waits for both.
constexpr int kPartThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kPartThreads) parts_kernel(const T* dy, int64_t stride, int64_t tokens, int64_t outs,
                                                             int64_t ld, __nv_bfloat16* out) {
  griddep_launch_dependents();
  const int64_t per = ld / 8, items = tokens * per;
  for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < items; i += (int64_t)gridDim.x * kPartThreads) {
    const int64_t t = i / per, c = (i - t * per) * 8;
    const T* p = dy + t * stride + c;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = c + k < outs ? Vec<T>::load(p + k) : 0.f;
    uint4* to = reinterpret_cast<uint4*>(out + t * ld + c);
    if constexpr (sizeof(T) == 2) {
      *to = Vec<__nv_bfloat16>::pack(v);
    } else {
      uint32_t h[3][8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float rest = v[k];
        const bool finite = fabsf(rest) < INFINITY;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          const uint32_t bits = __float_as_uint(rest) & 0xFFFF0000u;
          h[part][k] = finite ? bits >> 16 : part ? 0u : rest != rest ? 0x7FC0u : bits >> 16;
          rest -= __uint_as_float(bits);
        }
      }
#pragma unroll
      for (int part = 0; part < 3; ++part)
        to[part * (tokens * ld / 8)] =
            make_uint4(h[part][0] | h[part][1] << 16, h[part][2] | h[part][3] << 16, h[part][4] | h[part][5] << 16,
                       h[part][6] | h[part][7] << 16);
    }
  }
  griddep_wait();
}

// dW (+)= the splits' sums, in their order.
constexpr int kJoinThreads = 256;
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const float* sums, int64_t ld, int64_t split_stride, int splits,
                                                            T* out, int64_t stride, int64_t outs, int64_t cols,
                                                            int accumulate) {
  griddep_wait();
  const int64_t per = ld / 4, items = outs * per;
  for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < items; i += (int64_t)gridDim.x * kJoinThreads) {
    const int64_t r = i / per, c = (i - r * per) * 4;
    const float4* p = reinterpret_cast<const float4*>(sums + r * ld + c);
    float4 s = __ldcg(p);
    for (int k = 1; k < splits; ++k) {
      const float4 x = __ldcg(p + k * (split_stride / 4));
      s = make_float4(s.x + x.x, s.y + x.y, s.z + x.z, s.w + x.w);
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    T* q = out + r * stride + c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < cols) Vec<T>::store(q + k, accumulate ? Vec<T>::load(q + k) + v[k] : v[k]);
  }
}

// dW of no tokens.
template <typename T>
__global__ void __launch_bounds__(kJoinThreads) zero_kernel(T* out, int64_t stride, int64_t outs, int64_t cols) {
  const int64_t items = outs * cols;
  for (int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x; i < items; i += (int64_t)gridDim.x * kJoinThreads)
    Vec<T>::store(out + i / cols * stride + i % cols, 0.f);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
constexpr int kPairs = 76;  // of SMs on the device this is built for: the division of the tokens goes by it

struct GradPlan {
  int64_t tiles_m, tiles_n, steps, splits, split_steps;
  int parts;        // of dy; 0: read as it lies
  int64_t ld, x_ld; // of the parts, and of x in bf16
  int64_t sum_ld;   // of the splits' sums
  size_t x_bytes, parts_bytes, bytes;
};

// The tokens are divided by as many pairs as a tile can have.  8192 tokens, bf16 to fp32, us on the
// device with (1, 2, 4) parts: 8 tiles 54, 35, 27 (23 with the 9 that they get), 16 tiles 54, 37, 29,
// 38 tiles 56, 42, 46.  Above half the pairs more units than pairs would start a second round: 40 tiles
// 56, 62, 56, 48 tiles 56, 64, 58, 160 tiles 146, 149, 162; these stay whole, and 36 pairs idle
// beside 40 tiles, 68 in the last of three rounds of 160.
// A part is four steps at least: 1024 tokens of 2 tiles 12.9 us with one, two or four, 14.8 with
// eight; 512 tokens of 16 tiles 16.9, 16.9, 15.6, 15.0.
GradPlan plan_of(int64_t tokens, int64_t cols, int64_t outs, const void* dy, int64_t dy_stride, int32_t dtype) {
  GradPlan p = {};
  p.tiles_m = (outs + kTile - 1) / kTile;
  p.tiles_n = (cols + kTile - 1) / kTile;
  if (dtype == MUON_DTYPE_F32) p.parts = 3;
  else p.parts = aligned(dy, 16) && dy_stride % 8 == 0 ? 0 : 1;
  const int64_t passes = p.parts > 1 ? p.parts : 1;
  p.steps = (tokens + kTokens - 1) / kTokens;
  p.ld = (outs + 7) / 8 * 8;
  p.x_ld = (cols + 7) / 8 * 8;
  p.x_bytes = ((size_t)tokens * p.x_ld * 2 + 255) / 256 * 256;
  if (p.parts) p.parts_bytes = ((size_t)p.parts * tokens * p.ld * 2 + 255) / 256 * 256;
  const int64_t all = passes * p.steps, tiles = p.tiles_m * p.tiles_n;
  int64_t splits = tiles < kPairs ? kPairs / tiles : 1;
  if (splits > all / 4) splits = all / 4;
  if (splits < 1) splits = 1;
  p.split_steps = (all + splits - 1) / splits;
  p.splits = all ? (all + p.split_steps - 1) / p.split_steps : 1;
  p.sum_ld = (cols + 3) / 4 * 4;
  p.bytes = p.x_bytes + p.parts_bytes + (p.splits > 1 ? (size_t)p.splits * outs * p.sum_ld * 4 : 0);
  return p;
}

int32_t check_grad_args(const muon_checkpoint* c, const void* dy, int64_t dy_stride, int32_t dy_dtype, int64_t outs) {
  if (!c) return invalid("checkpoint is NULL");
  if (c->rows < 0 || c->rows > (1ll << 31) - 1 - kTokens) return invalid("rows must be in [0, 2^31 - 64)");
  if (c->cols < 1 || c->cols > (1ll << 30)) return invalid("cols must be in [1, 2^30]");
  if (outs < 1 || outs > (1ll << 30)) return invalid("outs must be in [1, 2^30]");
  if (dy_dtype != MUON_DTYPE_F32 && dy_dtype != MUON_DTYPE_BF16) return invalid("unknown dtype of dy");
  if (dy_stride != 0 && (dy_stride < outs || dy_stride > (1ll << 36))) return invalid("dy_stride must be 0 or at least outs");
  if (!aligned(dy, dy_dtype == MUON_DTYPE_BF16 ? 2 : 4)) return invalid("dy is not aligned to its type");
  return MUON_OK;
}

int grid_of(int64_t items, int threads, int sms) {
  const int64_t want = (items + threads - 1) / threads, most = 8ll * sms;
  return (int)(want < 1 ? 1 : want < most ? want : most);
}

template <typename T>
cudaError_t launch_join(const GradPlan& p, const float* sums, void* dw, int64_t stride, int64_t outs, int64_t cols,
                        int accumulate, int sms, cudaStream_t s) {
  return launch(join_kernel<T>, grid_of(outs * (p.sum_ld / 4), kJoinThreads, sms), kJoinThreads, 0, s, 1, true, sums,
                p.sum_ld, outs * p.sum_ld, (int)p.splits, static_cast<T*>(dw), stride, outs, cols, accumulate);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_weight_grad_workspace_bytes(const muon_checkpoint* checkpoint, const void* dy, int64_t dy_stride,
                                             int32_t dy_dtype, int64_t outs, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  const int32_t st = check_grad_args(checkpoint, dy, dy_stride, dy_dtype, outs);
  if (st != MUON_OK) return st;
  *bytes = plan_of(checkpoint->rows, checkpoint->cols, outs, dy, dy_stride ? dy_stride : outs, dy_dtype).bytes;
  return MUON_OK;
}

muon_status muon_checkpoint_weight_grad(const muon_checkpoint* checkpoint, const void* dy, int64_t dy_stride,
                                        int32_t dy_dtype, int64_t outs, void* dw, int64_t dw_stride, int32_t dw_dtype,
                                        int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_grad_args(checkpoint, dy, dy_stride, dy_dtype, outs);
  if (st != MUON_OK) return st;
  const int64_t rows = checkpoint->rows, cols = checkpoint->cols;
  if (rows > 0 && (!checkpoint->data || !aligned(checkpoint->data, 16)))
    return invalid("checkpoint data is NULL or not 16-byte aligned");
  if (rows > 0 && !dy) return invalid("dy is NULL");
  if (dw_dtype != MUON_DTYPE_F32 && dw_dtype != MUON_DTYPE_BF16) return invalid("unknown dtype of dw");
  if (!dw || !aligned(dw, dw_dtype == MUON_DTYPE_BF16 ? 2 : 4)) return invalid("dw is NULL or not aligned to its type");
  if (dw_stride != 0 && (dw_stride < cols || dw_stride > (1ll << 36))) return invalid("dw_stride must be 0 or at least cols");
  if (accumulate != 0 && accumulate != 1) return invalid("accumulate must be 0 or 1");
  const int64_t stride = dy_stride ? dy_stride : outs;
  const GradPlan p = plan_of(rows, cols, outs, dy, stride, dy_dtype);
  if (p.tiles_m * p.tiles_n * p.splits > (1ll << 31) - 1) return set_error(MUON_ERR_UNSUPPORTED, "more than 2^31 tiles");
  if ((int64_t)(p.parts > 1 ? p.parts : 1) * p.steps > (1ll << 31) - 1) return set_error(MUON_ERR_UNSUPPORTED, "too many tokens");
  if (p.bytes > 0 && (st = check_workspace(workspace, workspace_bytes, p.bytes)) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  const bool bf16_out = dw_dtype == MUON_DTYPE_BF16;
  const int64_t out_stride = dw_stride ? dw_stride : cols;
  if (rows == 0) {
    if (accumulate) return MUON_OK;
    const int grid = grid_of(outs * cols, kJoinThreads, sms);
    e = bf16_out ? launch(zero_kernel<__nv_bfloat16>, grid, kJoinThreads, 0, s, 1, false, static_cast<__nv_bfloat16*>(dw), out_stride, outs, cols)
                 : launch(zero_kernel<float>, grid, kJoinThreads, 0, s, 1, false, static_cast<float*>(dw), out_stride, outs, cols);
    return e == cudaSuccess ? MUON_OK : cuda_error(e);
  }
  GradArgs a = {};
  uint8_t* const space = static_cast<uint8_t*>(workspace);
  if ((e = launch_checkpoint_load(checkpoint, space, p.x_ld, s)) != cudaSuccess) return cuda_error(e);
  const void* operand = dy;
  int64_t ld = stride, count = 1;
  if (p.parts) {
    __nv_bfloat16* parts = reinterpret_cast<__nv_bfloat16*>(space + p.x_bytes);
    const int grid = grid_of(rows * (p.ld / 8), kPartThreads, sms);
    e = dy_dtype == MUON_DTYPE_BF16
            ? launch(parts_kernel<__nv_bfloat16>, grid, kPartThreads, 0, s, 1, true, static_cast<const __nv_bfloat16*>(dy), stride, rows, outs, p.ld, parts)
            : launch(parts_kernel<float>, grid, kPartThreads, 0, s, 1, true, static_cast<const float*>(dy), stride, rows, outs, p.ld, parts);
    if (e != cudaSuccess) return cuda_error(e);
    operand = parts;
    ld = p.ld;
    count = p.parts;
  }
  if (!encode_tensor_map(&a.dy, const_cast<void*>(operand), outs, rows, count, ld, 64, kTokens) ||
      !encode_tensor_map(&a.x, space, cols, rows, 1, p.x_ld, 64, kTokens))
    return set_error(MUON_ERR_CUDA, "cuTensorMapEncodeTiled rejected a tensor map");
  a.cols = (int32_t)cols;
  a.outs = (int32_t)outs;
  a.parts = (int32_t)count;
  a.steps = (int32_t)p.steps;
  a.tiles_n = (int32_t)p.tiles_n;
  a.tiles = (int32_t)(p.tiles_m * p.tiles_n);
  a.splits = (int32_t)p.splits;
  a.split_steps = (int32_t)p.split_steps;
  float* sums = nullptr;
  if (p.splits > 1) {
    sums = reinterpret_cast<float*>(space + p.x_bytes + p.parts_bytes);
    a.out = sums;
    a.stride = p.sum_ld;
    a.split_stride = outs * p.sum_ld;
  } else {
    a.out = dw;
    a.stride = out_stride;
    a.bf16 = bf16_out;
    a.accumulate = accumulate;
  }
  if ((e = cudaFuncSetAttribute(weight_grad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem)) != cudaSuccess)
    return cuda_error(e);
  const int64_t units = (int64_t)a.tiles * a.splits, pairs = sms / 2;
  e = launch(weight_grad_kernel, (int)(2 * (units < pairs ? units : pairs)), kGradThreads, kGradSmem, s, 2, true, a);
  if (e != cudaSuccess) return cuda_error(e);
  if (p.splits > 1) {
    e = bf16_out ? launch_join<__nv_bfloat16>(p, sums, dw, out_stride, outs, cols, accumulate, sms, s)
                 : launch_join<float>(p, sums, dw, out_stride, outs, cols, accumulate, sms, s);
    if (e != cudaSuccess) return cuda_error(e);
  }
  return MUON_OK;
}

}  // extern "C"
