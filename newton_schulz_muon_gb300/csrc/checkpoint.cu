// Activation checkpoints in 8 bits: saved, loaded, and those of a gated activation's two
// inputs saved in its forward pass and read in its backward pass.
//
//   h = gate s up,  s = 1 / (1 + e^-gate)
//   dgate = dh up s (1 + gate (1 - s)),  dup = dh gate s
//
// A thread takes one 16-byte unit of a row at a time (8 bf16 or 4 fp32 columns), so that the
// 4 or 8 lanes of a block of 32 columns find its largest magnitude with 2 or 3 shuffles and
// every access of a warp is to consecutive bytes.  A CTA takes several times as many
// consecutive units as it has threads; the loads of all of a thread's units are issued before
// the first is used.  Each element is read and written by one thread, which reads first: an
// output may be an input of the same layout.
//
// Bound by HBM, next to which stands the issue of instructions: magnitudes of bf16 are compared
// two at a time, and bounds and alignment are left out where all rows are whole blocks on 16-byte
// boundaries.  (Bytes to numbers by their bits, a permutation and a difference, instead of by
// conversions, which have a pipe of their own: loading 95 us instead of 73.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "checkpoint.cuh"
#include "checkpoint.h"
#include "device.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "muon.h"
#include "rows.cuh"

namespace muon {
namespace {

enum Pass { kSave, kLoad, kGatedForward, kGatedBackward };

constexpr int kCheckpointThreads = 128;
// Units of a thread: as many as the loads' latency needs, fewer where more matrices are in
// flight (8192 or, saved and loaded, 16384 x 9728 bf16, us: save 82 with 4, 79 with 6; forward
// 109, 101, 97 with 1, 2, 4; backward 121, 118, 119).
__host__ __device__ constexpr int items_of(int pass) { return pass == kSave ? 6 : pass == kGatedBackward ? 2 : 4; }

// A matrix of T, rows `stride` elements apart.
struct Matrix {
  void* p;
  int64_t stride;
};

struct CheckpointArgs {
  CheckpointView a, b;   // the checkpoint; gate's and up's
  Matrix x, y, z;        // inputs: x; gate, up; dh
  Matrix u, v, w;        // outputs: x; h; dgate, dup, h (p null: not wanted)
  int64_t items;         // units of all rows, padding included
  int32_t per_row;
};

// Unit `col / N` of a row; columns from `cols` on are 0.  kWhole: every unit lies in the row and on
// a 16-byte boundary.
template <typename T, bool kWhole>
__device__ __forceinline__ uint4 load_cols(const Matrix& m, int64_t row, int col, int cols) {
  constexpr int N = Vec<T>::N;
  const T* p = reinterpret_cast<const T*>(m.p) + row * m.stride + col;
  if constexpr (kWhole) {
    return *reinterpret_cast<const uint4*>(p);
  } else {
    if (col + N <= cols && (reinterpret_cast<uint64_t>(p) & 15) == 0) return *reinterpret_cast<const uint4*>(p);
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = col + i < cols ? Vec<T>::load(p + i) : 0.f;
    return Vec<T>::pack(v);
  }
}

template <typename T, bool kWhole>
__device__ __forceinline__ void store_cols(const Matrix& m, int64_t row, int col, int cols, const float (&v)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  T* p = reinterpret_cast<T*>(m.p) + row * m.stride + col;
  if constexpr (kWhole) {
    *reinterpret_cast<uint4*>(p) = Vec<T>::pack(v);
  } else if (col + N <= cols && (reinterpret_cast<uint64_t>(p) & 15) == 0) {
    *reinterpret_cast<uint4*>(p) = Vec<T>::pack(v);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (col + i < cols) Vec<T>::store(p + i, v[i]);
  }
}

// The bits of the largest magnitude of a block, of which a lane has the unit w.
template <typename T>
__device__ __forceinline__ uint32_t block_most(const uint4& w) {
  constexpr int kLanes = kBlockCols / Vec<T>::N;
  if constexpr (sizeof(T) == 2) {  // magnitudes of bf16 compare as 16-bit integers
    uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7FFF7FFFu, w.y & 0x7FFF7FFFu), __vmaxu2(w.z & 0x7FFF7FFFu, w.w & 0x7FFF7FFFu));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return max(m << 16, m & 0xFFFF0000u);
  } else {
    uint32_t m = max(max(w.x & 0x7FFFFFFFu, w.y & 0x7FFFFFFFu), max(w.z & 0x7FFFFFFFu, w.w & 0x7FFFFFFFu));
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    return m;
  }
}

// Quantises the unit w, whose values are v; the lanes of a block work together.
template <typename T>
__device__ __forceinline__ void save_unit(const CheckpointView& c, int64_t row, int unit, const uint4& w,
                                          const float (&v)[Vec<T>::N], bool live) {
  constexpr int N = Vec<T>::N, kLanes = kBlockCols / N;
  const uint32_t most = block_most<T>(w);
  if (!live) return;
  const int b = block_byte(most);
  const float scale = steps_per_unit(b);
  uint32_t q[N / 4];
#pragma unroll
  for (int i = 0; i < N; i += 4) q[i / 4] = quantize4(v[i], v[i + 1], v[i + 2], v[i + 3], scale);
  if (b >= 254) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = fminf(fmaxf(v[i + k] * scale, -127.f), 127.f);
      q[i / 4] = b == 255 ? 0u : quantize4(x[0], x[1], x[2], x[3], 1.f);
    }
  }
  int8_t* at = c.q + (row * c.blocks * kBlockCols + (int64_t)unit * N);
  if constexpr (N == 8) *reinterpret_cast<uint2*>(at) = make_uint2(q[0], q[1]);
  else *reinterpret_cast<uint32_t*>(at) = q[0];
  if (unit % kLanes == 0) c.b[row * c.blocks + unit / kLanes] = (uint8_t)b;
}

// A unit of a checkpoint as it lies in memory, and its values.
template <int N>
struct SavedUnit {
  uint32_t q[N / 4];
  int b;
};
template <int N>
__device__ __forceinline__ SavedUnit<N> fetch_unit(const CheckpointView& c, int64_t row, int unit) {
  SavedUnit<N> s;
  const int8_t* at = c.q + (row * c.blocks * kBlockCols + (int64_t)unit * N);
  if constexpr (N == 8) {
    const uint2 w = *reinterpret_cast<const uint2*>(at);
    s.q[0] = w.x;
    s.q[1] = w.y;
  } else {
    s.q[0] = *reinterpret_cast<const uint32_t*>(at);
  }
  s.b = c.b[row * c.blocks + unit / (kBlockCols / N)];
  return s;
}
template <int N>
__device__ __forceinline__ void values_of(const SavedUnit<N>& s, float (&v)[N]) {
  const float step = step_of(s.b);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = (float)(int8_t)(s.q[i / 4] >> (8 * (i % 4))) * step;
}

// 1 / (1 + e^-g) and 1 minus that, which is e^-g / (1 + e^-g).  For bf16, whose results keep 8
// bits, the approximate exponential and reciprocal, 2^-22 each and |g| 7.3e-8 for the exponent's
// rounding (6e-6 at the largest |g| that leaves a sigmoid, 88), and the difference.
template <typename T>
__device__ __forceinline__ float2 sigmoid(float g) {
  if constexpr (sizeof(T) == 2) {
    float s;
    asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(1.f + ex2(-1.4426950408889634f * g)));
    return make_float2(s, 1.f - s);
  } else {
    const float e = expf(-g), s = __frcp_rn(1.f + e);
    return make_float2(s, e == INFINITY ? 1.f : e * s);
  }
}

template <typename T, int kPass, bool kWhole>
__global__ void __launch_bounds__(kCheckpointThreads) checkpoint_kernel(const __grid_constant__ CheckpointArgs a) {
  constexpr int N = Vec<T>::N;
  constexpr int kCount = items_of(kPass);
  griddep_launch_dependents();
  const int64_t first = (int64_t)blockIdx.x * (kCheckpointThreads * kCount) + threadIdx.x;
  int64_t row;
  int unit;
  if (a.items <= 0xFFFFFFFFll) {
    row = (uint32_t)first / (uint32_t)a.per_row;
    unit = (int)((uint32_t)first % (uint32_t)a.per_row);
  } else {
    row = first / a.per_row;
    unit = (int)(first % a.per_row);
  }
  int64_t rows[kCount];
  int units[kCount];
  bool live[kCount];
#pragma unroll
  for (int k = 0; k < kCount; ++k) {
    rows[k] = row;
    units[k] = unit;
    live[k] = first + k * kCheckpointThreads < a.items;
    unit += kCheckpointThreads;
    if (unit >= a.per_row) {
      row += unit / a.per_row;
      unit %= a.per_row;
    }
  }
  const int cols = a.a.cols;
  if constexpr (kPass == kSave || kPass == kGatedForward) {
    uint4 x[kCount], y[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      x[k] = y[k] = make_uint4(0, 0, 0, 0);
      if (!live[k]) continue;
      x[k] = load_cols<T, kWhole>(a.x, rows[k], units[k] * N, cols);
      if (kPass == kGatedForward) y[k] = load_cols<T, kWhole>(a.y, rows[k], units[k] * N, cols);
    }
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      float g[N];
      Vec<T>::unpack(x[k], g);
      save_unit<T>(a.a, rows[k], units[k], x[k], g, live[k]);
      if constexpr (kPass == kGatedForward) {
        float up[N], h[N];
        Vec<T>::unpack(y[k], up);
        save_unit<T>(a.b, rows[k], units[k], y[k], up, live[k]);
#pragma unroll
        for (int i = 0; i < N; ++i) h[i] = g[i] * sigmoid<T>(g[i]).x * up[i];
        if (live[k]) store_cols<T, kWhole>(a.u, rows[k], units[k] * N, cols, h);
      }
    }
  } else {
    SavedUnit<N> s[kCount], t[kCount];
    uint4 z[kCount];
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      if (!live[k]) continue;
      s[k] = fetch_unit<N>(a.a, rows[k], units[k]);
      if (kPass == kGatedBackward) {
        t[k] = fetch_unit<N>(a.b, rows[k], units[k]);
        z[k] = load_cols<T, kWhole>(a.z, rows[k], units[k] * N, cols);
      }
    }
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int col = units[k] * N;
      if (!live[k] || (!kWhole && col >= cols)) continue;
      float g[N];
      values_of<N>(s[k], g);
      if constexpr (kPass == kLoad) {
        store_cols<T, kWhole>(a.u, rows[k], col, cols, g);
      } else {
        float up[N], dh[N], dg[N], du[N], h[N];
        values_of<N>(t[k], up);
        Vec<T>::unpack(z[k], dh);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float2 e = sigmoid<T>(g[i]);
          const float act = g[i] * e.x;
          dg[i] = dh[i] * up[i] * __fmaf_rn(act, e.y, e.x);
          du[i] = dh[i] * act;
          h[i] = act * up[i];
        }
        store_cols<T, kWhole>(a.u, rows[k], col, cols, dg);
        store_cols<T, kWhole>(a.v, rows[k], col, cols, du);
        if (a.w.p != nullptr) store_cols<T, kWhole>(a.w, rows[k], col, cols, h);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int32_t check_checkpoint(const muon_checkpoint* c) {
  if (!c) return invalid("checkpoint is NULL");
  if (c->rows < 0 || c->rows > (1ll << 31) - 1) return invalid("rows must be in [0, 2^31)");
  if (c->cols < 1 || c->cols > (1ll << 30)) return invalid("cols must be in [1, 2^30]");
  if (c->rows > 0 && !c->data) return invalid("checkpoint data is NULL");
  if (!aligned(c->data, 16)) return invalid("checkpoint data must be 16-byte aligned");
  return MUON_OK;
}

int32_t check_matrix(const void* p, int64_t stride, int64_t cols, int32_t dtype, Matrix* m) {
  if (!p) return invalid("a matrix is NULL");
  if (!aligned(p, dtype == MUON_DTYPE_BF16 ? 2 : 4)) return invalid("a matrix is not aligned to its type");
  if (stride != 0 && (stride < cols || stride > (1ll << 40))) return invalid("a row stride must be 0 or at least the columns");
  *m = Matrix{const_cast<void*>(p), stride ? stride : cols};
  return MUON_OK;
}

// An output in the place of an input: each element is read and written by one thread only where both
// have one row stride.
bool displaced(const Matrix& out, const Matrix& in, int64_t rows) {
  return rows > 1 && out.p == in.p && out.stride != in.stride;
}

CheckpointView view_of(const muon_checkpoint* c) {
  CheckpointView v;
  v.rows = c->rows;
  v.cols = (int32_t)c->cols;
  v.blocks = (int32_t)((c->cols + kBlockCols - 1) / kBlockCols);
  v.q = static_cast<int8_t*>(c->data);
  v.b = static_cast<uint8_t*>(c->data) + c->rows * v.blocks * kBlockCols;
  return v;
}

// Whether every unit of every row lies on a 16-byte boundary (where there is such a matrix).
bool whole(const Matrix& m, int n) { return !m.p || (aligned(m.p, 16) && m.stride % n == 0); }

template <typename T, int kPass>
cudaError_t launch_as(const CheckpointArgs& a, int64_t grid, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const bool all = a.a.cols % kBlockCols == 0 && whole(a.x, N) && whole(a.y, N) && whole(a.z, N) && whole(a.u, N) &&
                   whole(a.v, N) && whole(a.w, N);
  return launch(all ? checkpoint_kernel<T, kPass, true> : checkpoint_kernel<T, kPass, false>, (int)grid, kCheckpointThreads, 0,
                s, 1, false, a);
}

// The pass over a.a's rows; false: too many of them for a grid.
template <int kPass>
bool launch_pass(CheckpointArgs& a, int32_t dtype, cudaStream_t s, cudaError_t* e) {
  const int n = dtype == MUON_DTYPE_BF16 ? 8 : 4;
  a.per_row = a.a.blocks * (kBlockCols / n);
  a.items = a.a.rows * a.per_row;
  const int64_t per_cta = kCheckpointThreads * items_of(kPass);
  const int64_t grid = (a.items + per_cta - 1) / per_cta;
  if (grid > (1ll << 31) - 1) return false;
  *e = dtype == MUON_DTYPE_BF16 ? launch_as<__nv_bfloat16, kPass>(a, grid, s) : launch_as<float, kPass>(a, grid, s);
  return true;
}

template <int kPass>
int32_t run_checkpoint(CheckpointArgs& a, int32_t dtype, void* stream) {
  int sms;
  const int32_t st = find_device(&sms);
  if (st != MUON_OK) return st;
  cudaError_t e;
  if (!launch_pass<kPass>(a, dtype, static_cast<cudaStream_t>(stream), &e))
    return set_error(MUON_ERR_UNSUPPORTED, "more than 2^31 pieces of a checkpoint");
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

bool known(int32_t dtype) { return dtype == MUON_DTYPE_F32 || dtype == MUON_DTYPE_BF16; }

}  // namespace

cudaError_t launch_checkpoint_load(const muon_checkpoint* checkpoint, void* x, int64_t ld, cudaStream_t stream) {
  CheckpointArgs a = {};
  a.a = view_of(checkpoint);
  a.u = Matrix{x, ld};
  cudaError_t e;
  return launch_pass<kLoad>(a, MUON_DTYPE_BF16, stream, &e) ? e : cudaErrorInvalidConfiguration;
}

}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_checkpoint_bytes(int64_t rows, int64_t cols, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  if (rows < 0 || rows > (1ll << 31) - 1) return invalid("rows must be in [0, 2^31)");
  if (cols < 1 || cols > (1ll << 30)) return invalid("cols must be in [1, 2^30]");
  *bytes = (size_t)rows * (size_t)((cols + kBlockCols - 1) / kBlockCols) * (kBlockCols + 1);
  return MUON_OK;
}

muon_status muon_checkpoint_save(const void* x, int64_t x_stride, int32_t dtype, const muon_checkpoint* checkpoint,
                                 void* stream) {
  int32_t st = check_checkpoint(checkpoint);
  if (st != MUON_OK) return st;
  if (!known(dtype)) return invalid("unknown dtype");
  if (checkpoint->rows == 0) return MUON_OK;
  CheckpointArgs a = {};
  if ((st = check_matrix(x, x_stride, checkpoint->cols, dtype, &a.x)) != MUON_OK) return st;
  a.a = view_of(checkpoint);
  return run_checkpoint<kSave>(a, dtype, stream);
}

muon_status muon_checkpoint_load(const muon_checkpoint* checkpoint, void* x, int64_t x_stride, int32_t dtype,
                                 void* stream) {
  int32_t st = check_checkpoint(checkpoint);
  if (st != MUON_OK) return st;
  if (!known(dtype)) return invalid("unknown dtype");
  if (checkpoint->rows == 0) return MUON_OK;
  CheckpointArgs a = {};
  if ((st = check_matrix(x, x_stride, checkpoint->cols, dtype, &a.u)) != MUON_OK) return st;
  a.a = view_of(checkpoint);
  return run_checkpoint<kLoad>(a, dtype, stream);
}

muon_status muon_swiglu_forward(const void* gate, int64_t gate_stride, const void* up, int64_t up_stride, int32_t dtype,
                                void* h, int64_t h_stride, const muon_checkpoint* gate_checkpoint,
                                const muon_checkpoint* up_checkpoint, void* stream) {
  int32_t st = check_checkpoint(gate_checkpoint);
  if (st == MUON_OK) st = check_checkpoint(up_checkpoint);
  if (st != MUON_OK) return st;
  const int64_t rows = gate_checkpoint->rows, cols = gate_checkpoint->cols;
  if (up_checkpoint->rows != rows || up_checkpoint->cols != cols) return invalid("the checkpoints have two shapes");
  if (!known(dtype)) return invalid("unknown dtype");
  if (rows == 0) return MUON_OK;
  if (gate_checkpoint->data == up_checkpoint->data) return invalid("the checkpoints are one");
  CheckpointArgs a = {};
  if ((st = check_matrix(gate, gate_stride, cols, dtype, &a.x)) != MUON_OK) return st;
  if ((st = check_matrix(up, up_stride, cols, dtype, &a.y)) != MUON_OK) return st;
  if ((st = check_matrix(h, h_stride, cols, dtype, &a.u)) != MUON_OK) return st;
  if (displaced(a.u, a.x, rows) || displaced(a.u, a.y, rows))
    return invalid("h in place of gate or up must have its row stride");
  a.a = view_of(gate_checkpoint);
  a.b = view_of(up_checkpoint);
  return run_checkpoint<kGatedForward>(a, dtype, stream);
}

muon_status muon_swiglu_backward(const void* dh, int64_t dh_stride, int32_t dtype, const muon_checkpoint* gate_checkpoint,
                                 const muon_checkpoint* up_checkpoint, void* dgate, int64_t dgate_stride, void* dup,
                                 int64_t dup_stride, void* h, int64_t h_stride, void* stream) {
  int32_t st = check_checkpoint(gate_checkpoint);
  if (st == MUON_OK) st = check_checkpoint(up_checkpoint);
  if (st != MUON_OK) return st;
  const int64_t rows = gate_checkpoint->rows, cols = gate_checkpoint->cols;
  if (up_checkpoint->rows != rows || up_checkpoint->cols != cols) return invalid("the checkpoints have two shapes");
  if (!known(dtype)) return invalid("unknown dtype");
  if (rows == 0) return MUON_OK;
  CheckpointArgs a = {};
  if ((st = check_matrix(dh, dh_stride, cols, dtype, &a.z)) != MUON_OK) return st;
  if ((st = check_matrix(dgate, dgate_stride, cols, dtype, &a.u)) != MUON_OK) return st;
  if ((st = check_matrix(dup, dup_stride, cols, dtype, &a.v)) != MUON_OK) return st;
  if (h && (st = check_matrix(h, h_stride, cols, dtype, &a.w)) != MUON_OK) return st;
  if (dgate == dup || dgate == h || dup == h) return invalid("two outputs are one");
  if (displaced(a.u, a.z, rows) || displaced(a.v, a.z, rows) || displaced(a.w, a.z, rows))
    return invalid("an output in place of dh must have its row stride");
  a.a = view_of(gate_checkpoint);
  a.b = view_of(up_checkpoint);
  return run_checkpoint<kGatedBackward>(a, dtype, stream);
}

}  // extern "C"
