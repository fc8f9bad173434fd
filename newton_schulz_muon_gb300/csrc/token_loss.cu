// Losses on token log-probabilities, and their gradient with respect to the logits.
//
//   logp_t = z_y - log sum_j exp(z_j),  z = logits / temperature
//   dL/dz_j = dL/dlogp_t (1[j = y_t] - softmax(z)_j)
//
// The clipped policy loss needs only the row's own logp for dL/dlogp_t, so a row's
// gradient follows its log-probability in the same launch; the preference loss needs
// the sums over whole sequences first, so its forward and backward passes are launches
// of their own with a small one between them.
//
// Exponentials are taken in base 2 with c = log2(e) / temperature: a row's sum is
// s = sum_j 2^(c z_j - f) with the frame f = fl(c m), m = max_j z_j, and every later use
// takes the same f, so that its rounding cancels.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "device.cuh"
#include "epilogue.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "momentum.cuh"
#include "muon.h"

namespace muon {
namespace {

constexpr float kLn2 = 0.693147180559945309f;

// What a row kernel does with each row.
enum RowMode : int32_t {
  kLogp = 0,     // log-probabilities
  kForward = 1,  // log-probabilities and the row's frame and sum, for a later backward pass
  kPolicy = 2,   // the policy loss's terms and gradient
};

struct RowArgs {
  const void* logits;
  const int64_t* targets;
  const uint8_t* mask;
  int64_t tokens, vocab, stride, grad_stride;
  float c;               // log2(e) / temperature
  float inv_temp;
  float* logp;           // or null
  float2* frame;         // kForward: (m, s) of each row
  float* slope;          // kForward: cleared for rows of no sequence
  // kPolicy
  const float* old_logp;
  const float* ref_logp; // or null
  const float* adv;
  const float* inv_count; // token mean and sum: one weight for all positions
  const float* weight;    // sequence mean: [tokens]
  float low, high, beta, grad_scale;
  void* grad;             // or null
  float4* terms;          // [tokens]: w (-s + beta k), w (-s), w k, w [clipped]
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;  // elements of 16 bytes
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[4]) {
    v[0] = __uint_as_float(w.x); v[1] = __uint_as_float(w.y);
    v[2] = __uint_as_float(w.z); v[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float (&v)[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(u[i] << 16);
      v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                      pack_bf16x2(v[6], v[7]));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

// A partial sum of exponentials: s = sum_j 2^(c z_j - fl(c m)), m the largest z so far
// (-inf: nothing yet, or only logits of -inf).  c m leaves fp32's range for logits near
// the type's limits (a mask of its lowest value); the numbers there are so far apart that
// only those equal to m count, one each.
struct Sum {
  float m, s;
};

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < INFINITY; }

// Factor that takes a sum from the frame of m to that of the larger `to`.
__device__ __forceinline__ float reframe(float m, float to, float c) {
  if (m == to) return 1.f;  // both -inf among them
  const float f = to * c;
  return f == -INFINITY ? 0.f : ex2(m * c - f);  // a NaN stays one
}

__device__ __forceinline__ Sum merge(const Sum& a, const Sum& b, float c) {
  Sum r;
  r.m = fmaxf(a.m, b.m);
  r.s = a.s * reframe(a.m, r.m, c) + b.s * reframe(b.m, r.m, c);
  return r;
}

// 2^(c z - f) in the frame of m whose f = c m is out of range.
__device__ __forceinline__ float far_term(float z, float m) {
  if (z != z || z == INFINITY) return NAN;
  return z == m && z != -INFINITY ? 1.f : 0.f;
}

template <int N>
__device__ __forceinline__ void add_values(Sum& t, const float (&v)[N], float c) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < N; ++i) m = fmaxf(m, v[i]);
  if (!(m <= t.m)) {
    t.s *= t.s == 0.f ? 1.f : reframe(t.m, m, c);
    t.m = m;
  }
  const float f = t.m * c;
  if (finite(f)) {
#pragma unroll
    for (int i = 0; i < N; ++i) t.s += ex2(__fmaf_rn(v[i], c, -f));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) t.s += far_term(v[i], t.m);
  }
}

// log2 of the target's probability; also the exponent's form in pass 2.
__device__ __forceinline__ float log2_prob(float z, const Sum& t, float c) {
  const float f = t.m * c;
  const float d = finite(f) ? __fmaf_rn(z, c, -f) : log2f(far_term(z, t.m));
  return d - log2f(t.s);
}

__device__ __forceinline__ float term(float z, float c, float m, float f, bool near) {
  return near ? ex2(__fmaf_rn(z, c, -f)) : far_term(z, m);
}

__device__ __forceinline__ Sum warp_merge(Sum t, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum b;
    b.m = __shfl_xor_sync(0xFFFFFFFFu, t.m, o);
    b.s = __shfl_xor_sync(0xFFFFFFFFu, t.s, o);
    t = merge(t, b, c);
  }
  return t;
}

// A position's scalars, read before its logits are.
struct Position {
  int64_t y;
  float old_logp, ref, adv, w;
};

struct Outcome {
  float slope;  // dL/dlogp
  float4 terms;
};

__device__ __forceinline__ Outcome policy_terms(const RowArgs& a, const Position& p, float logp) {
  Outcome o;
  o.slope = 0.f;
  o.terms = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.w == 0.f) return o;  // a position of no sequence
  const float ratio = expf(logp - p.old_logp);
  // a ratio above fp32's range times a zero advantage is zero
  const float plain = p.adv == 0.f && ratio == INFINITY ? 0.f : ratio * p.adv;
  const float limit = fminf(fmaxf(ratio, a.low), a.high);
  const float held = p.adv == 0.f && limit == INFINITY ? 0.f : limit * p.adv;
  const bool clipped = held < plain;
  const float s = clipped ? held : plain;
  float k = 0.f;
  float slope = clipped ? 0.f : -plain;
  if (a.beta != 0.f) {
    const float d = p.ref - logp;
    const float e = expm1f(d);
    // e - d cancels for small d: its series there, (d^2 / 2)(1 + d/3 + d^2/12 + d^3/60 + ...)
    k = fabsf(d) < 0.1f
            ? 0.5f * d * d * (1.f + d * (1.f / 3.f) * (1.f + d * 0.25f * (1.f + d * 0.2f * (1.f + d * (1.f / 6.f)))))
            : e - d;
    slope -= a.beta * e;
  }
  o.slope = p.w * slope;
  o.terms = make_float4(p.w * (a.beta * k - s), p.w * -s, p.w * k, clipped ? p.w : 0.f);
  return o;
}

constexpr int kRowThreads = 512;
constexpr int kRowWarps = kRowThreads / 32;

// One CTA a row, the row read twice (the second time from L2).
template <typename T, int kMode>
__global__ void __launch_bounds__(kRowThreads) row_kernel(const __grid_constant__ RowArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Sum red[kRowWarps];
  __shared__ float2 back;  // dL/dz factor of the row, and the target's value
  const int tid = threadIdx.x;
  griddep_wait();
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T* z = reinterpret_cast<const T*>(a.logits) + t * a.stride;
    T* g = reinterpret_cast<T*>(a.grad) + t * a.grad_stride;
    const bool live = a.mask == nullptr || a.mask[t] != 0;
    const uint64_t mis = reinterpret_cast<uint64_t>(z) & 15;
    const int64_t head = min(a.vocab, (int64_t)(((16 - mis) & 15) / sizeof(T)));
    const int64_t nv = (a.vocab - head) / N;
    const int64_t tail = head + nv * N;
    const uint4* zv = reinterpret_cast<const uint4*>(z + head);
    if (!live) {
      if (tid == 0) {
        if (a.logp) a.logp[t] = 0.f;
        if (kMode == kForward) a.slope[t] = 0.f;
        if (kMode == kPolicy) a.terms[t] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      if (kMode == kPolicy && a.grad)
        for (int64_t j = tid; j < a.vocab; j += kRowThreads) Vec<T>::store(g + j, 0.f);
      continue;
    }
    Sum part{-INFINITY, 0.f};
    for (int64_t i = tid; i < nv; i += kRowThreads) {
      float v[N];
      Vec<T>::unpack(zv[i], v);
      add_values<N>(part, v, a.c);
    }
    const int64_t edge = tid < 16 ? (tid < head ? tid : -1) : (tid < 32 && tail + tid - 16 < a.vocab ? tail + tid - 16 : -1);
    if (edge >= 0) {
      float v[1] = {Vec<T>::load(z + edge)};
      add_values<1>(part, v, a.c);
    }
    part = warp_merge(part, a.c);
    if ((tid & 31) == 0) red[tid >> 5] = part;
    __syncthreads();
    Sum all = red[0];
#pragma unroll
    for (int w = 1; w < kRowWarps; ++w) all = merge(all, red[w], a.c);
    if (tid == 0) {
      const int64_t y = a.targets[t];
      const bool fits = y >= 0 && y < a.vocab;
      const float zy = fits ? Vec<T>::load(z + y) : NAN;
      const float logp = kLn2 * log2_prob(zy, all, a.c);
      if (a.logp) a.logp[t] = logp;
      if (kMode == kForward) {
        a.frame[t] = make_float2(all.m, all.s);
        a.slope[t] = 0.f;
      }
      if (kMode == kPolicy) {
        Position p;
        p.y = y;
        p.old_logp = a.old_logp[t];
        p.ref = a.ref_logp ? a.ref_logp[t] : 0.f;
        p.adv = a.adv[t];
        p.w = a.weight ? a.weight[t] : *a.inv_count;
        const Outcome o = policy_terms(a, p, logp);
        a.terms[t] = o.terms;
        const float f = o.slope * a.grad_scale * a.inv_temp;
        back = make_float2(-f / all.s, -f * expm1f(logp));
      }
    }
    __syncthreads();
    if (kMode == kPolicy && a.grad) {
      const float2 b = back;
      const int64_t y = a.targets[t];
      const float f = all.m * a.c;
      const bool near = finite(f);
      for (int64_t j = tid; j < a.vocab; j += kRowThreads) {
        const float e = term(Vec<T>::load(z + j), a.c, all.m, f, near);
        Vec<T>::store(g + j, j == y ? b.y : b.x * e);
      }
      __syncthreads();  // `back` and `red` are free for the next row
    }
  }
}

// The gradient of rows whose slope, frame and sum are known: one CTA a row.
template <typename T>
__global__ void __launch_bounds__(kRowThreads) backward_kernel(const __grid_constant__ RowArgs a) {
  griddep_wait();
  const int tid = threadIdx.x;
  for (int64_t r = blockIdx.x; r < a.tokens; r += gridDim.x) {
    const int64_t t = a.tokens - 1 - r;
    const T* z = reinterpret_cast<const T*>(a.logits) + t * a.stride;
    T* g = reinterpret_cast<T*>(a.grad) + t * a.grad_stride;
    const bool live = a.mask == nullptr || a.mask[t] != 0;
    const float f = live ? a.slope[t] * a.grad_scale * a.inv_temp : 0.f;
    if (f == 0.f) {
      for (int64_t j = tid; j < a.vocab; j += kRowThreads) Vec<T>::store(g + j, 0.f);
      continue;
    }
    const float2 fs = a.frame[t];
    const int64_t y = a.targets[t];
    const float at_y = -f * expm1f(a.logp[t]);
    const float factor = -f / fs.y;
    const float frame = fs.x * a.c;
    const bool near = finite(frame);
    for (int64_t j = tid; j < a.vocab; j += kRowThreads) {
      const float e = term(Vec<T>::load(z + j), a.c, fs.x, frame, near);
      Vec<T>::store(g + j, j == y ? at_y : factor * e);
    }
  }
}

// ---------------------------------------------------------------------------
// small kernels
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 512;

__device__ __forceinline__ int64_t clamp_offset(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

__device__ __forceinline__ int64_t block_sum(int64_t v) {
  __shared__ int64_t red[kSmallThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 32; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[kSmallThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kSmallThreads / 32; ++w) v += red[w];
  return v;
}

__device__ __forceinline__ int64_t live_count(const uint8_t* mask, int64_t a, int64_t b) {
  if (mask == nullptr) return b > a ? b - a : 0;
  int64_t n = 0;
  for (int64_t t = a + threadIdx.x; t < b; t += kSmallThreads) n += mask[t] != 0;
  return block_sum(n);
}

// Weight of every position under the token mean (or the sum: 1).
__global__ void __launch_bounds__(kSmallThreads) count_kernel(const uint8_t* mask, int64_t tokens, int mean,
                                                              float* inv_count) {
  float w = 1.f;
  if (mean) {
    const int64_t n = live_count(mask, 0, tokens);
    w = 1.f / (float)(n < 1 ? 1 : n);
  }
  if (threadIdx.x == 0) *inv_count = w;
}

// Sequence mean: one CTA a sequence writes the weights of its positions; CTA n_seqs
// clears those before the first and after the last.
__global__ void __launch_bounds__(kSmallThreads) weight_kernel(const uint8_t* mask, int64_t tokens,
                                                               const int64_t* offsets, int64_t n_seqs, float* weight) {
  const int64_t q = blockIdx.x;
  if (q == n_seqs) {
    const int64_t a = clamp_offset(offsets[0], 0, tokens), b = clamp_offset(offsets[n_seqs], a, tokens);
    for (int64_t t = threadIdx.x; t < a; t += kSmallThreads) weight[t] = 0.f;
    for (int64_t t = b + threadIdx.x; t < tokens; t += kSmallThreads) weight[t] = 0.f;
    return;
  }
  const int64_t a = clamp_offset(offsets[q], 0, tokens), b = clamp_offset(offsets[q + 1], a, tokens);
  const int64_t n = live_count(mask, a, b);
  const float w = 1.f / ((float)n_seqs * (float)(n < 1 ? 1 : n));
  for (int64_t t = a + threadIdx.x; t < b; t += kSmallThreads)
    weight[t] = mask == nullptr || mask[t] != 0 ? w : 0.f;
}

// stats = sum of the positions' terms.
__global__ void __launch_bounds__(kSmallThreads) stats_kernel(const float4* terms, int64_t tokens, float* stats) {
  griddep_wait();
  float h[4] = {0.f, 0.f, 0.f, 0.f}, l[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t t = threadIdx.x; t < tokens; t += kSmallThreads) {
    const float4 x = terms[t];
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s, e;
      two_sum(h[i], v[i], s, e);
      h[i] = s;
      l[i] += isfinite(s) ? e : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double s = block_sum((double)h[i] + (double)l[i]);
    if (threadIdx.x == 0) stats[i] = (float)s;
  }
}

struct PairArgs {
  const uint8_t* mask;
  const float* logp;
  const float* ref;
  const int64_t* offsets;
  int64_t tokens, n_pairs;
  float beta, smooth;
  int32_t mean;
  float* margins;   // or null
  float* seq_logp;  // or null
  float* pair_loss; // [n_pairs]
  float* slope;     // [tokens], or null
};

// One CTA a pair: both sums, the margin, and the slope of each of its positions.
__global__ void __launch_bounds__(kSmallThreads) pair_kernel(const __grid_constant__ PairArgs a) {
  griddep_wait();
  const int64_t i = blockIdx.x;
  double gain[2];
  int64_t lo[2], hi[2];
  float per[2];
  for (int k = 0; k < 2; ++k) {
    const int64_t q = k == 0 ? i : a.n_pairs + i;
    lo[k] = clamp_offset(a.offsets[q], 0, a.tokens);
    hi[k] = clamp_offset(a.offsets[q + 1], lo[k], a.tokens);
    float h = 0.f, l = 0.f;
    for (int64_t t = lo[k] + threadIdx.x; t < hi[k]; t += kSmallThreads) {
      float s, e;
      two_sum(h, a.logp[t], s, e);  // 0 where masked
      h = s;
      l += isfinite(s) ? e : 0.f;
    }
    double sum = block_sum((double)h + (double)l);
    const int64_t n = a.mean ? live_count(a.mask, lo[k], hi[k]) : 1;
    per[k] = 1.f / (float)(n < 1 ? 1 : n);
    if (a.mean) sum /= (double)(n < 1 ? 1 : n);
    if (threadIdx.x == 0 && a.seq_logp) a.seq_logp[q] = (float)sum;
    gain[k] = sum - (double)a.ref[q];
  }
  const float h = (float)((double)a.beta * (gain[0] - gain[1]));
  // log sigmoid(h) = min(h, 0) - log(1 + exp(-|h|))
  const float soft = log1pf(expf(-fabsf(h)));
  if (threadIdx.x == 0) {
    if (a.margins) a.margins[i] = h;
    a.pair_loss[i] = (1.f - a.smooth) * (soft - fminf(h, 0.f)) + a.smooth * (soft + fmaxf(h, 0.f));
  }
  if (a.slope) {
    const float up = 1.f / (1.f + expf(-h)), down = 1.f / (1.f + expf(h));
    const float d = a.beta / (float)a.n_pairs * (a.smooth * up - (1.f - a.smooth) * down);
    for (int k = 0; k < 2; ++k)
      for (int64_t t = lo[k] + threadIdx.x; t < hi[k]; t += kSmallThreads) a.slope[t] = (k == 0 ? d : -d) * per[k];
  }
}

__global__ void __launch_bounds__(kSmallThreads) pair_mean_kernel(const float* pair_loss, int64_t n, float* loss) {
  griddep_wait();
  double t = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kSmallThreads) t += (double)pair_loss[i];
  t = block_sum(t);
  if (threadIdx.x == 0) *loss = n > 0 ? (float)(t / (double)n) : 0.f;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int32_t invalid(const char* msg) { return set_error(MUON_ERR_INVALID, msg); }
int32_t cuda_error(cudaError_t e) { return set_error(MUON_ERR_CUDA, cudaGetErrorString(e)); }

bool aligned(const void* p, size_t a) { return reinterpret_cast<uint64_t>(p) % a == 0; }

int32_t check_batch(const muon_token_batch* b) {
  if (!b) return invalid("batch is NULL");
  if (b->tokens < 0 || b->tokens > (1ll << 31) - 1) return invalid("tokens must be in [0, 2^31)");
  if (b->vocab < 1 || b->vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (b->row_stride != 0 && (b->row_stride < b->vocab || b->row_stride > (1ll << 40)))
    return invalid("row_stride must be 0 or at least vocab");
  if (b->dtype != MUON_DTYPE_F32 && b->dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  if (!(b->temperature > 0.f) || std::isinf(b->temperature)) return invalid("temperature must be finite and > 0");
  if (b->tokens == 0) return MUON_OK;
  if (!b->logits || !b->targets) return invalid("logits or targets is NULL");
  if (!aligned(b->logits, b->dtype == MUON_DTYPE_BF16 ? 2 : 4) || !aligned(b->targets, 8))
    return invalid("logits or targets is not aligned to its type");
  return MUON_OK;
}

int32_t check_grad(const muon_token_batch* b, const void* grad, int64_t grad_stride) {
  if (!grad) return MUON_OK;
  if (!aligned(grad, b->dtype == MUON_DTYPE_BF16 ? 2 : 4)) return invalid("grad is not aligned to its type");
  if (grad_stride != 0 && (grad_stride < b->vocab || grad_stride > (1ll << 40)))
    return invalid("grad_stride must be 0 or at least vocab");
  const int64_t stride = b->row_stride ? b->row_stride : b->vocab;
  if (grad == b->logits && (grad_stride ? grad_stride : b->vocab) != stride)
    return invalid("grad in place of the logits must have their row stride");
  return MUON_OK;
}

int32_t check_workspace(const void* ws, size_t bytes, size_t need) {
  if (!ws || bytes < need) return set_error(MUON_ERR_NO_WORKSPACE, "workspace is NULL or too small");
  if (!aligned(ws, 16)) return invalid("workspace must be 16-byte aligned");
  return MUON_OK;
}

int32_t find_device(int* sms) {
  cudaError_t e;
  *sms = device_sms(&e);
  if (e != cudaSuccess) return cuda_error(e);
  if (*sms == 0) return set_error(MUON_ERR_UNSUPPORTED, "libmuon is built for sm_103a");
  return MUON_OK;
}

RowArgs row_args(const muon_token_batch* b) {
  RowArgs a = {};
  a.logits = b->logits;
  a.targets = b->targets;
  a.mask = b->mask;
  a.tokens = b->tokens;
  a.vocab = b->vocab;
  a.stride = b->row_stride ? b->row_stride : b->vocab;
  a.grad_stride = a.vocab;
  a.c = (float)(1.4426950408889634 / (double)b->temperature);
  a.inv_temp = (float)(1.0 / (double)b->temperature);
  a.grad_scale = 1.f;
  return a;
}

template <int kMode>
cudaError_t launch_rows(const RowArgs& a, int32_t dtype, int sms, bool dependent, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  const int grid = (int)(a.tokens < 4ll * sms ? a.tokens : 4ll * sms);
  return dtype == MUON_DTYPE_BF16
             ? launch(row_kernel<__nv_bfloat16, kMode>, grid, kRowThreads, 0, s, 1, dependent, a)
             : launch(row_kernel<float, kMode>, grid, kRowThreads, 0, s, 1, dependent, a);
}

cudaError_t launch_backward(const RowArgs& a, int32_t dtype, int sms, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  const int grid = (int)(a.tokens < 4ll * sms ? a.tokens : 4ll * sms);
  return dtype == MUON_DTYPE_BF16 ? launch(backward_kernel<__nv_bfloat16>, grid, kRowThreads, 0, s, 1, true, a)
                                  : launch(backward_kernel<float>, grid, kRowThreads, 0, s, 1, true, a);
}

// Workspace of the losses: per position 16 bytes (terms; or frame, slope and logp),
// 4 more for a weight, and 4 for each sequence.
size_t round16(size_t v) { return (v + 15) / 16 * 16; }

struct LossSpace {
  float4* terms;
  float2* frame;
  float *slope, *logp, *weight, *inv_count, *pair_loss;
  size_t bytes;
};

LossSpace loss_space(void* ws, int64_t tokens, int64_t n_seqs) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  LossSpace s;
  size_t off = 0;
  s.inv_count = reinterpret_cast<float*>(p + off); off += 16;
  s.terms = reinterpret_cast<float4*>(p + off);
  s.frame = reinterpret_cast<float2*>(p + off);
  s.slope = reinterpret_cast<float*>(p + off + 8 * (size_t)tokens);
  s.logp = reinterpret_cast<float*>(p + off + 12 * (size_t)tokens);
  off += 16 * (size_t)tokens;
  s.weight = reinterpret_cast<float*>(p + off); off += round16(4 * (size_t)tokens);
  s.pair_loss = reinterpret_cast<float*>(p + off); off += round16(4 * (size_t)n_seqs);
  s.bytes = off;
  return s;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

void muon_policy_config_default(muon_policy_config* cfg) {
  if (!cfg) return;
  *cfg = muon_policy_config{};
  cfg->clip_low = cfg->clip_high = 0.2f;
  cfg->grad_scale = 1.f;
  cfg->reduction = MUON_REDUCE_TOKEN_MEAN;
}

void muon_preference_config_default(muon_preference_config* cfg) {
  if (!cfg) return;
  *cfg = muon_preference_config{};
  cfg->beta = 0.1f;
  cfg->grad_scale = 1.f;
}

muon_status muon_loss_workspace_bytes(int64_t tokens, int64_t n_seqs, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  if (tokens < 0 || tokens > (1ll << 31) - 1 || n_seqs < 0 || n_seqs > (1ll << 31) - 1)
    return invalid("tokens and n_seqs must be in [0, 2^31)");
  *bytes = loss_space(nullptr, tokens, n_seqs).bytes;
  return MUON_OK;
}

muon_status muon_token_logprobs(const muon_token_batch* batch, float* logp, void* stream) {
  int32_t st = check_batch(batch);
  if (st != MUON_OK) return st;
  if (batch->tokens == 0) return MUON_OK;
  if (!logp || !aligned(logp, 4)) return invalid("logp is NULL or not aligned");
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  RowArgs a = row_args(batch);
  a.logp = logp;
  const cudaError_t e = launch_rows<kLogp>(a, batch->dtype, sms, false, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

muon_status muon_policy_loss(const muon_token_batch* batch, const muon_policy_config* cfg, const float* old_logp,
                             const float* ref_logp, const float* advantages, const int64_t* seq_offsets,
                             int64_t n_seqs, float* stats, float* logp, void* grad, int64_t grad_stride,
                             void* workspace, size_t workspace_bytes, void* stream) {
  int32_t st = check_batch(batch);
  if (st != MUON_OK) return st;
  muon_policy_config c;
  muon_policy_config_default(&c);
  if (cfg) c = *cfg;
  if (!(c.clip_low >= 0.f && c.clip_low <= 1.f) || !(c.clip_high >= 0.f)) return invalid("clip_low must be in [0, 1], clip_high >= 0");
  if (!std::isfinite(c.kl_beta) || !std::isfinite(c.grad_scale)) return invalid("kl_beta and grad_scale must be finite");
  if (c.reduction < MUON_REDUCE_TOKEN_MEAN || c.reduction > MUON_REDUCE_SUM) return invalid("unknown reduction");
  const bool by_seq = c.reduction == MUON_REDUCE_SEQUENCE_MEAN;
  if (n_seqs < 0 || n_seqs > (1ll << 31) - 2) return invalid("n_seqs must be in [0, 2^31 - 1)");
  if (by_seq && (n_seqs < 1 || !seq_offsets || !aligned(seq_offsets, 8))) return invalid("the sequence mean needs seq_offsets of at least one sequence");
  if (!stats || !aligned(stats, 4) || !aligned(logp, 4)) return invalid("stats is NULL, or stats or logp not aligned");
  if (batch->tokens > 0) {
    if (!old_logp || !advantages || !aligned(old_logp, 4) || !aligned(advantages, 4))
      return invalid("old_logp or advantages is NULL or not aligned");
    if (c.kl_beta != 0.f && (!ref_logp || !aligned(ref_logp, 4))) return invalid("the KL term needs ref_logp");
  }
  if ((st = check_grad(batch, grad, grad_stride)) != MUON_OK) return st;
  const LossSpace ws = loss_space(workspace, batch->tokens, n_seqs);
  if ((st = check_workspace(workspace, workspace_bytes, ws.bytes)) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (by_seq)
    e = launch(weight_kernel, (int)n_seqs + 1, kSmallThreads, 0, s, 1, false, batch->mask, (int64_t)batch->tokens,
               seq_offsets, (int64_t)n_seqs, ws.weight);
  else
    e = launch(count_kernel, 1, kSmallThreads, 0, s, 1, false, batch->mask, (int64_t)batch->tokens,
               (int)(c.reduction == MUON_REDUCE_TOKEN_MEAN), ws.inv_count);
  if (e != cudaSuccess) return cuda_error(e);
  RowArgs a = row_args(batch);
  a.logp = logp;
  a.old_logp = old_logp;
  a.ref_logp = c.kl_beta != 0.f ? ref_logp : nullptr;
  a.adv = advantages;
  a.inv_count = ws.inv_count;
  a.weight = by_seq ? ws.weight : nullptr;
  a.low = (float)(1.0 - (double)c.clip_low);
  a.high = (float)(1.0 + (double)c.clip_high);
  a.beta = c.kl_beta;
  a.grad_scale = c.grad_scale;
  a.grad = grad;
  if (grad_stride) a.grad_stride = grad_stride;
  a.terms = ws.terms;
  if ((e = launch_rows<kPolicy>(a, batch->dtype, sms, true, s)) != cudaSuccess) return cuda_error(e);
  e = launch(stats_kernel, 1, kSmallThreads, 0, s, 1, true, (const float4*)ws.terms, (int64_t)batch->tokens, stats);
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

muon_status muon_preference_loss(const muon_token_batch* batch, const muon_preference_config* cfg,
                                 const float* ref_logp, const int64_t* seq_offsets, int64_t n_pairs, float* loss,
                                 float* margins, float* seq_logp, void* grad, int64_t grad_stride, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  int32_t st = check_batch(batch);
  if (st != MUON_OK) return st;
  muon_preference_config c;
  muon_preference_config_default(&c);
  if (cfg) c = *cfg;
  if (!(c.beta > 0.f) || std::isinf(c.beta)) return invalid("beta must be finite and > 0");
  if (!(c.label_smoothing >= 0.f && c.label_smoothing <= 1.f)) return invalid("label_smoothing must be in [0, 1]");
  if (!std::isfinite(c.grad_scale)) return invalid("grad_scale must be finite");
  if (c.length_normalize != 0 && c.length_normalize != 1) return invalid("length_normalize must be 0 or 1");
  if (n_pairs < 0 || n_pairs > (1ll << 30) - 1) return invalid("n_pairs must be in [0, 2^30)");
  if (!loss || !aligned(loss, 4) || !aligned(margins, 4) || !aligned(seq_logp, 4))
    return invalid("loss is NULL, or loss, margins or seq_logp not aligned");
  if (n_pairs > 0 && (!ref_logp || !seq_offsets || !aligned(ref_logp, 4) || !aligned(seq_offsets, 8)))
    return invalid("ref_logp or seq_offsets is NULL or not aligned");
  if ((st = check_grad(batch, grad, grad_stride)) != MUON_OK) return st;
  const LossSpace ws = loss_space(workspace, batch->tokens, 2 * n_pairs);
  if ((st = check_workspace(workspace, workspace_bytes, ws.bytes)) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  RowArgs a = row_args(batch);
  a.logp = ws.logp;
  a.frame = ws.frame;
  a.slope = ws.slope;
  a.grad_scale = c.grad_scale;
  a.grad = grad;
  if (grad_stride) a.grad_stride = grad_stride;
  cudaError_t e = launch_rows<kForward>(a, batch->dtype, sms, false, s);
  if (e != cudaSuccess) return cuda_error(e);
  if (n_pairs > 0) {
    PairArgs p;
    p.mask = batch->mask;
    p.logp = ws.logp;
    p.ref = ref_logp;
    p.offsets = seq_offsets;
    p.tokens = batch->tokens;
    p.n_pairs = n_pairs;
    p.beta = c.beta;
    p.smooth = c.label_smoothing;
    p.mean = c.length_normalize;
    p.margins = margins;
    p.seq_logp = seq_logp;
    p.pair_loss = ws.pair_loss;
    p.slope = ws.slope;
    if ((e = launch(pair_kernel, (int)n_pairs, kSmallThreads, 0, s, 1, batch->tokens > 0, p)) != cudaSuccess)
      return cuda_error(e);
  }
  e = launch(pair_mean_kernel, 1, kSmallThreads, 0, s, 1, false, (const float*)ws.pair_loss, (int64_t)n_pairs, loss);
  if (e != cudaSuccess) return cuda_error(e);
  if (grad && (e = launch_backward(a, batch->dtype, sms, s)) != cudaSuccess) return cuda_error(e);
  return MUON_OK;
}

}  // extern "C"
