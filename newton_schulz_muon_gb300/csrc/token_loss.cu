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
// The sum over a row leaves the target out: with m the largest of the other logits,
//   S = sum_{j != y} e^(z_j - m),   x = z_y - m,
//   logp = -log1p(S e^-x) where x >= 0, else x - log(S + e^x),
// which keeps logp's digits (and those of 1 - p_y) where the target is nearly certain.
// Exponentials are taken in base 2, 2^(c (z - m)) with c = log2(e) / temperature: the
// difference is formed first, so that the largest term is exactly 1 and logits at the
// type's limits do not overflow.  A rounded c would shift every row's sum the same way,
// which the sum over a sequence adds up.  fp32 logits, which HBM delivers more slowly
// than the SMs can take them, use c as two floats; for bf16 logits, where every
// instruction counts, the eight elements of a 16-byte unit take the two floats next to c
// in the proportion that gives c in the mean (4096 x 131072 policy loss, when this was
// chosen: 0.400 ms with two floats, 0.370 ms with one; HBM's time is 0.285 ms).
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
#include "rows.cuh"

namespace muon {
namespace {

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
  const int32_t* order;   // live rows, then masked ones; null: by the mask as they come
  const int32_t* n_live;
  int64_t tokens, vocab, stride, grad_stride;
  float c_hi, c_lo;      // log2(e) / temperature = c_hi + c_lo, c_lo > 0
  float2 c_mix[4];       // the floats next to it, for the four pairs of a unit of bf16
  float inv_temp;        // 1 / temperature, and
  float inv_hi, inv_lo;  // in two floats, inv_lo > 0
  float* logp;           // or null
  float2* frame;         // kForward: (m, sum over the whole row) of each row
  float* slope;          // kForward: cleared for rows of no sequence
  // kPolicy
  const float* old_logp;
  const float* ref_logp; // or null
  const float* adv;
  const float* inv_count; // token mean and sum: one weight for all positions
  const float* weight;    // sequence mean: [tokens]
  float low, high, beta, grad_scale;
  void* grad;             // or null
  double* partials;       // 4 for each cluster: its rows' sums of w (-s + beta k), w (-s), w k, w [clipped]
  unsigned* ticket;       // zeroed by the kernel before
  float* stats;
  // shape of the launch
  int32_t log_cluster;    // 2^log_cluster CTAs a row
  int32_t stage_vecs;     // 16-byte units of one ring stage
};

// 2^(c (z - m)) of one value, and of elements 2 i and 2 i + 1 of a unit.  c_lo > 0, so that
// a difference of -inf stays one.
template <typename T>
struct Expo {
  float m, c_hi, c_lo;  // m finite or +inf
  F2 mix[4];
  __device__ __forceinline__ Expo(const RowArgs& a, float largest) : c_hi(a.c_hi), c_lo(a.c_lo) {
    frame(largest);
    if (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        mix[i] = make_f2(a.c_mix[i].x, a.c_mix[i].y);
        asm volatile("" : "+l"(mix[i].v));  // in registers: packed products take no other operands
      }
    }
  }
  // With no finite logit but the target's, any finite m gives the right zeros.
  __device__ __forceinline__ void frame(float largest) { m = largest == -INFINITY ? 0.f : largest; }
  __device__ __forceinline__ float one(float z) const {
    const float d = z - m;
    return ex2(__fmaf_rn(d, c_hi, d * c_lo));
  }
  __device__ __forceinline__ float2 two(const float* v, int i) const {
    const F2 d = add2(make_f2(v[2 * i], v[2 * i + 1]), make_f2(-m, -m));
    const float2 u = split(sizeof(T) == 2 ? mul2(d, mix[i]) : fma2(d, make_f2(c_hi, c_hi), mul2(d, make_f2(c_lo, c_lo))));
    return make_float2(ex2(u.x), ex2(u.y));
  }
};

// A partial sum of exponentials: s = sum_j 2^(c (z_j - m)), m the largest z so far
// (-inf: nothing yet, or only logits of -inf).
struct Sum {
  float m, s;
};

// Factor that takes a sum from the frame of m to that of the larger `to`.
__device__ __forceinline__ float reframe(const RowArgs& a, float m, float to) {
  if (m == to) return 1.f;  // both -inf among them
  const float d = m - to;   // a NaN stays one; `to` is not -inf
  return ex2(__fmaf_rn(d, a.c_hi, d * a.c_lo));
}

__device__ __forceinline__ Sum merge(const RowArgs& a, const Sum& x, const Sum& y) {
  Sum r;
  r.m = fmaxf(x.m, y.m);
  r.s = x.s * reframe(a, x.m, r.m) + y.s * reframe(a, y.m, r.m);
  return r;
}

// Merges the lanes' sums: the largest m first, then one factor a lane.
__device__ __forceinline__ Sum warp_merge(const RowArgs& a, const Sum& t) {
  Sum r;
  r.m = warp_max(t.m);
  r.s = t.s * reframe(a, t.m, r.m);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r.s += __shfl_xor_sync(0xFFFFFFFFu, r.s, o);
  return r;
}

// G 16-byte units of a row.
template <typename T, int G>
__device__ __forceinline__ void add_units(const RowArgs& a, Expo<T>& x, Sum& t, const uint4 (&w)[G]) {
  constexpr int N = Vec<T>::N;
  const float m = Vec<T>::max(w);
  if (!(m <= t.m)) {
    t.s *= reframe(a, t.m, m);
    t.m = m;
    x.frame(m);
  }
  F2 s0 = make_f2(0.f, 0.f), s1 = make_f2(0.f, 0.f);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float v[N];
    Vec<T>::unpack(w[g], v);
#pragma unroll
    for (int i = 0; i < N / 2; i += 2) {
      const float2 e0 = x.two(v, i), e1 = x.two(v, i + 1);
      s0 = add2(s0, make_f2(e0.x, e0.y));
      s1 = add2(s1, make_f2(e1.x, e1.y));
    }
  }
  const float2 r = split(add2(s0, s1));
  t.s += r.x + r.y;
}

__device__ __forceinline__ void add_value(const RowArgs& a, Sum& t, float v) {
  if (!(v <= t.m)) {
    t.s *= reframe(a, t.m, v);
    t.m = v;
  }
  if (v != -INFINITY) t.s += reframe(a, v, t.m);
}

// A row's log-probability, and the sum over the whole row in the frame of m.
struct Prob {
  float logp, s;
};

__device__ __forceinline__ Prob row_prob(const RowArgs& a, const Sum& t, float zy) {
  const float d = zy - t.m;
  const float x = __fmaf_rn(d, a.inv_hi, d * a.inv_lo);
  const float e = expf(x);
  Prob p;
  p.s = t.s + e;
  const float s = t.s > 1.f ? __fmaf_rn(t.s - 1.f, kExpLow, t.s) : t.s;  // a NaN stays one
  p.logp = x >= 0.f ? 0.f - log1pf(s * expf(-x)) : x - logf(s + e);
  if (zy == INFINITY) p.logp = NAN;
  return p;
}

// The gradient's elements: factor 2^(c (z_j - m)), and at_y at the target.  Both are zero
// for a row that does not move the loss: its elements are then, whatever its logits.
struct Factor {
  float m, factor, at_y;
  __device__ __forceinline__ bool none() const { return factor == 0.f && at_y == 0.f; }
};

__device__ __forceinline__ Factor row_factor(const RowArgs& a, float m, float s, float logp, float slope) {
  const float f = slope * a.grad_scale * a.inv_temp;
  return f == 0.f ? Factor{m, 0.f, 0.f} : Factor{m, -f / s, -f * expm1f(logp)};
}

// A position's scalars.
struct Position {
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

// ---------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------
// The 16-byte units that lie whole in a row, and the elements around them.
struct Row {
  int head;  // elements before the first unit
  int units;
  int tail;  // first element after the last unit
};

template <typename T>
__device__ __forceinline__ Row row_of(const T* z, int64_t vocab) {
  Row r;
  r.head = min((int)vocab, (int)((-reinterpret_cast<uint64_t>(z) & 15) / sizeof(T)));
  r.units = (int)(vocab - r.head) / Vec<T>::N;
  r.tail = r.head + r.units * Vec<T>::N;
  return r;
}

// The element of a row that lane `lane` of its edge warp looks after, or -1: lanes 0-7
// those before the first unit, 8-15 those after the last.
__device__ __forceinline__ int edge_of(const Row& r, int64_t vocab, int lane) {
  if (lane < 8) return lane < r.head ? lane : -1;
  return lane < 16 && r.tail + lane - 8 < vocab ? r.tail + lane - 8 : -1;
}

template <typename T>
__device__ __forceinline__ uint4 scaled_unit(const uint4& w, const Expo<T>& x, float factor) {
  constexpr int N = Vec<T>::N;
  float v[N];
  Vec<T>::unpack(w, v);
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float2 e = x.two(v, i);
    const float2 r = split(mul2(make_f2(e.x, e.y), make_f2(factor, factor)));
    v[2 * i] = r.x;
    v[2 * i + 1] = r.y;
  }
  return Vec<T>::pack(v);
}

// A unit of the gradient: one store where the gradient's row is aligned as the logits'
// row is, else its elements one by one.
template <typename T>
__device__ __forceinline__ void store_unit(T* g, const uint4& w, bool whole) {
  if (whole) {
    *reinterpret_cast<uint4*>(g) = w;
  } else {
    float v[Vec<T>::N];
    Vec<T>::unpack(w, v);  // exact both ways
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) Vec<T>::store(g + i, v[i]);
  }
}

template <typename T>
__device__ __forceinline__ bool aligned_unit(const T* g) {
  return (reinterpret_cast<uint64_t>(g) & 15) == 0;
}

constexpr int kMaxRowThreads = 512;  // that hold units of a row, beside the finishing warp
constexpr int kMaxCluster = 8;
constexpr int kInfo = 32;    // rows whose places and scalars a CTA holds at a time
constexpr int kSlots = 4;    // rows whose partial sums may be on their way
constexpr int kGroup = 4;    // 16-byte units a thread takes at a time
constexpr int64_t kKeptBytes = 80ll << 20;  // of logits that L2 holds from the forward pass to the backward pass

// A CTA's sums of its rows' terms, and whether it is the last to have them.
struct StatsShared {
  double sum[4];
  int32_t last;
};

// Shared memory beside the ring of rows: the partial sums of kSlots rows follow it, from
// every warp of the cluster.
struct RowShared {
  uint64_t full[kSlots];   // a slot has every partial sum of its row
  StatsShared stats;
  Factor factor[kSlots];   // by the row's slot
  // live rows by index modulo kInfo
  const uint4* src[kInfo]; // this CTA's units of the logits
  void* dst[kInfo];        // the gradient's elements there
  int32_t units[kInfo];    // how many; negative (~units): the gradient is not aligned there
  int32_t row[kInfo];
  int32_t unit[kInfo];     // the target's unit in this CTA's part; -1: elsewhere
  int32_t elem[kInfo];     // its element there + 16 times the thread that has it; with unit = -2 the edge lane
  float zy[kInfo];
  float old_logp[kInfo], ref[kInfo], adv[kInfo], w[kInfo];
  uint32_t live;
};

// Barriers 1 and 2 (by the row's parity): the finishing warp has written a row's factor.
__device__ __forceinline__ void factor_sync(int par, uint32_t count) {
  if (par) asm volatile("bar.sync 2, %0;" ::"r"(count) : "memory");
  else asm volatile("bar.sync 1, %0;" ::"r"(count) : "memory");
}
__device__ __forceinline__ void factor_arrive(int par, uint32_t count) {
  if (par) asm volatile("bar.arrive 2, %0;" ::"r"(count) : "memory");
  else asm volatile("bar.arrive 1, %0;" ::"r"(count) : "memory");
}

// Writes a partial sum to a slot of CTA `rank` of the cluster and counts it there.  The
// asynchronous store belongs to cluster launches; a CTA alone writes its own memory.
__device__ __forceinline__ void send(Sum* slot, uint64_t* full, int ncta, uint32_t rank, const Sum& v) {
  if (ncta == 1) {
    *slot = v;
    mbar_arrive(full);
    return;
  }
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(
                   mapa_shared(slot, rank)),
               "r"(__float_as_uint(v.m)), "r"(__float_as_uint(v.s)), "r"(mapa_shared(full, rank))
               : "memory");
}

// Sums of rows' terms, carried with their rounding errors.
struct Terms {
  float hi[4] = {0.f, 0.f, 0.f, 0.f}, lo[4] = {0.f, 0.f, 0.f, 0.f};
  __device__ __forceinline__ void add(const float4& t) {
    const float v[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float sum, err;
      two_sum(hi[k], v[k], sum, err);
      hi[k] = sum;
      lo[k] += fabsf(sum) < INFINITY ? err : 0.f;
    }
  }
  __device__ __forceinline__ void get(double* sum) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k] = (double)hi[k] + (double)lo[k];
  }
};

// The CTA's sums into the partials; the last of `n` CTAs to come adds all of them, in
// their order: kEach sums a warp, side by side (4 / kEach warps at least).
template <int kEach>
__device__ __forceinline__ void finish_stats(const RowArgs& a, StatsShared& sh, int64_t part, int64_t n) {
  constexpr int kWarps = 4 / kEach;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (threadIdx.x == 0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) a.partials[4 * part + k] = sh.sum[k];
    __threadfence();
    sh.last = atomicAdd(a.ticket, 1u) == (unsigned)n - 1;
  }
  __syncthreads();
  if (sh.last && warp < kWarps) {
    __threadfence();
    double sum[kEach] = {};
    for (int64_t k = lane; k < n; k += 32) {
#pragma unroll
      for (int j = 0; j < kEach; ++j) sum[j] += __ldcg(a.partials + 4 * k + warp + kWarps * j);
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum[j] += __shfl_xor_sync(0xFFFFFFFFu, sum[j], o);
      if (lane == 0) a.stats[warp + kWarps * j] = (float)sum[j];
    }
  }
}

// A cluster of 1 to 8 CTAs takes one row at a time and keeps it in shared memory between
// the sum and the gradient, so that every logit is read from HBM once.  Each thread copies
// its own 16-byte units into a ring of kStages rows (cp.async) and is the only one to read
// them, so that only the sums cross threads: every warp writes its partial sum to all CTAs
// of the cluster, and a warp of each CTA that holds no units forms the row's result from
// them.  While it does, the others write the gradient of the row before, whose stage then
// takes the row kStages - 1 further on, and sum the next row.
//
// The sums travel as asynchronous stores that count on a barrier of the receiver, so that no
// store of a gradient is waited for.  A warp sends row i after it has had the result of row
// i - 2 from its own CTA's finishing warp; that took the sums of row i - 2 from every CTA,
// which were sent after the results of row i - 4 there: slot i - 4 = i mod kSlots has been
// read in every CTA.
//
// Bound by HBM, and nearly as much by the SM's issue slots (55% taken on 608 x 131072 bf16
// rows: 14.5 instructions a logit, 9 of them the two exponentials, their unpacking and
// packing; the rest a row's fixed cost over 8 units a thread), which is why the warps read
// a row's places from shared memory and test nothing inside their loops.  4096 x 131072
// bf16, a fifth masked: 0.309 ms, 6.3 TB/s of compulsory traffic (with the row read twice
// from memory, stream_kernel: 0.483 ms; with 384 or 256 threads: 0.320 and 0.337 ms; when
// asynchronous stores took the place of a cluster barrier a row, 0.416 ms became 0.365 ms).
// 6250 x 32000 fp32: 0.245 ms, 5.9 TB/s.
template <typename T, int kMode, int kStages>
__global__ void __launch_bounds__(kMaxRowThreads + 32) row_kernel(const __grid_constant__ RowArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint4 ring[];
  RowShared& sh = *reinterpret_cast<RowShared*>(ring + (size_t)kStages * a.stage_vecs);
  const int tid = threadIdx.x, all = blockDim.x, nt = all - 32, lane = tid & 31, warp = tid >> 5, warps = all >> 5;
  const int ncta = 1 << a.log_cluster;
  const int rank = ncta > 1 ? (int)cluster_ctarank() : 0;
  const int64_t cid = blockIdx.x >> a.log_cluster, n_clusters = gridDim.x >> a.log_cluster;
  const bool has_grad = kMode == kPolicy && a.grad != nullptr;
  const bool finisher = warp == warps - 1;
  const T* const logits = reinterpret_cast<const T*>(a.logits);
  T* const grads = reinterpret_cast<T*>(a.grad);
  const int64_t my_rows = a.tokens > cid ? (a.tokens - cid + n_clusters - 1) / n_clusters : 0;
  Sum* const slots = reinterpret_cast<Sum*>(&sh + 1);  // [kSlots][ncta][warps]
  Terms acc;  // of the finishing warp

  auto part_of = [&](const Row& row, int& v0) {  // this CTA's units of a row
    const int per = (row.units + ncta - 1) >> a.log_cluster;
    v0 = rank * per;
    return max(0, min(per, row.units - v0));
  };

  griddep_launch_dependents();
  // a cluster's sums are counted in bytes, one CTA's (no cluster launch) in arrivals
  if (tid < kSlots) mbar_init(&sh.full[tid], ncta > 1 ? 1 : warps);
  fence_mbarrier_init();
  cluster_sync();

  // The cluster's n live rows.  With the list of all live rows (or no mask) they are its
  // entries cid, cid + n_clusters, ...; without it there are at most kInfo rows, live ones
  // and then the others in sh.row.
  int n;
  int64_t n_live = a.tokens;
  const bool listed = a.order != nullptr || a.mask == nullptr;
  auto row_at = [&](int64_t i) {
    const int64_t p = cid + i * n_clusters;
    return a.order ? __ldcg(a.order + p) : (int32_t)p;
  };
  if (listed) {
    if (a.order) {
      griddep_wait();
      n_live = __ldcg(a.n_live);
    }
    n = (int)(n_live > cid ? (n_live - cid + n_clusters - 1) / n_clusters : 0);
    if (tid < kInfo && tid < n) sh.row[tid] = row_at(tid);
  } else {
    if (warp == 0) {
      const bool live = tid < my_rows && a.mask[cid + tid * n_clusters] != 0;
      const unsigned bits = __ballot_sync(0xFFFFFFFFu, live);
      const int before = __popc(bits & ((1u << lane) - 1));
      if (tid < my_rows) sh.row[live ? before : (int)my_rows - 1 - (tid - before)] = (int32_t)(cid + tid * n_clusters);
      if (lane == 0) sh.live = bits;
    }
    __syncthreads();
    n = __popc(sh.live);
  }
  auto put_place = [&](int i, int64_t t) {
    const T* z = logits + t * a.stride;
    T* g = grads + t * a.grad_stride;
    const Row row = row_of(z, a.vocab);
    int v0;
    const int cnt = part_of(row, v0);
    const int64_t first = row.head + (int64_t)v0 * N;
    const int k = i % kInfo;
    sh.row[k] = (int32_t)t;
    sh.src[k] = reinterpret_cast<const uint4*>(z + first);
    sh.dst[k] = g + first;
    sh.units[k] = !has_grad || aligned_unit(g + first) ? cnt : ~cnt;
  };
  if (warp == 0) {
    __syncwarp();
    if (lane < n) put_place(lane, sh.row[lane]);
  }
  __syncthreads();

  // Starts the copy of live row i; the finishing warp's lanes get their elements of it.
  auto issue = [&](int i, int stage) {
    float e = -INFINITY;
    if (i < n) {
      const int k = i % kInfo;
      if (finisher) {
        const T* z = logits + sh.row[k] * a.stride;
        const int at = rank == 0 ? edge_of(row_of(z, a.vocab), a.vocab, lane) : -1;
        if (at >= 0) e = Vec<T>::load(z + at);
      } else {
        const int cnt = max(sh.units[k], ~sh.units[k]);
        const uint4* src = sh.src[k];
        uint4* dst = ring + (size_t)stage * a.stage_vecs;
        for (int l = tid; l < cnt; l += nt) cp_async_16(dst + l, src + l);
      }
    }
    cp_async_commit();
    return e;
  };
  float edge[kStages];  // of rows i - 1, i, i + 1, ...
  edge[0] = -INFINITY;
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) edge[i + 1] = issue(i, i);

  // A row's scalars, in three steps whose loads depend on one another.
  struct Info {
    int32_t row;
    int64_t y;
    float zy, old_logp, ref, adv, w;
  };
  auto load_scalars = [&](Info& f) {
    f.y = a.targets[f.row];
    if (kMode == kPolicy) {
      f.old_logp = a.old_logp[f.row];
      f.ref = a.ref_logp ? a.ref_logp[f.row] : 0.f;
      f.adv = a.adv[f.row];
    }
  };
  auto load_target = [&](Info& f) {
    f.zy = f.y >= 0 && f.y < a.vocab ? Vec<T>::load(logits + f.row * a.stride + f.y) : NAN;
  };
  auto load_weight = [&](Info& f) {
    if (kMode == kPolicy) f.w = a.weight ? __ldcg(a.weight + f.row) : __ldcg(a.inv_count);
  };
  auto put_scalars = [&](int i, const Info& f) {
    const int k = i % kInfo;
    const Row row = row_of(logits + f.row * a.stride, a.vocab);
    int v0;
    const int cnt = part_of(row, v0);
    int unit = -1, elem = 0;
    if (f.y >= row.head && f.y < row.tail) {
      const int u = ((int)f.y - row.head) / N - v0;
      if (u >= 0 && u < cnt) {
        unit = u;
        elem = ((int)f.y - row.head) % N + 16 * (u % nt);
      }
    } else if (f.y >= 0 && f.y < a.vocab) {
      unit = -2;
      elem = (int)(f.y < row.head ? f.y : 8 + f.y - row.tail);
    }
    sh.unit[k] = unit;
    sh.elem[k] = elem;
    sh.zy[k] = f.zy;
    if (kMode == kPolicy) {
      sh.old_logp[k] = f.old_logp;
      sh.ref[k] = f.ref;
      sh.adv[k] = f.adv;
      sh.w[k] = f.w;
    }
  };
  Info info = {};
  const bool mine = tid < kInfo && tid < n;
  if (mine) {
    info.row = sh.row[tid];
    load_scalars(info);
    load_target(info);
  }
  griddep_wait();
  if (mine) {
    load_weight(info);
    put_scalars(tid, info);
  }
  __syncthreads();

  bool arrived = true;
  if (finisher) {
    for (int i = 0; i < n; ++i) {
      const int par = i & 1, k = i % kInfo, slot = i % kSlots;
      const int64_t pos = sh.row[k];
      // the row's elements outside whole units are this warp's part of the sum
      const bool at_edge = sh.unit[k] == -2 && sh.elem[k] == lane;
      Sum t{-INFINITY, 0.f};
      if (!at_edge) add_value(a, t, edge[1]);
      t = warp_merge(a, t);
      if (ncta > 1 && lane == 0) mbar_arrive_expect_tx(&sh.full[slot], ncta * warps * (uint32_t)sizeof(Sum));
      if (lane < ncta) send(slots + (slot * ncta + rank) * warps + warp, &sh.full[slot], ncta, lane, t);
      // The 16 rows after this row's 16, a step a row, into the half that held the 16 before:
      // their gradients have been written once the sums of the row two before this are here.
      const int step = i & (kInfo / 2 - 1), base = i - step + kInfo / 2;
      if (base >= kInfo && base < n) {
        const bool in = lane < kInfo / 2 && base + lane < n;
        if (step == 0 && in) info.row = row_at(base + lane);
        if (step == 1 && in) load_scalars(info);
        if (step == 2 && in) load_target(info);
        if (step == 3 && in) load_weight(info);
        if (step == 4 && in) {
          put_place(base + lane, info.row);
          put_scalars(base + lane, info);
        }
      }
      __syncwarp();
      arrived = arrived && mbar_wait(&sh.full[slot], (uint32_t)(i / kSlots) & 1, nullptr, nullptr);
      arrived = __all_sync(0xFFFFFFFFu, arrived);
      // every warp of every CTA, in the same order in each
      t = Sum{-INFINITY, 0.f};
      for (int j = lane; j < ncta * warps; j += 32) t = merge(a, t, slots[slot * ncta * warps + j]);
      t = warp_merge(a, t);
      if (!arrived) t.s = NAN;  // a wait ran out: the results say so
      const Prob p = row_prob(a, t, sh.zy[k]);
      const bool writer = rank == 0 && lane == 0;
      if (writer && a.logp) a.logp[pos] = p.logp;
      if (kMode == kForward && writer) {
        a.frame[pos] = make_float2(t.m, p.s);
        a.slope[pos] = 0.f;
      }
      if (kMode == kPolicy) {
        const Position at{sh.old_logp[k], sh.ref[k], sh.adv[k], sh.w[k]};
        const Outcome o = policy_terms(a, at, p.logp);
        acc.add(o.terms);
        if (has_grad) {
          const Factor f = row_factor(a, t.m, p.s, p.logp, o.slope);
          if (lane == 0) sh.factor[slot] = f;
          T* g = grads + pos * a.grad_stride;
          const int e = rank == 0 ? edge_of(row_of(logits + pos * a.stride, a.vocab), a.vocab, lane) : -1;
          __syncwarp();
          factor_arrive(par, all);
          if (e >= 0) Vec<T>::store(g + e, f.none() ? 0.f : at_edge ? f.at_y : f.factor * Expo<T>(a, f.m).one(edge[1]));
        }
      }
      if (!has_grad) factor_arrive(par, all);  // the other warps keep the row's distance all the same
#pragma unroll
      for (int j = 0; j + 1 < kStages; ++j) edge[j] = edge[j + 1];
      edge[kStages - 1] = issue(i + kStages - 1, 0);
    }
  } else {
    int stage = 0, before = kStages - 1;  // of rows i and i - 1
    Expo<T> x(a, 0.f);
    for (int i = 0; i <= n; ++i) {
      if (i < n) {
        // the row's sum without its target: this thread's part, then the warp's
        cp_async_wait<kStages - 2>();
        const int k = i % kInfo, slot = i % kSlots;
        const int cnt = max(sh.units[k], ~sh.units[k]);
        uint4* src = ring + (size_t)stage * a.stage_vecs;
        const int unit = sh.unit[k], elem = sh.elem[k];
        if (unit >= 0 && elem >> 4 == tid) {  // the target leaves the sum
          uint4 w = src[unit];
          drop<T>(w, Vec<T>::mask_of(elem & 15));
          src[unit] = w;
        }
        Sum t{-INFINITY, 0.f};
        x.frame(t.m);
        int l = tid;
        for (; l + (kGroup - 1) * nt < cnt; l += kGroup * nt) {
          uint4 w[kGroup];
#pragma unroll
          for (int g = 0; g < kGroup; ++g) w[g] = src[l + g * nt];
          add_units<T>(a, x, t, w);
        }
        if (l + (kGroup - 2) * nt < cnt) {  // all but one of a group
          uint4 w[kGroup];
#pragma unroll
          for (int g = 0; g < kGroup - 1; ++g) w[g] = src[l + g * nt];
          w[kGroup - 1] = make_uint4(Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest);
          add_units<T>(a, x, t, w);
          l = cnt;
        }
        for (; l < cnt; l += nt) {
          const uint4 w[1] = {src[l]};
          add_units<T>(a, x, t, w);
        }
        t = warp_merge(a, t);
        if (lane < ncta) send(slots + (slot * ncta + rank) * warps + warp, &sh.full[slot], ncta, lane, t);
      }
      if (i > 0 && !has_grad) factor_sync((i - 1) & 1, all);
      if (i > 0 && has_grad) {
        // the gradient of the row before
        const int k = (i - 1) % kInfo;
        const bool whole = sh.units[k] >= 0;
        const int cnt = max(sh.units[k], ~sh.units[k]);
        const uint4* src = ring + (size_t)before * a.stage_vecs;
        T* g = static_cast<T*>(sh.dst[k]);
        factor_sync((i - 1) & 1, all);
        const Factor f = sh.factor[(i - 1) % kSlots];
        x.frame(f.m);
        int l = tid;
        if (f.none()) {
          for (; l < cnt; l += nt) store_unit(g + (int64_t)l * N, make_uint4(0, 0, 0, 0), whole);
        }
        if (whole) {
          for (; l + (kGroup - 1) * nt < cnt; l += kGroup * nt) {
            uint4 w[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) w[j] = src[l + j * nt];
#pragma unroll
            for (int j = 0; j < kGroup; ++j)
              store_unit(g + (int64_t)(l + j * nt) * N, scaled_unit<T>(w[j], x, f.factor), true);
          }
        }
        for (; l < cnt; l += nt) store_unit(g + (int64_t)l * N, scaled_unit<T>(src[l], x, f.factor), whole);
        const int unit = sh.unit[k], elem = sh.elem[k];
        if (unit >= 0 && elem >> 4 == tid) Vec<T>::store(g + (int64_t)unit * N + (elem & 15), f.at_y);
      }
      if (i < n) issue(i + kStages - 1, before);
      before = stage;
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  }

  // masked rows
  for (int64_t i = n; i < my_rows; ++i) {
    const int64_t t = listed ? row_at(i) : sh.row[i];
    if (rank == 0 && tid == 0) {
      if (a.logp) a.logp[t] = 0.f;
      if (kMode == kForward) a.slope[t] = 0.f;
    }
    if (!has_grad) continue;
    T* g = grads + t * a.grad_stride;
    const Row row = row_of(g, a.vocab);
    if (finisher) {
      const int e = rank == 0 ? edge_of(row, a.vocab, lane) : -1;
      if (e >= 0) Vec<T>::store(g + e, 0.f);
    } else {
      int v0;
      const int cnt = part_of(row, v0);
      uint4* dst = reinterpret_cast<uint4*>(g + row.head) + v0;
      for (int l = tid; l < cnt; l += nt) dst[l] = make_uint4(0, 0, 0, 0);
    }
  }
  if (kMode == kForward && blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  if (kMode == kPolicy && rank == 0) {
    if (finisher && lane == 0) acc.get(sh.stats.sum);
    finish_stats<1>(a, sh.stats, cid, n_clusters);
  }
  cluster_sync();  // no CTA of the cluster ends before the others have all it sent
}

// Rows of at most 32 kUnits 16-byte units (and the elements around them): one warp holds a
// row in registers, and nothing is shared between warps.  The row's largest logit is known
// before the first exponential.  Bound by the latency of a row's loads (16 warps an SM, 122
// registers) and by issue (53%): 20011 x 4099 bf16, a tenth masked, 0.062 ms, 5.0 TB/s of
// compulsory traffic; with a CTA a row (row_kernel) 0.094 ms; with the next row copied to
// shared memory meanwhile 0.073 ms (rows of 1024 to 4000 logits 0 to 12% slower so, too).
constexpr int kWarpRowThreads = 256;
constexpr int kWarpRowWarps = kWarpRowThreads / 32;

template <typename T, int kMode, int kUnits>
__global__ void __launch_bounds__(kWarpRowThreads, kUnits > 4 ? 2 : 3) warp_row_kernel(const __grid_constant__ RowArgs a) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool has_grad = kMode == kPolicy && a.grad != nullptr;
  const int64_t warps = (int64_t)gridDim.x * kWarpRowWarps;
  Terms acc;
  griddep_launch_dependents();
  bool waited = false;
  const int64_t first = (int64_t)blockIdx.x * kWarpRowWarps + warp;
  bool next_live = first < a.tokens && (a.mask == nullptr || a.mask[first] != 0);
  int64_t next_y = first < a.tokens ? a.targets[first] : 0;
  for (int64_t t = first; t < a.tokens; t += warps) {
    // the next row's mask and target are on their way while this row is worked on
    const bool live = next_live;
    const int64_t y = next_y;
    if (t + warps < a.tokens) {
      next_live = a.mask == nullptr || a.mask[t + warps] != 0;
      next_y = a.targets[t + warps];
    }
    if (!waited && !live) {
      griddep_wait();
      waited = true;
    }
    const T* z = reinterpret_cast<const T*>(a.logits) + t * a.stride;
    T* g = reinterpret_cast<T*>(a.grad) + t * a.grad_stride;
    if (!live) {
      if (lane == 0 && a.logp) a.logp[t] = 0.f;
      if (kMode == kForward && lane == 0) a.slope[t] = 0.f;
      if (has_grad) {
        const Row row = row_of(g, a.vocab);
        uint4* dst = reinterpret_cast<uint4*>(g + row.head);
        for (int u = lane; u < row.units; u += 32) dst[u] = make_uint4(0, 0, 0, 0);
        const int e = edge_of(row, a.vocab, lane);
        if (e >= 0) Vec<T>::store(g + e, 0.f);
      }
      continue;
    }
    const Row row = row_of(z, a.vocab);
    const uint4* src = reinterpret_cast<const uint4*>(z + row.head);
    uint4 w[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k)
      w[k] = k * 32 + lane < row.units ? src[k * 32 + lane]
                                       : make_uint4(Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest);
    const int edge = edge_of(row, a.vocab, lane);
    const float zedge = edge >= 0 ? Vec<T>::load(z + edge) : -INFINITY;
    const bool in = y >= 0 && y < a.vocab;
    const float zy = in ? Vec<T>::load(z + y) : NAN;
    Position at{0.f, 0.f, 0.f, 0.f};
    if (kMode == kPolicy) {
      at.old_logp = a.old_logp[t];
      if (a.ref_logp) at.ref = a.ref_logp[t];
      at.adv = a.adv[t];
    }
    if (!waited) {  // the first row's loads are under way
      griddep_wait();
      waited = true;
    }
    if (kMode == kPolicy) {
      at.w = a.weight ? __ldcg(a.weight + t) : __ldcg(a.inv_count);
    }
    const int unit = in && y >= row.head && y < row.tail ? ((int)y - row.head) / N : -1;
    const int owned = unit >= 0 && (unit & 31) == lane ? unit >> 5 : -1;
    const uint4 bits = Vec<T>::mask_of(((int)y - row.head) % N);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      int mine = owned;
      asm volatile("" : "+r"(mine));  // one test a register, not an indexed array
      if (mine == k) drop<T>(w[k], bits);  // the target leaves the sum
    }
    const bool at_edge = edge >= 0 && edge == y;
    const float others = at_edge ? -INFINITY : zedge;
    Sum s;
    s.m = warp_max(fmaxf(Vec<T>::max(w), others));
    const Expo<T> x(a, s.m);
    F2 s0 = make_f2(x.one(others), 0.f), s1 = make_f2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      float v[N];
      Vec<T>::unpack(w[k], v);
#pragma unroll
      for (int i = 0; i < N / 2; i += 2) {
        const float2 e0 = x.two(v, i), e1 = x.two(v, i + 1);
        s0 = add2(s0, make_f2(e0.x, e0.y));
        s1 = add2(s1, make_f2(e1.x, e1.y));
      }
    }
    const float2 r = split(add2(s0, s1));
    s.s = warp_sum(r.x + r.y);
    const Prob p = row_prob(a, s, zy);
    if (lane == 0) {
      if (a.logp) a.logp[t] = p.logp;
      if (kMode == kForward) {
        a.frame[t] = make_float2(s.m, p.s);
        a.slope[t] = 0.f;
      }
    }
    if (kMode == kPolicy) {
      const Outcome o = policy_terms(a, at, p.logp);
      acc.add(o.terms);
      if (has_grad) {
        const Factor f = row_factor(a, s.m, p.s, p.logp, o.slope);
        if (f.none() || !aligned_unit(g + row.head)) {  // zeros; or (then g is not z) element by element
          for (int j = lane; j < a.vocab; j += 32)
            Vec<T>::store(g + j, f.none() ? 0.f : j == y ? f.at_y : f.factor * x.one(Vec<T>::load(z + j)));
          continue;
        }
        T* dst = g + row.head + lane * N;
        if (kUnits * N > 64) {  // up to 64 exponentials stay in registers from the sum; more are taken again
#pragma unroll
          for (int k = 0; k < kUnits; ++k)
            asm volatile("" : "+r"(w[k].x), "+r"(w[k].y), "+r"(w[k].z), "+r"(w[k].w));
        }
#pragma unroll
        for (int k = 0; k < kUnits; ++k)
          if (k * 32 + lane < row.units) store_unit(dst + k * 32 * N, scaled_unit<T>(w[k], x, f.factor), true);
        if (owned >= 0) Vec<T>::store(g + y, f.at_y);
        if (edge >= 0) Vec<T>::store(g + edge, at_edge ? f.at_y : f.factor * x.one(zedge));
      }
    }
  }
  if (!waited) griddep_wait();
  if (kMode == kForward && blockIdx.x == 0 && threadIdx.x == 0) *a.ticket = 0;
  if (kMode == kPolicy) {
    __shared__ double part[kWarpRowWarps][4];
    __shared__ StatsShared stats;
    if (lane == 0) acc.get(part[warp]);
    __syncthreads();
    if (threadIdx.x < 4) {
      double sum = part[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < kWarpRowWarps; ++k) sum += part[k][threadIdx.x];
      stats.sum[threadIdx.x] = sum;
    }
    finish_stats<1>(a, stats, blockIdx.x, gridDim.x);
  }
}

// Rows straight from memory, one CTA a row: where nothing is written back a row need not
// stay on chip, and many CTAs an SM hide a row's end behind others' loads.  A different warp
// forms each row's result while the others go on to the next.  With a gradient (rows too
// long for a cluster's shared memory) the row is read a second time.  Bound by HBM: 16411 x
// 131072 bf16, a tenth masked, 0.567 ms, 6.8 TB/s (persistent CTAs with rows dealt out in
// turn: 0.614 ms, since masked rows leave some idle; row_kernel: 0.807 ms).
template <typename T, int kMode>
__global__ void __launch_bounds__(kMaxRowThreads) stream_kernel(const __grid_constant__ RowArgs a) {
  constexpr int N = Vec<T>::N;
  __shared__ Sum red[2][kMaxRowThreads / 32];
  __shared__ Factor factor;
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5, warps = nt >> 5;
  const bool has_grad = kMode == kPolicy && a.grad != nullptr;
  Terms acc;  // of the last warp
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const T* z = reinterpret_cast<const T*>(a.logits) + t * a.stride;
    T* g = reinterpret_cast<T*>(a.grad) + t * a.grad_stride;
    if (a.mask != nullptr && a.mask[t] == 0) {
      if (tid == 0 && a.logp) a.logp[t] = 0.f;
      if (kMode == kForward && tid == 0) a.slope[t] = 0.f;
      if (has_grad)
        for (int64_t j = tid; j < a.vocab; j += nt) Vec<T>::store(g + j, 0.f);
      continue;
    }
    const int64_t y = a.targets[t];
    const bool in = y >= 0 && y < a.vocab;
    const Row row = row_of(z, a.vocab);
    const uint4* src = reinterpret_cast<const uint4*>(z + row.head);
    const int unit = in && y >= row.head && y < row.tail ? ((int)y - row.head) / N : -1;
    const int elem = ((int)y - row.head) % N;
    // the unit is the target_k-th of the kGroup that its thread takes from target_l on
    const int target_l = unit >= 0 && unit % nt == tid ? unit - unit / nt % kGroup * nt : -1;
    const int target_k = unit / nt % kGroup;
    const int edge = tid < 16 ? edge_of(row, a.vocab, tid) : -1;
    Sum s{-INFINITY, 0.f};
    Expo<T> x(a, s.m);
    // the backward pass begins with the last rows: L2 keeps them rather than those before
    const uint64_t policy = l2_policy(kMode == kForward && (a.tokens - t) * a.vocab * (int)sizeof(T) > kKeptBytes);
    for (int l = tid; l < row.units; l += kGroup * nt) {
      uint4 w[kGroup];
#pragma unroll
      for (int k = 0; k < kGroup; ++k) {
        const int u = l + k * nt;
        w[k] = u < row.units ? (kMode == kForward ? load16(src + u, policy) : __ldg(src + u)) : make_uint4(Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest, Vec<T>::kLowest);
      }
      if (l == target_l) {  // the target leaves the sum
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
          if (k == target_k) drop<T>(w[k], Vec<T>::mask_of(elem));
      }
      add_units<T>(a, x, s, w);
    }
    const float zedge = edge >= 0 ? Vec<T>::load(z + edge) : -INFINITY;
    if (edge >= 0 && edge != y) add_value(a, s, zedge);
    s = warp_merge(a, s);
    if (lane == 0) red[turn & 1][warp] = s;
    __syncthreads();
    if (warp == (kMode == kPolicy ? warps - 1 : turn % warps)) {
      s = warp_merge(a, lane < warps ? red[turn & 1][lane] : Sum{-INFINITY, 0.f});
      const Prob p = row_prob(a, s, in ? Vec<T>::load(z + y) : NAN);
      if (lane == 0) {
        if (a.logp) a.logp[t] = p.logp;
        if (kMode == kForward) {
          a.frame[t] = make_float2(s.m, p.s);
          a.slope[t] = 0.f;
        }
      }
      if (kMode == kPolicy) {
        const Position at{a.old_logp[t], a.ref_logp ? a.ref_logp[t] : 0.f, a.adv[t],
                          a.weight ? __ldcg(a.weight + t) : __ldcg(a.inv_count)};
        const Outcome o = policy_terms(a, at, p.logp);
        acc.add(o.terms);
        if (lane == 0) factor = row_factor(a, s.m, p.s, p.logp, o.slope);
      }
    }
    ++turn;
    if (!has_grad) continue;  // red's other half takes the next row
    __syncthreads();
    const Factor f = factor;
    x.frame(f.m);
    const bool whole = aligned_unit(g + row.head);
    for (int l = tid; l < row.units; l += nt)
      store_unit(g + row.head + (int64_t)l * N, f.none() ? make_uint4(0, 0, 0, 0) : scaled_unit<T>(src[l], x, f.factor), whole);
    if (unit >= 0 && unit % nt == tid) Vec<T>::store(g + y, f.at_y);
    if (edge >= 0) Vec<T>::store(g + edge, f.none() ? 0.f : edge == y ? f.at_y : f.factor * x.one(zedge));
    __syncthreads();  // factor is free
  }
  if (kMode == kForward && blockIdx.x == 0 && tid == 0) *a.ticket = 0;
  if (kMode == kPolicy) {
    __shared__ StatsShared stats;
    if (warp == warps - 1 && lane == 0) acc.get(stats.sum);
    finish_stats<2>(a, stats, blockIdx.x, gridDim.x);  // a CTA may have two warps
  }
}

// The gradient of rows whose slope, frame and sum are known, a piece of kPiece units a
// CTA; the last rows first, whose logits the forward pass left in L2 (a gradient too large
// for L2 does not displace them: 1024 x 65536 fp32, forward and backward 125 us with the
// default policies, 117 us so).  Bound by HBM: with its forward pass 8192 x 131072 bf16, a
// quarter masked, in 0.79 ms, 6.8 TB/s of the three passes' traffic.
constexpr int kPieceThreads = 256;
constexpr int kPiece = kPieceThreads * kGroup;

template <typename T>
__global__ void __launch_bounds__(kPieceThreads) backward_kernel(const __grid_constant__ RowArgs a, int pieces) {
  constexpr int N = Vec<T>::N;
  const int tid = threadIdx.x;
  const uint64_t policy = l2_policy(a.tokens * a.vocab * (int)sizeof(T) > kKeptBytes);
  bool waited = false;
  for (int64_t r = blockIdx.x; r < a.tokens * pieces; r += gridDim.x) {
    const int64_t t = a.tokens - 1 - r / pieces;
    const int piece = (int)(r % pieces);
    const T* z = reinterpret_cast<const T*>(a.logits) + t * a.stride;
    T* g = reinterpret_cast<T*>(a.grad) + t * a.grad_stride;
    const bool live = a.mask == nullptr || a.mask[t] != 0;
    // the logits are on their way while the row's scalars are read (and, at first, while
    // the pair kernel runs)
    const Row row = row_of(z, a.vocab);
    const int v0 = piece * kPiece + tid;
    const uint4* src = reinterpret_cast<const uint4*>(z + row.head);
    uint4 w[kGroup];
    if (live) {
#pragma unroll
      for (int k = 0; k < kGroup; ++k)
        if (v0 + k * kPieceThreads < row.units) w[k] = src[v0 + k * kPieceThreads];
    }
    if (!waited) {
      griddep_wait();
      waited = true;
    }
    const float slope = live ? __ldcg(a.slope + t) : 0.f;
    if (slope == 0.f) {
      const Row out = row_of(g, a.vocab);
      uint4* dst = reinterpret_cast<uint4*>(g + out.head);
      for (int l = v0; l < min((piece + 1) * kPiece, out.units); l += kPieceThreads)
        store16(dst + l, make_uint4(0, 0, 0, 0), policy);
      const int e = piece == 0 && tid < 16 ? edge_of(out, a.vocab, tid) : -1;
      if (e >= 0) Vec<T>::store(g + e, 0.f);
      continue;
    }
    const float2 ms = __ldcg(a.frame + t);
    const int64_t y = a.targets[t];
    const Factor f = row_factor(a, ms.x, ms.y, __ldcg(a.logp + t), slope);
    const Expo<T> x(a, f.m);
    const bool whole = aligned_unit(g + row.head);
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const int u = v0 + k * kPieceThreads;
      if (u >= row.units) continue;
      T* dst = g + row.head + (int64_t)u * N;
      const uint4 o = scaled_unit<T>(w[k], x, f.factor);
      if (whole) store16(reinterpret_cast<uint4*>(dst), o, policy);
      else store_unit(dst, o, false);
    }
    const int unit = y >= row.head && y < row.tail ? ((int)y - row.head) / N : -1;
    if (unit >= v0 && unit < v0 + kPiece && (unit - v0) % kPieceThreads == 0) Vec<T>::store(g + y, f.at_y);
    const int e = piece == 0 && tid < 16 ? edge_of(row, a.vocab, tid) : -1;
    if (e >= 0) Vec<T>::store(g + e, e == y ? f.at_y : f.factor * x.one(Vec<T>::load(z + e)));
  }
  if (!waited) griddep_wait();
}

// ---------------------------------------------------------------------------
// small kernels
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 1024;

__device__ __forceinline__ int64_t clamp_offset(int64_t v, int64_t lo, int64_t hi) {
  return v < lo ? lo : v > hi ? hi : v;
}

template <int kThreads>
__device__ __forceinline__ int64_t block_sum(int64_t v) {
  __shared__ int64_t red[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += red[w];
  return v;
}

// A sum and the rounding errors that it left (64-bit additions are two a clock and SM).
struct Pair {
  float s = 0.f, err = 0.f;
  __device__ __forceinline__ void add(float v) {
    float t, e;
    two_sum(s, v, t, e);
    s = t;
    err += fabsf(t) < INFINITY ? e : 0.f;
  }
  __device__ __forceinline__ void add(const Pair& v) {
    add(v.s);
    err += v.err;
  }
};

template <int kThreads>
__device__ __forceinline__ int64_t live_count(const uint8_t* mask, int64_t a, int64_t b) {
  if (mask == nullptr) return b > a ? b - a : 0;
  int64_t n = 0;
  // 16 positions at a time between the first and the last 16-byte boundary
  const int64_t a16 = min(b, a + (int64_t)(-reinterpret_cast<uint64_t>(mask + a) & 15));
  const int64_t units = b > a16 ? (b - a16) / 16 : 0;
  const uint4* p = reinterpret_cast<const uint4*>(mask + a16);
  for (int64_t u = threadIdx.x; u < units; u += kThreads) {
    const uint4 w = p[u];
    // a byte that is not 0 becomes 0xff, so that every one counts 8 bits
    n += (__popc(__vcmpne4(w.x, 0)) + __popc(__vcmpne4(w.y, 0)) + __popc(__vcmpne4(w.z, 0)) + __popc(__vcmpne4(w.w, 0))) / 8;
  }
  for (int64_t t = a + threadIdx.x; t < a16; t += kThreads) n += mask[t] != 0;
  for (int64_t t = a16 + 16 * units + threadIdx.x; t < b; t += kThreads) n += mask[t] != 0;
  return block_sum<kThreads>(n);
}

// Lists the live positions, then (from the back) the masked ones, so that every cluster of
// the row kernel gets as many of each; returns the number of live ones.
__device__ __forceinline__ int64_t build_order(const uint8_t* mask, int64_t tokens, int32_t* order, int32_t* n_live) {
  constexpr int kEach = 16;
  __shared__ int totals[kSmallThreads / 32];
  const bool whole = (reinterpret_cast<uint64_t>(mask) & 15) == 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t live = 0;
  for (int64_t base = 0; base < tokens; base += kEach * kSmallThreads) {
    const int64_t t = base + kEach * threadIdx.x;
    unsigned bits = 0;
    if (whole && t + kEach <= tokens) {
      const uint4 w = *reinterpret_cast<const uint4*>(mask + t);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < kEach; ++j) bits |= ((u[j >> 2] >> (8 * (j & 3))) & 255u) != 0 ? 1u << j : 0u;
    } else {
#pragma unroll
      for (int j = 0; j < kEach; ++j)
        if (t + j < tokens && mask[t + j] != 0) bits |= 1u << j;
    }
    const int own = __popc(bits);
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) totals[warp] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kSmallThreads / 32; ++w) {
      before += w < warp ? totals[w] : 0;
      all += totals[w];
    }
    int64_t front = live + before + upto - own, back = tokens - 1 - (t - front);
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      if (t + j >= tokens) break;
      order[(bits >> j) & 1 ? front++ : back--] = (int32_t)(t + j);
    }
    live += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) *n_live = (int32_t)live;
  return live;
}

// Weight of every position under the token mean (or the sum: 1); the order if it is asked for.
__global__ void __launch_bounds__(kSmallThreads) count_kernel(const uint8_t* mask, int64_t tokens, int mean,
                                                              float* inv_count, unsigned* ticket, int32_t* order,
                                                              int32_t* n_live) {
  griddep_launch_dependents();
  if (threadIdx.x == 0) *ticket = 0;
  float w = 1.f;
  int64_t n = -1;
  if (order) n = build_order(mask, tokens, order, n_live);
  if (mean) {
    if (n < 0) n = live_count<kSmallThreads>(mask, 0, tokens);
    w = 1.f / (float)(n < 1 ? 1 : n);
  }
  if (threadIdx.x == 0) *inv_count = w;
}

// Sequence mean: one CTA a sequence writes the weights of its positions; CTA n_seqs
// clears those before the first and after the last, and does what concerns all.
__global__ void __launch_bounds__(kSmallThreads) weight_kernel(const uint8_t* mask, int64_t tokens,
                                                               const int64_t* offsets, int64_t n_seqs, float* weight,
                                                               unsigned* ticket, int32_t* order, int32_t* n_live) {
  griddep_launch_dependents();
  const int64_t q = blockIdx.x;
  if (q == n_seqs) {
    if (order) build_order(mask, tokens, order, n_live);
    if (threadIdx.x == 0) *ticket = 0;
    const int64_t a = clamp_offset(offsets[0], 0, tokens), b = clamp_offset(offsets[n_seqs], a, tokens);
    for (int64_t t = threadIdx.x; t < a; t += kSmallThreads) weight[t] = 0.f;
    for (int64_t t = b + threadIdx.x; t < tokens; t += kSmallThreads) weight[t] = 0.f;
    return;
  }
  const int64_t a = clamp_offset(offsets[q], 0, tokens), b = clamp_offset(offsets[q + 1], a, tokens);
  const int64_t n = live_count<kSmallThreads>(mask, a, b);
  const float w = 1.f / ((float)n_seqs * (float)(n < 1 ? 1 : n));
  for (int64_t t = a + threadIdx.x; t < b; t += kSmallThreads)
    weight[t] = mask == nullptr || mask[t] != 0 ? w : 0.f;
}

constexpr int kPairThreads = 512;

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
  float* loss;
  unsigned* ticket; // zeroed by the kernel before
};

// One CTA a pair: half of it sums each sequence, one thread forms the margin (in 64 bits:
// a difference of long sums), and each half writes the slopes of its positions.  The last
// CTA to come forms the mean over the pairs, in their order.  Bound by latency (6 us for
// sequences of 50 positions).
__global__ void __launch_bounds__(kPairThreads) pair_kernel(const __grid_constant__ PairArgs a) {
  constexpr int kHalf = kPairThreads / 2, kWarps = kPairThreads / 32;
  __shared__ Pair sums[kWarps];
  __shared__ int live[kWarps];
  __shared__ float slope[2];
  __shared__ int32_t last;
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, half = threadIdx.x / kHalf, at = threadIdx.x % kHalf;
  const int64_t i = blockIdx.x, q = half == 0 ? i : a.n_pairs + i;
  const int64_t lo = clamp_offset(a.offsets[q], 0, a.tokens), hi = clamp_offset(a.offsets[q + 1], lo, a.tokens);
  const float ref[2] = {a.ref[i], a.ref[a.n_pairs + i]};
  Pair part;
  int n = 0;
  if (a.mean)
    for (int64_t t = lo + at; t < hi; t += kHalf) n += a.mask == nullptr || a.mask[t] != 0;
  griddep_wait();
#pragma unroll 4
  for (int64_t t = lo + at; t < hi; t += kHalf) part.add(__ldcg(a.logp + t));  // 0 where masked
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Pair u;
    u.s = __shfl_xor_sync(0xFFFFFFFFu, part.s, o);
    u.err = __shfl_xor_sync(0xFFFFFFFFu, part.err, o);
    part.add(u);
    n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
  }
  if (lane == 0) {
    sums[warp] = part;
    live[warp] = n;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double gain[2];
    float per[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      Pair s = sums[k * kWarps / 2];
      int count = live[k * kWarps / 2];
#pragma unroll
      for (int w = 1; w < kWarps / 2; ++w) {
        s.add(sums[k * kWarps / 2 + w]);
        count += live[k * kWarps / 2 + w];
      }
      double sum = (double)s.s + (double)s.err;
      per[k] = a.mean ? 1.f / (float)max(count, 1) : 1.f;
      if (a.mean) sum /= (double)max(count, 1);
      if (a.seq_logp) a.seq_logp[k == 0 ? i : a.n_pairs + i] = (float)sum;
      gain[k] = sum - (double)ref[k];
    }
    const float h = (float)((double)a.beta * (gain[0] - gain[1]));
    if (a.margins) a.margins[i] = h;
    // log sigmoid(h) = min(h, 0) - log(1 + exp(-|h|))
    const float soft = log1pf(expf(-fabsf(h)));
    // an infinite margin (an answer with a token that cannot be taken) has a term of infinity,
    // which counts for nothing where its weight is zero
    const float won = a.smooth < 1.f ? (1.f - a.smooth) * (soft - fminf(h, 0.f)) : 0.f;
    const float lost = a.smooth > 0.f ? a.smooth * (soft + fmaxf(h, 0.f)) : 0.f;
    a.pair_loss[i] = won + lost;
    const float up = 1.f / (1.f + expf(-h)), down = 1.f / (1.f + expf(h));
    const float d = a.beta / (float)a.n_pairs * (a.smooth * up - (1.f - a.smooth) * down);
    slope[0] = d * per[0];
    slope[1] = -d * per[1];
    __threadfence();
    last = atomicAdd(a.ticket, 1u) == (unsigned)a.n_pairs - 1;
  }
  __syncthreads();
  if (a.slope)
    for (int64_t t = lo + at; t < hi; t += kHalf) a.slope[t] = slope[half];
  if (!last) return;
  __threadfence();
  part = Pair();
  for (int64_t k = threadIdx.x; k < a.n_pairs; k += kPairThreads) part.add(__ldcg(a.pair_loss + k));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Pair u;
    u.s = __shfl_xor_sync(0xFFFFFFFFu, part.s, o);
    u.err = __shfl_xor_sync(0xFFFFFFFFu, part.err, o);
    part.add(u);
  }
  if (lane == 0) sums[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    part = sums[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) part.add(sums[w]);
    *a.loss = (float)(((double)part.s + (double)part.err) / (double)a.n_pairs);
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
int32_t check_batch(const muon_token_batch* b) {
  if (!b) return invalid("batch is NULL");
  if (b->tokens < 0 || b->tokens > (1ll << 31) - 1) return invalid("tokens must be in [0, 2^31)");
  if (b->vocab < 1 || b->vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (b->row_stride != 0 && (b->row_stride < b->vocab || b->row_stride > (1ll << 40)))
    return invalid("row_stride must be 0 or at least vocab");
  if (b->dtype != MUON_DTYPE_F32 && b->dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  if (!(b->temperature >= 1e-20 && b->temperature <= 1e20)) return invalid("temperature must be in [1e-20, 1e20]");
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

RowArgs row_args(const muon_token_batch* b) {
  RowArgs a = {};
  a.logits = b->logits;
  a.targets = b->targets;
  a.mask = b->mask;
  a.tokens = b->tokens;
  a.vocab = b->vocab;
  a.stride = b->row_stride ? b->row_stride : b->vocab;
  a.grad_stride = a.vocab;
  const double c = 1.4426950408889634 / b->temperature;
  split_down(c, &a.c_hi, &a.c_lo);
  split_down(1.0 / b->temperature, &a.inv_hi, &a.inv_lo);
  // c = down + (up - down) k / 8 within a sixteenth of their distance
  const float near = (float)c, down = (double)near <= c ? near : std::nextafterf(near, 0.f);
  const float up = std::nextafterf(down, INFINITY);
  const int k = (int)std::lround(8.0 * (c - (double)down) / ((double)up - (double)down));
  for (int i = 0; i < 4; ++i) a.c_mix[i] = make_float2(2 * i < k ? up : down, 2 * i + 1 < k ? up : down);
  a.inv_temp = (float)(1.0 / b->temperature);
  a.grad_scale = 1.f;
  return a;
}

constexpr int kMaxParts = 2048;            // partial sums of the policy loss
constexpr int64_t kMostCtas = 2000000000;
constexpr size_t kSmemPerSm = 227 * 1024;  // what one CTA may have

// Shape of a row kernel's launch.  warp_units > 0: a warp a row; else cluster = 0: straight
// from memory, one CTA a row.
struct RowShape {
  int warp_units, cluster, stages, threads;
  size_t smem;
};

int row_threads(int64_t units, int cluster) {  // that hold units: about 8 each
  const int64_t want = ((units + cluster - 1) / cluster + 7) / 8;
  return (int)(want <= 128 ? 128 : want >= kMaxRowThreads ? kMaxRowThreads : (want + 31) / 32 * 32);
}

size_t row_smem(int64_t units, int cluster, int stages) {
  const size_t sums = (size_t)kSlots * cluster * (row_threads(units, cluster) / 32 + 1) * sizeof(Sum);
  return (size_t)stages * (size_t)((units + cluster - 1) / cluster) * 16 + sizeof(RowShared) + sums;
}

// Threads that hold units, of all CTAs that an SM has room for; 0: a CTA does not fit.  80 and
// 64 registers are those of the bf16 forms in the units that they are given out in (74 and 56
// used); fp32 rows use 56 with three rows too and may fit more often than this says.
int resident_threads(int64_t units, int cluster, int stages) {
  const size_t smem = row_smem(units, cluster, stages);
  if (smem > kSmemPerSm) return 0;
  const int threads = row_threads(units, cluster), all = threads + 32;
  const int by_smem = (int)((kSmemPerSm + 1024) / (smem + 1024));
  const int by_regs = 65536 / (all * (stages == 3 ? 80 : 64));
  return threads * (by_smem < by_regs ? by_smem : by_regs);
}

RowShape row_shape(int64_t vocab, int32_t dtype, int64_t tokens, int sms, bool resident) {
  const int64_t per_unit = dtype == MUON_DTYPE_BF16 ? 8 : 4;
  const int64_t units = vocab / per_unit < 1 ? 1 : vocab / per_unit;
  RowShape s = {};
  // few rows: more CTAs for each, while each still has some 8 KB of it
  int split = 1;
  while (split < kMaxCluster && tokens * split * 2 <= sms && units / split >= 1024) split *= 2;
  if (units <= 512 && split == 1) {
    s.warp_units = units <= 128 ? 4 : units <= 256 ? 8 : 16;
    return s;
  }
  const auto take = [&](int cluster, int stages) {
    s.cluster = cluster;
    s.stages = stages;
    s.smem = row_smem(units, cluster, stages);
  };
  if (split > 1) {
    for (int c = split; c <= kMaxCluster && s.cluster == 0; c *= 2)
      for (int stages = 3; stages >= 2 && s.cluster == 0; --stages)
        if (resident_threads(units, c, stages) > 0) take(c, stages);
  } else if (resident) {
    // Three rows of the ring keep HBM busy with some 480 threads an SM that hold units (448
    // where a CTA has the whole row: bf16 28000 logits 5790 GB/s of compulsory traffic, two
    // CTAs and rows 5460; but 110000 logits 5050 with four CTAs and three rows, 5490 with
    // eight and two), two rows with more; clusters of eight fill the SMs badly unless several
    // of their CTAs share one.  GB/s, CTAs a row / rows: bf16 50000 logits 4/2 5540, 2/3 5050,
    // 8/2 5120; 65536 2/3 6170, 4/2 5870; 90000 8/2 5420, 8/3 5190; 100000 8/2 5590, 4/2 5250,
    // 4/3 4790; 131072 4/3 5960, 4/2 4610; 200064 8/2 5290, 4/2 4870; 240000 8/3 4530, 8/2
    // 3590; fp32 20000 4/3 6100, 2/3 5130; 48000 8/2 6250, 8/3 6400; 120000 8/3 4940, 8/2
    // 3980; 131072 8/3 5530, 8/2 4480.
    for (int c = 1; c <= 4 && s.cluster == 0; c *= 2)
      if (resident_threads(units, c, 3) >= (c == 1 ? 448 : 480)) take(c, 3);
    int best = 0, best_cluster = 0;
    for (int c = 1; c <= kMaxCluster; c *= 2)
      if (resident_threads(units, c, 2) > best) {
        best = resident_threads(units, c, 2);
        best_cluster = c;
      }
    if (s.cluster == 0 && best < 576 && resident_threads(units, kMaxCluster, 3) >= 480) take(kMaxCluster, 3);
    if (s.cluster == 0 && best > 0) take(best_cluster, 2);
  }
  if (s.cluster == 0) {
    // many rows: small CTAs, whose ends overlap; few: enough threads to fill the SMs
    s.threads = units <= 8192 ? 64 : 256;
    while (s.threads < kMaxRowThreads && tokens * s.threads <= 512ll * sms && units >= 8 * s.threads) s.threads *= 2;
    if (resident) s.threads = 512;
    return s;
  }
  s.threads = row_threads(units, s.cluster);
  return s;
}

// Clusters of this kernel that the device holds at once.
template <typename K>
cudaError_t resident_clusters(K kernel, const RowShape& s, int* n) {
  struct Known {
    const void* kernel;
    int device, cluster, threads;
    size_t smem;
    int n;
  };
  static thread_local Known known[16];
  static thread_local int next = 0;
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  for (const Known& k : known)
    if (k.kernel == (const void*)kernel && k.device == device && k.cluster == s.cluster && k.threads == s.threads &&
        k.smem == s.smem) {
      *n = k.n;
      return cudaSuccess;
    }
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemPerSm);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)s.cluster);
  cfg.blockDim = dim3((unsigned)s.threads + 32);
  cfg.dynamicSmemBytes = s.smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)s.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaOccupancyMaxActiveClusters(n, kernel, &cfg);
  if (e != cudaSuccess) return e;
  if (*n < 1) *n = 1;
  known[next] = Known{(const void*)kernel, device, s.cluster, s.threads, s.smem, *n};
  next = (next + 1) % 16;
  return cudaSuccess;
}

template <typename T, int kMode>
cudaError_t launch_rows_as(RowArgs a, int32_t dtype, int sms, bool dependent, cudaStream_t s) {
  const RowShape shape = row_shape(a.vocab, dtype, a.tokens, sms, kMode == kPolicy && a.grad != nullptr);
  const int64_t rows = a.tokens < 1 ? 1 : a.tokens;
  if (shape.warp_units > 0) {
    auto kernel = shape.warp_units == 4 ? warp_row_kernel<T, kMode, 4>
                  : shape.warp_units == 8 ? warp_row_kernel<T, kMode, 8> : warp_row_kernel<T, kMode, 16>;
    const int64_t ctas = (rows + kWarpRowWarps - 1) / kWarpRowWarps, most = (shape.warp_units > 4 ? 2 : 3) * (int64_t)sms;
    return launch(kernel, (int)(ctas < most ? ctas : most), kWarpRowThreads, 0, s, 1, dependent, a);
  }
  if (shape.cluster == 0) {
    // without partial sums to keep, a CTA for each row balances masked ones by itself; the policy
    // loss has room for those of kMaxParts CTAs, which take rows in turn
    const int64_t most = kMode == kPolicy ? kMaxParts : rows;
    return launch(stream_kernel<T, kMode>, (int)(rows < most ? rows : most), shape.threads, 0, s, 1, dependent, a);
  }
  for (a.log_cluster = 0; (1 << a.log_cluster) < shape.cluster;) ++a.log_cluster;
  const int64_t units = a.vocab / Vec<T>::N < 1 ? 1 : a.vocab / Vec<T>::N;
  a.stage_vecs = (int32_t)((units + shape.cluster - 1) / shape.cluster);
  auto kernel = shape.stages == 3 ? row_kernel<T, kMode, 3> : row_kernel<T, kMode, 2>;
  int n = 0;
  const cudaError_t e = resident_clusters(kernel, shape, &n);
  if (e != cudaSuccess) return e;
  // without the list a cluster holds all its rows' scalars at once
  if (a.mask && !a.order && (rows + kInfo - 1) / kInfo > n) n = (int)((rows + kInfo - 1) / kInfo);
  if (n > kMaxParts) n = kMaxParts;
  if (n > rows) n = (int)rows;
  return launch(kernel, n * shape.cluster, shape.threads + 32, shape.smem, s, shape.cluster, dependent, a);
}

template <int kMode>
cudaError_t launch_rows(const RowArgs& a, int32_t dtype, int sms, bool dependent, cudaStream_t s) {
  return dtype == MUON_DTYPE_BF16 ? launch_rows_as<__nv_bfloat16, kMode>(a, dtype, sms, dependent, s)
                                  : launch_rows_as<float, kMode>(a, dtype, sms, dependent, s);
}

cudaError_t launch_backward(const RowArgs& a, int32_t dtype, cudaStream_t s) {
  if (a.tokens == 0) return cudaSuccess;
  const int64_t units = a.vocab / (dtype == MUON_DTYPE_BF16 ? 8 : 4);
  const int pieces = (int)((units < 1 ? 1 : units) + kPiece - 1) / kPiece;
  const int64_t all = a.tokens * pieces;
  // a CTA for each piece: 8192 x 131072 with a quarter masked, both passes, 0.912 ms with 8
  // CTAs an SM that take pieces in turn, 0.791 ms so
  const int grid = (int)(all < kMostCtas ? all : kMostCtas);
  return dtype == MUON_DTYPE_BF16 ? launch(backward_kernel<__nv_bfloat16>, grid, kPieceThreads, 0, s, 1, true, a, pieces)
                                  : launch(backward_kernel<float>, grid, kPieceThreads, 0, s, 1, true, a, pieces);
}

// Workspace of the losses.
size_t round16(size_t v) { return (v + 15) / 16 * 16; }

struct LossSpace {
  float* inv_count;
  unsigned* ticket;
  int32_t *n_live, *order;
  double* partials;
  float2* frame;
  float *slope, *logp, *weight, *pair_loss;
  size_t bytes;
};

LossSpace loss_space(void* ws, int64_t tokens, int64_t n_seqs) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  LossSpace s;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    uint8_t* at = p + off;
    off += round16(bytes);
    return static_cast<void*>(at);
  };
  s.inv_count = static_cast<float*>(take(4));
  s.ticket = static_cast<unsigned*>(take(4));
  s.n_live = static_cast<int32_t*>(take(4));
  s.order = static_cast<int32_t*>(take(4 * (size_t)tokens));
  s.partials = static_cast<double*>(take((size_t)kMaxParts * 4 * sizeof(double)));
  s.frame = static_cast<float2*>(take(8 * (size_t)tokens));
  s.slope = static_cast<float*>(take(4 * (size_t)tokens));
  s.logp = static_cast<float*>(take(4 * (size_t)tokens));
  s.weight = static_cast<float*>(take(4 * (size_t)tokens));
  s.pair_loss = static_cast<float*>(take(4 * (size_t)n_seqs));
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
  // Clusters that take several rows each get as many masked ones each; with few rows, or a
  // warp a row, the list would only be waited for (4096 x 131072, a fifth masked at random:
  // 0.365 ms without it, 0.352 ms with it; 20011 x 4099: 0.075 and 0.086 ms).  Few rows: fewer
  // CTAs than four an SM.  That counts no CTAs that share an SM, so where several do (50001
  // fp32 logits: four) a list is made from one row a cluster on, and waited for.
  const RowShape shape = row_shape(batch->vocab, batch->dtype, batch->tokens, sms, grad != nullptr);
  int32_t* order = batch->mask && shape.cluster > 0 && batch->tokens * shape.cluster >= 4ll * sms ? ws.order : nullptr;
  if (by_seq)
    e = launch(weight_kernel, (int)n_seqs + 1, kSmallThreads, 0, s, 1, false, batch->mask, (int64_t)batch->tokens,
               seq_offsets, (int64_t)n_seqs, ws.weight, ws.ticket, order, ws.n_live);
  else
    e = launch(count_kernel, 1, kSmallThreads, 0, s, 1, false, batch->mask, (int64_t)batch->tokens,
               (int)(c.reduction == MUON_REDUCE_TOKEN_MEAN), ws.inv_count, ws.ticket, order, ws.n_live);
  if (e != cudaSuccess) return cuda_error(e);
  RowArgs a = row_args(batch);
  a.order = order;
  a.n_live = ws.n_live;
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
  a.partials = ws.partials;
  a.ticket = ws.ticket;
  a.stats = stats;
  e = launch_rows<kPolicy>(a, batch->dtype, sms, true, s);
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
  a.ticket = ws.ticket;
  a.grad_scale = c.grad_scale;
  a.grad = grad;
  if (grad_stride) a.grad_stride = grad_stride;
  cudaError_t e;
  // clears the pair kernel's ticket too
  e = batch->tokens > 0 ? launch_rows<kForward>(a, batch->dtype, sms, false, s)
                        : cudaMemsetAsync(ws.ticket, 0, sizeof(unsigned), s);
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
    p.slope = grad ? ws.slope : nullptr;
    p.loss = loss;
    p.ticket = ws.ticket;
    if ((e = launch(pair_kernel, (int)n_pairs, kPairThreads, 0, s, 1, batch->tokens > 0, p)) != cudaSuccess)
      return cuda_error(e);
  }
  if (n_pairs == 0 && (e = cudaMemsetAsync(loss, 0, sizeof(float), s)) != cudaSuccess) return cuda_error(e);
  if (grad && (e = launch_backward(a, batch->dtype, s)) != cudaSuccess) return cuda_error(e);
  return MUON_OK;
}

}  // extern "C"
