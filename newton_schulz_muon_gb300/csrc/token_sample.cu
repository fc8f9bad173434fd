// Tokens sampled from logits, and drafted tokens verified against the target's
// probabilities, from given uniform numbers.
//
//   p = softmax(target logits / temperature), q the draft model's probabilities likewise
//   a draft x is taken while u q(x) < p(x);
//   the token after the a taken ones comes from max(p - q, 0) at row a where a draft was
//   refused there, else from p: the first token whose cumulated weight exceeds
//   u' (the sum of all weights).
//
// A row is cut into strips of consecutive 16-byte units, and each strip's sum of exponentials
// is kept (in the frame of its own largest logit).  The sums give the row's normaliser, and by
// them the strip that holds the sampled token is found: only that strip is read again, so
// that a row is read once.  A refused draft's row is read twice, since the difference of the
// probabilities needs both rows' normalisers first.
//
// Sampling: the strips of all rows are dealt out to the warps of the whole chip alike, and a
// second kernel draws the tokens, a warp a row.  (With a CTA a row 2048 rows of 131072 bf16
// logits took 117 us: the ends of rows, and 3.03 rounds of CTAs that took 4.  ROWS_US so.)
//
// Verification: a cluster of CTAs a sequence, whose rows are taken one after the other until a
// draft is refused (side by side where there are few sequences).  (Dealing out the strips of
// all sequences' rows too, position by position, with the verdict by the warp that finishes a
// row, took 246 us for 512 sequences of four drafts: a warp that judges falls behind, so that
// it is the last at the next row as well.  VERIFY_US so.)
//
// Sums over a strip are fp32 (1024 bf16 or 512 fp32 logits, 32 or 16 a lane and then the
// lanes'), sums over strips and the search for the token's strip are in 64 bits: a token's
// share of [0, 1) begins within a few 1e-8 of where it should.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "device.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "muon.h"
#include "rows.cuh"

namespace muon {
namespace {

constexpr int kLoads = 4;                  // 16-byte units a lane takes at a time
constexpr int kStripStep = 32 * kLoads;    // units that a warp takes at a time
constexpr int kMaxStrips = 512;            // of a row; longer rows have longer strips
constexpr int kMaxRound = 8;               // rows of a sequence side by side
constexpr int kMaxCluster = 8;
constexpr int kSampleWarps = 8;            // of a CTA, at most
constexpr int kSampleCtas = 4;             // CTAs an SM, by their registers

// Logits are divided by the temperature: exponents in base 2 are c = c_hi + c_lo times
// theirs, c_lo > 0 (so that -inf stays -inf).
struct Scale {
  float c_hi, c_lo, inv_hi, inv_lo;
};

// A sum of exponentials in the frame of m, the largest logit (-inf: none).
struct StripSum {
  float m, s;
};
struct RowSum {
  double s;
  float m;
  double rest;  // without the strip that holds the row's draft
};

struct SampleArgs {
  const void* target;
  const void* draft;         // null: drafts that were certain
  const uint8_t* mask;       // rows of a sampling call that take part; or null
  const int64_t* drafts;
  const float* draft_logp;   // or null
  const int64_t* offsets;    // [n_seqs + 1]
  const float* accept_u;
  const float* sample_u;
  int64_t* tokens;
  int64_t* counts;
  float* logp;
  int64_t target_stride, draft_stride;
  int64_t n_drafts, n_seqs;  // sampling: n_seqs rows
  Scale target_scale, draft_scale;
  int32_t vocab;
  int32_t strip_units;       // a multiple of kStripStep
  int32_t strips;            // of a row; of a CTA's part of it in verification
  // sampling
  int32_t each, pieces;      // strips that a warp takes at a time; of a row: strips / each, rounded up
  StripSum* sums;            // workspace, [rows][strips]
  // verification
  int32_t cluster;           // CTAs a sequence
  int32_t round;             // rows of a sequence taken side by side
};

__device__ __forceinline__ float factor(const Scale& c, float m, float to) {
  if (m == to) return 1.f;
  const float d = m - to;
  return ex2(__fmaf_rn(d, c.c_hi, d * c.c_lo));
}
__device__ __forceinline__ float frame_of(float m) { return m == -INFINITY ? 0.f : m; }

__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ double warp_scan64(double v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double w = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += w;
  }
  return v;
}

// A row in 16-byte units: unit u holds the elements u N - shift .. + N - 1, those outside
// the row being -inf.
template <typename T>
struct RowUnits {
  const T* z;
  int32_t vocab, shift, units;
  __device__ __forceinline__ RowUnits(const void* base, int64_t row, int64_t stride, int32_t v)
      : z(reinterpret_cast<const T*>(base) + row * stride), vocab(v) {
    shift = (int)(reinterpret_cast<uint64_t>(z) & 15) / (int)sizeof(T);
    units = (shift + vocab + Vec<T>::N - 1) / Vec<T>::N;
  }
  __device__ __forceinline__ int first(int u) const { return u * Vec<T>::N - shift; }
};

// The 16 bytes of elements e .. e + N - 1 of a row, -inf outside it; one load where they lie
// in the row and on a 16-byte boundary.
template <typename T>
__device__ __forceinline__ uint4 load_elems(const T* z, int32_t vocab, int e) {
  constexpr int N = Vec<T>::N;
  const T* p = z + e;
  if (e >= 0 && e + N <= vocab && (reinterpret_cast<uint64_t>(p) & 15) == 0)
    return __ldg(reinterpret_cast<const uint4*>(p));
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = e + i >= 0 && e + i < vocab ? Vec<T>::load(p + i) : -INFINITY;
  return Vec<T>::pack(v);
}

// Units first, first + stride, ... of a row, kLoads of them, -inf from unit u1 on.  inside: they
// all hold elements of the row only.
template <typename T>
__device__ __forceinline__ void load_units(const RowUnits<T>& row, int first, int stride, int u1, bool inside,
                                           uint4 (&w)[kLoads]) {
  constexpr uint32_t low = Vec<T>::kLowest;
  if (inside) {
    const uint4* p = reinterpret_cast<const uint4*>(row.z - row.shift) + first;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) w[k] = __ldg(p + k * stride);
  } else {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int u = first + k * stride;
      w[k] = u < u1 ? load_elems<T>(row.z, row.vocab, row.first(u)) : make_uint4(low, low, low, low);
    }
  }
}
// Whether the units [u, u + kStripStep) lie before u1 and hold elements of the row only.
template <typename T>
__device__ __forceinline__ bool step_inside(const RowUnits<T>& row, int u, int u1) {
  return u + kStripStep <= u1 && row.first(u) >= 0 && row.first(u + kStripStep) <= row.vocab;
}

// 2^(c (z - m)) of a unit's elements.
template <typename T>
__device__ __forceinline__ void exps(const Scale& c, float m, const uint4& w, float (&e)[Vec<T>::N]) {
  float v[Vec<T>::N];
  Vec<T>::unpack(w, v);
#pragma unroll
  for (int i = 0; i < Vec<T>::N; i += 2) {
    const F2 d = add2(make_f2(v[i], v[i + 1]), make_f2(-m, -m));
    const float2 u = split(fma2(d, make_f2(c.c_hi, c.c_hi), mul2(d, make_f2(c.c_lo, c.c_lo))));
    e[i] = ex2(u.x);
    e[i + 1] = ex2(u.y);
  }
}

// Adds a step's units to a strip's sum; the same in every lane.
template <typename T>
__device__ __forceinline__ void add_step(const Scale& c, const uint4 (&w)[kLoads], StripSum& t) {
  const float m = fmaxf(t.m, warp_max(Vec<T>::max(w)));
  F2 s0 = make_f2(0.f, 0.f), s1 = make_f2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    float e[Vec<T>::N];
    exps<T>(c, frame_of(m), w[k], e);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; i += 4) {
      s0 = add2(s0, make_f2(e[i], e[i + 1]));
      s1 = add2(s1, make_f2(e[i + 2], e[i + 3]));
    }
  }
  const float2 r = split(add2(s0, s1));
  t.s = t.s * factor(c, t.m, m) + warp_sum(r.x + r.y);
  t.m = m;
}

// The sums of the strips [k0, k1) of a row, into `to`.  A step's loads are under way while the
// step before is summed.
template <typename T>
__device__ __forceinline__ void sum_strips(const RowUnits<T>& row, const Scale& c, int strip_units, int k0, int k1,
                                           StripSum* to, int lane) {
  const int end = (int)min((int64_t)k1 * strip_units, (int64_t)row.units);
  int u = (int)min((int64_t)k0 * strip_units, (int64_t)row.units);
  uint4 w[kLoads];
  load_units<T>(row, u + lane, 32, end, step_inside<T>(row, u, end), w);
  StripSum t{-INFINITY, 0.f};
  int left = strip_units;  // of the strip
  for (int k = k0; k < k1;) {
    const int next = u + kStripStep;
    uint4 x[kLoads];
    load_units<T>(row, next + lane, 32, end, step_inside<T>(row, next, end), x);
    add_step<T>(c, w, t);
    left -= kStripStep;
    if (left == 0) {
      if (lane == 0) to[k - k0] = t;
      t = StripSum{-INFINITY, 0.f};
      left = strip_units;
      ++k;
    }
    u = next;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) w[i] = x[i];
  }
}

// The probabilities of both models at a refused draft.
struct Refused {
  float mp, ip, mq, iq;  // frames, and reciprocals of the sums
};

// max(p - q, 0) of the units first, first + stride, ... of the target's row, 0 from u1 on; each
// product rounded, so that equal rows leave 0.
template <typename T>
__device__ __forceinline__ void left_over(const SampleArgs& a, const Refused& f, const RowUnits<T>& p, const T* zq,
                                          int first, int stride, int u1, bool inside, float (&r)[kLoads * Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  constexpr uint32_t low = Vec<T>::kLowest;
  uint4 wp[kLoads], wq[kLoads];
  load_units<T>(p, first, stride, u1, inside, wp);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    const int u = first + k * stride;
    wq[k] = u < u1 ? load_elems<T>(zq, p.vocab, p.first(u)) : make_uint4(low, low, low, low);
  }
#pragma unroll
  for (int k = 0; k < kLoads; ++k) {
    float x[N], y[N];
    exps<T>(a.target_scale, f.mp, wp[k], x);
    exps<T>(a.draft_scale, f.mq, wq[k], y);
#pragma unroll
    for (int i = 0; i < N; ++i) r[k * N + i] = fmaxf(__fmul_rn(x[i], f.ip) - __fmul_rn(y[i], f.iq), 0.f);
  }
}

// Each lane's part of the sum over the units [u0, u1) without one token.
template <typename T>
__device__ __forceinline__ float sum_without(const RowUnits<T>& row, const Scale& c, float m, int u0, int u1, int token,
                                             int lane) {
  constexpr int N = Vec<T>::N;
  float s = 0.f;
  for (int u = u0; u < u1; u += kStripStep) {
    uint4 w[kLoads];
    load_units<T>(row, u + lane, 32, u1, step_inside<T>(row, u, u1), w);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      float e[N];
      exps<T>(c, m, w[k], e);
      const int at = token - row.first(u + k * 32 + lane);
#pragma unroll
      for (int i = 0; i < N; ++i) s += i == at ? 0.f : e[i];
    }
  }
  return s;
}

// log p of a token from the sum over the others, of which each lane has a part, in the row's
// frame m; so a nearly certain token keeps its digits.
template <typename T>
__device__ __forceinline__ float token_logp(const RowUnits<T>& row, const Scale& c, float m, double rest, int token) {
  float s = (float)warp_sum64(rest);
  const float d = Vec<T>::load(row.z + token) - m;
  const float x = __fmaf_rn(d, c.inv_hi, d * c.inv_lo);
  // x <= 0; at the row's largest logit, log1p keeps the digits of a nearly certain token
  s = __fmaf_rn(x == 0.f ? s : s - 1.f, kExpLow, s);
  return x == 0.f ? 0.f - log1pf(s) : x - logf(s + expf(x));
}

__device__ __forceinline__ bool usable(const RowSum& t) { return t.s > 0. && t.s < (double)INFINITY; }

// The weights that a token is drawn from.
enum Weights {
  kPlain,    // p
  kWithout,  // p without the refused draft
  kLeft,     // max(p - q, 0)
};

// What a warp draws with.  This code runs once a row, so that it is its instructions' and the
// tables' way to the SM that costs: loops are not unrolled more than the loads need, and what
// is read again is kept in shared memory.
struct DrawSpace {
  float weight[32][kLoads * 8 + 1];  // of a step's elements, a row a lane
};

// The strip in which the cumulated weight exceeds t (one of weight 0 never does), else the
// last of positive weight; -1: none.  before: the weights before the first strip, and then
// before the one that is found.  weight(k), k < strips.
template <typename F>
__device__ __forceinline__ int find_strip(int strips, double t, double* before, int lane, F weight) {
  // a lane's strips are consecutive ones
  const int per = (strips + 31) / 32, k0 = min(lane * per, strips), k1 = min(k0 + per, strips);
  double w = 0.;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) w += (double)weight(k);
  const double end = *before + warp_scan64(w, lane);
  const unsigned above = __ballot_sync(0xFFFFFFFFu, w > 0. && end > t);
  const unsigned some = __ballot_sync(0xFFFFFFFFu, w > 0.);
  if (some == 0) return -1;
  const int l = above ? __ffs(above) - 1 : 31 - __clz(some);
  double at = end - w, begun = at;
  int strip = 0;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    const double x = (double)weight(k);
    if (x > 0.) {
      strip = k;
      begun = at;
      if (at + x > t) break;
    }
    at += x;
  }
  *before = __shfl_sync(0xFFFFFFFFu, begun, l);
  return __shfl_sync(0xFFFFFFFFu, strip, l);
}

// The first element of the units [u0, u1) at which the cumulated weight exceeds t (one of
// weight 0 never does), else the last of positive weight; -1: none.  A lane takes kLoads units
// side by side and sums them in fp32; the lanes' sums are added in 64 bits, of which the SMs do
// few.  rest: the lane's part of the sum of p over the units without that element.
template <typename T>
__device__ __forceinline__ int find_element(const SampleArgs& a, DrawSpace& sh, const RowUnits<T>& row, int u0, int u1,
                                            double t, int kind, int without, const T* zq, const Refused& f, float m,
                                            float* rest, int lane) {
  constexpr int N = Vec<T>::N;
  const Scale& c = a.target_scale;
  int found = -1;
  double before = 0.;
#pragma unroll 1
  for (int at = u0; at < u1; at += kStripStep) {
    const int first = at + lane * kLoads;
    const bool inside = step_inside<T>(row, at, u1);
    float v = 0.f;
    if (kind == kLeft) {
      float x[kLoads * N];
      left_over<T>(a, f, row, zq, first, 1, u1, inside, x);
#pragma unroll
      for (int i = 0; i < kLoads * N; ++i) {
        sh.weight[lane][i] = x[i];
        v += x[i];
      }
    } else {
      uint4 z[kLoads];
      load_units<T>(row, first, 1, u1, inside, z);
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        float e[N];
        exps<T>(c, m, z[k], e);
        const int drop = kind == kWithout ? without - row.first(first + k) : -1;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float x = i == drop ? 0.f : e[i];
          sh.weight[lane][k * N + i] = x;
          v += x;
        }
      }
    }
    __syncwarp();
    const double upto = before + warp_scan64((double)v, lane);
    const unsigned above = __ballot_sync(0xFFFFFFFFu, v > 0.f && upto > t);
    const unsigned some = __ballot_sync(0xFFFFFFFFu, v > 0.f);
    if (some) {
      const int l = above ? __ffs(above) - 1 : 31 - __clz(some);
      // each lane takes one of that lane's elements
      const float x = lane < kLoads * N ? sh.weight[l][lane] : 0.f;
      float s = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float y = __shfl_up_sync(0xFFFFFFFFu, s, o);
        if (lane >= o) s += y;
      }
      const float need = (float)(t - __shfl_sync(0xFFFFFFFFu, upto - (double)v, l));
      const unsigned over = __ballot_sync(0xFFFFFFFFu, x > 0.f && s > need);
      const unsigned any = __ballot_sync(0xFFFFFFFFu, x > 0.f);
      const int e = above && over ? __ffs(over) - 1 : 31 - __clz(any);
      found = row.first(at + l * kLoads) + e;
      *rest = (lane == l ? 0.f : v) + (lane == e ? 0.f : x);
    }
    if (above) break;
    before = __shfl_sync(0xFFFFFFFFu, upto, 31);
    __syncwarp();
  }
  if (found >= 0 && (kind != kPlain || u1 - u0 > kStripStep)) *rest = sum_without<T>(row, c, m, u0, u1, found, lane);
  return found;
}

// ---------------------------------------------------------------------------
// sampling
// ---------------------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, kSampleCtas) rows_kernel(const __grid_constant__ SampleArgs a) {
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), jobs = a.n_seqs * a.pieces;
  for (int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); job < jobs; job += warps) {
    const int64_t t = job / a.pieces;
    if (a.mask != nullptr && a.mask[t] == 0) continue;
    const int k0 = (int)(job - t * a.pieces) * a.each;
    const RowUnits<T> row(a.target, t, a.target_stride, a.vocab);
    sum_strips<T>(row, a.target_scale, a.strip_units, k0, min(k0 + a.each, a.strips), a.sums + t * a.strips + k0, lane);
  }
}

// A warp draws a row's token.
constexpr int kDrawWarps = 4;
template <typename T>
__global__ void __launch_bounds__(kDrawWarps * 32) draw_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ DrawSpace space[kDrawWarps];
  __shared__ float weights[kDrawWarps][kMaxStrips];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  griddep_wait();
  if (t >= a.n_seqs) return;
  int64_t token = -1;
  float logp = 0.f;
  if (a.mask == nullptr || a.mask[t] != 0) {
    logp = NAN;
    const Scale& c = a.target_scale;
    const RowUnits<T> row(a.target, t, a.target_stride, a.vocab);
    const float2* sums = reinterpret_cast<const float2*>(a.sums + t * a.strips);
    const float u = fmaxf(a.sample_u[t], 0.f);
    float m = -INFINITY;
#pragma unroll 4
    for (int k = lane; k < a.strips; k += 32) m = fmaxf(m, __ldcg(sums + k).x);
    m = warp_max(m);
    double own = 0.;
#pragma unroll 1
    for (int k = lane; k < a.strips; k += 32) {
      const float2 x = __ldcg(sums + k);
      weights[warp][k] = x.y * factor(c, x.x, m);
      own += (double)weights[warp][k];
    }
    __syncwarp();
    const RowSum p{warp_sum64(own), m, 0.};
    if (usable(p)) {
      double before = 0.;
      const double at = u < 1.f ? (double)u * p.s : (double)INFINITY;  // 1 and above: the last token
      const int strip = find_strip(a.strips, at, &before, lane, [&](int k) { return weights[warp][k]; });
      const int u0 = strip * a.strip_units, u1 = min(u0 + a.strip_units, row.units);
      float rest;
      const int found = find_element<T>(a, space[warp], row, u0, u1, at - before, kPlain, -1, nullptr, Refused{}, m, &rest, lane);
      double others = (double)rest;
#pragma unroll 1
      for (int k = lane; k < a.strips; k += 32)
        if (k != strip) others += (double)weights[warp][k];
      if (found >= 0) {
        token = found;
        logp = token_logp<T>(row, c, m, others, found);
      }
    }
  }
  if (lane == 0) {
    a.tokens[t] = token;
    a.logp[t] = logp;
  }
}

// ---------------------------------------------------------------------------
// verification
// ---------------------------------------------------------------------------
constexpr int kMaxTaken = 64;
struct SampleShared {
  float taken_m[kMaxTaken];        // of taken drafts whose log p is not written yet: the row's
  double taken_rest[kMaxTaken];    // frame, and its sum without the draft's strip
  RowSum slice[2][2 * kMaxRound];  // this CTA's part of each row, read by the cluster's other CTAs
  RowSum total[2][2 * kMaxRound];
  double weights;                  // this CTA's part of the weights a token is drawn from
  DrawSpace draw;
};

__device__ __forceinline__ RowSum load_peer(const RowSum* p, int rank, int own) {
  if (rank == own) return *p;
  const uint32_t at = mapa_shared(p, (uint32_t)rank);
  RowSum r;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(r.s) : "r"(at) : "memory");
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(r.m) : "r"(at + 8) : "memory");
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(r.rest) : "r"(at + 16) : "memory");
  return r;
}

__device__ __forceinline__ double load_peer(const double* p, int rank) {
  double v;
  asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(mapa_shared(p, (uint32_t)rank)) : "memory");
  return v;
}

// A cluster of CTAs a sequence.  Its rows are taken `round` at a time until a draft is refused.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 3) verify_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ StripSum tables[];  // [2][target and draft][round][strips]
  __shared__ SampleShared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int64_t seq = blockIdx.x / a.cluster;
  // offsets out of order or range: nothing outside the arrays is touched
  const int64_t lo = min(max(a.offsets[seq], (int64_t)0), a.n_drafts);
  const int64_t n = min(max(a.offsets[seq + 1], lo), a.n_drafts) - lo;
  const int64_t row0 = lo + seq;  // the sequence's first row
  const bool both = a.draft != nullptr && a.draft_logp == nullptr;  // rows of both models a round
  const int set = a.round * a.strips;
  const int strip0 = rank * a.strips;
  // of the CTA's strips this warp's
  const int per_warp = (a.strips + warps - 1) / warps, mine0 = min(warp * per_warp, a.strips), mine1 = min(mine0 + per_warp, a.strips);
  auto exchange = [&] {
    if (a.cluster > 1) cluster_sync();
    else __syncthreads();
  };
  auto units_of = [&](const RowUnits<T>& row, int k, int& u0, int& u1) {  // of this CTA's strip k
    u0 = (int)min((int64_t)(strip0 + k) * a.strip_units, (int64_t)row.units);
    u1 = min(u0 + a.strip_units, row.units);
  };
  // sums a row's slices: warp-wide, the same in every lane
  auto merge = [&](const RowSum* slice, const Scale& c) {
    RowSum t{0., -INFINITY, 0.};
    if (lane < a.cluster) t = load_peer(slice, lane, rank);
    RowSum r;
    r.m = warp_max(t.m);
    const double f = (double)factor(c, t.m, r.m);
    r.s = warp_sum64(t.s * f);
    r.rest = warp_sum64(t.rest * f);
    return r;
  };
  // this CTA's part of a row's sums; skip: the strip of its draft
  auto slice_sum = [&](const StripSum* table, const Scale& c, int skip) {
    float m = -INFINITY;
    for (int k = lane; k < a.strips; k += 32) m = fmaxf(m, table[k].m);
    RowSum r;
    r.m = warp_max(m);
    float sum = 0.f, rest = 0.f;
    for (int k = lane; k < a.strips; k += 32) {
      const float x = table[k].s * factor(c, table[k].m, r.m);
      sum += x;
      rest += k == skip ? 0.f : x;
    }
    r.s = warp_sum64((double)sum);
    r.rest = warp_sum64((double)rest);
    return r;
  };
  // each lane's part of a row's sum without the strip k0 of this CTA
  auto other_strips = [&](const StripSum* table, const RowSum* slice, int k0, float m, const Scale& c) {
    float own = 0.f;
    for (int k = lane; k < a.strips; k += 32)
      if (k != k0) own += table[k].s * factor(c, table[k].m, m);
    double s = (double)own;
    if (lane < a.cluster && lane != rank) {
      const RowSum t = load_peer(slice, lane, rank);
      s += t.s * (double)factor(c, t.m, m);
    }
    return s;
  };
  // this CTA's strip that holds a token of the target's row, or one that is not its
  auto strip_of = [&](const RowUnits<T>& row, int64_t token) {
    return token < 0 ? -1 : ((int)token + row.shift) / N / a.strip_units - strip0;
  };
  // the drafts' scalars, of 32 positions at a time: the lane's
  int64_t pos0 = 0, y = -1;
  float u = 0.f, zy = -INFINITY, logq = 0.f;
  auto look = [&] {
    y = -1;
    if (pos0 + lane >= n) return;
    const int64_t d = lo + pos0 + lane;
    y = a.drafts[d];
    u = a.accept_u[d];
    if (y < 0 || y >= a.vocab) y = -1;
    if (y < 0) return;
    zy = Vec<T>::load(reinterpret_cast<const T*>(a.target) + (row0 + pos0 + lane) * a.target_stride + y);
    if (both) logq = Vec<T>::load(reinterpret_cast<const T*>(a.draft) + d * a.draft_stride + y);
    else if (a.draft_logp != nullptr) logq = a.draft_logp[d];
  };
  // tokens and log p of the taken drafts from `from` on, by the warps from w0 on
  auto emit = [&](int64_t from, int64_t to, int w0) {
#pragma unroll 1
    for (int64_t i = from + warp - w0; i < to; i += warps - w0) {
      const int64_t t = a.drafts[lo + i];
      const RowUnits<T> row(a.target, row0 + i, a.target_stride, a.vocab);
      const int k = strip_of(row, t);
      if (k < 0 || k >= a.strips) continue;  // another CTA's strip
      int u0, u1;
      units_of(row, k, u0, u1);
      const float m = sh.taken_m[i % kMaxTaken];
      const double rest = (lane == 0 ? sh.taken_rest[i % kMaxTaken] : 0.) +
                          (double)sum_without<T>(row, a.target_scale, m, u0, u1, (int)t, lane);
      const float lp = token_logp<T>(row, a.target_scale, m, rest, (int)t);
      if (lane == 0) {
        a.tokens[row0 + i] = t;
        a.logp[row0 + i] = lp;
      }
    }
  };

  int parity = 0, at = 0;  // at: the last row's place in its round
  int64_t base = 0, taken = 0, emitted = 0;
  bool refused = false;
  StripSum* table = tables;
  for (;; base += a.round, parity ^= 1) {
    const int rows = (int)min((int64_t)a.round, n + 1 - base);
    table = tables + (size_t)parity * 2 * set;
    if (base == 0 || base + rows > pos0 + 32) {
      pos0 = base;
      look();
    }
    const int off = (int)(base - pos0);  // the lane of the round's first row
    const int drafted = both ? (int)min((int64_t)rows, n - base) : 0;
    for (int r = 0; r < rows + drafted; ++r) {
      const bool q = r >= rows;
      const RowUnits<T> row(q ? a.draft : a.target, q ? lo + base + r - rows : row0 + base + r,
                            q ? a.draft_stride : a.target_stride, a.vocab);
      sum_strips<T>(row, q ? a.draft_scale : a.target_scale, a.strip_units, strip0 + mine0, strip0 + mine1,
                    table + (q ? set + (r - rows) * a.strips : r * a.strips) + mine0, lane);
    }
    __syncthreads();
    for (int r = warp; r < rows + drafted; r += warps) {
      const bool q = r >= rows;
      int skip = -1;
      if (!q) {
        const RowUnits<T> row(a.target, row0 + base + r, a.target_stride, a.vocab);
        skip = strip_of(row, __shfl_sync(0xFFFFFFFFu, y, off + r));
      }
      const RowSum t = slice_sum(table + (q ? set + (r - rows) * a.strips : r * a.strips),
                                 q ? a.draft_scale : a.target_scale, skip);
      if (lane == 0) sh.slice[parity][q ? kMaxRound + r - rows : r] = t;
    }
    exchange();
    if (a.cluster > 1) {
      for (int r = warp; r < rows + drafted; r += warps) {
        const bool q = r >= rows;
        const int slot = q ? kMaxRound + r - rows : r;
        const RowSum t = merge(&sh.slice[parity][slot], q ? a.draft_scale : a.target_scale);
        if (lane == 0) sh.total[parity][slot] = t;
      }
      __syncthreads();
    }
    const RowSum* totals = a.cluster > 1 ? sh.total[parity] : sh.slice[parity];
    at = rows - 1;
    // every warp of every CTA decides alike
    bool ok = true;
    if (lane >= off && lane < off + rows && pos0 + lane < n) {
      const RowSum p = totals[lane - off];
      const Scale& c = a.target_scale;
      const float d = zy - p.m;
      const float logp = __fmaf_rn(d, c.inv_hi, d * c.inv_lo) - logf((float)p.s);
      bool fine = usable(p) && y >= 0;
      float lq = logq;
      if (both) {
        const RowSum q = totals[kMaxRound + lane - off];
        const float e = logq - q.m;
        lq = __fmaf_rn(e, a.draft_scale.inv_hi, e * a.draft_scale.inv_lo) - logf((float)q.s);
        fine = fine && usable(q);
      }
      ok = fine && u < expf(logp - lq);
    }
    const unsigned bad = __ballot_sync(0xFFFFFFFFu, !ok) >> off;
    refused = bad != 0;
    if (refused) at = __ffs(bad) - 1;
    // rows of this round whose drafts were taken; their log p comes later, when it delays no row
    const int good = (int)min(refused ? (int64_t)at : (int64_t)rows, n - base);
    if (warp == 0 && lane < good) {
      sh.taken_m[(base + lane) % kMaxTaken] = totals[lane].m;
      sh.taken_rest[(base + lane) % kMaxTaken] = totals[lane].rest;
    }
    taken = base + good;
    if (refused || base + rows == n + 1) break;
    if (taken - emitted + a.round > kMaxTaken) {
      __syncthreads();
      emit(emitted, taken, 0);
      emitted = taken;
      __syncthreads();
    }
  }

  // the token after the drafts that were taken, from row `taken`
  const RowUnits<T> row(a.target, row0 + taken, a.target_stride, a.vocab);
  const RowSum* totals = a.cluster > 1 ? sh.total[parity] : sh.slice[parity];
  const RowSum p = totals[at];
  const StripSum* own = table + at * a.strips;
  const Scale& c = a.target_scale;
  bool fine = usable(p);
  int kind = kPlain;
  int64_t without = -1;
  Refused f{};
  const T* zq = nullptr;
  StripSum* left = table + set + at * a.strips;  // of the draft model's row, then of the difference
  int without_strip = -1;
  float without_sum = 0.f;
  if (refused && fine) {
    const int64_t d = lo + taken;
    if (a.draft == nullptr) {
      kind = kWithout;
      without = a.drafts[d];
      if (without >= 0 && without < a.vocab) {
        const int k = strip_of(row, without);
        if (k >= 0 && k < a.strips) {  // every warp sums the strip alike
          int u0, u1;
          units_of(row, k, u0, u1);
          const float s = sum_without<T>(row, c, p.m, u0, u1, (int)without, lane);
          without_strip = k;
          without_sum = warp_sum(s);
        }
      }
    } else {
      kind = kLeft;
      const RowUnits<T> draft(a.draft, d, a.draft_stride, a.vocab);
      zq = draft.z;
      RowSum q;
      if (both) {
        q = totals[kMaxRound + at];
      } else {
        sum_strips<T>(draft, a.draft_scale, a.strip_units, strip0 + mine0, strip0 + mine1, left + mine0, lane);
        __syncthreads();
        if (warp == 0) {
          const RowSum t = slice_sum(left, a.draft_scale, -1);
          if (lane == 0) sh.slice[parity][kMaxRound] = t;
        }
        exchange();
        q = merge(&sh.slice[parity][kMaxRound], a.draft_scale);
      }
      fine = usable(q);
      f = Refused{p.m, (float)(1. / p.s), q.m, (float)(1. / q.s)};
      if (fine) {
        for (int k = warp; k < a.strips; k += warps) {
          int u0, u1;
          units_of(row, k, u0, u1);
          float s = 0.f;
          for (int u = u0; u < u1; u += kStripStep) {
            float r[kLoads * N];
            left_over<T>(a, f, row, zq, u + lane, 32, u1, step_inside<T>(row, u, u1), r);
#pragma unroll
            for (int i = 0; i < kLoads * N; ++i) s += r[i];
          }
          s = warp_sum(s);
          if (lane == 0) left[k] = StripSum{0.f, s};
        }
        __syncthreads();
      }
    }
  }

  // the first warp draws the token, the others (or it alone) write the taken drafts
  __syncthreads();
  if (warp != 0 || warps == 1) emit(emitted, taken, warps == 1 ? 0 : 1);
  if (warp != 0) return;  // the cluster's barriers wait for the warps that are left

  int64_t token = -1;
  bool mine = rank == 0;  // this CTA writes the token
  float lp = NAN;
  if (fine) {
    auto plain = [&](int k) { return own[k].s * factor(c, own[k].m, p.m); };
    auto weight = [&](int k) { return kind == kLeft ? left[k].s : kind == kWithout && k == without_strip ? without_sum : plain(k); };
    // each CTA's share of the weights in its lane, and their running sum
    double v = 0.;
    if (kind != kPlain) {
#pragma unroll 1
      for (int k = lane; k < a.strips; k += 32) v += (double)weight(k);
      v = warp_sum64(v);
      if (a.cluster > 1) {
        if (lane == 0) sh.weights = v;
        cluster_sync();
        v = lane >= a.cluster ? 0. : lane == rank ? v : load_peer(&sh.weights, lane);
      } else if (lane > 0) {
        v = 0.;
      }
      // nothing is left over where the two models agree, and the refusal was one of rounding
      if (!__any_sync(0xFFFFFFFFu, v > 0.)) kind = kPlain;
    }
    if (kind == kPlain) {
      RowSum r{0., -INFINITY, 0.};
      if (lane < a.cluster) r = load_peer(&sh.slice[parity][at], lane, rank);
      v = r.s * (double)factor(c, r.m, p.m);
    }
    const double upto = warp_scan64(v, lane), sum = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const float su = fmaxf(a.sample_u[seq], 0.f);
    const double t = su < 1.f ? (double)su * sum : (double)INFINITY;  // 1 and above: the last token
    const unsigned over = __ballot_sync(0xFFFFFFFFu, v > 0. && upto > t);
    const unsigned any = __ballot_sync(0xFFFFFFFFu, v > 0.);
    const int owner = over ? __ffs(over) - 1 : 31 - __clz(any);
    mine = rank == owner;
    if (mine) {
      double before = __shfl_sync(0xFFFFFFFFu, upto - v, owner);
      const int strip = find_strip(a.strips, t, &before, lane, weight);
      int u0, u1;
      units_of(row, strip, u0, u1);
      float rest;
      const int found = find_element<T>(a, sh.draw, row, u0, u1, t - before, kind, (int)without, zq, f, p.m, &rest, lane);
      const double others = (double)rest + other_strips(own, &sh.slice[parity][at], strip, p.m, c);
      if (found >= 0) {
        token = found;
        lp = token_logp<T>(row, c, p.m, others, found);
      }
    }
  }
  if (mine && lane == 0) {
    a.tokens[row0 + taken] = token;
    a.logp[row0 + taken] = lp;
  }
  if (rank == 0) {
    if (lane == 0) a.counts[seq] = taken;
    for (int64_t r = taken + 1 + lane; r <= n; r += 32) {
      a.tokens[row0 + r] = -1;
      a.logp[row0 + r] = 0.f;
    }
  }
  if (a.cluster > 1) cluster_sync();  // no CTA leaves while another may read its sums
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
Scale scale_of(double temperature) {
  Scale c;
  split_down(1.4426950408889634 / temperature, &c.c_hi, &c.c_lo);
  split_down(1.0 / temperature, &c.inv_hi, &c.inv_lo);
  return c;
}

int32_t check_rows(const muon_token_batch* b) {
  if (b->tokens < 0 || b->tokens > (1ll << 31) - 1) return invalid("tokens must be in [0, 2^31)");
  if (b->vocab < 1 || b->vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (b->row_stride != 0 && (b->row_stride < b->vocab || b->row_stride > (1ll << 40)))
    return invalid("row_stride must be 0 or at least vocab");
  if (b->dtype != MUON_DTYPE_F32 && b->dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  if (!(b->temperature >= 1e-20 && b->temperature <= 1e20)) return invalid("temperature must be in [1e-20, 1e20]");
  if (!aligned(b->logits, b->dtype == MUON_DTYPE_BF16 ? 2 : 4)) return invalid("logits are not aligned to their type");
  return MUON_OK;
}

// Strips of a row: their length and number.
void strips_of(int64_t vocab, int32_t dtype, int32_t* units, int32_t* strips) {
  const int64_t per = dtype == MUON_DTYPE_BF16 ? 8 : 4;
  const int64_t all = (2 * (per - 1) + vocab) / per, steps = (all + kStripStep - 1) / kStripStep;
  const int64_t mult = (steps + kMaxStrips - 1) / kMaxStrips;
  *units = (int32_t)(mult * kStripStep);
  *strips = (int32_t)((steps + mult - 1) / mult);
}

// Sampling: strips that a warp takes at a time, four where every warp of the chip has several
// such pieces.
template <typename T>
cudaError_t run_rows(SampleArgs& a, int sms, cudaStream_t s) {
  const int64_t chip = (int64_t)sms * kSampleCtas * kSampleWarps, all = a.n_seqs * a.strips;
  a.each = all >= 32 * chip ? 4 : all >= 4 * chip ? 2 : 1;
  a.pieces = (a.strips + a.each - 1) / a.each;
  // one warp an SM first
  const int64_t jobs = a.n_seqs * a.pieces, per_sm = (jobs + sms - 1) / sms;
  const int64_t warps = per_sm < kSampleWarps ? per_sm : kSampleWarps, ctas = (jobs + warps - 1) / warps, most = (int64_t)sms * kSampleCtas;
  cudaError_t e = launch(rows_kernel<T>, (int)(ctas < most ? ctas : most), (int)(32 * warps), 0, s, 1, false, a);
  if (e != cudaSuccess) return e;
  const int64_t drawers = a.n_seqs < 4ll * sms ? 1 : kDrawWarps;
  return launch(draw_kernel<T>, (int)((a.n_seqs + drawers - 1) / drawers), (int)(32 * drawers), 0, s, 1, true, a);
}

// Verification: CTAs a sequence, rows side by side.
template <typename T>
cudaError_t run_verify(SampleArgs& a, int sms, cudaStream_t s) {
  const int64_t whole = a.strips;
  int64_t cluster = 1;
  while (cluster < kMaxCluster && a.n_seqs * cluster * 2 <= 3 * sms && whole > 2 * cluster) cluster *= 2;
  const int64_t most = (a.n_drafts + 2 * a.n_seqs - 1) / a.n_seqs;  // rows of a sequence, in the mean
  a.cluster = (int32_t)cluster;
  a.strips = (int32_t)((whole + cluster - 1) / cluster);
  a.round = 1;
  if (a.n_seqs * cluster <= sms) {
    const int64_t room = kMaxStrips / a.strips, want = most < kMaxRound ? most : kMaxRound;
    a.round = (int32_t)(want < room ? want : room);
  }
  const size_t smem = (size_t)4 * a.round * a.strips * sizeof(StripSum);
  const int warps = a.strips < kSampleWarps ? a.strips : kSampleWarps;
  return launch(verify_kernel<T>, (int)(a.n_seqs * cluster), 32 * warps, smem, s, (int)cluster, false, a);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_sample_workspace_bytes(int64_t tokens, int64_t vocab, int32_t dtype, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  if (tokens < 0 || tokens > (1ll << 31) - 1) return invalid("tokens must be in [0, 2^31)");
  if (vocab < 1 || vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (dtype != MUON_DTYPE_F32 && dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  int32_t units, strips;
  strips_of(vocab, dtype, &units, &strips);
  *bytes = (size_t)tokens * strips * sizeof(StripSum);
  return MUON_OK;
}

muon_status muon_sample_tokens(const muon_token_batch* batch, const float* uniforms, int64_t* tokens, float* logp,
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!batch) return invalid("batch is NULL");
  int32_t st = check_rows(batch);
  if (st != MUON_OK) return st;
  if (batch->tokens == 0) return MUON_OK;
  if (!batch->logits) return invalid("logits is NULL");
  if (!uniforms || !tokens || !logp) return invalid("uniforms, tokens or logp is NULL");
  if (!aligned(uniforms, 4) || !aligned(tokens, 8) || !aligned(logp, 4))
    return invalid("uniforms, tokens or logp is not aligned to its type");
  SampleArgs a = {};
  a.target = batch->logits;
  a.target_stride = batch->row_stride ? batch->row_stride : batch->vocab;
  a.mask = batch->mask;
  a.sample_u = uniforms;
  a.tokens = tokens;
  a.logp = logp;
  a.target_scale = a.draft_scale = scale_of(batch->temperature);
  a.vocab = (int32_t)batch->vocab;
  a.n_seqs = batch->tokens;
  strips_of(a.vocab, batch->dtype, &a.strip_units, &a.strips);
  a.sums = static_cast<StripSum*>(workspace);
  if ((st = check_workspace(workspace, workspace_bytes, (size_t)a.n_seqs * a.strips * sizeof(StripSum))) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = batch->dtype == MUON_DTYPE_BF16 ? run_rows<__nv_bfloat16>(a, sms, s) : run_rows<float>(a, sms, s);
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

muon_status muon_verify_drafts(const muon_token_batch* target, const muon_token_batch* draft, const float* draft_logp,
                               const int64_t* draft_offsets, int64_t n_seqs, const float* accept_uniforms,
                               const float* sample_uniforms, int64_t* tokens, int64_t* counts, float* logp,
                               void* stream) {
  if (!target || !draft) return invalid("target or draft is NULL");
  int32_t st = check_rows(target);
  if (st == MUON_OK) st = check_rows(draft);
  if (st != MUON_OK) return st;
  if (n_seqs < 0 || n_seqs > (1ll << 31) - 1) return invalid("n_seqs must be in [0, 2^31)");
  if (target->tokens != draft->tokens + n_seqs)
    return invalid("the target has a row for each draft and one more for each sequence");
  if (draft->vocab != target->vocab || draft->dtype != target->dtype)
    return invalid("target and draft must have one vocabulary and one dtype");
  if (target->mask || draft->mask) return invalid("target and draft take no mask");
  if (draft_logp && !draft->logits) return invalid("draft_logp without the draft model's logits");
  if (n_seqs == 0) return MUON_OK;
  if (!target->logits || !draft_offsets || !sample_uniforms || !tokens || !counts || !logp)
    return invalid("logits, draft_offsets, sample_uniforms, tokens, counts or logp is NULL");
  if (draft->tokens > 0 && (!draft->targets || !accept_uniforms)) return invalid("drafts or accept_uniforms is NULL");
  if (!aligned(draft->targets, 8) || !aligned(draft_offsets, 8) || !aligned(tokens, 8) || !aligned(counts, 8) ||
      !aligned(draft_logp, 4) || !aligned(accept_uniforms, 4) || !aligned(sample_uniforms, 4) || !aligned(logp, 4))
    return invalid("an array is not aligned to its type");
  SampleArgs a = {};
  a.target = target->logits;
  a.target_stride = target->row_stride ? target->row_stride : target->vocab;
  a.draft = draft->logits;
  a.draft_stride = draft->row_stride ? draft->row_stride : draft->vocab;
  a.drafts = draft->targets;
  a.draft_logp = draft_logp;
  a.offsets = draft_offsets;
  a.accept_u = accept_uniforms;
  a.sample_u = sample_uniforms;
  a.tokens = tokens;
  a.counts = counts;
  a.logp = logp;
  a.n_drafts = draft->tokens;
  a.target_scale = scale_of(target->temperature);
  a.draft_scale = scale_of(draft->temperature);
  a.vocab = (int32_t)target->vocab;
  a.n_seqs = n_seqs;
  strips_of(a.vocab, target->dtype, &a.strip_units, &a.strips);
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = target->dtype == MUON_DTYPE_BF16 ? run_verify<__nv_bfloat16>(a, sms, s) : run_verify<float>(a, sms, s);
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

}  // extern "C"
