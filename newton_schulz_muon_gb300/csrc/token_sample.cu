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
// Sampling: the strips of all rows are dealt out to the CTAs of the whole chip alike, and by each to
// its warps as they come free; a second kernel draws the tokens, a warp a row.  2048 rows of 131072
// bf16 logits, a tenth masked: 90 us, of which the strips are 74 (6.5 TB/s) and the draws 9.  (Strips
// dealt to the warps beforehand: 9 us more, since masked rows leave some with less; a CTA a row: 117
// us in all.)
//
// Verification: a CTA a row (a cluster of them where there are few rows), position by position
// over all sequences, judges the row's draft; rows of a sequence whose draft was refused before
// are left out as far as that is known when their CTA starts, which changes no result.  A second
// kernel draws the tokens, a CTA or cluster for each refused draft, a warp for each other sequence.
// 512 sequences of four drafts, 131072 bf16 logits: 149 us, of which 98 are verdicts, 25 the
// difference of 236 refused drafts' rows (5 TB/s), 10 the steps around it.  (The difference formed
// where the draft is refused: 164 us, the last of them on an empty chip; a CTA a sequence, row after
// row: 191 us, since 456 sequences run at first and the others when the chip is half empty; with
// four CTAs an SM more rows are under way that turn out not to count: 9 us more.)
//
// Sums over a strip are fp32 (1024 bf16 or 512 fp32 logits, or so many times as many that a row has
// kMaxStrips; 32 or 16 at a time a lane and then the lanes'), and so are a lane's up to 16 strips
// of a row; the lanes' sums and the search among them are in 64 bits, of which the SMs do few.  How
// far from where it should a token's share of [0, 1) began, at most of 13000 to 205000 draws a kind of
// row (1000 to 1000003 logits): 8e-8 with normal logits, 7e-7 with one token above many equal ones,
// whose small terms a lane adds to a large one.
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
  StripSum* sums;            // workspace, [rows][strips of a row]
  // verification
  StripSum* q_sums;          // workspace, [drafts][all strips], where there is a draft model
  int32_t cluster;           // CTAs a row or sequence
  int32_t all_strips;        // of a row
  int32_t positions;         // of a sequence that have a CTA each; it takes every positions-th row
  int32_t draws;             // sequences of one of finish_kernel's last CTAs
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

// Units first, first + stride, ... of a row, L of them, -inf from unit u1 on.  inside: they
// all hold elements of the row only.
template <typename T, int L>
__device__ __forceinline__ void load_units(const RowUnits<T>& row, int first, int stride, int u1, bool inside,
                                           uint4 (&w)[L]) {
  constexpr uint32_t low = Vec<T>::kLowest;
  if (inside) {
    const uint4* p = reinterpret_cast<const uint4*>(row.z - row.shift) + first;
#pragma unroll
    for (int k = 0; k < L; ++k) w[k] = __ldg(p + k * stride);
  } else {
#pragma unroll
    for (int k = 0; k < L; ++k) {
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

// The rows of both models at a refused draft.
struct Refused {
  float mp, mq;  // frames
  float ratio;   // of the draft model's sum of exponentials to the target's: 1 for equal rows, which leave 0
};

// Units of the target's row and the draft model's elements at the same places.
template <typename T, int L>
struct UnitPair {
  uint4 p[L], q[L];
  __device__ __forceinline__ void load(const RowUnits<T>& row, const T* zq, int first, int stride, int u1, bool inside) {
    constexpr uint32_t low = Vec<T>::kLowest;
    load_units<T>(row, first, stride, u1, inside, p);
    if (inside && ((reinterpret_cast<uint64_t>(row.z) ^ reinterpret_cast<uint64_t>(zq)) & 15) == 0) {
      const uint4* at = reinterpret_cast<const uint4*>(zq - row.shift) + first;
#pragma unroll
      for (int k = 0; k < L; ++k) q[k] = __ldg(at + k * stride);
    } else {
#pragma unroll
      for (int k = 0; k < L; ++k) {
        const int u = first + k * stride;
        q[k] = u < u1 ? load_elems<T>(zq, row.vocab, row.first(u)) : make_uint4(low, low, low, low);
      }
    }
  }
  // max(p - q, 0) of unit k, times the sum of the draft model's exponentials.
  __device__ __forceinline__ void left_over(const SampleArgs& a, const Refused& f, int k, float (&r)[Vec<T>::N]) const {
    float y[Vec<T>::N];
    exps<T>(a.target_scale, f.mp, p[k], r);
    exps<T>(a.draft_scale, f.mq, q[k], y);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; i += 2) {
      const float2 d = split(fma2(make_f2(r[i], r[i + 1]), make_f2(-f.ratio, -f.ratio), make_f2(y[i], y[i + 1])));
      r[i] = fmaxf(-d.x, 0.f);
      r[i + 1] = fmaxf(-d.y, 0.f);
    }
  }
};

// The sums of max(p - q, 0) over the strips [k0, k1), into `to`; a step's loads are under way
// while the step before is summed (512 sequences: 149 us with 8 warps a CTA; half steps 170, and
// 149, 155 and 170 with 12, 16 and 24 warps).
template <typename T>
__device__ __forceinline__ void sum_left(const SampleArgs& a, const Refused& f, const RowUnits<T>& row, const T* zq, int k0,
                                         int k1, StripSum* to, int lane) {
  const int end = (int)min((int64_t)k1 * a.strip_units, (int64_t)row.units);
  int u = (int)min((int64_t)k0 * a.strip_units, (int64_t)row.units);
  UnitPair<T, kLoads> now;
  now.load(row, zq, u + lane, 32, end, step_inside<T>(row, u, end));
  F2 sum = make_f2(0.f, 0.f);
  int left = a.strip_units;
  for (int k = k0; k < k1;) {
    UnitPair<T, kLoads> next;
    next.load(row, zq, u + kStripStep + lane, 32, end, step_inside<T>(row, u + kStripStep, end));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      float r[Vec<T>::N];
      now.left_over(a, f, i, r);
#pragma unroll
      for (int j = 0; j < Vec<T>::N; j += 2) sum = add2(sum, make_f2(r[j], r[j + 1]));
    }
    left -= kStripStep;
    if (left == 0) {
      const float2 halves = split(sum);
      const float whole = warp_sum(halves.x + halves.y);
      if (lane == 0) to[k - k0] = StripSum{0.f, whole};
      sum = make_f2(0.f, 0.f);
      left = a.strip_units;
      ++k;
    }
    u += kStripStep;
    now = next;
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

// Strips' weights, of which a lane has some consecutive ones: its sum, and the sum up to its last.
struct StripScan {
  float w;
  double end;
};
__device__ __forceinline__ void strips_of_lane(int strips, int lane, int& k0, int& k1) {
  const int per = (strips + 31) / 32;
  k0 = min(lane * per, strips);
  k1 = min(k0 + per, strips);
}
template <typename F>
__device__ __forceinline__ StripScan scan_strips(int strips, int lane, F weight) {
  int k0, k1;
  strips_of_lane(strips, lane, k0, k1);
  StripScan r{0.f, 0.};
#pragma unroll 1
  for (int k = k0; k < k1; ++k) r.w += weight(k);
  r.end = warp_scan64((double)r.w, lane);
  return r;
}

// The strip in which the cumulated weight exceeds t (one of weight 0 never does), else the
// last of positive weight; -1: none.  before: the weights before it.  weight(k), k < strips.
template <typename F>
__device__ __forceinline__ int find_strip(const StripScan& scan, int strips, double t, double* before, int lane, F weight) {
  const unsigned above = __ballot_sync(0xFFFFFFFFu, scan.w > 0.f && scan.end > t);
  const unsigned some = __ballot_sync(0xFFFFFFFFu, scan.w > 0.f);
  if (some == 0) return -1;
  const int l = above ? __ffs(above) - 1 : 31 - __clz(some);
  const double start = scan.end - (double)scan.w;
  const float need = (float)(t - start);
  int k0, k1;
  strips_of_lane(strips, lane, k0, k1);
  float at = 0.f, begun = 0.f;
  int strip = 0;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) {
    const float x = weight(k);
    if (x > 0.f) {
      strip = k;
      begun = at;
      if (at + x > need) break;
    }
    at += x;
  }
  *before = __shfl_sync(0xFFFFFFFFu, start + (double)begun, l);
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
      UnitPair<T, kLoads> z;
      z.load(row, zq, first, 1, u1, inside);
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        float x[N];
        z.left_over(a, f, k, x);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          sh.weight[lane][k * N + i] = x[i];
          v += x[i];
        }
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
// A CTA's jobs are dealt to its warps as they come, since masked rows take no time.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, kSampleCtas) rows_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ int next;
  if (threadIdx.x == 0) next = 0;
  __syncthreads();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t jobs = a.n_seqs * a.pieces;
  for (;;) {
    int n;
    if (lane == 0) n = atomicAdd(&next, 1);
    const int64_t job = (int64_t)blockIdx.x + (int64_t)__shfl_sync(0xFFFFFFFFu, n, 0) * gridDim.x;
    if (job >= jobs) break;
    const int64_t t = job / a.pieces;
    if (a.mask != nullptr && a.mask[t] == 0) continue;
    const int k0 = (int)(job - t * a.pieces) * a.each;
    const RowUnits<T> row(a.target, t, a.target_stride, a.vocab);
    sum_strips<T>(row, a.target_scale, a.strip_units, k0, min(k0 + a.each, a.strips), a.sums + t * a.strips + k0, lane);
  }
}

// Draws row r's token from the sums of its strips, which are kept in `own`.  A warp's time here is
// that of a chain of steps, in which 64-bit sums weigh most (a warp's takes an SM 16 cycles).
template <typename T>
__device__ __forceinline__ void draw_row(const SampleArgs& a, int64_t r, const StripSum* from, int strips, float u,
                                         StripSum* own, DrawSpace& sh, int64_t* token, float* logp, int lane) {
  const Scale& c = a.target_scale;
  const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
  const float2* sums = reinterpret_cast<const float2*>(from);
  float m = -INFINITY;
#pragma unroll 4
  for (int k = lane; k < strips; k += 32) {
    const float2 x = __ldcg(sums + k);
    own[k] = StripSum{x.x, x.y};
    m = fmaxf(m, x.x);
  }
  m = warp_max(m);
  __syncwarp();
  const StripScan scan = scan_strips(strips, lane, [&](int k) { return own[k].s *= factor(c, own[k].m, m); });
  const RowSum p{__shfl_sync(0xFFFFFFFFu, scan.end, 31), m, 0.};
  *token = -1;
  *logp = NAN;
  if (!usable(p)) return;
  auto weight = [&](int k) { return own[k].s; };
  double before = 0.;
  const double at = u < 1.f ? (double)u * p.s : (double)INFINITY;  // 1 and above: the last token
  const int strip = find_strip(scan, strips, at, &before, lane, weight);
  const int u0 = strip * a.strip_units, u1 = min(u0 + a.strip_units, row.units);
  float rest;
  const int found = find_element<T>(a, sh, row, u0, u1, at - before, kPlain, -1, nullptr, Refused{}, m, &rest, lane);
  int k0, k1;
  strips_of_lane(strips, lane, k0, k1);
  float others = 0.f;
#pragma unroll 1
  for (int k = k0; k < k1; ++k) others += k == strip ? 0.f : weight(k);
  if (found < 0) return;
  *token = found;
  *logp = token_logp<T>(row, c, m, (double)rest + (double)others, found);
}

constexpr int kDrawWarps = 4;  // of a CTA (1, 2 and 4 alike)
template <typename T>
__global__ void __launch_bounds__(kDrawWarps * 32) draw_kernel(const __grid_constant__ SampleArgs a) {
  __shared__ DrawSpace space[kDrawWarps];
  __shared__ StripSum table[kDrawWarps][kMaxStrips];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + warp;
  const bool live = t < a.n_seqs && (a.mask == nullptr || a.mask[t] != 0);
  const float u = live ? fmaxf(a.sample_u[t], 0.f) : 0.f;
  griddep_wait();
  if (t >= a.n_seqs) return;
  int64_t token = -1;
  float logp = 0.f;
  if (live) draw_row<T>(a, t, a.sums + t * a.strips, a.strips, u, table[warp], space[warp], &token, &logp, lane);
  if (lane == 0) {
    a.tokens[t] = token;
    a.logp[t] = logp;
  }
}

// ---------------------------------------------------------------------------
// verification
// ---------------------------------------------------------------------------
struct Sequence {
  int64_t lo, n, row0;  // first draft, drafts, first row
};
// Offsets out of order or range lead to nothing outside the arrays.
__device__ __forceinline__ Sequence sequence_of(const SampleArgs& a, int64_t s) {
  Sequence q;
  q.lo = min(max(a.offsets[s], (int64_t)0), a.n_drafts);
  q.n = min(max(a.offsets[s + 1], q.lo), a.n_drafts) - q.lo;
  q.row0 = q.lo + s;
  return q;
}

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

// A CTA's strips [strip0, strip0 + a.strips) of a row: the units of strip k.
template <typename T>
__device__ __forceinline__ void units_of(const SampleArgs& a, const RowUnits<T>& row, int strip, int& u0, int& u1) {
  u0 = (int)min((int64_t)strip * a.strip_units, (int64_t)row.units);
  u1 = min(u0 + a.strip_units, row.units);
}

// Adds up n strips (-1: no strip is left out of rest): warp-wide, the same in every lane.
__device__ __forceinline__ RowSum sum_table(const StripSum* table, int n, const Scale& c, int skip, int lane) {
  float m = -INFINITY;
#pragma unroll 4
  for (int k = lane; k < n; k += 32) m = fmaxf(m, table[k].m);
  RowSum r;
  r.m = warp_max(m);
  float sum = 0.f, rest = 0.f;
#pragma unroll 4
  for (int k = lane; k < n; k += 32) {
    const float x = table[k].s * factor(c, table[k].m, r.m);
    sum += x;
    rest += k == skip ? 0.f : x;
  }
  r.s = warp_sum64((double)sum);
  r.rest = warp_sum64((double)rest);
  return r;
}

// Adds up the CTAs' parts of a row.
__device__ __forceinline__ RowSum merge(const RowSum* slice, const Scale& c, int cluster, int rank, int lane) {
  if (cluster == 1) return *slice;
  RowSum t{0., -INFINITY, 0.};
  if (lane < cluster) t = load_peer(slice, lane, rank);
  RowSum r;
  r.m = warp_max(t.m);
  const double f = (double)factor(c, t.m, r.m);
  r.s = warp_sum64(t.s * f);
  r.rest = warp_sum64(t.rest * f);
  return r;
}

// Strip sums of a row of the target (and of the draft model's, where its probabilities are
// needed), the verdict on its draft and, as if it were taken, the draft's log p.
// counts[s], all ones at first, becomes the first refused position.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 3) judge_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ StripSum tables[];  // [target and draft][strips]
  __shared__ RowSum slice[2][2];
  __shared__ bool stop, refusing;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int64_t unit = blockIdx.x / a.cluster, first = unit / a.n_seqs, seq = unit - first * a.n_seqs;
  unsigned long long* const refused = reinterpret_cast<unsigned long long*>(a.counts) + seq;
  unsigned long long seen = ~0ull;  // the first refused position, as far as it is known
  if (a.cluster == 1 && threadIdx.x == 0) seen = __ldcg(refused);
  const Sequence e = sequence_of(a, seq);
  const bool both = a.draft != nullptr && a.draft_logp == nullptr;
  const int strip0 = rank * a.strips;
  // of the CTA's strips this warp's
  const int per_warp = (a.strips + warps - 1) / warps, mine0 = min(warp * per_warp, a.strips), mine1 = min(mine0 + per_warp, a.strips);
  griddep_launch_dependents();
  int parity = 0;
  for (int64_t i = first; i <= e.n; i += a.positions, parity ^= 1) {
    if (a.cluster == 1) {  // CTAs of a cluster must go the same way
      if (threadIdx.x == 0) {
        if (i != first) seen = __ldcg(refused);
        stop = seen < (unsigned long long)i;
      }
      __syncthreads();
      if (stop) break;
    }
    const int64_t r = e.row0 + i, d = e.lo + i;
    const bool drafted = i < e.n;
    int64_t y = -1;
    float u = 0.f, zy = 0.f, logq = 0.f;
    if (warp == 0 && drafted) {  // on their way while the row is read
      y = a.drafts[d];
      u = a.accept_u[d];
      if (!both && a.draft_logp != nullptr) logq = a.draft_logp[d];
    }
    const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
    sum_strips<T>(row, a.target_scale, a.strip_units, strip0 + mine0, strip0 + mine1, tables + mine0, lane);
    if (both && drafted) {
      const RowUnits<T> draft(a.draft, d, a.draft_stride, a.vocab);
      sum_strips<T>(draft, a.draft_scale, a.strip_units, strip0 + mine0, strip0 + mine1, tables + a.strips + mine0, lane);
    }
    if (warp == 0) {
      if (y < 0 || y >= a.vocab) y = -1;
      if (y >= 0) {
        zy = Vec<T>::load(row.z + y);
        if (both) logq = Vec<T>::load(reinterpret_cast<const T*>(a.draft) + d * a.draft_stride + y);
      }
    }
    __syncthreads();
    // the strips' sums, for the kernel that draws
    for (int k = threadIdx.x; k < a.strips && strip0 + k < a.all_strips; k += blockDim.x) {
      a.sums[r * a.all_strips + strip0 + k] = tables[k];
      if (both && drafted) a.q_sums[d * a.all_strips + strip0 + k] = tables[a.strips + k];
    }
    if (drafted) {
      const int strip = y < 0 ? -1 : ((int)y + row.shift) / N / a.strip_units - strip0;  // of the draft, in this CTA's
      if (warp == 0) {
        const RowSum p = sum_table(tables, a.strips, a.target_scale, strip, lane);
        if (lane == 0) slice[parity][0] = p;
        if (both) {
          const RowSum q = sum_table(tables + a.strips, a.strips, a.draft_scale, -1, lane);
          if (lane == 0) slice[parity][1] = q;
        }
        __syncwarp();
      }
      if (a.cluster > 1) cluster_sync();
      if (warp == 0) {
        if (lane == 0) refusing = false;
        const RowSum p = merge(&slice[parity][0], a.target_scale, a.cluster, rank, lane);
        const float x = zy - p.m;
        const float logp = __fmaf_rn(x, a.target_scale.inv_hi, x * a.target_scale.inv_lo) - logf((float)p.s);
        bool ok = usable(p) && y >= 0;
        if (both) {
          const RowSum q = merge(&slice[parity][1], a.draft_scale, a.cluster, rank, lane);
          const float z = logq - q.m;
          logq = __fmaf_rn(z, a.draft_scale.inv_hi, z * a.draft_scale.inv_lo) - logf((float)q.s);
          ok = ok && usable(q);
        }
        ok = ok && u < expf(logp - logq);
        if (!ok) {
          unsigned long long before = ~0ull;
          if (rank == 0 && lane == 0) before = atomicMin(refused, (unsigned long long)i);
          // not where an earlier draft was refused meanwhile; CTAs of a cluster go the same way
          if (lane == 0) refusing = a.cluster > 1 || before >= (unsigned long long)i;
        } else if (strip >= 0 && strip < a.strips) {
          int u0, u1;
          units_of(a, row, strip0 + strip, u0, u1);
          const double rest = (lane == 0 ? p.rest : 0.) + (double)sum_without<T>(row, a.target_scale, p.m, u0, u1, (int)y, lane);
          const float exact = token_logp<T>(row, a.target_scale, p.m, rest, (int)y);
          if (lane == 0) {
            a.tokens[r] = y;
            a.logp[r] = exact;
          }
        }
      }
    }
    __syncthreads();  // the tables are free
    // a refused draft's token needs the draft model's row, too, and no row behind it
    if (drafted && refusing) {
      if (a.draft != nullptr && !both) {
        const RowUnits<T> draft(a.draft, d, a.draft_stride, a.vocab);
        sum_strips<T>(draft, a.draft_scale, a.strip_units, strip0 + mine0, strip0 + mine1, tables + mine0, lane);
        __syncthreads();
        for (int k = threadIdx.x; k < a.strips && strip0 + k < a.all_strips; k += blockDim.x)
          a.q_sums[d * a.all_strips + strip0 + k] = tables[k];
      }
      break;
    }
  }
  if (a.cluster > 1) cluster_sync();  // no CTA leaves while another may read its sums
}

// The token after a sequence's taken drafts, and -1 behind it.  A refused draft's rows take a CTA or
// cluster; the grid's last CTAs draw for the sequences whose drafts were all taken, a warp for
// each (with a CTA for these too, the refused ones among 512 sequences of four drafts waited for
// them: 14 us more).
constexpr int kDraws = 4;  // sequences of one of the last CTAs
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 2) finish_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  extern __shared__ StripSum tables[];  // [2][strips]: of p, of the difference.  [draws][all strips]
  __shared__ double share;              // this CTA's part of the weights
  __shared__ DrawSpace space[kDraws];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t drawers = a.n_seqs * a.cluster;  // the first of the last CTAs
  if (blockIdx.x >= drawers) {
    const int64_t seq = (blockIdx.x - drawers) * a.draws + warp;
    if (warp >= a.draws || seq >= a.n_seqs) return;
    const Sequence e = sequence_of(a, seq);
    const float u = fmaxf(a.sample_u[seq], 0.f);
    griddep_wait();
    if (__ldcg(a.counts + seq) >= 0) return;  // refused
    const int64_t r = e.row0 + e.n;
    int64_t token;
    float logp;
    draw_row<T>(a, r, a.sums + r * a.all_strips, a.all_strips, u, tables + warp * a.all_strips, space[warp], &token, &logp, lane);
    if (lane == 0) {
      a.tokens[r] = token;
      a.logp[r] = logp;
      a.counts[seq] = e.n;
    }
    return;
  }
  const int rank = a.cluster > 1 ? (int)cluster_ctarank() : 0;
  const int64_t seq = blockIdx.x / a.cluster;
  const Sequence e = sequence_of(a, seq);
  const int strip0 = rank * a.strips;
  const int per_warp = (a.strips + warps - 1) / warps, mine0 = min(warp * per_warp, a.strips), mine1 = min(mine0 + per_warp, a.strips);
  const Scale& c = a.target_scale;
  griddep_wait();
  const unsigned long long first_refused = __ldcg(reinterpret_cast<unsigned long long*>(a.counts) + seq);
  // all taken: all ones, or the number of drafts where it has been drawn for
  if (first_refused >= (unsigned long long)e.n) return;
  const int64_t taken = (int64_t)first_refused, r = e.row0 + taken, d = e.lo + taken;
  const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
  // the row's sums, by every warp alike, and this CTA's strips of them
  const StripSum* const all = a.sums + r * a.all_strips;
  const RowSum p = sum_table(all, a.all_strips, c, -1, lane);
  StripSum* const own = tables;
  StripSum* const left = tables + a.strips;
  for (int k = threadIdx.x; k < a.strips; k += blockDim.x)
    own[k] = strip0 + k < a.all_strips ? all[strip0 + k] : StripSum{-INFINITY, 0.f};
  bool fine = usable(p);
  int kind = kPlain;
  int without = -1;
  int without_strip = -1;
  float without_sum = 0.f;
  Refused f{};
  const T* zq = nullptr;
  if (fine && a.draft == nullptr) {
    const int64_t x = a.drafts[d];
    if (x >= 0 && x < a.vocab) {  // any other is no token, and all of p is left
      kind = kWithout;
      without = (int)x;
      const int k = (without + row.shift) / N / a.strip_units;
      if (warp == 0 && k >= strip0 && k < strip0 + a.strips) {
        int u0, u1;
        units_of(a, row, k, u0, u1);
        without_strip = k - strip0;
        without_sum = warp_sum(sum_without<T>(row, c, p.m, u0, u1, without, lane));
      }
    }
  } else if (fine) {
    kind = kLeft;
    const RowUnits<T> draft(a.draft, d, a.draft_stride, a.vocab);
    zq = draft.z;
    const RowSum q = sum_table(a.q_sums + d * a.all_strips, a.all_strips, a.draft_scale, -1, lane);
    fine = usable(q);
    f = Refused{p.m, q.m, (float)(q.s / p.s)};
    if (fine) sum_left<T>(a, f, row, zq, strip0 + mine0, strip0 + mine1, left + mine0, lane);
  }
  __syncthreads();
  if (rank == 0 && (warp == 1 || warps == 1)) {
    for (int64_t i = taken + 1 + lane; i <= e.n; i += 32) {
      a.tokens[e.row0 + i] = -1;
      a.logp[e.row0 + i] = 0.f;
    }
  }
  if (warp != 0) return;  // the cluster's barriers wait for the warps that are left

  int64_t token = -1;
  bool mine = rank == 0;  // this CTA writes the token
  float lp = NAN;
  if (fine) {
    auto plain = [&](int k) { return own[k].s * factor(c, own[k].m, p.m); };
    auto weight = [&](int k) { return kind == kLeft ? left[k].s : kind == kWithout && k == without_strip ? without_sum : plain(k); };
    // each CTA's share of the weights in its lane, and their running sum
    StripScan scan;
    double v;
    for (;;) {
      scan = scan_strips(a.strips, lane, weight);
      v = __shfl_sync(0xFFFFFFFFu, scan.end, 31);
      if (a.cluster > 1) {
        if (lane == 0) share = v;
        cluster_sync();
        v = lane >= a.cluster ? 0. : lane == rank ? v : load_peer(&share, lane);
        cluster_sync();  // share is free
      } else if (lane > 0) {
        v = 0.;
      }
      // nothing is left over where the two models agree, and the refusal was one of rounding
      if (kind == kPlain || __any_sync(0xFFFFFFFFu, v > 0.)) break;
      kind = kPlain;
    }
    const double upto = warp_scan64(v, lane), sum = __shfl_sync(0xFFFFFFFFu, upto, 31);
    const float su = fmaxf(a.sample_u[seq], 0.f);
    const double t = su < 1.f ? (double)su * sum : (double)INFINITY;  // 1 and above: the last token
    const unsigned over = __ballot_sync(0xFFFFFFFFu, v > 0. && upto > t);
    const unsigned any = __ballot_sync(0xFFFFFFFFu, v > 0.);
    const int owner = over ? __ffs(over) - 1 : 31 - __clz(any);
    mine = rank == owner;
    if (mine) {
      const double here = t - __shfl_sync(0xFFFFFFFFu, upto - v, owner);  // of this CTA's weights
      double before = 0.;
      const int strip = find_strip(scan, a.strips, here, &before, lane, weight);
      int u0, u1;
      units_of(a, row, strip0 + strip, u0, u1);
      float rest;
      const int found = find_element<T>(a, space[0], row, u0, u1, here - before, kind, without, zq, f, p.m, &rest, lane);
      float others = 0.f;
#pragma unroll 4
      for (int k = lane; k < a.all_strips; k += 32)
        if (k != strip0 + strip) others += all[k].s * factor(c, all[k].m, p.m);
      if (found >= 0) {
        token = found;
        lp = token_logp<T>(row, c, p.m, (double)rest + (double)others, found);
      }
    }
  }
  if (mine && lane == 0) {
    a.tokens[r] = token;
    a.logp[r] = lp;
  }
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
// such pieces (2048 rows of 131072 bf16 logits: 90 us, 99 with two, 89 with eight).
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
  return launch(draw_kernel<T>, (int)((a.n_seqs + kDrawWarps - 1) / kDrawWarps), 32 * kDrawWarps, 0, s, 1, true, a);
}

// CTAs a row: as many as keep every SM busy with three, and have two strips each.
int cluster_of(int64_t units, int64_t strips, int sms) {
  int cluster = 1;
  while (cluster < kMaxCluster && units * cluster * 2 <= 3 * sms && strips > 2 * cluster) cluster *= 2;
  return cluster;
}

// The strips of a row divided among the CTAs of a cluster, and a CTA's warps.
int share_strips(SampleArgs& a, int64_t units, int sms) {
  a.cluster = cluster_of(units, a.all_strips, sms);
  a.strips = (a.all_strips + a.cluster - 1) / a.cluster;
  return a.strips < kSampleWarps ? a.strips : kSampleWarps;
}

template <typename T>
cudaError_t run_verify(SampleArgs& a, int sms, cudaStream_t s) {
  cudaError_t e = cudaMemsetAsync(a.counts, 0xFF, (size_t)a.n_seqs * sizeof(int64_t), s);
  if (e != cudaSuccess) return e;
  // the mean number of rows, rounded up, and twice as many where that costs no second round of
  // CTAs; longer sequences' CTAs take several
  const int64_t rows = a.n_drafts + a.n_seqs, most = 0x7FFFFFFF / kMaxCluster / a.n_seqs;
  int64_t positions = (rows + a.n_seqs - 1) / a.n_seqs;
  int warps = share_strips(a, rows, sms);
  if (a.n_seqs * positions * a.cluster <= 3 * sms) positions *= 2;
  a.positions = (int32_t)(positions < most ? positions : most < 1 ? 1 : most);
  e = launch(judge_kernel<T>, (int)(a.n_seqs * a.positions * a.cluster), 32 * warps, (size_t)2 * a.strips * sizeof(StripSum), s,
             a.cluster, false, a);
  if (e != cudaSuccess) return e;
  warps = share_strips(a, a.n_seqs, sms);
  a.draws = a.n_seqs < 4 * sms ? 1 : warps < kDraws ? warps : kDraws;
  const int64_t drawers = (a.n_seqs + a.draws - 1) / a.draws, ctas = (a.n_seqs + (drawers + a.cluster - 1) / a.cluster) * a.cluster;
  const int strips = 2 * a.strips > a.draws * a.all_strips ? 2 * a.strips : a.draws * a.all_strips;
  return launch(finish_kernel<T>, (int)ctas, 32 * warps, strips * sizeof(StripSum), s, a.cluster, true, a);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_sample_workspace_bytes(int64_t rows, int64_t vocab, int32_t dtype, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  if (rows < 0 || rows > (1ll << 32) - 1) return invalid("rows must be in [0, 2^32)");
  if (vocab < 1 || vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (dtype != MUON_DTYPE_F32 && dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  int32_t units, strips;
  strips_of(vocab, dtype, &units, &strips);
  *bytes = (size_t)rows * strips * sizeof(StripSum);
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
                               void* workspace, size_t workspace_bytes, void* stream) {
  if (!target || !draft) return invalid("target or draft is NULL");
  int32_t st = check_rows(target);
  if (st == MUON_OK) st = check_rows(draft);
  if (st != MUON_OK) return st;
  if (n_seqs < 0 || n_seqs > (1ll << 30) - 1) return invalid("n_seqs must be in [0, 2^30)");
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
  strips_of(a.vocab, target->dtype, &a.strip_units, &a.all_strips);
  const size_t row = (size_t)a.all_strips * sizeof(StripSum), rows = (size_t)(a.n_drafts + n_seqs);
  if ((st = check_workspace(workspace, workspace_bytes, (rows + (draft->logits ? (size_t)a.n_drafts : 0)) * row)) != MUON_OK)
    return st;
  a.sums = static_cast<StripSum*>(workspace);
  a.q_sums = draft->logits ? a.sums + rows * a.all_strips : nullptr;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = target->dtype == MUON_DTYPE_BF16 ? run_verify<__nv_bfloat16>(a, sms, s) : run_verify<float>(a, sms, s);
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

}  // extern "C"
