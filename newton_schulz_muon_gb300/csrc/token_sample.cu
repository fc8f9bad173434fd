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
// Strips of all rows are dealt out to the warps of the whole chip alike, a few strips a time,
// and a small kernel draws the tokens afterwards, a warp a row: with a CTA a row, 2048 rows of
// 131072 bf16 logits took 117 us (the ends of rows, and 3.03 rounds of CTAs that took 4), ROWS_US so.
// Drafts are verified position by position: the warp that finishes a row decides on its
// draft, and later rows of a sequence whose draft was refused are left out as far as that is
// known when their turn comes.  (What is left out changes no result.)
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
};

struct SampleArgs {
  const void* target;
  const void* draft;         // null: drafts that were certain
  const uint8_t* mask;       // rows of a sampling call that take part; or null
  const int64_t* drafts;
  const float* draft_logp;   // or null
  const int64_t* offsets;    // [n_seqs + 1]; null: sampling, a row a sequence
  const float* accept_u;
  const float* sample_u;
  int64_t* tokens;
  int64_t* counts;
  float* logp;
  int64_t target_stride, draft_stride;
  int64_t n_drafts, n_seqs;
  Scale target_scale, draft_scale;
  int32_t vocab;
  int32_t strip_units;       // a multiple of kStripStep
  int32_t strips;            // of a row
  int32_t each;              // strips that a warp takes at a time
  int32_t pieces;            // of a row: strips / each, rounded up
  int32_t both;              // the draft model's rows are read with the target's
  // workspace
  StripSum* p;               // [target rows][strips]
  StripSum* q;               // of the draft model: both, [drafts][strips]; else [n_seqs][strips], where a draft was refused
  float* left;               // [n_seqs][strips] max(p - q, 0)
  RowSum* p_total;           // [target rows]
  RowSum* q_total;           // [drafts] or [n_seqs]
  uint32_t* done;            // [target rows] pieces that are done; zero at first, as the next two
  uint32_t* q_done;          // [n_seqs]
  uint32_t* refused;         // [n_seqs] 2^31 - 1 minus the first refused draft, 0: none
  int64_t* longest;          // the most drafts of a sequence
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

// The sum of exponentials over the units [u0, u1) of a row; the same in every lane.
template <typename T>
__device__ __forceinline__ StripSum strip_sum(const RowUnits<T>& row, const Scale& c, int u0, int u1, int lane) {
  StripSum t{-INFINITY, 0.f};
  for (int u = u0; u < u1; u += kStripStep) {
    uint4 w[kLoads];
    load_units<T>(row, u + lane, 32, u1, step_inside<T>(row, u, u1), w);
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
  return t;
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

// The first element of the units [u0, u1) at which the cumulated weight exceeds t (a token
// of weight 0 never does), or the last of positive weight, or -1.  weights(first, inside, w):
// those of the units first .. first + kLoads - 1 (0 from u1 on), which a lane takes side by
// side.  A lane's weights are summed in fp32, the lanes' in 64 bits, of which the SMs do few.
template <typename T, typename F>
__device__ __forceinline__ int pick_element(const RowUnits<T>& row, int u0, int u1, double t, int lane, F weights) {
  constexpr int N = Vec<T>::N;
  double before = 0.;
  int last = -1;
  for (int u = u0; u < u1; u += kStripStep) {
    const int first = u + lane * kLoads;
    float w[kLoads * N];
    weights(first, step_inside<T>(row, u, u1), w);
    float s = 0.f;
    int positive = -1;
#pragma unroll
    for (int i = 0; i < kLoads * N; ++i) {
      s += w[i];
      if (w[i] > 0.f) positive = i;
    }
    const double upto = before + warp_scan64((double)s, lane);
    const unsigned over = __ballot_sync(0xFFFFFFFFu, positive >= 0 && upto > t);
    const unsigned any = __ballot_sync(0xFFFFFFFFu, positive >= 0);
    if (over) {
      const int l = __ffs(over) - 1;
      const float rest = (float)(t - (upto - (double)s));  // of the lane's weights
      int found = positive;
      float c = 0.f;
      bool passed = false;
#pragma unroll
      for (int i = 0; i < kLoads * N; ++i) {
        c += w[i];
        if (!passed && w[i] > 0.f && c > rest) {
          found = i;
          passed = true;
        }
      }
      return __shfl_sync(0xFFFFFFFFu, row.first(first) + found, l);
    }
    if (any) last = __shfl_sync(0xFFFFFFFFu, row.first(first) + positive, 31 - __clz(any));
    before = __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return last;
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

// log p of a token of the strip [u0, u1): the strip is summed again without the token, so
// that a nearly certain token keeps its digits.  rest: each lane's part of the sum over the
// other strips, in the row's frame m.
template <typename T>
__device__ __forceinline__ float token_logp(const RowUnits<T>& row, const Scale& c, float m, double rest, int u0, int u1,
                                            int token, int lane) {
  rest += (double)sum_without<T>(row, c, m, u0, u1, token, lane);
  float s = (float)warp_sum64(rest);
  const float d = Vec<T>::load(row.z + token) - m;
  const float x = __fmaf_rn(d, c.inv_hi, d * c.inv_lo);
  // x <= 0; at the row's largest logit, log1p keeps the digits of a nearly certain token
  s = __fmaf_rn(x == 0.f ? s : s - 1.f, kExpLow, s);
  return x == 0.f ? 0.f - log1pf(s) : x - logf(s + expf(x));
}

__device__ __forceinline__ bool usable(const RowSum& t) { return t.s > 0. && t.s < (double)INFINITY; }

// The sum over a row's strips, and of the lane's share of them (consecutive strips), in the
// frame of the largest.
__device__ __forceinline__ RowSum row_sum(const SampleArgs& a, const StripSum* t, const Scale& c, int lane) {
  float m = -INFINITY;
  for (int k = lane; k < a.strips; k += 32) m = fmaxf(m, __ldcg(reinterpret_cast<const float2*>(t) + k).x);
  RowSum r;
  r.m = warp_max(m);
  double s = 0.;
  for (int k = lane; k < a.strips; k += 32) {
    const float2 x = __ldcg(reinterpret_cast<const float2*>(t) + k);
    s += (double)(x.y * factor(c, x.x, r.m));
  }
  r.s = warp_sum64(s);
  return r;
}

__device__ __forceinline__ RowSum load_total(const RowSum* p) {
  RowSum r;
  r.s = __ldcg(&p->s);
  r.m = __ldcg(&p->m);
  return r;
}

// A sequence's drafts; offsets out of order or range lead to nothing outside the arrays.
struct Sequence {
  int64_t lo, n;
};
__device__ __forceinline__ Sequence sequence_of(const SampleArgs& a, int64_t s) {
  Sequence q;
  q.lo = min(max(a.offsets[s], (int64_t)0), a.n_drafts);
  q.n = min(max(a.offsets[s + 1], q.lo), a.n_drafts) - q.lo;
  return q;
}

// The sums of the strips [k0, k1) of a row.
template <typename T>
__device__ __forceinline__ void sum_strips(const SampleArgs& a, const RowUnits<T>& row, const Scale& c, int k0, int k1,
                                           StripSum* to, int lane) {
  for (int k = k0; k < k1; ++k) {
    const int u0 = (int)min((int64_t)k * a.strip_units, (int64_t)row.units), u1 = min(u0 + a.strip_units, row.units);
    const StripSum t = strip_sum<T>(row, c, u0, u1, lane);
    if (lane == 0) __stcg(reinterpret_cast<float2*>(to) + k, make_float2(t.m, t.s));
  }
}

// Whether the calling warp's piece is the last of `all`; what the other warps wrote is then
// visible to every lane.
__device__ __forceinline__ bool last_piece(uint32_t* done, uint32_t all, int lane) {
  uint32_t before = 0;
  if (lane == 0) {
    __threadfence();
    before = atomicAdd(done, 1u);
  }
  const bool last = __shfl_sync(0xFFFFFFFFu, before, 0) == all - 1;
  if (last) __threadfence();
  return last;
}

// Clears the counters and finds the longest sequence.
constexpr int kSetupThreads = 1024;
__global__ void __launch_bounds__(kSetupThreads) setup_kernel(const __grid_constant__ SampleArgs a) {
  griddep_launch_dependents();
  __shared__ long long most[kSetupThreads / 32];
  long long n = 0;
  for (int64_t s = threadIdx.x; s < a.n_seqs; s += kSetupThreads) {
    n = max(n, (long long)sequence_of(a, s).n);
    a.q_done[s] = 0;
    a.refused[s] = 0;
  }
  for (int64_t r = threadIdx.x; r < a.n_drafts + a.n_seqs; r += kSetupThreads) a.done[r] = 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n = max(n, __shfl_xor_sync(0xFFFFFFFFu, n, o));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kSetupThreads / 32; ++k) n = max(n, most[k]);
    *a.longest = n;
  }
}

// Strip sums of sampled rows.
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
    sum_strips<T>(a, row, a.target_scale, k0, min(k0 + a.each, a.strips), a.p + t * a.strips, lane);
  }
}

// Strip sums of the target's rows (and, where `both`, of the draft model's), position by
// position over all sequences, and the verdict on each draft.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, kSampleCtas) verify_kernel(const __grid_constant__ SampleArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  const int sets = a.both ? 2 : 1, per_row = a.pieces * sets;
  const int64_t jobs = (__ldcg(a.longest) + 1) * a.n_seqs * per_row;
  // a job's sequence and what is known of it are read while the job before is worked on
  int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  int64_t i = 0, s = 0;
  int piece = 0;
  Sequence q{0, -1};
  uint32_t refused = 0;
  auto look = [&](int64_t j) {
    if (j >= jobs) return;
    const int64_t r = j / per_row;
    piece = (int)(j - r * per_row);
    i = r / a.n_seqs;
    s = r - i * a.n_seqs;
    q = sequence_of(a, s);
    refused = __ldcg(a.refused + s);
  };
  look(job);
  while (job < jobs) {
    const int64_t at = i, seq = s;
    const Sequence own = q;
    const bool of_draft = piece >= a.pieces;
    const int k0 = (of_draft ? piece - a.pieces : piece) * a.each;
    const uint32_t known = refused;
    job += warps;
    look(job);
    // no such row, or one behind a refused draft
    if (at > own.n || (known != 0 && (int64_t)(0x7FFFFFFFu - known) < at)) continue;
    const int64_t r = own.lo + seq + at, d = own.lo + at;
    if (of_draft) {
      if (at == own.n) continue;
      const RowUnits<T> row(a.draft, d, a.draft_stride, a.vocab);
      sum_strips<T>(a, row, a.draft_scale, k0, min(k0 + a.each, a.strips), a.q + d * a.strips, lane);
    } else {
      const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
      sum_strips<T>(a, row, a.target_scale, k0, min(k0 + a.each, a.strips), a.p + r * a.strips, lane);
    }
    if (!last_piece(a.done + r, at < own.n ? per_row : a.pieces, lane)) continue;
    const RowSum p = row_sum(a, a.p + r * a.strips, a.target_scale, lane);
    if (lane == 0) a.p_total[r] = p;
    if (at == own.n) continue;
    RowSum dq{1., 0.f};
    if (a.both) {
      dq = row_sum(a, a.q + d * a.strips, a.draft_scale, lane);
      if (lane == 0) a.q_total[d] = dq;
    }
    if (lane == 0) {
      const int64_t y = a.drafts[d];
      bool ok = usable(p) && usable(dq) && y >= 0 && y < a.vocab;
      if (ok) {
        const float x = Vec<T>::load(reinterpret_cast<const T*>(a.target) + r * a.target_stride + y) - p.m;
        const float logp = __fmaf_rn(x, a.target_scale.inv_hi, x * a.target_scale.inv_lo) - logf((float)p.s);
        float logq = a.draft_logp != nullptr ? a.draft_logp[d] : 0.f;
        if (a.both) {
          const float z = Vec<T>::load(reinterpret_cast<const T*>(a.draft) + d * a.draft_stride + y) - dq.m;
          logq = __fmaf_rn(z, a.draft_scale.inv_hi, z * a.draft_scale.inv_lo) - logf((float)dq.s);
        }
        ok = a.accept_u[d] < expf(logp - logq);
      }
      if (!ok) atomicMax(a.refused + seq, 0x7FFFFFFFu - (uint32_t)at);
    }
  }
}

// Where sequence s stopped: its drafts, the number of them that were taken, whether the next
// was refused.
struct Stop {
  Sequence q;
  int64_t taken;
  bool refused;
};
__device__ __forceinline__ Stop stop_of(const SampleArgs& a, int64_t s) {
  Stop r;
  r.q = sequence_of(a, s);
  const uint32_t known = __ldcg(a.refused + s);
  r.refused = known != 0;
  r.taken = known ? (int64_t)(0x7FFFFFFFu - known) : r.q.n;
  return r;
}

// Strip sums of the draft model's row at each refused draft.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, kSampleCtas) refused_kernel(const __grid_constant__ SampleArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), jobs = a.n_seqs * a.pieces;
  for (int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); job < jobs; job += warps) {
    const int64_t s = job / a.pieces;
    const Stop e = stop_of(a, s);
    if (!e.refused) continue;
    const int k0 = (int)(job - s * a.pieces) * a.each;
    const RowUnits<T> row(a.draft, e.q.lo + e.taken, a.draft_stride, a.vocab);
    sum_strips<T>(a, row, a.draft_scale, k0, min(k0 + a.each, a.strips), a.q + s * a.strips, lane);
    if (!last_piece(a.q_done + s, a.pieces, lane)) continue;
    const RowSum q = row_sum(a, a.q + s * a.strips, a.draft_scale, lane);
    if (lane == 0) a.q_total[s] = q;
  }
}

__device__ __forceinline__ Refused refused_of(const SampleArgs& a, const Stop& e, int64_t s, bool* fine) {
  const RowSum p = load_total(a.p_total + e.q.lo + s + e.taken);
  const RowSum q = load_total(a.q_total + (a.both ? e.q.lo + e.taken : s));
  *fine = usable(p) && usable(q);
  return Refused{p.m, (float)(1. / p.s), q.m, (float)(1. / q.s)};
}

// Strip sums of max(p - q, 0) at each refused draft.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 3) left_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), jobs = a.n_seqs * a.pieces;
  for (int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); job < jobs; job += warps) {
    const int64_t s = job / a.pieces;
    const Stop e = stop_of(a, s);
    if (!e.refused) continue;
    bool fine;
    const Refused f = refused_of(a, e, s, &fine);
    if (!fine) continue;
    const RowUnits<T> row(a.target, e.q.lo + s + e.taken, a.target_stride, a.vocab);
    const RowUnits<T> draft(a.draft, e.q.lo + e.taken, a.draft_stride, a.vocab);
    const int k0 = (int)(job - s * a.pieces) * a.each;
    for (int k = k0; k < min(k0 + a.each, a.strips); ++k) {
      const int u0 = (int)min((int64_t)k * a.strip_units, (int64_t)row.units), u1 = min(u0 + a.strip_units, row.units);
      float sum = 0.f;
      for (int u = u0; u < u1; u += kStripStep) {
        float r[kLoads * N];
        left_over<T>(a, f, row, draft.z, u + lane, 32, u1, step_inside<T>(row, u, u1), r);
#pragma unroll
        for (int i = 0; i < kLoads * N; ++i) sum += r[i];
      }
      sum = warp_sum(sum);
      if (lane == 0) __stcg(a.left + s * a.strips + k, sum);
    }
  }
}

// The weights that a token is drawn from.
enum Weights {
  kPlain,    // p
  kWithout,  // p without the refused draft
  kLeft,     // max(p - q, 0)
};

// Draws the token of a row; the warp's lanes get the same token and log p.
template <typename T>
__device__ __forceinline__ void draw(const SampleArgs& a, int64_t r, int64_t s, int kind, int64_t without, const T* zq,
                                     const Refused& f, float u, int64_t* token, float* logp, int lane) {
  constexpr int N = Vec<T>::N;
  const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
  const Scale& c = a.target_scale;
  const float2* strips = reinterpret_cast<const float2*>(a.p + r * a.strips);
  *token = -1;
  *logp = NAN;
  // a lane's strips are consecutive ones
  const int per = (a.strips + 31) / 32, k0 = min(lane * per, a.strips), k1 = min(k0 + per, a.strips);
  float m = -INFINITY;
  for (int k = k0; k < k1; ++k) m = fmaxf(m, __ldcg(strips + k).x);
  m = warp_max(m);
  auto plain = [&](int k) {
    const float2 x = __ldcg(strips + k);
    return (double)(x.y * factor(c, x.x, m));
  };
  auto bounds = [&](int k, int& u0, int& u1) {
    u0 = (int)min((int64_t)k * a.strip_units, (int64_t)row.units);
    u1 = min(u0 + a.strip_units, row.units);
  };
  double own = 0.;  // of p
  for (int k = k0; k < k1; ++k) own += plain(k);
  const RowSum p{warp_sum64(own), m};
  if (!usable(p)) return;
  int without_strip = -1;
  float without_sum = 0.f;
  if (kind == kWithout && without >= 0 && without < a.vocab) {
    without_strip = ((int)without + row.shift) / N / a.strip_units;
    int u0, u1;
    bounds(without_strip, u0, u1);
    without_sum = warp_sum(sum_without<T>(row, c, m, u0, u1, (int)without, lane));
  }
  auto weight = [&](int k) {
    if (kind == kLeft) return (double)__ldcg(a.left + s * a.strips + k);
    return kind == kWithout && k == without_strip ? (double)without_sum : plain(k);
  };
  double w = own;
  if (kind != kPlain) {
    w = 0.;
    for (int k = k0; k < k1; ++k) w += weight(k);
    // nothing is left over where the two models agree, and the refusal was one of rounding
    if (!__any_sync(0xFFFFFFFFu, w > 0.)) {
      kind = kPlain;
      w = own;
    }
  }
  const double end = warp_scan64(w, lane), sum = __shfl_sync(0xFFFFFFFFu, end, 31);
  u = fmaxf(u, 0.f);
  const double t = u < 1.f ? (double)u * sum : (double)INFINITY;  // 1 and above: the last token
  const unsigned above = __ballot_sync(0xFFFFFFFFu, w > 0. && end > t);
  const unsigned some = __ballot_sync(0xFFFFFFFFu, w > 0.);
  const int l = above ? __ffs(above) - 1 : 31 - __clz(some);
  double before = end - w, begun = before;
  int strip = 0;
  for (int k = k0; k < k1; ++k) {
    const double x = weight(k);
    if (x > 0.) {
      strip = k;
      begun = before;
      if (before + x > t) break;
    }
    before += x;
  }
  strip = __shfl_sync(0xFFFFFFFFu, strip, l);
  before = __shfl_sync(0xFFFFFFFFu, begun, l);
  int u0, u1;
  bounds(strip, u0, u1);
  const int found = pick_element<T>(row, u0, u1, t - before, lane, [&](int first, bool inside, float(&w)[kLoads * N]) {
    if (kind == kLeft) {
      left_over<T>(a, f, row, zq, first, 1, u1, inside, w);
      return;
    }
    uint4 z[kLoads];
    load_units<T>(row, first, 1, u1, inside, z);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      float e[N];
      exps<T>(c, m, z[k], e);
#pragma unroll
      for (int i = 0; i < N; ++i) w[k * N + i] = kind == kWithout && row.first(first + k) + i == without ? 0.f : e[i];
    }
  });
  if (found < 0) return;
  // the lane's part of p without the token's strip
  double rest = 0.;
  for (int k = k0; k < k1; ++k)
    if (k != strip) rest += plain(k);
  *token = found;
  *logp = token_logp<T>(row, c, m, rest, u0, u1, found, lane);
}

// Sampling: a warp draws a row's token.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 2) draw_kernel(const __grid_constant__ SampleArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  griddep_wait();
  if (t >= a.n_seqs) return;
  int64_t token = -1;
  float logp = 0.f;
  if (a.mask == nullptr || a.mask[t] != 0)
    draw<T>(a, t, t, kPlain, -1, nullptr, Refused{}, a.sample_u[t], &token, &logp, lane);
  if (lane == 0) {
    a.tokens[t] = token;
    a.logp[t] = logp;
  }
}

// Verification: a warp writes a row's token: a taken draft, the drawn one, or -1.
template <typename T>
__global__ void __launch_bounds__(kSampleWarps * 32, 2) emit_kernel(const __grid_constant__ SampleArgs a) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & 31;
  griddep_wait();
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5), jobs = (__ldcg(a.longest) + 1) * a.n_seqs;
  for (int64_t job = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); job < jobs; job += warps) {
    const int64_t i = job / a.n_seqs, s = job - i * a.n_seqs;
    const Stop e = stop_of(a, s);
    if (i > e.q.n) continue;
    const int64_t r = e.q.lo + s + i, d = e.q.lo + i;
    int64_t token = -1;
    float logp = 0.f;
    if (i < e.taken) {
      token = a.drafts[d];
      const RowUnits<T> row(a.target, r, a.target_stride, a.vocab);
      const RowSum p = load_total(a.p_total + r);
      const int strip = ((int)token + row.shift) / N / a.strip_units;
      double rest = 0.;
      for (int k = lane; k < a.strips; k += 32) {
        const float2 x = __ldcg(reinterpret_cast<const float2*>(a.p + r * a.strips) + k);
        if (k != strip) rest += (double)(x.y * factor(a.target_scale, x.x, p.m));
      }
      const int u0 = strip * a.strip_units;
      logp = token_logp<T>(row, a.target_scale, p.m, rest, u0, min(u0 + a.strip_units, row.units), (int)token, lane);
    } else if (i == e.taken) {
      int kind = kPlain;
      bool fine = true;
      Refused f{};
      const T* zq = nullptr;
      if (e.refused) {
        kind = kWithout;
        if (a.draft != nullptr) {
          kind = kLeft;
          f = refused_of(a, e, s, &fine);
          zq = reinterpret_cast<const T*>(a.draft) + d * a.draft_stride;
        }
      }
      logp = NAN;
      if (fine) draw<T>(a, r, s, kind, e.refused ? a.drafts[d] : -1, zq, f, a.sample_u[s], &token, &logp, lane);
      if (lane == 0) a.counts[s] = e.taken;
    }
    if (lane == 0) {
      a.tokens[r] = token;
      a.logp[r] = logp;
    }
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

// The workspace's parts, each on a 16-byte boundary; sampling needs the first alone.
size_t sample_space(SampleArgs* a, void* base, int64_t n_drafts, int64_t n_seqs, int32_t strips, bool drafts) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    void* p = base ? static_cast<uint8_t*>(base) + at : nullptr;
    at += (bytes + 15) / 16 * 16;
    return p;
  };
  const size_t rows = (size_t)(n_drafts + n_seqs), q_rows = (size_t)(n_drafts > n_seqs ? n_drafts : n_seqs);
  StripSum* p = static_cast<StripSum*>(take(rows * strips * sizeof(StripSum)));
  if (a) a->p = p;
  if (!drafts) return at;
  SampleArgs none;
  SampleArgs& o = a ? *a : none;
  o.q = static_cast<StripSum*>(take(q_rows * strips * sizeof(StripSum)));
  o.left = static_cast<float*>(take((size_t)n_seqs * strips * sizeof(float)));
  o.p_total = static_cast<RowSum*>(take(rows * sizeof(RowSum)));
  o.q_total = static_cast<RowSum*>(take(q_rows * sizeof(RowSum)));
  o.done = static_cast<uint32_t*>(take(rows * sizeof(uint32_t)));
  o.q_done = static_cast<uint32_t*>(take((size_t)n_seqs * sizeof(uint32_t)));
  o.refused = static_cast<uint32_t*>(take((size_t)n_seqs * sizeof(uint32_t)));
  o.longest = static_cast<int64_t*>(take(sizeof(int64_t)));
  return at;
}

// Strips that a warp takes at a time: two where there are enough for every warp of the chip.
void deal_out(SampleArgs& a, int64_t rows, int sms) {
  const int64_t warps = (int64_t)sms * kSampleCtas * kSampleWarps;
  a.each = rows * a.strips >= 8 * warps ? 2 : 1;
  a.pieces = (a.strips + a.each - 1) / a.each;
}

// CTAs and warps of a CTA for `jobs` jobs of a warp: one warp an SM first.
struct Launch {
  int grid, block;
};
Launch launch_of(int64_t jobs, int sms) {
  const int64_t per_sm = (jobs + sms - 1) / sms;
  const int64_t warps = per_sm < 1 ? 1 : per_sm < kSampleWarps ? per_sm : kSampleWarps;
  const int64_t ctas = (jobs + warps - 1) / warps, most = (int64_t)sms * kSampleCtas;
  return Launch{(int)(ctas < 1 ? 1 : ctas < most ? ctas : most), (int)(32 * warps)};
}

template <typename T>
cudaError_t run_rows(const SampleArgs& a, int sms, cudaStream_t s) {
  const Launch l = launch_of(a.n_seqs * a.pieces, sms);
  cudaError_t e = launch(rows_kernel<T>, l.grid, l.block, 0, s, 1, false, a);
  if (e != cudaSuccess) return e;
  const int64_t warps = a.n_seqs < 4ll * sms ? 1 : 4;  // a row each
  return launch(draw_kernel<T>, (int)((a.n_seqs + warps - 1) / warps), (int)(32 * warps), 0, s, 1, true, a);
}

template <typename T>
cudaError_t run_verify(const SampleArgs& a, int sms, cudaStream_t s) {
  const int64_t rows = a.n_drafts + a.n_seqs;
  cudaError_t e = launch(setup_kernel, 1, kSetupThreads, 0, s, 1, false, a);
  if (e != cudaSuccess) return e;
  const Launch all = launch_of((rows + (a.both ? a.n_drafts : 0)) * a.pieces, sms);
  if ((e = launch(verify_kernel<T>, all.grid, all.block, 0, s, 1, true, a)) != cudaSuccess) return e;
  if (a.draft != nullptr && a.n_drafts > 0) {
    const Launch one = launch_of(a.n_seqs * a.pieces, sms);
    if (!a.both && (e = launch(refused_kernel<T>, one.grid, one.block, 0, s, 1, true, a)) != cudaSuccess) return e;
    if ((e = launch(left_kernel<T>, one.grid, one.block, 0, s, 1, true, a)) != cudaSuccess) return e;
  }
  const Launch out = launch_of(rows, sms);
  return launch(emit_kernel<T>, out.grid, out.block, 0, s, 1, true, a);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_sample_workspace_bytes(int64_t rows, int64_t n_seqs, int64_t vocab, int32_t dtype, size_t* bytes) {
  if (!bytes) return invalid("bytes is NULL");
  if (rows < 0 || rows > (1ll << 31) - 1 || n_seqs < 0 || n_seqs > rows) return invalid("rows must be in [0, 2^31), n_seqs in [0, rows]");
  if (vocab < 1 || vocab > (1ll << 30)) return invalid("vocab must be in [1, 2^30]");
  if (dtype != MUON_DTYPE_F32 && dtype != MUON_DTYPE_BF16) return invalid("unknown logits dtype");
  int32_t units, strips;
  strips_of(vocab, dtype, &units, &strips);
  *bytes = sample_space(nullptr, nullptr, rows - n_seqs, n_seqs, strips, true);
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
  const size_t need = sample_space(&a, workspace, 0, a.n_seqs, a.strips, false);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  deal_out(a, a.n_seqs, sms);
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
  a.both = draft->logits && !draft_logp;
  strips_of(a.vocab, target->dtype, &a.strip_units, &a.strips);
  const size_t need = sample_space(&a, workspace, a.n_drafts, n_seqs, a.strips, true);
  if ((st = check_workspace(workspace, workspace_bytes, need)) != MUON_OK) return st;
  int sms;
  if ((st = find_device(&sms)) != MUON_OK) return st;
  deal_out(a, target->tokens, sms);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = target->dtype == MUON_DTYPE_BF16 ? run_verify<__nv_bfloat16>(a, sms, s) : run_verify<float>(a, sms, s);
  return e == cudaSuccess ? MUON_OK : cuda_error(e);
}

}  // extern "C"
