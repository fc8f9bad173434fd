// Global gradient norm over many tensors, and clipping by it.
//
//   N = sqrt(sum g^2),  c = min(1, max_norm / (N + eps)),  out = c g
//
// Two passes, bound by HBM: every element is read once for N; where something has to
// be written it is read again (in a launch in the reverse order, so that what the first pass
// left in L2 is met first: its last kKeptBytes, read with the normal policy while all before
// them are marked to be evicted first), scaled and written.  The tensor table travels as a kernel
// parameter, so a call copies nothing to the device and waits for nothing on the host.  A set of
// more tensors than one table holds takes several launches a pass, first to last in both, each
// with kKeptBytes of its own: only within a launch does the second pass meet the latest reads first.
//
// Measured: the norm of a 36-layer model's 7.3 GB of bf16 gradients 1.02 ms (7.1 TB/s; in
// place below the limit that is the whole call); one layer's 202 MB of bf16 gradients into
// fp32 0.135 ms: 0.035 ms for the norm, 0.100 ms for 606 MB of the second pass (6.1 TB/s);
// 1003 tensors of up to 40000 elements, 141 MB, 0.042 ms.
//
// The unit of work is a chunk of kChunk elements of one tensor, taken by one warp: a
// set of a thousand small tensors spreads over the GPU like one large tensor does.
// A warp's chunks are warp, warp + warps, ...: every partial sum has a fixed place and
// order, so that a call gives the same bits each time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <cmath>

#include "device.cuh"
#include "kernels.h"
#include "epilogue.cuh"
#include "launch.cuh"
#include "momentum.cuh"
#include "muon.h"

namespace muon {
namespace {

constexpr int kChunk = 2048;       // elements of one warp's unit of work: 8 octets a lane
constexpr int kClipThreads = 256;
constexpr int kClipWarps = kClipThreads / 32;
constexpr int kClipCtasPerSm = 4;
constexpr int kClipMaxCtas = 1024; // partial sums of one launch
constexpr int64_t kKeptBytes = 80ll << 20;

// A plain tensor, and one of several blocks a stride apart.
struct PlainSeg {
  const void* g;
  void* out;
  int64_t elems;
  int32_t chunk0;   // first chunk of the tensor in its launch
  int32_t bf16;     // bit 0: g, bit 1: out
  __device__ __forceinline__ int64_t block(int&) const { return 0; }
};
struct BlockSeg {
  const void* g;
  void* out;
  int64_t elems;
  int32_t chunk0;
  int32_t bf16;
  int64_t stride;
  int32_t chunks_per_block;
  int32_t pad_;
  // element offset of the block that chunk `local` of the tensor lies in; `local` becomes the chunk in it
  __device__ __forceinline__ int64_t block(int& local) const {
    const int b = local / chunks_per_block;
    local -= b * chunks_per_block;
    return b * stride;
  }
};

// A launch takes up to kCap tensors.  The small tables keep the parameters of the usual
// call at 2 or 3 KB; the large ones fill the 32,764 bytes that a kernel may have.
template <typename S, int kCap>
struct ClipArgs {
  using Seg = S;
  static constexpr int kMost = kCap;
  S seg[kCap];
  int32_t n_segs, n_chunks;
  double* partials;        // of the whole call
  int32_t partial0;        // this launch's first partial sum (norm)
  int32_t n_partials;      // all of them (clip)
  float max_norm, eps;
  int32_t nonfinite;
  int32_t in_place;        // every tensor of this launch is
  int32_t kept;            // the launch's chunks from here on are left in L2
  float* result;
};

// A chunk: its tensor, and the part of a block that it is.
struct Chunk {
  const void* g;  // of the block
  void* out;
  bool g_bf16, out_bf16;
  int64_t begin;  // elements [begin, end) of the block
  int64_t end;
  int head;       // the block's elements before its first aligned octet
};

template <typename A>
__device__ __forceinline__ Chunk find_chunk(const A& a, int c, int& cur) {
  const int next = cur + 1 < a.n_segs ? a.seg[cur + 1].chunk0 : a.n_chunks;
  if (c < a.seg[cur].chunk0 || c >= next) {
    int lo = 0, hi = a.n_segs - 1;
    while (lo < hi) {  // last tensor with chunk0 <= c
      const int mid = (lo + hi + 1) >> 1;
      if (a.seg[mid].chunk0 <= c) lo = mid; else hi = mid - 1;
    }
    cur = lo;
  }
  const typename A::Seg& s = a.seg[cur];
  int local = c - s.chunk0;
  const int64_t at = s.block(local);
  Chunk k;
  k.g_bf16 = s.bf16 & 1;
  k.out_bf16 = s.bf16 & 2;
  const int shift = k.g_bf16 ? 1 : 2;
  k.g = static_cast<const uint8_t*>(s.g) + (at << shift);
  k.out = static_cast<uint8_t*>(s.out) + (at << (k.out_bf16 ? 1 : 2));
  k.head = (int)((-reinterpret_cast<uint64_t>(k.g) & ((8u << shift) - 1)) >> shift);  // to 16 (bf16) or 32 bytes
  if (k.head > s.elems) k.head = (int)s.elems;
  // chunk 0 takes the head too, so that the others start on a boundary
  k.begin = local == 0 ? 0 : min(s.elems, k.head + (int64_t)local * kChunk);
  k.end = min(s.elems, k.head + (int64_t)(local + 1) * kChunk);
  return k;
}

__device__ __forceinline__ void unpack8(const uint4& w, float (&v)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(u[i] << 16);
    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

// Sum of squares of a lane's part of a chunk in fp32, and the OR of its bits without signs.
struct Part {
  float s;
  uint32_t bits;
};

__device__ __forceinline__ void add_octet_bf16(const uint4& w, float& s0, float& s1, uint32_t& bits) {
  float v[8];
  unpack8(w, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s0 = __fmaf_rn(v[2 * i], v[2 * i], s0);
    s1 = __fmaf_rn(v[2 * i + 1], v[2 * i + 1], s1);
  }
  bits |= (w.x | w.y | w.z | w.w) & 0x7FFF7FFFu;
}

__device__ __forceinline__ void add_quad_f32(const uint4& w, float& s0, float& s1, uint32_t& bits) {
  const float x = __uint_as_float(w.x), y = __uint_as_float(w.y), z = __uint_as_float(w.z), u = __uint_as_float(w.w);
  s0 = __fmaf_rn(x, x, s0);
  s1 = __fmaf_rn(y, y, s1);
  s0 = __fmaf_rn(z, z, s0);
  s1 = __fmaf_rn(u, u, s1);
  bits |= (w.x | w.y | w.z | w.w) & 0x7FFFFFFFu;
}

__device__ __forceinline__ float load_elem(const void* p, int64_t i, int bf16) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

__device__ __forceinline__ uint4 load16(const void* p, uint64_t policy) {
  uint4 w;
  asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
               : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
               : "l"(p), "l"(policy)
               : "memory");
  return w;
}

__device__ __forceinline__ Part chunk_squares(const Chunk& k, int lane, uint64_t policy) {
  float s0 = 0.f, s1 = 0.f;
  uint32_t bits = 0;
  const int64_t vec0 = k.begin == 0 ? k.head : k.begin;  // on an octet's boundary
  const int n8 = (int)((k.end - vec0) >> 3);
  if (k.g_bf16) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(k.g) + vec0);
    if (n8 == kChunk / 8) {
      uint4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = load16(p + i * 32 + lane, policy);
#pragma unroll
      for (int i = 0; i < 8; ++i) add_octet_bf16(w[i], s0, s1, bits);
    } else {
      for (int i = lane; i < n8; i += 32) add_octet_bf16(p[i], s0, s1, bits);
    }
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(k.g) + vec0);
    if (n8 == kChunk / 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = load16(p + h * 256 + i * 32 + lane, policy);
#pragma unroll
        for (int i = 0; i < 8; ++i) add_quad_f32(w[i], s0, s1, bits);
      }
    } else {
      for (int i = lane; i < 2 * n8; i += 32) add_quad_f32(p[i], s0, s1, bits);
    }
  }
  // the elements before the first boundary and after the last whole octet, < 8 each
  const int64_t tail = vec0 + 8ll * n8;
  int64_t i = -1;
  if (lane < 8) {
    if (k.begin == 0 && lane < k.head) i = lane;
  } else if (lane < 16 && tail + (lane - 8) < k.end) {
    i = tail + (lane - 8);
  }
  if (i >= 0) {
    const float x = load_elem(k.g, i, k.g_bf16);
    s0 = __fmaf_rn(x, x, s0);
    bits |= __float_as_uint(x) & 0x7FFFFFFFu;
  }
  return Part{s0 + s1, bits};
}

// The same in 64 bits, for a chunk whose squares fp32 cannot hold.
__device__ __noinline__ double chunk_squares_wide(const Chunk& k, int lane) {
  double s = 0.0;
  for (int64_t i = k.begin + lane; i < k.end; i += 32) {
    const double x = (double)load_elem(k.g, i, k.g_bf16);
    s = fma(x, x, s);
  }
  return s;
}

// A lane adds at most kChunk / 32 + 1 = 65 squares in fp32, in two sums (relative error below
// 34 units of 2^-24 at the very worst, a few in practice), then carries the sum of its
// chunks as an unevaluated pair.  A chunk whose lane sums leave [2^-116, 2^90], where
// squares overflow or lose bits to underflow, is summed again in 64 bits; an all-zero
// one is not.
template <typename A>
__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const __grid_constant__ A a) {
  __shared__ double red[kClipWarps];
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = gridDim.x * kClipWarps;
  uint64_t first, normal;  // L2 policies
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(first));
  asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(normal));
  float hi = 0.f, lo = 0.f;
  double wide = 0.0;
  int cur = 0;
  for (int c = blockIdx.x * kClipWarps + warp; c < a.n_chunks; c += warps) {
    const Chunk k = find_chunk(a, c, cur);
    const Part p = chunk_squares(k, lane, c < a.kept ? first : normal);
    const bool fits = p.s <= 0x1p90f && (p.s >= 0x1p-116f || p.bits == 0);
    if (__all_sync(0xFFFFFFFFu, fits)) {
      float s, e;
      two_sum(hi, p.s, s, e);
      hi = s;
      lo += e;
    } else {
      wide += chunk_squares_wide(k, lane);
    }
  }
  // 64-bit additions are two a clock and SM: the pairs are merged in fp32
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    float s, e;
    two_sum(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o), s, e);
    hi = s;
    lo += e + __shfl_xor_sync(0xFFFFFFFFu, lo, o);
  }
  if (__any_sync(0xFFFFFFFFu, wide != 0.0)) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) wide += __shfl_xor_sync(0xFFFFFFFFu, wide, o);
  }
  if (lane == 0) red[warp] = (double)hi + (double)lo + wide;
  __syncthreads();
  if (threadIdx.x == 0) {
    double t = red[0];
#pragma unroll
    for (int w = 1; w < kClipWarps; ++w) t += red[w];
    a.partials[a.partial0 + blockIdx.x] = t;
  }
}

// The call's sum of squares, in the same order in every CTA; by one warp of it, since
// 64-bit additions are two a clock and SM.
__device__ __forceinline__ double total_of(const double* partials, int n) {
  __shared__ double total;
  if (threadIdx.x < 32) {
    double t = 0.0;
    for (int i = threadIdx.x; i < n; i += 32) t += __ldcg(partials + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    if (threadIdx.x == 0) total = t;
  }
  __syncthreads();
  return total;
}

__global__ void __launch_bounds__(kClipThreads) norm_result_kernel(const double* partials, int n, float* norm) {
  griddep_wait();
  const double t = total_of(partials, n);
  if (threadIdx.x == 0) *norm = (float)sqrt(t);
}

// The product is rounded to fp32 and, for a bf16 output, again when it is packed.
__device__ __forceinline__ float scaled(float x, float c, bool zero) { return zero ? 0.f : c * x; }

template <bool kBf16>
struct Octet;  // eight elements as loaded
template <>
struct Octet<true> {
  uint4 w;
  __device__ __forceinline__ void load(const void* g, int64_t i) {
    w = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(g) + i));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack8(w, v); }
};
template <>
struct Octet<false> {
  float w[8];
  __device__ __forceinline__ void load(const void* g, int64_t i) {  // 32-byte aligned
    asm volatile("ld.global.L2::evict_first.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]), "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7])
                 : "l"(static_cast<const float*>(g) + i)
                 : "memory");
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w[e];
  }
};

// fp32 octets leave as whole 32-byte sectors where they are aligned to them (404 MB from
// 202 MB of bf16: 138 us in halves, 105 us so).
template <bool kBf16>
__device__ __forceinline__ void store8(void* out, int64_t i, const float (&r)[8], bool sectors) {
  if (kBf16) {
    __stcs(reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(out) + i),
           make_uint4(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]), pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7])));
  } else if (sectors) {
    asm volatile("st.global.L2::evict_first.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(static_cast<float*>(out) + i),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + i);
    __stcs(p, make_float4(r[0], r[1], r[2], r[3]));
    __stcs(p + 1, make_float4(r[4], r[5], r[6], r[7]));
  }
}

template <bool kIn, bool kOut>
__device__ __forceinline__ void scale_octets(const Chunk& k, int64_t vec0, int n8, float c, bool zero, int lane) {
  constexpr int kEach = 4;  // octets of a lane on their way at a time
  const bool sectors = ((reinterpret_cast<uint64_t>(k.out) + 4 * (uint64_t)vec0) & 31) == 0;
  int i = lane;
  for (; i + 32 * (kEach - 1) < n8; i += 32 * kEach) {
    Octet<kIn> w[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) w[j].load(k.g, vec0 + 8ll * (i + 32 * j));
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
      float v[8];
      w[j].get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = scaled(v[e], c, zero);
      store8<kOut>(k.out, vec0 + 8ll * (i + 32 * j), v, sectors);
    }
  }
  for (; i < n8; i += 32) {
    Octet<kIn> w;
    float v[8];
    w.load(k.g, vec0 + 8ll * i);
    w.get(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = scaled(v[e], c, zero);
    store8<kOut>(k.out, vec0 + 8ll * i, v, sectors);
  }
}

__device__ __forceinline__ void scale_elem(const Chunk& k, int64_t i, float c, bool zero) {
  const float r = scaled(load_elem(k.g, i, k.g_bf16), c, zero);
  if (k.out_bf16) static_cast<__nv_bfloat16*>(k.out)[i] = __float2bfloat16_rn(r);
  else static_cast<float*>(k.out)[i] = r;
}

template <typename A>
__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const __grid_constant__ A a) {
  griddep_wait();
  const double sumsq = total_of(a.partials, a.n_partials);
  const double norm = sqrt(sumsq);
  float c = 1.f;
  if (!isfinite(sumsq)) {
    c = a.nonfinite == MUON_NONFINITE_ZERO ? 0.f : 1.f;
  } else {
    const double den = norm + (double)a.eps;
    if (den > (double)a.max_norm) c = (float)((double)a.max_norm / den);
  }
  const bool zero = !isfinite(sumsq) && c == 0.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.result[0] = (float)norm;
    a.result[1] = c;
  }
  if (c == 1.f && a.in_place) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int warps = gridDim.x * kClipWarps;
  int cur = a.n_segs - 1;
  for (int r = blockIdx.x * kClipWarps + warp; r < a.n_chunks; r += warps) {
    const Chunk k = find_chunk(a, a.n_chunks - 1 - r, cur);
    if (c == 1.f && k.out == k.g) continue;
    const int64_t vec0 = k.begin == 0 ? k.head : k.begin;
    if (((reinterpret_cast<uint64_t>(k.out) + ((uint64_t)vec0 << (k.out_bf16 ? 1 : 2))) & 15) != 0) {
      // out is not aligned where g is: element by element
      for (int64_t i = k.begin + lane; i < k.end; i += 32) scale_elem(k, i, c, zero);
      continue;
    }
    const int n8 = (int)((k.end - vec0) >> 3);
    if (k.g_bf16) {
      if (k.out_bf16) scale_octets<true, true>(k, vec0, n8, c, zero, lane);
      else scale_octets<true, false>(k, vec0, n8, c, zero, lane);
    } else {
      if (k.out_bf16) scale_octets<false, true>(k, vec0, n8, c, zero, lane);
      else scale_octets<false, false>(k, vec0, n8, c, zero, lane);
    }
    const int64_t tail = vec0 + 8ll * n8;
    if (lane < 8) {
      if (k.begin == 0 && lane < k.head) scale_elem(k, lane, c, zero);
    } else if (lane < 16 && tail + (lane - 8) < k.end) {
      scale_elem(k, tail + (lane - 8), c, zero);
    }
  }
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
using PlainSmall = ClipArgs<PlainSeg, 64>;
using PlainLarge = ClipArgs<PlainSeg, 1020>;
using BlockSmall = ClipArgs<BlockSeg, 64>;
using BlockLarge = ClipArgs<BlockSeg, 640>;
static_assert(sizeof(PlainLarge) <= 32764 && sizeof(BlockLarge) <= 32764, "kernel parameters");

int64_t elem_size(int32_t dtype) { return dtype == MUON_DTYPE_BF16 ? 2 : 4; }

int64_t chunks_per_block(const muon_grad& t) { return (t.elems + kChunk - 1) / kChunk; }

constexpr int64_t kMostChunks = 2000000000ll;  // of a launch

const char* check_grad(const muon_grad& t) {
  if (t.elems < 0 || t.count < 0) return "gradient: elems and count must be >= 0";
  if (t.elems > (1ll << 40) || t.count > (1ll << 31) - 1) return "gradient: too many elements";
  if (t.stride_elems != 0 && (t.stride_elems < t.elems || t.stride_elems > (1ll << 40)))
    return "gradient: stride_elems must be 0 or at least elems";
  if (t.dtype != MUON_DTYPE_F32 && t.dtype != MUON_DTYPE_BF16) return "gradient: unknown dtype";
  if (t.elems == 0 || t.count == 0) return nullptr;
  if ((double)chunks_per_block(t) * (double)t.count > (double)kMostChunks) return "gradient: too many elements";
  if (!t.g) return "gradient pointer is NULL";
  if (reinterpret_cast<uint64_t>(t.g) % elem_size(t.dtype)) return "gradient pointer is not aligned to its type";
  return nullptr;
}

const char* check_out(const muon_grad& t) {
  if (t.elems == 0 || t.count == 0) return nullptr;
  if (!t.out || t.out == t.g) {
    if (t.out_dtype != t.dtype) return "gradient in place: out_dtype must be dtype";
    return nullptr;
  }
  if (t.out_dtype != MUON_DTYPE_F32 && t.out_dtype != MUON_DTYPE_BF16) return "gradient: unknown out_dtype";
  if (reinterpret_cast<uint64_t>(t.out) % elem_size(t.out_dtype)) return "out pointer is not aligned to its type";
  return nullptr;
}

void put_stride(PlainSeg&, const muon_grad&) {}
void put_stride(BlockSeg& s, const muon_grad& t) {
  s.stride = t.stride_elems ? t.stride_elems : t.elems;
  s.chunks_per_block = (int32_t)chunks_per_block(t);
}

// Launches of at most kMost tensors and 2e9 chunks cover the call's tensors in order: fills
// one from tensor `i` on, and leaves `i` at the first that it did not take.
template <typename A>
void fill_args(const muon_grad* grads, int64_t n, int64_t& i, A& a) {
  int64_t chunks = 0;
  a.n_segs = 0;
  a.in_place = 1;
  for (; i < n && a.n_segs < A::kMost; ++i) {
    const muon_grad& t = grads[i];
    if (t.elems == 0 || t.count == 0) continue;
    const int64_t all = chunks_per_block(t) * t.count;
    if (chunks + all > kMostChunks) break;
    typename A::Seg& s = a.seg[a.n_segs++];
    const bool in_place = !t.out || t.out == t.g;
    s.g = t.g;
    s.out = in_place ? t.g : t.out;
    s.elems = t.elems;
    s.chunk0 = (int32_t)chunks;
    s.bf16 = (t.dtype == MUON_DTYPE_BF16 ? 1 : 0) | ((in_place ? t.dtype : t.out_dtype) == MUON_DTYPE_BF16 ? 2 : 0);
    put_stride(s, t);
    if (!in_place) a.in_place = 0;
    chunks += all;
  }
  a.n_chunks = (int32_t)chunks;
  a.kept = 0;
  int64_t room = kKeptBytes / kChunk;  // bytes an element times chunks
  for (int k = a.n_segs - 1; k >= 0; --k) {
    const int64_t size = (a.seg[k].bf16 & 1) ? 2 : 4, mine = (k + 1 < a.n_segs ? a.seg[k + 1].chunk0 : chunks) - a.seg[k].chunk0;
    if (mine * size > room) {
      a.kept = (int32_t)(a.seg[k].chunk0 + mine - room / size);
      break;
    }
    room -= mine * size;
  }
}

int grid_for(int32_t n_chunks, int sms) {
  int64_t ctas = ((int64_t)n_chunks + kClipWarps - 1) / kClipWarps;
  const int64_t most = sms * kClipCtasPerSm < kClipMaxCtas ? sms * kClipCtasPerSm : kClipMaxCtas;
  return (int)(ctas < 1 ? 1 : ctas > most ? most : ctas);
}

// An upper bound of the launches that a set needs: by the smallest tables.
int64_t launches_for(const muon_grad* grads, int64_t n) {
  int64_t launches = 0, segs = 0, chunks = 0;
  for (int64_t i = 0; i < n; ++i) {
    const int64_t all = grads[i].elems > 0 ? chunks_per_block(grads[i]) * grads[i].count : 0;
    if (all == 0) continue;
    if (launches == 0 || segs == PlainSmall::kMost || chunks + all > kMostChunks) {
      ++launches;
      segs = chunks = 0;
    }
    ++segs;
    chunks += all;
  }
  return launches;
}

template <typename A>
int32_t run_clip(const muon_grad* grads, int64_t n, bool clip, float max_norm, float eps, int32_t nonfinite,
                 float* result, double* partials, int sms, cudaStream_t s) {
  A a;
  a.partials = partials;
  a.n_partials = 0;
  a.max_norm = max_norm;
  a.eps = eps;
  a.nonfinite = nonfinite;
  a.result = result;
  int64_t i = 0;
  cudaError_t e;
  int launches = 0;
  while (i < n) {
    fill_args(grads, n, i, a);
    if (a.n_chunks == 0) continue;
    const int grid = grid_for(a.n_chunks, sms);
    a.partial0 = a.n_partials;
    a.n_partials += grid;
    e = launch(clip_norm_kernel<A>, grid, kClipThreads, 0, s, 1, false, a);
    if (e != cudaSuccess) return cuda_error(e);
    ++launches;
  }
  if (!clip) {
    e = launch(norm_result_kernel, 1, kClipThreads, 0, s, 1, launches > 0, (const double*)partials, (int)a.n_partials,
               result);
    return e == cudaSuccess ? MUON_OK : cuda_error(e);
  }
  if (launches <= 1) {  // the table is filled already (or empty: the result alone)
    if (launches == 0) a.n_segs = a.n_chunks = a.in_place = 0;
    e = launch(clip_scale_kernel<A>, grid_for(a.n_chunks, sms), kClipThreads, 0, s, 1, launches > 0, a);
    return e == cudaSuccess ? MUON_OK : cuda_error(e);
  }
  for (i = 0; i < n;) {
    fill_args(grads, n, i, a);
    if (a.n_chunks == 0) continue;
    e = launch(clip_scale_kernel<A>, grid_for(a.n_chunks, sms), kClipThreads, 0, s, 1, false, a);
    if (e != cudaSuccess) return cuda_error(e);
  }
  return MUON_OK;
}

int32_t clip_entry(const muon_grad* grads, int64_t n, bool clip, float max_norm, float eps, int32_t nonfinite,
                   float* result, void* workspace, size_t workspace_bytes, void* stream) {
  if (n < 0 || (n > 0 && !grads)) return set_error(MUON_ERR_INVALID, "gradient array is NULL or its length negative");
  if (!result || reinterpret_cast<uint64_t>(result) % 4) return set_error(MUON_ERR_INVALID, "result is NULL or not aligned");
  for (int64_t i = 0; i < n; ++i) {
    const char* bad = check_grad(grads[i]);
    if (!bad && clip) bad = check_out(grads[i]);
    if (bad) return set_error(MUON_ERR_INVALID, bad);
  }
  if (clip) {
    if (!(max_norm >= 0.f)) return set_error(MUON_ERR_INVALID, "max_norm must be >= 0");
    if (!(eps >= 0.f) || std::isinf(eps)) return set_error(MUON_ERR_INVALID, "eps must be finite and >= 0");
    if (nonfinite != MUON_NONFINITE_KEEP && nonfinite != MUON_NONFINITE_ZERO)
      return set_error(MUON_ERR_INVALID, "unknown nonfinite policy");
  }
  size_t need = 0;
  const int32_t st = muon_clip_workspace_bytes(grads, n, &need);
  if (st != MUON_OK) return st;
  if (!workspace || workspace_bytes < need) return set_error(MUON_ERR_NO_WORKSPACE, "workspace is NULL or too small");
  if (reinterpret_cast<uint64_t>(workspace) % 16) return set_error(MUON_ERR_INVALID, "workspace must be 16-byte aligned");
  cudaError_t e;
  const int sms = device_sms(&e);
  if (e != cudaSuccess) return cuda_error(e);
  if (sms == 0) return set_error(MUON_ERR_UNSUPPORTED, "libmuon is built for sm_103a");
  double* partials = static_cast<double*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool plain = true;
  for (int64_t i = 0; i < n; ++i) plain = plain && grads[i].count <= 1;
  auto run = plain ? (n <= PlainSmall::kMost ? run_clip<PlainSmall> : run_clip<PlainLarge>)
                   : (n <= BlockSmall::kMost ? run_clip<BlockSmall> : run_clip<BlockLarge>);
  return run(grads, n, clip, max_norm, eps, nonfinite, result, partials, sms, s);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status muon_clip_workspace_bytes(const muon_grad* grads, int64_t n, size_t* bytes) {
  if (!bytes || n < 0 || (n > 0 && !grads)) return set_error(MUON_ERR_INVALID, "NULL argument or negative length");
  for (int64_t i = 0; i < n; ++i)
    if (const char* bad = check_grad(grads[i])) return set_error(MUON_ERR_INVALID, bad);
  const int64_t launches = launches_for(grads, n);
  *bytes = (size_t)(launches < 1 ? 1 : launches) * kClipMaxCtas * sizeof(double);
  return MUON_OK;
}

muon_status muon_grad_norm(const muon_grad* grads, int64_t n, float* norm, void* workspace, size_t workspace_bytes,
                           void* stream) {
  return clip_entry(grads, n, false, 0.f, 0.f, 0, norm, workspace, workspace_bytes, stream);
}

muon_status muon_clip_grad_norm(const muon_grad* grads, int64_t n, float max_norm, float eps, int32_t nonfinite,
                                float* result, void* workspace, size_t workspace_bytes, void* stream) {
  return clip_entry(grads, n, true, max_norm, eps, nonfinite, result, workspace, workspace_bytes, stream);
}

}  // extern "C"
