// The global norm of a list of gradients and clipping by it, in place:
//   norm = sqrt(sum over all elements g^2);   g <- g * min(1, max_norm / norm).
//
// Bandwidth-bound: every element is read once for the norm, and read and written once more
// where the norm is above max_norm.  Two launches.  The first leaves a partial sum a CTA; in
// the second every CTA adds the same partial sums in the same order, so that none waits for
// another, and returns at once where nothing is to be scaled.
//
// Measured: 340 M bf16 elements in 48 tensors, clipped, 311 to 334 us (three passes over 680 MB at
// 6.1 to 6.6 TB/s; the norm alone 115); 38.7 M fp32 and 37 k bf16 elements 73 to 78 us; 48 tensors of
// 1536 fp32 elements 8 us on the GPU and 41 with the host's side.  Measured and not kept: loads and stores
// marked as read once (332 to 340), CTAs of 512 threads (338), chunks of 16 KB (339), six
// CTAs an SM; walking the second pass forwards costs 3 us.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace {

constexpr int CL_THREADS = 256;
constexpr int CL_HELD = 8;                                  // 16-byte vectors a thread holds at a time
constexpr int CL_VECS = CL_THREADS * CL_HELD;               // vectors of a chunk (32 KB)
// CTAs an SM: registers for the vectors, and for the scaling some more.
constexpr int CL_NORM_CTAS = 4, CL_SCALE_CTAS = 3;
constexpr int CL_MAX_CTAS = 1024;
// Tensors of a launch.  The table travels in the kernel's parameters, and a launch is charged
// for all of them (48 tensors: 8 us a call less with the small one).
constexpr int CL_ENTRIES = 1000, CL_FEW = 64;

// Chunks are counted from the 16-byte boundary at or below a tensor's first element, so that
// tensors of any alignment move in whole vectors but for their ends.
struct ClipEntry {
  void* base;           // that boundary
  long long first;      // elements between it and the tensor
  long long end;        // one past the last element, from the boundary
  int begin;            // first chunk of the launch
  int bf16_;
};
template <int kEntries>
struct ClipParams {
  int n, chunks, ctas;
  int add;                         // partial sums of an earlier launch are already there
  int only;                        // the norm alone is wanted
  double* part;
  double max_norm;
  float* norm;
  ClipEntry e[kEntries];
};
static_assert(sizeof(ClipParams<CL_ENTRIES>) < 32700, "ClipParams too large");

// The chunk's tensor, given that of an earlier chunk: mostly the same or the next one.
template <class P>
__device__ __forceinline__ int entry_of(const P& p, int chunk, int from) {
  int lo = 0, hi = p.n - 1;
  if (p.e[from].begin <= chunk) {
    if (from == hi || p.e[from + 1].begin > chunk) return from;
    lo = from + 1;
  }
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.e[mid].begin <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A thread's share of a chunk, zeros outside the tensor.  Returns whether every vector of
// the chunk lies inside.
template <typename T>
__device__ __forceinline__ bool load_share(const ClipEntry& e, long long v0, uint4 (&q)[CL_HELD]) {
  constexpr int V = 16 / (int)sizeof(T);
  const uint4* base = static_cast<const uint4*>(e.base);
  if (v0 * V >= e.first && (v0 + CL_VECS) * V <= e.end) {
#pragma unroll
    for (int k = 0; k < CL_HELD; ++k) q[k] = base[v0 + k * CL_THREADS + threadIdx.x];
    return true;
  }
#pragma unroll
  for (int k = 0; k < CL_HELD; ++k) {
    const long long v = v0 + k * CL_THREADS + threadIdx.x, c = v * V;
    q[k] = make_uint4(0, 0, 0, 0);
    if (c >= e.first && c + V <= e.end) {
      q[k] = base[v];
    } else if (c + V > e.first && c < e.end) {
      T x[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        x[i] = c + i >= e.first && c + i < e.end ? static_cast<const T*>(e.base)[c + i] : from_f32<T>(0.f);
      q[k] = *reinterpret_cast<const uint4*>(x);
    }
  }
  return false;
}
__device__ __forceinline__ void widen(const uint4& q, f32x2 (&v)[4], const bf16*) {
  v[0] = cvt2(q.x); v[1] = cvt2(q.y); v[2] = cvt2(q.z); v[3] = cvt2(q.w);
}
__device__ __forceinline__ void widen(const uint4& q, f32x2 (&v)[2], const float*) {
  v[0] = make2(__uint_as_float(q.x), __uint_as_float(q.y));
  v[1] = make2(__uint_as_float(q.z), __uint_as_float(q.w));
}
template <typename T>
__device__ __forceinline__ float squares(const uint4 (&q)[CL_HELD], float scale) {
  constexpr int P = 8 / (int)sizeof(T);
  f32x2 s[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int k = 0; k < CL_HELD; ++k) {
    f32x2 v[P];
    widen(q[k], v, static_cast<const T*>(nullptr));
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (scale != 1.f) v[i] = mul2(v[i], both(scale));
      s[i & 1] = fma2(v[i], v[i], s[i & 1]);
    }
  }
  const f32x2 t = add2(s[0], s[1]);
  return lo2(t) + hi2(t);
}
// Squares of up to 64 numbers, in fp32 where they stay in its range (a sum of 2^-80 has lost
// at most 2^-40 of itself to squares that are subnormal), else of the numbers times a power
// of two: a gradient of 1e25 has a norm, and so has one of 1e-25.
template <typename T>
__device__ __forceinline__ double sum_share(const uint4 (&q)[CL_HELD]) {
  const float s = squares<T>(q, 1.f);
  if (s >= 0x1p-80f && s <= 0x1p120f) return (double)s;
  if (s < 0x1p-80f) return (double)squares<T>(q, 0x1p100f) * 0x1p-200;
  return (double)squares<T>(q, 0x1p-70f) * 0x1p140;
}

// Sum over the CTA, in a fixed order; every thread gets it.
__device__ __forceinline__ double cta_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll
  for (int i = 0; i < CL_THREADS / 32; ++i) v += red[i];
  return v;
}

// Partial sums: a CTA's chunks are the same in every run, so the norm repeats bit for bit.
// A thread's up to 64 squares are added in fp32, everything above in 64 bits.
template <class P>
__global__ void __launch_bounds__(CL_THREADS, CL_NORM_CTAS) clip_norm_kernel(const __grid_constant__ P p) {
  __shared__ double red[CL_THREADS / 32];
  allow_next();
  await_previous();
  double acc = 0.0;
  int at = 0;
  for (int c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    at = entry_of(p, c, at);
    const ClipEntry& e = p.e[at];
    const long long v0 = (long long)(c - e.begin) * CL_VECS;
    uint4 q[CL_HELD];
    if (e.bf16_) {
      load_share<bf16>(e, v0, q);
      acc += sum_share<bf16>(q);
    } else {
      load_share<float>(e, v0, q);
      acc += sum_share<float>(q);
    }
  }
  acc = cta_sum(acc, red);
  if (threadIdx.x == 0) p.part[blockIdx.x] = p.add ? p.part[blockIdx.x] + acc : acc;
}

// max_norm / norm as a number that fp32 holds in full and two powers of two, 1 unless the quotient is
// below 2^-100 (a subnormal factor would have lost its bits, not only where the results are subnormal).
struct Factor {
  float f, p[2];
};
__device__ __forceinline__ Factor factor_of(double q) {
  if (!(q < 0x1p-100 && q > 0.0)) return {(float)q, {1.f, 1.f}};
  int e;
  const double m = frexp(q, &e);
  e = max(e, -280);                       // (2^128 times that is no number of fp32 any more)
  return {(float)m, {ldexpf(1.f, e / 2), ldexpf(1.f, e - e / 2)}};
}

template <typename T>
__device__ __forceinline__ void scale_share(const ClipEntry& e, long long v0, const Factor& coef) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2;
  uint4 q[CL_HELD];
  const bool inside = load_share<T>(e, v0, q);
  uint4* base = static_cast<uint4*>(e.base);
#pragma unroll
  for (int k = 0; k < CL_HELD; ++k) {
    f32x2 v[P];
    widen(q[k], v, static_cast<const T*>(nullptr));
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = mul2(v[i], both(coef.f));
    if (coef.p[0] != 1.f) {
#pragma unroll
      for (int i = 0; i < P; ++i) v[i] = mul2(mul2(v[i], both(coef.p[0])), both(coef.p[1]));
    }
    uint4 o;
    if (sizeof(T) == 2)
      o = make_uint4(pack_bf16x2(lo2(v[0]), hi2(v[0])), pack_bf16x2(lo2(v[1]), hi2(v[1])),
                     pack_bf16x2(lo2(v[2 % P]), hi2(v[2 % P])), pack_bf16x2(lo2(v[3 % P]), hi2(v[3 % P])));
    else
      o = make_uint4(__float_as_uint(lo2(v[0])), __float_as_uint(hi2(v[0])), __float_as_uint(lo2(v[1])),
                     __float_as_uint(hi2(v[1])));
    const long long at = v0 + k * CL_THREADS + threadIdx.x, c = at * V;
    if (inside || (c >= e.first && c + V <= e.end)) {
      base[at] = o;
    } else if (c + V > e.first && c < e.end) {
      const T* x = reinterpret_cast<const T*>(&o);
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i >= e.first && c + i < e.end) static_cast<T*>(e.base)[c + i] = x[i];
    }
  }
}

// norm and, where it is above max_norm, the scaling.  The chunks are taken from the last to
// the first: the norm's pass has left the last ones in L2.
template <class P>
__global__ void __launch_bounds__(CL_THREADS, CL_SCALE_CTAS) clip_scale_kernel(const __grid_constant__ P p) {
  __shared__ double red[CL_THREADS / 32];
  await_previous();
  double s = 0.0;
  for (int i = threadIdx.x; i < p.ctas; i += CL_THREADS) s += __ldcg(p.part + i);
  const double norm = sqrt(cta_sum(s, red));
  if (p.norm && blockIdx.x == 0 && threadIdx.x == 0) *p.norm = (float)norm;
  if (p.only || norm <= p.max_norm) return;      // a NaN goes on, and makes every gradient NaN
  const Factor coef = factor_of(p.max_norm / norm);
  int at = p.n - 1;
  for (int c = p.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    if (p.e[at].begin > c) at = at > 0 && p.e[at - 1].begin <= c ? at - 1 : entry_of(p, c, 0);
    const ClipEntry& e = p.e[at];
    const long long v0 = (long long)(c - e.begin) * CL_VECS;
    if (e.bf16_) scale_share<bf16>(e, v0, coef);
    else scale_share<float>(e, v0, coef);
  }
}

// Whether two of the tensors share memory: scaled in place, their elements would be scaled
// by two threads at once.
int overlap(const muon_grad* g, int n, bool* found) {
  try {
    static thread_local std::vector<std::pair<uintptr_t, uintptr_t>> span;
    span.clear();
    for (int i = 0; i < n; ++i)
      if (g[i].numel > 0) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(g[i].G);
        span.push_back({a, a + (uintptr_t)g[i].numel * (g[i].dtype == MUON_DTYPE_BF16 ? 2 : 4)});
      }
    std::sort(span.begin(), span.end());
    *found = false;
    for (size_t i = 1; i < span.size(); ++i) *found = *found || span[i].first < span[i - 1].second;
  } catch (...) {        // no memory for the list
    return MUON_ERR_WORKSPACE;
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" size_t muon_clip_workspace_size(void) { return CL_MAX_CTAS * sizeof(double); }

extern "C" int muon_clip_grad_norm(const muon_grad* grads, int n, double max_norm, float* norm, void* ws,
                                   size_t ws_bytes, muon_stream_t stream) {
  begin_launches();
  if (n < 0 || !(max_norm >= 0.0) || !norm || reinterpret_cast<uintptr_t>(norm) % 4) return MUON_ERR_INVALID;
  if (n > 0 && !grads) return MUON_ERR_INVALID;
  for (int i = 0; i < n; ++i) {
    const muon_grad& a = grads[i];
    if (a.numel < 0) return MUON_ERR_INVALID;
    if (a.dtype != MUON_DTYPE_F32 && a.dtype != MUON_DTYPE_BF16) return MUON_ERR_UNSUPPORTED;
    if (a.numel == 0) continue;
    if (a.numel >= (1LL << 42)) return MUON_ERR_UNSUPPORTED;
    if (!a.G || reinterpret_cast<uintptr_t>(a.G) % (a.dtype == MUON_DTYPE_BF16 ? 2 : 4)) return MUON_ERR_INVALID;
  }
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 8 || ws_bytes < muon_clip_workspace_size()) return MUON_ERR_WORKSPACE;
  if (std::isfinite(max_norm)) {        // (the norm alone may count a tensor twice)
    bool found = false;
    if (int rc = overlap(grads, n, &found)) return rc;
    if (found) return MUON_ERR_INVALID;
  }
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int most = std::min(sms * CL_NORM_CTAS, CL_MAX_CTAS);
  static thread_local ClipParams<CL_ENTRIES> p;
  static thread_local ClipParams<CL_FEW> few;
  p.part = static_cast<double*>(ws);
  p.max_norm = max_norm;
  p.only = !std::isfinite(max_norm);
  // Fills the table from tensor *i on; returns whether there was anything.
  auto fill = [&](int* i) {
    int j = 0;
    long long chunks = 0;
    for (; *i < n && j < CL_ENTRIES; ++*i) {
      const muon_grad& a = grads[*i];
      if (a.numel == 0) continue;
      const int es = a.dtype == MUON_DTYPE_BF16 ? 2 : 4;
      const uintptr_t at = reinterpret_cast<uintptr_t>(a.G), base = at & ~uintptr_t(15);
      const long long first = (long long)(at - base) / es, end = first + a.numel;
      const long long nc = (end * es + 16LL * CL_VECS - 1) / (16LL * CL_VECS);
      if (chunks + nc >= (1LL << 30)) break;
      p.e[j++] = ClipEntry{reinterpret_cast<void*>(base), first, end, (int)chunks, es == 2};
      chunks += nc;
    }
    p.n = j;
    p.chunks = (int)chunks;
  };
  auto launch = [&](bool scale, int grid) {
    count_launch();
    if (p.n > CL_FEW)
      return scale ? launch_after(clip_scale_kernel<ClipParams<CL_ENTRIES>>, dim3(grid), dim3(CL_THREADS), 0, s, p)
                   : launch_after(clip_norm_kernel<ClipParams<CL_ENTRIES>>, dim3(grid), dim3(CL_THREADS), 0, s, p);
    few.n = p.n;
    few.chunks = p.chunks;
    few.ctas = p.ctas;
    few.add = p.add;
    few.only = p.only;
    few.part = p.part;
    few.max_norm = p.max_norm;
    few.norm = p.norm;
    std::copy(p.e, p.e + p.n, few.e);
    return scale ? launch_after(clip_scale_kernel<ClipParams<CL_FEW>>, dim3(grid), dim3(CL_THREADS), 0, s, few)
                 : launch_after(clip_norm_kernel<ClipParams<CL_FEW>>, dim3(grid), dim3(CL_THREADS), 0, s, few);
  };
  // the norm's launches leave as many partial sums as the largest of them has CTAs
  int launches = 0, i = 0;
  fill(&i);
  const bool one = i >= n;
  const int ctas = one ? std::max(1, std::min(most, p.chunks)) : most;
  while (true) {
    if (p.n == 0 && i < n) return MUON_ERR_UNSUPPORTED;
    p.ctas = ctas;
    p.add = launches > 0;
    p.norm = nullptr;
    if (launch(false, ctas) != cudaSuccess) return MUON_ERR_CUDA;
    ++launches;
    if (i >= n) break;
    fill(&i);
  }
  if (!one) {
    i = 0;
    fill(&i);
  }
  for (int k = 0; k < launches; ++k) {
    if (k > 0) fill(&i);
    p.ctas = ctas;
    p.norm = k == 0 ? norm : nullptr;
    if (k > 0 && p.only) break;
    const int grid = p.only ? 1 : std::max(1, std::min(sms * CL_SCALE_CTAS, p.chunks));
    if (launch(true, grid) != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}
