// Root-mean-square norm behind a residual's addition, forward and backward:
//   t = x + r (rounded to their type),   y = t rstd w,   rstd = 1/sqrt(mean(t^2) + eps)
//   dt = dtotal + rstd (g - xh mean(g xh)),   g = dy w,  xh = t rstd;   dw = sum_rows dy xh
// and, forward, y in 8 bits: e4m3 codes with one fp32 scale for each row and 128 columns.
// Every sum is fp32.  t is rounded before it is normed: it is what the residual stream keeps
// and what the backward pass reads.
//
// Bandwidth-bound.  Measured, of a copy's 6.68 TB/s: 32768 x 1536 bf16 with a residual, forward
// with the output in 8 bits 59 us (6.0 TB/s), backward with the weight's gradient 68 us (5.9; the
// column sums' kernel 4 of them); 32768 x 1537 bf16, rows off every 16-byte boundary, 85 and 87 us (4.7),
// in 8 bits 150 (2.4); 32768 x 1536 fp32 with a residual, forward 120 us (6.7), in 8 bits 101 (6.5),
// backward 124 (6.5); 5003 x 1537 fp32 forward 32 us (3.8), backward 24.6 (3.7).  What bounds the odd bf16
// rows is instructions: windows, masks and, in 8 bits, elements through shared memory; the odd fp32
// ones waits: a chain of copy, barrier and sum for each row, 8 rows a CTA, with 39% of the issue slots
// and 37% of DRAM's time in use.
#include <algorithm>
#include <cmath>
#include <cuda_fp8.h>

#include "rows.cuh"

namespace muon {
namespace {

using namespace rows;

constexpr int RMS_GROUP = MUON_RMS_GROUP;      // columns that share a scale
constexpr float RMS_LEAST_SCALE = 0x1p-100f;   // so that the reciprocal of a scale is finite
constexpr int RMS_LOOP_THREADS = 512;
constexpr int RMS_CTAS = 152;                  // lines of column sums at most

struct RmsFwd {
  const void *x, *r, *w;
  void *total, *y;
  uint8_t* codes;
  float *scales, *rstd;
  long long ldx, ldr, ldt, ldy, ldc, rows;
  int dim, w_bf16, groups;
  float eps;
};

// Max that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// The scale of a group whose largest magnitude is `most`, rounded to nearest, and its reciprocal within an ulp.
// The quotient is the product with the constant's reciprocal, corrected once by its exact remainder
// (Markstein): right for every mantissa; a remainder of an infinity is none.
__device__ __forceinline__ float2 scale_of(float most) {
  constexpr float R = 1.f / 448.f;
  const float q = most * R, s = fmaf(fmaf(-448.f, q, most), R, q);
  const float scale = max_nan(most <= 0x1.fffffep127f ? s : most, RMS_LEAST_SCALE);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scale));
  return make_float2(scale, inv);
}
// Two numbers to the nearest e4m3 codes (448 at most, NaN as NaN).
__device__ __forceinline__ uint32_t code2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Of two neighbouring codes (the first the smaller in magnitude) the one nearest to the fp32 quotient y/s.  That
// is their midpoint, and the even code is taken, where y/s is within half an ulp of it; else it is
// on y's side.  The midpoint has 5 bits: y - midpoint s is exact, and so are the comparisons.
__device__ __forceinline__ uint32_t nearer(uint32_t a, uint32_t b, float y, float s) {
  if (a == b) return a;
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)((a & 0x7Fu) | (b & 0x7Fu) << 8), __NV_E4M3);
  const __half2 v(h);
  const float mid = 0.5f * (__low2float(v) + __high2float(v)), d = fmaf(-mid, s, fabsf(y));
  const float power = __uint_as_float(__float_as_uint(mid) & 0x7F800000u), half = power * 0x1p-24f * s;
  if (d > half) return b;
  if (d < (mid == power ? -0.5f * half : -half)) return a;   // (numbers below a power of two lie closer)
  return b & 1u ? a : b;
}
// The codes nearest to y/s of kPairs pairs, two bytes each, in words; the quotient is rounded to fp32 first.  (bf16 numbers
// and weights make quotients that are midpoints of two codes, up to the roundings of y and s, of some 1 in
// 5000: the quotient's own rounding makes most of them midpoints again, which go to the even code.)
// y times the reciprocal is within 2^-22 of the quotient: where its neighbours 2^-21 below and above have one
// code, that is the code.
template <int kPairs>
__device__ __forceinline__ void codes_of(const f32x2* y, const float2& scale, uint32_t* w) {
  static_assert(kPairs % 2 == 0, "");
  const f32x2 below = both(scale.y * (1.f - 0x1p-21f)), above = both(scale.y * (1.f + 0x1p-21f));
#pragma unroll
  for (int i = 0; i < kPairs; i += 2) {
    const f32x2 a = mul2(y[i], below), b = mul2(y[i + 1], below), c = mul2(y[i], above), d = mul2(y[i + 1], above);
    uint32_t lo = code2(lo2(a), hi2(a)) | code2(lo2(b), hi2(b)) << 16;
    const uint32_t hi = code2(lo2(c), hi2(c)) | code2(lo2(d), hi2(d)) << 16;
    if (lo != hi) {
      uint32_t out = 0;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        const f32x2 p = k < 2 ? y[i] : y[i + 1];
        out |= nearer(lo >> 8 * k & 0xFFu, hi >> 8 * k & 0xFFu, k & 1 ? hi2(p) : lo2(p), scale.x) << 8 * k;
      }
      lo = out;
    }
    w[i / 2] = lo;
  }
}

// ---------------------------------------------------------------------------
// forward: rows whose pointers and strides allow 16-byte vectors
// ---------------------------------------------------------------------------

// x + r, rounded to their type, over x.
__device__ __forceinline__ void add16(uint4& x, const uint4& r, const bf16*) {
  auto sum = [](uint32_t a, uint32_t b) {
    const f32x2 s = add2(cvt2(a), cvt2(b));
    return pack_bf16x2(lo2(s), hi2(s));
  };
  x = make_uint4(sum(x.x, r.x), sum(x.y, r.y), sum(x.z, r.z), sum(x.w, r.w));
}
__device__ __forceinline__ void add16(uint4& x, const uint4& r, const float*) {
  auto sum = [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
  x = make_uint4(sum(x.x, r.x), sum(x.y, r.y), sum(x.z, r.z), sum(x.w, r.w));
}
// A vector of y to codes; its group of 128 columns lies in 16 neighbouring lanes (bf16) or in
// the warp (fp32).  The magnitudes' bits are compared as whole numbers: a NaN is the largest.
template <int V>
__device__ __forceinline__ void store_codes(const RmsFwd& p, long long row, int c, bool inside, const f32x2* y) {
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < V / 2; ++i)
    most = max(most, max(__float_as_uint(lo2(y[i])) & 0x7FFFFFFFu, __float_as_uint(hi2(y[i])) & 0x7FFFFFFFu));
#pragma unroll
  for (int o = RMS_GROUP / V / 2; o > 0; o >>= 1) most = max(most, __shfl_xor_sync(0xffffffffu, most, o));
  const float2 scale = scale_of(__uint_as_float(most));
  if (!inside) return;
  uint32_t w[V / 4];
  codes_of<V / 2>(y, scale, w);
  uint8_t* o = p.codes + row * p.ldc + c;
  if constexpr (V == 8) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (c % RMS_GROUP == 0) p.scales[row * p.groups + c / RMS_GROUP] = scale.x;
}

// A warp a row (kWarp) or a CTA a row.  The row stays in registers, as loaded, between its
// sum and its output, so that it is read once; all of a thread's loads are in flight together.
constexpr int RMS_WARPS = 8;
constexpr int RMS_MOST_THREADS = 512;
template <typename T, int kN, bool kWarp, int kW, bool kEight>
__global__ void __launch_bounds__(kWarp ? 32 * RMS_WARPS : RMS_MOST_THREADS) rms_forward_kernel(const RmsFwd p) {
  constexpr int V = 16 / (int)sizeof(T), C = V / 2, kSure = kWarp ? sure_of(kN) : 0;
  __shared__ __align__(8) float red[kWarp ? 2 : 128];
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x, size = kWarp ? 32 : blockDim.x;
  const long long r = kWarp ? (long long)blockIdx.x * RMS_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && r >= p.rows) return;
  Raw<T, V, kN> raw;
  raw.template load<kSure>(static_cast<const T*>(p.x) + r * p.ldx, t, size, p.dim);
  if (p.r) {
    Raw<T, V, kN> res;
    res.template load<kSure>(static_cast<const T*>(p.r) + r * p.ldr, t, size, p.dim);
#pragma unroll
    for (int k = 0; k < kN; ++k) add16(raw.q[k], res.q[k], static_cast<const T*>(nullptr));
    if (p.total) {
      T* total = static_cast<T*>(p.total) + r * p.ldt;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int c = (k * size + t) * V;
        if (k < kSure || c < p.dim) *reinterpret_cast<uint4*>(total + c) = raw.q[k];
      }
    }
  }
  f32x2 q = both(0.f);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    f32x2 v[C];
    raw.get(k, v);
#pragma unroll
    for (int i = 0; i < C; ++i) q = fma2(v[i], v[i], q);
  }
  const float ssq = lo2(q) + hi2(q);
  const float sum = kWarp ? warp_sum(ssq) : Group{t, size, 0, red}.sum(ssq, 0.f, 0).x;
  const float rs = 1.0f / sqrtf(sum * (1.f / (float)p.dim) + p.eps);
  raw.hold();
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = (k * size + t) * V;
    const bool inside = k < kSure || c < p.dim;
    f32x2 v[C], w[C];
    raw.get(k, v);
    if (kW == W_ASK || inside) weights<V, kW>(p.w, p.w_bf16, c, p.dim, 1.f, w);
    else
#pragma unroll
      for (int i = 0; i < C; ++i) w[i] = both(0.f);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = mul2(mul2(v[i], both(rs)), w[i]);
    if constexpr (kEight) store_codes<V>(p, r, c, inside, v);
    if (inside && (!kEight || p.y)) store16(static_cast<T*>(p.y) + r * p.ldy + c, v);
  }
  if (p.rstd && t == 0) p.rstd[r] = rs;
}

// ---------------------------------------------------------------------------
// rows of any alignment, through shared memory
// ---------------------------------------------------------------------------
// A row that starts off a 16-byte boundary is fetched in whole 16-byte words, from the one
// that holds its first element to the one that holds its last, and lies in shared memory as
// far behind a boundary as it does in global memory; results are staged likewise, at their own
// distance, and leave in whole words but for the ends.  (An element a thread moves 4 or 2
// bytes where a word moves 16: LSU-bound.)
// 16 bytes from `bytes` on (0 .. 15, a multiple of the element's size) of two words.
template <typename T>
__device__ __forceinline__ uint4 window(const uint4& lo, const uint4& hi, int bytes) {
  uint32_t a[7] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z};
  const uint32_t last = hi.w;
  uint32_t b[5];
  if (bytes & 8) {
#pragma unroll
    for (int i = 0; i < 5; ++i) a[i] = a[i + 2];
    a[5] = last;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) b[i] = bytes & 4 ? a[i + 1] : a[i];
  if (sizeof(T) == 2 && (bytes & 2)) {
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __funnelshift_r(b[i], b[i + 1], 16);
  }
  return make_uint4(b[0], b[1], b[2], b[3]);
}
template <typename T>
__device__ __forceinline__ void fetch_row(T* slot, const T* row, int dim, int t, int size) {
  const int off = behind(row), words = (int)(((off + dim) * sizeof(T) + 15) / 16);
  const uint4* src = reinterpret_cast<const uint4*>(row - off);
  for (int i = t; i < words; i += size) copy16(reinterpret_cast<uint4*>(slot) + i, src + i);
}
// slot holds the row from its `behind` on.
template <typename T>
__device__ __forceinline__ void flush_row(T* row, const T* slot, int dim, int t, int size) {
  constexpr int V = 16 / (int)sizeof(T);
  const int off = behind(row), end = off + dim, words = (end + V - 1) / V;
  T* dst = row - off;
  for (int i = t; i < words; i += size) {
    if (i * V >= off && i * V + V <= end) {
      reinterpret_cast<uint4*>(dst)[i] = reinterpret_cast<const uint4*>(slot)[i];
    } else {
      for (int c = max(i * V, off); c < min(i * V + V, end); ++c) dst[c] = slot[c];
    }
  }
}
template <typename T> __host__ __device__ constexpr int slot_bytes(int dim) {
  return (int)((dim * (long long)sizeof(T) + 31 + 15) / 16 * 16);
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.commit_group;\ncp.async.wait_group 0;" ::: "memory"); }

// The threads of a row (threadIdx.x) beside those of other rows (threadIdx.y).
struct RowThreads {
  int t, size, id;
  __device__ __forceinline__ void sync() const {
    if (size == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(size) : "memory");
  }
  // red: a float for each warp; every thread gets the sum, in a fixed order.  A second call needs a
  // sync() between.
  __device__ __forceinline__ float sum(float v, float* red) const {
    v = warp_sum(v);
    if (size == 32) return v;
    if ((t & 31) == 0) red[t >> 5] = v;
    sync();
    v = 0.f;
    for (int i = 0; i < size >> 5; ++i) v += red[i];
    return v;
  }
};

// Rows that start off the words' boundaries, in registers all the same, cut at the words of y
// (and of total, which has to lie like it).  A row that lies otherwise is read as windows of
// two words, and so are the weights; the words at the row's ends are masked, and stored by elements.
// Columns [pos - o, ...) of a row that begins o elements behind `base`; words without any
// element of the row are not read.
template <typename E>
__device__ __forceinline__ uint4 load_at(const E* base, int pos, int end) {
  constexpr int V = 16 / (int)sizeof(E), S = sizeof(E) == 2 ? 3 : 2;
  const int j = pos >> S, sh = pos & (V - 1);
  const uint4 none = make_uint4(0, 0, 0, 0);
  const uint4* q = reinterpret_cast<const uint4*>(base);
  const uint4 lo = j >= 0 && j * V < end ? q[j] : none;
  if (sh == 0) return lo;
  const uint4 hi = j + 1 >= 0 && (j + 1) * V < end ? q[j + 1] : none;
  return window<E>(lo, hi, sh * (int)sizeof(E));
}
template <typename T>
__device__ __forceinline__ void store_word(T* row, int c, int dim, const uint4& q) {
  constexpr int V = 16 / (int)sizeof(T);
  if (c >= 0 && c + V <= dim) {
    *reinterpret_cast<uint4*>(row + c) = q;
  } else {
    const T* x = reinterpret_cast<const T*>(&q);
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i >= 0 && c + i < dim) row[c + i] = x[i];
  }
}
template <typename T>
__device__ __forceinline__ uint4 packed(const f32x2* v) {
  if constexpr (sizeof(T) == 2)
    return make_uint4(pack_bf16x2(lo2(v[0]), hi2(v[0])), pack_bf16x2(lo2(v[1]), hi2(v[1])), pack_bf16x2(lo2(v[2]), hi2(v[2])),
                      pack_bf16x2(lo2(v[3]), hi2(v[3])));
  else
    return make_uint4(__float_as_uint(lo2(v[0])), __float_as_uint(hi2(v[0])), __float_as_uint(lo2(v[1])), __float_as_uint(hi2(v[1])));
}
// The weights of V columns from any c on, 0 outside the row.
template <int V, class P>
__device__ __forceinline__ void weights_at(const P& p, int c, f32x2* v) {
  if (!p.w) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = both(1.f);
  } else if (p.w_bf16) {
    const bf16* w = static_cast<const bf16*>(p.w);
    const int o = behind(w);
    const uint4 a = load_at(w - o, c + o, p.dim + o);
    v[0] = cvt2(a.x);
    v[1] = cvt2(a.y);
    if constexpr (V == 8) {
      v[2] = cvt2(a.z);
      v[3] = cvt2(a.w);
    }
  } else {
    const float* w = static_cast<const float*>(p.w);
    const int o = behind(w);
#pragma unroll
    for (int h = 0; h < V / 4; ++h) {
      const uint4 a = load_at(w - o, c + 4 * h + o, p.dim + o);
      v[2 * h] = make2(__uint_as_float(a.x), __uint_as_float(a.y));
      v[2 * h + 1] = make2(__uint_as_float(a.z), __uint_as_float(a.w));
    }
  }
  if (c < 0 || c + V > p.dim) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (c + i < 0 || c + i >= p.dim) v[i / 2] = i & 1 ? make2(lo2(v[i / 2]), 0.f) : make2(0.f, hi2(v[i / 2]));
  }
}
template <typename T, int kN, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * RMS_WARPS : RMS_MOST_THREADS) rms_forward_words_kernel(const RmsFwd p) {
  constexpr int V = 16 / (int)sizeof(T), C = V / 2;
  __shared__ __align__(8) float red[kWarp ? 2 : 128];
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x, size = kWarp ? 32 : blockDim.x, dim = p.dim;
  const long long r = kWarp ? (long long)blockIdx.x * RMS_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && r >= p.rows) return;
  T* y = static_cast<T*>(p.y) + r * p.ldy;
  const int off = behind(y);
  auto column = [&](int k) { return (k * size + t) * V - off; };
  auto row_word = [&](const T* row, int k) {
    const int c = column(k), o = behind(row);
    const uint4 q = load_at(row - o, c + o, dim + o);
    return c < 0 || c + V > dim ? masked_word<T>(q, -c, dim - c) : q;
  };
  Raw<T, V, kN> raw;
  const T* x = static_cast<const T*>(p.x) + r * p.ldx;
#pragma unroll
  for (int k = 0; k < kN; ++k) raw.q[k] = row_word(x, k);
  if (p.r) {
    const T* res = static_cast<const T*>(p.r) + r * p.ldr;
    Raw<T, V, kN> b;
#pragma unroll
    for (int k = 0; k < kN; ++k) b.q[k] = row_word(res, k);
#pragma unroll
    for (int k = 0; k < kN; ++k) add16(raw.q[k], b.q[k], static_cast<const T*>(nullptr));
    if (p.total) {
      T* total = static_cast<T*>(p.total) + r * p.ldt;
#pragma unroll
      for (int k = 0; k < kN; ++k) store_word(total, column(k), dim, raw.q[k]);
    }
  }
  f32x2 q = both(0.f);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    f32x2 v[C];
    raw.get(k, v);
#pragma unroll
    for (int i = 0; i < C; ++i) q = fma2(v[i], v[i], q);
  }
  const float ssq = lo2(q) + hi2(q);
  const float sum = kWarp ? warp_sum(ssq) : Group{t, size, 0, red}.sum(ssq, 0.f, 0).x;
  const float rs = 1.0f / sqrtf(sum * (1.f / (float)dim) + p.eps);
  raw.hold();
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = column(k);
    f32x2 v[C];
    raw.get(k, v);
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = mul2(v[i], both(rs));
    if (p.w && c < dim) {
      f32x2 w[C];
      weights_at<V>(p, c, w);
#pragma unroll
      for (int i = 0; i < C; ++i) v[i] = mul2(v[i], w[i]);
    }
    store_word(y, c, dim, packed<T>(v));
  }
  if (p.rstd && t == 0) p.rstd[r] = rs;
}

constexpr int RMS_ODD_GROUPS = 8;                 // rows a CTA at most
constexpr int RMS_ODD_SMEM = 200 * 1024;
// Slots: x, then y (or codes); the residual, or y without one; t with one.
template <typename T, bool kEight>
__global__ void __launch_bounds__(512) rms_forward_odd_kernel(const RmsFwd p, int slot) {
  extern __shared__ uint4 dyn[];
  __shared__ float red[RMS_ODD_GROUPS][16];
  const long long row = (long long)blockIdx.x * blockDim.y + threadIdx.y;
  if (row >= p.rows) return;
  const RowThreads g{(int)threadIdx.x, (int)blockDim.x, 1 + (int)threadIdx.y};
  const int slots = p.r ? 3 : 2, t = g.t, lane = t & 31, warp = t >> 5, nw = g.size >> 5;
  uint8_t* mine = reinterpret_cast<uint8_t*>(dyn) + (size_t)threadIdx.y * slots * slot;
  T* A = reinterpret_cast<T*>(mine);
  T* B = reinterpret_cast<T*>(mine + slot);
  T* D = reinterpret_cast<T*>(mine + 2 * slot);
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  fetch_row(A, x, p.dim, t, g.size);
  const T* a = A + behind(x);
  const T* b = nullptr;
  T* total = nullptr;
  T* d = nullptr;
  if (p.r) {
    const T* r = static_cast<const T*>(p.r) + row * p.ldr;
    fetch_row(B, r, p.dim, t, g.size);
    b = B + behind(r);
    if (p.total) total = static_cast<T*>(p.total) + row * p.ldt;
    d = D + (total ? behind(total) : 0);
  }
  copies_done();
  g.sync();
  float q = 0.f;
  if (p.r) {
#pragma unroll 4
    for (int c = t; c < p.dim; c += g.size) {
      const T v = from_f32<T>(to_f32(a[c]) + to_f32(b[c]));
      d[c] = v;
      q = fmaf(to_f32(v), to_f32(v), q);
    }
    a = d;
  } else {
#pragma unroll 4
    for (int c = t; c < p.dim; c += g.size) q = fmaf(to_f32(a[c]), to_f32(a[c]), q);
  }
  const float rs = 1.0f / sqrtf(g.sum(q, red[threadIdx.y]) * (1.f / (float)p.dim) + p.eps);
  if (g.size == 32) __syncwarp();      // (with more warps the sum has waited for all of d)
  if (total) flush_row(total, D, p.dim, t, g.size);
  // with a residual x's slot is free, without one the residual's
  T* Y = p.r ? A : B;
  T* y = p.y ? static_cast<T*>(p.y) + row * p.ldy : nullptr;
  auto norm_at = [&](int c) {
    const float v = to_f32(a[c]) * rs;
    return p.w ? v * ld_w(p.w, p.w_bf16, c) : v;
  };
  if constexpr (kEight) {
    uint8_t* codes = p.codes + row * p.ldc;
    uint8_t* o = reinterpret_cast<uint8_t*>(Y) + behind(codes);
    for (int k = warp; k < p.groups; k += nw) {
      float v[4];
      uint32_t most = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = k * RMS_GROUP + 32 * j + lane;
        v[j] = c < p.dim ? norm_at(c) : 0.f;
        most = max(most, __float_as_uint(v[j]) & 0x7FFFFFFFu);
      }
      most = __reduce_max_sync(0xffffffffu, most);
      const float2 scale = scale_of(__uint_as_float(most));
      if (lane == 0) p.scales[row * p.groups + k] = scale.x;
      const f32x2 pairs[2] = {make2(v[0], v[1]), make2(v[2], v[3])};
      uint32_t code;
      codes_of<2>(pairs, scale, &code);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = k * RMS_GROUP + 32 * j + lane;
        if (c < p.dim) {
          o[c] = (uint8_t)(code >> 8 * j);
          if (y) st1(y + c, v[j]);
        }
      }
    }
    g.sync();
    flush_row(codes, reinterpret_cast<const uint8_t*>(Y), p.dim, t, g.size);
  } else {
    T* o = Y + behind(y);
#pragma unroll 4
    for (int c = t; c < p.dim; c += g.size) o[c] = from_f32<T>(norm_at(c));
    g.sync();
    flush_row(y, static_cast<const T*>(Y), p.dim, t, g.size);
  }
  if (p.rstd && t == 0) p.rstd[row] = rs;
}

// Rows of any length: a CTA a row, three passes, the later ones from cache.
template <typename T>
__global__ void __launch_bounds__(RMS_LOOP_THREADS) rms_forward_loop_kernel(const RmsFwd p) {
  __shared__ float red[32];
  const long long row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = p.r ? static_cast<const T*>(p.r) + row * p.ldr : nullptr;
  T* total = p.total ? static_cast<T*>(p.total) + row * p.ldt : nullptr;
  auto sum_at = [&](int c) { return r ? to_f32(from_f32<T>(ld1(x + c) + ld1(r + c))) : ld1(x + c); };
  float q = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += RMS_LOOP_THREADS) {
    const float v = sum_at(c);
    if (total) st1(total + c, v);
    q = fmaf(v, v, q);
  }
  const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)p.dim + p.eps);
  // (block_sum's barriers order the writes of `total` before its reads by other threads)
  const T* t = total ? total : x;
  const bool again = r && !total;
  auto norm_at = [&](int c) {
    const float v = (again ? sum_at(c) : ld1(t + c)) * rs;
    return p.w ? v * ld_w(p.w, p.w_bf16, c) : v;
  };
  if (p.codes) {
    const int lane = threadIdx.x & 31;
    for (int g = threadIdx.x >> 5; g < p.groups; g += RMS_LOOP_THREADS / 32) {
      float v[4], most = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = g * RMS_GROUP + 32 * j + lane;
        v[j] = c < p.dim ? norm_at(c) : 0.f;
        most = max_nan(most, fabsf(v[j]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, o));
      const float2 scale = scale_of(most);
      if (lane == 0) p.scales[row * p.groups + g] = scale.x;
      const f32x2 pairs[2] = {make2(v[0], v[1]), make2(v[2], v[3])};
      uint32_t code;
      codes_of<2>(pairs, scale, &code);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = g * RMS_GROUP + 32 * j + lane;
        if (c < p.dim) {
          p.codes[row * p.ldc + c] = (uint8_t)(code >> 8 * j);
          if (p.y) st1(static_cast<T*>(p.y) + row * p.ldy + c, v[j]);
        }
      }
    }
  } else {
    T* y = static_cast<T*>(p.y) + row * p.ldy;
    for (int c = threadIdx.x; c < p.dim; c += RMS_LOOP_THREADS) st1(y + c, norm_at(c));
  }
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rs;
}

struct RmsBwd {
  const void *dy, *t, *w, *dtotal;
  const float* rstd;
  void* dx;
  float* part;             // [line][dim] sums over a line's rows, or null
  long long lddy, ldt, lddt, lddx, rows;
  int dim, w_bf16;
};

// A persistent CTA of several row groups (threadIdx.y).  A thread owns the same columns of
// every row its group takes, so the weights and the columns' sums stay in its registers; at
// the end the groups' sums are joined in shared memory in a fixed order and the CTA writes
// one line.  Rows come through a ring of asynchronous copies, R - 1 rows ahead.
constexpr int RMS_GROUPS = 16;
// 16 columns a thread leave 512 threads of an SM 128 registers each, 8 leave 768 some 80.  Rows
// that need windows and masks have more instructions a column to hide: 8 (32768 x 1537 bf16
// 88 us against 93, 5003 x 1537 fp32 25.4 against 27.5); the others 16 (32768 x 1536 bf16 69.1
// against 70.2).
__host__ __device__ constexpr int rms_threads(int columns, bool odd) { return odd && columns <= 8 ? 768 : 512; }
constexpr int RMS_RING = 3;
constexpr int RMS_GUARD = 8;       // words (one would do, and leave every access across two lines)

// The groups' sums of E columns a thread, to the CTA's line.
template <int E, class Column, class Sum>
__device__ __forceinline__ void join_columns(const RmsBwd& p, Column column, Sum sum) {
  extern __shared__ uint4 dyn[];
  const int g = threadIdx.y;
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                              // the ring's memory is free for the sums
  float* sums = reinterpret_cast<float*>(dyn);  // [groups - 1][dim]
  if (g > 0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (column(e) >= 0 && column(e) < p.dim) sums[(size_t)(g - 1) * p.dim + column(e)] = sum(e);
  }
  __syncthreads();
  if (g > 0) return;
  float* o = p.part + (size_t)blockIdx.x * p.dim;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = column(e);
    if (c >= 0 && c < p.dim) {
      float a = sum(e);
      for (int j = 0; j < (int)blockDim.y - 1; ++j) a += sums[(size_t)j * p.dim + c];
      o[c] = a;
    }
  }
}

// Rows in 16-byte words.  Where all of them start on a word (!kOdd) each thread reads only what
// it copied itself, so the ring needs no barrier.  Others (kOdd) are cut at the words of dx:
// a group's rows lie a multiple of 16 bytes apart (a number of rows that is one of the
// elements of a word), so the place of a row's first element in its word, and with it a
// thread's columns, stay.  A stream that starts elsewhere in its words than dx is read through a window
// of two words, which the threads beside have copied.
template <typename T, int kN, bool kDt, int R, bool kOdd>
__global__ void __launch_bounds__(rms_threads(kN * 16 / (int)sizeof(T), kOdd), 1) rms_backward_kernel(const RmsBwd p) {
  extern __shared__ uint4 dyn[];
  __shared__ float red[2][RMS_GROUPS][24];
  constexpr int V = 16 / (int)sizeof(T), C = V / 2, P = kN * C, S = kDt ? 3 : 2;
  allow_next();
  const RowThreads g{(int)threadIdx.x, (int)blockDim.x, 1 + (int)threadIdx.y};
  const int t = g.t, groups = blockDim.y;
  const float inv = 1.f / (float)p.dim;
  const long long step = (long long)gridDim.x * groups;
  long long r = (long long)blockIdx.x * groups + threadIdx.y, rf = r;
  T* dx = static_cast<T*>(p.dx) + r * p.lddx;
  const T *tf = static_cast<const T*>(p.t) + r * p.ldt, *gf = static_cast<const T*>(p.dy) + r * p.lddy;
  const T* df = kDt ? static_cast<const T*>(p.dtotal) + r * p.lddt : nullptr;
  // where in its first word a row of each begins
  const int off = kOdd ? behind(dx) : 0, ot = kOdd ? behind(tf) : 0, og = kOdd ? behind(gf) : 0, od = kOdd && kDt ? behind(df) : 0;
  dx -= off;
  tf -= ot;
  gf -= og;
  if (kDt) df -= od;
  const bool shifted = kOdd && (ot != off || og != off || (kDt && od != off));
  // a thread's word k begins at this column
  auto column = [&](int k) { return (k * g.size + t) * V - off; };
  f32x2 w[P], sw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) sw[i] = both(0.f);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    if constexpr (kOdd) {
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const int c = column(k) + 2 * i;
        auto at = [&](int c) { return c >= 0 && c < p.dim ? (p.w ? ld_w(p.w, p.w_bf16, c) : 1.f) : 0.f; };
        w[k * C + i] = make2(at(c), at(c + 1));
      }
    } else {
      weights<V>(p.w, p.w_bf16, column(k), p.dim, 1.f, w + k * C);
    }
  }
  // [slot][stream][word], with room at either end
  constexpr int G = kOdd ? RMS_GUARD : 0;
  const int W = kN * g.size + 2 * G;
  uint4* const mine = dyn + (size_t)threadIdx.y * (R * S * W) + G + t;
  auto fetch = [&](int slot) {                  // one group of copies, empty past the last row
    if (rf < p.rows) {
      uint4* d = mine + slot * (S * W);
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int c = (k * g.size + t) * V;
        if (c < p.dim + ot) copy16(d + k * g.size, tf + c);
        if (c < p.dim + og) copy16(d + W + k * g.size, gf + c);
        if (kDt && c < p.dim + od) copy16(d + 2 * W + k * g.size, df + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    rf += step;
    tf += step * p.ldt;
    gf += step * p.lddy;
    if (kDt) df += step * p.lddt;
  };
  if constexpr (!kOdd) {
    // words that are never copied to belong to columns past the row: zero
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (column(k) >= p.dim)
        for (int s = 0; s < S * R; ++s) mine[s * W + k * g.size] = make_uint4(0, 0, 0, 0);
  }
  for (int s = 0; s < R - 1; ++s) fetch(s);
  // word k of a stream that begins `o` elements into its words
  auto word = [&](const uint4* d, int k, int o) {
    if (!shifted || o == off) return d[k * g.size];
    const int from = o - off, back = from < 0;
    const uint4* e = d + k * g.size - back;
    return window<T>(e[0], e[1], (from + back * V) * (int)sizeof(T));
  };
  bool edge[kN];                                // words that reach past the row's ends
#pragma unroll
  for (int k = 0; k < kN; ++k) edge[k] = kOdd && (column(k) < 0 || column(k) + V > p.dim);
  float rs_n = r < p.rows ? p.rstd[r] : 0.f;
  int parity = 0, at = 0;
  for (; r < p.rows; r += step, dx += step * p.lddx) {
    fetch(at == 0 ? R - 1 : at - 1);
    const float rs = rs_n;
    if (r + step < p.rows) rs_n = p.rstd[r + step];
    asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory");
    if (shifted) g.sync();                      // the neighbours' copies are there
    const uint4* d = mine + at * (S * W);
    at = at + 1 == R ? 0 : at + 1;
    f32x2 xh[P], gr[P], s = both(0.f);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      uint4 a = word(d, k, ot), b = word(d + W, k, og);
      if (edge[k]) {
        a = masked_word<T>(a, -column(k), p.dim - column(k));
        b = masked_word<T>(b, -column(k), p.dim - column(k));
      }
      widen(a, xh + k * C, static_cast<const T*>(nullptr));
      widen(b, gr + k * C, static_cast<const T*>(nullptr));
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      xh[i] = mul2(xh[i], both(rs));
      sw[i] = fma2(gr[i], xh[i], sw[i]);
      gr[i] = mul2(gr[i], w[i]);
      s = fma2(gr[i], xh[i], s);
    }
    const float m = g.sum(lo2(s) + hi2(s), red[parity][threadIdx.y]) * inv;
    parity ^= 1;
    const f32x2 c1 = both(rs), c2 = both(-rs * m);
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = column(k);
      f32x2 v[C];
      if (kDt) widen(word(d + 2 * W, k, od), v, static_cast<const T*>(nullptr));
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const f32x2 a = fma2(gr[k * C + i], c1, mul2(xh[k * C + i], c2));
        v[i] = kDt ? add2(v[i], a) : a;
      }
      if (!edge[k]) {
        if (kOdd || c < p.dim) store16(dx + c + off, v);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i >= 0 && c + i < p.dim) st1(dx + off + c + i, elem(v, i));
      }
    }
    if (shifted) g.sync();                      // the slot is read before its next row arrives
  }
  if (p.part)
    join_columns<kN * V>(p, [&](int e) { return column(e / V) + e % V; }, [&](int e) { return elem(sw, e); });
}

// Rows wider than that: dx, a CTA a row with the row in registers, and the columns' sums over
// slabs of rows in a pass of their own.  kOdd: rows off the words' boundaries, cut at dx's.
template <typename T, int kN, bool kOdd>
__global__ void __launch_bounds__(kN == 4 ? 768 : RMS_MOST_THREADS) rms_dx_kernel(const RmsBwd p) {
  constexpr int V = 16 / (int)sizeof(T), C = V / 2;
  __shared__ float red[24];
  const RowThreads g{(int)threadIdx.x, (int)blockDim.x, 0};
  const long long r = blockIdx.x;
  T* dx = static_cast<T*>(p.dx) + r * p.lddx;
  const int off = kOdd ? behind(dx) : 0;
  auto column = [&](int k) { return (k * g.size + g.t) * V - off; };
  auto word = [&](const T* row, int k) {
    const int c = column(k);
    if constexpr (!kOdd) return c < p.dim ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    const int o = behind(row);
    const uint4 q = load_at(row - o, c + o, p.dim + o);
    return c < 0 || c + V > p.dim ? masked_word<T>(q, -c, p.dim - c) : q;
  };
  auto weight = [&](int k, f32x2* w) {
    if constexpr (!kOdd) weights<V>(p.w, p.w_bf16, column(k), p.dim, 1.f, w);
    else weights_at<V>(p, column(k), w);
  };
  Raw<T, V, kN> a, b;
#pragma unroll
  for (int k = 0; k < kN; ++k) a.q[k] = word(static_cast<const T*>(p.t) + r * p.ldt, k);
#pragma unroll
  for (int k = 0; k < kN; ++k) b.q[k] = word(static_cast<const T*>(p.dy) + r * p.lddy, k);
  const float rs = p.rstd[r];
  f32x2 s = both(0.f);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    f32x2 x[C], y[C], w[C];
    a.get(k, x);
    b.get(k, y);
    weight(k, w);
#pragma unroll
    for (int i = 0; i < C; ++i) s = fma2(mul2(y[i], w[i]), mul2(x[i], both(rs)), s);
  }
  a.hold();
  b.hold();
  const float m = -rs * (g.sum(lo2(s) + hi2(s), red) * (1.f / (float)p.dim));
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = column(k);
    if (c >= p.dim) continue;
    f32x2 x[C], y[C], w[C];
    a.get(k, x);
    b.get(k, y);
    weight(k, w);
#pragma unroll
    for (int i = 0; i < C; ++i) y[i] = fma2(mul2(y[i], w[i]), both(rs), mul2(mul2(x[i], both(rs)), both(m)));
    if (p.dtotal) {
      widen(word(static_cast<const T*>(p.dtotal) + r * p.lddt, k), x, static_cast<const T*>(nullptr));
#pragma unroll
      for (int i = 0; i < C; ++i) y[i] = add2(x[i], y[i]);
    }
    if constexpr (!kOdd) store16(dx + c, y);
    else store_word(dx, c, p.dim, packed<T>(y));
  }
}
// A word of columns a thread.  Rows a number of slabs apart that is one of a word's elements
// begin at the same place in their words (kOdd: those of t).
constexpr int RMS_SLAB_THREADS = 128;
template <typename T, bool kOdd>
__global__ void __launch_bounds__(RMS_SLAB_THREADS) rms_slab_kernel(const RmsBwd p) {
  constexpr int V = 16 / (int)sizeof(T), P = V / 2, H = 4;     // H rows in flight
  const int off = kOdd ? behind(static_cast<const T*>(p.t) + blockIdx.y * p.ldt) : 0;
  const int og = kOdd ? behind(static_cast<const T*>(p.dy) + blockIdx.y * p.lddy) : 0;
  const int c = (blockIdx.x * RMS_SLAB_THREADS + threadIdx.x) * V - off;
  if (c >= p.dim) return;
  f32x2 s[P];
#pragma unroll
  for (int i = 0; i < P; ++i) s[i] = both(0.f);
  auto word = [&](const T* row, int o) {
    if constexpr (!kOdd) return *reinterpret_cast<const uint4*>(row + c);
    return load_at(row - o, c + o, p.dim + o);
  };
  for (long long r0 = blockIdx.y; r0 < p.rows; r0 += (long long)gridDim.y * H) {
    uint4 a[H], b[H];
    float rs[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const long long r = r0 + (long long)gridDim.y * h, q = r < p.rows ? r : r0;
      a[h] = word(static_cast<const T*>(p.t) + q * p.ldt, off);
      b[h] = word(static_cast<const T*>(p.dy) + q * p.lddy, og);
      rs[h] = r < p.rows ? p.rstd[r] : 0.f;
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (h > 0 && r0 + (long long)gridDim.y * h >= p.rows) break;
      f32x2 x[P], y[P];
      widen(a[h], x, static_cast<const T*>(nullptr));
      widen(b[h], y, static_cast<const T*>(nullptr));
#pragma unroll
      for (int i = 0; i < P; ++i) s[i] = fma2(y[i], mul2(x[i], both(rs[h])), s[i]);
    }
  }
  float* o = p.part + (size_t)blockIdx.y * p.dim;
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (!kOdd || (c + e >= 0 && c + e < p.dim)) o[c + e] = elem(s, e);   // (what lies outside the row was summed, too)
}

// Rows of any length: dx with the row read twice.
template <typename T>
__global__ void __launch_bounds__(RMS_LOOP_THREADS) rms_backward_loop_kernel(const RmsBwd p) {
  __shared__ float red[32];
  const long long r = blockIdx.x;
  const float rs = p.rstd[r];
  const T* t = static_cast<const T*>(p.t) + r * p.ldt;
  const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
  const T* dt = p.dtotal ? static_cast<const T*>(p.dtotal) + r * p.lddt : nullptr;
  T* dx = static_cast<T*>(p.dx) + r * p.lddx;
  float s = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += RMS_LOOP_THREADS)
    s = fmaf(ld1(dy + c) * (p.w ? ld_w(p.w, p.w_bf16, c) : 1.f), ld1(t + c) * rs, s);
  const float m = block_sum(s, red) / (float)p.dim;
  for (int c = threadIdx.x; c < p.dim; c += RMS_LOOP_THREADS) {
    const float g = ld1(dy + c) * (p.w ? ld_w(p.w, p.w_bf16, c) : 1.f);
    const float v = rs * (g - ld1(t + c) * rs * m);
    st1(dx + c, dt ? v + ld1(dt + c) : v);
  }
}

// Column sums of the lines: 32 columns a CTA, 32 threads a column over the lines (each a
// fixed set), then a fixed tree.
__global__ void __launch_bounds__(1024) rms_columns_kernel(const float* part, int lines, int dim, void* dw, int w_bf16) {
  __shared__ float tile[32][33];
  await_previous();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < dim) {
    float v[(RMS_CTAS + 31) / 32];               // all of them asked for at once
#pragma unroll
    for (int i = 0; i < (RMS_CTAS + 31) / 32; ++i) {
      const int l = 32 * i + threadIdx.y;
      v[i] = l < lines ? part[(size_t)l * dim + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < (RMS_CTAS + 31) / 32; ++i) s += v[i];
  }
  tile[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(tile[threadIdx.x][threadIdx.y]);
  const int oc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && oc < dim) st_w(dw, w_bf16, oc, s);
}

template <typename T, int kN, bool kWarp, bool kEight>
void forward_launch(const RmsFwd& p, int threads, cudaStream_t s) {
  const unsigned grid = (unsigned)(kWarp ? cdiv(p.rows, RMS_WARPS) : p.rows);
  if constexpr (kWarp) {
    if (p.w && p.w_bf16) { rms_forward_kernel<T, kN, kWarp, W_BF16, kEight><<<grid, threads, 0, s>>>(p); return; }
    if (p.w) { rms_forward_kernel<T, kN, kWarp, W_F32, kEight><<<grid, threads, 0, s>>>(p); return; }
  }
  rms_forward_kernel<T, kN, kWarp, W_ASK, kEight><<<grid, threads, 0, s>>>(p);
}

// Threads of a row of so many elements through shared memory: 16 elements each.
int odd_threads(int dim) { return std::min(512, 32 * cdiv(dim, 512)); }

// A warp a row while a lane holds its share of x and of the residual in registers (8 vectors
// each: 2048 bf16 columns), then a CTA a row with 4 to 8 vectors a thread.
template <typename T, bool kEight>
cudaError_t forward(const RmsFwd& p, bool vec, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  const int words = cdiv(p.dim - 1LL, V) + 1;       // that a row may touch
  // whether total's rows begin where y's do in their words
  const bool alike = !p.total || ((uintptr_t)p.total % 16 == (uintptr_t)p.y % 16 && (p.rows == 1 || (p.ldt - p.ldy) % V == 0));
  const int n = p.dim / V, need = cdiv(n, 32), slot = slot_bytes<T>(std::min(p.dim, 1 << 20)), slots = p.r ? 3 : 2;
  count_launch();
  if (vec && need <= 8) {
    by_accesses(need, [&](auto N) {
      if constexpr (decltype(N)::value <= 8) forward_launch<T, decltype(N)::value, true, kEight>(p, 32 * RMS_WARPS, s);
    });
  } else if (vec && n <= 8 * RMS_MOST_THREADS) {
    int threads = 64;
    while (threads * 8 < n) threads *= 2;
    const int each = cdiv(n, threads);
    if (each <= 5) forward_launch<T, 5, false, kEight>(p, threads, s);
    else if (each == 6) forward_launch<T, 6, false, kEight>(p, threads, s);
    else forward_launch<T, 8, false, kEight>(p, threads, s);
  } else if (!kEight && alike && words <= 8 * RMS_MOST_THREADS) {
    if (words <= 256) {
      by_accesses(cdiv(words, 32), [&](auto N) {
        if constexpr (decltype(N)::value <= 8)
          rms_forward_words_kernel<T, decltype(N)::value, true><<<cdiv(p.rows, RMS_WARPS), 32 * RMS_WARPS, 0, s>>>(p);
      });
    } else {
      int threads = 64;
      while (threads * 8 < words) threads *= 2;
      if (cdiv(words, threads) <= 6) rms_forward_words_kernel<T, 6, false><<<(unsigned)p.rows, threads, 0, s>>>(p);
      else rms_forward_words_kernel<T, 8, false><<<(unsigned)p.rows, threads, 0, s>>>(p);
    }
  } else if ((long long)slots * slot <= RMS_ODD_SMEM) {
    const int threads = odd_threads(p.dim);
    // a few rows a CTA, as long as an SM still holds several CTAs
    const int groups = std::max(1, std::min(std::min(256 / threads, RMS_ODD_GROUPS), 48 * 1024 / (slots * slot)));
    const int smem = groups * slots * slot;
    if (smem > 40 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(rms_forward_odd_kernel<T, kEight>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, RMS_ODD_SMEM);
      if (e != cudaSuccess) return e;
    }
    rms_forward_odd_kernel<T, kEight><<<cdiv(p.rows, groups), dim3(threads, groups), smem, s>>>(p, slot);
  } else {
    rms_forward_loop_kernel<T><<<(unsigned)p.rows, RMS_LOOP_THREADS, 0, s>>>(p);
  }
  return cudaGetLastError();
}

template <class K>
cudaError_t allow_smem(K kern, size_t smem) {
  return smem <= 40 * 1024 ? cudaSuccess : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, RMS_ODD_SMEM);
}

// Row groups of a persistent CTA of so many threads a row and bytes of shared memory a group.
int row_groups(int most, int threads, size_t bytes, const RmsBwd& p, size_t* smem) {
  int groups = std::max(1, std::min(most / threads, threads == 32 ? RMS_GROUPS : 15));   // (15 barriers)
  auto need = [&](int g) { return std::max(bytes * g, p.part ? (size_t)(g - 1) * p.dim * 4 : 0); };
  while (groups > 1 && need(groups) > (size_t)RMS_ODD_SMEM) --groups;
  *smem = need(groups);
  return groups;
}

template <typename T, int kN, bool kOdd>
cudaError_t backward_words(const RmsBwd& p, int threads, int* lines, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  auto bytes = [&](int ring, int streams) { return (size_t)ring * streams * (kN * threads + (kOdd ? 2 * RMS_GUARD : 0)) * 16; };
  auto go = [&](auto kern, size_t each) {
    size_t smem = 0;
    const int groups = row_groups(rms_threads(kN * V, kOdd), threads, each, p, &smem);
    const cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    int n = (int)std::min<long long>(cdiv(p.rows, groups), RMS_CTAS);
    if (kOdd)       // a number of rows at a time that is one of a word's elements (152 are)
      while (n * groups % V) ++n;
    *lines = n;
    count_launch();
    kern<<<n, dim3(threads, groups), smem, s>>>(p);
    return cudaGetLastError();
  };
  if (!p.dtotal) return go(rms_backward_kernel<T, kN, false, RMS_RING, kOdd>, bytes(RMS_RING, 2));
  // (three streams of more than 5460 fp32 columns fill the memory with a row less ahead)
  if (bytes(RMS_RING, 3) > (size_t)RMS_ODD_SMEM) return go(rms_backward_kernel<T, kN, true, 2, kOdd>, bytes(2, 3));
  return go(rms_backward_kernel<T, kN, true, RMS_RING, kOdd>, bytes(RMS_RING, 3));
}

// A thread's columns: 16, but 8 where 16 would leave a row to less than two warps, and for rows
// off the words' boundaries where 768 threads cover them.
template <typename T>
cudaError_t backward(const RmsBwd& p, bool vec, int* lines, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  *lines = 0;
  if (p.rows == 0) return cudaSuccess;
  const int n = vec ? p.dim / V : cdiv(p.dim - 1LL, V) + 1;     // words a row may touch
  auto threads = [&](int each) { return 32 * cdiv(n, 32LL * each); };
  if (vec && n <= 32 * 16 / V) return backward_words<T, 8 / V, false>(p, threads(8 / V), lines, s);
  if (vec && threads(16 / V) <= rms_threads(16, false)) return backward_words<T, 16 / V, false>(p, threads(16 / V), lines, s);
  if (!vec && threads(8 / V) <= rms_threads(8, true)) return backward_words<T, 8 / V, true>(p, threads(8 / V), lines, s);
  if (!vec && threads(16 / V) <= rms_threads(16, true)) return backward_words<T, 16 / V, true>(p, threads(16 / V), lines, s);
  // the columns' sums before dx, which may be dy itself
  if (p.part) {
    *lines = (int)std::min<long long>((p.rows + V - 1) / V * V, RMS_CTAS);   // (152 is a multiple of V)
    const dim3 grid(cdiv(n, RMS_SLAB_THREADS), *lines);
    count_launch();
    if (vec) rms_slab_kernel<T, false><<<grid, RMS_SLAB_THREADS, 0, s>>>(p);
    else rms_slab_kernel<T, true><<<grid, RMS_SLAB_THREADS, 0, s>>>(p);
  }
  count_launch();
  auto dx = [&](auto kern, int each) { kern<<<(unsigned)p.rows, 32 * cdiv(n, 32LL * each), 0, s>>>(p); };
  if (n <= 4 * 768) vec ? dx(rms_dx_kernel<T, 4, false>, 4) : dx(rms_dx_kernel<T, 4, true>, 4);
  else if (n <= 8 * RMS_MOST_THREADS) vec ? dx(rms_dx_kernel<T, 8, false>, 8) : dx(rms_dx_kernel<T, 8, true>, 8);
  else rms_backward_loop_kernel<T><<<(unsigned)p.rows, RMS_LOOP_THREADS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" int muon_rmsnorm_forward(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                                    int64_t rows, int64_t dim, int x_dtype, int w_dtype, float eps, void* total,
                                    int64_t ldt, void* y, int64_t ldy, uint8_t* codes, int64_t ldc, float* scales,
                                    float* rstd, muon_stream_t stream) {
  begin_launches();
  if (!sizes_ok(rows, dim) || !(eps >= 0.f)) return MUON_ERR_INVALID;
  if (!known(x_dtype) || !known(w_dtype)) return MUON_ERR_UNSUPPORTED;
  if ((codes != nullptr) != (scales != nullptr)) return MUON_ERR_INVALID;
  if (rows == 0) return MUON_OK;
  if (!x || ldx < dim || (!y && !codes) || (y && ldy < dim) || (codes && ldc < dim)) return MUON_ERR_INVALID;
  if ((residual && ldr < dim) || (total && (!residual || ldt < dim || total == y))) return MUON_ERR_INVALID;
  const size_t xs = dt_size(x_dtype), ws = dt_size(w_dtype);
  if (!is_aligned(x, xs) || !is_aligned(residual, xs) || !is_aligned(total, xs) || !is_aligned(y, xs) ||
      !is_aligned(weight, ws) || !is_aligned(scales, 4) || !is_aligned(rstd, 4))
    return MUON_ERR_INVALID;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RmsFwd p{x, residual, weight, total, y, codes, scales, rstd, ldx, ldr, ldt, ldy, ldc, rows,
                 (int)dim, w_dtype == MUON_DTYPE_BF16, cdiv(dim, RMS_GROUP), eps};
  const bool vec = dim * xs % 16 == 0 && vec_rows(x, ldx, rows, xs) && (!residual || vec_rows(residual, ldr, rows, xs)) &&
                   (!total || vec_rows(total, ldt, rows, xs)) && (!y || vec_rows(y, ldy, rows, xs)) &&
                   is_aligned(weight, 16) && (!codes || (is_aligned(codes, 16 / xs) && (rows == 1 || ldc % (16 / xs) == 0)));
  const cudaError_t e = x_dtype == MUON_DTYPE_BF16 ? (codes ? forward<bf16, true>(p, vec, s) : forward<bf16, false>(p, vec, s))
                                                   : (codes ? forward<float, true>(p, vec, s) : forward<float, false>(p, vec, s));
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" size_t muon_rmsnorm_workspace_size(int64_t rows, int64_t dim) {
  if (!sizes_ok(rows, dim)) return (size_t)-1;
  return (size_t)RMS_CTAS * (size_t)dim * sizeof(float);
}

extern "C" int muon_rmsnorm_backward(const void* dy, int64_t lddy, const void* total, int64_t ldt, const void* weight,
                                     const float* rstd, const void* dtotal, int64_t lddt, int64_t rows, int64_t dim,
                                     int x_dtype, int w_dtype, void* dx, int64_t lddx, void* dweight, void* ws,
                                     size_t ws_bytes, muon_stream_t stream) {
  begin_launches();
  if (!sizes_ok(rows, dim)) return MUON_ERR_INVALID;
  if (!known(x_dtype) || !known(w_dtype)) return MUON_ERR_UNSUPPORTED;
  const size_t xs = dt_size(x_dtype), wsz = dt_size(w_dtype);
  if (rows > 0) {
    if (!dy || !total || !rstd || !dx || lddy < dim || ldt < dim || lddx < dim || (dtotal && lddt < dim))
      return MUON_ERR_INVALID;
    if (!is_aligned(dy, xs) || !is_aligned(total, xs) || !is_aligned(dx, xs) || !is_aligned(dtotal, xs) || !is_aligned(rstd, 4))
      return MUON_ERR_INVALID;
  }
  if (!is_aligned(weight, wsz) || !is_aligned(dweight, wsz)) return MUON_ERR_INVALID;
  if (rows == 0 && !dweight) return MUON_OK;
  if (dweight && (!ws || !is_aligned(ws, 256) || ws_bytes < muon_rmsnorm_workspace_size(rows, dim)))
    return MUON_ERR_WORKSPACE;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const RmsBwd p{dy, total, weight, dtotal, rstd, dx, dweight ? static_cast<float*>(ws) : nullptr, lddy, ldt, lddt, lddx,
                 rows, (int)dim, w_dtype == MUON_DTYPE_BF16};
  const bool vec = dim * xs % 16 == 0 && vec_rows(total, ldt, rows, xs) && vec_rows(dy, lddy, rows, xs) &&
                   vec_rows(dx, lddx, rows, xs) && (!dtotal || vec_rows(dtotal, lddt, rows, xs)) && is_aligned(weight, 16);
  int lines = 0;
  if ((x_dtype == MUON_DTYPE_BF16 ? backward<bf16>(p, vec, &lines, s) : backward<float>(p, vec, &lines, s)) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (dweight) {
    count_launch();
    if (launch_after(rms_columns_kernel, dim3(cdiv(dim, 32)), dim3(32, 32), 0, s, p.part, lines, (int)dim, dweight,
                     p.w_bf16) != cudaSuccess)
      return MUON_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
