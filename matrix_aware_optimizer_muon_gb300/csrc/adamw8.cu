// AdamW with both moments held in 8 bits (block-wise scales, stochastic rounding).
//
// A moment's code is the top of its fp32 bit pattern, counted from a base the block
// shares: value = float_bits((code + base) << 20), so encoding is an integer add of
// the random bits, a shift and a subtraction, and decoding an add and a shift.  The
// update itself is adamw.cu's:
//   m <- b1*m + (1-b1)*g;  v <- b2*v + (1-b2)*g^2;
//   p <- p - lr*( (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps) + wd*p ).
//
// Measured: 335.5 M bf16 parameters and gradients, step 575 us (5.9 TB/s, 86% of a copy's
// rate; three quarters of the issue slots) and unpacking 289 us (7.0 TB/s); 38.6 M fp32
// parameters with bf16 gradients 88 us (6.2 TB/s) and 37 us.  A warp with a code 0 or a
// number below its block's least takes the plain functions: 654 us where 3e-4 of the first
// moments are 0 (gradients that change sign), 1010 us where all are (rows no token touched).
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace {

constexpr int A8_MAX_PARAMS = 256;
constexpr int A8_BLOCK = MUON_ADAMW8_BLOCK;

struct Adamw8Entry {
  void* P;
  const void* G;
  uint8_t *m, *v, *ms, *vs;
  long long numel;
  long long first;
  int block_begin;
  int vec;
};
struct Adamw8Params {
  Adamw8Entry e[A8_MAX_PARAMS];
  int n;
  uint32_t key;        // from (seed, t)
  // each number twice, as the operand of a paired instruction
  f32x2 neg_lr, beta1, beta2, eps, wd;
  f32x2 omb1, omb2;    // 1 - beta1, 1 - beta2, formed in double precision on the host
  f32x2 inv_bc1;       // 1 / (1 - beta1^t)
  f32x2 root;          // 2^-12 / sqrt(1 - beta2^t)
};
static_assert(sizeof(Adamw8Params) < 32000, "Adamw8Params too large");

// 32 random bits: two rounds of xor-shift and multiplication by an odd constant
// (the fractions of the golden ratio and of sqrt 2).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x ^= x >> 16;
  x *= 0x9E3779B9u;
  x ^= x >> 15;
  x *= 0x6A09E667u;
  return x ^ (x >> 16);
}

__device__ __forceinline__ int scale_of(uint32_t top_bits) { return min((int)((top_bits >> 20) + 9) >> 3, 255); }
__device__ __forceinline__ uint32_t base_m(int s) { return 8u * (uint32_t)max(s - 16, 0); }
__device__ __forceinline__ uint32_t base_v(int s) { return 8u * (uint32_t)max(s - 32, 0); }

__device__ __forceinline__ float decode_m(uint32_t c, uint32_t base) {
  const uint32_t k = c & 127u;
  if (k == 0) return c ? __uint_as_float(0x7FC00000u) : 0.f;
  return __uint_as_float(((k + base) << 20) | ((c & 128u) << 24));
}
__device__ __forceinline__ float decode_v(uint32_t c, uint32_t base) {
  return c ? __uint_as_float((c + base) << 20) : 0.f;
}

// r: 16 random bits.  Adding r (and half of its last place) below the kept bits and
// dropping them rounds up with a probability equal to the remainder.
__device__ __forceinline__ uint32_t encode_m(float m, uint32_t base, uint32_t r) {
  const uint32_t a = __float_as_uint(m) & 0x7FFFFFFFu;
  if (a >= 0x7F800000u) return 128u;
  uint32_t k;
  if (a < ((base + 1) << 20)) k = (((float)r + 0.5f) * 0x1p-16f) * __uint_as_float((base + 1) << 20) < __uint_as_float(a);
  else k = min(((a + (r << 4) + 8u) >> 20) - base, 127u);
  return k | ((m < 0.f && k) ? 128u : 0u);
}
__device__ __forceinline__ uint32_t encode_v(float v, uint32_t base, uint32_t r) {
  const uint32_t a = __float_as_uint(v);
  const int k = (int)((a + (r << 4) + 8u) >> 20) - (int)base;
  return (uint32_t)min(max(k, a ? 1 : 0), 255);
}

// 10 bytes an element for bf16 parameters and gradients (2+2 P, 2 G, 1+1 a moment's codes
// twice): at HBM's rate an SM has 54 issue slots and 27 of the integer pipe an element,
// and the coding is integer work, so instructions count.  A thread owns 16 consecutive
// elements: whole 16- and 32-byte vectors, 8 threads a block of 128 (a maximum takes three
// shuffles), no shared memory.  The common case is coded without selects:
//   decoding   byte * 2^20 + base (a multiply-add), the sign as a factor +-1;
//   encoding   |m| * 16 + random * 256 - base * 2^24 leaves the code in the top byte,
//              which byte permutes collect;
// zero codes, numbers below a block's least, NaN and Inf are found by a test per thread and
// sent through the plain functions above.
constexpr int A8_THREADS = 128;
constexpr int A8_EACH = 16;
constexpr int A8_WORDS = A8_EACH / 4;      // of a moment's codes
constexpr int A8_CHUNK = A8_THREADS * A8_EACH;

// 16 elements as loaded, converted later, so that all of a thread's loads are in flight.
template <int kWords>
__device__ __forceinline__ void load_words(const void* p, uint32_t* w) {
  if constexpr (kWords == 4) {
    const uint4 q = *static_cast<const uint4*>(p);
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i) ld_v8(static_cast<const uint8_t*>(p) + 32 * i, w + 8 * i);
  }
}
template <int kWords>
__device__ __forceinline__ void store_words(void* p, const uint32_t* w) {
  if constexpr (kWords == 4) {
    *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kWords / 8; ++i) st_v8(static_cast<uint8_t*>(p) + 32 * i, w + 8 * i);
  }
}
template <typename T> struct RawN { uint32_t w[A8_EACH * sizeof(T) / 4]; };
template <typename T>
__device__ __forceinline__ void ld_all(const T* p, RawN<T>& r) {
  load_words<A8_EACH * sizeof(T) / 4>(p, r.w);
}
template <typename T>
__device__ __forceinline__ void ld_some(const T* p, int n, RawN<T>& r) {
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    if constexpr (sizeof(T) == 4) {
      r.w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    } else {
      const uint32_t h = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
      r.w[i / 2] = i & 1 ? r.w[i / 2] | (h << 16) : h;
    }
  }
}
// elements 2j and 2j + 1
template <typename T>
__device__ __forceinline__ f32x2 get2(const RawN<T>& r, int j) {
  if constexpr (sizeof(T) == 4) return make2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
  else return cvt2(r.w[j]);
}
template <typename T>
__device__ __forceinline__ void st_all(T* p, const f32x2 (&v)[A8_EACH / 2]) {
  uint32_t w[A8_EACH * sizeof(T) / 4];
#pragma unroll
  for (int j = 0; j < A8_EACH / 2; ++j) {
    if constexpr (sizeof(T) == 4) {
      w[2 * j] = __float_as_uint(lo2(v[j]));
      w[2 * j + 1] = __float_as_uint(hi2(v[j]));
    } else {
      w[j] = pack_bf16x2(lo2(v[j]), hi2(v[j]));
    }
  }
  store_words<A8_EACH * sizeof(T) / 4>(p, w);
}

// Square root and reciprocal of the update: the hardware's approximations (2 ulp at most);
// what they feed is lr times a number near 1, added to a parameter of 24 or 8 bits.  They
// flush what is below 2^-126, so the root is taken of 2^24 v; a thread that holds a v whose
// product with 2^24 could overflow (or that is NaN) asks for each element.
constexpr float A8_ROOT_SCALE = 0x1p24f, A8_ROOT_MAX = 0x1p103f;
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float root_any(float v) {   // 2^12 times the root
  return v > A8_ROOT_MAX ? 0x1p12f * sqrt_approx(v) : sqrt_approx(v * A8_ROOT_SCALE);
}
__device__ __forceinline__ f32x2 updated(const Adamw8Params& q, f32x2 p, f32x2 m, f32x2 root) {
  const f32x2 d = fma2(root, q.root, q.eps);
  const f32x2 u = mul2(mul2(m, q.inv_bc1), make2(rcp_approx(lo2(d)), rcp_approx(hi2(d))));
  return fma2(q.neg_lr, fma2(q.wd, p, u), p);
}

// Largest and smallest magnitude of three (a NaN makes the largest NaN).
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float min3_abs(float a, float b, float c) {
  float y;
  asm("min.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// over the threads of a block of codes
__device__ __forceinline__ uint32_t max_of_block(uint32_t x) {
#pragma unroll
  for (int o = A8_BLOCK / A8_EACH / 2; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}
// nonzero if a byte of w is zero
__device__ __forceinline__ uint32_t zero_byte(uint32_t w) { return (w - 0x01010101u) & ~w & 0x80808080u; }
__device__ __forceinline__ uint32_t byte_of(uint32_t w, int i) { return __byte_perm(w, 0, 0x4440 | i); }
// byte i of w as a code counted from base
__device__ __forceinline__ float code_bits(uint32_t w, int i, uint32_t base) {
  return __uint_as_float(byte_of(w, i) * 0x100000u + (base << 20));
}
// the top bytes of four words
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x0073), 0x5410);
}

// The uncommon cases, out of line so that they hold no registers of the common one.
struct CodesN {
  uint32_t m[A8_WORDS], v[A8_WORDS];
};
struct MomentsN {
  f32x2 m[A8_EACH / 2], v[A8_EACH / 2];
};
__device__ __noinline__ MomentsN decode_any(const CodesN c, uint32_t bm, uint32_t bv) {
  MomentsN o;
#pragma unroll
  for (int j = 0; j < A8_EACH / 2; ++j) {
    const int i = 2 * (j % 2);
    o.m[j] = make2(decode_m(byte_of(c.m[j / 2], i), bm), decode_m(byte_of(c.m[j / 2], i + 1), bm));
    o.v[j] = make2(decode_v(byte_of(c.v[j / 2], i), bv), decode_v(byte_of(c.v[j / 2], i + 1), bv));
  }
  return o;
}
__device__ __forceinline__ float element(const f32x2 (&a)[A8_EACH / 2], int i) {
  return i & 1 ? hi2(a[i / 2]) : lo2(a[i / 2]);
}
// NaN and Inf stay out of the block's scales: a NaN is kept in m, an infinite square holds
// the largest code.
__device__ __forceinline__ float held(float v) { return v != v ? 0.f : fminf(v, FLT_MAX); }
__device__ __noinline__ uint2 finite_tops(const MomentsN x) {
  uint2 t = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    const uint32_t a = __float_as_uint(element(x.m, i)) & 0x7FFFFFFFu;
    t.x = max(t.x, a < 0x7F800000u ? a : 0u);
    t.y = max(t.y, __float_as_uint(held(element(x.v, i))));
  }
  return t;
}
__device__ __noinline__ CodesN encode_any(const MomentsN x, uint32_t bm, uint32_t bv, uint32_t x0) {
  CodesN c = {};
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    uint32_t r = (x0 ^ i) * 0x9E3779B9u;
    r = (r ^ (r >> 15)) * 0x6A09E667u;
    r ^= r >> 16;
    c.m[i / 4] |= encode_m(element(x.m, i), bm, r & 0xFFFFu) << (8 * (i % 4));
    c.v[i / 4] |= encode_v(held(element(x.v, i)), bv, r >> 16) << (8 * (i % 4));
  }
  return c;
}

// CTAs an SM should hold, and so registers a thread.  Each CTA takes one chunk and leaves:
// its loads overlap the others' arithmetic.  Measured on 335 M bf16 elements (step and
// unpacking together): 32 warps an SM 883 us, 24 967, 16 1134; in CTAs of 128 threads
// instead of 256 868; loops over 2, 4 or 8 chunks 1035, 979, 945; a persistent kernel with
// the next chunk's data on their way to shared memory a fifth slower than one chunk a CTA.
constexpr int a8_ctas(int bytes) { return bytes == 4 ? 8 : 6; }
template <typename PT, typename GT>
__global__ void __launch_bounds__(A8_THREADS, a8_ctas(sizeof(PT) + sizeof(GT)))
    adamw8_kernel(const __grid_constant__ Adamw8Params q) {
  const int b = blockIdx.x;
  int lo = 0;
  if (q.n <= 4) {
#pragma unroll
    for (int i = 1; i < 4; ++i) lo += i < q.n && q.e[i].block_begin <= b;
  } else {
    int hi = q.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (q.e[mid].block_begin <= b) lo = mid; else hi = mid - 1;
    }
  }
  const Adamw8Entry& e = q.e[lo];
  // what the whole CTA shares is 64 bits wide, a thread's place in its chunk 32
  const long long c0 = (long long)(b - e.block_begin) * A8_CHUNK;
  const int left = (int)min(e.numel - c0, (long long)A8_CHUNK);
  const int off = threadIdx.x * A8_EACH;
  const int n = min(max(left - off, 0), A8_EACH);
  // past the last block of codes: nothing to do, but the shuffles below need the thread
  const bool codes = off < (left + A8_BLOCK - 1) / A8_BLOCK * A8_BLOCK;
  PT* P = reinterpret_cast<PT*>(e.P) + c0;
  const GT* G = reinterpret_cast<const GT*>(e.G) + c0;
  uint8_t *mp = e.m + c0, *vp = e.v + c0, *msp = e.ms + c0 / A8_BLOCK, *vsp = e.vs + c0 / A8_BLOCK;
  const bool whole = n == A8_EACH && e.vec;
  RawN<PT> pr;
  RawN<GT> gr;
  CodesN codes_n = {};
  uint32_t (&mw)[A8_WORDS] = codes_n.m, (&vw)[A8_WORDS] = codes_n.v;
  int ms = 0, vs = 0;
  if (codes) {
    load_words<A8_WORDS>(mp + off, mw);
    load_words<A8_WORDS>(vp + off, vw);
    ms = msp[off / A8_BLOCK];
    vs = vsp[off / A8_BLOCK];
  }
  if (whole) {
    ld_all(P + off, pr);
    ld_all(G + off, gr);
  } else {
    ld_some(P + off, n, pr);
    ld_some(G + off, n, gr);
  }
  MomentsN now;
  f32x2 (&m2)[A8_EACH / 2] = now.m, (&v2)[A8_EACH / 2] = now.v;
  {
    const uint32_t bm = base_m(ms), bv = base_v(vs);
    uint32_t zeros = 0;
#pragma unroll
    for (int k = 0; k < A8_WORDS; ++k) {
      const uint32_t mag = mw[k] & 0x7F7F7F7Fu, one = (mw[k] & 0x80808080u) | 0x3F3F3F3Fu;
      zeros |= zero_byte(mag) | zero_byte(vw[k]);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 2 * h;
        // +-1: top byte 0x3F or 0xBF, then 0x80
        m2[2 * k + h] = mul2(make2(code_bits(mag, i, bm), code_bits(mag, i + 1, bm)),
                             make2(__uint_as_float(__byte_perm(one, 0x80u, 0x0455 | (i << 12))),
                                   __uint_as_float(__byte_perm(one, 0x80u, 0x0455 | ((i + 1) << 12)))));
        v2[2 * k + h] = make2(code_bits(vw[k], i, bv), code_bits(vw[k], i + 1, bv));
      }
    }
    if (zeros) now = decode_any(codes_n, bm, bv);
  }
#pragma unroll
  for (int j = 0; j < A8_EACH / 2; ++j) {
    const f32x2 g = get2(gr, j);
    m2[j] = fma2(q.beta1, m2[j], mul2(q.omb1, g));
    v2[j] = fma2(q.beta2, v2[j], mul2(mul2(q.omb2, g), g));
  }
  if (!whole) {
#pragma unroll
    for (int i = 0; i < A8_EACH; ++i) {
      if (i >= n) {   // codes past the end stay 0
        m2[i / 2] = i & 1 ? make2(lo2(m2[i / 2]), 0.f) : make2(0.f, hi2(m2[i / 2]));
        v2[i / 2] = i & 1 ? make2(lo2(v2[i / 2]), 0.f) : make2(0.f, hi2(v2[i / 2]));
      }
    }
  }
  float mt = 0.f, vt = 0.f, mlow = INFINITY, vlow = INFINITY;
#pragma unroll
  for (int j = 0; j < A8_EACH / 2; ++j) {
    mt = max3_abs(mt, lo2(m2[j]), hi2(m2[j]));
    vt = max3_abs(vt, lo2(v2[j]), hi2(v2[j]));
    mlow = min3_abs(mlow, lo2(m2[j]), hi2(m2[j]));
    vlow = min3_abs(vlow, lo2(v2[j]), hi2(v2[j]));
  }
  f32x2 p[A8_EACH / 2];
  if (vt <= A8_ROOT_MAX) {
#pragma unroll
    for (int j = 0; j < A8_EACH / 2; ++j) {
      const f32x2 x = mul2(v2[j], both(A8_ROOT_SCALE));
      p[j] = updated(q, get2(pr, j), m2[j], make2(sqrt_approx(lo2(x)), sqrt_approx(hi2(x))));
    }
  } else {
#pragma unroll
    for (int j = 0; j < A8_EACH / 2; ++j)
      p[j] = updated(q, get2(pr, j), m2[j], make2(root_any(lo2(v2[j])), root_any(hi2(v2[j]))));
  }
  if (whole) {
    st_all(P + off, p);
  } else {
#pragma unroll
    for (int i = 0; i < A8_EACH; ++i)
      if (i < n) st1(P + off + i, element(p, i));
  }
  uint32_t mtop = __float_as_uint(mt), vtop = __float_as_uint(vt);
  const bool odd = max(mtop, vtop) >= 0x7F800000u;
  if (odd) {
    const uint2 t = finite_tops(now);
    mtop = t.x;
    vtop = t.y;
  }
  ms = scale_of(max_of_block(mtop));
  vs = scale_of(max_of_block(vtop));
  if (!codes) return;
  const uint32_t bm = base_m(ms), bv = base_v(vs);
  const unsigned long long at = (unsigned long long)(e.first + c0);
  // mix32 of (at + i) ^ key: i is in the lowest bits, so its first xor-shift is shared
  uint32_t key = mix32(q.key + (uint32_t)(at >> 32));
  const uint32_t low = (uint32_t)at + off;
  if (low < (uint32_t)at) key = mix32(q.key + (uint32_t)(at >> 32) + 1u);
  uint32_t x0 = low ^ key;
  x0 ^= x0 >> 16;
  // a block at the end of fp32's range is the one whose codes can pass the top
  if (odd || __float_as_uint(mlow) < ((bm + 1) << 20) || __float_as_uint(vlow) < ((bv + 1) << 20) || ms == 255 || vs == 255) {
    codes_n = encode_any(now, bm, bv, x0);
  } else {
    const uint32_t km = 128u - (bm << 24), kv = 128u - (bv << 24);   // half of the random bits' last place
#pragma unroll
    for (int k = 0; k < A8_WORDS; ++k) {
      uint32_t a[4], c[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t x = (x0 ^ (4 * k + i)) * 0x9E3779B9u;
        x = (x ^ (x >> 15)) * 0x6A09E667u;
        const uint32_t up = x >> 16, down = (x ^ up) & 0xFFFFu;
        a[i] = __float_as_uint(element(m2, 4 * k + i)) * 16u + (down * 256u + km);   // the sign is shifted out
        c[i] = __float_as_uint(element(v2, 4 * k + i)) * 16u + (up * 256u + kv);
      }
      const uint32_t sgn = top_bytes(__float_as_uint(lo2(m2[2 * k])), __float_as_uint(hi2(m2[2 * k])),
                                     __float_as_uint(lo2(m2[2 * k + 1])), __float_as_uint(hi2(m2[2 * k + 1])));
      mw[k] = top_bytes(a[0], a[1], a[2], a[3]) | (sgn & 0x80808080u);
      vw[k] = top_bytes(c[0], c[1], c[2], c[3]);
    }
  }
  store_words<A8_WORDS>(mp + off, mw);
  store_words<A8_WORDS>(vp + off, vw);
  if (threadIdx.x % (A8_BLOCK / A8_EACH) == 0) {
    msp[off / A8_BLOCK] = (uint8_t)ms;
    vsp[off / A8_BLOCK] = (uint8_t)vs;
  }
}

// 16 codes of one moment per thread: 16 bytes in, 32 out.  The values are the top halves of
// their fp32 bits.
template <bool kFirst>
__device__ __forceinline__ void unpack16(const uint4 w4, int sc, bf16* out) {
  const uint32_t base = kFirst ? base_m(sc) : base_v(sc);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  uint32_t o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t c = byte_of(w[j / 2], 2 * (j % 2)), d = byte_of(w[j / 2], 2 * (j % 2) + 1);
    o[j] = __byte_perm(__float_as_uint(kFirst ? decode_m(c, base) : decode_v(c, base)),
                       __float_as_uint(kFirst ? decode_m(d, base) : decode_v(d, base)), 0x7632);
  }
  st_v8(out, o);
}
__global__ void __launch_bounds__(256) adamw8_unpack_kernel(const uint8_t* m, const uint8_t* ms, const uint8_t* v,
                                                            const uint8_t* vs, long long numel, bf16* mo, bf16* vo) {
  const long long i0 = ((long long)blockIdx.x * 256 + threadIdx.x) * 16;
  if (i0 >= numel) return;
  uint4 mc = {}, vc = {};
  int sm = 0, sv = 0;
  if (m) { mc = *reinterpret_cast<const uint4*>(m + i0); sm = ms[i0 / A8_BLOCK]; }
  if (v) { vc = *reinterpret_cast<const uint4*>(v + i0); sv = vs[i0 / A8_BLOCK]; }
  if (m) unpack16<true>(mc, sm, mo + i0);
  if (v) unpack16<false>(vc, sv, vo + i0);
}

f32x2 twice(float x) {
  uint32_t w;
  std::memcpy(&w, &x, 4);
  return f32x2{(uint64_t)w << 32 | w};
}
bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" int muon_adamw8_step(const muon_adamw8_param* params, int n, int64_t t, float lr, double beta1,
                                double beta2, float eps, float weight_decay, uint32_t seed, muon_stream_t stream) {
  begin_launches();
  if (n < 0 || t < 1) return MUON_ERR_INVALID;
  if (n == 0) return MUON_OK;
  if (!params) return MUON_ERR_INVALID;
  if (!(beta1 >= 0.0 && beta1 < 1.0 && beta2 >= 0.0 && beta2 < 1.0 && eps >= 0.f)) return MUON_ERR_INVALID;
  const int p_dt = params[0].p_dtype, g_dt = params[0].g_dtype;
  for (int i = 0; i < n; ++i) {
    const muon_adamw8_param& a = params[i];
    if (a.numel < 0 || a.first < 0 || a.first % A8_BLOCK) return MUON_ERR_INVALID;
    if (a.p_dtype != p_dt || a.g_dtype != g_dt) return MUON_ERR_UNSUPPORTED;
    if ((p_dt != MUON_DTYPE_F32 && p_dt != MUON_DTYPE_BF16) || (g_dt != MUON_DTYPE_F32 && g_dt != MUON_DTYPE_BF16))
      return MUON_ERR_UNSUPPORTED;
    if (a.numel == 0) continue;
    if (!a.P || !a.G || !a.m || !a.v || !a.m_scale || !a.v_scale) return MUON_ERR_INVALID;
    if (!is_aligned(a.P, dt_size(p_dt)) || !is_aligned(a.G, dt_size(g_dt)) || !is_aligned(a.m, 16) ||
        !is_aligned(a.v, 16))
      return MUON_ERR_INVALID;
    if (a.numel / A8_CHUNK >= (1LL << 30)) return MUON_ERR_UNSUPPORTED;
  }
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local Adamw8Params q;
  const double bc1 = 1.0 - std::pow(beta1, (double)t);
  const double bc2 = 1.0 - std::pow(beta2, (double)t);
  int i = 0;
  while (i < n) {
    q.key = mix32(seed ^ mix32((uint32_t)t));
    q.neg_lr = twice(-lr);
    q.beta1 = twice((float)beta1);
    q.beta2 = twice((float)beta2);
    q.omb1 = twice((float)(1.0 - beta1));
    q.omb2 = twice((float)(1.0 - beta2));
    q.eps = twice(eps);
    q.wd = twice(weight_decay);
    q.inv_bc1 = twice((float)(1.0 / bc1));
    q.root = twice((float)(0x1p-12 / std::sqrt(bc2)));
    int j = 0;
    long long blocks = 0;
    for (; i < n && j < A8_MAX_PARAMS; ++i) {
      const muon_adamw8_param& a = params[i];
      if (a.numel == 0) continue;
      const long long nb = (a.numel + A8_CHUNK - 1) / A8_CHUNK;
      if (blocks + nb >= (1LL << 31)) {
        if (j == 0) return MUON_ERR_UNSUPPORTED;
        break;
      }
      q.e[j++] = Adamw8Entry{a.P, a.G, a.m, a.v, a.m_scale, a.v_scale, (long long)a.numel, (long long)a.first,
                             (int)blocks, is_aligned(a.P, 32) && is_aligned(a.G, 32)};
      blocks += nb;
    }
    q.n = j;
    if (j == 0) continue;
    const bool pb = p_dt == MUON_DTYPE_BF16, gb = g_dt == MUON_DTYPE_BF16;
    if (pb && gb) adamw8_kernel<bf16, bf16><<<(unsigned)blocks, A8_THREADS, 0, s>>>(q);
    else if (pb) adamw8_kernel<bf16, float><<<(unsigned)blocks, A8_THREADS, 0, s>>>(q);
    else if (gb) adamw8_kernel<float, bf16><<<(unsigned)blocks, A8_THREADS, 0, s>>>(q);
    else adamw8_kernel<float, float><<<(unsigned)blocks, A8_THREADS, 0, s>>>(q);
    if (cudaGetLastError() != cudaSuccess) return MUON_ERR_CUDA;
    count_launch();
  }
  return MUON_OK;
}

extern "C" int muon_adamw8_unpack(const uint8_t* m, const uint8_t* m_scale, const uint8_t* v, const uint8_t* v_scale,
                                  int64_t numel, void* m_out, void* v_out, muon_stream_t stream) {
  begin_launches();
  if (numel < 0 || numel % A8_BLOCK) return MUON_ERR_INVALID;
  if ((m != nullptr) != (m_out != nullptr) || (v != nullptr) != (v_out != nullptr)) return MUON_ERR_INVALID;
  if ((m && !m_scale) || (v && !v_scale)) return MUON_ERR_INVALID;
  if (!is_aligned(m, 16) || !is_aligned(v, 16) || !is_aligned(m_out, 32) || !is_aligned(v_out, 32))
    return MUON_ERR_INVALID;
  if (numel == 0 || (!m && !v)) return MUON_OK;
  const long long blocks = (numel / 16 + 255) / 256;
  if (blocks >= (1LL << 31)) return MUON_ERR_UNSUPPORTED;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  adamw8_unpack_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      m, m_scale, v, v_scale, numel, static_cast<bf16*>(m_out), static_cast<bf16*>(v_out));
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
