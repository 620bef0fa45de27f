// AdamW with both moments held in 8 bits (block-wise scales, stochastic rounding).
//
// A moment's code is the top of its fp32 bit pattern, counted from a base the block
// shares: value = float_bits((code + base) << 20), so encoding is an integer add of
// the random bits, a shift and a subtraction, and decoding an add and a shift.  The
// update itself is adamw.cu's:
//   m <- b1*m + (1-b1)*g;  v <- b2*v + (1-b2)*g^2;
//   p <- p - lr*( (m/(1-b1^t)) / (sqrt(v/(1-b2^t)) + eps) + wd*p ).
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
  float lr, beta1, beta2, eps, wd;
  float omb1, omb2;    // 1 - beta1, 1 - beta2, formed in double precision on the host
  float inv_bc1;       // 1 / (1 - beta1^t)
  float inv_sqrt_bc2;  // 1 / sqrt(1 - beta2^t)
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

// Bandwidth-bound: 10 bytes an element for bf16 parameters and gradients (2+2 P, 2 G, 1+1
// a moment's codes twice).  A thread owns 16 consecutive elements, so that every array is
// read and written in whole 16- or 32-byte vectors; 8 threads make a block of 128, whose
// two maxima take three shuffles each, and no value passes through shared memory.
constexpr int A8_THREADS = 256;
constexpr int A8_EACH = 16;
constexpr int A8_CHUNK = A8_THREADS * A8_EACH;

// 16 elements as loaded, converted later, so that all of a thread's loads are in flight.
template <typename T> struct Raw16 { uint32_t w[4 * sizeof(T)]; };
template <typename T>
__device__ __forceinline__ void ld16(const T* p, Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) ld_v8(reinterpret_cast<const uint8_t*>(p) + 32 * i, r.w + 8 * i);
}
template <typename T>
__device__ __forceinline__ void ld16_some(const T* p, int n, Raw16<T>& r) {
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    if (sizeof(T) == 4) {
      r.w[i] = i < n ? reinterpret_cast<const uint32_t*>(p)[i] : 0u;
    } else {
      const uint32_t h = i < n ? reinterpret_cast<const uint16_t*>(p)[i] : 0u;
      r.w[i / 2] = i & 1 ? r.w[i / 2] | (h << 16) : h;
    }
  }
}
template <typename T>
__device__ __forceinline__ float get16(const Raw16<T>& r, int i) {
  if (sizeof(T) == 4) return __uint_as_float(r.w[i]);
  return __uint_as_float(i & 1 ? r.w[i / 2] & 0xFFFF0000u : r.w[i / 2] << 16);
}
template <typename T>
__device__ __forceinline__ void st16(T* p, const float (&v)[A8_EACH]) {
  uint32_t w[4 * sizeof(T)];
#pragma unroll
  for (int i = 0; i < (int)(4 * sizeof(T)); ++i)
    w[i] = sizeof(T) == 4 ? __float_as_uint(v[i % A8_EACH]) : pack_bf16x2(v[(2 * i) % A8_EACH], v[(2 * i + 1) % A8_EACH]);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) st_v8(reinterpret_cast<uint8_t*>(p) + 32 * i, w + 8 * i);
}

// Square root and quotient of the update: the hardware's approximations (2 ulp at most);
// what they feed is lr times a number near 1, added to a parameter of 24 or 8 bits.
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t max_of_8(uint32_t x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

template <typename PT, typename GT>
__global__ void __launch_bounds__(A8_THREADS) adamw8_kernel(const __grid_constant__ Adamw8Params q) {
  int lo = 0, hi = q.n - 1;
  const int b = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (q.e[mid].block_begin <= b) lo = mid; else hi = mid - 1;
  }
  const Adamw8Entry& e = q.e[lo];
  const long long i0 = (long long)(b - e.block_begin) * A8_CHUNK + threadIdx.x * A8_EACH;
  const long long blk = i0 / A8_BLOCK;
  // past the last block of codes: nothing to do, but the shuffles below need the thread
  const bool codes = i0 < (e.numel + A8_BLOCK - 1) / A8_BLOCK * A8_BLOCK;
  const int n = (int)min(max(e.numel - i0, 0LL), (long long)A8_EACH);
  PT* P = reinterpret_cast<PT*>(e.P) + i0;
  const GT* G = reinterpret_cast<const GT*>(e.G) + i0;
  const bool whole = n == A8_EACH && e.vec;
  Raw16<PT> pr;
  Raw16<GT> gr;
  uint4 mc = make_uint4(0, 0, 0, 0), vc = mc;
  int ms = 0, vs = 0;
  if (codes) {
    mc = *reinterpret_cast<const uint4*>(e.m + i0);
    vc = *reinterpret_cast<const uint4*>(e.v + i0);
    ms = e.ms[blk];
    vs = e.vs[blk];
  }
  if (whole) {
    ld16(P, pr);
    ld16(G, gr);
  } else {
    ld16_some(P, n, pr);
    ld16_some(G, n, gr);
  }
  float m[A8_EACH], v[A8_EACH], p[A8_EACH];
  uint32_t mtop = 0, vtop = 0;
  {
    const uint32_t bm = base_m(ms), bv = base_v(vs);
    const uint32_t mw[4] = {mc.x, mc.y, mc.z, mc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
#pragma unroll
    for (int i = 0; i < A8_EACH; ++i) {
      const float g = get16(gr, i);
      m[i] = q.beta1 * decode_m((mw[i / 4] >> (8 * (i % 4))) & 255u, bm) + q.omb1 * g;
      v[i] = q.beta2 * decode_v((vw[i / 4] >> (8 * (i % 4))) & 255u, bv) + q.omb2 * g * g;
      p[i] = get16(pr, i);
      p[i] -= q.lr * (__fdividef(m[i] * q.inv_bc1, sqrt_approx(v[i]) * q.inv_sqrt_bc2 + q.eps) + q.wd * p[i]);
      // codes past the end stay 0; a NaN is kept in m; infinite squares hold the largest code
      if (i >= n) m[i] = v[i] = 0.f;
      v[i] = v[i] != v[i] ? 0.f : fminf(v[i], FLT_MAX);
      const uint32_t a = __float_as_uint(m[i]) & 0x7FFFFFFFu;
      mtop = max(mtop, a < 0x7F800000u ? a : 0u);
      vtop = max(vtop, __float_as_uint(v[i]));
    }
  }
  if (whole) {
    st16(P, p);
  } else {
#pragma unroll
    for (int i = 0; i < A8_EACH; ++i)
      if (i < n) st1(P + i, p[i]);
  }
  ms = scale_of(max_of_8(mtop));
  vs = scale_of(max_of_8(vtop));
  if (!codes) return;
  const uint32_t bm = base_m(ms), bv = base_v(vs);
  const unsigned long long at = (unsigned long long)(e.first + i0);
  const uint32_t key = mix32(q.key + (uint32_t)(at >> 32));
  uint32_t mw[4] = {}, vw[4] = {};
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    const uint32_t r = mix32(((uint32_t)at + i) ^ key);
    mw[i / 4] |= encode_m(m[i], bm, r & 0xFFFFu) << (8 * (i % 4));
    vw[i / 4] |= encode_v(v[i], bv, r >> 16) << (8 * (i % 4));
  }
  *reinterpret_cast<uint4*>(e.m + i0) = make_uint4(mw[0], mw[1], mw[2], mw[3]);
  *reinterpret_cast<uint4*>(e.v + i0) = make_uint4(vw[0], vw[1], vw[2], vw[3]);
  if ((threadIdx.x & 7) == 0) {
    e.ms[blk] = (uint8_t)ms;
    e.vs[blk] = (uint8_t)vs;
  }
}

// 16 codes of one moment per thread: 16 bytes in, 32 out.
template <bool kFirst>
__device__ __forceinline__ void unpack16(const uint8_t* c, const uint8_t* s, bf16* out, long long i0) {
  const uint4 w4 = *reinterpret_cast<const uint4*>(c + i0);
  const int sc = s[i0 / A8_BLOCK];
  const uint32_t base = kFirst ? base_m(sc) : base_v(sc);
  const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
  float v[A8_EACH];
#pragma unroll
  for (int i = 0; i < A8_EACH; ++i) {
    const uint32_t k = (w[i / 4] >> (8 * (i % 4))) & 255u;
    v[i] = kFirst ? decode_m(k, base) : decode_v(k, base);
  }
  st16(out + i0, v);
}
__global__ void __launch_bounds__(256) adamw8_unpack_kernel(const uint8_t* m, const uint8_t* ms, const uint8_t* v,
                                                            const uint8_t* vs, long long numel, bf16* mo, bf16* vo) {
  const long long i0 = ((long long)blockIdx.x * 256 + threadIdx.x) * A8_EACH;
  if (i0 >= numel) return;
  if (m) unpack16<true>(m, ms, mo, i0);
  if (v) unpack16<false>(v, vs, vo, i0);
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
    q.lr = lr;
    q.beta1 = (float)beta1;
    q.beta2 = (float)beta2;
    q.omb1 = (float)(1.0 - beta1);
    q.omb2 = (float)(1.0 - beta2);
    q.eps = eps;
    q.wd = weight_decay;
    q.inv_bc1 = (float)(1.0 / bc1);
    q.inv_sqrt_bc2 = (float)(1.0 / std::sqrt(bc2));
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
  const long long blocks = (numel / A8_EACH + 255) / 256;
  if (blocks >= (1LL << 31)) return MUON_ERR_UNSUPPORTED;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  adamw8_unpack_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      m, m_scale, v, v_scale, numel, static_cast<bf16*>(m_out), static_cast<bf16*>(v_out));
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
