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

// One block of 128 elements per CTA, one element per thread.
template <typename PT, typename GT>
__global__ void __launch_bounds__(A8_BLOCK) adamw8_kernel(const __grid_constant__ Adamw8Params q) {
  __shared__ uint32_t top[2];
  int lo = 0, hi = q.n - 1;
  const int b = blockIdx.x;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (q.e[mid].block_begin <= b) lo = mid; else hi = mid - 1;
  }
  const Adamw8Entry& e = q.e[lo];
  const long long blk = b - e.block_begin;
  const long long i = blk * A8_BLOCK + threadIdx.x;
  if (threadIdx.x < 2) top[threadIdx.x] = 0;
  __syncthreads();
  const bool in = i < e.numel;
  float m = 0.f, v = 0.f;
  if (in) {
    const float g = ld1(reinterpret_cast<const GT*>(e.G) + i);
    m = q.beta1 * decode_m(e.m[i], base_m(e.ms[blk])) + q.omb1 * g;
    v = q.beta2 * decode_v(e.v[i], base_v(e.vs[blk])) + q.omb2 * g * g;
    PT* P = reinterpret_cast<PT*>(e.P) + i;
    const float p = ld1(P);
    st1(P, p - q.lr * ((m * q.inv_bc1) / (sqrtf(v) * q.inv_sqrt_bc2 + q.eps) + q.wd * p));
    if (v != v) v = 0.f;   // the NaN is kept in m
    v = fminf(v, FLT_MAX);
    const uint32_t a = __float_as_uint(m) & 0x7FFFFFFFu;
    if (a < 0x7F800000u) atomicMax(&top[0], a);
    atomicMax(&top[1], __float_as_uint(v));
  }
  __syncthreads();
  const int sm = scale_of(top[0]), sv = scale_of(top[1]);
  const unsigned long long at = (unsigned long long)(e.first + i);
  const uint32_t r = mix32((uint32_t)at ^ mix32(q.key + (uint32_t)(at >> 32)));
  e.m[i] = (uint8_t)encode_m(m, base_m(sm), r & 0xFFFFu);
  e.v[i] = (uint8_t)encode_v(v, base_v(sv), r >> 16);
  if (threadIdx.x == 0) {
    e.ms[blk] = (uint8_t)sm;
    e.vs[blk] = (uint8_t)sv;
  }
}

__global__ void __launch_bounds__(256) adamw8_unpack_kernel(const uint8_t* m, const uint8_t* ms, const uint8_t* v,
                                                            const uint8_t* vs, long long numel, bf16* mo, bf16* vo) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
  if (i >= numel) return;
  if (m) mo[i] = __float2bfloat16_rn(decode_m(m[i], base_m(ms[i / A8_BLOCK])));
  if (v) vo[i] = __float2bfloat16_rn(decode_v(v[i], base_v(vs[i / A8_BLOCK])));
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
    if (a.numel / A8_BLOCK >= (1LL << 30)) return MUON_ERR_UNSUPPORTED;
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
      const long long nb = (a.numel + A8_BLOCK - 1) / A8_BLOCK;
      if (blocks + nb >= (1LL << 31)) {
        if (j == 0) return MUON_ERR_UNSUPPORTED;
        break;
      }
      q.e[j++] = Adamw8Entry{a.P, a.G, a.m, a.v, a.m_scale, a.v_scale, (long long)a.numel, (long long)a.first,
                             (int)blocks, 0};
      blocks += nb;
    }
    q.n = j;
    if (j == 0) continue;
    const bool pb = p_dt == MUON_DTYPE_BF16, gb = g_dt == MUON_DTYPE_BF16;
    if (pb && gb) adamw8_kernel<bf16, bf16><<<(unsigned)blocks, A8_BLOCK, 0, s>>>(q);
    else if (pb) adamw8_kernel<bf16, float><<<(unsigned)blocks, A8_BLOCK, 0, s>>>(q);
    else if (gb) adamw8_kernel<float, bf16><<<(unsigned)blocks, A8_BLOCK, 0, s>>>(q);
    else adamw8_kernel<float, float><<<(unsigned)blocks, A8_BLOCK, 0, s>>>(q);
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
  const long long blocks = (numel + 255) / 256;
  if (blocks >= (1LL << 31)) return MUON_ERR_UNSUPPORTED;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  adamw8_unpack_kernel<<<(unsigned)blocks, 256, 0, static_cast<cudaStream_t>(stream)>>>(
      m, m_scale, v, v_scale, numel, static_cast<bf16*>(m_out), static_cast<bf16*>(v_out));
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
