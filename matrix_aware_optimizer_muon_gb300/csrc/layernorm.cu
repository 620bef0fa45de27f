// Layer norm, forward and backward, with the reduction of the weight's and bias's
// gradients:
//   y  = (x - mean) rstd w + b,          rstd = 1/sqrt(var + eps)
//   dx = rstd (g - sum(g)/D - xh sum(g xh)/D),   g = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,   db = sum_rows dy
// Every sum is fp32.
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace {

constexpr int LN_THREADS = 256;

template <typename T, typename WT>
__global__ void __launch_bounds__(LN_THREADS) ln_forward_kernel(const T* x, long long ldx, const WT* w, const WT* b,
                                                                int dim, float eps, T* y, long long ldy, float* mean,
                                                                float* rstd) {
  __shared__ float red[32];
  const long long r = blockIdx.x;
  const T* xr = x + r * ldx;
  T* yr = y + r * ldy;
  float s = 0.f;
  for (int c = threadIdx.x; c < dim; c += LN_THREADS) s += ld1(xr + c);
  const float mu = block_sum(s, red) / (float)dim;
  float q = 0.f;
  for (int c = threadIdx.x; c < dim; c += LN_THREADS) {
    const float d = ld1(xr + c) - mu;
    q += d * d;
  }
  const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)dim + eps);
  for (int c = threadIdx.x; c < dim; c += LN_THREADS) {
    const float xh = (ld1(xr + c) - mu) * rs;
    st1(yr + c, (w ? xh * ld1(w + c) : xh) + (b ? ld1(b + c) : 0.f));
  }
  if (threadIdx.x == 0) {
    if (mean) mean[r] = mu;
    if (rstd) rstd[r] = rs;
  }
}

template <typename T, typename WT>
__global__ void __launch_bounds__(LN_THREADS) ln_backward_kernel(const T* dy, long long lddy, const T* x, long long ldx,
                                                                 const WT* w, const float* mean, const float* rstd,
                                                                 int dim, T* dx, long long lddx) {
  __shared__ float red[32];
  const long long r = blockIdx.x;
  const float mu = mean[r], rs = rstd[r];
  const T* xr = x + r * ldx;
  const T* dyr = dy + r * lddy;
  T* dxr = dx + r * lddx;
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < dim; c += LN_THREADS) {
    const float g = ld1(dyr + c) * (w ? ld1(w + c) : 1.f);
    s1 += g;
    s2 += g * ((ld1(xr + c) - mu) * rs);
  }
  const float c1 = block_sum(s1, red) / (float)dim;
  const float c2 = block_sum(s2, red) / (float)dim;
  for (int c = threadIdx.x; c < dim; c += LN_THREADS) {
    const float g = ld1(dyr + c) * (w ? ld1(w + c) : 1.f);
    st1(dxr + c, rs * (g - c1 - (ld1(xr + c) - mu) * rs * c2));
  }
}

// Column sums over a slab of rows; part: [slabs][2][dim].
constexpr int LN_SLABS = 152;
template <typename T>
__global__ void __launch_bounds__(LN_THREADS) ln_slab_kernel(const T* dy, long long lddy, const T* x, long long ldx,
                                                             const float* mean, const float* rstd, long long rows,
                                                             int dim, float* part) {
  const int c = blockIdx.x * LN_THREADS + threadIdx.x;
  if (c >= dim) return;
  float sw = 0.f, sb = 0.f;
  for (long long r = blockIdx.y; r < rows; r += gridDim.y) {
    const float g = ld1(dy + r * lddy + c);
    sw += g * ((ld1(x + r * ldx + c) - mean[r]) * rstd[r]);
    sb += g;
  }
  part[(size_t)blockIdx.y * 2 * dim + c] = sw;
  part[(size_t)blockIdx.y * 2 * dim + dim + c] = sb;
}

template <typename WT>
__global__ void __launch_bounds__(LN_THREADS) ln_columns_kernel(const float* part, int slabs, int dim, WT* dw, WT* db) {
  const int c = blockIdx.x * LN_THREADS + threadIdx.x;
  if (c >= dim) return;
  float sw = 0.f, sb = 0.f;
  for (int i = 0; i < slabs; ++i) {
    sw += part[(size_t)i * 2 * dim + c];
    sb += part[(size_t)i * 2 * dim + dim + c];
  }
  if (dw) st1(dw + c, sw);
  if (db) st1(db + c, sb);
}

bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
bool known(int dt) { return dt == MUON_DTYPE_F32 || dt == MUON_DTYPE_BF16; }
bool sizes_ok(int64_t rows, int64_t dim) { return rows >= 0 && rows < (1LL << 31) && dim >= 1 && dim < (1LL << 31); }

// f(T*, WT*) for the dtype pair
template <class F>
void by_types(int x_dt, int w_dt, F f) {
  if (x_dt == MUON_DTYPE_BF16) {
    if (w_dt == MUON_DTYPE_BF16) f((bf16*)nullptr, (bf16*)nullptr);
    else f((bf16*)nullptr, (float*)nullptr);
  } else {
    if (w_dt == MUON_DTYPE_BF16) f((float*)nullptr, (bf16*)nullptr);
    else f((float*)nullptr, (float*)nullptr);
  }
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" int muon_layernorm_forward(const void* x, int64_t ldx, const void* weight, const void* bias, int64_t rows,
                                      int64_t dim, int x_dtype, int w_dtype, float eps, void* y, int64_t ldy,
                                      float* mean, float* rstd, muon_stream_t stream) {
  begin_launches();
  if (!sizes_ok(rows, dim) || !(eps >= 0.f)) return MUON_ERR_INVALID;
  if (!known(x_dtype) || !known(w_dtype)) return MUON_ERR_UNSUPPORTED;
  if (rows == 0) return MUON_OK;
  if (!x || !y || ldx < dim || ldy < dim) return MUON_ERR_INVALID;
  const size_t xs = dt_size(x_dtype), ws = dt_size(w_dtype);
  if (!is_aligned(x, xs) || !is_aligned(y, xs) || !is_aligned(weight, ws) || !is_aligned(bias, ws) ||
      !is_aligned(mean, 4) || !is_aligned(rstd, 4))
    return MUON_ERR_INVALID;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  by_types(x_dtype, w_dtype, [&](auto* tx, auto* tw) {
    using T = std::remove_pointer_t<decltype(tx)>;
    using WT = std::remove_pointer_t<decltype(tw)>;
    ln_forward_kernel<T, WT><<<(unsigned)rows, LN_THREADS, 0, s>>>((const T*)x, ldx, (const WT*)weight,
                                                                  (const WT*)bias, (int)dim, eps, (T*)y, ldy, mean,
                                                                  rstd);
  });
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" size_t muon_layernorm_workspace_size(int64_t rows, int64_t dim) {
  if (!sizes_ok(rows, dim)) return (size_t)-1;
  return (size_t)LN_SLABS * 2 * (size_t)dim * sizeof(float);
}

extern "C" int muon_layernorm_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* weight,
                                       const float* mean, const float* rstd, int64_t rows, int64_t dim, int x_dtype,
                                       int w_dtype, void* dx, int64_t lddx, void* dweight, void* dbias, void* ws,
                                       size_t ws_bytes, muon_stream_t stream) {
  begin_launches();
  if (!sizes_ok(rows, dim)) return MUON_ERR_INVALID;
  if (!known(x_dtype) || !known(w_dtype)) return MUON_ERR_UNSUPPORTED;
  const size_t xs = dt_size(x_dtype), wsz = dt_size(w_dtype);
  if (rows > 0) {
    if (!dy || !x || !mean || !rstd || !dx || lddy < dim || ldx < dim || lddx < dim) return MUON_ERR_INVALID;
    if (!is_aligned(dy, xs) || !is_aligned(x, xs) || !is_aligned(dx, xs) || !is_aligned(mean, 4) || !is_aligned(rstd, 4))
      return MUON_ERR_INVALID;
  }
  if (!is_aligned(weight, wsz) || !is_aligned(dweight, wsz) || !is_aligned(dbias, wsz)) return MUON_ERR_INVALID;
  const bool sums = dweight || dbias;
  if (rows == 0 && !sums) return MUON_OK;
  if (sums && (!ws || !is_aligned(ws, 256) || ws_bytes < muon_layernorm_workspace_size(rows, dim)))
    return MUON_ERR_WORKSPACE;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned cblocks = (unsigned)((dim + LN_THREADS - 1) / LN_THREADS);
  by_types(x_dtype, w_dtype, [&](auto* tx, auto* tw) {
    using T = std::remove_pointer_t<decltype(tx)>;
    using WT = std::remove_pointer_t<decltype(tw)>;
    if (sums) {
      const int slabs = (int)(rows < LN_SLABS ? rows : LN_SLABS);
      if (slabs > 0) {
        ln_slab_kernel<T><<<dim3(cblocks, slabs), LN_THREADS, 0, s>>>((const T*)dy, lddy, (const T*)x, ldx, mean, rstd,
                                                                     rows, (int)dim, (float*)ws);
        count_launch();
      }
      ln_columns_kernel<WT><<<cblocks, LN_THREADS, 0, s>>>((const float*)ws, slabs, (int)dim, (WT*)dweight,
                                                           (WT*)dbias);
      count_launch();
    }
    if (rows > 0) {
      ln_backward_kernel<T, WT><<<(unsigned)rows, LN_THREADS, 0, s>>>((const T*)dy, lddy, (const T*)x, ldx,
                                                                     (const WT*)weight, mean, rstd, (int)dim, (T*)dx,
                                                                     lddx);
      count_launch();
    }
  });
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
