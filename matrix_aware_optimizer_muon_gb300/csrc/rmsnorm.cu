// Root-mean-square norm behind a residual's addition, forward and backward:
//   t = x + r (rounded to their type),   y = t rstd w,   rstd = 1/sqrt(mean(t^2) + eps)
//   dt = dtotal + rstd (g - xh mean(g xh)),   g = dy w,  xh = t rstd;   dw = sum_rows dy xh
// and, forward, y in 8 bits: e4m3 codes with one fp32 scale for each row and 128 columns.
// Every sum is fp32.  t is rounded before it is normed: it is what the residual stream keeps
// and what the backward pass reads.
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
// The scale of a group whose largest magnitude is `most`.
__device__ __forceinline__ float scale_of(float most) { return max_nan(most / 448.f, RMS_LEAST_SCALE); }
// Two numbers to the nearest e4m3 codes (448 at most, NaN as NaN).
__device__ __forceinline__ uint32_t code2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
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
      const float scale = scale_of(most), inv = 1.f / scale;
      if (lane == 0) p.scales[row * p.groups + g] = scale;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = g * RMS_GROUP + 32 * j + lane;
        if (c < p.dim) {
          p.codes[row * p.ldc + c] = (uint8_t)code2(v[j] * inv, 0.f);
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

// Rows of any length: dx with the row read twice, and the columns' sums over slabs of rows.
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
constexpr int RMS_SLAB_THREADS = 256;
template <typename T>
__global__ void __launch_bounds__(RMS_SLAB_THREADS) rms_slab_kernel(const RmsBwd p) {
  const int c = blockIdx.x * RMS_SLAB_THREADS + threadIdx.x;
  if (c >= p.dim) return;
  float s = 0.f;
  for (long long r = blockIdx.y; r < p.rows; r += gridDim.y)
    s = fmaf(ld1(static_cast<const T*>(p.dy) + r * p.lddy + c), ld1(static_cast<const T*>(p.t) + r * p.ldt + c) * p.rstd[r], s);
  p.part[(size_t)blockIdx.y * p.dim + c] = s;
}

// Column sums of the lines: 32 columns a CTA, 32 threads a column over the lines (each a
// fixed set), then a fixed tree.
__global__ void __launch_bounds__(1024) rms_columns_kernel(const float* part, int lines, int dim, void* dw, int w_bf16) {
  __shared__ float tile[32][33];
  await_previous();
  const int c = blockIdx.x * 32 + threadIdx.x;
  float s = 0.f;
  if (c < dim)
    for (int i = threadIdx.y; i < lines; i += 32) s += part[(size_t)i * dim + c];
  tile[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(tile[threadIdx.x][threadIdx.y]);
  const int oc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && oc < dim) st_w(dw, w_bf16, oc, s);
}

template <typename T>
void forward(const RmsFwd& p, cudaStream_t s) {
  count_launch();
  rms_forward_loop_kernel<T><<<(unsigned)p.rows, RMS_LOOP_THREADS, 0, s>>>(p);
}

template <typename T>
cudaError_t backward(const RmsBwd& p, int* lines, cudaStream_t s) {
  *lines = 0;
  if (p.rows == 0) return cudaSuccess;
  if (p.part) {       // before dx, which may be dy itself
    *lines = (int)std::min<long long>(p.rows, RMS_CTAS);
    rms_slab_kernel<T><<<dim3(cdiv(p.dim, RMS_SLAB_THREADS), *lines), RMS_SLAB_THREADS, 0, s>>>(p);
    count_launch();
  }
  rms_backward_loop_kernel<T><<<(unsigned)p.rows, RMS_LOOP_THREADS, 0, s>>>(p);
  count_launch();
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
  if (x_dtype == MUON_DTYPE_BF16) forward<bf16>(p, s);
  else forward<float>(p, s);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
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
  int lines = 0;
  if ((x_dtype == MUON_DTYPE_BF16 ? backward<bf16>(p, &lines, s) : backward<float>(p, &lines, s)) != cudaSuccess)
    return MUON_ERR_CUDA;
  if (dweight) {
    count_launch();
    if (launch_after(rms_columns_kernel, dim3(cdiv(dim, 32)), dim3(32, 32), 0, s, p.part, lines, (int)dim, dweight,
                     p.w_bf16) != cudaSuccess)
      return MUON_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
