// Layer norm, forward and backward, with the reduction of the weight's and bias's
// gradients:
//   y  = (x - mean) rstd w + b,          rstd = 1/sqrt(var + eps)
//   dx = rstd (g - sum(g)/D - xh sum(g xh)/D),   g = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,   db = sum_rows dy
// Every sum is fp32.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace {

// Bandwidth-bound: the forward pass reads x and writes y, the backward pass reads x and
// dy and writes dx.  A row stays in registers between its reductions, so that it is read
// once.  Rows whose pointers and strides allow it move in 16-byte vectors (kVec), the
// others one element a thread with neighbouring threads on neighbouring elements, which
// keeps every access coalesced whatever the alignment.
constexpr int LN_WARPS = 8;          // rows per CTA where a warp owns a row
constexpr int LN_LOOP_THREADS = 512; // rows too long for registers

// Weights come as fp32 or bf16 (a flag: they are read from L1, the branch is uniform).
__device__ __forceinline__ float ld_w(const void* w, int w_bf16, int c) {
  return w_bf16 ? ld1(static_cast<const bf16*>(w) + c) : static_cast<const float*>(w)[c];
}
__device__ __forceinline__ void st_w(void* w, int w_bf16, int c, float v) {
  if (w_bf16) st1(static_cast<bf16*>(w) + c, v);
  else static_cast<float*>(w)[c] = v;
}

// kV consecutive elements: 16 bytes, or one element.
template <typename T, int kV> struct Pack;
template <typename T> struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ float get(int) const { return to_f32(v); }
  __device__ __forceinline__ void put(const float (&x)[1]) { v = from_f32<T>(x[0]); }
  __device__ __forceinline__ void store(T* p) const { *p = v; }
};
template <> struct Pack<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
  __device__ __forceinline__ void put(const float (&x)[4]) { v = make_float4(x[0], x[1], x[2], x[3]); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float4*>(p) = v; }
};
template <> struct Pack<bf16, 8> {
  uint32_t w[4];
  __device__ __forceinline__ void load(const bf16* p) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
  }
  __device__ __forceinline__ float get(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
  __device__ __forceinline__ void put(const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
  }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]); }
};
template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }

// kV consecutive weights (with kV > 1 their vectors are aligned too).
template <int kV>
__device__ __forceinline__ void ld_wv(const void* w, int w_bf16, int c, float (&o)[kV]) {
  if (kV == 1) {
    o[0] = ld_w(w, w_bf16, c);
  } else if (w_bf16) {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i) ld4(static_cast<const bf16*>(w) + c + 4 * i, o + 4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i) ld4(static_cast<const float*>(w) + c + 4 * i, o + 4 * i);
  }
}

// The threads of one row: a warp, or `size` threads with a barrier of their own.
struct Group {
  int t, size, id;       // thread, threads, barrier (0: the whole CTA's)
  float* red;            // 2 x 32 floats
  __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(size) : "memory"); }
  __device__ __forceinline__ float2 sum(float a, float b, int parity) const {
    a = warp_sum(a);
    b = warp_sum(b);
    // two buffers in turn: a warp may be one reduction ahead of the slowest
    float2* slot = reinterpret_cast<float2*>(red) + 32 * parity;
    if ((t & 31) == 0) slot[t >> 5] = make_float2(a, b);
    sync();
    const float2 q = (t & 31) < (size >> 5) ? slot[t & 31] : make_float2(0.f, 0.f);
    return make_float2(warp_sum(q.x), warp_sum(q.y));
  }
};

struct LnFwd {
  const void *x, *w, *b;
  void* y;
  float *mean, *rstd;
  long long ldx, ldy, rows;
  int dim, w_bf16;
  float eps;
};

template <typename T, int kV, int kN, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * LN_WARPS : 1024) ln_forward_kernel(const LnFwd p) {
  __shared__ float red[kWarp ? 1 : 128];
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x, size = kWarp ? 32 : blockDim.x;
  const long long r = kWarp ? (long long)blockIdx.x * LN_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && r >= p.rows) return;
  const Group grp{t, size, 0, red};
  const T* x = static_cast<const T*>(p.x) + r * p.ldx;
  T* y = static_cast<T*>(p.y) + r * p.ldy;
  Pack<T, kV> raw[kN];
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if ((k * size + t) * kV < p.dim) raw[k].load(x + (k * size + t) * kV);
  const float inv = 1.f / (float)p.dim;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if ((k * size + t) * kV < p.dim)
#pragma unroll
      for (int i = 0; i < kV; ++i) s += raw[k].get(i);
  const float mu = (kWarp ? warp_sum(s) : grp.sum(s, 0.f, 0).x) * inv;
  float q = 0.f;
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if ((k * size + t) * kV < p.dim)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const float d = raw[k].get(i) - mu;
        q = fmaf(d, d, q);
      }
  const float rs = 1.0f / sqrtf((kWarp ? warp_sum(q) : grp.sum(q, 0.f, 1).x) * inv + p.eps);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = (k * size + t) * kV;
    if (c < p.dim) {
      float w[kV], b[kV];
#pragma unroll
      for (int i = 0; i < kV; ++i) { w[i] = 1.f; b[i] = 0.f; }
      if (p.w) ld_wv<kV>(p.w, p.w_bf16, c, w);
      if (p.b) ld_wv<kV>(p.b, p.w_bf16, c, b);
#pragma unroll
      for (int i = 0; i < kV; ++i) b[i] = fmaf((raw[k].get(i) - mu) * rs, w[i], b[i]);
      raw[k].put(b);
      raw[k].store(y + c);
    }
  }
  if (t == 0) {
    if (p.mean) p.mean[r] = mu;
    if (p.rstd) p.rstd[r] = rs;
  }
}

// Rows longer than the registers of a CTA: three passes, the later ones from cache.
template <typename T>
__global__ void __launch_bounds__(LN_LOOP_THREADS) ln_forward_loop_kernel(const LnFwd p) {
  __shared__ float red[32];
  const long long r = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + r * p.ldx;
  T* y = static_cast<T*>(p.y) + r * p.ldy;
  float s = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += LN_LOOP_THREADS) s += ld1(x + c);
  const float mu = block_sum(s, red) / (float)p.dim;
  float q = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += LN_LOOP_THREADS) {
    const float d = ld1(x + c) - mu;
    q = fmaf(d, d, q);
  }
  const float rs = 1.0f / sqrtf(block_sum(q, red) / (float)p.dim + p.eps);
  for (int c = threadIdx.x; c < p.dim; c += LN_LOOP_THREADS) {
    const float xh = (ld1(x + c) - mu) * rs;
    st1(y + c, (p.w ? xh * ld_w(p.w, p.w_bf16, c) : xh) + (p.b ? ld_w(p.b, p.w_bf16, c) : 0.f));
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[r] = mu;
    if (p.rstd) p.rstd[r] = rs;
  }
}

struct LnBwd {
  const void *dy, *x, *w;
  const float *mean, *rstd;
  void* dx;
  float* part;           // [CTA][2][dim] sums over the CTA's rows, or null
  long long lddy, ldx, lddx, rows;
  int dim, w_bf16;
};

// A persistent CTA of several row groups (threadIdx.y).  A thread owns the same columns of
// every row its group takes, so the columns' sums stay in its registers; at the end the
// groups' sums are joined in shared memory in a fixed order and the CTA writes one line.
constexpr int LN_GROUPS = 8;
constexpr int ln_bwd_ctas(int columns) { return columns > 8 ? 1 : 2; }   // CTAs of 512 threads an SM, by registers
template <typename T, int kV, int kN>
__global__ void __launch_bounds__(512, ln_bwd_ctas(kV * kN)) ln_backward_kernel(const LnBwd p) {
  extern __shared__ float sums[];               // [groups - 1][2][dim]
  __shared__ float red[LN_GROUPS * 128];
  const int t = threadIdx.x, size = blockDim.x, grp_i = threadIdx.y, groups = blockDim.y;
  const Group grp{t, size, 1 + grp_i, red + 128 * grp_i};
  const float inv = 1.f / (float)p.dim;
  float sw[kN][kV], sb[kN][kV];
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int i = 0; i < kV; ++i) sw[k][i] = sb[k][i] = 0.f;
  int parity = 0;
  for (long long r = (long long)blockIdx.x * groups + grp_i; r < p.rows; r += (long long)gridDim.x * groups) {
    const T* x = static_cast<const T*>(p.x) + r * p.ldx;
    const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
    Pack<T, kV> xr[kN], gr[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if ((k * size + t) * kV < p.dim) {
        xr[k].load(x + (k * size + t) * kV);
        gr[k].load(dy + (k * size + t) * kV);
      }
    const float mu = p.mean[r], rs = p.rstd[r];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = (k * size + t) * kV;
      if (c < p.dim) {
        float w[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) w[i] = 1.f;
        if (p.w) ld_wv<kV>(p.w, p.w_bf16, c, w);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float d = gr[k].get(i), xh = (xr[k].get(i) - mu) * rs, g = d * w[i];
          sw[k][i] = fmaf(d, xh, sw[k][i]);
          sb[k][i] += d;
          s1 += g;
          s2 = fmaf(g, xh, s2);
        }
      }
    }
    const float2 c12 = grp.sum(s1, s2, parity);
    parity ^= 1;
    const float c1 = c12.x * inv, c2 = c12.y * inv;
    T* dx = static_cast<T*>(p.dx) + r * p.lddx;
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = (k * size + t) * kV;
      if (c < p.dim) {
        float w[kV];
#pragma unroll
        for (int i = 0; i < kV; ++i) w[i] = 1.f;
        if (p.w) ld_wv<kV>(p.w, p.w_bf16, c, w);
#pragma unroll
        for (int i = 0; i < kV; ++i) {
          const float xh = (xr[k].get(i) - mu) * rs;
          w[i] = rs * (gr[k].get(i) * w[i] - c1 - xh * c2);
        }
        gr[k].put(w);
        gr[k].store(dx + c);
      }
    }
  }
  if (!p.part) return;
  if (grp_i > 0) {
    float* o = sums + (size_t)(grp_i - 1) * 2 * p.dim;
#pragma unroll
    for (int k = 0; k < kN; ++k)
#pragma unroll
      for (int i = 0; i < kV; ++i) {
        const int c = (k * size + t) * kV + i;
        if (c < p.dim) { o[c] = sw[k][i]; o[p.dim + c] = sb[k][i]; }
      }
  }
  __syncthreads();
  if (grp_i > 0) return;
  float* o = p.part + (size_t)blockIdx.x * 2 * p.dim;
#pragma unroll
  for (int k = 0; k < kN; ++k)
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const int c = (k * size + t) * kV + i;
      if (c < p.dim) {
        for (int j = 0; j < groups - 1; ++j) {
          sw[k][i] += sums[(size_t)j * 2 * p.dim + c];
          sb[k][i] += sums[(size_t)j * 2 * p.dim + p.dim + c];
        }
        o[c] = sw[k][i];
        o[p.dim + c] = sb[k][i];
      }
    }
}

// Long rows: dx with the row read three times (from cache after the first), and the
// columns' sums over slabs of rows in a pass of their own.
template <typename T>
__global__ void __launch_bounds__(LN_LOOP_THREADS) ln_backward_loop_kernel(const LnBwd p) {
  __shared__ float red[32];
  const long long r = blockIdx.x;
  const float mu = p.mean[r], rs = p.rstd[r];
  const T* x = static_cast<const T*>(p.x) + r * p.ldx;
  const T* dy = static_cast<const T*>(p.dy) + r * p.lddy;
  T* dx = static_cast<T*>(p.dx) + r * p.lddx;
  float s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x; c < p.dim; c += LN_LOOP_THREADS) {
    const float g = ld1(dy + c) * (p.w ? ld_w(p.w, p.w_bf16, c) : 1.f);
    s1 += g;
    s2 = fmaf(g, (ld1(x + c) - mu) * rs, s2);
  }
  const float c1 = block_sum(s1, red) / (float)p.dim;
  const float c2 = block_sum(s2, red) / (float)p.dim;
  for (int c = threadIdx.x; c < p.dim; c += LN_LOOP_THREADS) {
    const float g = ld1(dy + c) * (p.w ? ld_w(p.w, p.w_bf16, c) : 1.f);
    st1(dx + c, rs * (g - c1 - (ld1(x + c) - mu) * rs * c2));
  }
}
constexpr int LN_SLAB_THREADS = 256;
template <typename T>
__global__ void __launch_bounds__(LN_SLAB_THREADS) ln_slab_kernel(const LnBwd p) {
  const int c = blockIdx.x * LN_SLAB_THREADS + threadIdx.x;
  if (c >= p.dim) return;
  float sw = 0.f, sb = 0.f;
  for (long long r = blockIdx.y; r < p.rows; r += gridDim.y) {
    const float g = ld1(static_cast<const T*>(p.dy) + r * p.lddy + c);
    sw = fmaf(g, (ld1(static_cast<const T*>(p.x) + r * p.ldx + c) - p.mean[r]) * p.rstd[r], sw);
    sb += g;
  }
  p.part[(size_t)blockIdx.y * 2 * p.dim + c] = sw;
  p.part[(size_t)blockIdx.y * 2 * p.dim + p.dim + c] = sb;
}

// Column sums of the lines the CTAs wrote: 32 columns a CTA, 32 threads a column over the
// lines (each a fixed set), then a fixed tree.
__global__ void __launch_bounds__(1024) ln_columns_kernel(const float* part, int lines, int dim, void* dw, void* db,
                                                          int w_bf16) {
  __shared__ float tile[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
  void* out = which ? db : dw;
  if (!out) return;
  float s = 0.f;
  if (c < dim)
    for (int i = threadIdx.y; i < lines; i += 32) s += part[((size_t)i * 2 + which) * dim + c];
  tile[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = warp_sum(tile[threadIdx.x][threadIdx.y]);
  const int oc = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && oc < dim) st_w(out, w_bf16, oc, s);
}

bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
bool known(int dt) { return dt == MUON_DTYPE_F32 || dt == MUON_DTYPE_BF16; }
bool sizes_ok(int64_t rows, int64_t dim) { return rows >= 0 && rows < (1LL << 31) && dim >= 1 && dim < (1LL << 31); }

int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Whether rows of p (ld elements apart) and the weights can be read in 16-byte vectors.
bool vec_rows(const void* p, int64_t ld, int64_t rows, size_t es) {
  return is_aligned(p, 16) && (rows <= 1 || (size_t)ld * es % 16 == 0);
}

template <typename T, int kV, bool kWarp>
bool forward_n(const LnFwd& p, int need, int threads, cudaStream_t s) {
  const unsigned grid = (unsigned)(kWarp ? cdiv(p.rows, LN_WARPS) : p.rows);
#define MUON_LN_FWD(N)                                                   \
  if (need <= N) {                                                       \
    ln_forward_kernel<T, kV, N, kWarp><<<grid, threads, 0, s>>>(p);      \
    return true;                                                         \
  }
  if constexpr (kV > 1 && kWarp) {
    MUON_LN_FWD(1) MUON_LN_FWD(2) MUON_LN_FWD(3) MUON_LN_FWD(4) MUON_LN_FWD(6) MUON_LN_FWD(8) MUON_LN_FWD(12)
    MUON_LN_FWD(16)
  } else if constexpr (kV > 1) {
    MUON_LN_FWD(1) MUON_LN_FWD(2) MUON_LN_FWD(4)
  } else if constexpr (kWarp) {
    MUON_LN_FWD(2) MUON_LN_FWD(8) MUON_LN_FWD(16)
  } else {
    MUON_LN_FWD(4) MUON_LN_FWD(8) MUON_LN_FWD(16)
  }
#undef MUON_LN_FWD
  return false;
}

// A warp per row while a lane holds its share of the row in registers (16 accesses);
// above that a CTA per row.
template <typename T>
void forward(const LnFwd& p, bool vec, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  if (vec) {
    const int nv = p.dim / V;
    if (forward_n<T, V, true>(p, cdiv(nv, 32), 32 * LN_WARPS, s)) return;
    const int threads = 32 * cdiv(nv, 32LL * cdiv(nv, 1024));
    if (forward_n<T, V, false>(p, cdiv(nv, threads), threads, s)) return;
  } else {
    if (forward_n<T, 1, true>(p, cdiv(p.dim, 32), 32 * LN_WARPS, s)) return;
    const int threads = 32 * cdiv(p.dim, 32LL * std::max(8, cdiv(p.dim, 1024)));
    if (forward_n<T, 1, false>(p, cdiv(p.dim, threads), threads, s)) return;
  }
  ln_forward_loop_kernel<T><<<(unsigned)p.rows, LN_LOOP_THREADS, 0, s>>>(p);
}

// The backward pass's CTAs, at most two on each of 152 SMs; every CTA writes one line of
// partial sums.
constexpr int LN_CTAS = 304;
constexpr int LN_MAX_SUMS = 96 * 1024;   // shared memory for the groups' sums

template <typename T, int kV, int kN>
bool backward_n(const LnBwd& p, int threads, int* lines, cudaStream_t s, cudaError_t* err) {
  int groups = std::max(1, std::min(512 / threads, LN_GROUPS));
  while (groups > 1 && (size_t)(groups - 1) * 2 * p.dim * 4 > LN_MAX_SUMS) --groups;
  const int grid = (int)std::min<long long>((p.rows + groups - 1) / groups, LN_CTAS / 2 * ln_bwd_ctas(kV * kN));
  const size_t smem = p.part ? (size_t)(groups - 1) * 2 * p.dim * 4 : 0;
  if (smem > 32 * 1024 &&
      (*err = cudaFuncSetAttribute(ln_backward_kernel<T, kV, kN>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   LN_MAX_SUMS)) != cudaSuccess)
    return true;
  ln_backward_kernel<T, kV, kN><<<grid, dim3(threads, groups), smem, s>>>(p);
  *lines = grid;
  return true;
}

// Threads of a row: as many as it has accesses, at most 512, then up to kN accesses each.
template <typename T, int kV>
bool backward_v(const LnBwd& p, int accesses, int* lines, cudaStream_t s, cudaError_t* err) {
  auto threads = [&](int n) { return 32 * cdiv(accesses, 32LL * n); };
  if (threads(1) <= (kV > 1 ? 512 : 128)) return backward_n<T, kV, 1>(p, threads(1), lines, s, err);
  if (threads(2) <= (kV > 1 ? 512 : 128)) return backward_n<T, kV, 2>(p, threads(2), lines, s, err);
  if constexpr (kV < 8) {
    if (threads(4) <= 512) return backward_n<T, kV, 4>(p, threads(4), lines, s, err);
  }
  if constexpr (kV == 1) {
    if (threads(8) <= 512) return backward_n<T, kV, 8>(p, threads(8), lines, s, err);
    if (threads(16) <= 512) return backward_n<T, kV, 16>(p, threads(16), lines, s, err);
  }
  return false;
}

template <typename T>
cudaError_t backward(const LnBwd& p, bool vec, int* lines, cudaStream_t s) {
  cudaError_t err = cudaSuccess;
  *lines = 0;
  if (p.rows == 0) return err;
  bool done = vec ? backward_v<T, vec_of<T>()>(p, p.dim / vec_of<T>(), lines, s, &err)
                  : backward_v<T, 1>(p, p.dim, lines, s, &err);
  if (err != cudaSuccess) return err;
  if (!done) {
    if (p.part) {
      *lines = (int)std::min<long long>(p.rows, LN_CTAS);
      ln_slab_kernel<T><<<dim3(cdiv(p.dim, LN_SLAB_THREADS), *lines), LN_SLAB_THREADS, 0, s>>>(p);
      count_launch();
    }
    ln_backward_loop_kernel<T><<<(unsigned)p.rows, LN_LOOP_THREADS, 0, s>>>(p);
  }
  count_launch();
  return cudaGetLastError();
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
  const LnFwd p{x, weight, bias, y, mean, rstd, ldx, ldy, rows, (int)dim, w_dtype == MUON_DTYPE_BF16, eps};
  const bool vec = dim * xs % 16 == 0 && vec_rows(x, ldx, rows, xs) && vec_rows(y, ldy, rows, xs) &&
                   is_aligned(weight, 16) && is_aligned(bias, 16);
  if (x_dtype == MUON_DTYPE_BF16) forward<bf16>(p, vec, s);
  else forward<float>(p, vec, s);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" size_t muon_layernorm_workspace_size(int64_t rows, int64_t dim) {
  if (!sizes_ok(rows, dim)) return (size_t)-1;
  return (size_t)LN_CTAS * 2 * (size_t)dim * sizeof(float);
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
  const LnBwd p{dy, x, weight, mean, rstd, dx, sums ? static_cast<float*>(ws) : nullptr, lddy, ldx, lddx, rows,
                (int)dim, w_dtype == MUON_DTYPE_BF16};
  const bool vec = dim * xs % 16 == 0 && vec_rows(x, ldx, rows, xs) && vec_rows(dy, lddy, rows, xs) &&
                   vec_rows(dx, lddx, rows, xs) && is_aligned(weight, 16);
  int lines = 0;
  const cudaError_t e = x_dtype == MUON_DTYPE_BF16 ? backward<bf16>(p, vec, &lines, s) : backward<float>(p, vec, &lines, s);
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  if (sums) {
    ln_columns_kernel<<<dim3(cdiv(dim, 32), 2), dim3(32, 32), 0, s>>>(p.part, lines, (int)dim, dweight, dbias, p.w_bf16);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
