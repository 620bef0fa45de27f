// Layer norm, forward and backward, with the reduction of the weight's and bias's
// gradients:
//   y  = (x - mean) rstd w + b,          rstd = 1/sqrt(var + eps)
//   dx = rstd (g - sum(g)/D - xh sum(g xh)/D),   g = dy w,  xh = (x - mean) rstd
//   dw = sum_rows dy xh,   db = sum_rows dy
// Every sum is fp32.  Measured, of HBM's 6.79 TB/s (a copy): 32768 x 1536 bf16 forward
// 36.7 us (5.5 TB/s), backward with both column sums 61.5 us (4.9 TB/s; 55 of them the rows'
// kernel, 4 the column sums'); 5003 x 1537 fp32 rows of no alignment backward 25.7 us
// (3.6 TB/s).  What is left: the forward pass and the rows' kernel wait for memory at half
// of the issue slots; fp32 arithmetic in single instead of paired instructions takes the
// same time.
#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace muon {
namespace {

using namespace rows;

// Bandwidth-bound: the forward pass reads x and writes y, the backward pass reads x and
// dy and writes dx.  A row stays in registers between its reductions, so that it is read
// once.  Rows whose pointers and strides allow it move in 16-byte vectors (kVec), the
// others one element a thread with neighbouring threads on neighbouring elements, which
// keeps every access coalesced whatever the alignment.
constexpr int LN_WARPS = 8;          // rows per CTA where a warp owns a row
constexpr int LN_LOOP_THREADS = 512; // rows too long for registers

struct LnFwd {
  const void *x, *w, *b;
  void* y;
  float *mean, *rstd;
  long long ldx, ldy, rows;
  int dim, w_bf16;
  float eps;
};

// CTAs of a warp-a-row kernel an SM should hold: registers for the row and about 32 more.
constexpr int ln_fwd_ctas(int n, bool warp) { return warp ? 256 / (4 * n + 32) : 1; }
template <typename T, int kV, int kN, bool kWarp, int kW, int kSize>
__global__ void __launch_bounds__(kWarp ? 32 * LN_WARPS : kSize ? kSize : 1024, ln_fwd_ctas(kN, kWarp)) ln_forward_kernel(const LnFwd p) {
  constexpr int kSure = kWarp || kSize ? sure_of(kN) : 0;
  __shared__ __align__(8) float red[kWarp ? 2 : 128];
  const int t = kWarp ? threadIdx.x & 31 : threadIdx.x, size = kWarp ? 32 : kSize ? kSize : blockDim.x;
  const long long r = kWarp ? (long long)blockIdx.x * LN_WARPS + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && r >= p.rows) return;
  const Group grp{t, size, 0, red};
  const T* x = static_cast<const T*>(p.x) + r * p.ldx;
  T* y = static_cast<T*>(p.y) + r * p.ldy;
  using S = Share<kV, kN>;
  // The row stays in registers as loaded and is widened again for each of the three
  // passes: held as fp32 pairs it would leave room for half as many warps (measured on
  // 32768 x 1536 bf16: 53 us instead of 37).
  Raw<T, kV, kN> raw;
  raw.template load<kSure>(x, t, size, p.dim);
  constexpr int C = kV == 1 ? 1 : kV / 2;   // pairs of an access
  const float inv = 1.f / (float)p.dim;
  f32x2 s = both(0.f), q = both(0.f);
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    f32x2 v[C];
    raw.get(k, v);
#pragma unroll
    for (int i = 0; i < C; ++i) s = add2(s, v[i]);
  }
  const float sum = lo2(s) + hi2(s);
  const float mu = (kWarp ? warp_sum(sum) : grp.sum(sum, 0.f, 0).x) * inv;
  raw.hold();
#pragma unroll
  for (int k = 0; k < kN; ++k)
    if (k < kSure || (k * size + t) * kV < p.dim) {
      f32x2 v[C];
      raw.get(k, v);
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const f32x2 d = add2(v[i], kV == 1 ? make2(-mu, 0.f) : both(-mu));
        q = fma2(d, d, q);
      }
    }
  const float ssq = lo2(q) + hi2(q);
  const float rs = 1.0f / sqrtf((kWarp ? warp_sum(ssq) : grp.sum(ssq, 0.f, 1).x) * inv + p.eps);
  raw.hold();
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = (k * size + t) * kV;
    if (k < kSure || c < p.dim) {
      f32x2 v[C], w[C], b[C];
      raw.get(k, v);
      weights<kV, kW>(p.w, p.w_bf16, c, p.dim, 1.f, w);
      weights<kV, kW>(p.b, p.w_bf16, c, p.dim, 0.f, b);
#pragma unroll
      for (int i = 0; i < C; ++i) b[i] = fma2(mul2(add2(v[i], both(-mu)), both(rs)), w[i], b[i]);
      if constexpr (kV > 1) store16(y + c, b);
      else st1(y + c, lo2(b[0]));
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
// every row its group takes, so the weights and the columns' sums stay in its registers; at
// the end the groups' sums are joined in shared memory in a fixed order and the CTA writes
// one line.  Rows come through a ring of asynchronous copies in shared memory that each
// thread keeps for itself (it reads only what it copied: no barrier), because the registers
// are taken: 6 KB a row of 1536 bf16 pairs, ln_ring() - 1 rows ahead.  Rows that need
// element-wise access are fetched one row ahead into registers (5003 x 1537 fp32: 25.9 us; two
// or three rows ahead 28.4 and 28.6, through 4-byte asynchronous copies 28.4).
constexpr int LN_GROUPS = 8;
__host__ __device__ constexpr int ln_ring(int n) { return n <= 2 ? 4 : 3; }

// 512 threads leave each 128 registers.  Measured on 32768 x 1536 bf16: 512 threads (5 rows at
// once) 61.5 us, 384 63.6, 640 (spilling) 90.7; a ring of 3, 4 or 6 rows 61.1 to 62.5.
constexpr int LN_BWD_THREADS = 512;
template <typename T, int kV, int kN, int kSize>
__global__ void __launch_bounds__(LN_BWD_THREADS, 1) ln_backward_kernel(const LnBwd p) {
  extern __shared__ uint4 dyn[];
  __shared__ __align__(8) float red[LN_GROUPS * 128];
  using S = Share<kV, kN>;
  constexpr int kSure = kSize ? sure_of(kN) : 0;
  const int t = threadIdx.x, size = kSize ? kSize : blockDim.x, grp_i = threadIdx.y, groups = blockDim.y;
  const int nthr = size * groups, tid = grp_i * size + t;
  const Group grp{t, size, 1 + grp_i, red + 128 * grp_i};
  const float inv = 1.f / (float)p.dim;
  const long long step = (long long)gridDim.x * groups;
  long long r = (long long)blockIdx.x * groups + grp_i;
  f32x2 w[S::P], sw[S::P], sb[S::P];
#pragma unroll
  for (int i = 0; i < S::P; ++i) sw[i] = sb[i] = both(0.f);
  if constexpr (kV > 1) {
#pragma unroll
    for (int k = 0; k < kN; ++k) weights<kV>(p.w, p.w_bf16, (k * size + t) * kV, p.dim, 1.f, w + k * (kV / 2));
  } else {
    f32x2 a[2];
#pragma unroll
    for (int k = 0; k < kN; k += 2) {
      weights<1>(p.w, p.w_bf16, k * size + t, p.dim, 1.f, a);
      a[1] = both(0.f);
      if (k + 1 < kN) weights<1>(p.w, p.w_bf16, (k + 1) * size + t, p.dim, 1.f, a + 1);
      w[k / 2] = make2(lo2(a[0]), lo2(a[1]));
    }
  }
  constexpr int R = ln_ring(kN);
  // where the next row to be fetched lies, and the row at hand
  const T* xf = static_cast<const T*>(p.x) + r * p.ldx;
  const T* gf = static_cast<const T*>(p.dy) + r * p.lddy;
  T* dx = static_cast<T*>(p.dx) + r * p.lddx;
  const float *mean = p.mean + r, *rstd = p.rstd + r;
  const long long sx = step * p.ldx, sg = step * p.lddy, sd = step * p.lddx;
  long long rf = r;
  uint4* const mine = dyn + tid;                // [slot][x, dy][access][thread]
  auto fetch = [&](int slot) {                  // one group of copies, empty past the last row
    if (rf < p.rows) {
      uint4* d = mine + slot * (2 * kN) * nthr;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int c = (k * size + t) * kV;
        if (k < kSure || c < p.dim) {
          copy16(d + k * nthr, xf + c);
          copy16(d + (kN + k) * nthr, gf + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    rf += step;
    xf += sx;
    gf += sg;
  };
  Raw<T, kV, kN> xn, gn;
  float mu_n = 0.f, rs_n = 0.f;
  if constexpr (kV > 1) {
    // slots that are never copied to belong to columns past the row: zero
#pragma unroll
    for (int k = kSure; k < kN; ++k)
      if ((k * size + t) * kV >= p.dim)
        for (int s = 0; s < 2 * R; ++s) mine[(s * kN + k) * nthr] = make_uint4(0, 0, 0, 0);
    for (int s = 0; s < R - 1; ++s) fetch(s);
  } else if (r < p.rows) {
    xn.template load<kSure>(xf, t, size, p.dim);
    gn.template load<kSure>(gf, t, size, p.dim);
  }
  if (r < p.rows) { mu_n = *mean; rs_n = *rstd; }
  int parity = 0, at = 0;
  for (; r < p.rows; r += step) {
    f32x2 xh[S::P], g[S::P];
    const float mu = mu_n, rs = rs_n;
    if constexpr (kV > 1) {
      fetch(at == 0 ? R - 1 : at - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(R - 1) : "memory");
      const uint4* d = mine + at * (2 * kN) * nthr;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        widen(d[k * nthr], xh + k * (kV / 2), static_cast<const T*>(nullptr));
        widen(d[(kN + k) * nthr], g + k * (kV / 2), static_cast<const T*>(nullptr));
      }
      at = at + 1 == R ? 0 : at + 1;
    } else {
      xn.pairs(xh);
      gn.pairs(g);
    }
    if (r + step < p.rows) {
      mean += step;
      rstd += step;
      mu_n = *mean;
      rs_n = *rstd;
      if constexpr (kV == 1) {
        xf += sx;
        gf += sg;
        xn.template load<kSure>(xf, t, size, p.dim);
        gn.template load<kSure>(gf, t, size, p.dim);
      }
    }
    f32x2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < S::P; ++i) {
      xh[i] = mul2(add2(xh[i], both(-mu)), both(rs));
      sw[i] = fma2(g[i], xh[i], sw[i]);
      sb[i] = add2(sb[i], g[i]);
      g[i] = mul2(g[i], w[i]);
      s1 = add2(s1, g[i]);
      s2 = fma2(g[i], xh[i], s2);
    }
    const float2 c12 = grp.sum(lo2(s1) + hi2(s1), lo2(s2) + hi2(s2), parity);
    parity ^= 1;
    const f32x2 c1 = both(-rs * (c12.x * inv)), c2 = both(-rs * (c12.y * inv));
#pragma unroll
    for (int i = 0; i < S::P; ++i) g[i] = fma2(xh[i], c2, fma2(g[i], both(rs), c1));
    store_row<T, kV, kN, kSure>(dx, g, t, size, p.dim);
    dx += sd;
  }
  if (!p.part) return;
  if constexpr (kV > 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();                              // the ring's memory is free for the sums
  float* sums = reinterpret_cast<float*>(dyn);  // [groups - 1][2][dim]
  if (grp_i > 0) {
    float* o = sums + (size_t)(grp_i - 1) * 2 * p.dim;
#pragma unroll
    for (int e = 0; e < S::E; ++e) {
      const int c = ((e / kV) * size + t) * kV + e % kV;
      if (c < p.dim) { o[c] = elem(sw, e); o[p.dim + c] = elem(sb, e); }
    }
  }
  __syncthreads();
  if (grp_i > 0) return;
  float* o = p.part + (size_t)blockIdx.x * 2 * p.dim;
#pragma unroll
  for (int e = 0; e < S::E; ++e) {
    const int c = ((e / kV) * size + t) * kV + e % kV;
    if (c < p.dim) {
      float a = elem(sw, e), b = elem(sb, e);
      for (int j = 0; j < groups - 1; ++j) {
        a += sums[(size_t)j * 2 * p.dim + c];
        b += sums[(size_t)j * 2 * p.dim + p.dim + c];
      }
      o[c] = a;
      o[p.dim + c] = b;
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
  await_previous();
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

template <typename T, int kV, int kN, bool kWarp, int kSize>
void forward_launch(const LnFwd& p, int threads, cudaStream_t s) {
  const unsigned grid = (unsigned)(kWarp ? cdiv(p.rows, LN_WARPS) : p.rows);
  if constexpr (kV > 1 && kWarp) {
    if (p.w && p.b && p.w_bf16) { ln_forward_kernel<T, kV, kN, kWarp, W_BF16, kSize><<<grid, threads, 0, s>>>(p); return; }
    if (p.w && p.b) { ln_forward_kernel<T, kV, kN, kWarp, W_F32, kSize><<<grid, threads, 0, s>>>(p); return; }
  }
  ln_forward_kernel<T, kV, kN, kWarp, W_ASK, kSize><<<grid, threads, 0, s>>>(p);
}

// A warp per row while a lane holds its share of the row in registers (16 accesses, 8 of
// single elements); above that a CTA per row.
template <typename T>
void forward(const LnFwd& p, bool vec, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  const int n = vec ? p.dim / V : p.dim;   // accesses
  const int need = cdiv(n, 32);
  if (vec && need <= 16) {
    by_accesses(need, [&](auto N) { forward_launch<T, V, decltype(N)::value, true, 32>(p, 32 * LN_WARPS, s); });
  } else if (vec && n <= 4096) {
    const int threads = 32 * cdiv(n, 32LL * cdiv(n, 1024)), each = cdiv(n, threads);
    if (each == 1) forward_launch<T, V, 1, false, 0>(p, threads, s);
    else if (each == 2) forward_launch<T, V, 2, false, 0>(p, threads, s);
    else forward_launch<T, V, 4, false, 0>(p, threads, s);
  } else if (!vec && need <= 8) {
    by_accesses(need, [&](auto N) {
      if constexpr (decltype(N)::value <= 8) forward_launch<T, 1, decltype(N)::value, true, 32>(p, 32 * LN_WARPS, s);
    });
  } else if (!vec && n <= 256 * 16) {
    by_accesses(cdiv(n, 256), [&](auto N) { forward_launch<T, 1, decltype(N)::value, false, 256>(p, 256, s); });
  } else if (!vec && n <= 1024 * 16) {
    by_accesses(cdiv(n, 1024), [&](auto N) {
      if constexpr (decltype(N)::value >= 4) forward_launch<T, 1, decltype(N)::value, false, 1024>(p, 1024, s);
    });
  } else {
    ln_forward_loop_kernel<T><<<(unsigned)p.rows, LN_LOOP_THREADS, 0, s>>>(p);
  }
}

// The backward pass's CTAs: one on each SM (its registers fill it); every CTA writes one
// line of partial sums.
constexpr int LN_CTAS = 152;
constexpr int LN_MAX_SMEM = 200 * 1024;

template <typename T, int kV, int kN, int kSize>
cudaError_t backward_launch(const LnBwd& p, int threads, int* lines, cudaStream_t s) {
  int groups = std::max(1, std::min(LN_BWD_THREADS / threads, LN_GROUPS));
  auto smem_of = [&](int g) {
    const size_t ring = kV > 1 ? (size_t)ln_ring(kN) * 2 * kN * 16 * threads * g : 0;
    return std::max(ring, p.part ? (size_t)(g - 1) * 2 * p.dim * 4 : 0);
  };
  while (groups > 1 && smem_of(groups) > (size_t)LN_MAX_SMEM) --groups;
  const size_t smem = smem_of(groups);
  if (smem > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(ln_backward_kernel<T, kV, kN, kSize>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, LN_MAX_SMEM);
    if (e != cudaSuccess) return e;
  }
  *lines = (int)std::min<long long>((p.rows + groups - 1) / groups, LN_CTAS);
  ln_backward_kernel<T, kV, kN, kSize><<<*lines, dim3(threads, groups), smem, s>>>(p);
  count_launch();
  return cudaGetLastError();
}

// 16 columns a thread (registers hold their sums, weights and the row), 8 for rows that 16
// would leave to less than two warps.  Element-wise rows: a fixed number of threads, so that
// an access is an offset the instruction holds, and as few columns each as cover the row.
template <typename T>
cudaError_t backward(const LnBwd& p, bool vec, int* lines, cudaStream_t s) {
  constexpr int V = vec_of<T>();
  cudaError_t e = cudaSuccess;
  *lines = 0;
  if (p.rows == 0) return e;
  const int n = vec ? p.dim / V : p.dim;
  auto threads = [&](int each) { return 32 * cdiv(n, 32LL * each); };
  if (vec && n <= 32 * 16 / V) return backward_launch<T, V, 8 / V, 0>(p, threads(8 / V), lines, s);
  if (vec && threads(16 / V) <= LN_BWD_THREADS) return backward_launch<T, V, 16 / V, 0>(p, threads(16 / V), lines, s);
  if (!vec && n <= 256) {
    by_accesses(cdiv(n, 32), [&](auto N) {
      if constexpr (decltype(N)::value <= 8) e = backward_launch<T, 1, decltype(N)::value, 32>(p, 32, lines, s);
    });
    return e;
  }
  if (!vec && n <= 256 * 12) {
    by_accesses(cdiv(n, 256), [&](auto N) {
      if constexpr (decltype(N)::value <= 12) e = backward_launch<T, 1, decltype(N)::value, 256>(p, 256, lines, s);
    });
    return e;
  }
  if (!vec && n <= 512 * 16) {
    by_accesses(cdiv(n, 512), [&](auto N) {
      if constexpr (decltype(N)::value >= 6) e = backward_launch<T, 1, decltype(N)::value, 512>(p, 512, lines, s);
    });
    return e;
  }
  if (p.part) {
    *lines = (int)std::min<long long>(p.rows, LN_CTAS);
    ln_slab_kernel<T><<<dim3(cdiv(p.dim, LN_SLAB_THREADS), *lines), LN_SLAB_THREADS, 0, s>>>(p);
    count_launch();
  }
  ln_backward_loop_kernel<T><<<(unsigned)p.rows, LN_LOOP_THREADS, 0, s>>>(p);
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
    count_launch();
    if (launch_after(ln_columns_kernel, dim3(cdiv(dim, 32), 2), dim3(32, 32), 0, s, p.part, lines, (int)dim, dweight,
                     dbias, p.w_bf16) != cudaSuccess)
      return MUON_ERR_CUDA;
  }
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
