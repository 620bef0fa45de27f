// Log probabilities of a few rows (a decoding step, a short answer to be scored), forward and
// backward, without the tiles of the others:
//   forward   z = H W^T and its statistics, W read once;
//   backward  z again, g from it, dW = g^T H and dH = g W, W read and dW written once.
//
// With few rows a call is bound by W's bytes, and the tiles of 256 rows leave most of
// themselves empty; 32-bit operands would besides be written and read
// again as three bf16 parts.  fp32 products, and those of W's rows that begin off a 16-byte word: the rows of H lie
// in shared memory as fp32 numbers; a warp reads four rows of W at a time, so that a word of H serves four
// products, and adds in fp32 (a lane dim/32 products, then a tree).  bf16 forward: matrix instructions
// that take W from registers.  What a statistic or a key is, ce.h says: the kernels that
// join them are those of the other path.
#include <algorithm>
#include <type_traits>

#include "ce.h"
#include "rows.cuh"

namespace muon {
namespace ce {
namespace {

constexpr int FEW_THREADS = 256;
constexpr int FEW_WARPS = FEW_THREADS / 32;
constexpr int FEW_AT_ONCE = 4;              // rows of W a warp multiplies at a time
constexpr int FEW_BLOCK = 128;              // columns of a statistic; 32 where that leaves SMs without work
constexpr int FEW_PIECE = FEW_WARPS * FEW_AT_ONCE;   // rows of W a CTA takes at a time in the backward pass
static_assert(FEW_PIECE == KEY_COLS, "a short block is a group of the keys, a step of each warp");
constexpr float FEW_FLOOR = -200.f;

// How rows of W are read: by elements, by 16-byte words, or, where they begin off a word, by
// words all the same, against four copies of H that lie 0 to 3 columns on.  The copies are for
// bf16 (50257 x 2501, 1 row 57 us, by elements 127; 2 rows 111 and 146); of fp32 numbers elements are as
// wide as lanes need them (50257 x 1001, 4 rows 48 us, by copies 72, and by windows of two
// words 121).
enum Read { ELEMENTS, WORDS, SHIFTED };
constexpr int FEW_LEAD = 4, FEW_REST = 24;  // zeros in front of a copy's row, and all that it is longer than dp

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
size_t padded(int64_t dim) { return (size_t)(dim + 7) / 8 * 8; }

// The rows of H as fp32 numbers, zeros behind them and in rows without a use.
template <typename T, int R>
__device__ __forceinline__ void stage_rows(const Few& p, float* h, int dp) {
  for (int r = 0; r < R; ++r) {
    bool live = r < p.rows;
    if (live && p.masked) {
      const long long lab = p.labels[r];
      live = lab != p.ignore && lab >= 0 && lab < p.vocab;
    }
    const T* x = static_cast<const T*>(p.H) + r * p.ldh;
    for (int c = threadIdx.x; c < dp; c += FEW_THREADS) h[r * dp + c] = live && c < p.dim ? ld1(x + c) : 0.f;
  }
}

// Its copies: column c of copy j is at FEW_LEAD + j + c.
template <typename T, int R>
__device__ __forceinline__ void stage_copies(const Few& p, float* h, int dq) {
  for (int r = 0; r < R; ++r) {
    const T* x = static_cast<const T*>(p.H) + r * p.ldh;
    for (int i = threadIdx.x; i < dq; i += FEW_THREADS)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = i - j - FEW_LEAD;
        h[(j * R + r) * dq + i] = r < p.rows && c >= 0 && c < p.dim ? ld1(x + c) : 0.f;
      }
  }
}

__device__ __forceinline__ void widen_word(const uint4& q, f32x2 (&v)[4], const bf16*) {
  v[0] = cvt2(q.x); v[1] = cvt2(q.y); v[2] = cvt2(q.z); v[3] = cvt2(q.w);
}
__device__ __forceinline__ void widen_word(const uint4& q, f32x2 (&v)[2], const float*) {
  v[0] = make2(__uint_as_float(q.x), __uint_as_float(q.y));
  v[1] = make2(__uint_as_float(q.z), __uint_as_float(q.w));
}

// Elements k to k + 3 of a word.
template <typename T>
__device__ __forceinline__ void four_of(const uint4& q, int k, float (&x)[4], const T* type) {
  f32x2 all[8 / sizeof(T)];
  widen_word(q, all, type);
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = j & 1 ? hi2(all[(k + j) / 2]) : lo2(all[(k + j) / 2]);
}
__device__ __forceinline__ float add_four(const float (&x)[4], const float4& y, float v) {
  return fmaf(x[3], y.w, fmaf(x[2], y.z, fmaf(x[1], y.y, fmaf(x[0], y.x, v))));
}

// The products of FEW_AT_ONCE rows of W from v0 on with the R rows of H, summed over the warp:
// lane l has product l * n / 32 (row of W times R plus row of H) of the n, the first of two
// where n is 64.  kSquares: lane l also gets the squares' sum of row l / 8 of W.
template <typename T, int R, Read kRead, bool kSquares>
__device__ __forceinline__ float2 products(const Few& p, const float* h, int dp, long long v0, int lane, float& squares) {
  constexpr int N = FEW_AT_ONCE * R;
  float v[N], sq[FEW_AT_ONCE];                  // (pairs of numbers would take twice the registers)
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
#pragma unroll
  for (int i = 0; i < FEW_AT_ONCE; ++i) sq[i] = 0.f;
  const auto square = [&](int i, const float (&x)[4]) {
    if constexpr (kSquares) sq[i] = add_four(x, make_float4(x[0], x[1], x[2], x[3]), sq[i]);
  };
  const T* w[FEW_AT_ONCE];
#pragma unroll
  for (int i = 0; i < FEW_AT_ONCE; ++i)         // (rows behind the last are the last's; nobody looks at them)
    w[i] = static_cast<const T*>(p.W) + min(v0 + i, p.vocab - 1) * p.ldw;
  constexpr int V = 16 / (int)sizeof(T);
  if constexpr (kRead == WORDS) {
#pragma unroll 2
    for (int c = lane * V; c < p.dim; c += 32 * V) {
      uint4 q[FEW_AT_ONCE];
#pragma unroll
      for (int i = 0; i < FEW_AT_ONCE; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(w[i] + c));
#pragma unroll
      for (int k = 0; k < V; k += 4) {
        float x[FEW_AT_ONCE][4];
#pragma unroll
        for (int i = 0; i < FEW_AT_ONCE; ++i) {
          four_of(q[i], k, x[i], static_cast<const T*>(nullptr));
          square(i, x[i]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 y = *reinterpret_cast<const float4*>(h + r * dp + c + k);
#pragma unroll
          for (int i = 0; i < FEW_AT_ONCE; ++i) v[i * R + r] = add_four(x[i], y, v[i * R + r]);
        }
      }
    }
  } else if constexpr (kRead == SHIFTED) {
    const int dq = dp + FEW_REST;
    int o[FEW_AT_ONCE];                         // elements of the row's first word before it
    const float* y0[FEW_AT_ONCE];
#pragma unroll
    for (int i = 0; i < FEW_AT_ONCE; ++i) {
      o[i] = rows::behind(w[i]);
      w[i] -= o[i];
      y0[i] = h + (o[i] & 3) * R * dq + FEW_LEAD - (o[i] & ~3);
    }
    const auto step = [&](int c, auto kind) {
      constexpr bool edge = decltype(kind)::value;
      if (edge && c >= p.dim + V - 1) return;   // (the copies end there)
      uint4 q[FEW_AT_ONCE];
#pragma unroll
      for (int i = 0; i < FEW_AT_ONCE; ++i)
        q[i] = !edge || c < p.dim + o[i] ? __ldg(reinterpret_cast<const uint4*>(w[i] + c)) : make_uint4(0, 0, 0, 0);
      if constexpr (edge) {
#pragma unroll
        for (int i = 0; i < FEW_AT_ONCE; ++i) q[i] = rows::masked_word<T>(q[i], o[i] - c, p.dim + o[i] - c);
      }
#pragma unroll
      for (int k = 0; k < V; k += 4)
#pragma unroll
        for (int i = 0; i < FEW_AT_ONCE; ++i) {
          float x[4];
          four_of(q[i], k, x, static_cast<const T*>(nullptr));
          square(i, x);
#pragma unroll
          for (int r = 0; r < R; ++r)
            v[i * R + r] = add_four(x, *reinterpret_cast<const float4*>(y0[i] + r * dq + c + k), v[i * R + r]);
        }
    };
    // words that reach over the row's ends are masked: in the first step and the last ones
    constexpr int STEP = 32 * V;
    int c = lane * V, c0 = STEP;
    step(c, std::true_type());
#pragma unroll 2
    for (; c0 + STEP <= p.dim; c0 += STEP) step(c += STEP, std::false_type());
#pragma unroll 1
    for (; c0 < p.dim + V - 1; c0 += STEP) step(c += STEP, std::true_type());
  } else {
    constexpr int H = 4;                        // elements in flight
    for (int c0 = lane; c0 < p.dim; c0 += 32 * H) {
      float x[H][FEW_AT_ONCE];
#pragma unroll
      for (int k = 0; k < H; ++k)
#pragma unroll
        for (int i = 0; i < FEW_AT_ONCE; ++i) x[k][i] = c0 + 32 * k < p.dim ? ld1(w[i] + c0 + 32 * k) : 0.f;
#pragma unroll
      for (int k = 0; k < H; ++k) {
        if constexpr (kSquares) {
#pragma unroll
          for (int i = 0; i < FEW_AT_ONCE; ++i) sq[i] = fmaf(x[k][i], x[k][i], sq[i]);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float y = c0 + 32 * k < p.dim ? h[r * dp + c0 + 32 * k] : 0.f;
#pragma unroll
          for (int i = 0; i < FEW_AT_ONCE; ++i) v[i * R + r] = fmaf(x[k][i], y, v[i * R + r]);
        }
      }
    }
  }
  if constexpr (kSquares) {
    const bool a = lane & 16, b = lane & 8;
    sq[0] = (a ? sq[2] : sq[0]) + __shfl_xor_sync(0xffffffffu, a ? sq[0] : sq[2], 16);
    sq[1] = (a ? sq[3] : sq[1]) + __shfl_xor_sync(0xffffffffu, a ? sq[1] : sq[3], 16);
    sq[0] = (b ? sq[1] : sq[0]) + __shfl_xor_sync(0xffffffffu, b ? sq[0] : sq[1], 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sq[0] += __shfl_xor_sync(0xffffffffu, sq[0], o);
    squares = sq[0];
  }
  // each exchange halves what a lane holds, as long as there is more than one
  int n = N;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < N / 2; ++i)
        if (i < n) {
          const float keep = up ? v[i + n] : v[i], give = up ? v[i] : v[i + n];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return make_float2(v[0], N > 32 ? v[1 % N] : 0.f);
}

// The shares of H's rows (in shared memory, each `len` numbers with zeros behind the row's), a warp a row.
template <typename T>
__device__ __forceinline__ void write_shares(const Few& p, const T* h, int len, int lane, int warp, float* share) {
  for (int r = warp; r < p.rows; r += FEW_WARPS) {
    constexpr int V = 16 / (int)sizeof(T);      // (a row's length here is a multiple of that)
    f32x2 sums = both(0.f);
    float most = 0.f;
#pragma unroll 4
    for (int c = lane * V; c < len; c += 32 * V) {
      f32x2 x[V / 2];
      widen_word(*reinterpret_cast<const uint4*>(h + (size_t)r * len + c), x, static_cast<const T*>(nullptr));
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        sums = fma2(x[i], x[i], sums);
        most = fmaxf(most, fmaxf(fabsf(lo2(x[i])), fabsf(hi2(x[i]))));
      }
    }
    const float s = warp_sum(lo2(sums) + hi2(sums));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    if (lane == 0) share[r] = share_of(s, most, p.share);
  }
}

// A row's statistic of a block of logits, its keys and its token's logit, by a warp.  z: the row's
// first of kParts shares of the logits, which lie `apart`; share and squares: for the keys,
// the row's share and kParts shares of the squares of W's rows.
template <int kBlock, int kParts, bool kKeys>
__device__ __forceinline__ void write_block(const Few& p, const float* z, int apart, int r, int blk, int lane, float share,
                                            const float* squares) {
  constexpr int G = kBlock / KEY_COLS;
  const long long b0 = (long long)blk * kBlock;
  float x[G], mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    float v = z[32 * j + lane];
#pragma unroll
    for (int i = 1; i < kParts; ++i) v += z[i * apart + 32 * j + lane];
    x[j] = b0 + 32 * j + lane < p.vocab ? v : -INFINITY;
    mx = fmaxf(mx, x[j]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  const float ref = mx == -INFINITY ? 0.f : mx;
  float s = 0.f, t = 0.f;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float d = x[j] - ref, e = __expf(d);
    s += e;
    t = fmaf(e, fmaxf(d, FEW_FLOOR), t);
  }
  s = warp_sum(s);
  t = warp_sum(t);
  if (lane == 0) p.stat[(size_t)r * p.parts + blk] = make_float4(mx, s, t, 0.f);
  if constexpr (kKeys) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      float sq = squares[32 * j + lane];
#pragma unroll
      for (int i = 1; i < kParts; ++i) sq += squares[i * kBlock + 32 * j + lane];
      const float most = fmaxf(fmaf(share, length_of(sq), x[j]), -0x1.fffffep127f);
      const float own = __uint_as_float((__float_as_uint(most) & ~KEY_MASK) | (KEY_MASK - lane));
      float a = own;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
      float b = own == a ? -INFINITY : own;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, o));
      if (lane == j) p.keys[((size_t)r * p.parts + blk) * G + j] = make_float2(a, b);
    }
  }
  const long long at = p.labels ? p.labels[r] - b0 : -1;
#pragma unroll
  for (int j = 0; j < G; ++j)
    if (at == 32 * j + lane && b0 + at < p.vocab) p.zlabel[r] = x[j];
}

template <typename T, int R, Read kRead, int kBlock, bool kKeys>
__global__ void __launch_bounds__(FEW_THREADS) few_forward_kernel(const Few p) {
  extern __shared__ __align__(16) float few_smem[];
  __shared__ float share[R], squares[kKeys ? kBlock : 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dp = p.dp;
  float* h = few_smem;                          // [R][dp], or the four copies
  float* z = h + (kRead == SHIFTED ? 4 * R * (dp + FEW_REST) : R * dp);   // [R][kBlock]
  allow_next();
  await_previous();
  if constexpr (kRead == SHIFTED) stage_copies<T, R>(p, h, dp + FEW_REST);
  else stage_rows<T, R>(p, h, dp);
  if constexpr (kKeys) {
    __syncthreads();
    write_shares(p, h, kRead == SHIFTED ? dp + FEW_REST : dp, lane, warp, share);
  }
  for (int blk = blockIdx.x; blk < p.parts; blk += gridDim.x) {
    __syncthreads();                            // h is staged; the last block's z are read
    const long long b0 = (long long)blk * kBlock;
    for (int i = warp * FEW_AT_ONCE; i < kBlock; i += FEW_PIECE) {
      if (b0 + i >= p.vocab) break;
      float sq = 0.f;
      const float2 v = products<T, R, kRead, kKeys>(p, h, dp, b0 + i, lane, sq);
      if (kKeys && lane % 8 == 0) squares[i + lane / 8] = sq;
      constexpr int N = FEW_AT_ONCE * R;
      if constexpr (N > 32) {
        const int at = lane * (N / 32);
        z[(at % R) * kBlock + i + at / R] = v.x;
        z[((at + 1) % R) * kBlock + i + (at + 1) / R] = v.y;
      } else if (lane % (32 / N) == 0) {
        const int at = lane / (32 / N);
        z[(at % R) * kBlock + i + at / R] = v.x;
      }
    }
    __syncthreads();
    for (int r = warp; r < p.rows; r += FEW_WARPS)
      write_block<kBlock, 1, kKeys>(p, z + r * kBlock, 0, r, blk, lane, kKeys ? share[r] : 0.f, squares);
  }
}

// bf16 rows of W from words, by matrix instructions: 16 rows of W are one's rows and 8 rows of H its
// columns, so that a warp takes W from global memory straight to registers, a lane 16 bytes of each of two
// rows, and H's word with the same columns from shared memory.  (The tensor cores' larger tiles would
// pass W through shared memory, and be filled to 1/32 by 8 rows.)  Which column of W stands at which k of an
// instruction does not matter as long as H's stands there too: a lane's four pairs are k
// 2t, 2t + 1 and 2t + 8, 2t + 9 of two of them.  Sums are taken over into fp32 numbers every 128 columns.
// Short blocks: two warps take 16 of the 32 columns each, of four quarters of the row; long
// ones: a warp takes 16 of the 128 columns.  The squares of W's rows (kKeys) are summed 16 pairs at a time in
// bf16 (within 2^-5, which the share allows for), then in fp32.
__device__ __forceinline__ void mma_16x8(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ float squares_of(const uint4 (&q)[N]) {
  __nv_bfloat162 s[2] = {__floats2bfloat162_rn(0.f, 0.f), __floats2bfloat162_rn(0.f, 0.f)};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&w[j]);
      s[j & 1] = __hfma2(x, x, s[j & 1]);
    }
  }
  const __nv_bfloat162 a = s[0], b = s[1];
  return (__low2float(a) + __high2float(a)) + (__low2float(b) + __high2float(b));
}
// A row of H is an odd multiple of 64 bytes long, so that eight lanes' words lie in different banks.
__host__ __device__ constexpr int mma_stride(int dim) { return (dim + 31) / 32 % 2 ? (dim + 31) / 32 * 32 : (dim + 63) / 32 * 32; }
template <int R, int kBlock, bool kKeys>
__global__ void __launch_bounds__(FEW_THREADS) few_mma_kernel(const Few p) {
  extern __shared__ __align__(16) float few_smem[];
  constexpr int S = kBlock == KEY_COLS ? 4 : 1, ZS = kBlock + 4, STEPS = 4;   // STEPS of 32 columns at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane / 4, t = lane % 4, ds = mma_stride(p.dim);
  bf16* h = reinterpret_cast<bf16*>(few_smem);  // [R][ds]
  float* z = reinterpret_cast<float*>(h + R * ds);   // [S][R][ZS]
  __shared__ float share[R], squares[kKeys ? S * kBlock : 1];
  allow_next();
  await_previous();
  for (int r = 0; r < R; ++r) {
    const bf16* x = static_cast<const bf16*>(p.H) + r * p.ldh;
    const bool live = r < p.rows, words = rows::behind(x) == 0;   // (the number of columns is a multiple of 8)
    for (int c = threadIdx.x * 8; c < ds; c += FEW_THREADS * 8) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (live && c < p.dim) {
        if (words) {
          q = *reinterpret_cast<const uint4*>(x + c);
        } else {
          bf16* e = reinterpret_cast<bf16*>(&q);
#pragma unroll
          for (int i = 0; i < 8; ++i) e[i] = x[c + i];
        }
      }
      *reinterpret_cast<uint4*>(h + r * ds + c) = q;
    }
  }
  const int group = S == 4 ? warp % 2 : warp, part = S == 4 ? warp / 2 : 0;
  const int chunks = (p.dim + 31) / 32, lo = chunks * part / S, hi = chunks * (part + 1) / S;
  const bf16* y = h + g * ds + t * 8;
  if constexpr (kKeys) {
    __syncthreads();
    write_shares(p, h, ds, lane, warp, share);
  }
  for (int blk = blockIdx.x; blk < p.parts; blk += gridDim.x) {
    __syncthreads();                            // h is staged; the last block's z are read
    const long long v0 = (long long)blk * kBlock + group * 16;
    if (v0 < p.vocab) {
      // (rows behind the last are the last's; nobody looks at them)
      const bf16* w0 = static_cast<const bf16*>(p.W) + min(v0 + g, p.vocab - 1) * p.ldw + t * 8;
      const bf16* w1 = static_cast<const bf16*>(p.W) + min(v0 + g + 8, p.vocab - 1) * p.ldw + t * 8;
      float sum[R / 8][4] = {}, first = 0.f, last = 0.f;
      for (int k = lo; k < hi; k += STEPS) {
        uint4 a[STEPS], b[STEPS];
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          const bool in = k + i < hi && (k + i) * 32 + t * 8 < p.dim;
          a[i] = in ? __ldg(reinterpret_cast<const uint4*>(w0 + (k + i) * 32)) : make_uint4(0, 0, 0, 0);
          b[i] = in ? __ldg(reinterpret_cast<const uint4*>(w1 + (k + i) * 32)) : make_uint4(0, 0, 0, 0);
        }
        float d[R / 8][4] = {};
        if constexpr (kKeys) {
          first += squares_of(a);
          last += squares_of(b);
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
          if (k + i >= hi) break;
#pragma unroll
          for (int n = 0; n < R / 8; ++n) {
            const uint4 c = *reinterpret_cast<const uint4*>(y + n * 8 * ds + (k + i) * 32);
            mma_16x8(d[n], a[i].x, b[i].x, a[i].y, b[i].y, c.x, c.y);
            mma_16x8(d[n], a[i].z, b[i].z, a[i].w, b[i].w, c.z, c.w);
          }
        }
#pragma unroll
        for (int n = 0; n < R / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[n][i] += d[n][i];
      }
#pragma unroll
      for (int n = 0; n < R / 8; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          z[(part * R + n * 8 + 2 * t + i % 2) * ZS + group * 16 + g + i / 2 * 8] = sum[n][i];
      if constexpr (kKeys) {
#pragma unroll
        for (int o = 1; o < 4; o *= 2) {        // (the four lanes of a row)
          first += __shfl_xor_sync(0xffffffffu, first, o);
          last += __shfl_xor_sync(0xffffffffu, last, o);
        }
        if (t == 0) squares[part * kBlock + group * 16 + g] = first;
        if (t == 1) squares[part * kBlock + group * 16 + g + 8] = last;
      }
    }
    __syncthreads();
    for (int r = warp; r < p.rows; r += FEW_WARPS)
      write_block<kBlock, S, kKeys>(p, z + r * ZS, R * ZS, r, blk, lane, kKeys ? share[r] : 0.f, squares);
  }
}

// The columns a thread takes at a time in the second half of a piece.
template <typename T, bool kVec> struct Columns {
  static constexpr int E = kVec ? 4 : 1;
};
__device__ __forceinline__ void load_columns(const float* p, float (&v)[4]) { ld4(p, v); }
__device__ __forceinline__ void load_columns(const bf16* p, float (&v)[4]) { ld4(p, v); }
template <typename T> __device__ __forceinline__ void load_columns(const T* p, float (&v)[1]) { v[0] = ld1(p); }
template <typename T> __device__ __forceinline__ void store_columns(T* p, const float (&v)[4]) { st4(p, v); }
template <typename T> __device__ __forceinline__ void store_columns(T* p, const float (&v)[1]) { st1(p, v[0]); }

// Pieces of FEW_PIECE rows of W: their logits and g, a warp four rows; then, a thread some
// columns, dW's rows (written) and their share of dH (kept in shared memory until the end).
// W's second read of a piece comes from L2.
template <typename T, int R, bool kVec>
__global__ void __launch_bounds__(FEW_THREADS) few_backward_kernel(const Few p) {
  extern __shared__ __align__(16) float few_smem[];
  __shared__ __align__(16) float g[FEW_PIECE][R < 4 ? 4 : R];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, dp = p.dp;
  float* h = few_smem;                          // [R][dp]
  float* dh = h + R * dp;                       // [R][dp]
  constexpr int N = FEW_AT_ONCE * R, E = Columns<T, kVec>::E;
  allow_next();
  await_previous();
  stage_rows<T, R>(p, h, dp);
  if (p.dh_part)
    for (int i = threadIdx.x; i < R * dp; i += FEW_THREADS) dh[i] = 0.f;
  // what g is made of in the row of H that this lane's product belongs to
  const int mine = lane / (N < 32 ? 32 / N : 1), row = mine % R;
  float a = 0.f, b = 0.f, lse = 0.f, ah = 0.f;
  long long label = -1;
  const bool lost = __ldcg(p.status) & DEV_TIMEOUT;
  if (row < p.rows) {
    const long long lab = p.labels[row];
    if (lab != p.ignore && lab >= 0 && lab < p.vocab) {
      label = lab;
      lse = p.lse[row];
      if (p.g_logprob) a = p.g_logprob[row];
      if (p.g_entropy) b = p.g_entropy[row];
      ah = b == 0.f && !p.g_entropy ? a : fmaf(b, p.entropy[row], a);
    }
  }
  for (long long v0 = (long long)blockIdx.x * FEW_PIECE; v0 < p.vocab; v0 += (long long)gridDim.x * FEW_PIECE) {
    __syncthreads();                            // h is staged; the last piece's g are read
    const long long w0 = v0 + warp * FEW_AT_ONCE;
    if (w0 < p.vocab) {
      float none;
      const float z = products<T, R, kVec ? WORDS : ELEMENTS, false>(p, h, dp, w0, lane, none).x;
      if (N >= 32 || lane % (32 / N) == 0) {
        const long long v = w0 + mine / R;
        const float d = z - lse;
        float x = -__expf(d) * fmaf(b, fmaxf(d, FEW_FLOOR), ah);
        if (v == label) x += a;
        if (label < 0) x = 0.f;                 // no gradient, whatever the row holds
        if (lost) x = __int_as_float(0x7FC00000);
        g[warp * FEW_AT_ONCE + mine / R][row] = x;
      }
    }
    __syncthreads();
    const int n = (int)min(p.vocab - v0, (long long)FEW_PIECE);
    for (int c = threadIdx.x * E; c < p.dim; c += FEW_THREADS * E) {
      float hc[R][E], dc[R][E];
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          hc[r][i] = h[r * dp + c + i];
          dc[r][i] = 0.f;
        }
      const T* w = static_cast<const T*>(p.W) + v0 * p.ldw + c;
      T* dw = static_cast<T*>(p.dW) + v0 * p.dim + c;
#pragma unroll 8
      for (int v = 0; v < n; ++v) {
        float x[E], o[E], gv[R];
        if (p.dh_part) load_columns(w + v * p.ldw, x);
#pragma unroll
        for (int r = 0; r < R; ++r) gv[r] = g[v][r];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            o[i] = fmaf(gv[r], hc[r][i], o[i]);
            if (p.dh_part) dc[r][i] = fmaf(gv[r], x[i], dc[r][i]);
          }
        if (p.dW) store_columns(dw + (long long)v * p.dim, o);
      }
      if (p.dh_part)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < E; ++i) dh[r * dp + c + i] += dc[r][i];
    }
  }
  if (p.dh_part) {
    __syncthreads();
    float* o = p.dh_part + (size_t)blockIdx.x * R * dp;
    for (int i = threadIdx.x; i < R * dp; i += FEW_THREADS) o[i] = dh[i];
  }
}

// dH from the CTAs' shares: 32 columns of a row a CTA, 8 threads a column over the shares
// (each a fixed set), joined in order.
template <typename T>
__global__ void __launch_bounds__(256) few_join_kernel(const float* part, int ctas, int R, int dp, int dim, T* dH) {
  __shared__ float sum[8][33];
  await_previous();
  const int c = blockIdx.x * 32 + threadIdx.x, r = blockIdx.y;
  float s = 0.f;
  if (c < dim) {
#pragma unroll 4
    for (int i = threadIdx.y; i < ctas; i += 8) s += part[((size_t)i * R + r) * dp + c];
  }
  sum[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y || c >= dim) return;
  for (int i = 1; i < 8; ++i) s += sum[i][threadIdx.x];
  st1(dH + (long long)r * dim + c, s);
}

int padded_rows(int64_t rows) { return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }
int mma_rows(int64_t rows) { return rows <= 8 ? 8 : 16; }
size_t forward_smem(int64_t rows, int64_t dim) { return padded_rows(rows) * (padded(dim) + FEW_BLOCK) * 4; }
size_t mma_smem(int64_t rows, int64_t dim) {
  return mma_rows(rows) * ((size_t)mma_stride((int)dim) * 2 + std::max<size_t>(4 * (KEY_COLS + 4), FEW_BLOCK + 4) * 4);
}
size_t copies_smem(int64_t rows, int64_t dim) { return padded_rows(rows) * (4 * (padded(dim) + FEW_REST) + FEW_BLOCK) * 4; }
size_t backward_smem(int64_t rows, int64_t dim) { return padded_rows(rows) * padded(dim) * 8; }
constexpr size_t FEW_SMEM = 200 * 1024, MMA_SMEM = 60 * 1024;

template <class K>
cudaError_t run(K kern, Few& p, size_t smem, int64_t work, int most, int* grid, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FEW_SMEM);
  if (e != cudaSuccess) return e;
  // as many CTAs as run at once; each takes pieces in turn
  int per_sm = 0, sms = 0;
  if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, FEW_THREADS, smem)) != cudaSuccess) return e;
  if (require_device(&sms) != MUON_OK) return cudaErrorNoDevice;
  *grid = (int)std::max<int64_t>(1, std::min<int64_t>({work, (int64_t)per_sm * sms, most}));
  count_launch();
  return launch_after(kern, dim3(*grid), dim3(FEW_THREADS), smem, s, p);
}
template <typename T, Read kRead, int kBlock>
cudaError_t forward_of(Few& p, cudaStream_t s) {
  int grid = 0;
  const size_t smem = kRead == SHIFTED ? copies_smem(p.rows, p.dim) : forward_smem(p.rows, p.dim);
  // (a lane's sum of one column in 32, and the tree)
  p.share = UNIT_FP32 * (float)(cdiv(p.dim, 32) + 16);
  auto go = [&](auto rows) {
    constexpr int R = decltype(rows)::value;
    return p.keys ? run(few_forward_kernel<T, R, kRead, kBlock, true>, p, smem, cdiv(p.vocab, kBlock), 1 << 30, &grid, s)
                  : run(few_forward_kernel<T, R, kRead, kBlock, false>, p, smem, cdiv(p.vocab, kBlock), 1 << 30, &grid, s);
  };
  const int R = padded_rows(p.rows);
  if (R == 1) return go(std::integral_constant<int, 1>());
  if constexpr (sizeof(T) == 4) {
    if (R == 4) return go(std::integral_constant<int, 4>());
    if (R == 8) return go(std::integral_constant<int, 8>());
    if (R == 16) return go(std::integral_constant<int, 16>());
  }
  return go(std::integral_constant<int, 2>());
}
template <typename T, int kBlock>
cudaError_t forward_by(Few& p, bool vec, cudaStream_t s) {
  if constexpr (sizeof(T) == 4) {
    if (vec) return forward_of<T, WORDS, kBlock>(p, s);
  } else {
    if (vec) {
      int grid = 0;
      const int R = mma_rows(p.rows);
      // (eight instructions, and a take-over every 128 columns)
      p.share = 1.02f * UNIT_TENSOR * (float)(cdiv(p.dim, 128) + 16);
      auto go = [&](auto kern) { return run(kern, p, mma_smem(p.rows, p.dim), cdiv(p.vocab, kBlock), 1 << 30, &grid, s); };
      if (p.keys) return R == 8 ? go(few_mma_kernel<8, kBlock, true>) : go(few_mma_kernel<16, kBlock, true>);
      return R == 8 ? go(few_mma_kernel<8, kBlock, false>) : go(few_mma_kernel<16, kBlock, false>);
    }
    if (copies_smem(p.rows, p.dim) <= FEW_SMEM / 2) return forward_of<T, SHIFTED, kBlock>(p, s);
  }
  return forward_of<T, ELEMENTS, kBlock>(p, s);
}
template <typename T, bool kVec>
cudaError_t backward_of(Few& p, T* dH, cudaStream_t s) {
  int grid = 0;
  const int R = padded_rows(p.rows);
  const size_t smem = backward_smem(p.rows, p.dim);
  auto go = [&](auto kern) { return run(kern, p, smem, cdiv(p.vocab, FEW_PIECE), FEW_MAX_CTAS, &grid, s); };
  cudaError_t e;
  if (R == 1) e = go(few_backward_kernel<T, 1, kVec>);
  else if (R == 2) e = go(few_backward_kernel<T, 2, kVec>);
  else if (sizeof(T) == 2 || R == 4) e = go(few_backward_kernel<T, 4, kVec>);
  else e = go(few_backward_kernel<T, sizeof(T) == 2 ? 4 : 8, kVec>);
  if (e != cudaSuccess || !dH) return e;
  count_launch();
  return launch_after(few_join_kernel<T>, dim3(cdiv(p.dim, 32), p.rows), dim3(32, 8), 0, s, p.dh_part, grid, R, p.dp, p.dim, dH);
}

}  // namespace

// Up to how many rows this is the faster way (microseconds here and by tiles, 32768 x 1536):
// fp32 forward 16 rows 98 and 203, 8 rows 58 and 199, backward 4 rows 116 and 431, 8 rows 145 and
// 422; bf16 backward 1 row 66 and 98, 4 rows 74 and 99, 8 rows 118 and 98; bf16 forward in words 8 rows 21 and
// 29, with 8 alternatives (where tiles read W once more for its rows' lengths, and these sum their squares on
// the way) 36 and 62, 16 rows 29 and 29, 45 and 62, 24 rows 51 and 30; of 131072 x 2560 8 rows 122 and 128.  Longer rows leave an SM fewer warps (32768 x 4096, 8 rows 74 and 61): tiles.
// bf16 rows off the words: 1 row of 50257 x 2501 57 and 150, 4 rows have no kernel here.
bool few_rows(int64_t rows, int64_t dim, bool f32, bool backward, bool vec) {
  if (rows < 1 || dim >= (1 << 20)) return false;
  if (backward) return rows <= (f32 ? 8 : 4) && backward_smem(rows, dim) <= FEW_SMEM;
  if (!f32 && vec) return rows <= 16 && mma_smem(rows, dim) <= MMA_SMEM;
  return rows <= (f32 ? 16 : 2) && forward_smem(rows, dim) <= FEW_SMEM;
}
size_t few_bytes(int64_t rows, int64_t dim) { return (size_t)FEW_MAX_CTAS * padded_rows(rows) * padded(dim) * 4; }

// Columns of a statistic: short blocks where long ones are fewer than two an SM (microseconds, short and
// long: fp32 1 row of 1622 x 2240 10 and 26, of 32768 x 1536 43 and 49, of 50257 x 1536 62 and 58; bf16 8 rows of
// 32768 x 1536 21 and 23, of 131072 x 512 36 and 33).
int few_block(int64_t vocab) { return vocab < 2LL * 152 * FEW_BLOCK ? KEY_COLS : FEW_BLOCK; }

cudaError_t few_forward(Few p, bool f32, bool vec, cudaStream_t s) {
  p.dp = (int)padded(p.dim);
  p.masked = 0;
  if (few_block(p.vocab) == KEY_COLS) return f32 ? forward_by<float, KEY_COLS>(p, vec, s) : forward_by<bf16, KEY_COLS>(p, vec, s);
  return f32 ? forward_by<float, FEW_BLOCK>(p, vec, s) : forward_by<bf16, FEW_BLOCK>(p, vec, s);
}
cudaError_t few_backward(Few p, bool f32, bool vec, void* dH, cudaStream_t s) {
  p.dp = (int)padded(p.dim);
  p.masked = 1;
  if (!dH) p.dh_part = nullptr;
  if (f32)
    return vec ? backward_of<float, true>(p, static_cast<float*>(dH), s) : backward_of<float, false>(p, static_cast<float*>(dH), s);
  return vec ? backward_of<bf16, true>(p, static_cast<bf16*>(dH), s) : backward_of<bf16, false>(p, static_cast<bf16*>(dH), s);
}

}  // namespace ce
}  // namespace muon
