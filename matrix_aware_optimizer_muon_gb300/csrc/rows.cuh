// Rows in registers, for the norms: a thread's share of a row as 16-byte vectors or single
// elements, the weights beside it, sums over the threads of a row, and what the host side
// asks of sizes and alignments.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace rows {

// Weights come as fp32 or bf16 (a flag: they are read from L1, the branch is uniform).
__device__ __forceinline__ float ld_w(const void* w, int w_bf16, int c) {
  return w_bf16 ? ld1(static_cast<const bf16*>(w) + c) : static_cast<const float*>(w)[c];
}
__device__ __forceinline__ void st_w(void* w, int w_bf16, int c, float v) {
  if (w_bf16) st1(static_cast<bf16*>(w) + c, v);
  else static_cast<float*>(w)[c] = v;
}

// A thread's share of a row: kN accesses of kV elements (16 bytes, or one element),
// `stride` elements apart, as pairs.  What lies past the row reads as zero.
template <int kV, int kN> struct Share {
  static constexpr int E = kV * kN;
  static constexpr int P = (E + 1) / 2;
};
template <typename T> constexpr int vec_of() { return 16 / (int)sizeof(T); }
__device__ __forceinline__ float elem(const f32x2* v, int i) { return i & 1 ? hi2(v[i / 2]) : lo2(v[i / 2]); }

// 16 bytes of the row as loaded, to pairs.
__device__ __forceinline__ void widen(const uint4& q, f32x2* v, const bf16*) {
  v[0] = cvt2(q.x); v[1] = cvt2(q.y); v[2] = cvt2(q.z); v[3] = cvt2(q.w);
}
__device__ __forceinline__ void widen(const uint4& q, f32x2* v, const float*) {
  v[0] = make2(__uint_as_float(q.x), __uint_as_float(q.y));
  v[1] = make2(__uint_as_float(q.z), __uint_as_float(q.w));
}
__device__ __forceinline__ void store16(bf16* p, const f32x2* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(lo2(v[0]), hi2(v[0])), pack_bf16x2(lo2(v[1]), hi2(v[1])),
                                            pack_bf16x2(lo2(v[2]), hi2(v[2])), pack_bf16x2(lo2(v[3]), hi2(v[3])));
}
__device__ __forceinline__ void store16(float* p, const f32x2* v) {
  *reinterpret_cast<float4*>(p) = make_float4(lo2(v[0]), hi2(v[0]), lo2(v[1]), hi2(v[1]));
}

// The row's raw registers, all loads in flight together.
template <typename T, int kV, int kN> struct Raw {
  uint4 q[kN];
  template <int kSure = 0>
  __device__ __forceinline__ void load(const T* x, int t, int size, int dim) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int c = (k * size + t) * kV;
      q[k] = k < kSure || c < dim ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void get(int k, f32x2* v) const { widen(q[k], v, static_cast<const T*>(nullptr)); }
  // keeps the compiler from holding widened values across this point
  __device__ __forceinline__ void hold() {
#pragma unroll
    for (int k = 0; k < kN; ++k) asm volatile("" : "+r"(q[k].x), "+r"(q[k].y), "+r"(q[k].z), "+r"(q[k].w));
  }
};
template <typename T, int kN> struct Raw<T, 1, kN> {
  T e[kN];
  template <int kSure = 0>
  __device__ __forceinline__ void load(const T* x, int t, int size, int dim) {
#pragma unroll
    for (int k = 0; k < kN; ++k) e[k] = k < kSure || k * size + t < dim ? x[k * size + t] : from_f32<T>(0.f);
  }
  __device__ __forceinline__ void get(int k, f32x2* v) const { v[0] = make2(to_f32(e[k]), 0.f); }
  __device__ __forceinline__ void hold() {}
  __device__ __forceinline__ void pairs(f32x2* v) const {
#pragma unroll
    for (int k = 0; k < kN; k += 2) v[k / 2] = make2(to_f32(e[k]), k + 1 < kN ? to_f32(e[(k + 1) % kN]) : 0.f);
  }
};
template <typename T, int kV, int kN, int kSure>
__device__ __forceinline__ void store_row(T* y, const f32x2* v, int t, int size, int dim) {
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int c = (k * size + t) * kV;
    if (k < kSure || c < dim) {
      if constexpr (kV > 1) store16(y + c, v + k * (kV / 2));
      else st1(y + c, elem(v, k));
    }
  }
}

// What the weights are: asked at run time, or known to be all there in one type (the
// forward pass's common cases: asking costs it a sixth of its instructions).
enum { W_ASK = 0, W_F32 = 1, W_BF16 = 2 };

// The weights of access k (with kV > 1 their vectors are aligned too); `none` without any.
template <int kV, int kW = W_ASK>
__device__ __forceinline__ void weights(const void* w, int w_bf16, int c, int dim, float none, f32x2* v) {
  if constexpr (kV == 1) {
    v[0] = both(c < dim ? (w ? ld_w(w, w_bf16, c) : none) : 0.f);
  } else if (kW == W_ASK && (c >= dim || !w)) {
#pragma unroll
    for (int i = 0; i < kV / 2; ++i) v[i] = both(c < dim ? none : 0.f);
  } else if (kW == W_BF16 || (kW == W_ASK && w_bf16)) {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i) {
      const uint2 q = *reinterpret_cast<const uint2*>(static_cast<const bf16*>(w) + c + 4 * i);
      v[2 * i] = cvt2(q.x);
      v[2 * i + 1] = cvt2(q.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kV / 4; ++i) {
      const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(w) + c + 4 * i);
      v[2 * i] = make2(q.x, q.y);
      v[2 * i + 1] = make2(q.z, q.w);
    }
  }
}

// The threads of one row: a warp, or `size` threads with a barrier of their own.
struct Group {
  int t, size, id;       // thread, threads, barrier (0: the whole CTA's)
  float* red;            // 2 x 32 floats
  __device__ __forceinline__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(size) : "memory"); }
  // Sums of a and b over the group.  The halves of a warp take one of the two each after the
  // first exchange; the warps' sums are added in order by everyone.
  __device__ __forceinline__ float2 sum(float a, float b, int parity) const {
    const bool up = t & 16;
    float v = up ? b : a;
    v += __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (size == 32) return make_float2(__shfl_sync(0xffffffffu, v, 0), __shfl_sync(0xffffffffu, v, 16));
    // two buffers in turn: a warp may be one reduction ahead of the slowest
    float* slot = red + 64 * parity;
    if ((t & 15) == 0) slot[t >> 4] = v;
    sync();
    f32x2 q = both(0.f);
    for (int i = 0; i < size >> 5; ++i) q = add2(q, *reinterpret_cast<const f32x2*>(slot + 2 * i));
    return make_float2(lo2(q), hi2(q));
  }
};

// How many of a thread's n accesses lie inside the row for every thread: the launcher takes
// the least n that covers the row out of 1 .. 8, 10, 12, 16.
__host__ __device__ constexpr int sure_of(int n) { return n <= 8 ? n - 1 : n <= 12 ? n - 2 : n - 4; }

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// A row that starts off a 16-byte word: elements between the word's start and the row's.
template <typename T> __device__ __forceinline__ int behind(const T* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
}
// A word's elements outside [lo, hi) become zeros.
template <typename T>
__device__ __forceinline__ uint4 masked_word(uint4 q, int lo, int hi) {
  T* x = reinterpret_cast<T*>(&q);
#pragma unroll
  for (int i = 0; i < 16 / (int)sizeof(T); ++i)
    if (i < lo || i >= hi) x[i] = from_f32<T>(0.f);
  return q;
}

inline bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
inline bool known(int dt) { return dt == MUON_DTYPE_F32 || dt == MUON_DTYPE_BF16; }
// (so that a column or a row past the end by a block's stride still fits an int)
inline bool sizes_ok(int64_t rows, int64_t dim) { return rows >= 0 && rows <= (1LL << 30) && dim >= 1 && dim <= (1LL << 30); }

inline int cdiv(long long a, long long b) { return (int)((a + b - 1) / b); }

// Whether rows of p (ld elements apart) and the weights can be read in 16-byte vectors.
inline bool vec_rows(const void* p, int64_t ld, int64_t rows, size_t es) {
  return is_aligned(p, 16) && (rows <= 1 || (size_t)ld * es % 16 == 0);
}

// f(std::integral_constant<int, N>) for the least N of sure_of's list that is >= need.
template <class F>
bool by_accesses(int need, F f) {
  switch (need <= 8 ? need : need <= 10 ? 10 : need <= 12 ? 12 : 16) {
#define MUON_ROWS_N(N) \
  case N: f(std::integral_constant<int, N>()); return need <= 16;
    MUON_ROWS_N(1) MUON_ROWS_N(2) MUON_ROWS_N(3) MUON_ROWS_N(4) MUON_ROWS_N(5) MUON_ROWS_N(6) MUON_ROWS_N(7) MUON_ROWS_N(8)
    MUON_ROWS_N(10) MUON_ROWS_N(12) MUON_ROWS_N(16)
#undef MUON_ROWS_N
  }
  return false;
}

}  // namespace rows
}  // namespace muon
