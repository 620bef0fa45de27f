// Softmax cross entropy of the logits z = H W^T, without keeping the logits.
//
//   forward:  per row and 128 columns of the vocabulary, max and sum of exponentials
//             (in the product's epilogue); lse = max + log(sum) joined over them;
//             loss = lse - z[label].
//   backward: g = c (exp(z - lse) - onehot) by pieces of the vocabulary;
//             dH += g W_piece,  dW_piece = g^T H.
//
// Log probabilities of given tokens, entropy and the largest logits, likewise:
//
//   forward:  lse and z[token] as above; with S = sum e^(z-m) and T = sum e^(z-m) (z-m)
//             (m the row's max) the entropy is log S - T/S; the two largest logits of each
//             32 columns, from which the alternatives are chosen and ranked (top_kernel).
//   backward: g = a (onehot - p) - b p (log p + H), a and b the gradients of log probability
//             and entropy; the same two products.
//
// The products run in ce_gemm.cu (those of a few rows' log probabilities in
// logprob_few.cu); here are the plan of a call, the join and the copies
// that bring operands into a layout TMA can read.
//
// Log probabilities measured: 8192 x 2560 x 131072 bf16 forward 3.1 to 3.3 ms without
// alternatives (1.66 to 1.77 PFLOP/s), 3.6 to 3.7 with 8, backward 10.5; 1021 x 1536 x 50257 bf16
// 119 and, with 5, 178 us; 8 x 1536 x 32768 bf16 25 and 35.  Alternatives cost the product's
// epilogue 7% (their keys), the lengths of W's rows a pass over W (26 us for 154 MB), and their
// kernel 8 us for 8 rows, 25 for 1021.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "ce.h"
#include "common.cuh"

namespace muon {
namespace ce {
namespace {

constexpr size_t HEADER = 256;     // status word, join ticket
constexpr int TICKET_WORD = 16;    // of the header

// A piece's g is rows x piece bf16 (three times that for 32-bit operands), twice: one
// piece is multiplied while the next is computed.  Every piece costs a launch and a pass
// over dH's sums.  8192 x 2560 x 131072 backward: 48 MB 11.1 ms, 96 10.6, 192 10.5, 384
// 10.3, 1024 10.2.
constexpr int64_t G_BYTES = 512 << 20;
constexpr int64_t MIN_PIECE = 2048;
constexpr int MAX_SPLITS = 16;
// K steps (of 64) between take-overs of the tensor cores' sums into registers (for 32-bit
// operands, of the leading parts' products).  Error against 64 bits and time: bf16 forward
// 2560 wide, 8 steps 2.1e-7 of lse, 20 steps 5.1e-7, one take-over at the end 1.0e-6, and for
// 8192 x 131072 3.44, 3.20 and 3.17 ms; 32-bit 1021 x 1001 x 10007 backward, 4 steps 3.9e-7
// of dH and 314 us, 8 steps 6.9e-7 and 304, 16 steps 1.3e-6 and 302.
constexpr int SEG_BF16 = 20, SEG_F32 = 4;
// The same for bf16 products whose sums are rounded to bf16 (the backward pass).  Up to 2^16
// products of one sign the truncation's bias is 3e-4, well below that rounding's 4e-3, and a
// launch of no longer sums takes the form without take-overs; it grows in proportion (2^22
// rows: 2.4e-2 of dW).
constexpr int SEG_LONG = 1024;
// The log probabilities' products: segments of one length, SEG_BF16 steps at most; short ones
// where a single row of tiles waits for W anyway (one row's log probability may be small against
// its logits, and the logits' error is its own).
constexpr int SEG_FEW = 12;

size_t up(size_t x) { return (x + 255) / 256 * 256; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// ---------------------------------------------------------------------------
// small kernels
// ---------------------------------------------------------------------------

// Rows whose label carries no gradient become zeros: dW sums g^T H over all rows, and a
// zero of g times a NaN or an infinity that such a row may hold (padding) would be NaN.
struct RowMask {
  const int64_t* labels;   // null: every row as it is
  long long vocab, ignore;
};
__device__ __forceinline__ bool masked(const RowMask& k, long long r) {
  if (!k.labels) return false;
  const long long lab = k.labels[r];
  return lab == k.ignore || lab < 0 || lab >= k.vocab;
}

// Rows of any stride and alignment to bf16 rows of ldo elements (a multiple of 8):
// bf16 as it is, fp32 as `parts` bf16 numbers that add up to it (8 bits each).  A warp a
// row, a lane two neighbouring columns of each 64, PACK_HELD of them in flight.
// A part that more parts follow stays within bf16's range: fp32's largest numbers (a mask of
// the type's lowest value) would round to an infinity and leave a NaN for the next.  What no
// part can hold, infinities and NaN, is left to the last one, which is multiplied with the other
// operand's leading part alone.
constexpr float BF16_MAX = 0x1.FEp127f;
__device__ __forceinline__ float in_bf16_range(float x) { return fminf(fmaxf(x, -BF16_MAX), BF16_MAX); }
constexpr int PACK_HELD = 8;
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(const T* in, long long ld, long long rows, int dim, bf16* out,
                                                   long long ldo, int parts, long long part_stride, RowMask mask) {
  allow_next();
  await_previous();
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const bool zero = masked(mask, r);
  const T* x = in + r * ld;
  for (int c0 = (threadIdx.x & 31) * 2; c0 < dim; c0 += 64 * PACK_HELD) {
    float a[PACK_HELD], b[PACK_HELD];
#pragma unroll
    for (int i = 0; i < PACK_HELD; ++i) {
      const int c = c0 + 64 * i;
      a[i] = c < dim && !zero ? ld1(x + c) : 0.f;
      b[i] = c + 1 < dim && !zero ? ld1(x + c + 1) : 0.f;
    }
    bf16* o = out + r * ldo + c0;
    for (int q = 0; q < parts; ++q, o += part_stride) {
#pragma unroll
      for (int i = 0; i < PACK_HELD; ++i) {
        const uint32_t w = q + 1 < parts ? pack_bf16x2(in_bf16_range(a[i]), in_bf16_range(b[i])) : pack_bf16x2(a[i], b[i]);
        if (c0 + 64 * i < dim) *reinterpret_cast<uint32_t*>(o + 64 * i) = w;
        a[i] -= __uint_as_float(w << 16);
        b[i] -= __uint_as_float(w & 0xFFFF0000u);
      }
    }
  }
}

// The same for bf16 rows that are whole 16-byte vectors, ldo = dim.
__global__ void __launch_bounds__(256) mask_kernel(const bf16* in, long long ld, long long rows, int dim, bf16* out,
                                                   RowMask mask) {
  allow_next();
  await_previous();
  const long long r = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (r >= rows) return;
  const bool zero = masked(mask, r);
  const uint4* x = reinterpret_cast<const uint4*>(in + r * ld);
  uint4* o = reinterpret_cast<uint4*>(out + r * dim);
  for (int c0 = threadIdx.x & 31; c0 < dim / 8; c0 += 32 * PACK_HELD) {
    uint4 v[PACK_HELD];
#pragma unroll
    for (int i = 0; i < PACK_HELD; ++i)
      v[i] = c0 + 32 * i < dim / 8 && !zero ? x[c0 + 32 * i] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < PACK_HELD; ++i)
      if (c0 + 32 * i < dim / 8) o[c0 + 32 * i] = v[i];
  }
}

// What the keys of the log probabilities' tiles need of the operands: the lengths of W's rows, by
// column and the largest of each KEY_COLS (minus one where one is four times as long as another: these are
// told apart, for a few long rows would raise their neighbours' bounds too), and the shares of H's
// rows.  A CTA has KEY_COLS rows, a warp four.  W is read once more for them, at 5 to 6 TB/s, from its end
// on: the product starts with what was read last.
struct Lengths {
  const void *h, *w;
  long long ldh, ldw, rows, vocab;
  int dim, hvec, wvec, groups;       // vec: rows in 16-byte words
  float share;
  float *hshare, *wlen, *wgroup;
};
template <typename T>
__global__ void __launch_bounds__(256) lengths_kernel(const Lengths p) {
  constexpr int V = 16 / (int)sizeof(T), N = 4, HELD = 2;
  __shared__ float all[KEY_COLS];
  allow_next();
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool is_h = (int)blockIdx.x >= p.groups;
  const long long block = is_h ? (long long)blockIdx.x - p.groups : p.groups - 1 - (long long)blockIdx.x;
  const long long rows = is_h ? p.rows : p.vocab, r0 = block * KEY_COLS + warp * N;
  const T* x[N];
#pragma unroll
  for (int i = 0; i < N; ++i)        // (rows behind the last are the last's)
    x[i] = static_cast<const T*>(is_h ? p.h : p.w) + min(r0 + i, rows - 1) * (is_h ? p.ldh : p.ldw);
  f32x2 s[N];
  float most[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = both(0.f);
    most[i] = 0.f;
  }
  auto take = [&](int i, float a, float b) {
    s[i] = fma2(make2(a, b), make2(a, b), s[i]);
    if (is_h) most[i] = fmaxf(most[i], fmaxf(fabsf(a), fabsf(b)));
  };
  const int dim = r0 < rows ? p.dim : 0, words = (is_h ? p.hvec : p.wvec) ? dim / V : 0;
  for (int c0 = lane; c0 < words; c0 += 32 * HELD) {
    uint4 q[N][HELD];
#pragma unroll
    for (int k = 0; k < HELD; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i)
        q[i][k] = c0 + 32 * k < words ? reinterpret_cast<const uint4*>(x[i])[c0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < HELD; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t w[4] = {q[i][k].x, q[i][k].y, q[i][k].z, q[i][k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (sizeof(T) == 2) take(i, __uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xFFFF0000u));
          else if (j % 2 == 0) take(i, __uint_as_float(w[j]), __uint_as_float(w[(j + 1) % 4]));
        }
      }
  }
  for (int c = words * V + lane; c < dim; c += 32)
#pragma unroll
    for (int i = 0; i < N; ++i) take(i, ld1(x[i] + c), 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float sum = warp_sum(lo2(s[i]) + hi2(s[i]));
    if (is_h) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) most[i] = fmaxf(most[i], __shfl_xor_sync(0xffffffffu, most[i], o));
      if (lane == 0 && r0 + i < rows) p.hshare[r0 + i] = share_of(sum, most[i], p.share);
    } else if (lane == 0) {
      all[warp * N + i] = length_of(sum);
    }
  }
  if (is_h) return;
  __syncthreads();
  if (warp) return;
  const long long v = block * KEY_COLS + lane;
  const float len = all[lane];
  float hi = len, lo = len;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
  }
  p.wlen[v] = len;
  if (lane == 0) p.wgroup[block] = hi > 4.f * lo ? -1.f : hi;
}

// Whether a wait of this call's products (or of an earlier call that nobody asked about) ran
// out: what they left unwritten must not pass for a result, so the last kernel of a call
// writes NaN instead.  A caller without a workspace to ask sees it too.
__device__ __forceinline__ bool is_lost(const unsigned int* status) { return __ldcg(status) & DEV_TIMEOUT; }
__device__ __forceinline__ float not_a_number() { return __int_as_float(0x7FC00000); }
template <typename T>
__device__ void fill_lost(T* p, long long n) {
  if (!p) return;
  for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
    st1(p + i, not_a_number());
}

// One warp a row: joins its partial sums (JOIN_HELD a lane at a time), writes lse and
// loss.  Each block adds its rows' losses up; the last block to finish adds the blocks'.
constexpr int JOIN_WARPS = 8;
constexpr int JOIN_HELD = 8;   // partial sums a lane keeps at a time
__global__ void __launch_bounds__(32 * JOIN_WARPS) join_kernel(const float2* part, int parts, long long rows,
                                                               const int64_t* labels, long long vocab, long long ignore,
                                                               const float* zlabel, float* loss, float* lse,
                                                               float* stats, float2* sums, unsigned int* ticket,
                                                               const unsigned int* status) {
  __shared__ float red[32];
  __shared__ float2 mine[JOIN_WARPS];
  __shared__ bool last;
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r = (long long)blockIdx.x * JOIN_WARPS + warp;
  float2 sum = make_float2(0.f, 0.f);   // this row's loss, and 1 if it counts
  const bool lost = is_lost(status);
  if (r < rows && lost) {
    sum = make_float2(not_a_number(), not_a_number());
    if (lane == 0) lse[r] = loss[r] = not_a_number();
  } else if (r < rows) {
    const float2* q = part + (size_t)r * parts;
    const long long lab = labels[r];
    const bool counted = lab != ignore, known = counted && lab >= 0 && lab < vocab;
    const float zl = known ? zlabel[r] : 0.f;
    float mx = -INFINITY, s = 0.f;
    for (int t0 = 0; t0 < parts; t0 += 32 * JOIN_HELD) {
      float2 w[JOIN_HELD];
      float m = mx;
#pragma unroll
      for (int i = 0; i < JOIN_HELD; ++i) {
        const int t = t0 + 32 * i + lane;
        w[i] = t < parts ? q[t] : make_float2(-INFINITY, 0.f);
      }
#pragma unroll
      for (int i = 0; i < JOIN_HELD; ++i) m = fmaxf(m, w[i].x);
      const float ref = m == -INFINITY ? 0.f : m;
      s = mx == -INFINITY ? s : s * expf(mx - ref);
#pragma unroll
      for (int i = 0; i < JOIN_HELD; ++i) s += w[i].x == -INFINITY ? w[i].y : w[i].y * expf(w[i].x - ref);
      mx = m;
    }
    float top = mx;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float ref = top == -INFINITY ? 0.f : top;
    s = warp_sum(mx == -INFINITY ? s : s * expf(mx - ref));
    const float l = ref + logf(s);
    const float x = known ? l - zl : counted ? not_a_number() : 0.f;
    if (lane == 0) {
      lse[r] = l;
      loss[r] = x;
    }
    sum = make_float2(x, counted ? 1.f : 0.f);
  }
  if (!stats) return;
  if (lane == 0) mine[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 b = make_float2(0.f, 0.f);
    for (int i = 0; i < JOIN_WARPS; ++i) { b.x += mine[i].x; b.y += mine[i].y; }
    mine[0] = b;
    last = true;
    if (gridDim.x > 1) {
      sums[blockIdx.x] = b;
      __threadfence();
      last = atomicAdd(ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  float s = mine[0].x, c = mine[0].y;
  if (gridDim.x > 1) {
    __threadfence();
    s = c = 0.f;
    for (unsigned i = threadIdx.x; i < gridDim.x; i += 32 * JOIN_WARPS) {
      const float2 b = __ldcg(sums + i);
      s += b.x;
      c += b.y;
    }
    s = block_sum(s, red);
    c = block_sum(c, red);
  }
  if (threadIdx.x == 0) {
    stats[0] = s / fmaxf(c, 1.f);
    stats[1] = c;
    *ticket = 0;
  }
}

// ---------------------------------------------------------------------------
// log probabilities: the join and the alternatives
// ---------------------------------------------------------------------------
struct LogprobRows {
  const float4* stat;        // [row][parts]
  const float2* keys;        // [row][groups], with alternatives
  int parts, groups;
  long long rows;
  const int64_t* labels;     // or null: no token is given
  long long vocab, ignore;
  const float* zlabel;
  float *logprob, *entropy, *lse;
  const unsigned int* status;
  // alternatives
  const void *H, *W;
  long long ldh, ldw;
  int dim, top, vec;
  long long* ids;
  float* alternatives;
};

// A running max with the sums that are relative to it.
struct Moments {
  float m, s, t;
};
// Adds sums relative to w.x, made relative to `ref` >= w.x.  A part whose max is minus
// infinity has sums of 0, or NaN where it holds one; one far below ref adds nothing, whose
// distance has to stay finite.
__device__ __forceinline__ void add_moments(Moments& a, const float4& w, float ref) {
  const float d = fmaxf(w.x - ref, -1000.f), f = expf(d);
  const bool none = w.x == -INFINITY;
  a.s += none ? w.y : f * w.y;
  a.t += none ? w.z : f * fmaf(d, w.y, w.z);
}
__device__ __forceinline__ Moments join_moments(const float4* q, int parts, int i0, int step) {
  Moments a = {-INFINITY, 0.f, 0.f};
  for (int t0 = i0; t0 < parts; t0 += step * 4) {
    float4 w[4];
    float m = a.m;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + step * i;
      w[i] = t < parts ? q[t] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
      m = fmaxf(m, w[i].x);
    }
    const float ref = m == -INFINITY ? 0.f : m;
    Moments b = {m, 0.f, 0.f};
    add_moments(b, make_float4(a.m, a.s, a.t, 0.f), ref);
#pragma unroll
    for (int i = 0; i < 4; ++i) add_moments(b, w[i], ref);
    a = b;
  }
  return a;
}
__device__ __forceinline__ Moments warp_moments(const Moments& a) {
  float top = a.m;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  Moments b = {top, 0.f, 0.f};
  add_moments(b, make_float4(a.m, a.s, a.t, 0.f), top == -INFINITY ? 0.f : top);
  b.s = warp_sum(b.s);
  b.t = warp_sum(b.t);
  return b;
}

// A row's results; returns its lse.  An infinite logit makes its sums NaN, and so everything.
__device__ __forceinline__ float write_row(const LogprobRows& p, long long r, const Moments& a, bool counted, bool writes) {
  const float ls = logf(a.s), lse = (a.m == -INFINITY ? 0.f : a.m) + ls;
  if (writes) {
    const long long lab = p.labels ? p.labels[r] : 0;
    const bool known = lab >= 0 && lab < p.vocab;
    p.lse[r] = lse;
    if (p.labels) p.logprob[r] = !counted ? 0.f : known ? p.zlabel[r] - lse : not_a_number();
    p.entropy[r] = !counted ? 0.f : known ? ls - a.t / a.s : not_a_number();
  }
  return lse;
}
__device__ __forceinline__ void write_lost(const LogprobRows& p, long long r) {
  p.lse[r] = p.entropy[r] = not_a_number();
  if (p.labels) p.logprob[r] = not_a_number();
}

// Without alternatives: a warp a row, or all of a CTA's where the rows are fewer than the SMs.
template <bool kWide>
__global__ void __launch_bounds__(32 * JOIN_WARPS) logprob_kernel(const LogprobRows p) {
  __shared__ float4 sums[JOIN_WARPS];
  await_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long r = kWide ? blockIdx.x : (long long)blockIdx.x * JOIN_WARPS + warp;
  if (r >= p.rows) return;
  if (is_lost(p.status)) {
    if (kWide ? threadIdx.x == 0 : lane == 0) write_lost(p, r);
    return;
  }
  const float4* stat = p.stat + (size_t)r * p.parts;
  Moments a = warp_moments(join_moments(stat, p.parts, kWide ? threadIdx.x : lane, kWide ? 32 * JOIN_WARPS : 32));
  if (kWide) {
    if (lane == 0) sums[warp] = make_float4(a.m, a.s, a.t, 0.f);
    __syncthreads();
    if (warp) return;
    a = warp_moments(join_moments(sums, JOIN_WARPS, lane, 32));
  }
  write_row(p, r, a, !p.labels || p.labels[r] != p.ignore, lane == 0);
}

// With alternatives: a CTA a row.  The products' logits are off by some 1e-6 of their
// partial sums, which is enough to swap neighbours (and where large terms cancel, ones far apart), so
// they only choose candidates, and the candidates' logits are summed again, to 2^-45 of their
// largest partial sum.  The keys are upper bounds on the exact logits (ce.h):
//   1. the top-th largest of the threads' largest keys (two each where there are few), by merging
//      the warps' lists in order;
//   2. candidates: columns whose key is not below that by more than MARGIN of the largest
//      logit; of 32 columns whose two keys both qualify, all (a third may hide behind them);
//   3. their logits again, a warp each; 4. their ranks, ties to the lower index;
//   5. if the top-th best of them is not below what was the least key of a candidate, nothing else
//      can be among the best.  (MARGIN lets keys of up to some 10000 columns pass.)
// Where it is, and where ties or bounds full of neighbours make more candidates than fit, the row's
// groups of 32 columns are walked in order instead, against the top-th best so far.
// Many rows: 128 threads, so that many rows are at hand (4096 x 32000 with 8 alternatives, by 64,
// 128 and 256 threads: 255, 237 and 349 us).  Few rows, whose every wait shows: 512, a
// candidate a warp and a row's words asked for at once.
constexpr int TOP_MANY = 128, TOP_FEW = 512, TOP_FEW_ROWS = 152;
constexpr int TOP_CANDIDATES = 512;
constexpr int TOP_WHOLE = 14;                // groups taken whole
constexpr float TOP_MARGIN = 0x1p-10f, TOP_LEAST_MARGIN = 1e-18f;   // (rows of zeros: above what the least length makes of them)
// A bound may be above its key by this share of it (twice 31 ulp of the column's bits, a rounding).
constexpr float KEY_SHARE = 0x1p-16f, KEY_LEAST = 1e-30f;
constexpr float MASKED = -0x1p120f;          // logits down here are masks, of the type's lowest value or less
static_assert(TOP_WHOLE * KEY_COLS + MUON_LOGPROB_MAX_TOP <= TOP_CANDIDATES, "");

// s + e <- s + e + p, exactly but for e's own rounding.
__device__ __forceinline__ void add_exact(float& s, float& e, float p) {
  const float t = __fadd_rn(s, p), b = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(p, b)));
  s = t;
}
// s + e over the warp, in every lane (64-bit additions would hold the warps up): the same
// number in each, for a lane and its partner round the same sums.  (What the addition of s and so
// drops is a number of its own; e + eo comes first, which does not depend on whose is whose.)
__device__ __forceinline__ double warp_exact(float s, float e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o), eo = __shfl_xor_sync(0xffffffffu, e, o);
    e = __fadd_rn(e, eo);
    add_exact(s, e, so);
  }
  return (double)s + (double)e;
}
// The logits of a row and N rows of W as sums of exact products: those of bf16 numbers are
// exact in fp32, those of fp32 ones come in two parts.  kHeld vectors are asked for at once (the
// order of the sums does not depend on it).
template <int N, int kHeld>
__device__ __forceinline__ void logits(const bf16* h, const bf16* const* w, int dim, int vec, int lane, double* out) {
  float s[N][2] = {}, e[N][2] = {};
  const int whole = vec ? dim / 8 : 0;
  const uint4 none = make_uint4(0, 0, 0, 0);
  for (int c0 = lane; c0 < whole; c0 += 32 * kHeld) {
    uint4 a[kHeld], b[N][kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int c = c0 + 32 * i;
      a[i] = c < whole ? reinterpret_cast<const uint4*>(h)[c] : none;
#pragma unroll
      for (int q = 0; q < N; ++q) b[q][i] = c < whole ? reinterpret_cast<const uint4*>(w[q])[c] : none;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const uint32_t y[4] = {b[q][i].x, b[q][i].y, b[q][i].z, b[q][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          add_exact(s[q][0], e[q][0], __fmul_rn(__uint_as_float(x[j] << 16), __uint_as_float(y[j] << 16)));
          add_exact(s[q][1], e[q][1], __fmul_rn(__uint_as_float(x[j] & 0xFFFF0000u), __uint_as_float(y[j] & 0xFFFF0000u)));
        }
      }
    }
  }
  for (int c = whole * 8 + lane; c < dim; c += 32)
#pragma unroll
    for (int q = 0; q < N; ++q) add_exact(s[q][0], e[q][0], __fmul_rn(ld1(h + c), ld1(w[q] + c)));
#pragma unroll
  for (int q = 0; q < N; ++q) {
    add_exact(s[q][0], e[q][0], s[q][1]);
    out[q] = warp_exact(s[q][0], __fadd_rn(e[q][0], e[q][1]));
  }
}
template <int N, int kHeld>
__device__ __forceinline__ void logits(const float* h, const float* const* w, int dim, int, int lane, double* out) {
  float s[N] = {}, e[N] = {};
  for (int c0 = lane; c0 < dim; c0 += 64 * kHeld) {
    float a[2 * kHeld], b[N][2 * kHeld];
#pragma unroll
    for (int i = 0; i < 2 * kHeld; ++i) {
      const int c = c0 + 32 * i;
      a[i] = c < dim ? h[c] : 0.f;
#pragma unroll
      for (int q = 0; q < N; ++q) b[q][i] = c < dim ? w[q][c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 2 * kHeld; ++i)
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const float x = __fmul_rn(a[i], b[q][i]);
        e[q] = __fadd_rn(e[q], __fmaf_rn(a[i], b[q][i], -x));   // what the product's rounding dropped
        add_exact(s[q], e[q], x);
      }
  }
#pragma unroll
  for (int q = 0; q < N; ++q) out[q] = warp_exact(s[q], e[q]);
}

// A number's place among the doubles as a whole number (comparisons of doubles take 16 cycles a
// warp); one that is masked or not a number has none.
constexpr long long NO_PLACE = -0x7FFFFFFFFFFFFFFFLL - 1;
__device__ __forceinline__ long long place_of(double v) {
  const long long b = __double_as_longlong(v + 0.0);      // (-0 is 0)
  return v > MASKED ? b ^ ((b >> 63) & 0x7FFFFFFFFFFFFFFFLL) : NO_PLACE;
}
__device__ __forceinline__ double at_place(long long k) {
  return __longlong_as_double(k ^ ((k >> 63) & 0x7FFFFFFFFFFFFFFFLL));
}

constexpr int TOP_HELD = 8;                  // pairs of groups whose keys a thread keeps (65536 entries)
template <int kThreads> struct TopShared {
  long long value[TOP_CANDIDATES];           // place_of a logit
  int id[TOP_CANDIDATES];
  float key[kThreads];
  float4 warp[kThreads / 32];
  int whole[TOP_WHOLE];
  long long kept_value[MUON_LOGPROB_MAX_TOP];
  int kept_id[MUON_LOGPROB_MAX_TOP];
  int count, wholes;
  float bound;
};

// The warp's numbers in descending order, one a lane.
__device__ __forceinline__ float sort_lanes(float v, int lane) {
#pragma unroll
  for (int n = 2; n <= 32; n *= 2)
#pragma unroll
    for (int m = n / 2; m > 0; m /= 2) {
      const float o = __shfl_xor_sync(0xffffffffu, v, m);
      v = ((lane & n) == 0) == ((lane & m) == 0) ? fmaxf(v, o) : fminf(v, o);
    }
  return v;
}

// The 32 largest of two warps' numbers, both in descending order, in descending order.
__device__ __forceinline__ float merge_lanes(float a, float b, int lane) {
  float v = fmaxf(a, __shfl_sync(0xffffffffu, b, 31 - lane));
#pragma unroll
  for (int m = 16; m > 0; m /= 2) {
    const float o = __shfl_xor_sync(0xffffffffu, v, m);
    v = (lane & m) == 0 ? fmaxf(v, o) : fminf(v, o);
  }
  return v;
}

// The best `top` of n candidates, in order, to kept_*; the others' places hold -1.  An id of
// -1, a masked value or a NaN is no candidate.
template <int kThreads>
__device__ __forceinline__ void rank(TopShared<kThreads>& sh, int n, int top) {
  for (int i = threadIdx.x; i < top; i += kThreads) sh.kept_id[i] = -1;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const long long v = sh.value[i];
    const int id = sh.id[i];
    if (id < 0 || v == NO_PLACE) continue;
    int better = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) {
      const long long u = sh.value[j];
      const int other = sh.id[j];
      better += other >= 0 && (u > v || (u == v && other < id));
    }
    if (better < top) {
      sh.kept_value[better] = v;
      sh.kept_id[better] = id;
    }
  }
  __syncthreads();
}

// The values of N ids of a warp, as many apart as there are warps, from i on.  (An id of -1 has
// no row; its value is never looked at.)
template <int N, int kHeld, typename T, int kThreads>
__device__ __forceinline__ void evaluate_some(TopShared<kThreads>& sh, int i, const LogprobRows& p, const T* h, int lane) {
  const T* w[N];
  double v[N];
#pragma unroll
  for (int q = 0; q < N; ++q) w[q] = static_cast<const T*>(p.W) + max(sh.id[i + q * (kThreads / 32)], 0) * p.ldw;
  logits<N, kHeld>(h, w, p.dim, p.vec, lane, v);
#pragma unroll
  for (int q = 0; q < N; ++q)
    if (lane == q) sh.value[i + q * (kThreads / 32)] = place_of(v[q]);
}
// The values of the first n ids, two of them a warp at a time where there are as many.
template <typename T, int kThreads>
__device__ __forceinline__ void evaluate(TopShared<kThreads>& sh, int n, const LogprobRows& p, const T* h) {
  constexpr int W = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int i = warp;
  for (; i + W < n; i += 2 * W) evaluate_some<2, 2>(sh, i, p, h, lane);
  if (i < n) evaluate_some<1, kThreads == TOP_FEW ? 6 : 2>(sh, i, p, h, lane);
  __syncthreads();
}

template <typename T, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreads == TOP_FEW ? 1 : 8) top_kernel(const LogprobRows p) {
  constexpr int TOP_THREADS = kThreads, TOP_WARPS = kThreads / 32;
  __shared__ TopShared<kThreads> sh;
  await_previous();
  const long long r = blockIdx.x;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, top = p.top;
  long long* ids = p.ids + r * top;
  float* alternatives = p.alternatives + r * top;
  const bool lost = is_lost(p.status), counted = !p.labels || p.labels[r] != p.ignore;
  // the row's sums
  const Moments mine = warp_moments(join_moments(p.stat + (size_t)r * p.parts, p.parts, t, TOP_THREADS));
  if (lane == 0) sh.warp[warp] = make_float4(mine.m, mine.s, mine.t, 0.f);
  if (t == 0) sh.count = sh.wholes = 0;
  // the thread's two largest keys
  const int groups = p.groups;
  const float2* keys = p.keys + (size_t)r * groups;
  const float4* pairs = reinterpret_cast<const float4*>(keys);
  float4 held[TOP_HELD];
  float k1 = -INFINITY, k2 = -INFINITY;
  auto take = [&](const float4& k) {
    k2 = fmaxf(k2, fmaxf(fminf(k1, k.x), k.y));
    k1 = fmaxf(k1, k.x);
    k2 = fmaxf(k2, fmaxf(fminf(k1, k.z), k.w));
    k1 = fmaxf(k1, k.z);
  };
  // a group a thread where that covers them (every key counts below), two otherwise
  const bool single = groups <= TOP_THREADS;
#pragma unroll
  for (int i = 0; i < TOP_HELD; ++i) {
    const int g = single ? groups : t + i * TOP_THREADS;
    held[i] = g < groups / 2 ? pairs[g] : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
  }
  if (single && t < groups) {
    const float2 k = keys[t];
    held[0] = make_float4(k.x, k.y, -INFINITY, -INFINITY);
  }
#pragma unroll
  for (int i = 0; i < TOP_HELD; ++i) take(held[i]);
  for (int g = t + TOP_HELD * TOP_THREADS; g < groups / 2; g += TOP_THREADS) take(pairs[g]);
  // (few groups: the second largest count, too)
  float best = sort_lanes(k1, lane);
  if (groups < 4 * TOP_THREADS) best = merge_lanes(best, sort_lanes(k2, lane), lane);
  sh.key[t] = best;
  if (t == 0) sh.bound = -INFINITY;
  __syncthreads();
  Moments all = {-INFINITY, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < TOP_WARPS; ++i) all.m = fmaxf(all.m, sh.warp[i].x);
#pragma unroll
  for (int i = 0; i < TOP_WARPS; ++i) add_moments(all, sh.warp[i], all.m == -INFINITY ? 0.f : all.m);
  if (lost && t == 0) write_lost(p, r);
  const float lse = lost ? not_a_number() : write_row(p, r, all, counted, t == 0);
  if (!counted || !isfinite(lse)) {
    // nothing to rank: an ignored row, one whose logits are all minus infinity, or not numbers
    for (int i = t; i < top; i += TOP_THREADS) {
      ids[i] = -1;
      alternatives[i] = counted && lse != -INFINITY ? not_a_number() : -INFINITY;
    }
    return;
  }
  // 1. the top-th largest of the threads' keys (-inf where there are fewer)
  if (warp == 0) {
#pragma unroll
    for (int w = 1; w < TOP_WARPS; ++w) best = merge_lanes(best, sh.key[32 * w + lane], lane);
    if (lane == top - 1 && best > MASKED) sh.bound = best;
  }
  __syncthreads();
  const float bound = sh.bound;
  float least = bound - (TOP_MARGIN * fmaxf(fabsf(all.m), bound == -INFINITY ? 0.f : fabsf(bound)) + TOP_LEAST_MARGIN);
  const T* h = static_cast<const T*>(p.H) + r * p.ldh;
  // 2. candidates
  auto choose = [&](float a, float b, int g) {
    if (!(a >= least && a > MASKED)) return;
    if (b >= least && b > MASKED) {
      const int at = atomicAdd(&sh.wholes, 1);
      if (at < TOP_WHOLE) sh.whole[at] = g;
    } else {
      const int at = atomicAdd(&sh.count, 1);
      if (at < TOP_CANDIDATES) sh.id[at] = g * KEY_COLS + (int)(KEY_MASK - (__float_as_uint(a) & KEY_MASK));
    }
  };
  if (k1 >= least) {
#pragma unroll
    for (int i = 0; i < TOP_HELD; ++i) {
      const int g = t + i * TOP_THREADS;
      choose(held[i].x, held[i].y, single ? t : 2 * g);
      choose(held[i].z, held[i].w, 2 * g + 1);
    }
    for (int g = t + TOP_HELD * TOP_THREADS; g < groups / 2; g += TOP_THREADS) {
      const float4 k = pairs[g];
      choose(k.x, k.y, 2 * g);
      choose(k.z, k.w, 2 * g + 1);
    }
  }
  __syncthreads();
  // 5. what no key below `least` can reach, and the least key that can reach the top-th best
  auto enough = [&] {
    return least == -INFINITY || (sh.kept_id[top - 1] >= 0 && sh.kept_value[top - 1] >= place_of((double)least + (KEY_SHARE * fabsf(least) + KEY_LEAST)));
  };
  auto lower = [&] {
    if (sh.kept_id[top - 1] < 0) return -INFINITY;
    const float v = __double2float_rd(at_place(sh.kept_value[top - 1]));
    return __fsub_rd(v, __fmaf_ru(KEY_SHARE, fabsf(v), KEY_LEAST));
  };
  const int singles = sh.count, wholes = sh.wholes;
  const bool fits = wholes <= TOP_WHOLE && singles + wholes * KEY_COLS <= TOP_CANDIDATES;
  int walks = 2;                 // the first with `least` as it is, where the candidates do not fit
  if (fits) {
    const int n = singles + wholes * KEY_COLS;
    for (int i = singles + t; i < n; i += TOP_THREADS) {
      const int c = sh.whole[(i - singles) / KEY_COLS] * KEY_COLS + (i - singles) % KEY_COLS;
      sh.id[i] = c < p.vocab ? c : -1;
    }
    __syncthreads();
    // 3.
    evaluate(sh, n, p, h);
    rank(sh, n, top);
    walks = 0;
    if (!enough()) {
      least = lower();
      walks = 1;
    }
  } else {
    // a row of zeros (padding): every logit is 0
    bool zero = true;
    for (int c = t; c < p.dim; c += TOP_THREADS) zero = zero && ld1(h + c) == 0.f;
    if (__syncthreads_and(zero)) {
      for (int i = t; i < top; i += TOP_THREADS) {
        ids[i] = i < p.vocab ? i : -1;
        alternatives[i] = i < p.vocab ? -lse : -INFINITY;
      }
      return;
    }
  }
  // every group against the best so far, KEY_COLS columns at a time; a second walk goes on with the
  // keys that the first left out
  int kept = 0;
  double worst = -INFINITY;        // of the kept, when there are `top`
  for (float above = INFINITY; walks > 0; --walks) {
    __syncthreads();
    for (int g = 0; g < groups; ++g) {
      const float k = keys[g].x;   // (the same for every thread)
      if (!(k >= least && k > MASKED) || k >= above || (double)k + (KEY_SHARE * fabsf(k) + KEY_LEAST) < worst) continue;
      const long long c = (long long)g * KEY_COLS + t;
      if (t < KEY_COLS) sh.id[t] = c < p.vocab ? (int)c : -1;
      if (t < kept) {
        sh.value[KEY_COLS + t] = sh.kept_value[t];
        sh.id[KEY_COLS + t] = sh.kept_id[t];
      }
      __syncthreads();
      evaluate(sh, KEY_COLS, p, h);
      rank(sh, KEY_COLS + kept, top);
      kept = 0;
      while (kept < top && sh.kept_id[kept] >= 0) ++kept;
      if (kept == top) worst = at_place(sh.kept_value[top - 1]);
      __syncthreads();
    }
    if (walks == 1 || enough()) break;
    above = least;
    least = lower();
  }
  for (int i = t; i < top; i += TOP_THREADS) {
    const int id = sh.kept_id[i];
    ids[i] = id;
    alternatives[i] = id < 0 ? -INFINITY : (float)(at_place(sh.kept_value[i]) - (double)lse);
  }
}

// dH from the sums of each range of K; a block a row.
template <typename T>
__global__ void __launch_bounds__(256) split_sum_kernel(const float* acc, int splits, long long rows, int dim,
                                                        long long ldacc, T* out, float scale, const float* upstream,
                                                        const float* stats, const unsigned int* status, T* dW,
                                                        long long vocab) {
  await_previous();
  if (is_lost(status)) {
    fill_lost(out, rows * dim);
    fill_lost(dW, vocab * dim);
    return;
  }
  const long long r = blockIdx.x;
  const float u = shared_factor(scale, upstream, stats);
  for (int c = threadIdx.x; c < dim; c += 256) {
    const float* a = acc + r * ldacc + c;
    float s = 0.f;
#pragma unroll 4
    for (int k = 0; k < splits; ++k) s += a[(size_t)k * rows * ldacc];
    st1(out + r * dim + c, s * u);
  }
}

// The last kernel of a backward pass that sums no ranges.
constexpr int LOST_CTAS = 32;
template <typename T>
__global__ void __launch_bounds__(256) lost_kernel(const unsigned int* status, T* dH, long long nh, T* dW, long long nw) {
  await_previous();
  if (!is_lost(status)) return;
  fill_lost(dH, nh);
  fill_lost(dW, nw);
}

// ---------------------------------------------------------------------------
// plan
// ---------------------------------------------------------------------------
struct CePlan {
  int parts, nterms;
  int64_t dp;                  // row length of a packed copy
  bool pack_h, pack_w;
  size_t hp, wp;               // packed copies
  size_t zlabel, part, sums;   // forward
  size_t stat, keys, hshare, wlen;   // forward of the log probabilities
  size_t few;                  // their backward pass with few rows
  int64_t piece, npieces;
  int splits;
  size_t g[2];
  size_t g_part;               // elements of one part of g
  size_t acc;
  int64_t ldacc;
  size_t total;
};

int check(const muon_linear_ce* a) {
  if (!a) return MUON_ERR_INVALID;
  const int64_t lim = 1LL << 30;   // so that a tile's rows and columns past the end still fit an int
  if (a->rows < 0 || a->rows > lim || a->vocab < 1 || a->vocab > lim || a->dim < 1 || a->dim > lim ||
      a->ldh < a->dim || a->ldw < a->dim)
    return MUON_ERR_INVALID;
  if (a->dtype != MUON_DTYPE_F32 && a->dtype != MUON_DTYPE_BF16) return MUON_ERR_UNSUPPORTED;
  if (a->ldh >= (1LL << 38) || a->ldw >= (1LL << 38)) return MUON_ERR_UNSUPPORTED;
  // tiles are counted in 31 bits
  if (cdiv(a->rows, TILE) * cdiv(a->vocab, TILE) >= (1LL << 30) || cdiv(a->rows, TILE) * cdiv(a->dim, TILE) >= (1LL << 26) ||
      cdiv(a->vocab, TILE) * cdiv(a->dim, TILE) >= (1LL << 30))
    return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}
int check_pointers(const muon_linear_ce* a, bool no_labels = false) {
  if (!a->W || !is_aligned(a->W, dt_size(a->dtype))) return MUON_ERR_INVALID;
  if (a->rows && (!a->H || (!a->labels && !no_labels) || !is_aligned(a->H, dt_size(a->dtype)) || !is_aligned(a->labels, 8)))
    return MUON_ERR_INVALID;
  return MUON_OK;
}

// A tile's time in K steps: its epilogue overlaps the next tile's MMAs, and alone takes as
// long as some 12 steps (64 rows: 3.5 us a tile of dW, one K step long).
int64_t tile_cost(int64_t steps) { return std::max<int64_t>(steps, 12) + 2; }

// Ranges the K of a dH tile is cut into: a tile over a whole piece must not outlast half
// of a CTA pair's share of the launch (the tiles are handed out longest first).
int split_count(int64_t rows, int64_t dim, int64_t piece, int64_t npairs) {
  const int64_t kp = cdiv(piece, BK), mt = cdiv(rows, TILE), dt = cdiv(dim, TILE), vt = cdiv(piece, TILE);
  const int64_t work = mt * dt * kp + vt * dt * tile_cost(cdiv(rows, BK)) + mt * vt * tile_cost(cdiv(dim, BK));
  const int64_t share = std::max<int64_t>(work / (2 * npairs), 8);
  return (int)std::min<int64_t>(std::max<int64_t>(1, cdiv(kp, share)), MAX_SPLITS);
}

// Whether W can be read in 16-byte words.
bool words_of_w(const muon_linear_ce* a) {
  const size_t es = dt_size(a->dtype);
  return is_aligned(a->W, 16) && a->ldw * es % 16 == 0 && a->dim * es % 16 == 0;
}

// top: -1 for the cross entropy's forward pass, else the log probabilities' with so many
// alternatives.
void make_plan(const muon_linear_ce* a, int backward, CePlan* P, int top = -1) {
  const bool f32 = a->dtype == MUON_DTYPE_F32;
  P->parts = f32 ? 3 : 1;
  P->nterms = f32 ? 6 : 1;
  P->dp = (a->dim + 7) / 8 * 8;
  P->pack_h = f32 || a->ldh % 8 || !is_aligned(a->H, 16);
  P->pack_w = f32 || a->ldw % 8 || !is_aligned(a->W, 16);
  size_t at = HEADER;
  auto take = [&](size_t bytes) { const size_t p = at; at += up(bytes); return p; };
  // room for H's copy in any case: for the backward pass, and so that a workspace fits
  // whatever H's alignment
  auto copies = [&] {
    P->hp = take((size_t)P->parts * a->rows * P->dp * 2);
    P->wp = P->pack_w ? take((size_t)P->parts * a->vocab * P->dp * 2) : at;
  };
  // (few rows' kernels read the operands where they lie, and no rows need nothing)
  if (top < 0 || (a->rows > 0 && !few_rows(a->rows, a->dim, f32, false, words_of_w(a)))) copies();
  P->zlabel = take((size_t)a->rows * 4);
  if (top < 0) {
    P->part = take((size_t)a->rows * 2 * cdiv(a->vocab, TILE) * sizeof(float2));
    P->sums = take((size_t)cdiv(a->rows, JOIN_WARPS) * sizeof(float2));
  } else {
    int64_t stats = a->rows * 2;                // of a tile's columns; more where a few of the rows would have more
    for (int64_t n = 1; n <= std::min<int64_t>(a->rows, 16); ++n)
      if (few_rows(n, a->dim, f32, false, false) || few_rows(n, a->dim, f32, false, true))
        stats = std::max(stats, n * (TILE / few_block(a->vocab)));
    P->stat = take((size_t)stats * cdiv(a->vocab, TILE) * sizeof(float4));
    P->keys = take(top ? (size_t)a->rows * (TILE / KEY_COLS) * cdiv(a->vocab, TILE) * sizeof(float2) : 0);
    P->hshare = take(top ? (size_t)a->rows * 4 : 0);
    P->wlen = take(top ? (size_t)cdiv(a->vocab, TILE) * (TILE + TILE / KEY_COLS) * 4 : 0);
  }
  P->total = at;
  if (!backward) return;
  at = HEADER;
  if (top >= 0) {
    // (for more rows too, so that their workspace serves a few of them)
    for (int64_t n = 1; n <= 8; n *= 2)
      if (n < 2 * a->rows && few_rows(n, a->dim, f32, true, false)) P->total = std::max(P->total, at + up(few_bytes(n, a->dim)));
    if (few_rows(a->rows, a->dim, f32, true, false)) P->few = at;
    if (a->rows == 0 || P->few) return;
  }
  copies();
  const int64_t want = G_BYTES / (2 * P->parts * std::max<int64_t>(a->rows, 1));
  P->piece = std::min(std::max(want / TILE * TILE, MIN_PIECE), cdiv(a->vocab, TILE) * TILE);
  if (const int tiles = (test_flags() / MUON_DEBUG_CE_PIECE) & 255) P->piece = std::min<int64_t>(P->piece, (int64_t)tiles * TILE);
  // pieces of one size, as far as tiles allow
  P->npieces = cdiv(a->vocab, P->piece);
  P->piece = cdiv(cdiv(a->vocab, P->npieces), TILE) * TILE;
  P->npieces = cdiv(a->vocab, P->piece);
  P->splits = split_count(a->rows, a->dim, P->piece, 76);
  P->g_part = (size_t)a->rows * P->piece;
  for (int i = 0; i < 2; ++i) P->g[i] = P->npieces > 1 || i == 0 ? take(P->parts * P->g_part * 2) : P->g[0];
  P->ldacc = P->dp;
  P->acc = P->npieces > 1 || P->splits > 1 ? take((size_t)P->splits * a->rows * P->ldacc * 4) : 0;
  P->total = std::max(P->total, at);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------
struct Operand {
  const bf16* p;
  int64_t rows, cols, ld, part_stride;
  int parts;
};

bool map_of(CUtensorMap* m, const Operand& o) {
  return encode_tmap_bf16(m, o.p, (uint64_t)o.cols, (uint64_t)o.rows, (uint64_t)o.parts, (uint64_t)o.ld * 2,
                          (uint64_t)o.part_stride * 2, 64, BOX);
}

template <typename T>
cudaError_t pack(const void* in, int64_t ld, int64_t rows, int64_t dim, bf16* out, int64_t ldo, int parts,
                 const RowMask& mask, cudaStream_t s) {
  count_launch();
  return launch_after(pack_kernel<T>, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const T*>(in),
                      (long long)ld, (long long)rows, (int)dim, out, (long long)ldo, parts, (long long)(rows * ldo), mask);
}

// H or W as the products read it: where it lies, or a copy of it.  mask: the rows of H that
// carry a gradient are wanted, and zeros for the others.
cudaError_t operand(Operand* o, const muon_linear_ce* a, const CePlan& P, bool h, bool mask, char* ws, cudaStream_t s) {
  const void* src = h ? a->H : a->W;
  const int64_t rows = h ? a->rows : a->vocab, ld = h ? a->ldh : a->ldw;
  const bool copy = h ? P.pack_h : P.pack_w;
  if (!copy && !mask) {
    *o = Operand{static_cast<const bf16*>(src), rows, a->dim, ld, rows * ld, 1};
    return cudaSuccess;
  }
  bf16* dst = reinterpret_cast<bf16*>(ws + (h ? P.hp : P.wp));
  *o = Operand{dst, rows, a->dim, P.dp, rows * P.dp, P.parts};
  const RowMask k = {mask ? a->labels : nullptr, a->vocab, a->ignore_index};
  if (!copy && a->dim % 8 == 0) {
    count_launch();
    return launch_after(mask_kernel, dim3((unsigned)cdiv(rows, 8)), dim3(256), 0, s, static_cast<const bf16*>(src),
                        (long long)ld, (long long)rows, (int)a->dim, dst, k);
  }
  return a->dtype == MUON_DTYPE_BF16 ? pack<bf16>(src, ld, rows, a->dim, dst, P.dp, 1, k, s)
                                     : pack<float>(src, ld, rows, a->dim, dst, P.dp, 3, k, s);
}

void common_params(Params* p, const muon_linear_ce* a, const CePlan& P, char* ws) {
  std::memset(static_cast<void*>(p), 0, sizeof(Params));
  p->nterms = P.nterms;
  p->parts = P.parts;
  // (part of A, part of B), smallest products first
  static const unsigned char ta[MAX_TERMS] = {2, 0, 1, 1, 0, 0}, tb[MAX_TERMS] = {0, 2, 1, 0, 1, 0};
  if (P.nterms > 1) {
    std::memcpy(p->ta, ta, sizeof(ta));
    std::memcpy(p->tb, tb, sizeof(tb));
  }
  p->f32_out = a->dtype == MUON_DTYPE_F32;
  p->labels = a->labels;
  p->vocab = a->vocab;
  p->ignore = a->ignore_index;
  p->status = reinterpret_cast<unsigned int*>(ws);
  p->timeout_ns = wait_limit_ns();
  p->debug_flags = test_flags();
}

// Row tiles that are walked together for each column tile, so that their rows of A stay in
// L2: the forward pass keeps all of 8192 rows there; the products with g, whose operands are
// larger, and g itself beside them do better with fewer.  8192 x 2560 x 131072 in a loop:
// forward 8 row tiles 3.46 ms, 16 3.39, 32 3.35; backward, g and its products, 32 and 32
// 10.56 ms, 16 and 16 10.28, 32 and 12 10.37, 32 and 8 10.30, 16 and 8 10.25.
constexpr int GROUP_FORWARD = 32, GROUP_GRAD = 16, GROUP_G = 8;

void shape(Job* j, int64_t m, int64_t n, int64_t k, int group) {
  j->m = (int)m;
  j->n = (int)n;
  j->mtiles = (int)cdiv(m, TILE);
  j->ntiles = (int)cdiv(n, TILE);
  j->group = std::min(group, j->mtiles);
  j->splits = 1;
  j->nkb = (int)cdiv(k, BK);
  j->tiles = j->mtiles * j->ntiles;
}

// Hands the launch's tiles out so that the pairs' work evens out: jobs in order of their
// tiles' lengths, the tiles of each filling the pairs up to a common level, round by round
// (so that pairs work on neighbouring tiles at a time).  Launches with more tiles than the
// table holds go round robin, where one tile more or less no longer matters.  Returns
// whether the table is used.
bool lay_out(OrderedParams* p, int npairs) {
  std::sort(p->job, p->job + p->njobs, [](const Job& x, const Job& y) { return x.nkb > y.nkb; });
  int t = 0;
  for (int j = 0; j < p->njobs; ++j) {
    p->job[j].begin = t;
    t += p->job[j].tiles;
  }
  p->tiles = t;
  // (and what the levels are counted in has to fit 31 bits)
  long long work = 0;
  for (int j = 0; j < p->njobs; ++j) work += (long long)p->job[j].tiles * tile_cost(p->nterms * (int64_t)p->job[j].nkb);
  if (p->njobs < 2 || t > MAX_ORDER || t <= npairs || work >= (1LL << 30)) return false;
  int load[MAX_PAIRS] = {}, by_load[MAX_PAIRS];
  int count[MAX_JOBS][MAX_PAIRS];
  int total[MAX_PAIRS] = {};
  for (int j = 0; j < p->njobs; ++j) {
    const int cost = (int)tile_cost((int64_t)p->nterms * p->job[j].nkb);
    const int tiles = p->job[j].tiles;
    // the highest level up to which whole tiles can fill the pairs ...
    auto below = [&](int level) {
      int n = 0;
      for (int i = 0; i < npairs; ++i) n += level > load[i] ? (level - load[i]) / cost : 0;
      return n;
    };
    int most = 0;
    long long sum = (long long)cost * tiles;
    for (int i = 0; i < npairs; ++i) { most = std::max(most, load[i]); sum += load[i]; }
    int lo = *std::min_element(load, load + npairs), hi = std::max<int>(most, (int)(sum / npairs)) + cost + 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (below(mid) <= tiles) lo = mid; else hi = mid - 1;
    }
    int left = tiles;
    for (int i = 0; i < npairs; ++i) {
      by_load[i] = i;
      count[j][i] = lo > load[i] ? (lo - load[i]) / cost : 0;
      load[i] += count[j][i] * cost;
      left -= count[j][i];
    }
    // ... and the rest, less than one a pair, to those with the least work
    std::sort(by_load, by_load + npairs, [&](int x, int y) { return load[x] != load[y] ? load[x] < load[y] : x < y; });
    for (int i = 0; i < left; ++i) {
      ++count[j][by_load[i]];
      load[by_load[i]] += cost;
    }
    for (int i = 0; i < npairs; ++i) total[i] += count[j][i];
  }
  int fill[MAX_PAIRS];
  p->start[0] = 0;
  for (int i = 0; i < npairs; ++i) {
    fill[i] = p->start[i];
    p->start[i + 1] = (unsigned short)(p->start[i] + total[i]);
  }
  t = 0;
  for (int j = 0; j < p->njobs; ++j)
    for (const int end = t + p->job[j].tiles; t < end;)
      for (int i = 0; i < npairs; ++i)
        if (count[j][i] > 0) {
          --count[j][i];
          p->order[fill[i]++] = (unsigned short)t++;
        }
  return true;
}

template <typename T>
cudaError_t finish(const muon_linear_ce* a, const CePlan& P, const float* acc, const Params& p, T* dH, T* dW, cudaStream_t s) {
  count_launch();
  if (dH && P.splits > 1)
    return launch_after(split_sum_kernel<T>, dim3((unsigned)a->rows), dim3(256), 0, s, acc, P.splits, a->rows, a->dim,
                        P.ldacc, dH, p.scale, p.upstream, p.stats, p.status, dW, a->vocab);
  return launch_after(lost_kernel<T>, dim3(LOST_CTAS), dim3(256), 0, s, p.status, dH, a->rows * a->dim, dW,
                      a->vocab * a->dim);
}

int result_vec(const void* out, int64_t ld, int dt) {
  const size_t row = (size_t)ld * dt_size(dt);
  if (is_aligned(out, 32) && row % 32 == 0) return 2;
  return is_aligned(out, 16) && row % 16 == 0 ? 1 : 0;
}

Few few_args(const muon_linear_ce* a, char* ws) {
  Few f = {};
  f.H = a->H;
  f.W = a->W;
  f.labels = a->labels;
  f.ldh = a->ldh;
  f.ldw = a->ldw;
  f.vocab = a->vocab;
  f.ignore = a->ignore_index;
  f.rows = (int)a->rows;
  f.dim = (int)a->dim;
  f.status = reinterpret_cast<const unsigned int*>(ws);
  return f;
}

// The keys' shares and lengths: of bf16 operands as the products read them, of 32-bit ones as they are.
cudaError_t lengths(const muon_linear_ce* a, const Operand& H, const Operand& W, float share, float* hshare,
                    float* wlen, float* wgroup, cudaStream_t s) {
  const bool f32 = a->dtype == MUON_DTYPE_F32;
  const size_t es = dt_size(a->dtype);
  Lengths q = {};
  q.h = f32 ? a->H : H.p;
  q.w = f32 ? a->W : W.p;
  q.ldh = f32 ? a->ldh : H.ld;
  q.ldw = f32 ? a->ldw : W.ld;
  q.rows = a->rows;
  q.vocab = a->vocab;
  q.dim = (int)a->dim;
  q.hvec = is_aligned(q.h, 16) && q.ldh * es % 16 == 0;
  q.wvec = is_aligned(q.w, 16) && q.ldw * es % 16 == 0;
  q.groups = (int)(cdiv(a->vocab, TILE) * (TILE / KEY_COLS));   // (of whole tiles)
  q.share = share;
  q.hshare = hshare;
  q.wlen = wlen;
  q.wgroup = wgroup;
  count_launch();
  const dim3 grid((unsigned)(q.groups + cdiv(a->rows, KEY_COLS)));
  return f32 ? launch_after(lengths_kernel<float>, grid, dim3(256), 0, s, q)
             : launch_after(lengths_kernel<bf16>, grid, dim3(256), 0, s, q);
}

// The last kernel of a forward pass.
int join_rows(const muon_linear_ce* a, int top, const Params& p, int parts, float* logprob, float* entropy, float* lse,
              int64_t* ids, float* alternatives, cudaStream_t s) {
  LogprobRows q = {};
  q.stat = p.stat;
  q.keys = p.keys;
  q.parts = parts;
  q.groups = (int)(TILE / KEY_COLS * cdiv(a->vocab, TILE));
  q.rows = a->rows;
  q.labels = a->labels;
  q.vocab = a->vocab;
  q.ignore = a->ignore_index;
  q.zlabel = p.zlabel;
  q.logprob = logprob;
  q.entropy = entropy;
  q.lse = lse;
  q.status = p.status;
  q.H = a->H;
  q.W = a->W;
  q.ldh = a->ldh;
  q.ldw = a->ldw;
  q.dim = (int)a->dim;
  q.top = top;
  q.ids = reinterpret_cast<long long*>(ids);
  q.alternatives = alternatives;
  const size_t es = dt_size(a->dtype);
  q.vec = is_aligned(a->H, 16) && is_aligned(a->W, 16) && a->ldh * es % 16 == 0 && a->ldw * es % 16 == 0;
  count_launch();
  cudaError_t e;
  if (top == 0)
    e = a->rows <= TOP_FEW_ROWS ? launch_after(logprob_kernel<true>, dim3((unsigned)a->rows), dim3(32 * JOIN_WARPS), 0, s, q)
                                : launch_after(logprob_kernel<false>, dim3((unsigned)cdiv(a->rows, JOIN_WARPS)),
                                               dim3(32 * JOIN_WARPS), 0, s, q);
  else if (a->rows <= TOP_FEW_ROWS)
    e = a->dtype == MUON_DTYPE_BF16 ? launch_after(top_kernel<bf16, TOP_FEW>, dim3((unsigned)a->rows), dim3(TOP_FEW), 0, s, q)
                                    : launch_after(top_kernel<float, TOP_FEW>, dim3((unsigned)a->rows), dim3(TOP_FEW), 0, s, q);
  else
    e = a->dtype == MUON_DTYPE_BF16 ? launch_after(top_kernel<bf16, TOP_MANY>, dim3((unsigned)a->rows), dim3(TOP_MANY), 0, s, q)
                                    : launch_after(top_kernel<float, TOP_MANY>, dim3((unsigned)a->rows), dim3(TOP_MANY), 0, s, q);
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

// What g is made of in each row.
struct RowGrads {
  bool policy;                                             // of log probabilities and entropies
  const float *lse, *row_grad, *stats, *upstream;          // cross entropy
  float scale;
  const float *entropy, *g_logprob, *g_entropy;            // log probabilities
};

int backward_pass(const muon_linear_ce* a, const RowGrads& rows, void* dH, void* dW, void* ws, size_t ws_bytes,
                  cudaStream_t s) {
  const size_t es = dt_size(a->dtype);
  if (!is_aligned(dH, es) || !is_aligned(dW, es)) return MUON_ERR_INVALID;
  CePlan P = {};
  make_plan(a, 1, &P, rows.policy ? 0 : -1);
  if (!ws || !is_aligned(ws, 256) || ws_bytes < P.total) return MUON_ERR_WORKSPACE;
  if (!dH && !dW) return MUON_OK;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  if (a->rows == 0) {
    if (dW && cudaMemsetAsync(dW, 0, (size_t)a->vocab * a->dim * es, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (prepare() != cudaSuccess) return MUON_ERR_CUDA;
  char* w = static_cast<char*>(ws);
  if (rows.policy && P.few) {
    Few f = few_args(a, w);
    f.lse = rows.lse;
    f.entropy = rows.entropy;
    f.g_logprob = rows.g_logprob;
    f.g_entropy = rows.g_entropy;
    f.dh_part = reinterpret_cast<float*>(w + P.few);
    f.dW = dW;
    const bool vec = words_of_w(a) && is_aligned(dW, 16);
    return few_backward(f, a->dtype == MUON_DTYPE_F32, vec, dH, s) == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  }
  static thread_local OrderedParams p;
  Operand H, W;
  if (operand(&H, a, P, true, dW != nullptr, w, s) != cudaSuccess || operand(&W, a, P, false, false, w, s) != cudaSuccess)
    return MUON_ERR_CUDA;
  CUtensorMap hmap, wmap;
  if (!map_of(&hmap, H) || !map_of(&wmap, W)) return MUON_ERR_CUDA;
  const bool f32 = a->dtype == MUON_DTYPE_F32;
  const int npairs = pairs();
  float* acc = P.acc ? reinterpret_cast<float*>(w + P.acc) : nullptr;
  // launch i computes g of piece i and multiplies g of piece i - 1
  for (int64_t i = 0; i <= P.npieces; ++i) {
    common_params(&p, a, P, w);
    p.lse = rows.lse;
    p.row_grad = rows.row_grad;
    p.stats = rows.stats;
    p.upstream = rows.upstream;
    p.scale = rows.scale;
    p.entropy = rows.entropy;
    p.g_logprob = rows.g_logprob;
    p.g_entropy = rows.g_entropy;
    if (i > 0) {
      const int64_t v0 = (i - 1) * P.piece, c = std::min(P.piece, a->vocab - v0);
      const Operand G{reinterpret_cast<const bf16*>(w + P.g[(i - 1) & 1]), a->rows, c, P.piece, (int64_t)P.g_part, P.parts};
      if (dH) {
        Job& j = p.job[p.njobs++];
        j.kind = DH;
        if (!map_of(&j.a, G)) return MUON_ERR_CUDA;
        j.b = wmap;
        j.b_mn = 1;
        j.b_k0 = (int)v0;
        shape(&j, a->rows, a->dim, c, GROUP_G);
        j.splits = P.splits;
        j.nkb = (int)cdiv(j.nkb, P.splits);
        j.tiles *= P.splits;
        j.acc = acc;
        j.ldacc = P.ldacc;
        j.first = i == 1;
        j.last = i == P.npieces;
        j.out = P.splits == 1 ? dH : nullptr;
        j.ldo = a->dim;
        j.vec = result_vec(dH, a->dim, a->dtype);
        j.seg_kb = f32 ? SEG_F32 : SEG_LONG;
      }
      if (dW) {
        Job& j = p.job[p.njobs++];
        j.kind = DW;
        if (!map_of(&j.a, G)) return MUON_ERR_CUDA;
        j.b = hmap;
        j.a_mn = j.b_mn = 1;
        shape(&j, c, a->dim, a->rows, GROUP_G);
        j.out = static_cast<char*>(dW) + (size_t)v0 * a->dim * es;
        j.ldo = a->dim;
        j.vec = result_vec(j.out, a->dim, a->dtype);
        j.seg_kb = f32 ? SEG_F32 : SEG_LONG;
      }
    }
    if (i < P.npieces) {
      Job& j = p.job[p.njobs++];
      j.kind = rows.policy ? POLICY : GRAD;
      j.a = hmap;
      j.b = wmap;
      p.v0 = i * P.piece;
      j.b_n0 = (int)p.v0;
      shape(&j, a->rows, std::min<int64_t>(P.piece, a->vocab - p.v0), a->dim, GROUP_GRAD);
      j.out = w + P.g[i & 1];
      j.ldo = P.piece;
      j.part_stride = (long long)P.g_part;
      j.seg_kb = f32 ? SEG_F32 : SEG_LONG;
    }
    bool promote = f32;
    for (int k = 0; k < p.njobs; ++k) promote = promote || p.job[k].nkb > SEG_LONG;
    const bool ordered = lay_out(&p, npairs);
    if (launch(p, ordered, promote, rows.policy, s) != cudaSuccess) return MUON_ERR_CUDA;
  }
  const cudaError_t e = f32 ? finish<float>(a, P, acc, p, static_cast<float*>(dH), static_cast<float*>(dW), s)
                            : finish<bf16>(a, P, acc, p, static_cast<bf16*>(dH), static_cast<bf16*>(dW), s);
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

}  // namespace
}  // namespace ce
}  // namespace muon

using namespace muon;

extern "C" size_t muon_linear_ce_workspace_size(const muon_linear_ce* a, int backward) {
  if (ce::check(a) != MUON_OK) return (size_t)-1;
  ce::CePlan P = {};
  ce::make_plan(a, backward, &P);
  return P.total;
}

extern "C" int muon_linear_ce_forward(const muon_linear_ce* a, float* loss, float* lse, float* stats, void* ws,
                                      size_t ws_bytes, muon_stream_t stream) {
  using namespace ce;
  begin_launches();
  if (int rc = check(a)) return rc;
  if (int rc = check_pointers(a)) return rc;
  if (a->rows && (!loss || !lse)) return MUON_ERR_INVALID;
  if (!is_aligned(loss, 4) || !is_aligned(lse, 4) || !is_aligned(stats, 4)) return MUON_ERR_INVALID;
  CePlan P = {};
  make_plan(a, 0, &P);
  if (!ws || !is_aligned(ws, 256) || ws_bytes < P.total) return MUON_ERR_WORKSPACE;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {
    if (stats && cudaMemsetAsync(stats, 0, 8, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (prepare() != cudaSuccess) return MUON_ERR_CUDA;
  char* w = static_cast<char*>(ws);
  static thread_local OrderedParams p;
  common_params(&p, a, P, w);
  p.part = reinterpret_cast<float2*>(w + P.part);
  p.zlabel = reinterpret_cast<float*>(w + P.zlabel);
  Operand H, W;
  if (operand(&H, a, P, true, false, w, s) != cudaSuccess || operand(&W, a, P, false, false, w, s) != cudaSuccess)
    return MUON_ERR_CUDA;
  Job& j = p.job[0];
  j.kind = LOGITS;
  if (!map_of(&j.a, H) || !map_of(&j.b, W)) return MUON_ERR_CUDA;
  shape(&j, a->rows, a->vocab, a->dim, GROUP_FORWARD);
  j.seg_kb = P.nterms > 1 ? SEG_F32 : SEG_BF16;
  p.njobs = 1;
  p.tiles = j.tiles;
  if (launch(p, false, true, false, s) != cudaSuccess) return MUON_ERR_CUDA;
  count_launch();
  if (launch_after(join_kernel, dim3((unsigned)cdiv(a->rows, JOIN_WARPS)), dim3(32 * JOIN_WARPS), 0, s, p.part,
                   2 * j.ntiles, a->rows, a->labels, a->vocab, a->ignore_index, p.zlabel, loss, lse, stats,
                   reinterpret_cast<float2*>(w + P.sums), reinterpret_cast<unsigned int*>(w) + TICKET_WORD, p.status) !=
      cudaSuccess)
    return MUON_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" int muon_linear_ce_backward(const muon_linear_ce* a, const float* lse, const float* row_grad,
                                       const float* stats, const float* upstream, float grad_scale, void* dH,
                                       void* dW, void* ws, size_t ws_bytes, muon_stream_t stream) {
  using namespace ce;
  begin_launches();
  if (int rc = check(a)) return rc;
  if (int rc = check_pointers(a)) return rc;
  if (a->rows && !lse) return MUON_ERR_INVALID;
  if (!is_aligned(lse, 4) || !is_aligned(row_grad, 4) || !is_aligned(stats, 4) || !is_aligned(upstream, 4))
    return MUON_ERR_INVALID;
  const RowGrads rows = {false, lse, row_grad, stats, upstream, grad_scale, nullptr, nullptr, nullptr};
  return backward_pass(a, rows, dH, dW, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" size_t muon_linear_logprob_workspace_size(const muon_linear_ce* a, int top, int backward) {
  if (ce::check(a) != MUON_OK || top < 0 || top > MUON_LOGPROB_MAX_TOP) return (size_t)-1;
  ce::CePlan P = {};
  ce::make_plan(a, backward, &P, top);
  return P.total;
}

extern "C" int muon_linear_logprob_forward(const muon_linear_ce* a, int top, float* logprob, float* entropy, float* lse,
                                           int64_t* ids, float* alternatives, void* ws, size_t ws_bytes,
                                           muon_stream_t stream) {
  using namespace ce;
  begin_launches();
  if (int rc = check(a)) return rc;
  if (int rc = check_pointers(a, true)) return rc;
  if (top < 0 || top > MUON_LOGPROB_MAX_TOP) return MUON_ERR_INVALID;
  if (a->rows && (!entropy || !lse || (a->labels && !logprob) || (top && (!ids || !alternatives)))) return MUON_ERR_INVALID;
  if (!is_aligned(logprob, 4) || !is_aligned(entropy, 4) || !is_aligned(lse, 4) || !is_aligned(ids, 8) ||
      !is_aligned(alternatives, 4))
    return MUON_ERR_INVALID;
  CePlan P = {};
  make_plan(a, 0, &P, top);
  if (!ws || !is_aligned(ws, 256) || ws_bytes < P.total) return MUON_ERR_WORKSPACE;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) return MUON_OK;
  if (prepare() != cudaSuccess) return MUON_ERR_CUDA;
  char* w = static_cast<char*>(ws);
  static thread_local OrderedParams p;
  common_params(&p, a, P, w);
  p.stat = reinterpret_cast<float4*>(w + P.stat);
  p.keys = top ? reinterpret_cast<float2*>(w + P.keys) : nullptr;
  p.zlabel = reinterpret_cast<float*>(w + P.zlabel);
  const bool w_vec = words_of_w(a);
  Job& j = p.job[0];
  shape(&j, a->rows, a->vocab, a->dim, GROUP_FORWARD);
  if (few_rows(a->rows, a->dim, a->dtype == MUON_DTYPE_F32, false, w_vec)) {
    Few f = few_args(a, w);
    f.stat = p.stat;
    f.keys = p.keys;
    f.zlabel = p.zlabel;
    f.parts = TILE / few_block(a->vocab) * j.ntiles;
    if (few_forward(f, a->dtype == MUON_DTYPE_F32, w_vec, s) != cudaSuccess) return MUON_ERR_CUDA;
    return join_rows(a, top, p, f.parts, logprob, entropy, lse, ids, alternatives, s);
  }
  Operand H, W;
  if (operand(&H, a, P, true, false, w, s) != cudaSuccess || operand(&W, a, P, false, false, w, s) != cudaSuccess)
    return MUON_ERR_CUDA;
  j.kind = LOGPROB;
  if (!map_of(&j.a, H) || !map_of(&j.b, W)) return MUON_ERR_CUDA;
  j.seg_kb = P.nterms > 1 ? SEG_F32 : j.mtiles == 1 ? SEG_FEW : (int)cdiv(j.nkb, cdiv(j.nkb, SEG_BF16));
  p.njobs = 1;
  p.tiles = j.tiles;
  const bool promote = P.nterms > 1 || j.nkb > j.seg_kb;
  if (top) {
    // roundings on the way of one product: the segment's (four steps of 16 products a K step) and the
    // take-overs'; for 32-bit operands also the other terms', 2^-7 of the result, and what no term holds
    const float steps = 4.f * (float)std::min(j.seg_kb, j.nkb) + (float)cdiv(j.nkb, j.seg_kb) + (P.nterms > 1 ? 32.f : 4.f);
    float *hshare = reinterpret_cast<float*>(w + P.hshare), *wlen = reinterpret_cast<float*>(w + P.wlen);
    float* wgroup = wlen + (size_t)j.ntiles * TILE;
    if (lengths(a, H, W, UNIT_TENSOR * steps, hshare, wlen, wgroup, s) != cudaSuccess) return MUON_ERR_CUDA;
    p.hshare = hshare;
    p.wlen = wlen;
    p.wgroup = wgroup;
  }
  if (launch(p, false, promote, true, s) != cudaSuccess) return MUON_ERR_CUDA;
  return join_rows(a, top, p, 2 * j.ntiles, logprob, entropy, lse, ids, alternatives, s);
}

extern "C" int muon_linear_logprob_backward(const muon_linear_ce* a, const float* lse, const float* entropy,
                                            const float* g_logprob, const float* g_entropy, void* dH, void* dW,
                                            void* ws, size_t ws_bytes, muon_stream_t stream) {
  using namespace ce;
  begin_launches();
  if (int rc = check(a)) return rc;
  if (int rc = check_pointers(a)) return rc;
  if (a->rows && (!lse || (g_entropy && !entropy))) return MUON_ERR_INVALID;
  if (!is_aligned(lse, 4) || !is_aligned(entropy, 4) || !is_aligned(g_logprob, 4) || !is_aligned(g_entropy, 4))
    return MUON_ERR_INVALID;
  const RowGrads rows = {true, lse, nullptr, nullptr, nullptr, 1.f, entropy, g_logprob, g_entropy};
  return backward_pass(a, rows, dH, dW, ws, ws_bytes, static_cast<cudaStream_t>(stream));
}
