// Softmax cross entropy of the logits z = H W^T, without keeping the logits.
//
//   forward:  per row and 128 columns of the vocabulary, max and sum of exponentials
//             (in the product's epilogue); lse = max + log(sum) joined over them;
//             loss = lse - z[label].
//   backward: g = c (exp(z - lse) - onehot) by pieces of the vocabulary;
//             dH += g W_piece,  dW_piece = g^T H.
//
// The products run in ce_gemm.cu; here are the plan of a call, the join and the copies
// that bring operands into a layout TMA can read.
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
int check_pointers(const muon_linear_ce* a) {
  if (!a->W || !is_aligned(a->W, dt_size(a->dtype))) return MUON_ERR_INVALID;
  if (a->rows && (!a->H || !a->labels || !is_aligned(a->H, dt_size(a->dtype)) || !is_aligned(a->labels, 8)))
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

void make_plan(const muon_linear_ce* a, int backward, CePlan* P) {
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
  P->hp = take((size_t)P->parts * a->rows * P->dp * 2);
  P->wp = P->pack_w ? take((size_t)P->parts * a->vocab * P->dp * 2) : at;
  const size_t common = at;
  P->zlabel = take((size_t)a->rows * 4);
  P->part = take((size_t)a->rows * 2 * cdiv(a->vocab, TILE) * sizeof(float2));
  P->sums = take((size_t)cdiv(a->rows, JOIN_WARPS) * sizeof(float2));
  P->total = at;
  if (!backward) return;
  at = common;
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

}  // namespace
}  // namespace ce
}  // namespace muon

using namespace muon;

extern "C" size_t muon_linear_ce_workspace_size(const muon_linear_ce* a, int backward) {
  if (ce::check(a) != MUON_OK) return (size_t)-1;
  ce::CePlan P;
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
  if (launch(p, false, true, s) != cudaSuccess) return MUON_ERR_CUDA;
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
  const size_t es = dt_size(a->dtype);
  if (a->rows && !lse) return MUON_ERR_INVALID;
  if (!is_aligned(lse, 4) || !is_aligned(row_grad, 4) || !is_aligned(stats, 4) || !is_aligned(upstream, 4) ||
      !is_aligned(dH, es) || !is_aligned(dW, es))
    return MUON_ERR_INVALID;
  CePlan P = {};
  make_plan(a, 1, &P);
  if (!ws || !is_aligned(ws, 256) || ws_bytes < P.total) return MUON_ERR_WORKSPACE;
  if (!dH && !dW) return MUON_OK;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {
    if (dW && cudaMemsetAsync(dW, 0, (size_t)a->vocab * a->dim * es, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  if (prepare() != cudaSuccess) return MUON_ERR_CUDA;
  char* w = static_cast<char*>(ws);
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
    p.lse = lse;
    p.row_grad = row_grad;
    p.stats = stats;
    p.upstream = upstream;
    p.scale = grad_scale;
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
      j.kind = GRAD;
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
    if (launch(p, ordered, promote, s) != cudaSuccess) return MUON_ERR_CUDA;
  }
  const cudaError_t e = f32 ? finish<float>(a, P, acc, p, static_cast<float*>(dH), static_cast<float*>(dW), s)
                            : finish<bf16>(a, P, acc, p, static_cast<bf16*>(dH), static_cast<bf16*>(dW), s);
  if (e != cudaSuccess) return MUON_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
