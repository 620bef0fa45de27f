// Softmax cross entropy of the logits z = H W^T, without keeping the logits.
//
//   forward:  per piece of the vocabulary, max and sum of exponentials of each row;
//             lse = max + log(sum), joined over the pieces; loss = lse - z[label].
//   backward: g = c (exp(z - lse) - onehot) by pieces of the vocabulary;
//             dH += g W_piece,  dW_piece = g^T H.
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "internal.h"

namespace muon {
namespace ce {

constexpr int BT = 64, BKS = 16, THREADS = 256;   // 64 x 64 tile, 4 x 4 a thread
constexpr int64_t PIECE = 4096;                   // vocabulary columns of one backward piece

struct Gemm {
  // C[i, j] = sum_k A[i*sai + k*sak] * B[j*sbj + k*sbk], i < m, j < n, k < kk
  const void *A, *B;
  long long sai, sak, sbj, sbk;
  long long m, n, kk;
  // LOGITS epilogues
  const int64_t* labels;
  long long v0, vocab, ignore;
  float2* part;          // FWD: [column tiles][m]
  float* zlabel;         // FWD
  const float *lse, *row_grad, *stats;
  float scale;
  void* out;             // GRAD: fp32 g; DH: fp32 running sum; DW: result
  long long ldo;
  void* fin;             // DH: result, on the last piece
  int first, last;
};
enum { FWD = 0, GRAD = 1, DH = 2, DW = 3 };

template <int kEpi, typename TA, typename TB, typename TO>
__global__ void __launch_bounds__(THREADS) gemm_kernel(const Gemm p) {
  __shared__ float As[BKS][BT + 1], Bs[BKS][BT + 1];
  __shared__ float2 red[BT][17];
  const long long i0 = (long long)blockIdx.y * BT, j0 = (long long)blockIdx.x * BT;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const TA* A = static_cast<const TA*>(p.A);
  const TB* B = static_cast<const TB*>(p.B);
  float acc[4][4] = {};
  for (long long k0 = 0; k0 < p.kk; k0 += BKS) {
    for (int t = threadIdx.x; t < BT * BKS; t += THREADS) {
      int i, k;
      if (p.sak == 1) { i = t / BKS; k = t % BKS; } else { i = t % BT; k = t / BT; }
      As[k][i] = (i0 + i < p.m && k0 + k < p.kk) ? ld1(A + (i0 + i) * p.sai + (k0 + k) * p.sak) : 0.f;
      if (p.sbk == 1) { i = t / BKS; k = t % BKS; } else { i = t % BT; k = t / BT; }
      Bs[k][i] = (j0 + i < p.n && k0 + k < p.kk) ? ld1(B + (j0 + i) * p.sbj + (k0 + k) * p.sbk) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < BKS; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) { a[u] = As[k][ty * 4 + u]; b[u] = Bs[k][tx * 4 + u]; }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) acc[u][w] = fmaf(a[u], b[w], acc[u][w]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const long long i = i0 + ty * 4 + u;
    if (kEpi == FWD) {
      float mx = -INFINITY, s = 0.f;
      const long long lab = i < p.m ? p.labels[i] : -1;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const long long j = j0 + tx * 4 + w;
        if (j < p.n) mx = fmaxf(mx, acc[u][w]);
        if (j < p.n && i < p.m && j == lab) p.zlabel[i] = acc[u][w];
      }
      const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (j0 + tx * 4 + w < p.n) s += expf(acc[u][w] - ref);
      red[ty * 4 + u][tx] = make_float2(mx, s);
    } else if (kEpi == GRAD) {
      if (i >= p.m) continue;
      const long long lab = p.labels[i];
      float c = p.scale;
      if (p.row_grad) c *= p.row_grad[i];
      if (p.stats) c /= fmaxf(p.stats[1], 1.f);
      const bool counted = lab != p.ignore && lab >= 0 && lab < p.vocab;
      for (int w = 0; w < 4; ++w) {
        const long long j = j0 + tx * 4 + w;
        if (j >= p.n) continue;
        const float g = counted ? c * (expf(acc[u][w] - p.lse[i]) - (p.v0 + j == lab ? 1.f : 0.f)) : 0.f;
        static_cast<float*>(p.out)[i * p.ldo + j] = g;
      }
    } else {
      for (int w = 0; w < 4; ++w) {
        const long long j = j0 + tx * 4 + w;
        if (i >= p.m || j >= p.n) continue;
        if (kEpi == DH) {
          float* o = static_cast<float*>(p.out) + i * p.ldo + j;
          const float v = acc[u][w] + (p.first ? 0.f : *o);
          if (p.last) st1(static_cast<TO*>(p.fin) + i * p.ldo + j, v);
          else *o = v;
        } else {
          st1(static_cast<TO*>(p.out) + i * p.ldo + j, acc[u][w]);
        }
      }
    }
  }
  if (kEpi == FWD) {
    __syncthreads();
    if (threadIdx.x < BT && i0 + threadIdx.x < p.m) {
      float mx = -INFINITY, s = 0.f;
      for (int t = 0; t < 16; ++t) mx = fmaxf(mx, red[threadIdx.x][t].x);
      const float ref = mx == -INFINITY ? 0.f : mx;
      for (int t = 0; t < 16; ++t) {
        const float2 q = red[threadIdx.x][t];
        s += q.x == -INFINITY ? q.y : q.y * expf(q.x - ref);
      }
      p.part[(size_t)blockIdx.x * p.m + i0 + threadIdx.x] = make_float2(mx, s);
    }
  }
}

// Joins the pieces of each row; one thread a row.
__global__ void join_kernel(const float2* part, int parts, long long rows, const int64_t* labels, long long vocab,
                            long long ignore, const float* zlabel, float* loss, float* lse) {
  const long long r = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (r >= rows) return;
  float mx = -INFINITY, s = 0.f;
  for (int t = 0; t < parts; ++t) mx = fmaxf(mx, part[(size_t)t * rows + r].x);
  const float ref = mx == -INFINITY ? 0.f : mx;
  for (int t = 0; t < parts; ++t) {
    const float2 q = part[(size_t)t * rows + r];
    s += q.x == -INFINITY ? q.y : q.y * expf(q.x - ref);
  }
  const float l = ref + logf(s);
  lse[r] = l;
  const long long lab = labels[r];
  loss[r] = lab == ignore ? 0.f : (lab < 0 || lab >= vocab) ? __int_as_float(0x7FC00000) : l - zlabel[r];
}

// Mean loss over the rows that are not ignored; one block, fixed order.
__global__ void __launch_bounds__(1024) stats_kernel(const float* loss, const int64_t* labels, long long rows,
                                                     long long ignore, float* stats) {
  __shared__ float red[32];
  float s = 0.f, c = 0.f;
  for (long long r = threadIdx.x; r < rows; r += 1024)
    if (labels[r] != ignore) { s += loss[r]; c += 1.f; }
  s = block_sum(s, red);
  c = block_sum(c, red);
  if (threadIdx.x == 0) {
    stats[0] = s / fmaxf(c, 1.f);
    stats[1] = c;
  }
}

constexpr size_t HEADER = 256;
size_t up(size_t x) { return (x + 255) / 256 * 256; }
size_t dt_size(int dt) { return dt == MUON_DTYPE_BF16 ? 2 : 4; }
bool is_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check(const muon_linear_ce* a) {
  if (!a) return MUON_ERR_INVALID;
  const int64_t lim = 1LL << 31;
  if (a->rows < 0 || a->rows >= lim || a->vocab < 1 || a->vocab >= lim || a->dim < 1 || a->dim >= lim ||
      a->ldh < a->dim || a->ldw < a->dim)
    return MUON_ERR_INVALID;
  if (a->dtype != MUON_DTYPE_F32 && a->dtype != MUON_DTYPE_BF16) return MUON_ERR_UNSUPPORTED;
  return MUON_OK;
}
int check_pointers(const muon_linear_ce* a) {
  if (!a->W || !is_aligned(a->W, dt_size(a->dtype))) return MUON_ERR_INVALID;
  if (a->rows && (!a->H || !a->labels || !is_aligned(a->H, dt_size(a->dtype)) || !is_aligned(a->labels, 8)))
    return MUON_ERR_INVALID;
  return MUON_OK;
}

template <int kEpi, typename TA, typename TB, typename TO>
void launch(const Gemm& p, cudaStream_t s) {
  gemm_kernel<kEpi, TA, TB, TO><<<dim3((unsigned)((p.n + BT - 1) / BT), (unsigned)((p.m + BT - 1) / BT)), THREADS, 0,
                                  s>>>(p);
  count_launch();
}

template <typename T>
void backward(const muon_linear_ce* a, Gemm base, void* dH, void* dW, float* g, float* acc, cudaStream_t s) {
  const size_t es = sizeof(T);
  for (int64_t v0 = 0; v0 < a->vocab; v0 += PIECE) {
    const int64_t c = std::min(PIECE, a->vocab - v0);
    const char* Wp = static_cast<const char*>(a->W) + (size_t)v0 * a->ldw * es;
    Gemm p = base;
    p.A = a->H; p.sai = a->ldh; p.sak = 1; p.B = Wp; p.sbj = a->ldw; p.sbk = 1;
    p.m = a->rows; p.n = c; p.kk = a->dim; p.v0 = v0; p.out = g; p.ldo = PIECE;
    launch<GRAD, T, T, float>(p, s);
    if (dH) {
      p.A = g; p.sai = PIECE; p.sak = 1; p.B = Wp; p.sbj = 1; p.sbk = a->ldw;
      p.m = a->rows; p.n = a->dim; p.kk = c; p.out = acc; p.fin = dH; p.ldo = a->dim;
      p.first = v0 == 0; p.last = v0 + c == a->vocab;
      launch<DH, float, T, T>(p, s);
    }
    if (dW) {
      p.A = g; p.sai = 1; p.sak = PIECE; p.B = a->H; p.sbj = 1; p.sbk = a->ldh;
      p.m = c; p.n = a->dim; p.kk = a->rows; p.out = static_cast<char*>(dW) + (size_t)v0 * a->dim * es; p.ldo = a->dim;
      launch<DW, float, T, T>(p, s);
    }
  }
}

}  // namespace ce
}  // namespace muon

using namespace muon;

extern "C" size_t muon_linear_ce_workspace_size(const muon_linear_ce* a, int backward) {
  if (ce::check(a) != MUON_OK) return (size_t)-1;
  const size_t n = (size_t)a->rows;
  const size_t fwd = ce::up(n * 4) + ce::up(n * ((a->vocab + ce::BT - 1) / ce::BT) * 8);
  const size_t bwd = ce::up(n * ce::PIECE * 4) + ce::up(n * a->dim * 4);
  return ce::HEADER + (backward ? std::max(fwd, bwd) : fwd);
}

extern "C" int muon_linear_ce_forward(const muon_linear_ce* a, float* loss, float* lse, float* stats, void* ws,
                                      size_t ws_bytes, muon_stream_t stream) {
  begin_launches();
  if (int rc = ce::check(a)) return rc;
  if (int rc = ce::check_pointers(a)) return rc;
  if (a->rows && (!loss || !lse)) return MUON_ERR_INVALID;
  if (!ce::is_aligned(loss, 4) || !ce::is_aligned(lse, 4) || !ce::is_aligned(stats, 4)) return MUON_ERR_INVALID;
  if (!ws || !ce::is_aligned(ws, 256) || ws_bytes < muon_linear_ce_workspace_size(a, 0)) return MUON_ERR_WORKSPACE;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(ws) + ce::HEADER;
  ce::Gemm p = {};
  p.zlabel = reinterpret_cast<float*>(w);
  p.part = reinterpret_cast<float2*>(w + ce::up((size_t)a->rows * 4));
  p.labels = a->labels; p.vocab = a->vocab; p.ignore = a->ignore_index;
  p.A = a->H; p.sai = a->ldh; p.sak = 1; p.B = a->W; p.sbj = a->ldw; p.sbk = 1;
  p.m = a->rows; p.n = a->vocab; p.kk = a->dim;
  if (a->rows) {
    if (a->dtype == MUON_DTYPE_BF16) ce::launch<ce::FWD, bf16, bf16, float>(p, s);
    else ce::launch<ce::FWD, float, float, float>(p, s);
    ce::join_kernel<<<(unsigned)((a->rows + 127) / 128), 128, 0, s>>>(
        p.part, (int)((a->vocab + ce::BT - 1) / ce::BT), a->rows, a->labels, a->vocab, a->ignore_index, p.zlabel, loss,
        lse);
    count_launch();
  }
  if (stats) {
    ce::stats_kernel<<<1, 1024, 0, s>>>(loss, a->labels, a->rows, a->ignore_index, stats);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

extern "C" int muon_linear_ce_backward(const muon_linear_ce* a, const float* lse, const float* row_grad,
                                       const float* stats, float grad_scale, void* dH, void* dW, void* ws,
                                       size_t ws_bytes, muon_stream_t stream) {
  begin_launches();
  if (int rc = ce::check(a)) return rc;
  if (int rc = ce::check_pointers(a)) return rc;
  const size_t es = ce::dt_size(a->dtype);
  if (a->rows && !lse) return MUON_ERR_INVALID;
  if (!ce::is_aligned(lse, 4) || !ce::is_aligned(row_grad, 4) || !ce::is_aligned(stats, 4) ||
      !ce::is_aligned(dH, es) || !ce::is_aligned(dW, es))
    return MUON_ERR_INVALID;
  if (!ws || !ce::is_aligned(ws, 256) || ws_bytes < muon_linear_ce_workspace_size(a, 1)) return MUON_ERR_WORKSPACE;
  if (!dH && !dW) return MUON_OK;
  int sms = 0;
  if (int rc = require_device(&sms)) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->rows == 0) {
    if (dW && cudaMemsetAsync(dW, 0, (size_t)a->vocab * a->dim * es, s) != cudaSuccess) return MUON_ERR_CUDA;
    return MUON_OK;
  }
  char* w = static_cast<char*>(ws) + ce::HEADER;
  float* g = reinterpret_cast<float*>(w);
  float* acc = reinterpret_cast<float*>(w + ce::up((size_t)a->rows * ce::PIECE * 4));
  ce::Gemm p = {};
  p.labels = a->labels; p.vocab = a->vocab; p.ignore = a->ignore_index;
  p.lse = lse; p.row_grad = row_grad; p.stats = stats; p.scale = grad_scale;
  if (a->dtype == MUON_DTYPE_BF16) ce::backward<bf16>(a, p, dH, dW, g, acc, s);
  else ce::backward<float>(a, p, dH, dW, g, acc, s);
  return cudaGetLastError() == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}
