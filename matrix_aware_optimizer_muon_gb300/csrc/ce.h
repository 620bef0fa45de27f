// Linear cross entropy: what the host side (linear_ce.cu) hands to the tensor-core
// kernel (ce_gemm.cu).
#pragma once

#include "internal.h"

namespace muon {
namespace ce {

constexpr int TILE = 256;          // output tile of a CTA pair, both ways
constexpr int BK = 64;             // K step
constexpr int BOX = 64;            // rows of a TMA box
constexpr int MAX_JOBS = 3;
constexpr int MAX_PAIRS = 80;
constexpr int MAX_ORDER = 12000;   // tiles of a launch whose order the host lays out
constexpr int MAX_TERMS = 6;

enum Kind : int {
  LOGITS = 0,   // per row and 128 columns: max and sum of exponentials; the label's logit
  GRAD = 1,     // g = c (exp(z - lse) - onehot), in bf16 (or three bf16 parts)
  DH = 2,       // g W, summed over the pieces in fp32
  DW = 3        // g^T H
};

// One product of a launch: out[m, n] = sum_k A[m, k] B[n, k].  A K-major operand's map
// covers (k, row), an MN-major one's (row, k), in boxes of 64 x 64.  The maps' third
// coordinate is the bf16 part of a 32-bit operand.
struct Job {
  CUtensorMap a, b;
  int kind;
  int a_mn, b_mn;
  int m, n;              // valid rows and columns of the output
  int b_n0, b_k0;        // first row, or first k, of the piece inside B's map
  int mtiles, ntiles, group;  // tiles; row tiles that are walked together
  int tiles, begin;      // number of tiles, first tile of the launch
  int splits;            // DH: K is cut into so many ranges, each with sums of its own
  int nkb, seg_kb;       // K steps of one range; K steps after which a sum is taken over (promoted)
  // outputs
  void* out;             // GRAD: g;  DH, DW: result (rows of ldo elements) or null
  long long ldo;
  long long part_stride; // GRAD: elements between the parts of g
  float* acc;            // DH: running sums [splits][m][ldacc]
  long long ldacc;
  int first, last;       // DH: first piece, last piece of the vocabulary
  int vec;               // DH, DW: result rows start 32-byte aligned (2), 16-byte aligned (1) or neither (0)
};

struct Params {
  Job job[MAX_JOBS];
  int njobs;
  int tiles;
  int nterms, parts;
  unsigned char ta[MAX_TERMS], tb[MAX_TERMS];  // parts of A and B multiplied in each term
  int f32_out;
  // logits
  const int64_t* labels;
  long long vocab, ignore, v0;   // v0: first vocabulary row of the GRAD piece
  float2* part;                  // LOGITS: [row][2 * ntiles]
  float* zlabel;
  const float *lse, *row_grad, *stats, *upstream;
  float scale;
  unsigned int* status;
  unsigned long long timeout_ns;
  int debug_flags;
};
// The same with the tiles laid out by the host: pair i takes order[start[i] .. start[i + 1]).
// A launch whose tiles go round robin is not charged for the table.
struct OrderedParams : Params {
  unsigned short start[MAX_PAIRS + 1];
  unsigned short order[MAX_ORDER];
};
static_assert(sizeof(OrderedParams) < 32000, "ce::OrderedParams too large");

cudaError_t prepare();           // kernel attributes and occupancy of the current device, once
int pairs();                     // CTA pairs that run at once
cudaError_t launch(const OrderedParams& p, bool ordered, bool promote, cudaStream_t s);

#ifdef __CUDACC__
// The factor that all rows share.
__device__ __forceinline__ float shared_factor(float scale, const float* upstream, const float* stats) {
  if (upstream) scale *= *upstream;
  if (stats) scale /= fmaxf(stats[1], 1.f);
  return scale;
}
#endif

}  // namespace ce
}  // namespace muon
