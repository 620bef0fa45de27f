// Linear cross entropy: what the host side (linear_ce.cu) hands to the tensor-core
// kernel (ce_gemm.cu).
#pragma once

#include "internal.h"

namespace muon {
namespace ce {

constexpr int TILE = 256;          // output tile of a CTA pair, both ways
constexpr int BK = 64;             // K step
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
// covers (k, row); an MN-major one's (row, k).  The maps' third coordinate is the bf16
// part of a 32-bit operand.
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
  const float *lse, *row_grad, *stats;
  float scale;
  unsigned int* status;
  unsigned long long timeout_ns;
  int debug_flags;
  int ordered;                   // tiles follow order[start[pair] .. start[pair + 1]), else round robin
  unsigned short start[MAX_PAIRS + 1];
  unsigned short order[MAX_ORDER];
};
static_assert(sizeof(Params) < 32000, "ce::Params too large");

cudaError_t prepare();           // kernel attributes and occupancy of the current device, once
int pairs();                     // CTA pairs that run at once
cudaError_t launch(const Params& p, bool promote, cudaStream_t s);

}  // namespace ce
}  // namespace muon
