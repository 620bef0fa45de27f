// Linear cross entropy and log probabilities: what the host side (linear_ce.cu) hands to
// the tensor-core kernel (ce_gemm.cu).
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
  DW = 3,       // g^T H
  LOGPROB = 4,  // LOGITS, and the sum that the entropy takes and the largest of each 32 columns
  POLICY = 5    // GRAD of log probabilities and entropies
};

// The two largest of 32 columns as keys: the number's lowest 5 bits hold 31 minus the
// column, so that two maxima a logit find them without carrying an index.  The numbers are
// upper bounds on the exact logits: a first sum is off by a share of |h||w| (the rows'
// lengths), however small the sum itself is, and that share is added before the key is made.
constexpr int KEY_COLS = 32;
constexpr unsigned KEY_MASK = KEY_COLS - 1;
// The share: a unit for each rounding that a product can pass on its way into the sum (fp32
// additions 2^-24 each; a step of the tensor cores, which truncate, measured 2^-24 for 16 products of one
// sign and allowed four times that), and a fiftieth for the lengths' own sums.
constexpr float UNIT_FP32 = 0x1.05p-24f, UNIT_TENSOR = 0x1.05p-22f;

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
  float4* stat;                  // LOGPROB: [row][2 * ntiles] max m, sum of e^(z-m), sum of e^(z-m) (z-m)
  float2* keys;                  // LOGPROB: [row][8 * ntiles], or null
  // with keys: [row] share of |h|, [column] length of a row of W, [32 columns] the largest, or -1 where
  // their lengths differ (a whole tile's, with some finite length behind the vocabulary)
  const float *hshare, *wlen, *wgroup;
  const float *entropy, *g_logprob, *g_entropy;   // POLICY
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
cudaError_t launch(const OrderedParams& p, bool ordered, bool promote, bool logprob, cudaStream_t s);

// A call with few rows (logprob_few.cu).
constexpr int FEW_MAX_CTAS = 608;
struct Few {
  const void *H, *W;
  const int64_t* labels;
  long long ldh, ldw, vocab, ignore;
  int rows, dim, dp, masked;     // dp: padded row of the staged H;  masked: rows without a token count as zeros
  const unsigned int* status;
  // forward: as in Params, parts statistics a row
  float4* stat;
  float2* keys;
  float* zlabel;
  int parts;                     // statistics a row
  float share;                   // with keys: what a logit may be off by, over |h||w|
  // backward
  const float *lse, *entropy, *g_logprob, *g_entropy;
  float* dh_part;                // [CTA][rows, padded][dp], or null
  void* dW;
};
bool few_rows(int64_t rows, int64_t dim, bool f32, bool backward, bool vec);   // whether it is one; vec: W in 16-byte words
size_t few_bytes(int64_t rows, int64_t dim);     // of dh_part
int few_block(int64_t vocab);                    // columns of a statistic
cudaError_t few_forward(Few p, bool f32, bool vec, cudaStream_t s);
cudaError_t few_backward(Few p, bool f32, bool vec, void* dH, cudaStream_t s);

#ifdef __CUDACC__
// A row's length from the sum of its squares, between 2^-60 and 2^63: what fp32's squares lose
// below is too much of a bound and never too little; longer rows are masks (a product of two
// such lengths stays away from a masked logit's 2^120).
__device__ __forceinline__ float length_of(float squares) { return sqrtf(fminf(fmaxf(squares, 0x1p-120f), 0x1p126f)); }
// The share of a row of H; none for a row of zeros, whose logits are exact.
__device__ __forceinline__ float share_of(float squares, float largest, float share) {
  return largest == 0.f ? 0.f : fminf(share * length_of(squares), 0x1p50f);
}
// The factor that all rows share.
__device__ __forceinline__ float shared_factor(float scale, const float* upstream, const float* stats) {
  if (upstream) scale *= *upstream;
  if (stats) scale /= fmaxf(stats[1], 1.f);
  return scale;
}
#endif

}  // namespace ce
}  // namespace muon
