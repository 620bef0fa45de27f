// The products of the linear cross entropy on the sm_103a tensor cores (tcgen05, TMEM,
// TMA), with the softmax fused into their epilogues.
//
// A 2-CTA cluster (cta_group::2) computes a 256 x 256 output tile; each CTA stages its
// 128 rows of A and 128 rows of B (32 KB a K step of 64).
// 384 threads a CTA:
//   warps 0, 2  TMA producers (one lane each) of A and of B, a ring of STAGES K steps.
//               Two, and in boxes of 64 rows: a request takes a lane about 100 cycles
//               to issue, and one of 128 rows 400 to serve.  Loads alone would feed
//               1.50 PFLOP/s from one lane in boxes of 128, 1.68 in boxes of 64, 2.54
//               from two lanes (the MMAs alone run at 2.08);
//   warp 1      tensor-memory allocation; in the even CTA one lane issues the MMAs;
//   warps 4..11 epilogue, two per TMEM lane quarter, 128 of the 256 columns each: a
//               thread owns one row, so a row's max and sum need no shuffles.
// Two 256-column fp32 accumulators: the epilogue of a tile overlaps the next one's MMAs.
//
// One launch runs up to three products (jobs) over one list of tiles.  The backward
// pass multiplies g of piece i twice (dH and dW) while it computes g of piece i+1, so
// the short lists of dH tiles never leave SMs idle at the end of a launch of their own.
//
// The tensor cores add to the fp32 accumulator with truncation; its bias grows with the
// number of K steps (measured: 2.3e-7 of a sum of 256 bf16 products, 1e-6 of 1024,
// 9e-6 of 8192).  Taking it over while the MMAs run is slow, for they have the tensor
// memory's ports most of the time.  The kPromote form takes the accumulator over into registers every
// seg_kb K steps and adds there with rounding to nearest (five take-overs of a tile of
// 2560 products instead of two cost 8%).  It serves the logits of the forward pass, whose
// loss is fp32, every product of 32-bit operands, and launches with sums of more than 2^16
// products; shorter ones that are rounded to bf16 (4e-3) do without.
//
// 32-bit operands come as three bf16 parts (24 bits of mantissa); the six products of
// parts down to 2^-16 of the leading one are summed, smallest first.
//
// Measured (8192 rows, 2560 wide, 131072 entries, bf16, in loops of 0.1 to 0.3 s, several
// GPUs): forward 3.16 to 3.45 ms (1.59 to 1.74 PFLOP/s), backward 9.9 to 11.1 ms (1.49 to
// 1.66).  In turn on one GPU the forward pass took 3.21, 3.36 and 3.45 ms and the library's
// product of the same operands, which writes the logits, 2.98, 3.16 and 3.11.  The tensor pipe is
// busy 78% (forward), 79% (g) and 89% (the products with g) of the time in single launches,
// at 1.65 to 1.8 GHz; in loops the 1.4 kW power cap sets the clock.  Without its
// exponentials the forward pass takes 4% less; waits that suspend the thread for longer, and
// sharing an operand among clusters of four CTAs, change nothing.
// 8 rows read the vocabulary matrix at 5.9 TB/s after some 11 us of launches and set-up.
//
// Exponentials are __expf: off by 2 ulp near 0 and by 1.2 |x| ulp further down, where they
// count less (x <= 0; at -16 they are 1e-7 of the largest and 1.2e-6 of that off).  A row's sum is
// within some 1e-7 of itself by them, less than the sum over 2^17 entries and the logits'
// own error (4e-7 of the loss) bring.  The bf16 gradient rounds by 4e-3.
#include <map>
#include <mutex>

#include "ce.h"
#include "common.cuh"
#include "ptx.cuh"

namespace muon {
namespace ce {
namespace {

constexpr int HALF = TILE / 2;
constexpr int OP_BYTES = HALF * BK * 2;        // one operand's 128 rows of a K step
constexpr int STAGE_BYTES = 2 * OP_BYTES;
constexpr int BOX_BYTES = BOX * BK * 2;        // two boxes an operand, one above the other in either major
constexpr int STAGES = 6;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int CHUNKS = 4;                      // 32-column chunks of an epilogue warp
constexpr uint32_t TMEM_COLS = 512;
constexpr int XPOSE = 32 * 17;                  // floats an epilogue warp stages: 32 rows of 16 columns
constexpr int SMEM = STAGES * STAGE_BYTES + 1024 + 256 + EPI_WARPS * XPOSE * 4;

// A job's numbers, copied to shared memory: every role reads them for every tile, and with
// the tile table in the parameters the constant cache does not hold them.
struct Work {
  int kind, a_mn, b_mn, m, n, b_n0, b_k0, mtiles, ntiles, group, begin, splits, nkb, seg_kb, first, last, vec;
  void* out;
  float* acc;
  long long ldo, ldacc, part_stride;
};

struct Tile {
  int job, tm, tn, split;
};

__device__ __forceinline__ Tile decode(const Work* jobs, int njobs, int t) {
  Tile ti;
  int j = 0;
  while (j + 1 < njobs && jobs[j + 1].begin <= t) ++j;
  const Work& J = jobs[j];
  ti.job = j;
  int r = t - J.begin;
  ti.split = 0;
  if (J.splits > 1) {
    const int per = J.mtiles * J.ntiles;
    ti.split = r / per;
    r -= ti.split * per;
  }
  int g = 0, rows = J.mtiles;
  if (J.group < rows) {
    g = r / (J.group * J.ntiles);
    r -= g * J.group * J.ntiles;
    rows = min(J.group, J.mtiles - g * J.group);
  }
  ti.tn = r / rows;
  ti.tm = g * J.group + (r - ti.tn * rows);
  return ti;
}

// The pair's k-th tile, or -1.
__device__ __forceinline__ int tile_at(const OrderedParams& p, int pair, int, int k) {
  const int i = p.start[pair] + k;
  return i < p.start[pair + 1] ? p.order[i] : -1;
}
__device__ __forceinline__ int tile_at(const Params& p, int pair, int npairs, int k) {
  const int t = pair + k * npairs;
  return t < p.tiles ? t : -1;
}

// A tile's K steps run through its terms, the products of the operands' leading parts
// last.  The accumulator is taken over after each segment: SMALL_SEG steps of the other
// terms (2^-8 of the result at most, and their truncation with them), seg_kb of the last.
constexpr int SMALL_SEG = 256;
__device__ __forceinline__ int segment_at(const Work& J, int nterms, int kb) {
  const int small = (nterms - 1) * J.nkb;
  return kb < small ? min(SMALL_SEG, small - kb) : min(J.seg_kb, nterms * J.nkb - kb);
}
__device__ __forceinline__ int segments(const Work& J, int nterms) {
  return ((nterms - 1) * J.nkb + SMALL_SEG - 1) / SMALL_SEG + (J.nkb + J.seg_kb - 1) / J.seg_kb;
}

// Bounded wait: on expiry the status word and the CTA's abort flag are set and every
// role leaves its loop.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* abort_flag, const Params& p,
                                         bool honor_abort) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    if (honor_abort && *abort_flag) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      *abort_flag = 1;
      atomicOr(p.status, DEV_TIMEOUT);
      return false;
    }
  }
}

// 32 consecutive results of one row: cols of them are inside the matrix.
template <typename T>
__device__ __forceinline__ void store_row(T* dst, const float (&v)[32], int cols, int vec) {
  if (cols >= 32 && vec) {
    if (sizeof(T) == 2) {
      uint32_t w[16];
#pragma unroll
      for (int h = 0; h < 16; ++h) w[h] = pack_bf16x2(v[2 * h], v[2 * h + 1]);
      if (vec == 2) {
        st_v8(dst, w);
        st_v8(reinterpret_cast<uint8_t*>(dst) + 32, w + 8);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<uint4*>(dst)[q] = make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        reinterpret_cast<float4*>(dst)[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < cols) st1(dst + j, v[j]);
  }
}

// The same for rows that start on no vector boundary: 32 rows (row0 the first, m the
// matrix's) by way of shared memory, so that a store covers 16 neighbouring columns of two
// rows instead of one element of 32 (a sector each).  Called by whole warps.
template <typename T>
__device__ __forceinline__ void store_staged(T* out, long long ldo, int row0, int m, int c0, int cols,
                                             const float (&v)[32], float* stage, int lane) {
  const int cc = lane & 15, rr = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) stage[lane * 17 + j] = v[16 * h + j];
    __syncwarp();
    if (16 * h + cc < cols) {
      T* o = out + (size_t)(row0 + rr) * ldo + c0 + 16 * h + cc;
      const float* x = stage + rr * 17 + cc;
#pragma unroll 4
      for (int i = 0; i < 16; ++i, o += 2 * ldo)
        if (row0 + rr + 2 * i < m) st1(o, x[2 * i * 17]);
    }
  }
}

// Row constants of a GRAD tile: c (0 for a row without gradient), lse and the label's
// column inside the piece.
struct RowIn {
  float c, lse;
  long long label;
};
__device__ __forceinline__ RowIn row_in(const Params& p, int r) {
  const long long lab = p.labels[r];
  RowIn x;
  x.lse = p.lse[r];
  x.label = lab - p.v0;
  const float c = p.row_grad ? p.row_grad[r] : 1.f;
  x.c = (lab == p.ignore || lab < 0 || lab >= p.vocab) ? 0.f : c;
  // a row without gradient gives zeros even where its logits or lse are not finite
  if (lab == p.ignore || lab < 0 || lab >= p.vocab) x.lse = INFINITY;
  return x;
}

// g goes into both products as an operand of the tensor cores, so in the operands' type: bf16
// (an error of 2.2e-3 of dH and dW with their own rounding, which alone is 1.7e-3), or three
// bf16 parts for 32 bits.
__device__ __forceinline__ void finish_grad(const Params& p, const Work& J, int r, int c0, float (&v)[32],
                                            const RowIn& x) {
  if (r >= J.m || c0 >= J.n) return;
  const bool dead = x.lse == INFINITY && x.c == 0.f;
  const int at = x.label >= c0 && x.label < c0 + 32 ? (int)(x.label - c0) : -1;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    float e = __expf(v[j] - x.lse);
    if (j == at) e -= 1.f;
    v[j] = dead ? 0.f : x.c * e;
  }
  bf16* dst = static_cast<bf16*>(J.out) + (size_t)r * J.ldo + c0;
  store_row(dst, v, J.n - c0, 2);
  for (int q = 1; q < p.parts; ++q) {
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
    store_row(dst + q * J.part_stride, v, J.n - c0, 2);
  }
}

__device__ __forceinline__ void finish_sum(const Params& p, const Work& J, int split, int r, int c0, float u,
                                           float* stage, int lane, float (&v)[32]) {
  if (c0 >= J.n) return;
  const int cols = J.n - c0;
  if (J.kind == DH && J.acc) {
    const bool more = !J.last || !J.out;
    if (r < J.m) {
      float* a = J.acc + ((size_t)split * J.m + r) * J.ldacc + c0;
      if (!J.first) {
        if (cols >= 32) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[8];
            ld_v8(a + 8 * q, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * q + j] += __uint_as_float(w[j]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j < cols) v[j] += a[j];
        }
      }
      if (more) store_row(a, v, cols, 2);
    }
    if (more) return;
  }
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] *= u;
  if (J.vec) {
    if (r >= J.m) return;
    if (p.f32_out) store_row(static_cast<float*>(J.out) + (size_t)r * J.ldo + c0, v, cols, J.vec);
    else store_row(static_cast<bf16*>(J.out) + (size_t)r * J.ldo + c0, v, cols, J.vec);
  } else {
    if (p.f32_out) store_staged(static_cast<float*>(J.out), J.ldo, r - lane, J.m, c0, cols, v, stage, lane);
    else store_staged(static_cast<bf16*>(J.out), J.ldo, r - lane, J.m, c0, cols, v, stage, lane);
  }
}

// Max, sum of exponentials and the label's logit over this thread's 128 columns.
__device__ __forceinline__ void finish_logits(const Params& p, const Work& J, const Tile& ti, int half, int r, int cbase,
                                              const float (&acc)[CHUNKS][32]) {
  if (r >= J.m) return;
  const int cols = J.n - cbase;
  float mx = -INFINITY;
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (k * 32 + j < cols) mx = fmaxf(mx, acc[k][j]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float s = 0.f;
#pragma unroll
  for (int k = 0; k < CHUNKS; ++k) {
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (k * 32 + j < cols) q += __expf(acc[k][j] - ref);
    s += q;
  }
  p.part[(size_t)r * (2 * J.ntiles) + 2 * ti.tn + half] = make_float2(mx, s);
  const long long at = p.labels[r] - cbase;
  if (at >= 0 && at < HALF && at < cols) {
    float z = 0.f;
#pragma unroll
    for (int k = 0; k < CHUNKS; ++k)
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (k * 32 + j == (int)at) z = acc[k][j];
    p.zlabel[r] = z;
  }
}

template <bool kPromote, class P>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1) ce_kernel(const __grid_constant__ P p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* mdone = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mdone + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  __shared__ Work jobs[MAX_JOBS];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)ptx::cluster_ctarank();
  const bool even = rank == 0;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      ptx::mbar_init(&full[s], 2);         // the even CTA's producers of A and B
      ptx::mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      ptx::mbar_init(&tfull[a], 1);
      ptx::mbar_init(&tempty[a], 2 * EPI_WARPS);
    }
    ptx::mbar_init(mdone, 1);
    *abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 2 && lane < p.njobs) {
    const Job& J = p.job[lane];
    jobs[lane] = Work{J.kind, J.a_mn, J.b_mn, J.m, J.n, J.b_n0, J.b_k0, J.mtiles, J.ntiles, J.group, J.begin, J.splits,
                      J.nkb, J.seg_kb, J.first, J.last, J.vec, J.out, J.acc, J.ldo, J.ldacc, J.part_stride};
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(tmem_slot, TMEM_COLS);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem_base = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  allow_next();
  await_previous();

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers (both CTAs)
    const bool is_b = warp == 2;
    if (lane == 0 && !(p.debug_flags & MUON_DEBUG_STALL_PRODUCER)) {
      for (int j = 0; j < p.njobs; ++j) ptx::prefetch_tmap(is_b ? &p.job[j].b : &p.job[j].a);
      int stage = 0;
      uint32_t phase = 0, pending = 0, pend_phase = 0;
      bool stop = false;
      for (int i = 0, t; !stop && (t = tile_at(p, pair, npairs, i)) >= 0; ++i) {
        const Tile ti = decode(jobs, p.njobs, t);
        const Work J = jobs[ti.job];
        const CUtensorMap* map = is_b ? &p.job[ti.job].b : &p.job[ti.job].a;
        const bool mn = is_b ? J.b_mn : J.a_mn;
        // A box that lies wholly past the output's rows or columns is not fetched (what the
        // MMAs make of stale data there is never read), but each CTA's first always is: a
        // producer that fetched nothing would not hold the MMAs back, and could lose count
        // of the phases of `empty`
        const int t0 = is_b ? ti.tn * TILE : ti.tm * TILE, left = (is_b ? J.n : J.m) - t0;
        const int boxes = left > rank * HALF + BOX ? 2 : 1;
        const uint32_t bytes = ((left > BOX ? 2 : 1) + (left > HALF + BOX ? 2 : 1)) * BOX_BYTES;   // of both CTAs
        const int r0 = t0 + rank * HALF + (is_b ? J.b_n0 : 0);
        const int k0 = ti.split * J.nkb * BK + (is_b ? J.b_k0 : 0);
        for (int term = 0; term < p.nterms && !stop; ++term) {
          const int z = is_b ? p.tb[term] : p.ta[term];
          for (int kb = 0; kb < J.nkb; ++kb) {
            if (!wait_for(&empty[stage], phase ^ 1u, abort_flag, p, true)) { stop = true; break; }
            const uint32_t fb = ptx::mapa_shared(ptx::smem_addr(&full[stage]), 0);
            if (even) ptx::mbar_arrive_expect_tx(&full[stage], bytes);
            const uint32_t d = ptx::smem_addr(smem + stage * STAGE_BYTES) + (is_b ? OP_BYTES : 0);
            const int k = k0 + kb * BK;
#pragma unroll
            for (int q = 0; q < 2; ++q)
              if (q < boxes)
                ptx::tma_load_3d_pair(d + q * BOX_BYTES, map, fb, mn ? r0 + q * BOX : k, mn ? k : r0 + q * BOX, z);
            pending |= 1u << stage;
            pend_phase = (pend_phase & ~(1u << stage)) | (phase << stage);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
        }
      }
      // Every issued copy lands before a CTA leaves.  The even CTA's barriers count both
      // CTAs' copies; the odd CTA waits for it at the cluster barrier.
      if (even)
        for (int s = 0; s < STAGES; ++s)
          if (pending & (1u << s)) wait_for(&full[s], (pend_phase >> s) & 1u, abort_flag, p, false);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (even CTA)
    if (even && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      int it = 0;   // accumulator uses
      bool stop = false;
      for (int i = 0, t; !stop && (t = tile_at(p, pair, npairs, i)) >= 0; ++i) {
        const Tile ti = decode(jobs, p.njobs, t);
        const Work J = jobs[ti.job];
        const uint32_t idesc = ptx::idesc_bf16_f32(TILE, TILE, J.a_mn, J.b_mn);
        // K-major: 8-row groups 1024 B apart, a K step of 16 is 32 B.  MN-major: atoms of
        // 64 rows 8 KB apart, 8-K groups 1024 B apart, a K step of 16 is 2 KB.
        const uint32_t a_lbo = J.a_mn ? OP_BYTES / 2 : 16, a_step = J.a_mn ? 2048 : 32;
        const uint32_t b_lbo = J.b_mn ? OP_BYTES / 2 : 16, b_step = J.b_mn ? 2048 : 32;
        const int total = p.nterms * J.nkb;
        for (int kb = 0; kb < total && !stop;) {
          const int run = segment_at(J, p.nterms, kb);
          const int acc = it & 1;
          if (!wait_for(&tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1u, abort_flag, p, true)) { stop = true; break; }
          ptx::tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * TILE);
          for (int q = 0; q < run; ++q) {
            if (!wait_for(&full[stage], phase, abort_flag, p, true)) { stop = true; break; }
            ptx::tc_fence_after();
            const uint32_t sa = ptx::smem_addr(smem + stage * STAGE_BYTES);
            const uint32_t sb = sa + OP_BYTES;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k)
              ptx::mma_bf16_pair(d, ptx::smem_desc_sw128(sa + k * a_step, a_lbo, 1024),
                                 ptx::smem_desc_sw128(sb + k * b_step, b_lbo, 1024), idesc, (q > 0 || k > 0) ? 1u : 0u);
            ptx::mma_commit_pair_mc(&empty[stage], 3);
            if (++stage == STAGES) { stage = 0; phase ^= 1u; }
          }
          if (stop) break;
          ptx::mma_commit_pair_mc(&tfull[acc], 3);
          ++it;
          kb += run;
        }
      }
      // all issued MMAs complete before either CTA releases its tensor memory
      ptx::mma_commit_pair_mc(mdone, 1);
      wait_for(mdone, 0, abort_flag, p, false);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue (both CTAs)
    const int quarter = warp & 3, half = (warp - 4) >> 2;
    const float u = shared_factor(p.scale, p.upstream, p.stats);
    float* stage = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES + 256) + (warp - 4) * XPOSE;
    int it = 0;
    bool stop = false;
    for (int i = 0, t; !stop && (t = tile_at(p, pair, npairs, i)) >= 0; ++i) {
      const Tile ti = decode(jobs, p.njobs, t);
      const Work& J = jobs[ti.job];
      const int r = ti.tm * TILE + rank * HALF + quarter * 32 + lane;
      const int cbase = ti.tn * TILE + half * HALF;
      RowIn x = {};
      if (J.kind == GRAD && r < J.m) x = row_in(p, r);
      const int nseg = kPromote ? segments(J, p.nterms) : 1;
      float acc[kPromote ? CHUNKS : 1][32];
      for (int seg = 0; seg < nseg; ++seg, ++it) {
        const int a = it & 1;
        int ok = 1;
        if (lane == 0) ok = wait_for(&tfull[a], (uint32_t)(it >> 1) & 1u, abort_flag, p, true) ? 1 : 0;
        if (!__shfl_sync(0xffffffffu, ok, 0)) { stop = true; break; }
        ptx::tc_fence_after();
        const uint32_t tb = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(a * TILE + half * HALF);
#pragma unroll
        for (int k = 0; k < CHUNKS; ++k) {
          if constexpr (kPromote) {
            ptx::tmem_add_32x32b_x16(tb + k * 32, acc[k], seg == 0);
            ptx::tmem_add_32x32b_x16(tb + k * 32 + 16, acc[k] + 16, seg == 0);
          } else {
            float v[32];
            ptx::tmem_ld_32x32b_x32(tb + k * 32, v);
            if (J.kind == GRAD) finish_grad(p, J, r, cbase + k * 32, v, x);
            else finish_sum(p, J, ti.split, r, cbase + k * 32, u, stage, lane, v);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (even) ptx::mbar_arrive(&tempty[a]);
          else ptx::mbar_arrive_cluster(ptx::mapa_shared(ptx::smem_addr(&tempty[a]), 0));
        }
      }
      if constexpr (kPromote) {
        if (!stop && J.kind == LOGITS) {
          finish_logits(p, J, ti, half, r, cbase, acc);
        } else if (!stop) {
#pragma unroll
          for (int k = 0; k < CHUNKS; ++k) {
            if (J.kind == GRAD) finish_grad(p, J, r, cbase + k * 32, acc[k], x);
            else finish_sum(p, J, ti.split, r, cbase + k * 32, u, stage, lane, acc[k]);
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  ptx::cluster_sync();   // no CTA leaves while its pair may still read its shared memory
  ptx::tc_fence_after();
  if (warp == 1) ptx::tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

template <class K>
cudaError_t allow(K kern) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
}
std::mutex g_mu;
std::map<int, int> g_pairs;   // device -> CTA pairs that run at once

}  // namespace

cudaError_t prepare() {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_pairs.count(dev)) return cudaSuccess;
  if ((e = allow(ce_kernel<false, Params>)) != cudaSuccess || (e = allow(ce_kernel<true, Params>)) != cudaSuccess ||
      (e = allow(ce_kernel<false, OrderedParams>)) != cudaSuccess ||
      (e = allow(ce_kernel<true, OrderedParams>)) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  int n = 0;
  if ((e = cudaOccupancyMaxActiveClusters(&n, ce_kernel<true, Params>, &cfg)) != cudaSuccess) return e;
  g_pairs[dev] = n < MAX_PAIRS ? n : MAX_PAIRS;
  return cudaSuccess;
}

int pairs() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_pairs.find(dev);
  return it == g_pairs.end() ? 0 : it->second;
}

cudaError_t launch(const OrderedParams& p, bool ordered, bool promote, cudaStream_t s) {
  if (p.tiles <= 0) return cudaSuccess;
  const int n = pairs();
  if (n < 1) return cudaErrorInvalidConfiguration;
  const int grid = 2 * (p.tiles < n ? p.tiles : n);
  count_launch();
  if (promote && ordered) return launch_after(ce_kernel<true, OrderedParams>, grid, THREADS, SMEM, s, p);
  if (promote) return launch_after(ce_kernel<true, Params>, grid, THREADS, SMEM, s, p);
  if (ordered) return launch_after(ce_kernel<false, OrderedParams>, grid, THREADS, SMEM, s, p);
  return launch_after(ce_kernel<false, Params>, grid, THREADS, SMEM, s, p);
}

}  // namespace ce
}  // namespace muon
