// Cross entropy of the LM head without the logits, and its gradient.
//
//   z_rv = h_r . w_v          lse_r = log sum_v exp(z_rv)         nll_r = lse_r - z_r,t(r)
//   D_rv = g_r (exp(z_rv - lse_r) - [v = t(r)])     dH = D W      dW = D^T H
//
// The loss makes one product (2 R V d operations, R = rows that take part) and keeps one
// (maximum, sum of exponentials) pair per row and column group instead of the logits.  The
// gradient makes the product again, piece of the vocabulary by piece, writes D for the piece
// (bf16, at most kPieceBytes of it), and multiplies it from both sides: 6 R V d operations.
//
// Rows with a negative target are left out before the first product: `head_rows_kernel` lists the
// others and copies them together, so that they cost nothing and what they hold (NaN, garbage
// of a padded batch) reaches no sum.  When every row takes part the rows are read in place.
//
// What bounds it and what it reaches (B200, other inputs on every pass):
//   loss, 4096 rows, 4096 x 8192     187 us   1.47 PFLOP/s  (a plain bf16 product sustains 1.40,
//                                             in bursts 1.67: tensor pipe and power)
//   gradient, a quarter left out     468 us   1.32 PFLOP/s  likewise
//   loss, 8 rows, 1024 x 32000       18.6 us  3.5 TB/s      reading 65 MB (a bare read: 14), two tails
//   gradient, 128 rows, likewise     63 us    2.1 TB/s      see head_narrow_kernel
//   fp32 loss, 331 rows, 256 x 1001  12.3 us                latency of three kernels
//
// One kernel does all products (`head_gemm_kernel`): persistent CTAs (or pairs, cta_group::2),
// 128 x BN (256 x 256) tiles, TMA loads into an mbarrier ring, tcgen05.mma into one of two
// accumulators in tensor memory while eight warps drain the other one.  K-major and MN-major
// operands differ in their boxes and descriptors only, so D and W are multiplied as they lie.
//
// bf16 (the logits' operands may be fp16): products of the given values, fp32 sums.  D is rounded
// to bf16 (half a step, 2^-8 relative to each of its values); "What rounding D to bf16 costs"
// below says what becomes of the remainders.
// fp32: every operand is split into three bf16 parts (8 + 8 + 8 significant bits) and the six
// products that reach 2^-16 of the largest are summed, smallest first (2^-23 is left out).
#include "head.h"

#include <algorithm>
#include <type_traits>

#include "ends.h"
#include "tensormap.h"

namespace smdm {

namespace {

constexpr int kThreads = 320;        // producer warp, MMA warp, 8 epilogue warps
constexpr int kEpiWarps = 8;
constexpr int kABytes = 128 * 128;   // 128 rows x 64 bf16
constexpr int kStagingBytes = kEpiWarps * 4096;
constexpr int kMaxStages = 8;
constexpr int kSmemLimit = 227 * 1024;
// D (and split weights) held at once.  Pieces that stay in L2 were slower, their kernels' tails
// cost more than the traffic: 64 MB 437 us and 32 MB 487 us against 437 for 4096 rows of
// 4096 x 8192 with a quarter left out, 420 and 482 against 378 for 2400 rows of 1024 x 32000.
constexpr size_t kPieceBytes = size_t(256) << 20;
constexpr float kLog2e = 1.4426950408889634f;

enum Mode : int { kLoss = 0, kDlog = 1, kGrad = 2 };

// Device-side counts, written by head_rows_kernel.
struct HeadMeta {
  int n;       // rows that take part
  int dense;   // 1: all of them do, and the caller's hidden is read in place
};

struct HeadDev {
  const HeadMeta* meta;     // null: row i is the caller's row i
  const int* row_idx;       // row that takes part -> row of the caller's tensors
  const int* target;
  int rows;
  int d, v0, vc;            // width; first column and columns of this piece
  int w_row0;               // row of the weight map that holds column v0
  int terms;                // products of parts per chunk (the schedule's weight of a chunk)
  int d_parts;              // bf16 parts of D
  int h_plane, w_plane, d_plane;   // rows between the parts of H, W, D in their maps
  int a_box;                // rows of A that one box brings (K-major H)
  int nstages, staging_off, bar_off;
  // With one row of tiles every slot starts at another place of K where the weight rows lie a
  // multiple of 2 KB apart: all slots at the same place of such rows keep to few of HBM's channels.
  // Loss of 8 / 128 rows of 1024 x 32000 19.0 -> 18.3, 20.1 -> 18.8 us, 100 rows of 4096 x 8192
  // 23.2 -> 20.3; rows of 1 or 3 KB are no faster for it (13.4 -> 13.8, 19.4 -> 19.7).
  int spread;
  int half;                 // the logits' operands are fp16
  // loss
  float2* part;             // [column group][r_pad]
  int part0;                // first column group of this piece
  int r_pad;
  float* tlogit;            // [r_pad]
  // D
  const int* row_tgt;       // [r_pad] targets of the listed rows
  float* delta;             // [r_pad] remainder of D at the row's target; null: not kept
  const int* run;           // [r_pad] rows with its target if it is the first of them, else 0
  int2* ids;                // [vocab] first listed row with the id as its target, and their number
  const __nv_bfloat16* rest;   // [r_pad][d_pad] sums of the remainders' part of dW (see RestArgs)
  const void* hidden;       // the caller's rows
  long long ld_hidden;
  const __nv_bfloat16* hid; // the listed rows
  const void* head;         // the caller's weights
  long long ld_head;
  int head_vec;             // they start on 16-byte boundaries
  const float* lse;
  const float* grad_nll;
  __nv_bfloat16* dlog;      // [parts][r_pad][ld_dlog]
  int ld_dlog;
  int d_rows;               // rows of D that are read (one row tile: 16, 64 or 128)
  // gradients
  int do_h, do_w, splits;
  float* acc;               // [splits][r_pad][d_pad] or null: dH is written directly
  int acc_add;              // add to acc (a later piece)
  int d_pad;
  void* out_h;              // [rows][d]
  void* out_w;              // row v0 of [vocab][d]
  int vec_ok;               // output rows start on 16-byte boundaries
  uint32_t* status;
};

__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
  return idesc_f16(M, N, a_mn, b_mn) | (1u << 7) | (1u << 10);   // A and B formats: bf16
}

// One unit of work: a tile of a product and the K range of it.
struct Unit {
  int kind;      // 0: H x W^T (loss, D); 1: dH; 2: dW
  int m0, n0;    // first row / column
  int k0, nk;    // first 64-wide K chunk, chunks
  int split;
};

// Fixed cost of a tile in K chunks, for the balance of the two gradients' tiles.
constexpr int kTileCost = 6;

// Operands in parts.  P = 1: bf16 operands.  P = 3 (fp32): both operands in three.  A pipeline
// stage holds a 64-wide K chunk of all parts, and the products of parts that count are summed
// from it, smallest first.
template <int P> constexpr int kAParts = P;
template <int P> constexpr int kBParts = P;
template <int P> constexpr int kProducts = P == 3 ? 6 : 1;
// parts of A and B in product t (t = 0 the smallest)
template <int P> __host__ __device__ constexpr int part_a(int t) {
  return P == 3 ? (0x021010 >> (4 * (5 - t))) & 15 : 0;
}
template <int P> __host__ __device__ constexpr int part_b(int t) {
  return P == 3 ? (0x201100 >> (4 * (5 - t))) & 15 : 0;
}

// The tensor core cuts its fp32 sums instead of rounding them, always towards zero.  Measured on sums
// of one sign, every 16-term step takes 1e-8 (terms of like size) to 1e-7 of the final value off:
// 1.6e-3 over 2^18 rows, as much as bf16's rounding.  It therefore sums kSegment chunks at a
// time, and the epilogue threads add the segments in registers, rounded to nearest: 24 or 32 steps
// for logits (the loss's, and the gradient's: what is left of exp(z - lse) - 1 at a certain target
// is as exact as z and lse are to each other) and for everything of the fp32 path.  The bf16
// gradients are rounded to 8 bits next; their segments are kWholeK chunks (512 steps, 5e-5 of the
// value at most, 1/40 of that rounding), and K ranges up to that long are summed whole, by a
// kernel of its own: the registers for the sums cost up to 10 % (200 rows of 1024 x 32000:
// 92.7 -> 101 us).
constexpr int kWholeK = 128;
template <int kMode, int P> constexpr int kSegment = P == 3 ? 1 : kMode == kGrad ? kWholeK : 8;
template <int kMode, int P, bool kLong>
constexpr bool kPromote = P == 3 || kMode != kGrad || kLong;

// 64-wide K chunks per pipeline stage.  Waiting for a stage and releasing it takes the issuing
// warp about 300 clocks, as much as the MMAs of a narrow tile, so those take two at a time.
template <int kMode, int CG, int BN, int P>
constexpr int kChunks = kMode != kGrad && P == 1 && CG == 1 && BN <= 128 ? 2 : 1;

// What rounding D to bf16 costs, and what is done about it.  Alone it makes dW's error 1.4 times its
// own rounding's, and dH's up to 1.7 times where a few rows with large weights make up the norm.
// A row's largest entry is its target's (it is minus the sum of the others), so its remainder
// delta_r is kept in fp32, and added to
//   row r of dH     delta_r times the weights of r's target,
//   row v of dW     the sum of delta_r h_r over the rows r whose target is v (head_rest_kernel),
// by the epilogues before they round: both errors fall back to the output's own rounding, whatever
// the rows' weights.  (A row that is certain of another id has a second entry as large, which is
// rounded: up to 1.2 times in its row of dH, 1.4 times in that id's row of dW.)
// One row tile (head_narrow_kernel) keeps the remainders of all entries.

// The work of one slot (CTA or pair) p of P.  Loss and D: tiles round robin, in groups of 16 row
// tiles so that a group's rows stay in L2 while the weights pass once.  Gradients: the dH units
// round robin, then the dW tiles so that every slot ends at about the same number of K chunks
// (a tile's fixed cost counted as kTileCost chunks).
template <int kMode, int CG, int BN>
struct Schedule {
  int p, P, n, kc, mt, nt;
  int kw, nh, nw, mt_w, nt_d, my_h, qa, my_w, n_rem;
  int kch, kper;

  SMDM_DEV Schedule(const HeadDev& a, int n_, int p_, int P_) : p(p_), P(P_), n(n_) {
    constexpr int MT = 128 * CG;
    mt = (n + MT - 1) / MT;
    if constexpr (kMode != kGrad) {
      kc = (a.d + 63) >> 6;
      nt = (a.vc + BN - 1) / BN;
    } else {
      nt_d = (a.d + BN - 1) / BN;
      kch = (a.vc + 63) >> 6;
      kper = (kch + a.splits - 1) / a.splits;
      kw = (n + 63) >> 6;
      mt_w = (a.vc + MT - 1) / MT;
      nh = a.do_h ? mt * nt_d * a.splits : 0;
      nw = a.do_w ? mt_w * nt_d : 0;
      const int c = nh / P;
      n_rem = nh % P;                       // slots with c + 1 dH units
      my_h = c + (p < n_rem ? 1 : 0);
      // finishing time T of all slots, raised from the mean until every dW tile fits.  In fp32:
      // every thread of the grid computes the same values, and rounding only moves the balance.
      const float ch = (float)kper * a.terms + kTileCost, cw = (float)kw * a.terms + kTileCost;
      auto fit = [&](float T, float used) {
        return T > used ? (int)fminf(__fdividef(T - used, cw), (float)nw) : 0;
      };
      float T = ((float)nh * ch + (float)nw * cw) / (float)P;
      int qb;
      while (true) {
        qa = fit(T, (c + 1) * ch);          // dW tiles of the slots with c + 1 dH units
        qb = fit(T, c * ch);
        if ((long long)n_rem * qa + (long long)(P - n_rem) * qb >= nw) break;
        T += 0.25f * cw + T * 1e-6f;
      }
      // this slot's dW tiles below nw (see get(): its t-th tile's number grows with t)
      my_w = min(qa, p < nw ? (nw - 1 - p) / P + 1 : 0);
      if (p >= n_rem && my_w == qa) {
        const int rest = nw - qa * P - (p - n_rem);
        if (rest > 0) my_w += min(qb - qa, (rest - 1) / (P - n_rem) + 1);
      }
    }
  }

  SMDM_DEV bool get(const HeadDev& a, int i, Unit& u) const {
    constexpr int MT = 128 * CG;
    if constexpr (kMode != kGrad) {
      const long long t = (long long)p + (long long)i * P;
      if (t >= (long long)mt * nt) return false;
      constexpr int G = 16;
      const int per = G * nt;
      const int g = (int)(t / per), in = (int)(t % per);
      const int gm = min(G, mt - g * G);
      u.kind = 0;
      u.m0 = (g * G + in % gm) * MT;
      u.n0 = (in / gm) * BN;
      u.k0 = 0;
      u.nk = kc;
      u.split = 0;
      return true;
    } else {
      // odd slots take their dW tiles first: dH reads the weights, dW writes their gradient, and
      // the two halves of the traffic overlap
      if (i >= my_h + my_w) return false;
      if (p & 1) i = i < my_w ? i + my_h : i - my_w;
      if (i < my_h) {
        const int t = p + i * P;
        const int tile = t / a.splits;
        u.kind = 1;
        u.split = t % a.splits;
        u.m0 = (tile % mt) * MT;
        u.n0 = (tile / mt) * BN;
        u.k0 = u.split * kper;
        u.nk = max(0, min(kper, kch - u.k0));
        return true;
      }
      const int t = i - my_h;
      // rounds in which every slot has a tile, then those of the slots with fewer dH units
      const int q = t < qa ? t * P + p : qa * P + (t - qa) * (P - n_rem) + (p - n_rem);
      u.kind = 2;
      u.split = 0;
      u.m0 = (q / nt_d) * MT;
      u.n0 = (q % nt_d) * BN;
      u.k0 = 0;
      u.nk = kw;
      return true;
    }
  }
};

// x = p0 + p1 + p2 with bf16 parts; an infinity or NaN stays in the first part alone.
SMDM_DEV void split3(float x, __nv_bfloat16& p0, __nv_bfloat16& p1, __nv_bfloat16& p2) {
  p0 = __float2bfloat16_rn(x);
  float r = x - __bfloat162float(p0);
  if (!(fabsf(x) <= 3.3895314e38f)) r = 0.f;
  p1 = __float2bfloat16_rn(r);
  p2 = __float2bfloat16_rn(r - __bfloat162float(p1));
}

SMDM_DEV float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// One lane of a converged warp.  The producer and MMA warps run their loops as whole warps, so
// that loop counters, addresses and descriptors are warp-uniform, and only the instructions
// that one thread must issue are under this predicate.  With the loops inside `if (lane == 0)`
// instead an MMA took 65 clocks to issue whatever its size, and a 64-wide chunk about 500.
SMDM_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
// mbar_wait by a whole warp.
SMDM_DEV bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}

SMDM_DEV uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A warp's 32 rows x 128 (or 64) bytes, swizzled by row so that neither the writes (a lane per
// row) nor the reads (lanes along a row) collide on banks.
template <int RB>
SMDM_DEV uint8_t* stage_at(uint8_t* st, int row, int chunk) {
  constexpr int C = RB / 16;
  return st + row * RB + ((chunk ^ ((RB == 128 ? row : row >> 1) & (C - 1))) << 4);
}

// Write the staged rows to global memory: RB bytes of every row, at column `col` (elements) of
// the row that `row_ptr(row)` gives (null: skip), of which `cols` columns exist.
// kLast: nothing reads the data again soon (a gradient), so it need not stay in L2.
template <typename T, int RB, bool kLast, typename RowPtr>
SMDM_DEV void flush_rows(uint8_t* st, int lane, int col, int cols, bool vec, RowPtr row_ptr) {
  constexpr int C = RB / 16, E = 16 / (int)sizeof(T), RPI = 32 / C;
  __syncwarp();
  // (All reads first, then the stores.  What bounds a flush is that an SM takes 32 bytes of stores
  // per clock, measured: 1024 clocks for eight warps' 32 KB at least, 1450 seen.)
  uint4 v[C];
#pragma unroll
  for (int it = 0; it < C; ++it)
    v[it] = *reinterpret_cast<const uint4*>(stage_at<RB>(st, it * RPI + lane / C, lane % C));
  const int c0 = col + lane % C * E;
#pragma unroll
  for (int it = 0; it < C; ++it) {
    T* dst = row_ptr(it * RPI + lane / C);
    if (dst && c0 < cols) {
      if (vec && c0 + E <= cols) {
        if constexpr (kLast) __stcs(reinterpret_cast<uint4*>(dst + c0), v[it]);
        else *reinterpret_cast<uint4*>(dst + c0) = v[it];
      } else {
        const T* e = reinterpret_cast<const T*>(&v[it]);
#pragma unroll
        for (int k = 0; k < E; ++k)
          if (c0 + k < cols) dst[c0 + k] = e[k];
      }
    }
  }
  __syncwarp();
}

// 32 values of this lane's row -> staging chunks starting at chunk c0.
template <int RB>
SMDM_DEV void stage_bf16(uint8_t* st, int lane, int c0, const float* v) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint4 w;
    w.x = pack_bf16(v[8 * k + 0], v[8 * k + 1]);
    w.y = pack_bf16(v[8 * k + 2], v[8 * k + 3]);
    w.z = pack_bf16(v[8 * k + 4], v[8 * k + 5]);
    w.w = pack_bf16(v[8 * k + 6], v[8 * k + 7]);
    *reinterpret_cast<uint4*>(stage_at<RB>(st, lane, c0 + k)) = w;
  }
}
SMDM_DEV void stage_f32(uint8_t* st, int lane, const float* v) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    *reinterpret_cast<float4*>(stage_at<128>(st, lane, k)) =
        make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
}

// 32 columns of a row of a gradient: plus f times the row w of the other operand.
SMDM_DEV void add_row(const __nv_bfloat16* w, bool vec, float f, int col, int d, float* v) {
  w += col;
  if (vec && col + 32 <= d) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 u = *reinterpret_cast<const uint4*>(w + 8 * k);
      const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[8 * k + 2 * j] = fmaf(f, __uint_as_float(x[j] << 16), v[8 * k + 2 * j]);
        v[8 * k + 2 * j + 1] = fmaf(f, __uint_as_float(x[j] & 0xffff0000u), v[8 * k + 2 * j + 1]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (col + j < d) v[j] = fmaf(f, __bfloat162float(w[j]), v[j]);
  }
}

// kMode: what is computed.  CG: CTAs per tile (2: a pair on two SMs, M = 256).  BN: tile
// columns.  P: operand parts; 3 is the fp32 path.  kLong: K in segments (kWholeK).
template <int kMode, int CG, int BN, int P, bool kLong>
__global__ void __launch_bounds__(kThreads, 1)
    head_gemm_kernel(const __grid_constant__ CUtensorMap tm_h,    // caller's hidden (K-major box)
                     const __grid_constant__ CUtensorMap tm_hc,   // listed rows, or same box
                     const __grid_constant__ CUtensorMap tm_w,    // weights
                     const __grid_constant__ CUtensorMap tm_dk,   // D, K-major box
                     const __grid_constant__ CUtensorMap tm_dm,   // D, MN-major box
                     const HeadDev a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  constexpr int kBRows = BN / CG;                    // rows (columns of the product) of B here
  constexpr bool F32 = P == 3;
  constexpr int kBPart = kBRows * 128;
  constexpr int KS = kChunks<kMode, CG, BN, P>;
  constexpr int kStage = KS * (kAParts<P> * kABytes + kBParts<P> * kBPart);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + a.bar_off);
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* acc_full = bars + 2 * kMaxStages;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(acc_empty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.nstages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps * CG);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_hc);
    tma_prefetch_desc(&tm_w);
  }
  if constexpr (CG == 2) cluster_sync_all();
  if (warp == 1) {
    if constexpr (CG == 2) {
      tmem_alloc_pair(tmem_holder, 2 * BN);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, 2 * BN);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  griddep_launch();
  griddep_wait();

  // (no meta: every row of the caller's hidden, listed or not)
  const int n = a.meta ? a.meta->n : a.rows;
  const bool dense = a.meta ? a.meta->dense != 0 : true;
  const Schedule<kMode, CG, BN> sch(a, n, blockIdx.x / CG, gridDim.x / CG);
  auto lead_addr = [&](uint64_t* bar) -> uint32_t {
    return CG == 2 ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar);
  };

  if (warp == 0) {
    {
      const uint64_t pol = policy_evict_normal();
      int stage = 0;
      uint32_t phase = 0;
      Unit u;
      bool ok = true;
      const CUtensorMap* th = dense ? &tm_h : &tm_hc;
      const int h_plane = dense ? 0 : a.h_plane;
      for (int i = 0; ok && sch.get(a, i, u); ++i) {
        const int m0 = u.m0 + (int)rank * 128;
        const int n0 = u.n0 + (int)rank * kBRows;
        int kx = 0, span = 0;              // loss and D: where this slot is in K, and K's end
        if constexpr (kMode != kGrad) {
          span = (u.nk + KS - 1) / KS * KS;
          if (a.spread && sch.mt == 1) kx = (int)(blockIdx.x / CG) * KS % span;
        }
        for (int k = u.k0; k < u.k0 + u.nk; k += KS) {
          if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, a.status)) { ok = false; break; }
          uint8_t* A = smem + stage * kStage;
          uint8_t* B = A + KS * kAParts<P> * kABytes;
          if (elect_one()) {
            const int ab = u.kind == 0 ? a.a_box * 128 : kABytes;
            if (leader)
              mbar_arrive_expect_tx(&full[stage],
                                    CG * KS * (kAParts<P> * ab + kBParts<P> * kBPart));
            const uint32_t fb = lead_addr(&full[stage]);
            auto load = [&](uint8_t* dst, const CUtensorMap* m, int x, int y) {
              if constexpr (CG == 2) tma_load_2d_pair(dst, m, fb, x, y, pol);
              else tma_load_2d(dst, m, &full[stage], x, y, pol);
            };
#pragma unroll
            for (int p = 0; p < kAParts<P>; ++p) {
              if constexpr (kMode != kGrad) {
                // (a chunk past the row's end arrives as zeros)
#pragma unroll
                for (int s = 0; s < KS; ++s)
                  load(A + (s * kAParts<P> + p) * kABytes, th, (kx + s) * 64, p * h_plane + m0);
              } else if (u.kind == 1) {   // dH: D (K = columns, contiguous)
                load(A + p * kABytes, &tm_dk, k * 64, p * a.d_plane + m0);
              } else {                    // dW: D (M contiguous)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  load(A + p * kABytes + j * 8192, &tm_dm, m0 + j * 64, p * a.d_plane + k * 64);
              }
            }
#pragma unroll
            for (int p = 0; p < kBParts<P>; ++p) {
              if constexpr (kMode != kGrad) {
#pragma unroll
                for (int s = 0; s < KS; ++s)
                  load(B + (s * kBParts<P> + p) * kBPart, &tm_w, (kx + s) * 64,
                       a.w_row0 + p * a.w_plane + n0);
              } else {                    // dH: W, dW: H (N contiguous)
                const CUtensorMap* tb = u.kind == 1 ? &tm_w : th;
                const int y = (u.kind == 1 ? a.w_row0 + p * a.w_plane : p * h_plane) + k * 64;
#pragma unroll
                for (int j = 0; j < kBRows / 64; ++j)
                  load(B + p * kBPart + j * 8192, tb, n0 + j * 64, y);
              }
            }
          }
          __syncwarp();
          if constexpr (kMode != kGrad) kx = kx + KS == span ? 0 : kx + KS;
          if (++stage == a.nstages) { stage = 0; phase ^= 1; }
        }
      }
      // The MMAs' completions arrive on these barriers, a pair's from the first CTA: wait until
      // every stage is released so that no arrival lands after this CTA has exited.
      for (int s = 0; ok && s < a.nstages; ++s) {
        if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, a.status)) break;
        if (++stage == a.nstages) { stage = 0; phase ^= 1; }
      }
    }
  } else if (warp == 1) {
    if (leader) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      Unit u;
      bool ok = true;
      for (int i = 0; ok && sch.get(a, i, u); ++i) {
        const int total = (u.nk + KS - 1) / KS;      // stages
        // K-major: the next 16 K values lie 32 bytes on; MN-major: 16 rows of 128 bytes on,
        // with 8192 bytes between 64-element runs along M or N
        const int a_mn = u.kind == 2, b_mn = u.kind != 0;
        const uint32_t idesc = kMode != kGrad && P == 1 && a.half
                                   ? idesc_f16(128 * CG, BN, a_mn, b_mn)
                                   : idesc_bf16(128 * CG, BN, a_mn, b_mn);
        const uint32_t a_lbo = a_mn ? 8192 : 16, b_lbo = b_mn ? 8192 : 16;
        const uint32_t a_step = a_mn ? 2048 >> 4 : 32 >> 4, b_step = b_mn ? 2048 >> 4 : 32 >> 4;
        // (no chunks at all: nothing to sum, the epilogue writes zeros)
        for (int c0 = 0; ok && c0 < total;) {
          const int c1 = kPromote<kMode, P, kLong> ? min(total, c0 + kSegment<kMode, P> / KS) : total;
          if (!warp_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, a.status)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tbase + acc * BN;
          for (int c = c0; c < c1; ++c) {
            if (!warp_wait(&full[stage], phase, abort_flag, a.status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t a_addr = smem_u32(smem + stage * kStage);
            const uint64_t ad = sdesc_sw128(a_addr, a_lbo, 1024);
            const uint64_t bd = sdesc_sw128(a_addr + KS * kAParts<P> * kABytes, b_lbo, 1024);
            if (elect_one()) {
#pragma unroll
              for (int t = 0; t < kProducts<P> * KS; ++t) {
                constexpr int NP = kProducts<P>;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                  const uint32_t accum = (c > c0 || t > 0 || kk > 0) ? 1u : 0u;
                  const int pa = t / NP * kAParts<P> + part_a<P>(t % NP);
                  const int pb = t / NP * kBParts<P> + part_b<P>(t % NP);
                  const uint64_t da = ad + (pa * kABytes >> 4) + kk * a_step;
                  const uint64_t db = bd + (pb * kBPart >> 4) + kk * b_step;
                  if constexpr (CG == 2) umma_f16_pair(d, da, db, idesc, accum);
                  else umma_f16(d, da, db, idesc, accum);
                }
              }
              if constexpr (CG == 2) umma_commit_pair(&empty[stage]);
              else umma_commit(&empty[stage]);
            }
            __syncwarp();
            if (++stage == a.nstages) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          if (elect_one()) {
            if constexpr (CG == 2) umma_commit_pair(&acc_full[acc]);
            else umma_commit(&acc_full[acc]);
          }
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
          c0 = c1;
        }
      }
    }
  } else {
    // Epilogue: a warp reads the 32 accumulator rows of its lane quarter (warp % 4), one row per
    // lane; warps 2-5 take the tile's first half of the columns, warps 6-9 the second.
    const int q = warp & 3, half = (warp - 2) >> 2;
    constexpr int HC = BN / 2;             // columns of a half
    uint8_t* st = smem + a.staging_off + (warp - 2) * 4096;
    int acc = 0;
    uint32_t acc_phase = 0;
    Unit u;
    for (int i = 0; sch.get(a, i, u); ++i) {
      const int row = u.m0 + (int)rank * 128 + q * 32 + lane;   // row of the product
      const bool empty_sum = u.nk == 0;
      int my_row = 0, tgt = -1;
      float lse = 0.f, g = 0.f;
      if (kMode != kGrad || u.kind == 1) {
        if (row < n) {
          my_row = a.meta ? a.row_idx[row] : row;
          if constexpr (kMode != kGrad) tgt = a.target[my_row] - a.v0 - u.n0 - half * HC;
          if constexpr (kMode == kDlog) {
            lse = a.lse[my_row];
            g = a.grad_nll[my_row];
          }
          if constexpr (kMode == kGrad && !F32) {
            // (kind 1) the row's target, where this unit's columns hold it
            if (a.delta) {
              const int t = a.row_tgt[row] - a.v0;
              if (t >= u.k0 * 64 && t < min(a.vc, (u.k0 + u.nk) * 64)) {
                tgt = t + a.v0;
                g = a.delta[row];
              }
            }
          }
        }
      }
      // the remainder of D at this row's target, or the remainders whose target is this row's id
      const __nv_bfloat16* with = nullptr;
      if constexpr (kMode == kGrad && !F32) {
        if (u.kind == 1) {
          if (tgt >= 0) with = static_cast<const __nv_bfloat16*>(a.head) + (size_t)tgt * a.ld_head;
        } else if (a.rest && row < a.vc) {
          const int2 id = a.ids[a.v0 + row];
          if (id.y == 1) {
            with = dense ? static_cast<const __nv_bfloat16*>(a.hidden) + (size_t)id.x * a.ld_hidden
                         : a.hid + (size_t)id.x * a.d_pad;
            g = a.delta[id.x];
          } else if (id.y > 1) {
            with = a.rest + (size_t)id.x * a.d_pad;
            g = 1.f;
          }
        }
      }
      const bool with_vec = u.kind == 2 || a.head_vec;
      const uint32_t lanes = uint32_t(q * 32) << 16;
      // a wait that gave up only flags the status word; the results are then garbage but the
      // kernel ends
      auto acquire = [&]() {
        mbar_wait(&acc_full[acc], acc_phase, abort_flag, a.status);
        tc_fence_after();
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (CG == 2) mbar_arrive_cluster(lead_addr(&acc_empty[acc]));
          else mbar_arrive(&acc_empty[acc]);
        }
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      };
      // Promoted sums: this thread's HC columns live in registers once the last segment is in.
      constexpr bool kRegs = kPromote<kMode, P, kLong>;
      constexpr int NB = HC / 32;
      float sum[kRegs ? HC : 1];
      if constexpr (kRegs) {
#pragma unroll
        for (int j = 0; j < HC; ++j) sum[j] = 0.f;
        for (int c0 = 0; c0 < u.nk; c0 += kSegment<kMode, P>) {   // (chunks; a stage never splits)
          acquire();
#pragma unroll
          for (int c = 0; c < NB; ++c) {
            float v[32];
            tmem_ld32(tbase + lanes + acc * BN + half * HC + c * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) sum[c * 32 + j] += v[j];
          }
          release();
        }
      } else if (!empty_sum) {
        acquire();
      }
      const uint32_t tacc = tbase + lanes + acc * BN + half * HC;
      auto load = [&](int c, float* v) {
        if constexpr (kRegs) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = sum[c * 32 + j];
        } else if (!empty_sum) {
          tmem_ld32(tacc + c * 32, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
      };
      const int ccol = u.n0 + half * HC;   // first column of this half
      if constexpr (kMode == kLoss) {
        // running maximum and sum of this row over the half's columns
        const int ncol = min(HC, a.vc - ccol);
        float m = -INFINITY, s = 0.f;
#pragma unroll
        for (int c = 0; c < NB; ++c) {
          if (c * 32 >= ncol) break;
          float v[32];
          load(c, v);
          if (c * 32 + 32 > ncol) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j >= ncol) v[j] = -INFINITY;
          }
          float x[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) x[j & 3] = fmaxf(x[j & 3], v[j]);
          const float mn = fmaxf(m, fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
          // the target's logit, in the few chunks that hold one
          const int rel = tgt - c * 32;
          const bool mine = row < n && rel >= 0 && rel < 32;
          if (__any_sync(0xffffffffu, mine)) {
            float tv = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (j == rel) tv = v[j];
            if (mine) a.tlogit[row] = tv;
          }
          float y[4] = {0.f, 0.f, 0.f, 0.f};
          const float ref = mn == -INFINITY ? 0.f : mn;   // (no column above -inf so far)
#pragma unroll
          for (int j = 0; j < 32; ++j) y[j & 3] += ex2((v[j] - ref) * kLog2e);
          s = s * ex2((m - ref) * kLog2e) + ((y[0] + y[1]) + (y[2] + y[3]));
          m = mn;
        }
        if (row < n)
          a.part[(size_t)(a.part0 + 2 * (u.n0 / BN) + half) * a.r_pad + row] = make_float2(m, s);
      } else if constexpr (kMode == kDlog) {
        // 32-column blocks per staged pass (two of 128 columns' sums would spill: 190 -> 195 us for
        // 4096 rows of 4096 x 8192)
        constexpr int PC = !F32 && HC == 64 ? 2 : 1;
        constexpr int RB = 64 * PC;
        auto rp = [&](int plane) {
          return [&, plane](int r) -> __nv_bfloat16* {
            const int rr = row - lane + r;
            return rr < a.d_rows ? a.dlog + ((size_t)plane * a.d_plane + rr) * a.ld_dlog : nullptr;
          };
        };
#pragma unroll(kRegs ? NB : 1)
        for (int c = 0; c < NB; c += PC) {
          const int col = ccol + c * 32;
          // rows past the last one and columns past the vocabulary become zeros: the products
          // that follow read them
          const int lim = row < n ? a.vc - col : 0;
          const int rel = tgt - c * 32;
          float v[32 * PC];
#pragma unroll
          for (int s2 = 0; s2 < PC; ++s2) load(c + s2, v + 32 * s2);
          // (most blocks hold no target, no row past the last and no column past the vocabulary)
          const bool plain = __all_sync(0xffffffffu, lim >= 32 * PC && (rel < 0 || rel >= 32 * PC));
          if (plain && !F32) {
            const float off = -lse * kLog2e;
#pragma unroll
            for (int j = 0; j < 32 * PC; ++j) v[j] = ex2(fmaf(v[j], kLog2e, off)) * g;
          } else {
            float tv = 0.f;
#pragma unroll
            for (int j = 0; j < 32 * PC; ++j) {
              float p = ex2((v[j] - lse) * kLog2e);
              if (j == rel) p -= 1.f;
              v[j] = j < lim ? p * g : 0.f;
              if (j == rel) tv = v[j];
            }
            if (!F32 && a.delta && row < n && rel >= 0 && rel < 32 * PC) {
              a.delta[row] = tv - __bfloat162float(__float2bfloat16_rn(tv));
              const int k = a.ids ? a.run[row] : 0;
              if (k > 0) a.ids[a.v0 + col + rel] = make_int2(row, k);
            }
          }
          // the parts one after the other, each the rounding of what the ones before leave (more
          // than one of bf16 only in tiles of 64 columns)
          const int parts = F32 || BN == 64 ? a.d_parts : 1;
          for (int pl = 0; pl < parts; ++pl) {
#pragma unroll
            for (int s2 = 0; s2 < PC; ++s2) stage_bf16<RB>(st, lane, s2 * 4, v + 32 * s2);
            flush_rows<__nv_bfloat16, RB, false>(st, lane, col, a.ld_dlog, true, rp(pl));
            if (pl + 1 < parts) {
#pragma unroll
              for (int j = 0; j < 32 * PC; j += 2) {
                const uint32_t hi = pack_bf16(v[j], v[j + 1]);
                v[j] -= __uint_as_float(hi << 16);
                v[j + 1] -= __uint_as_float(hi & 0xffff0000u);
              }
            }
          }
        }
      } else if (u.kind == 1 && a.acc) {
        // fp32 sums of this piece and K range
        float* base = a.acc + (size_t)u.split * a.r_pad * a.d_pad;
#pragma unroll(kRegs ? NB : 1)
        for (int c = 0; c < NB; ++c) {
          const int col = ccol + c * 32;
          float v[32];
          load(c, v);
          if (!F32 && with) add_row(with, with_vec, g, col, a.d, v);
          stage_f32(st, lane, v);
          if (a.acc_add) {
            __syncwarp();
#pragma unroll
            for (int it = 0; it < 8; ++it) {
              const int r = it * 4 + (lane >> 3), ch = lane & 7;
              if (row - lane + r < n && col + ch * 4 < a.d_pad) {
                float4* s4 = reinterpret_cast<float4*>(stage_at<128>(st, r, ch));
                const float4 o = *reinterpret_cast<const float4*>(
                    base + (size_t)(row - lane + r) * a.d_pad + col + ch * 4);
                float4 w = *s4;
                w.x += o.x; w.y += o.y; w.z += o.z; w.w += o.w;
                *s4 = w;
              }
            }
          }
          flush_rows<float, 128, false>(st, lane, col, a.d_pad, true, [&](int r) -> float* {
            return row - lane + r < n ? base + (size_t)(row - lane + r) * a.d_pad : nullptr;
          });
        }
      } else {
        // a gradient in its own type: dH rows at the caller's rows, dW rows in order
        using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
        const int lim = u.kind == 1 ? n : a.vc;
        T* base = static_cast<T*>(u.kind == 1 ? a.out_h : a.out_w);
        auto rp = [&](int r) -> T* {
          const int rr = row - lane + r;
          const int at = u.kind == 1 ? __shfl_sync(0xffffffffu, my_row, r) : rr;
          return rr < lim ? base + (size_t)at * a.d : nullptr;
        };
        constexpr int PC = (!F32 && HC >= 64) ? 2 : 1;
        constexpr int RB = F32 ? 128 : 64 * PC;
#pragma unroll(kRegs ? NB : 1)
        for (int c = 0; c < NB; c += PC) {
#pragma unroll
          for (int s2 = 0; s2 < PC; ++s2) {
            float v[32];
            load(c + s2, v);
            if (!F32 && with) add_row(with, with_vec, g, ccol + (c + s2) * 32, a.d, v);
            if constexpr (F32) stage_f32(st, lane, v);
            else stage_bf16<RB>(st, lane, s2 * 4, v);
          }
          flush_rows<T, RB, true>(st, lane, ccol + c * 32, a.d, a.vec_ok != 0, rp);
        }
      }
      if (!kRegs && !empty_sum) release();
    }
  }
  if (*abort_flag) let_land();
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync_all();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 2) tmem_dealloc_pair(tbase, 2 * BN);
    else tmem_dealloc(tbase, 2 * BN);
  }
}

// ------------------------------------------------------------------------------------------
// Gradients of one row tile (at most 128 rows that take part, bf16)
// ------------------------------------------------------------------------------------------
// With so few rows both products of D are bound by bytes: dH reads the weights, dW writes their
// gradient.  A CTA keeps 128 columns of everything: its columns of the hidden rows stay in shared
// memory, its columns of dH stay in tensor memory, and for 64 vocabulary rows at a time it loads
// D once for both products and its columns of the weights, adds to dH, and drains dW.  That
// moves half of the bytes of separate tiles from L2 to the SMs, and the reads of one vocabulary
// block overlap the writes of the last.
//
//   dH [128 r][128 c]  += D [128 r][64 v] W [64 v][128 c]        (both parts of D)
//   dW^T [128 c][64 v]  = H^T [128 c][r] D [r][64 v]
//
// dW comes out transposed (a lane per column), so that 64 vocabulary rows are enough for an
// M = 128 product; the epilogue turns it around by an exchange between neighbouring lanes and
// through shared memory (without the exchange, two bytes of a lane at a time, 5 us more).  What
// bounds the loop: loads alone take 20 us, the writes of dW 7, the products 5 that do not
// overlap.  An MMA of N columns reads 4 KB of A and 32 N bytes of B from shared memory, 128 bytes
// per clock; H^T therefore goes to tensor memory once and is dW's A operand from there.
//
// With 1024 x 32000 weights, other weights on every pass: 128 rows 62 us, 8 rows 56 us for the whole
// gradient, 34 and 32 of them here; 79 and 84 us with head_gemm_kernel's tiles.  With H^T in shared
// memory 9 us more; a deeper ring of stages changed nothing.
constexpr int kNarrowD = 2 * 128 * 128;         // a stage: D, two parts of [128 r][64 v]
constexpr int kNarrowW = 2 * 64 * 128;          // and W, two runs of 64 columns [64 v][64 c]
constexpr int kNarrowStage = kNarrowD + kNarrowW;
constexpr int kNarrowStages = 3;
constexpr int kNarrowBlocks = 256;              // of 8 steps each: 2e-4 at most (see kWholeK)
constexpr int kNarrowH = 2 * 128 * 128;         // H: two runs of 64 columns [128 r][64 c]

// Lane l holds 32 values of column l; afterwards, rounded to bf16, columns l & ~1 and l | 1 of the
// values 2 k + l % 2 in a[k].
SMDM_DEV void pair_columns(const float* v, int lane, uint32_t* a) {
  const bool odd = lane & 1;
  const uint32_t lo = odd ? 0x1054 : 0x5410, hi = odd ? 0x3276 : 0x7632;
#pragma unroll
  for (int k = 0; k < 8; ++k) {              // values 4 k and 4 k + 2, or 4 k + 1 and 4 k + 3
    const uint32_t e = pack_bf16(v[4 * k], v[4 * k + 2]), o = pack_bf16(v[4 * k + 1], v[4 * k + 3]);
    const uint32_t mine = odd ? o : e;
    const uint32_t other = __shfl_xor_sync(0xffffffffu, odd ? e : o, 1);
    a[2 * k] = __byte_perm(mine, other, lo);
    a[2 * k + 1] = __byte_perm(mine, other, hi);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    head_narrow_kernel(const __grid_constant__ CUtensorMap tm_h,    // box {64, 64}
                       const __grid_constant__ CUtensorMap tm_hc,
                       const __grid_constant__ CUtensorMap tm_w,    // box {64, 64}
                       const __grid_constant__ CUtensorMap tm_dk,   // box {64, 128}
                       const HeadDev a, int slots) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sh_h = smem + kNarrowStages * kNarrowStage;
  uint8_t* sh_st = sh_h + kNarrowH;
  uint64_t* full = reinterpret_cast<uint64_t*>(sh_st + kStagingBytes);
  uint64_t* empty = full + kNarrowStages;
  uint64_t* acc_full = empty + kNarrowStages;    // [2] dW
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* h_full = acc_empty + 2;
  uint64_t* dh_full = h_full + 1;
  uint64_t* ht_full = dh_full + 1;               // H^T is in tensor memory
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(ht_full + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kNarrowStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps);
    }
    mbar_init(h_full, 1);
    mbar_init(dh_full, 1);
    mbar_init(ht_full, kEpiWarps);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_w);
    tma_prefetch_desc(&tm_dk);
  }
  if (warp == 1) {
    tmem_alloc(tmem_holder, 512);                // dH: 128 columns; dW: 2 x 64; H^T: 64
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_holder;
  griddep_launch();
  griddep_wait();

  const int n = a.meta->n;
  const bool dense = a.meta->dense != 0;
  const int c0 = blockIdx.x * 128, slot = blockIdx.y;
  const int blocks = n > 0 ? (a.vc + 63) >> 6 : 0;   // 64-row blocks of the vocabulary
  const int mine = slot < blocks ? (blocks - 1 - slot) / slots + 1 : 0;

  if (warp == 0) {
    const uint64_t pol = policy_evict_normal();
    if (mine > 0 && elect_one()) {
      const CUtensorMap* th = dense ? &tm_h : &tm_hc;
      mbar_arrive_expect_tx(h_full, kNarrowH);
      for (int j = 0; j < 2; ++j)
        for (int k = 0; k < 2; ++k)
          tma_load_2d(sh_h + j * 16384 + k * 8192, th, h_full, c0 + j * 64, k * 64, pol);
    }
    __syncwarp();
    int stage = 0;
    uint32_t phase = 0;
    for (int i = 0; i < mine; ++i) {
      if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, a.status)) break;
      if (elect_one()) {
        uint8_t* D = smem + stage * kNarrowStage;
        uint8_t* W = D + kNarrowD;
        const int v = (slot + i * slots) * 64;
        mbar_arrive_expect_tx(&full[stage], 2 * a.d_rows * 128 + kNarrowW);
        for (int p = 0; p < 2; ++p)
          tma_load_2d(D + p * 16384, &tm_dk, &full[stage], v, p * a.d_plane, pol);
        for (int j = 0; j < 2; ++j)
          tma_load_2d(W + j * 8192, &tm_w, &full[stage], c0 + j * 64, a.w_row0 + v, pol);
      }
      __syncwarp();
      if (++stage == kNarrowStages) { stage = 0; phase ^= 1; }
    }
    // every stage released: the last products are done (also those of a dH that is not wanted)
    for (int s = 0; s < kNarrowStages; ++s) {
      if (!warp_wait(&empty[stage], phase ^ 1, abort_flag, a.status)) break;
      if (++stage == kNarrowStages) { stage = 0; phase ^= 1; }
    }
  } else if (warp == 1) {
    bool ok = mine > 0 && warp_wait(ht_full, 0, abort_flag, a.status);
    const uint32_t id_w = idesc_bf16(128, 64, 0, 1), id_h = idesc_bf16(128, 128, 0, 1);
    int stage = 0, acc = 0;
    uint32_t phase = 0, acc_phase = 0;
    for (int i = 0; ok && i < mine; ++i) {
      if (!warp_wait(&full[stage], phase, abort_flag, a.status)) { ok = false; break; }
      if (!warp_wait(&acc_empty[acc], acc_phase ^ 1, abort_flag, a.status)) { ok = false; break; }
      tc_fence_after();
      const uint32_t d_addr = smem_u32(smem + stage * kNarrowStage);
      const uint64_t db = sdesc_sw128(d_addr, 16, 1024);     // D, both ways it is read
      const uint64_t wd = sdesc_sw128(d_addr + kNarrowD, 8192, 1024);
      if (elect_one()) {
        // dW first: its epilogue can start while dH is added to
        // (straight-line code: a runtime loop around each MMA costs its issue half again)
        auto dw = [&](auto steps) {
#pragma unroll
          for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int kk = 0; kk < decltype(steps)::value; ++kk)
              umma_f16_ts(tbase + 128 + acc * 64, tbase + 256 + kk * 8,
                          db + p * (16384 >> 4) + kk * (2048 >> 4), id_w,
                          (p == 0 || kk > 0) ? 1u : 0u);
        };
        if (n > 64) dw(std::integral_constant<int, 8>());
        else if (n > 16) dw(std::integral_constant<int, 4>());
        else dw(std::integral_constant<int, 1>());
        umma_commit(&acc_full[acc]);
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_f16(tbase, db + p * (16384 >> 4) + kk * (32 >> 4), wd + kk * (2048 >> 4), id_h,
                     (i > 0 || p == 0 || kk > 0) ? 1u : 0u);
        umma_commit(&empty[stage]);
        if (i == mine - 1) umma_commit(dh_full);
      }
      __syncwarp();
      if (++stage == kNarrowStages) { stage = 0; phase ^= 1; }
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
  } else {
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t lanes = uint32_t(q * 32) << 16;
    uint8_t* st = sh_st + (warp - 2) * 4096;
    __nv_bfloat16* out_w = static_cast<__nv_bfloat16*>(a.out_w);
    int acc = 0;
    uint32_t acc_phase = 0;
    if (mine > 0) {
      // H^T: lane c, a 32-bit column for every two rows; this warp's 32 columns and 64 rows
      mbar_wait(h_full, 0, abort_flag, a.status);
      const int c = q * 32 + lane;
      const uint8_t* src = sh_h + (c >> 6) * 16384 + (c & 7) * 2;
      uint32_t w[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const int r = half * 64 + 2 * j;       // (rows of 128 bytes, 16-byte words swizzled)
        const uint32_t lo = *reinterpret_cast<const uint16_t*>(
            src + r * 128 + ((((c & 63) >> 3) ^ (r & 7)) << 4));
        const uint32_t hi = *reinterpret_cast<const uint16_t*>(
            src + (r + 1) * 128 + ((((c & 63) >> 3) ^ ((r + 1) & 7)) << 4));
        w[j] = lo | (hi << 16);
      }
      tmem_st32(tbase + lanes + 256 + half * 32, w);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ht_full);
    }
    for (int i = 0; i < mine; ++i) {
      mbar_wait(&acc_full[acc], acc_phase, abort_flag, a.status);
      tc_fence_after();
      float v[32];                               // column c0 + 32 q + lane, 32 vocabulary rows
      tmem_ld32(tbase + lanes + 128 + acc * 64 + half * 32, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
      if (!a.do_w) continue;
      // [32 v][32 c]: a store writes two rows, a word of every bank
      uint32_t* t = reinterpret_cast<uint32_t*>(st);
      uint32_t x[16];
      pair_columns(v, lane, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) t[(2 * k + (lane & 1)) * 16 + (lane >> 1)] = x[k];
      __syncwarp();
      const int v0 = (slot + i * slots) * 64 + half * 32, c = c0 + q * 32 + (lane & 3) * 8;
      uint4 w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = *reinterpret_cast<const uint4*>(t + (k * 8 + (lane >> 2)) * 16 + (lane & 3) * 4);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = v0 + k * 8 + (lane >> 2);
        if (r >= a.vc || c >= a.d) continue;
        __nv_bfloat16* dst = out_w + (size_t)r * a.d + c;
        if (a.vec_ok && c + 8 <= a.d) {
          __stcs(reinterpret_cast<uint4*>(dst), w[k]);
        } else {
          const __nv_bfloat16* e = reinterpret_cast<const __nv_bfloat16*>(&w[k]);
          for (int x = 0; x < 8; ++x)
            if (c + x < a.d) dst[x] = e[x];
        }
      }
    }
    if (a.do_w && n == 0) {
      // no row takes part: zeros
      for (int v = slot * 8 + (warp - 2); v < a.vc; v += slots * 8)
        for (int c = c0 + lane; c < min(a.d, c0 + 128); c += 32)
          out_w[(size_t)v * a.d + c] = __nv_bfloat16(0.f);
    }
    if (a.do_h) {
      // this slot's sums of dH (zeros when it had no block)
      if (mine > 0) {
        mbar_wait(dh_full, 0, abort_flag, a.status);
        tc_fence_after();
      }
      const int row = q * 32 + lane;
      float* base = a.acc + (size_t)slot * a.r_pad * a.d_pad;
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int col = c0 + half * 64 + b * 32;
        float v[32];
        if (mine > 0) {
          tmem_ld32(tbase + lanes + half * 64 + b * 32, v);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        }
        stage_f32(st, lane, v);
        if (a.acc_add) {
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            const int r = it * 4 + (lane >> 3), ch = lane & 7;
            if (row - lane + r < n && col + ch * 4 < a.d_pad) {
              float4* s4 = reinterpret_cast<float4*>(stage_at<128>(st, r, ch));
              const float4 o = *reinterpret_cast<const float4*>(
                  base + (size_t)(row - lane + r) * a.d_pad + col + ch * 4);
              float4 w = *s4;
              w.x += o.x; w.y += o.y; w.z += o.z; w.w += o.w;
              *s4 = w;
            }
          }
        }
        flush_rows<float, 128, false>(st, lane, col, a.d_pad, true, [&](int r) -> float* {
          return row - lane + r < n ? base + (size_t)(row - lane + r) * a.d_pad : nullptr;
        });
      }
    }
  }
  if (*abort_flag) let_land();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

// ------------------------------------------------------------------------------------------
// Rows
// ------------------------------------------------------------------------------------------
struct RowsArgs {
  int rows, d, d_pad, vocab, r_pad, per;   // per: rows of one CTA
  int row_ctas;
  bool f32, in_place, vec, pad_rows;
  long long ld;
  const void* hidden;
  const int* target;
  int* counts;                 // [row_ctas] listed rows of every CTA; null: the CTAs count them
  HeadMeta* meta;
  int* row_idx;
  __nv_bfloat16* out;          // [parts][r_pad][d_pad]
  const void* hidden16;        // fp16 rows of the same shape, contiguous; null: none
  __nv_bfloat16* out16;        // their copies
  int* row_tgt;                // [r_pad] targets of the listed rows; null: not wanted
  int4* perm;                  // [r_pad] listed rows in order of (target, row), as (row, its `run`,
                               // target, 0); null: not wanted
  int* run;                    // [r_pad] (see HeadDev)
  int* inv;                    // instead of those two, with counts: caller's row -> listed row
  int2* ids;                   // [vocab] to clear; null: not wanted
  float *nll, *lse;            // loss: zero for the rows that take no part
  void* grad_hidden;           // gradient: likewise
  bool gvec;
  uint32_t* status;
};

// Copy (bf16) or split (fp32) one row of d elements into d_pad bf16 columns, zeros behind the
// row, by one warp; x null: all zeros.  vec: the row starts on a 16-byte boundary and d fills
// whole 16-byte words.  Four loads per lane are in flight.
template <typename T>
SMDM_DEV void put_row(const T* x, int d, int d_pad, bool vec, __nv_bfloat16* o, size_t plane,
                      int lane) {
  constexpr int B = 4;
  if (vec || !x) {
    constexpr int E = 16 / (int)sizeof(T);
    for (int c0 = lane * E; c0 < d_pad; c0 += B * 32 * E) {
      uint4 r[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int c = c0 + b * 32 * E;
        r[b] = x && c < d ? *reinterpret_cast<const uint4*>(x + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int c = c0 + b * 32 * E;
        if (c >= d_pad) break;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint4*>(o + c) = r[b];
        } else {
          const uint32_t w[4] = {r[b].x, r[b].y, r[b].z, r[b].w};
          __nv_bfloat16 p[3][4];
#pragma unroll
          for (int k = 0; k < 4; ++k) split3(__uint_as_float(w[k]), p[0][k], p[1][k], p[2][k]);
#pragma unroll
          for (int k = 0; k < 3; ++k)
            *reinterpret_cast<uint2*>(o + k * plane + c) = *reinterpret_cast<const uint2*>(p[k]);
        }
      }
    }
    return;
  }
  for (int c0 = lane; c0 < d_pad; c0 += 2 * B * 32) {
    T r[2 * B];
#pragma unroll
    for (int b = 0; b < 2 * B; ++b) r[b] = c0 + b * 32 < d ? x[c0 + b * 32] : T(0.f);
#pragma unroll
    for (int b = 0; b < 2 * B; ++b) {
      const int c = c0 + b * 32;
      if (c >= d_pad) break;
      if constexpr (sizeof(T) == 2) {
        o[c] = r[b];
      } else {
        split3(r[b], o[c], o[plane + c], o[2 * plane + c]);
      }
    }
  }
}

SMDM_DEV void copy_row(const RowsArgs& a, int src, __nv_bfloat16* out, int dst, int lane) {
  if (a.hidden16)              // (moved as they are, whatever two-byte type they have)
    put_row(static_cast<const __nv_bfloat16*>(a.hidden16) + (size_t)src * a.d, a.d, a.d_pad, true,
            a.out16 + (size_t)dst * a.d_pad, 0, lane);
  const size_t plane = (size_t)a.r_pad * a.d_pad;
  __nv_bfloat16* o = out + (size_t)dst * a.d_pad;
  if (a.f32)
    put_row(static_cast<const float*>(a.hidden) + (size_t)src * a.ld, a.d, a.d_pad, a.vec, o, plane,
            lane);
  else
    put_row(static_cast<const __nv_bfloat16*>(a.hidden) + (size_t)src * a.ld, a.d, a.d_pad, a.vec,
            o, plane, lane);
}

// The weight rows of one piece that TMA cannot read in place: fp32 ones, split into three bf16
// parts, or bf16 ones whose rows do not start on 16-byte boundaries.
struct WeightArgs {
  const void* w;
  long long ld;
  int vc, vc_pad;      // rows, and rows to fill (zeros behind)
  bool vec;
  __nv_bfloat16* out;  // [parts][vc_pad][d_pad]
  int ctas;            // 0: nothing to do
};

SMDM_DEV void put_weights(const RowsArgs& a, const WeightArgs& w, int cta) {
  const int lane = threadIdx.x & 31;
  const size_t plane = (size_t)w.vc_pad * a.d_pad;
  for (int v = cta * 8 + (threadIdx.x >> 5); v < w.vc_pad; v += w.ctas * 8) {
    __nv_bfloat16* o = w.out + (size_t)v * a.d_pad;
    if (a.f32)
      put_row(v < w.vc ? static_cast<const float*>(w.w) + (size_t)v * w.ld : nullptr, a.d, a.d_pad,
              w.vec, o, plane, lane);
    else
      put_row(v < w.vc ? static_cast<const __nv_bfloat16*>(w.w) + (size_t)v * w.ld : nullptr, a.d,
              a.d_pad, w.vec, o, plane, lane);
  }
}

// Sum over a CTA of 256 threads.
SMDM_DEV int cta_sum(int s, int* red) {
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = 0;
  for (int w = 0; w < 8; ++w) s += red[w];
  return s;
}

// How many rows of every CTA of head_rows_kernel take part.
__global__ void __launch_bounds__(256) head_count_kernel(RowsArgs a) {
  griddep_launch();
  griddep_wait();
  __shared__ int red[8];
  const int r0 = blockIdx.x * a.per, r1 = min(a.rows, r0 + a.per);
  int s = 0;
  for (int base = r0 + threadIdx.x; base < r1; base += 8 * 256) {
    int t[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) t[k] = base + k * 256 < r1 ? a.target[base + k * 256] : -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += t[k] >= 0 && t[k] < a.vocab;
  }
  s = cta_sum(s, red);
  if (threadIdx.x == 0) a.counts[blockIdx.x] = s;
}

// List the rows that take part, in order, and copy them together.  Every CTA needs to know how
// many listed rows precede its own and whether all rows are listed: up to kListRows rows it reads
// all targets (from L2), which takes less time than a second launch; of more rows a kernel in
// front has counted each CTA's.  The CTAs behind row_ctas lay out the first
// piece's weights meanwhile, where those cannot be read in place.
// For the remainders of D the rows are also put in order of their targets: up to kListRows rows
// with kOwn rows per CTA, which compares them with all targets as it reads them; more rows are
// sorted (launch_sort_ids).
constexpr int kOwn = 8;

__global__ void __launch_bounds__(256) head_rows_kernel(RowsArgs a, WeightArgs w) {
  griddep_launch();
  griddep_wait();
  if ((int)blockIdx.x >= a.row_ctas) {
    put_weights(a, w, blockIdx.x - a.row_ctas);
    return;
  }
  __shared__ int red[2][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.x * a.per, r1 = min(a.rows, r0 + a.per);
  __shared__ int2 s_rank[8][kOwn];
  int before = 0, total = 0;
  if (a.perm) {
    // as below, and for the CTA's own rows (kOwn at most) how many listed rows have a smaller
    // target, how many the same, and how many of those come before
    int own[kOwn], less[kOwn], same[kOwn];       // same: << 16 those before
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      own[j] = r0 + j < r1 ? a.target[r0 + j] : -1;
      less[j] = same[j] = 0;
    }
    for (int base = tid; base < a.rows; base += 8 * 256) {
      int t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = a.target[min(base + k * 256, a.rows - 1)];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = base + k * 256;
        const bool on = r < a.rows && t[k] >= 0 && t[k] < a.vocab;
        if (!on) t[k] = 0x7fffffff;              // neither below nor equal to any target
        total += on;
        before += on && r < r0;
        const int one = r < r0 ? 0x10001 : 1;    // (the own rows among themselves: below)
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
          less[j] += t[k] < own[j];
          same[j] += t[k] == own[j] ? one : 0;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
      const int x = __reduce_add_sync(0xffffffffu, less[j]);
      int y = __reduce_add_sync(0xffffffffu, same[j]);
      if (warp == 0)
        for (int i = 0; i < j; ++i) y += own[i] == own[j] ? 0x10000 : 0;
      if (lane == 0) s_rank[warp][j] = make_int2(x, y);
    }
  } else if (a.counts) {
    for (int i = tid; i < a.row_ctas; i += 256) {
      const int c = a.counts[i];
      total += c;
      if (i < (int)blockIdx.x) before += c;
    }
  } else {
    for (int base = tid; base < a.rows; base += 8 * 256) {
      int t[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) t[k] = a.target[min(base + k * 256, a.rows - 1)];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = base + k * 256;
        const bool on = r < a.rows && t[k] >= 0 && t[k] < a.vocab;
        total += on;
        if (r < r0) before += on;
      }
    }
  }
  const int n = cta_sum(total, red[0]);
  int at = cta_sum(before, red[1]);
  const bool dense = a.in_place && n == a.rows;
  if (a.ids)
    for (int v = blockIdx.x * 256 + tid; v < a.vocab; v += a.row_ctas * 256)
      a.ids[v] = make_int2(0, 0);
  if (tid == 0 && blockIdx.x == 0) {
    a.meta->n = n;
    a.meta->dense = dense ? 1 : 0;
  }
  // 32 rows at a time: every warp works out the same listed positions, then takes every 8th row
  for (int b = r0; b < r1; b += 32) {
    const int r = b + lane;
    const int t = r < r1 ? a.target[r] : -1;
    const bool on = t >= 0 && t < a.vocab;
    if (t >= a.vocab && warp == 0 && a.status) atomicOr(a.status, kStatusBounds);
    const uint32_t mask = __ballot_sync(0xffffffffu, on);
    const int pos = at + __popc(mask & ((1u << lane) - 1u));
    at += __popc(mask);
    if (warp == 0 && r < r1) {
      if (on) {
        a.row_idx[pos] = r;
        if (a.row_tgt) a.row_tgt[pos] = t;
        if (a.inv) a.inv[r] = pos;
        if (a.perm) {
          int2 k = make_int2(0, 0);
          for (int i = 0; i < 8; ++i) {
            k.x += s_rank[i][r - r0].x;
            k.y += s_rank[i][r - r0].y;
          }
          const int run = k.y < 0x10000 ? k.y : 0;
          a.perm[k.x + (k.y >> 16)] = make_int4(pos, run, t, 0);
          a.run[pos] = run;
        }
      } else if (a.nll) {
        a.nll[r] = 0.f;
        a.lse[r] = 0.f;
      }
    }
    for (int i = warp; i < min(32, r1 - b); i += 8) {
      const int p = __shfl_sync(0xffffffffu, pos, i);
      if ((mask >> i) & 1u) {
        if (!dense) copy_row(a, b + i, a.out, p, lane);
      } else if (a.grad_hidden) {
        const size_t es = a.f32 ? 4 : 2;
        uint8_t* g = static_cast<uint8_t*>(a.grad_hidden) + (size_t)(b + i) * a.d * es;
        if (a.gvec) {
          for (size_t c = lane * 16; c < a.d * es; c += 512)
            *reinterpret_cast<uint4*>(g + c) = make_uint4(0, 0, 0, 0);
        } else if (a.f32) {
          for (int c = lane; c < a.d; c += 32) reinterpret_cast<float*>(g)[c] = 0.f;
        } else {
          for (int c = lane; c < a.d; c += 32)
            reinterpret_cast<__nv_bfloat16*>(g)[c] = __nv_bfloat16(0.f);
        }
      }
    }
  }
  // the rows up to the next multiple of 64 (128 with one row tile) are summed over by dW: zeros,
  // every CTA its share
  if (a.pad_rows && !dense) {
    const int end = a.rows <= 128 ? 128 : (n + 63) & ~63;
    const size_t plane = (size_t)a.r_pad * a.d_pad;
    for (int r = n + blockIdx.x * 8 + warp; r < end; r += a.row_ctas * 8)
      for (int p = 0; p < (a.f32 ? 3 : 1); ++p)
        for (int c = lane * 8; c < a.d_pad; c += 256)
          *reinterpret_cast<uint4*>(a.out + p * plane + (size_t)r * a.d_pad + c) =
              make_uint4(0, 0, 0, 0);
  }
}

// The order of the listed rows by (target, row), and `run` of every row, from the sorted (target,
// caller's row) words.
__global__ void __launch_bounds__(256)
    head_perm_kernel(const HeadMeta* meta, const unsigned long long* sorted, const int* inv,
                     int4* perm, int* run) {
  griddep_launch();
  griddep_wait();
  const int n = meta->n, p = blockIdx.x * 256 + threadIdx.x;
  if (p >= n) return;
  const unsigned long long w = sorted[p];
  const unsigned key = (unsigned)(w >> 32);
  const int row = inv[(unsigned)w];
  int lo = p + 1, hi = n;                    // the end of the rows with this target
  if (p > 0 && (unsigned)(sorted[p - 1] >> 32) == key) lo = hi = p;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if ((unsigned)(sorted[mid] >> 32) == key) lo = mid + 1;
    else hi = mid;
  }
  perm[p] = make_int4(row, lo - p, (int)key, 0);
  run[row] = lo - p;
}

// rest[x] = the sum of delta_r h_r over the listed rows r with one target, in row order, for the
// targets of a piece that two or more rows have (one row's is added as it lies); x is the first of
// them.  A CTA takes 256 columns and the targets that begin at 32 places of the rows in order of
// their targets: a warp each, all warps together for one of more than kRestLong rows.  Summed in
// fp32, eight rows in flight per warp; kept in bf16, which is 2^-9 of 2^-9 of D's part of dW.
// 4096 rows with a quarter left out, 4096 x 8192: 13 us, mostly the latency of loads that follow one
// another; 786432 rows of 64 over 64 ids: 0.5 ms of 6.
struct RestArgs {
  const HeadMeta* meta;
  const int4* perm;
  const float* delta;
  const void* hidden;          // the caller's rows
  long long ld_hidden;
  const __nv_bfloat16* hid;    // the listed rows
  int d, d_pad, slabs, v0, vc;
  __nv_bfloat16* out;          // [r_pad][d_pad]
};

constexpr int kRestWarps = 8, kRestLong = 64;

__global__ void __launch_bounds__(kRestWarps * 32) head_rest_kernel(RestArgs a) {
  griddep_launch();
  griddep_wait();
  __shared__ __align__(16) float part[kRestWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int p0 = (int)(blockIdx.x / a.slabs) * 32, c = (int)(blockIdx.x % a.slabs) * 256 + lane * 8;
  const int4 at = a.perm[p0 + lane];         // (past the last row: nothing that is used)
  const int n = a.meta->n;
  if (p0 >= n) return;
  // both kinds of rows start on 16 bytes and fill 16-byte words
  const bool dense = a.meta->dense != 0;
  const __nv_bfloat16* h = dense ? static_cast<const __nv_bfloat16*>(a.hidden) : a.hid;
  const long long ld = dense ? a.ld_hidden : a.d_pad;
  const bool in = c < (dense ? a.d : a.d_pad);
  // the target that begins at this lane's place
  const int row = at.x;
  const int count = p0 + lane < n && at.z >= a.v0 && at.z < a.v0 + a.vc ? at.y : 0;
  float s[8];
  // the rows at the places [from, to)
  auto sum = [&](int from, int to) {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 0.f;
    for (; from < to; from += 32) {
      const int cnt = min(32, to - from);
      const int r = lane < cnt ? a.perm[from + lane].x : 0;
      const float delta = lane < cnt ? a.delta[r] : 0.f;
      for (int e0 = 0; e0 < cnt; e0 += 8) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = __shfl_sync(0xffffffffu, r, e0 + k);
          x[k] = in && e0 + k < cnt ? *reinterpret_cast<const uint4*>(h + (size_t)e * ld + c)
                                    : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (e0 + k >= cnt) break;
          const float f = __shfl_sync(0xffffffffu, delta, e0 + k);
          const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s[2 * j] = fmaf(f, __uint_as_float(w[j] << 16), s[2 * j]);
            s[2 * j + 1] = fmaf(f, __uint_as_float(w[j] & 0xffff0000u), s[2 * j + 1]);
          }
        }
      }
    }
  };
  auto put = [&](int to) {
    if (c >= a.d_pad) return;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack_bf16(s[2 * j], s[2 * j + 1]);
    *reinterpret_cast<uint4*>(a.out + (size_t)to * a.d_pad + c) = make_uint4(w[0], w[1], w[2], w[3]);
  };
  int turn = 0;
  const uint32_t few = __ballot_sync(0xffffffffu, count > 1 && count <= kRestLong);
  for (uint32_t m = few; m; m &= m - 1, ++turn) {
    if (turn % kRestWarps != warp) continue;
    const int i = __ffs(m) - 1;
    sum(p0 + i, p0 + i + __shfl_sync(0xffffffffu, count, i));
    put(__shfl_sync(0xffffffffu, row, i));
  }
  for (uint32_t m = __ballot_sync(0xffffffffu, count > kRestLong); m; m &= m - 1) {
    const int i = __ffs(m) - 1, k = __shfl_sync(0xffffffffu, count, i);
    const int per = (k + kRestWarps - 1) / kRestWarps, from = p0 + i + min(k, warp * per);
    sum(from, min(p0 + i + k, from + per));
#pragma unroll
    for (int j = 0; j < 8; j += 4)
      *reinterpret_cast<float4*>(&part[warp][lane * 8 + j]) =
          make_float4(s[j], s[j + 1], s[j + 2], s[j + 3]);
    __syncthreads();
    if (warp == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s[j] = 0.f;
        for (int w = 0; w < kRestWarps; ++w) s[j] += part[w][lane * 8 + j];
      }
      put(__shfl_sync(0xffffffffu, row, i));
    }
    __syncthreads();
  }
}

// The weights of a later piece.
__global__ void __launch_bounds__(256) head_weights_kernel(RowsArgs a, WeightArgs w) {
  griddep_launch();
  griddep_wait();
  put_weights(a, w, blockIdx.x);
}

// nll and lse of the listed rows from the column groups' (maximum, sum) pairs.  32 rows per CTA
// (a lane each), 32 warps over the groups; a warp has eight pairs in flight.
__global__ void __launch_bounds__(1024)
    head_finish_kernel(const HeadMeta* meta, const int* row_idx, const int* target, int rows,
                       int vocab, const float2* part, int n_part, int r_pad, const float* tlogit,
                       float* nll, float* lse, uint32_t* status) {
  griddep_launch();
  griddep_wait();
  __shared__ float2 sh[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int n = meta ? meta->n : rows;
  const int row = blockIdx.x * 32 + lane;
  if (blockIdx.x * 32 >= n) return;
  float m = -INFINITY, s = 0.f;
  for (int i0 = g; i0 < n_part; i0 += 32 * 8) {
    float2 p[8];
    float mn = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + k * 32;
      p[k] = (row < n && i < n_part) ? part[(size_t)i * r_pad + row] : make_float2(-INFINITY, 0.f);
      mn = fmaxf(mn, p[k].x);
    }
    s *= s == 0.f ? 0.f : ex2((m - mn) * kLog2e);
#pragma unroll
    for (int k = 0; k < 8; ++k)        // (a group past the vocabulary's end has sum 0)
      if (p[k].y != 0.f) s += p[k].y * ex2((p[k].x - mn) * kLog2e);
    m = mn;
  }
  sh[g][lane] = make_float2(m, s);
  __syncthreads();
  // warp g: row g of the CTA, a lane per group range
  const float2 p = sh[lane][g];
  m = p.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  s = p.y != 0.f ? p.y * ex2((p.x - m) * kLog2e) : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int out = blockIdx.x * 32 + g;
  if (lane == 0 && out < n) {
    const float l = logf(s);
    const int r = meta ? row_idx[out] : out;
    const int t = target[r];
    const bool on = t >= 0 && t < vocab;      // (without the list: also rows that take no part)
    if (t >= vocab && status) atomicOr(status, kStatusBounds);
    lse[r] = on ? m + l : 0.f;
    nll[r] = on ? (m - tlogit[out]) + l : 0.f;
  }
}

// dH from its fp32 sums: the K ranges in order, rounded once, at the caller's rows.
template <bool F32>
__global__ void __launch_bounds__(256)
    head_sum_kernel(const HeadMeta* meta, const int* row_idx, const float* acc, int splits,
                    int r_pad, int d, int d_pad, void* out) {
  griddep_launch();
  griddep_wait();
  const int n = meta->n;
  const size_t plane = (size_t)r_pad * d_pad;
  const int d4 = d_pad >> 2;
  const long long total = (long long)n * d4;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (long long)gridDim.x * 256) {
    const int r = (int)(i / d4), c = (int)(i % d4) * 4;
    if (c >= d) continue;
    const float* p = acc + (size_t)r * d_pad + c;
    float4 s = *reinterpret_cast<const float4*>(p);
#pragma unroll 8
    for (int k = 1; k < splits; ++k) {
      const float4 t = *reinterpret_cast<const float4*>(p + k * plane);
      s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
    }
    const float v[4] = {s.x, s.y, s.z, s.w};
    const size_t o = (size_t)row_idx[r] * d + c;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (c + k < d) {
        if constexpr (F32) static_cast<float*>(out)[o + k] = v[k];
        else static_cast<__nv_bfloat16*>(out)[o + k] = __float2bfloat16_rn(v[k]);
      }
  }
}

// The same for many K ranges and few rows: a CTA per row and 128 columns, eight warps over the
// ranges (each in order), then the warps' sums in order.
__global__ void __launch_bounds__(256)
    head_sum_deep_kernel(const HeadMeta* meta, const int* row_idx, const float* acc, int splits,
                         int r_pad, int d, int d_pad, __nv_bfloat16* out) {
  griddep_launch();
  griddep_wait();
  __shared__ __align__(16) float sh[8][128];
  const int r = blockIdx.y;
  if (r >= meta->n) return;
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int c = blockIdx.x * 128 + lane * 4;
  const size_t plane = (size_t)r_pad * d_pad;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (c < d_pad) {
    const float* p = acc + (size_t)r * d_pad + c;
#pragma unroll 4
    for (int k = g; k < splits; k += 8) {
      const float4 t = *reinterpret_cast<const float4*>(p + k * plane);
      s.x += t.x; s.y += t.y; s.z += t.z; s.w += t.w;
    }
  }
  *reinterpret_cast<float4*>(&sh[g][lane * 4]) = s;
  __syncthreads();
  const int cc = blockIdx.x * 128 + threadIdx.x;
  if (threadIdx.x < 128 && cc < d) {
    float t = 0.f;
    for (int i = 0; i < 8; ++i) t += sh[i][threadIdx.x];
    out[(size_t)row_idx[r] * d + cc] = __float2bfloat16_rn(t);
  }
}

// ------------------------------------------------------------------------------------------
// Host side
// ------------------------------------------------------------------------------------------
// Rows up to which head_rows_kernel's CTAs read all targets, and its CTAs at most.
constexpr int kListRows = 8192, kListCtas = 1024;

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int sm_count() {
  static int cached[64];
  int dev = 0, n = 148;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return n;
  if (!cached[dev] &&
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    cached[dev] = n;
  return cached[dev] ? cached[dev] : n;
}

struct Plan {
  bool few;           // head_few.cu takes the call
  int parts, terms, r_pad, d_pad;
  int d_parts, g_terms;   // bf16 parts of D; products summed by the gradients
  bool staged;        // weights go through a bf16 copy of each piece
  int piece, n_pieces;
  bool rest;          // D's remainders at the targets
  size_t meta, counts, row_idx, hid, hid16, part, tlogit, wst, dlog, acc, total;
  size_t row_tgt, delta, ids, run, perm, inv, sort[2], rest_rows;      // (rest)
  int cfg, cfg_g;     // tile configuration of the logits' product and of the gradients'
  int splits, n_part;
  int narrow;         // > 0: head_narrow_kernel, with this many vocabulary slots (= splits)
};

// Tile configurations: {CTAs per tile, columns}.  tile_cost() picks the one whose rounds of tiles
// end first.  Measured, 64 / 128 / 256 columns / pairs of 256: 4096 rows of 4096 x 8192
// 494 / 277 / 205 / 181 us; 8 rows of it 21 / 24 / 31 / - us (32 tiles of 256 columns leave most SMs
// idle); 8 rows of 1024 x 32000 24 / 20 / 18.5 / 22 us.
constexpr int kCfgCG[4] = {1, 1, 1, 2};
constexpr int kCfgBN[4] = {64, 128, 256, 256};

bool weight_in_place(int d, long long ld, bool f32) { return !f32 && d % 8 == 0 && ld % 8 == 0; }

// SM clocks of one K chunk with `m` rows of A and operands in `parts`: its MMAs, its bytes at 64
// per clock, or the threads that issue it.
double chunk_clocks(int cfg, long long m, int parts) {
  const int cg = kCfgCG[cfg], bn = kCfgBN[cfg];
  const int prod = parts == 3 ? 6 : parts, bp = parts == 3 ? 3 : 1;
  const double mma = prod * std::max(bn * 2.0, 200.0);
  const double bytes = (parts * kABytes * std::min<long long>(m, 128) / 128.0 + bp * bn / cg * 128.0) / 64.0;
  return std::max(mma + 150.0, bytes);
}

// Time of the product: rounds of tiles times a K chunk's time.
double tile_cost(int cfg, long long m, long long n, int sms, int parts) {
  const int cg = kCfgCG[cfg], bn = kCfgBN[cfg];
  const long long tiles = ((m + 128 * cg - 1) / (128 * cg)) * ((n + bn - 1) / bn);
  const long long slots = sms / cg;
  return (double)((tiles + slots - 1) / slots) * chunk_clocks(cfg, m, parts);
}

int pick_cfg(long long m, long long n, int sms, int parts) {
  int best = 0;
  double bc = 0;
  for (int c = 0; c < 4; ++c) {
    if (c == 2 && parts != 1) continue;
    const double t = tile_cost(c, m, n, sms, parts);
    if (c == 0 || t <= bc) { bc = t; best = c; }
  }
  return best;
}

// Vocabulary slots of head_narrow_kernel: one column group per CTA, a CTA per SM.
int narrow_slots(int d, int sms) { return std::max(1, sms / ((d + 127) / 128)); }

Plan make_plan(int rows, int d, int vocab, long long ld_head, bool f32, bool grad, bool half) {
  Plan p{};
  const int sms = sm_count();
  p.parts = f32 ? 3 : 1;
  p.terms = f32 ? 6 : 1;
  p.r_pad = (int)up(rows, 256);
  p.d_pad = (int)up(d, 64);
  p.staged = !weight_in_place(d, ld_head, f32);
  p.few = head_few_fits(rows, d) && p.staged;
  if (p.few) {
    p.total = head_few_bytes(rows, d, vocab, sms);
    return p;
  }
  p.d_parts = f32 ? 3 : rows <= 128 ? 2 : 1;
  p.g_terms = f32 ? 6 : 1;
  p.rest = grad && p.d_parts == 1;
  // widest piece whose D (gradient) and weight copy (when made) stay below kPieceBytes
  size_t per_col = 0;
  if (grad) per_col = (size_t)p.d_parts * p.r_pad * 2;
  if (p.staged) per_col = std::max(per_col, (size_t)p.parts * p.d_pad * 2);
  const int v_pad = (int)up(vocab, 256);
  p.piece = v_pad;
  if (per_col) p.piece = (int)std::min<size_t>(v_pad, std::max<size_t>(256, kPieceBytes / per_col / 256 * 256));
  // one row tile: no slot of head_narrow_kernel sums more than kNarrowBlocks blocks into its dH
  if (grad && !f32 && rows <= 128)
    p.piece = (int)std::min<long long>(p.piece, (long long)narrow_slots(d, sms) * kNarrowBlocks * 64);
  p.n_pieces = (vocab + p.piece - 1) / p.piece;
  // pieces of equal width
  p.piece = (int)up((vocab + p.n_pieces - 1) / p.n_pieces, 256);
  p.n_pieces = (vocab + p.piece - 1) / p.piece;
  p.cfg = pick_cfg(rows, std::min(p.piece, vocab), sms, p.parts);
  const int bn = kCfgBN[p.cfg];
  p.n_part = 2 * ((p.piece + bn - 1) / bn) * p.n_pieces;
  p.splits = 1;
  if (grad) {
    // The configuration whose slots finish both products first.  K ranges of dH are cut until a
    // unit takes no more than a slot's share of all the work.
    const long long kh = p.piece / 64, kw = (rows + 63) / 64;
    double best = 0;
    for (int c : {0, 1, 3}) {
      const int mt = 128 * kCfgCG[c], bnc = kCfgBN[c], slots = sms / kCfgCG[c];
      const long long nt = (d + bnc - 1) / bnc;
      const double ch = chunk_clocks(c, 128, p.d_parts), epi = bnc * 8.0 / ch;   // (a tile's fixed cost)
      const long long nh = (rows + mt - 1) / mt * nt, nw = (p.piece + mt - 1) / mt * nt;
      const double uh = (double)kh, uw = (double)kw + epi;
      const double share = (nh * (uh + epi) + nw * uw) / slots;
      const int s = (int)std::min<double>(std::min<long long>(32, kh), std::max(1.0, uh / std::max(share, 2.0)));
      const double t = ch * std::max(std::max(share, uw), uh / s + epi);
      if (c == 0 || t <= best) { best = t; p.cfg_g = c; p.splits = s; }
    }
    // one row tile: a column group per CTA, as many vocabulary slots as fill the SMs
    if (!f32 && rows <= 128) {
      p.narrow = (int)std::min<long long>(narrow_slots(d, sms), kh);
      p.splits = p.narrow;
      p.cfg = 0;
    }
  }
  size_t off = 0;
  auto take = [&](size_t b) {
    const size_t o = off;
    off = up(off + b, 1024);
    return o;
  };
  p.meta = take(256);
  p.counts = take(rows > kListRows ? kListCtas * 4 : 0);
  p.row_idx = take((size_t)p.r_pad * 4);
  p.hid = take((size_t)p.parts * p.r_pad * p.d_pad * 2);
  if (grad && half) p.hid16 = take((size_t)p.r_pad * p.d_pad * 2);
  if (!grad) {
    p.part = take((size_t)p.n_part * p.r_pad * 8);
    p.tlogit = take((size_t)p.r_pad * 4);
  }
  if (p.staged) p.wst = take((size_t)p.parts * p.piece * p.d_pad * 2);
  if (grad) {
    p.dlog = take((size_t)p.d_parts * p.r_pad * p.piece * 2);
    if (p.rest) {
      p.row_tgt = take((size_t)p.r_pad * 4);
      p.delta = take((size_t)p.r_pad * 4);
      p.ids = take((size_t)vocab * 8);
      p.run = take((size_t)p.r_pad * 4);
      p.perm = take((size_t)p.r_pad * 16);
      if (rows > kListRows) {
        p.inv = take((size_t)rows * 4);
        for (size_t& k : p.sort) k = take((size_t)rows * 8);
      }
      p.rest_rows = take((size_t)p.r_pad * p.d_pad * 2);
    }
    if (p.narrow || p.splits > 1 || p.n_pieces > 1) p.acc = take((size_t)p.splits * p.r_pad * p.d_pad * 4);
  }
  p.total = off;
  return p;
}

bool encode_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t ld,
                 uint32_t box_inner, uint32_t box_outer) {
  EncodeTiledFn fn = get_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {inner, outer};
  cuuint64_t strides[1] = {ld * 2};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
  CUtensorMap h, hc, w, dk, dm;
};

// Clusters of the pair kernels that fit the device at once (some SM groups are odd).
template <typename K>
int max_pairs(K kern, int smem) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  return n;
}

template <int kMode, int CG, int BN, int P, bool kLong = false>
cudaError_t launch_one(const Maps& m, HeadDev a, long long units, int sms, cudaStream_t st) {
  constexpr int kStage = kChunks<kMode, CG, BN, P> *
                         (kAParts<P> * kABytes + kBParts<P> * (BN / CG * 128));
  const int budget = kSmemLimit - 1024 - kStagingBytes - 512;
  a.nstages = std::min(kMaxStages, budget / kStage);
  a.staging_off = a.nstages * kStage;
  a.bar_off = a.staging_off + kStagingBytes;
  const int smem = a.bar_off + 512 + 1024;
  auto kern = head_gemm_kernel<kMode, CG, BN, P, kLong>;
  // per device: the shared-memory opt-in and the number of pairs that fit
  static int ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit);
    if (e != cudaSuccess) return e;
    int n = sms;
    if (CG == 2) {
      n = max_pairs(kern, smem);
      if (n <= 0) n = sms / 2;
    }
    ready[dev] = n;
  }
  long long slots = std::min<long long>(ready[dev], units);
  if (slots < 1) slots = 1;
  return launch_pdl(kern, dim3((unsigned)(slots * CG)), dim3(kThreads), (size_t)smem, st, CG, m.h,
                    m.hc, m.w, m.dk, m.dm, a);
}

template <int kMode, int P, bool kLong = false>
cudaError_t launch_cfg(int cfg, const Maps& m, const HeadDev& a, long long units, int sms,
                       cudaStream_t st) {
  switch (cfg) {
    case 0: return launch_one<kMode, 1, 64, P, kLong>(m, a, units, sms, st);
    case 1: return launch_one<kMode, 1, 128, P, kLong>(m, a, units, sms, st);
    case 2:
      if constexpr (kMode != kGrad && P == 1) return launch_one<kMode, 1, 256, P>(m, a, units, sms, st);
      break;
    case 3: return launch_one<kMode, 2, 256, P, kLong>(m, a, units, sms, st);
  }
  return cudaErrorInvalidValue;
}

template <int kMode>
cudaError_t launch_mode(int parts, int cfg, const Maps& m, const HeadDev& a, long long units,
                        int sms, cudaStream_t st) {
  if (parts == 3) return launch_cfg<kMode, 3>(cfg, m, a, units, sms, st);
  if constexpr (kMode == kGrad) {
    const long long rows = a.do_w ? a.rows : 0, ids = a.do_h ? (a.vc + a.splits - 1) / a.splits : 0;
    if (std::max(rows, ids) > 64 * kWholeK)
      return launch_cfg<kMode, 1, true>(cfg, m, a, units, sms, st);
  }
  return launch_cfg<kMode, 1>(cfg, m, a, units, sms, st);
}

cudaError_t launch_narrow(const Maps& m, const HeadDev& a, int slots, cudaStream_t st) {
  constexpr int smem = kNarrowStages * kNarrowStage + kNarrowH + kStagingBytes + 512 + 1024;
  static_assert(smem <= kSmemLimit, "narrow kernel's shared memory");
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(head_narrow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  return launch_pdl(head_narrow_kernel, dim3((a.d + 127) / 128, slots), dim3(kThreads),
                    (size_t)smem, st, 1, m.h, m.hc, m.w, m.dk, a, slots);
}

#define TRY(x)                        \
  do {                                \
    cudaError_t e_ = (x);             \
    if (e_ != cudaSuccess) return e_; \
  } while (0)

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Call {
  const HeadArgs& h;
  Plan p;
  int sms;
  uint8_t* ws;
  bool in_place;    // the caller's hidden can be read by TMA
  bool loss;
  template <typename T> T* at(size_t off) const { return reinterpret_cast<T*>(ws + off); }

  Call(const HeadArgs& a, bool grad)
      : h(a), p(make_plan(a.rows, a.d, a.vocab, a.ld_head, a.f32, grad, a.half)), sms(sm_count()),
        ws(static_cast<uint8_t*>(a.ws)), loss(!grad) {
    in_place = !a.f32 && a.d % 8 == 0 && a.ld_hidden % 8 == 0 && aligned16(a.hidden);
  }

  RowsArgs row_args() const {
    RowsArgs r{};
    r.rows = h.rows;
    r.d = h.d;
    r.d_pad = p.d_pad;
    r.vocab = h.vocab;
    r.r_pad = p.r_pad;
    const bool order = p.rest && h.grad_head, counted = h.rows > kListRows;
    r.per = order && !counted ? kOwn : std::max(8, (h.rows + kListCtas - 1) / kListCtas);
    r.row_ctas = (h.rows + r.per - 1) / r.per;
    r.f32 = h.f32;
    r.in_place = in_place;
    r.pad_rows = !loss;
    r.vec = whole_words(h.hidden, h.ld_hidden);
    r.ld = h.ld_hidden;
    r.hidden = h.hidden;
    r.target = h.target;
    r.counts = counted ? at<int>(p.counts) : nullptr;
    r.meta = at<HeadMeta>(p.meta);
    r.row_idx = at<int>(p.row_idx);
    r.out = at<__nv_bfloat16>(p.hid);
    if (!loss && h.half) {
      r.hidden16 = h.hidden16;
      r.out16 = at<__nv_bfloat16>(p.hid16);
    }
    r.nll = h.nll;
    r.lse = h.lse_out;
    if (p.rest) {
      r.row_tgt = at<int>(p.row_tgt);
      if (order) r.ids = at<int2>(p.ids);
      if (order && counted) {
        r.inv = at<int>(p.inv);
      } else if (order) {
        r.perm = at<int4>(p.perm);
        r.run = at<int>(p.run);
      }
    }
    r.grad_hidden = h.grad_hidden;
    r.gvec = whole_words(h.grad_hidden, h.d);
    r.status = h.status;
    return r;
  }
  // rows of h.d elements, ld apart, that start on 16-byte boundaries and fill 16-byte words
  bool whole_words(const void* t, long long ld) const {
    const int es = h.f32 ? 4 : 2;
    return aligned16(t) && (long long)h.d * es % 16 == 0 && ld * es % 16 == 0;
  }
  WeightArgs weight_args(int v0, int vc) const {
    WeightArgs w{};
    if (!p.staged) return w;
    const size_t es = h.f32 ? 4 : 2;
    w.w = static_cast<const uint8_t*>(h.head) + (size_t)v0 * h.ld_head * es;
    w.ld = h.ld_head;
    w.vc = vc;
    w.vc_pad = (int)up(vc, 256);
    w.vec = whole_words(w.w, h.ld_head);
    w.out = at<__nv_bfloat16>(p.wst);
    w.ctas = std::min(w.vc_pad / 8, sms * 8);
    return w;
  }
  // The loss of at most 128 rows that lie on 16-byte boundaries skips the list: they fill one
  // row of tiles either way, and a row of the product that takes no part touches no other.  (Not
  // the gradient: dW sums over the rows.)
  bool listed() const { return !(loss && in_place && !p.staged && h.rows <= 128); }
  // Launches of rows().
  int row_launches() const {
    if (!listed()) return 0;
    if (h.rows <= kListRows) return 1;
    return 2 + (p.rest && h.grad_head ? sort_ids_launches(h.rows) + 1 : 0);
  }
  HeadMeta* meta() const { return listed() ? at<HeadMeta>(p.meta) : nullptr; }
  // The rows that take part, and the first piece's weights.
  cudaError_t rows(cudaStream_t st) const {
    if (!listed()) return cudaSuccess;
    const RowsArgs r = row_args();
    const WeightArgs w = weight_args(0, std::min(p.piece, h.vocab));
    if (r.counts) TRY(launch_pdl(head_count_kernel, dim3(r.row_ctas), dim3(256), 0, st, 1, r));
    TRY(launch_pdl(head_rows_kernel, dim3(r.row_ctas + w.ctas), dim3(256), 0, st, 1, r, w));
    if (!r.inv) return cudaSuccess;
    const unsigned long long* sorted = nullptr;
    TRY(launch_sort_ids(h.target, h.rows, h.vocab, at<unsigned long long>(p.sort[0]),
                        at<unsigned long long>(p.sort[1]), nullptr, 0, nullptr, st, &sorted));
    return launch_pdl(head_perm_kernel, dim3((h.rows + 255) / 256), dim3(256), 0, st, 1,
                      (const HeadMeta*)r.meta, sorted, (const int*)r.inv, at<int4>(p.perm),
                      at<int>(p.run));
  }
  // The weights of a later piece: read in place, or copied into the workspace.
  cudaError_t weights(int v0, int vc, cudaStream_t st) const {
    if (!p.staged || v0 == 0) return cudaSuccess;
    const WeightArgs w = weight_args(v0, vc);
    return launch_pdl(head_weights_kernel, dim3(w.ctas), dim3(256), 0, st, 1, row_args(), w);
  }
  // The operands of the logits, where they are others than the gradient's products have.
  bool half_maps(Maps* m, uint32_t h_rows, uint32_t w_rows) const {
    return encode_bf16(&m->h, h.hidden16, h.d, h.rows, h.d, 64, h_rows) &&
           encode_bf16(&m->hc, at<uint8_t>(p.hid16), p.d_pad, p.r_pad, p.d_pad, 64, h_rows) &&
           encode_bf16(&m->w, h.head16, h.d, h.vocab, h.d, 64, w_rows);
  }
  bool weight_map(CUtensorMap* m, int vc, uint32_t box_rows) const {
    if (p.staged)
      return encode_bf16(m, at<uint8_t>(p.wst), p.d_pad, (uint64_t)p.parts * up(vc, 256), p.d_pad,
                         64, box_rows);
    return encode_bf16(m, h.head, h.d, h.vocab, h.ld_head, 64, box_rows);
  }
  bool hidden_maps(CUtensorMap* in, CUtensorMap* listed, uint32_t box_rows) const {
    bool ok = encode_bf16(listed, at<uint8_t>(p.hid), p.d_pad, (uint64_t)p.parts * p.r_pad,
                          p.d_pad, 64, box_rows);
    if (in_place) ok &= encode_bf16(in, h.hidden, h.d, h.rows, h.ld_hidden, 64, box_rows);
    else *in = *listed;
    return ok;
  }
  HeadDev dev(int v0, int vc) const {
    HeadDev a{};
    a.meta = meta();
    a.rows = h.rows;
    a.row_idx = at<int>(p.row_idx);
    a.target = h.target;
    a.d = h.d;
    a.v0 = v0;
    a.vc = vc;
    a.w_row0 = p.staged ? 0 : v0;
    a.spread = (p.staged ? p.d_pad : h.ld_head) * 2 % 2048 == 0;
    a.terms = p.terms;
    a.h_plane = p.r_pad;
    a.w_plane = p.staged ? (int)up(vc, 256) : 0;
    a.d_plane = p.r_pad;
    a.r_pad = p.r_pad;
    a.d_pad = p.d_pad;
    a.status = h.status;
    a.half = h.half;
    return a;
  }
  // fp16 operands are read in place only
  bool half_ok() const {
    if (!h.half) return true;
    if (h.f32 || !in_place || p.staged) return false;
    return loss || (h.hidden16 && h.head16 && aligned16(h.hidden16) && aligned16(h.head16));
  }
  // Rows of D that head_narrow_kernel reads for rows that take part: its steps over them.
  int narrow_rows() const { return h.rows <= 16 ? 16 : h.rows <= 64 ? 64 : 128; }
  // rows of A that one box brings: no more than there are (a multiple of 8)
  int a_box() const { return (int)std::min<size_t>(128, up(h.rows, 8)); }
};

}  // namespace

size_t head_workspace_bytes(int rows, int d, int vocab, bool f32, bool grad, bool half) {
  // the layout that copies the weights is the larger one; it serves every row stride
  return std::max(make_plan(rows, d, vocab, 0, f32, grad, half).total,
                  make_plan(rows, d, vocab, 1, f32, grad, half).total);
}

bool head_needs_aligned_weight(int d, long long ld_head, bool f32) {
  return weight_in_place(d, ld_head, f32);
}

int head_loss_launches(const HeadArgs& a) {
  const Call c(a, false);
  const Plan& p = c.p;
  if (p.few) return 1 + head_few_groups(a.rows, a.d);
  return 1 + c.row_launches() + p.n_pieces + (p.staged ? p.n_pieces - 1 : 0);
}

int head_grad_launches(const HeadArgs& a) {
  const Call c(a, true);
  const Plan& p = c.p;
  if (p.few) return 1 + head_few_groups(a.rows, a.d) + (a.grad_hidden ? 1 : 0);
  const bool sums = p.narrow || p.splits > 1 || p.n_pieces > 1;
  return c.row_launches() + (p.rest && a.grad_head ? 3 : 2) * p.n_pieces +
         (p.staged ? p.n_pieces - 1 : 0) + (sums && a.grad_hidden ? 1 : 0);
}

cudaError_t launch_head_loss(const HeadArgs& h, cudaStream_t st) {
  const Call c(h, false);
  const Plan& p = c.p;
  if (!c.half_ok()) return cudaErrorInvalidValue;
  if (p.few) return launch_head_few_loss(h, c.sms, st);
  TRY(c.rows(st));
  const int cg = kCfgCG[p.cfg], bn = kCfgBN[p.cfg];
  for (int i = 0; i < p.n_pieces; ++i) {
    const int v0 = i * p.piece, vc = std::min(p.piece, h.vocab - v0);
    TRY(c.weights(v0, vc, st));
    Maps m;
    HeadDev a = c.dev(v0, vc);
    a.a_box = c.a_box();
    if (!c.hidden_maps(&m.h, &m.hc, a.a_box) || !c.weight_map(&m.w, vc, bn / cg))
      return cudaErrorInvalidValue;
    m.dk = m.dm = m.hc;
    a.part = c.at<float2>(p.part);
    a.part0 = 2 * (p.piece / bn) * i;
    a.tlogit = c.at<float>(p.tlogit);
    const long long units = (long long)((h.rows + 128 * cg - 1) / (128 * cg)) * ((vc + bn - 1) / bn);
    TRY(launch_mode<kLoss>(p.parts, p.cfg, m, a, units, c.sms, st));
  }
  const int last = h.vocab - (p.n_pieces - 1) * p.piece;
  const int n_part = 2 * (p.piece / bn) * (p.n_pieces - 1) + 2 * ((last + bn - 1) / bn);
  return launch_pdl(head_finish_kernel, dim3((h.rows + 31) / 32), dim3(1024),
                    0, st, 1, c.meta(), c.at<int>(p.row_idx), h.target, h.rows, h.vocab,
                    c.at<float2>(p.part), n_part, p.r_pad, c.at<float>(p.tlogit), h.nll, h.lse_out,
                    h.status);
}

cudaError_t launch_head_grad(const HeadArgs& h, cudaStream_t st) {
  const Call c(h, true);
  const Plan& p = c.p;
  if (!c.half_ok()) return cudaErrorInvalidValue;
  if (p.few) return launch_head_few_grad(h, c.sms, st);
  TRY(c.rows(st));
  const int cg = kCfgCG[p.cfg], bn = kCfgBN[p.cfg];
  const int gcg = kCfgCG[p.cfg_g], gbn = kCfgBN[p.cfg_g];
  const size_t es = h.f32 ? 4 : 2;
  const bool sums = p.narrow || p.splits > 1 || p.n_pieces > 1;
  for (int i = 0; i < p.n_pieces; ++i) {
    const int v0 = i * p.piece, vc = std::min(p.piece, h.vocab - v0);
    TRY(c.weights(v0, vc, st));
    Maps m;
    HeadDev a = c.dev(v0, vc);
    a.a_box = c.a_box();
    if (!(h.half ? c.half_maps(&m, a.a_box, bn / cg)
                 : c.hidden_maps(&m.h, &m.hc, a.a_box) && c.weight_map(&m.w, vc, bn / cg)))
      return cudaErrorInvalidValue;
    m.dk = m.dm = m.hc;
    a.d_parts = p.d_parts;
    a.d_rows = p.narrow ? c.narrow_rows() : p.r_pad;
    a.lse = h.lse;
    a.grad_nll = h.grad_nll;
    a.dlog = c.at<__nv_bfloat16>(p.dlog);
    a.ld_dlog = p.piece;
    if (p.rest) {
      a.row_tgt = c.at<int>(p.row_tgt);
      a.delta = c.at<float>(p.delta);
      if (h.grad_head) {
        a.run = c.at<int>(p.run);
        a.ids = c.at<int2>(p.ids);
        a.hidden = h.hidden;
        a.ld_hidden = h.ld_hidden;
        a.hid = c.at<__nv_bfloat16>(p.hid);
        a.rest = c.at<__nv_bfloat16>(p.rest_rows);
      }
      a.head = h.head;
      a.ld_head = h.ld_head;
      a.head_vec = c.whole_words(h.head, h.ld_head);
    }
    const long long units = (long long)((h.rows + 128 * cg - 1) / (128 * cg)) * ((vc + bn - 1) / bn);
    TRY(launch_mode<kDlog>(p.parts, p.cfg, m, a, units, c.sms, st));
    if (a.rest) {
      const int slabs = (p.d_pad + 255) / 256;
      const RestArgs r{a.meta, c.at<int4>(p.perm), a.delta, h.hidden, h.ld_hidden,
                       c.at<__nv_bfloat16>(p.hid), h.d, p.d_pad, slabs, v0, vc,
                       c.at<__nv_bfloat16>(p.rest_rows)};
      const long long ctas = (long long)((h.rows + 31) / 32) * slabs;
      TRY(launch_pdl(head_rest_kernel, dim3((unsigned)ctas), dim3(kRestWarps * 32), 0, st, 1, r));
    }
    // both products of D: 64-row boxes for the MN-major operands
    if (!c.hidden_maps(&m.h, &m.hc, 64) || !c.weight_map(&m.w, vc, 64) ||
        !encode_bf16(&m.dk, a.dlog, p.piece, (uint64_t)p.d_parts * p.r_pad, p.piece, 64,
                     p.narrow ? a.d_rows : 128) ||
        !encode_bf16(&m.dm, a.dlog, p.piece, (uint64_t)p.d_parts * p.r_pad, p.piece, 64, 64))
      return cudaErrorInvalidValue;
    a.terms = p.g_terms;
    a.do_h = h.grad_hidden != nullptr;
    a.do_w = h.grad_head != nullptr;
    a.splits = p.splits;
    a.acc = sums ? c.at<float>(p.acc) : nullptr;
    a.acc_add = i > 0;
    a.out_h = h.grad_hidden;
    a.out_w = h.grad_head ? static_cast<uint8_t*>(h.grad_head) + (size_t)v0 * h.d * es : nullptr;
    a.vec_ok = (size_t)h.d * es % 16 == 0 && (!h.grad_hidden || aligned16(h.grad_hidden)) &&
               (!h.grad_head || aligned16(h.grad_head));
    if (p.narrow) {
      TRY(launch_narrow(m, a, p.narrow, st));
      continue;
    }
    const long long nt = (h.d + gbn - 1) / gbn;
    const long long gu = (a.do_h ? nt * ((h.rows + 128 * gcg - 1) / (128 * gcg)) * p.splits : 0) +
                         (a.do_w ? nt * ((vc + 128 * gcg - 1) / (128 * gcg)) : 0);
    TRY(launch_mode<kGrad>(p.d_parts, p.cfg_g, m, a, gu, c.sms, st));
  }
  if (sums && h.grad_hidden) {
    if (p.narrow)
      return launch_pdl(head_sum_deep_kernel, dim3((h.d + 127) / 128, h.rows), dim3(256), 0, st, 1,
                        c.at<HeadMeta>(p.meta), c.at<int>(p.row_idx), c.at<float>(p.acc),
                        p.splits, p.r_pad, h.d, p.d_pad,
                        static_cast<__nv_bfloat16*>(h.grad_hidden));
    const long long n4 = (long long)h.rows * (p.d_pad / 4);
    const int grid = (int)std::min<long long>((n4 + 255) / 256, (long long)c.sms * 16);
    auto k = h.f32 ? head_sum_kernel<true> : head_sum_kernel<false>;
    TRY(launch_pdl(k, dim3(grid), dim3(256), 0, st, 1, c.at<HeadMeta>(p.meta),
                   c.at<int>(p.row_idx), c.at<float>(p.acc), p.splits, p.r_pad, h.d, p.d_pad,
                   h.grad_hidden));
  }
  return cudaSuccess;
}

}  // namespace smdm
