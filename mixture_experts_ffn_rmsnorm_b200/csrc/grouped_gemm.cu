// Ragged products grouped by expert on the 5th-generation tensor cores, and
// their gradients (moe_grouped_gemm, moe_grouped_gemm_dgrad,
// moe_grouped_gemm_wgrad).
//
// Expert e owns rows off[e] <= p < off[e + 1] of the sorted row tensors and
// the matrix W_e [N, K]:
//   forward         y[p, n]   = act(sum_k W_e[n, k] x[p, k])
//   data gradient   dx[p, k]  = sum_n W_e[n, k] dy[p, n]
//   weight gradient dW_e[n, k] = sum_p dy[p, n] x[p, k]
// Each is C[r, c] = sum_q A[c, q] B[r, q] per expert, with c the contiguous
// dimension of the output.  c is the tensor cores' M (TMEM lanes) and r their
// N (TMEM columns): N comes in steps of 16, so a group of few rows costs a
// narrow MMA instead of a padded 128-row one, and a warp's lanes hold
// neighbouring elements of an output row.
//   forward:         c = n, r = rows, q = k: A = W_e K-major,  B = x K-major
//   data gradient:   c = k, r = rows, q = n: A = W_e MN-major, B = dy K-major
//   weight gradient: c = k, r = n, q = rows: A = x MN-major,   B = dy MN-major
// (a TMA box of 64 contiguous elements x 64 rows lands in shared memory as an
// MN-major tile as it is; nothing is transposed).
//
// Structure: CG CTAs (1, or a cluster of 2) work on one tile of 128 * CG c's
// x NB r's at a time, persistently, tile indices handed out round-robin over
// a list that every CTA derives from `off` by itself (no workspace, nothing
// shared between calls).
//   warp 0    issues the TMA loads into a ring of stages;
//   warp 1    (of the pair's rank 0) issues the tcgen05.mma;
//   warp 2    weight gradient: zeroes the rows of a group's last k-block that
//             belong to the next group, in shared memory;
//   warps 4-11 read the accumulators from TMEM and store them, while the MMA
//             warp fills the other accumulator.
// In a pair each CTA loads its 128 c's of A and half of the r's of B, and
// reads its half of the accumulator: 64 bytes of shared-memory fill per cycle
// at the tensor cores' full rate instead of 96 for one CTA with the same NB.
// Every wait is bounded; a timeout sets a status bit and the CTA winds down.
//
// What bounds it and what it reaches (sustained, H = 2688, I = 1856, 128 experts;
// the range over several B200s): few rows a group, the weights' stream: 8 tokens 64
// to 69 us, 48 rows a group 204 to 221 us (6.5 to 6.0 TB/s); many, the tensor cores
// under the 1000 W cap: dense 8192 x 4096 x 4096 194 us (1417 TFLOP/s; in a burst
// 172 us).  384 rows a group on average but 7300 on the hottest, 504 to 563 us (970
// to 870 TFLOP/s): light groups stream weights and heavy ones compute, one after the
// other.  Even groups of 130 to 500 rows take 1.3 to 1.5 times the larger of both,
// DRAM and the tensor cores each busy 60 % of the time; which role waits there has not
// been measured.  Weight gradients of few rows, the writes: 48 rows a group 247 to
// 268 us (5.4 to 5.0 TB/s; plain stores of zeros to the same 1.28 GB take 320), 256
// rows in FP32 325 to 343 us.
#include <cuda_fp16.h>

#include <climits>

#include "handle_free.h"
#include "moe_internal.h"
#include "ptx_pair.cuh"

namespace moe {
namespace {

enum Mode : int { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int kThreads = 384;
constexpr int kEpiWarps = 8;
static_assert(kThreads >= MOE_MAX_EXPERTS, "one thread per group derives the tile list");
constexpr int kBK = 64;        // elements of q per k-block (128 bytes)

struct GroupedArgs {
  CUtensorMap tmA;     // forward: 128-row boxes; else 64-row boxes
  // K-major: boxes of 16, 32, 64 and 128 rows; weight gradient: [0] of 64, [1]
  // and [2] of 1 and 4, for zeros
  CUtensorMap tmB[4];
  CUtensorMap tmO;     // weight gradient with `tma_out`: a round's 32 or 64 r's x 32 c's of the output
  const int* off;
  int groups;
  int rows;  // rows of the row tensors: no group may end behind it
  int C;     // extent of c
  int Q;     // extent of q (forward, data gradient)
  int R;     // extent of r (weight gradient)
  void* out;
  long long ldo;           // elements
  long long group_stride;  // elements (weight gradient)
  uint32_t fmt;            // 0 = FP16, 1 = BF16
  int relu2;
  int accumulate;  // out += (FP32 only)
  int tma_out;     // weight gradient: whole chunks leave by TMA
  int vec;         // 16-byte stores: base, ldo and group_stride allow them
  int* status;
};

template <Mode M, int CG, int NB, int KPS, int STAGES, int EB>
struct Traits {
  static constexpr bool kAMN = M != kFwd;
  static constexpr bool kBMN = M == kWgrad;
  static constexpr int kABytes = 128 * 128;          // one k-block of A in one CTA
  static constexpr int kBBytes = NB / CG * 128;      // one k-block of B in one CTA
  static constexpr int kStageBytes = KPS * (kABytes + kBBytes);
  static constexpr int kTileC = 128 * CG;
  static constexpr int kTmemCols = 2 * NB;
  static constexpr int kChunk = 32 * 32 * EB;  // 32 r's x 32 c's of the epilogue
  // chunks a warp stores at a time: each round waits for its staging tile,
  // fences it and issues one copy, 340 cycles of a chunk's 620
  static constexpr int kRound = M == kWgrad && EB == 2 ? 2 : 1;
  static constexpr int kWarpStaging = kRound * kChunk;
  static constexpr int kStagingBytes = kEpiWarps * kWarpStaging;
  // The tensor cores truncate as they accumulate: a sum of q products loses about
  // q * 1e-9 of itself, where all have one sign q * 6e-9 (measured: 9e-6 and 5e-5 at
  // 8192; in one piece 2^20 products 1.2e-3 and 6.9e-3, more than an FP16 rounding).
  // So sums start anew every 128 k-blocks, 8192 products, and the pieces are added up,
  // rounding to nearest, in TMEM: the epilogue adds the sum so far to the next piece
  // before it hands the accumulator back.  For an FP32 result they start anew every
  // 768 rows (7e-7 and 4e-6): two are joined in the epilogue, which takes both
  // accumulators then, and every two sums in memory.  (128 groups of 780 rows, 1024 x
  // 2688: 819 us with each added up in memory, 694 with pairs.)
  static constexpr int kSegment = EB == 4 ? 12 : 128;  // k-blocks
  // Weight gradient: a group's last k-block is loaded this many k-blocks ahead of
  // its turn, in which time the rows behind the group's last one are cleared
  // (128 groups of 500 / 333 / 261 / 135 rows, 2688 x 1856, us: 0 ahead 725 / 553
  // / 497 / 346, 1 ahead 688 / 533 / 492 / 340, 2 ahead 709 / 538 / 481 / 351, 3
  // ahead 741 / 572 / 493 / 346).
  static constexpr int kAhead = 1;
  static_assert(M != kWgrad || kAhead < STAGES, "");
  // behind the stages and the staging tiles: barriers, the groups' bounds, row
  // tiles before each group, a scan's sums
  static constexpr int kBarriers = (3 * STAGES + 7) * 8;
  static constexpr int kSmem = STAGES * kStageBytes + kStagingBytes + kBarriers +
                               (2 * (MOE_MAX_EXPERTS + 1) + kThreads / 32) * 4;
  static_assert(kSegment % KPS == 0, "");
  static_assert(!kBMN || KPS == 1, "the tail of a group is one k-block of one stage");
  static_assert(kTmemCols >= 32 && (kTmemCols & (kTmemCols - 1)) == 0 && kTmemCols <= 512, "");
  static_assert(kSmem <= 232448, "");
};

// Weight gradient: place in the order of a tile's loads of the k-block that has
// rows to clear (nk: there is none).  The others keep their order.
template <typename Tr>
__device__ __forceinline__ int tail_place(int nk, int cnt) {
  if ((cnt & 15) == 0) return nk;  // whole steps of 16 rows
  return max(nk - 1 - Tr::kAhead, (nk - 1) / Tr::kSegment * Tr::kSegment);
}

struct GTile {
  int e;
  int row0;  // forward, data gradient: first row; weight gradient: first q row
  int cnt;   // rows of the group
  int r0;    // first r of the tile, inside the group
  int nr;    // r's of the tile
  int c0;    // first c of the tile
  int nk;    // k-blocks
};

// The tiles of one CTA (pair), in order.  Tile number u of the launch is c tile
// u % ct of row tile u / ct, row tiles counted over all groups (pre[e] = row
// tiles of the groups before e); CTA (pair) i takes the tiles i, i + step, ...
// The quotient and the remainder are carried along, so that the next tile
// costs a few additions (with a division, and the group's bounds read again,
// the roles spent 1400 cycles a tile on it, more than on a tile of one k-block).
template <Mode M, int TILE_C, int NB>
struct Walk {
  int ct, step_q, step_r;
  int q, r;         // row tile and c tile of the next tile
  int e = 0, lo = 0, hi;  // current group and its row tiles
  GTile t;

  __device__ __forceinline__ Walk(const GroupedArgs& p, const int* off, const int* pre, int first,
                                  int step)
      : ct((p.C + TILE_C - 1) / TILE_C), step_q(step / ct), step_r(step % ct), q(first / ct),
        r(first % ct), hi(pre[1]) {
    group(p, off, 0);
  }

  __device__ __forceinline__ void group(const GroupedArgs& p, const int* off, int g) {
    t.e = g;
    t.row0 = off[g];
    t.cnt = off[g + 1] - t.row0;
    t.nk = ((M == kWgrad ? t.cnt : p.Q) + kBK - 1) / kBK;
  }

  __device__ __forceinline__ bool next(const GroupedArgs& p, const int* off, const int* pre) {
    if (q >= hi) {
      do {
        if (++e >= p.groups) return false;
        lo = hi;
        hi = pre[e + 1];
      } while (q >= hi);
      group(p, off, e);
    }
    t.c0 = r * TILE_C;
    t.r0 = (q - lo) * NB;
    t.nr = min(NB, (M == kWgrad ? p.R : t.cnt) - t.r0);
    q += step_q;
    r += step_r;
    if (r >= ct) {
      r -= ct;
      ++q;
    }
    return true;
  }
};

__device__ __forceinline__ void give_up(const GroupedArgs& p, volatile int* abort) {
  *abort = 1;
  if (p.status) atomicOr(p.status, kStatusWaitTimeout);
}

// mbar_wait for a warp whose turn may be many tiles away: the limit holds for
// the time in which *begun, the count of tiles begun, stands still.
__device__ __forceinline__ bool mbar_wait_turn(uint64_t* bar, uint32_t parity, volatile int* begun,
                                               volatile int* abort) {
  int seen = *begun;
  long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (*abort) return false;
    const int now = *begun;
    if (now != seen) {
      seen = now;
      t0 = clock64();
    }
    if (clock64() - t0 > kWaitLimitCycles) return false;
  }
  return true;
}

// N TMEM columns from `base + to` on, in this warp's lanes: plus those from `base +
// from` on.
template <int N>
__device__ __noinline__ void add_columns(uint32_t base, uint32_t from, uint32_t to) {
#pragma unroll 1
  for (int j = 0; j < N; j += 16) {
    uint32_t s[2][16];
    tmem_ld_32x32b_x16(base + from + uint32_t(j), s[0]);
    tmem_ld_32x32b_x16(base + to + uint32_t(j), s[1]);
    tmem_ld_wait_regs(s);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      s[1][i] = __float_as_uint(__uint_as_float(s[0][i]) + __uint_as_float(s[1][i]));
    tmem_st_32x32b_x16(base + to + uint32_t(j), s[1]);
  }
  tmem_st_wait();
}

__device__ __forceinline__ float relu2(float v) {
  return v <= 0.f ? 0.f : v * v;  // NaN stays NaN
}

__device__ __forceinline__ uint32_t pack_16(uint32_t lo, uint32_t hi, bool bf16) {
  const float a = __uint_as_float(lo), b = __uint_as_float(hi);
  if (bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of the 16-byte block (8 c's) `b` of row r in a warp's 32 x 32
// staging tile of 16-bit elements: 64 bytes a row, blocks permuted so that
// neither stmatrix (8 rows of one block) nor the row-wise reads conflict.
__device__ __forceinline__ uint32_t staging_at(uint32_t r, uint32_t b) {
  return r * 64 + ((b ^ ((r >> 1) & 3)) * 16);
}

// A chunk of 32 r's (TMEM columns) x 32 c's (this warp's TMEM lanes), to an
// output of 16-bit elements.  The accumulators come as fragments of 8 x 8
// matrices (c x r); two neighbouring r's are rounded into one register, and a
// transposing stmatrix leaves rows of 32 c's in shared memory, which go out
// as 16-byte stores.  (With one 2-byte store per element and lane into the
// staging tile, by four warps, a weight gradient of 48 rows a group took 655
// us; this, by eight, 317.)
__device__ __forceinline__ void stage_chunk_16(const GroupedArgs& p, uint32_t (&lo)[16],
                                               uint32_t (&hi)[16], uint32_t staging) {
  const uint32_t lane = threadIdx.x & 31;
  if (p.relu2) {
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      lo[j] = __float_as_uint(relu2(__uint_as_float(lo[j])));
      hi[j] = __float_as_uint(relu2(__uint_as_float(hi[j])));
    }
  }
  uint32_t m[2][8];
  if (p.fmt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[0][j] = pack_16(lo[2 * j], lo[2 * j + 1], true);
      m[1][j] = pack_16(hi[2 * j], hi[2 * j + 1], true);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[0][j] = pack_16(lo[2 * j], lo[2 * j + 1], false);
      m[1][j] = pack_16(hi[2 * j], hi[2 * j + 1], false);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    stmatrix_x4_trans(staging + staging_at(8 * i + (lane & 7), lane >> 3), m[0][2 * i],
                      m[0][2 * i + 1], m[1][2 * i], m[1][2 * i + 1]);
}

// A staged chunk to the output, its first n rows.
__device__ __forceinline__ void store_chunk_16(const GroupedArgs& p, uint32_t staging, uint16_t* o,
                                               int cw, int n) {
  const uint32_t lane = threadIdx.x & 31;
  if (p.vec && cw + 32 <= p.C) {
    const uint32_t b = lane & 3;
    uint16_t* dst = o + (long long)(lane >> 2) * p.ldo + cw + b * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = 8 * i + (lane >> 2);
      uint4 u;
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                   : "r"(staging + staging_at(r, b)));
      if (int(r) < n) *reinterpret_cast<uint4*>(dst + 8LL * i * p.ldo) = u;
    }
  } else {
    const bool cvalid = cw + int(lane) < p.C;
#pragma unroll 4
    for (int r = 0; r < 32; ++r) {
      uint16_t u;
      asm volatile("ld.shared.u16 %0, [%1];"
                   : "=h"(u)
                   : "r"(staging + staging_at(r, lane >> 3) + (lane & 7) * 2));
      if (r < n && cvalid) o[(long long)r * p.ldo + cw + lane] = u;
    }
  }
}

// An FP32 chunk (lane = c): staged as 128-byte rows with the 16-byte blocks
// permuted as the TMA store's 128-byte swizzle has them.
__device__ __forceinline__ void stage_chunk_32(const uint32_t (&acc)[32], uint32_t staging) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (uint32_t r = 0; r < 32; ++r)
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(staging + r * 128 +
                                                 (((lane >> 2) ^ (r & 7)) * 16) + (lane & 3) * 4),
                 "r"(acc[r])
                 : "memory");
}

// The same without staging: a warp's store of one r is 128 contiguous bytes.
// (add: the elements are this lane's alone, in every segment of a sum.)
__device__ __forceinline__ void store_chunk_32(const GroupedArgs& p, const uint32_t (&acc)[32],
                                               float* o, int n, bool add) {
  if (add) {
    float old[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) old[j] = j < n ? o[j * p.ldo] : 0.f;
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) o[j * p.ldo] = old[j] + __uint_as_float(acc[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (j < n) o[j * p.ldo] = __uint_as_float(acc[j]);
  }
}

template <Mode M, int CG, int NB, int KPS, int STAGES, int EB>
__global__ void __launch_bounds__(kThreads, 1)
    ragged_gemm_kernel(const __grid_constant__ GroupedArgs p) {
  using Tr = Traits<M, CG, NB, KPS, STAGES, EB>;
  extern __shared__ __align__(1024) uint8_t tiles[];
  uint8_t* staging = tiles + STAGES * Tr::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + Tr::kStagingBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* tail = empty + STAGES;
  uint64_t* tfull = tail + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* begun = abort + 1;  // tiles the producer has begun
  static_assert(Tr::kBarriers == (3 * STAGES + 5) * 8 + 16, "");
  int* s_off = reinterpret_cast<int*>(full) + Tr::kBarriers / 4;  // groups' bounds
  int* s_pre = s_off + MOE_MAX_EXPERTS + 1;
  int* s_scan = s_pre + MOE_MAX_EXPERTS + 1;

  const int warp = uniform(int(threadIdx.x >> 5));
  const int lane = threadIdx.x & 31;
  const uint32_t rank = CG == 2 ? cluster_rank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], CG);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], kEpiWarps * CG);
    }
    mbar_init(drain, 1);
    *abort = 0;
    *begun = 0;
    fence_barrier_init();
    tma_prefetch_desc(&p.tmA);
    tma_prefetch_desc(&p.tmB[0]);
  }
  if (warp == 1) tmem_alloc_cg<CG>(tmem_slot, Tr::kTmemCols);
  // (programmatic dependent launch: the above overlaps the kernel before)
  pdl_wait();
  pdl_trigger();

  // the work list: row tiles of each group, prefix sums
  {
    const int e = threadIdx.x;
    int n = 0;
    bool bad = false;
    if (e < p.groups) {
      const int a = p.off[e], b = p.off[e + 1];
      const bool good = a >= 0 && a <= b && b <= p.rows;
      if (!good && p.status && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
      bad = !good;
      const int cnt = good ? b - a : 0;
      s_off[e] = a;
      if (e + 1 == p.groups) s_off[p.groups] = b;
      n = ((M == kWgrad ? p.R : cnt) + NB - 1) / NB;
      if (M == kWgrad && cnt == 0 && p.accumulate) n = 0;  // nothing to add
      if (M == kWgrad && !good) n = 0;  // a bad group's gradient is left as it was
    }
    // inclusive sums: within each warp, then over the warps
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int up = __shfl_up_sync(0xffffffffu, n, d);
      if (lane >= d) n += up;
    }
    // (the sign says that the warp has met a bad entry)
    const bool met = M != kWgrad && __any_sync(0xffffffffu, bad);
    if (lane == 31) s_scan[warp] = met ? n | INT_MIN : n;
    __syncthreads();
    bool fell = met;
    for (int i = 0; i < warp; ++i) {
      n += s_scan[i] & INT_MAX;
      fell |= M != kWgrad && s_scan[i] < 0;
    }
    // Where `off` falls, a group may begin below the end of one before it.  The
    // rows they share have one owner, the first: the later group counts as empty.
    // (A weight gradient's groups share no output.)  Threads whose own group or
    // one before it is bad add up again, each by itself; a barrier that carries
    // the flag cost every launch 0.2 us.
    if (fell && e < p.groups) {
      n = 0;
      for (int i = 0, top = 0; i <= e; ++i) {
        const int a = s_off[i], b = s_off[i + 1];
        if (a >= top && a <= b && b <= p.rows) n += (b - a + NB - 1) / NB;
        if (a <= p.rows) top = max(top, a);
      }
    }
    if (e == 0) s_pre[0] = 0;
    if (e < p.groups) s_pre[e + 1] = n;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (CG == 2) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  Walk<M, Tr::kTileC, NB> walk(p, s_off, s_pre, int(blockIdx.x) / CG, int(gridDim.x) / CG);
  const uint32_t tiles_u32 = smem_u32(tiles);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int it = 1; ok && uniform(walk.next(p, s_off, s_pre)); ++it) {
      if (M == kWgrad && lane == 0) *begun = it;
      const int nk = uniform(walk.t.nk), nr = uniform(walk.t.nr), cnt = uniform(walk.t.cnt);
      const int e = uniform(walk.t.e), row0 = uniform(walk.t.row0), r0 = uniform(walk.t.r0);
      const int nmma = (nr + 15) & ~15;
      const int nb = nmma / CG;  // r's of B this CTA loads
      const int ca = uniform(walk.t.c0) + int(rank) * 128;
      const int rb = r0 + int(rank) * nb;
      // B of one k-block: one K-major box of 16, 32, 64 or 128 rows (several
      // smaller ones cost more than the rows they save), or MN-major boxes
      // of 64
      int nbox = 1, size = 0;
      uint32_t bbytes;
      if (Tr::kBMN) {
        nbox = (nb + 63) / 64;
        bbytes = nbox * 64 * 128;
      } else {
        size = nb <= 16 ? 0 : nb <= 32 ? 1 : nb <= 64 ? 2 : 3;
        bbytes = 2048u << size;
      }
      const int place = M == kWgrad ? tail_place<Tr>(nk, cnt) : nk;
      for (int kb0 = 0; kb0 < nk; kb0 += KPS) {
        ok = uniform(mbar_wait(&empty[stage], phase ^ 1u, abort));
        if (!ok) break;
        const int kbn = min(KPS, nk - kb0);
        const uint32_t bytes = uint32_t(kbn) * (Tr::kABytes + bbytes);
        const bool is_tail = M == kWgrad && kb0 == place;
        const int first = M != kWgrad || kb0 < place ? kb0 : is_tail ? nk - 1 : kb0 - 1;
        const uint32_t st = tiles_u32 + stage * Tr::kStageBytes;
        if (elect_one()) {
          uint32_t bar;
          if (is_tail) {
            mbar_arrive_expect_tx(&tail[stage], bytes);
            bar = smem_u32(&tail[stage]);
          } else if (CG == 2) {
            bar = map_to_rank(smem_u32(&full[stage]), 0);
            mbar_arrive_expect_tx_at(bar, bytes);
          } else {
            mbar_arrive_expect_tx(&full[stage], bytes);
            bar = smem_u32(&full[stage]);
          }
#pragma unroll
          for (int kk = 0; kk < KPS; ++kk) {
            if (kk >= kbn) break;
            const int q = (first + kk) * kBK;
            const uint32_t sa = st + kk * (Tr::kABytes + Tr::kBBytes), sb = sa + Tr::kABytes;
            if constexpr (M == kFwd) {
              tma_load_3d<CG>(sa, &p.tmA, bar, q, ca, e);
            } else {
              const int y = M == kDgrad ? q : row0 + q;
              const int z = M == kDgrad ? e : 0;
              tma_load_3d<CG>(sa, &p.tmA, bar, ca, y, z);
              tma_load_3d<CG>(sa + 8192, &p.tmA, bar, ca + 64, y, z);
            }
            if constexpr (M == kWgrad) {
              for (int h = 0; h < nbox; ++h)
                tma_load_3d<CG>(sb + h * 8192, &p.tmB[0], bar, rb + h * 64, row0 + q, 0);
            } else {
              tma_load_3d<CG>(sb, &p.tmB[size], bar, q, row0 + rb, 0);
            }
          }
        }
        __syncwarp();
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      if (lane == 0) give_up(p, abort);
      const long long t0 = clock64();  // let the copies in flight land before the CTA may exit
      while (clock64() - t0 < 4000000) {
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    // The whole warp walks the tiles with warp-uniform values and one lane
    // issues: from a single lane's divergent branch each tcgen05.mma took
    // about 180 cycles to issue, more than the 128 of its 256 x 256 x 16
    // product.
    if (rank == 0) {
      int stage = 0, it = 0, tail_stage = 0;
      uint32_t phase = 0, tail_phase = 0;
      bool ok = true;
      const auto advance = [&] {
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      };
      while (ok && uniform(walk.next(p, s_off, s_pre))) {
        const int nk = uniform(walk.t.nk), nr = uniform(walk.t.nr), cnt = uniform(walk.t.cnt);
        if (nk == 0) continue;
        const int place = M == kWgrad ? tail_place<Tr>(nk, cnt) : nk;
        const uint32_t idesc = make_idesc_16(128 * CG, (nr + 15) & ~15, p.fmt, Tr::kAMN, Tr::kBMN);
        const int last = (cnt - (nk - 1) * kBK + 15) / 16;  // weight gradient: steps with rows
        for (int seg = 0; seg < nk && ok; seg += Tr::kSegment) {
          const int end = Tr::kSegment < nk - seg ? seg + Tr::kSegment : nk;
          const int ab = it & 1;
          ok = uniform(mbar_wait(&tempty[ab], ((it >> 1) & 1) ^ 1u, abort));
          if (!ok) break;
          ++it;
          tc_fence_after();
          const uint32_t d = tmem_base + uint32_t(ab * NB);
          for (int kb0 = seg; kb0 < end; kb0 += KPS) {
            // a group's last k-block with rows to clear
            const bool is_tail = M == kWgrad && place < nk && kb0 + 1 == nk;
            if (M == kWgrad && kb0 == place) {  // its stage; its turn comes last
              tail_stage = stage;
              tail_phase = phase;
              advance();
            }
            const int at = is_tail ? tail_stage : stage;
            ok = uniform(mbar_wait(&full[at], is_tail ? tail_phase : phase, abort));
            if (!ok) break;
            tc_fence_after();
            const int kbn = min(KPS, nk - kb0);
            const uint32_t sa0 = tiles_u32 + at * Tr::kStageBytes;
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < KPS; ++kk) {
                if (kk >= kbn) break;
                const uint32_t sa = sa0 + kk * (Tr::kABytes + Tr::kBBytes), sb = sa + Tr::kABytes;
                const uint64_t ad =
                    Tr::kAMN ? smem_desc_mn_sw128(sa, 8192) : smem_desc_k_sw128(sa);
                const uint64_t bd =
                    Tr::kBMN ? smem_desc_mn_sw128(sb, 8192) : smem_desc_k_sw128(sb);
                const int ks = M == kWgrad && kb0 + 1 == nk ? last : kBK / 16;
#pragma unroll
                for (int s = 0; s < kBK / 16; ++s)
                  if (M != kWgrad || s < ks)
                    umma_f16_cg<CG>(d, ad + s * (Tr::kAMN ? 128 : 2),
                                    bd + s * (Tr::kBMN ? 128 : 2), idesc,
                                    (kb0 - seg) | kk | s ? 1u : 0u);
              }
              umma_commit_cg<CG>(&empty[at]);
            }
            __syncwarp();
            if (!is_tail) advance();
          }
          if (ok && elect_one()) umma_commit_cg<CG>(&tfull[ab]);
          __syncwarp();
        }
      }
      if (!ok && lane == 0) give_up(p, abort);
      // every MMA issued has completed once `drain` flips (in both CTAs)
      if (elect_one()) umma_commit_cg<CG>(drain);
      __syncwarp();
      int zero = 0;
      mbar_wait(drain, 0, &zero);
    }
  } else if (M == kWgrad && warp == 2) {
    // ---------------------------------------- rows behind a group's last one
    // Cleared by copies of boxes that lie behind the tensor's last row, which
    // TMA fills with zeros: they complete on the MMA's barrier like the loads
    // before them.  (Plain stores have to be released to the pair's other CTA,
    // about a microsecond a tail: 48 rows a group 259 us, this 245; 500 rows
    // 773 and 680.)
    // The tile it waits for may come after many that it has nothing to do with,
    // longer than a wait's limit (the other roles wait for one tile at most).
    int total = 0;
    uint32_t used = 0;  // phase bit of each barrier
    while (uniform(walk.next(p, s_off, s_pre))) {
      const int nk = uniform(walk.t.nk), cnt = uniform(walk.t.cnt);
      const int place = tail_place<Tr>(nk, cnt);
      const int stage = (total + place) % STAGES;
      total += nk;
      if (place == nk) continue;
      if (!uniform(mbar_wait_turn(&tail[stage], (used >> stage) & 1u, begun, abort))) {
        if (lane == 0) give_up(p, abort);
        break;
      }
      used ^= 1u << stage;
      const int nb = ((uniform(walk.t.nr) + 15) & ~15) / CG;
      const int blocks = 2 + (nb + 63) / 64;
      const int valid = cnt & (kBK - 1), n = -valid & 15;  // rows to clear
      if (elect_one()) {
        uint32_t bar = smem_u32(&full[stage]);
        if (CG == 2) {
          bar = map_to_rank(bar, 0);
          mbar_arrive_expect_tx_at(bar, uint32_t(blocks * n) * 128);
        } else {
          mbar_arrive_expect_tx(&full[stage], uint32_t(blocks * n) * 128);
        }
        for (int h = 0; h < blocks; ++h) {
          uint32_t dst = tiles_u32 + stage * Tr::kStageBytes + h * 8192 + valid * 128;
          for (int r = 0; r < n;) {
            const int size = n - r >= 4 ? 2 : 1;
            tma_load_3d<CG>(dst, &p.tmB[size], bar, 0, p.rows, 0);
            r += size == 2 ? 4 : 1;
            dst += size == 2 ? 512 : 128;
          }
        }
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int half = (warp - 4) >> 2;  // chunks of 32 r's: even or odd ones
    const uint32_t st = smem_u32(staging) + (warp - 4) * Tr::kWarpStaging;
    int it = 0;
    bool ok = true;
    while (ok && uniform(walk.next(p, s_off, s_pre))) {
      const int nk = uniform(walk.t.nk), nr = uniform(walk.t.nr), r0 = uniform(walk.t.r0);
      const int e = uniform(walk.t.e);
      const int cw = uniform(walk.t.c0) + int(rank) * 128 + q * 32;
      const long long row = M == kWgrad ? r0 : (long long)(uniform(walk.t.row0)) + r0;
      const long long base = (M == kWgrad ? e * p.group_stride : 0) + row * p.ldo;
      for (int seg = 0; seg == 0 || (EB == 4 && seg < nk && ok); seg += 2 * Tr::kSegment) {
        int ab = it & 1;
        const bool two = EB == 4 && nk - seg > Tr::kSegment;  // sums to join
        if (nk > 0) {
          ok = uniform(mbar_wait(&tfull[ab], (it >> 1) & 1, abort));
          ++it;
          if (two && ok) {
            ok = uniform(mbar_wait(&tfull[ab ^ 1], (it >> 1) & 1, abort));
            ++it;
          }
          if (EB == 2) {
            // the pieces of a long sum: each takes in the sum before it
            for (int done = Tr::kSegment; done < nk && ok; done += Tr::kSegment) {
              ok = uniform(mbar_wait(&tfull[ab ^ 1], (it >> 1) & 1, abort));
              ++it;
              if (!ok) break;
              tc_fence_after();
              if (cw < p.C)
                for (int j0 = half * 32 * Tr::kRound; j0 < nr; j0 += 64 * Tr::kRound)
                  add_columns<32 * Tr::kRound>(tmem_base + (uint32_t(q * 32) << 16) + uint32_t(j0),
                                               uint32_t(ab * NB), uint32_t((ab ^ 1) * NB));
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                if (CG == 2)
                  mbar_arrive_at(map_to_rank(smem_u32(&tempty[ab]), 0));
                else
                  mbar_arrive(&tempty[ab]);
              }
              ab ^= 1;
            }
          }
          if (!ok) {
            if (lane == 0) give_up(p, abort);
            break;
          }
          tc_fence_after();
        }
        const uint32_t tb = tmem_base + (uint32_t(q * 32) << 16) + uint32_t(ab * NB);
        const bool mine = cw < p.C;  // the warp has c's to store
        const bool bulk = M == kWgrad && p.tma_out;
        const bool add = EB == 4 && (p.accumulate || seg > 0);
        if (EB == 4 && bulk && seg > 0) {  // the sums before are in memory
          if (elect_one()) bulk_wait_all();
          __syncwarp();
        }
#pragma unroll 1
        for (int j0 = half * 32 * Tr::kRound; j0 < nr && mine; j0 += 64 * Tr::kRound) {
          // the bulk store of the round before has read the staging tile
          if (bulk) {
            if (elect_one()) bulk_wait_read<0>();
            __syncwarp();
          }
          if constexpr (EB == 4) {
            uint32_t r[32];
            if (two) {
              const uint32_t tb2 = tmem_base + (uint32_t(q * 32) << 16) + uint32_t((ab ^ 1) * NB);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t s[2][16];
                tmem_ld_32x32b_x16(tb + uint32_t(j0 + 16 * h), s[0]);
                tmem_ld_32x32b_x16(tb2 + uint32_t(j0 + 16 * h), s[1]);
                tmem_ld_wait_regs(s);
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  r[16 * h + j] =
                      __float_as_uint(__uint_as_float(s[0][j]) + __uint_as_float(s[1][j]));
              }
            } else if (nk > 0) {
              tmem_ld_32x32b_x32(tb + uint32_t(j0), r);
              tmem_ld_wait();
            } else {  // an empty group's gradient
#pragma unroll
              for (int j = 0; j < 32; ++j) r[j] = 0u;
            }
            if (bulk)
              stage_chunk_32(r, st);
            else if (cw + lane < p.C)
              store_chunk_32(p, r, static_cast<float*>(p.out) + base + j0 * p.ldo + cw + lane,
                             nr - j0, add);
          } else {
            uint32_t r[2 * Tr::kRound][16];
            if (nk > 0) {
#pragma unroll
              for (int c = 0; c < Tr::kRound; ++c) {
                tmem_ld_16x256b_x4(tb + uint32_t(j0 + 32 * c), r[2 * c]);
                tmem_ld_16x256b_x4(tb + (16u << 16) + uint32_t(j0 + 32 * c), r[2 * c + 1]);
              }
              tmem_ld_wait_regs(r);
            } else {
#pragma unroll
              for (int c = 0; c < 2 * Tr::kRound; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) r[c][j] = 0u;
            }
#pragma unroll
            for (int c = 0; c < Tr::kRound; ++c)
              stage_chunk_16(p, r[2 * c], r[2 * c + 1], st + c * Tr::kChunk);
            if (!bulk) {
              __syncwarp();
#pragma unroll
              for (int c = 0; c < Tr::kRound; ++c)
                store_chunk_16(p, st + c * Tr::kChunk,
                               static_cast<uint16_t*>(p.out) + base + (j0 + 32 * c) * p.ldo, cw,
                               nr - j0 - 32 * c);
              __syncwarp();
            }
          }
          if (bulk) {
            fence_proxy_async_smem();
            __syncwarp();
            if (elect_one()) {
              if (add)
                tma_add_3d(&p.tmO, st, cw, r0 + j0, e);
              else
                tma_store_3d(&p.tmO, st, cw, r0 + j0, e);
              bulk_commit();
            }
          }
        }
        if (nk > 0) {
          tc_fence_before();
          __syncwarp();
          if (lane < 1 + two) {
            if (CG == 2)
              mbar_arrive_at(map_to_rank(smem_u32(&tempty[ab ^ lane]), 0));
            else
              mbar_arrive(&tempty[ab ^ lane]);
          }
        }
      }
    }
    if (M == kWgrad && elect_one()) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  __syncwarp();
  if constexpr (CG == 2) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_cg<CG>(tmem_base, Tr::kTmemCols);
  }
  if constexpr (CG == 2) {
    __syncwarp();
    cluster_sync();
  }
}

template <Mode M, int CG, int NB, int KPS, int STAGES, int EB>
struct Variant {
  using Tr = Traits<M, CG, NB, KPS, STAGES, EB>;

  // On the current device, before the first launch: loads the kernel, too.
  static cudaError_t set_up() {
    return cudaFuncSetAttribute(ragged_gemm_kernel<M, CG, NB, KPS, STAGES, EB>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, Tr::kSmem);
  }

  static cudaError_t launch(const GroupedArgs& a, int sms, long long max_tiles,
                            cudaStream_t stream) {
    const int units = sms / CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(CG * (max_tiles < units ? max_tiles : units)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Tr::kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, ragged_gemm_kernel<M, CG, NB, KPS, STAGES, EB>, a);
  }

  // Tiles of `groups` groups with `rows` rows in all, at most.
  static long long tiles_of(const GroupedArgs& a) {
    const long long ct = (a.C + Tr::kTileC - 1) / Tr::kTileC;
    if (M == kWgrad) return a.groups * ct * ((a.R + NB - 1) / NB);
    return ct * (a.rows / NB + (a.groups < a.rows ? a.groups : a.rows));
  }
};

struct Operand {
  const void* base;
  long long ld;  // elements
  int inner, rows, groups;
};

bool map_of(CUtensorMap* m, const Operand& o, uint32_t fmt, int box_rows, bool swizzle = true) {
  return make_map_3d(m, fmt ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                     o.base, uint64_t(o.inner), uint64_t(o.rows), uint64_t(o.groups),
                     uint64_t(o.ld) * 2, uint64_t(o.ld) * 2 * uint64_t(o.groups > 1 ? o.rows : 1),
                     uint32_t(box_rows), 128, swizzle);
}

template <Mode M, int CG, int NB, int KPS, int STAGES, int EB>
moe_status run_variant(GroupedArgs& a, const Operand& A, const Operand& B, int sms,
                       cudaStream_t stream) {
  using V = Variant<M, CG, NB, KPS, STAGES, EB>;
  bool ok = map_of(&a.tmA, A, a.fmt, M == kFwd ? 128 : 64);
  if (M == kWgrad)
    // and boxes of zeros: 1 and 4 rows
    ok = ok && map_of(&a.tmB[0], B, a.fmt, 64) && map_of(&a.tmB[1], A, a.fmt, 1, false) &&
         map_of(&a.tmB[2], A, a.fmt, 4, false);
  else
    for (int i = 0; i < 4 && (16 << i) <= NB / CG; ++i)
      ok = ok && map_of(&a.tmB[i], B, a.fmt, 16 << i);
  if (M == kWgrad && a.tma_out)
    ok = ok && make_map_3d(&a.tmO,
                           EB == 4  ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                           : a.fmt  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                           EB, a.out, uint64_t(a.C), uint64_t(a.R), uint64_t(a.groups),
                           uint64_t(a.ldo) * EB, uint64_t(a.group_stride) * EB, 32 * V::Tr::kRound,
                           32 * EB);
  if (!ok) return MOE_ERR_CUDA;
  if (V::launch(a, sms, V::tiles_of(a), stream) != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// All of an operator's variants, so that a call whose sizes take another one than
// the first call's finds it ready (inside a stream capture, say).
template <Mode M>
cudaError_t set_up_variants() {
  const auto all = [](auto... v) {
    cudaError_t e = cudaSuccess;
    ((e = e != cudaSuccess ? e : decltype(v)::set_up()), ...);
    return e;
  };
  if constexpr (M == kWgrad)
    return all(Variant<M, 1, 128, 1, 6, 4>(), Variant<M, 2, 256, 1, 6, 4>(),
               Variant<M, 1, 128, 1, 6, 2>(), Variant<M, 2, 256, 1, 6, 2>());
  else
    return all(Variant<M, 1, 64, 2, 4, 2>(), Variant<M, 2, 128, 1, 8, 2>(),
               Variant<M, 2, 256, 1, 6, 2>());
}

// Rules every operand keeps: a leading dimension that covers the row, in
// 16-byte steps (a TMA stride), and a 16-byte aligned base.
moe_status check_sizes(int num_experts, int rows, int K, int N, int dtype) {
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS) return MOE_ERR_INVALID_CONFIG;
  if (K < 1 || K > MOE_GROUPED_MAX_FEATURES || N < 1 || N > MOE_GROUPED_MAX_FEATURES)
    return MOE_ERR_INVALID_CONFIG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_CONFIG;
  if (rows < 0 || rows > MOE_GROUPED_MAX_ROWS) return MOE_ERR_TOKENS_OUT_OF_RANGE;
  return MOE_OK;
}

constexpr int64_t kMaxLd = (int64_t(1) << 22) - 8;  // a group's stride stays below TMA's 2^40 bytes

bool bad_ld(int64_t ld, int width, bool tma) {
  return ld < width || ld > kMaxLd || (tma && (ld & 7));
}

template <Mode M>
moe_status dispatch(GroupedArgs& a, const Operand& A, const Operand& B, bool out_f32,
                    cudaStream_t stream) {
  int dev = 0, sms = 0;
  const moe_status st = current_device(&dev, &sms);
  if (st != MOE_OK) return st;
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (set_up_variants<M>() != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    ready[dev].store(true, std::memory_order_release);
  }
  // Tiles a launch is likely to have: half of the groups end in a part of a
  // row tile.
  const auto tiles = [&](int cg, int nb) {
    const long long ct = (a.C + 128 * cg - 1) / (128 * cg);
    if (M == kWgrad) return a.groups * ct * ((a.R + nb - 1) / nb);
    const int used = a.groups < a.rows ? a.groups : a.rows;
    return ct * (a.rows / nb + (used + 1) / 2);
  };
  if constexpr (M != kWgrad) {
    // The row tile that covers an average group, and a smaller one where the
    // tiles would leave SMs idle.  128 groups of K = 2688, N = 1856, forward,
    // with row tiles of 64 / 128 / 256: 1 row a group 184 / 188 / 195 us, 48
    // 206 / 209 / 216, 64 213 / 214 / 224, 80 282 / 226 / 234, 128 311 / 254 /
    // 260, 160 413 / 338 / 295, 256 553 / 420 / 357.  The mean stands
    // for skewed groups, too: 48 rows on average, the hottest 900, 211 / 207 / 212 us (K =
    // 1856, N = 2688: 226 / 210 / 212); 96 on average, the hottest 1810, 263 / 231 / 235.
    // One group of 2048 rows,
    // K = 1024, N = 512: 6.9 us with 64-row tiles, 11.3 with 256; 8192 rows, N =
    // 1024: 17.6 with 256 (132 tiles for 74 pairs).
    int nb = a.rows <= 64LL * a.groups ? 64 : a.rows <= 128LL * a.groups ? 128 : 256;
    if (nb == 256 && tiles(2, 256) < sms / 2) nb = 128;
    if (nb == 128 && tiles(2, 128) < sms / 2) nb = 64;
    if (nb == 64) return run_variant<M, 1, 64, 2, 4, 2>(a, A, B, sms, stream);
    if (nb == 128) return run_variant<M, 2, 128, 1, 8, 2>(a, A, B, sms, stream);
    return run_variant<M, 2, 256, 1, 6, 2>(a, A, B, sms, stream);
  } else {
    // Small gradients: single CTAs and 128 x 128 tiles, four times as many (one
    // group of 571 rows, K = 856, N = 768: 8.0 us for 10.4; two of 200 rows,
    // 376 x 872: 7.1 for 9.2).
    const bool few = tiles(2, 256) < sms / 2;
    if (out_f32)
      return few ? run_variant<M, 1, 128, 1, 6, 4>(a, A, B, sms, stream)
                 : run_variant<M, 2, 256, 1, 6, 4>(a, A, B, sms, stream);
    return few ? run_variant<M, 1, 128, 1, 6, 2>(a, A, B, sms, stream)
               : run_variant<M, 2, 256, 1, 6, 2>(a, A, B, sms, stream);
  }
}

}  // namespace
}  // namespace moe

using moe::aligned_to;

extern "C" moe_status moe_grouped_gemm(const void* x, int64_t ldx, const void* w, int64_t ldw,
                                       const int32_t* off, int32_t num_experts, int32_t rows,
                                       int32_t in_features, int32_t out_features, int32_t dtype,
                                       int32_t activation, void* y, int64_t ldy, int32_t* status,
                                       void* stream) {
  const moe_status st = moe::check_sizes(num_experts, rows, in_features, out_features, dtype);
  if (st != MOE_OK) return st;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_RELU2) return MOE_ERR_INVALID_CONFIG;
  if (moe::bad_ld(ldx, in_features, true) || moe::bad_ld(ldw, in_features, true) ||
      moe::bad_ld(ldy, out_features, false))
    return MOE_ERR_INVALID_CONFIG;
  if (rows == 0) return MOE_OK;
  if (!x || !w || !off || !y) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(y, 2) || !aligned_to(off, 4) ||
      !aligned_to(status, 4))
    return MOE_ERR_MISALIGNED;
  moe::GroupedArgs a = {};
  a.off = off;
  a.groups = num_experts;
  a.rows = rows;
  a.C = out_features;
  a.Q = in_features;
  a.out = y;
  a.ldo = ldy;
  a.fmt = dtype == MOE_DTYPE_BF16;
  a.relu2 = activation == MOE_ACT_RELU2;
  a.vec = aligned_to(y, 16) && (ldy & 7) == 0;
  a.status = status;
  return moe::dispatch<moe::kFwd>(a, {w, ldw, in_features, out_features, num_experts},
                                  {x, ldx, in_features, rows, 1}, false,
                                  static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_grouped_gemm_dgrad(const void* dy, int64_t lddy, const void* w,
                                             int64_t ldw, const int32_t* off, int32_t num_experts,
                                             int32_t rows, int32_t in_features,
                                             int32_t out_features, int32_t dtype, void* dx,
                                             int64_t lddx, int32_t* status, void* stream) {
  const moe_status st = moe::check_sizes(num_experts, rows, in_features, out_features, dtype);
  if (st != MOE_OK) return st;
  if (moe::bad_ld(lddy, out_features, true) || moe::bad_ld(ldw, in_features, true) ||
      moe::bad_ld(lddx, in_features, false))
    return MOE_ERR_INVALID_CONFIG;
  if (rows == 0) return MOE_OK;
  if (!dy || !w || !off || !dx) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(dy, 16) || !aligned_to(w, 16) || !aligned_to(dx, 2) || !aligned_to(off, 4) ||
      !aligned_to(status, 4))
    return MOE_ERR_MISALIGNED;
  moe::GroupedArgs a = {};
  a.off = off;
  a.groups = num_experts;
  a.rows = rows;
  a.C = in_features;
  a.Q = out_features;
  a.out = dx;
  a.ldo = lddx;
  a.fmt = dtype == MOE_DTYPE_BF16;
  a.vec = aligned_to(dx, 16) && (lddx & 7) == 0;
  a.status = status;
  return moe::dispatch<moe::kDgrad>(a, {w, ldw, in_features, out_features, num_experts},
                                    {dy, lddy, out_features, rows, 1}, false,
                                    static_cast<cudaStream_t>(stream));
}

extern "C" moe_status moe_grouped_gemm_wgrad(const void* dy, int64_t lddy, const void* x,
                                             int64_t ldx, const int32_t* off, int32_t num_experts,
                                             int32_t rows, int32_t in_features,
                                             int32_t out_features, int32_t dtype, void* dw,
                                             int64_t lddw, int32_t out_dtype, int32_t accumulate,
                                             int32_t* status, void* stream) {
  const moe_status st = moe::check_sizes(num_experts, rows, in_features, out_features, dtype);
  if (st != MOE_OK) return st;
  if (out_dtype != dtype && out_dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_CONFIG;
  if (accumulate != 0 && (accumulate != 1 || out_dtype != MOE_DTYPE_F32))
    return MOE_ERR_INVALID_CONFIG;
  if (moe::bad_ld(lddy, out_features, true) || moe::bad_ld(ldx, in_features, true) ||
      moe::bad_ld(lddw, in_features, false))
    return MOE_ERR_INVALID_CONFIG;
  if (!off || !dw || (rows > 0 && (!dy || !x))) return MOE_ERR_NULL_POINTER;
  const bool f32 = out_dtype == MOE_DTYPE_F32;
  if ((rows > 0 && (!aligned_to(dy, 16) || !aligned_to(x, 16))) || !aligned_to(dw, f32 ? 4 : 2) ||
      !aligned_to(off, 4) || !aligned_to(status, 4))
    return MOE_ERR_MISALIGNED;
  moe::GroupedArgs a = {};
  a.off = off;
  a.groups = num_experts;
  a.rows = rows;
  a.C = in_features;
  a.R = out_features;
  a.out = dw;
  a.ldo = lddw;
  a.group_stride = (long long)(out_features)*lddw;
  a.fmt = dtype == MOE_DTYPE_BF16;
  a.accumulate = accumulate;
  a.vec = !f32 && aligned_to(dw, 16) && (lddw & 7) == 0;
  // whole 16-byte blocks, or a store would write to the end of a row's last one,
  // and a group's stride below TMA's 2^40 bytes
  const int block = f32 ? 4 : 8;
  a.tma_out = aligned_to(dw, 16) && in_features % block == 0 && lddw % block == 0 &&
              a.group_stride < (1LL << 37);
  a.status = status;
  // no rows: every group is empty and no map is read through; the maps still
  // want a valid, aligned address
  static char none[16] __attribute__((aligned(16)));
  if (rows == 0) dy = x = none;
  const int r = rows > 0 ? rows : 1;
  return moe::dispatch<moe::kWgrad>(a, {x, ldx, in_features, r, 1}, {dy, lddy, out_features, r, 1},
                                    f32, static_cast<cudaStream_t>(stream));
}
