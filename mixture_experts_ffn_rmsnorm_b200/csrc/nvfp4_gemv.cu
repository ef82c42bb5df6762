// Matrix-vector products of a few tokens with their experts' NVFP4 matrices
// (moe_nvfp4_gemv): the W4A16 form of a decode step's expert projections
// (MoeLayer's W4A16 kernels).
//
//   y[t, j, n] = act(s2[e] * sum_k E2M1(w[e, n, k]) * E4M3(s[e, n, k / 16]) * x[t(, j), k]),
//   e = idx[t, j].
//
// Bound: HBM; a step reads the chosen experts' 9/16 byte per weight once and
// little else.  Unpacking 4-bit weights on the CUDA cores costs more than the
// stream (conversion, scale and mma.sync take about 230 instructions per 2048
// weights: 38 us where the bytes take 17.6, 8 tokens over 39 experts), so the
// block-scaled tensor cores (tcgen05.mma kind::mxf4nvf4, scale vectors of 16)
// take the weights and their scales as they are stored.  Their other operand
// is E2M1 too, and a token row becomes one exactly, in digits: with a power of
// two of its own, 2^s, a row's elements are whole numbers X = 2^s x of
// magnitude below 2^46 (the largest at least 2^45), and X = sum_i d_i 8^i with
// sixteen digits d_i in -4..3, each an E2M1 value (in halves).  Row n of the
// other operand is digit n % 16 of token n / 16; sixteen accumulator columns
// join as sum_i 8^i acc_i.  Every FP16 row fits (2^15 down to 2^-24), and of a
// BF16 row every element down to 2^-38 of its largest.  What does not fit
// (smaller ones, infinities and NaN) has no digits: it counts as zero there and
// is added in the epilogue from the stored weights.  So a token's
// elements count in full, whatever stands beside them.  (Eight digits, half the
// columns, round to 2^-22 of the row's largest: with an FP16 60000 at a weight
// of zero the outputs of elements around 0.1 were off by 4 %.)
//
// Layout: routed rows of one expert share passes of up to 4 rows over its
// matrix.  All passes' blocks of 64 weight rows ("units") form one list, cut
// into contiguous ranges, one per CTA; a CTA takes two neighbouring units of a
// pass as one tile of 128 rows (the MMA's M) where it can.
//   warp 20    TMA: 256 inputs (128 bytes) of a tile's rows into a ring stage,
//              and the tile's scales as one copy;
//   warps 0-3  the MMAs, every third or fourth stage each and into an
//              accumulator of its own: a warp takes longer to wait for a stage
//              and issue its four MMAs than the MMAs themselves take;
//   warps 4-7  epilogue: a lane is a weight row, so the lanes' results are
//              neighbours in y;
//   warps 8-11 scales from shared memory through registers into TMEM, a
//              lane quarter each (read from global memory by the row, 4 to 8
//              bytes a lane, they took 1000 cycles a stage; handed on with
//              tcgen05.cp, the four copies of a stage held up its MMAs);
//   warps 12-19 the token rows' digits, a pass ahead of its MMAs.
// Results do not depend on the grid.
//
// Measured (one B200, a graph of eight calls with routings of their own): one
// token, six experts of 2688 x 1856, 9.4 us (17 MB; launch 2.2 us, passes, digits
// and the MMAs of one tile follow one another); 8 tokens, about 41 experts of 1856 x
// 2688, 26.0 us (4.4 TB/s).
#include <cuda_fp16.h>

#include "handle_free.h"
#include "ptx_pair.cuh"

namespace moe {
namespace {

constexpr int kGemvThreads = 672;
constexpr int kProducer = 20;  // warp
constexpr int kUnitRows = 64;
constexpr int kHalf = 8;            // digits of 24 bits
constexpr int kDigits = 2 * kHalf;
constexpr int kMaxPassRows = 4;
constexpr int kStageK = 256;         // inputs of a stage: 128 bytes a row
constexpr int kStageBytes = 128 * 128;  // a stage's weights
constexpr int kMaxStages = 12;
constexpr int kMaxRows = MOE_NVFP4_MAX_ROWS;
constexpr int kGemvSmemMax = 232448;
// TMEM columns: two accumulators (of a chain for each MMA warp), the tokens'
// scales (ones), the stages' scales (16 columns each: 4 bytes of a row per 64
// inputs, 4 x 32 rows)
constexpr int kChains = 4;  // MMA warps, at most
constexpr int kTmemCols = 512;
constexpr int kWideChains = 3, kWideStages = 6;  // with passes of kMaxPassRows
static_assert(2 * kChains * 2 * kDigits + 16 + kMaxStages * 16 <= kTmemCols, "");
static_assert(2 * kWideChains * kMaxPassRows * kDigits + 16 + kWideStages * 16 <= kTmemCols, "");
constexpr int kConverters = 8 * 32;  // threads that write digits

struct GemvArgs {
  CUtensorMap tmW;  // [E * N, K / 2] bytes, boxes of 128 bytes x 64 rows
  const void* x;
  long long ldx;
  int per_slot;
  const int* idx;
  int R, top_k;
  const uint8_t* scale;
  long long scale_bytes;  // E * N * K / 16
  const float* scale2;
  const uint8_t* w;
  int E, K, N;
  int relu2;
  void* y;
  long long ldy;
  int* status;
  int rp;      // rows of a pass, at most (1, 2 or 4)
  int xrows;   // their digit rows: rp * 16, also an accumulator's columns
  int col_sfb;  // TMEM column of the tokens' scales; the stages' follow 16 later
  int stages;
  int issuers;    // MMA warps (3 or 4); divides stages
  int xbufs;      // passes whose digits are in shared memory (1 or 2)
  int raws;       // tiles whose scales are in shared memory (1 or 2)
  int raw_bytes;  // of one tile
};

static_assert(kMaxRows <= 32767 && MOE_MAX_EXPERTS <= 256, "int16 / uint8 tables");
struct Setup {
  int16_t id[kMaxRows];       // expert of each routed row (-1: none)
  int16_t sorted[kMaxRows];   // routed rows by expert
  int16_t pass_at[kMaxRows];  // first row in `sorted`, rows and expert of each pass
  int16_t pass_n[kMaxRows];   // (before: rank of each row among its expert's)
  uint8_t pass_e[kMaxRows];
  int count[MOE_MAX_EXPERTS];
  int first[MOE_MAX_EXPERTS];
  int passes;
  int xrow[2][kMaxPassRows];      // token rows in each digit buffer
  int top[2][kMaxPassRows];       // their largest exponents
  uint32_t odd[2][kMaxPassRows];  // their blocks of 256 that hold elements without digits
  uint32_t amax[kMaxPassRows][8];
  int changed;  // the last pass whose token rows differ from those of its buffer
  volatile int abort;
};

// Bounded wait.  Once one has run out, every wait of the CTA returns at once:
// the warps go on through their barriers and store nothing.
__device__ __forceinline__ bool wait_for(const GemvArgs& p, uint64_t* bar, uint32_t parity,
                                         volatile int* abort) {
  if (mbar_wait(bar, parity, abort)) return true;
  *abort = 1;
  if (p.status) atomicOr(p.status, kStatusWaitTimeout);
  return false;
}

// D[tmem] (+)= A * SFA x (B * SFB)^T: E2M1 operands, one E4M3 scale per 16.
__device__ __forceinline__ void umma_nvfp4(uint32_t d, uint64_t adesc, uint64_t bdesc,
                                           uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, [%4], "
      "[%5], p;\n\t}\n" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// Block-scaled instruction descriptor: E2M1 x E2M1, K-major, unsigned E4M3
// scales (bit 23 clear), scale ids 0, M = 128.
__device__ __forceinline__ uint32_t nvfp4_idesc(uint32_t N) {
  return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ int expert_of(const GemvArgs& p, int r) {
  const int e = p.idx[r];
  const bool good = unsigned(e) < unsigned(p.E);
  if (!good && p.status && blockIdx.x == 0) atomicOr(p.status, kStatusBadIndex);
  return good ? e : -1;
}

// The passes of up to 32 routed rows, by one warp with a row per lane (a
// decode step's few tokens: nothing but shuffles between the ids' arrival and
// the first weight load).
__device__ __forceinline__ void group_few_rows(const GemvArgs& p, Setup& S) {
  const int lane = threadIdx.x & 31;
  const uint32_t before = (1u << lane) - 1u;
  const int e = lane < p.R ? expert_of(p, lane) : -1;
  const uint32_t same = __match_any_sync(0xffffffffu, e);
  const int rank = __popc(same & before), count = __popc(same);
  const int chunk = rank / p.rp * p.rp;  // rank of the pass's first row
  const uint32_t leaders = __ballot_sync(0xffffffffu, e >= 0 && rank == chunk);
  uint32_t rest = same;
  for (int i = 0; i < chunk; ++i) rest &= rest - 1;
  const int pass = __popc(leaders & ((1u << (__ffs(rest) - 1)) - 1u));
  if (lane < p.R) S.id[lane] = int16_t(e);
  if (e >= 0) {
    S.sorted[pass * p.rp + rank - chunk] = int16_t(lane);
    if (rank == chunk) {
      S.pass_e[pass] = uint8_t(e);
      S.pass_at[pass] = int16_t(pass * p.rp);
      S.pass_n[pass] = int16_t(min(p.rp, count - rank));
    }
  }
  if (lane == 0) S.passes = __popc(leaders);
}

// The passes of any number of rows, by one warp; S.id is set and S.count zero.
__device__ __forceinline__ void group_rows(const GemvArgs& p, Setup& S) {
  const int lane = threadIdx.x & 31;
  // rank of each row among the rows of its expert, in row order
  for (int r0 = 0; r0 < p.R; r0 += 32) {
    const int r = r0 + lane;
    const int e = r < p.R ? S.id[r] : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    int rank = 0;
    if (e >= 0) rank = S.count[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && (same >> lane) == 1u) S.count[e] = rank + 1;  // the highest lane
    if (r < p.R) S.pass_n[r] = int16_t(rank);
    __syncwarp();
  }
  // first sorted position and first pass of each expert
  constexpr int kPer = MOE_MAX_EXPERTS / 32;
  int rows[kPer], nr = 0, np = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    rows[i] = S.count[lane * kPer + i];
    nr += rows[i];
    np += (rows[i] + p.rp - 1) / p.rp;
  }
  int sr = nr, sp = np;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int a = __shfl_up_sync(0xffffffffu, sr, d), b = __shfl_up_sync(0xffffffffu, sp, d);
    if (lane >= d) {
      sr += a;
      sp += b;
    }
  }
  if (lane == 31) S.passes = sp;
  int base = sr - nr, pass = sp - np;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    S.first[lane * kPer + i] = base;
    base += rows[i];
  }
  __syncwarp();
  for (int r = lane; r < p.R; r += 32) {
    const int e = S.id[r];
    if (e >= 0) S.sorted[S.first[e] + S.pass_n[r]] = int16_t(r);
  }
  __syncwarp();
  base = sr - nr;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    for (int a = 0; a < rows[i]; a += p.rp, ++pass) {
      S.pass_e[pass] = uint8_t(lane * kPer + i);
      S.pass_at[pass] = int16_t(base + a);
      S.pass_n[pass] = int16_t(min(p.rp, rows[i] - a));
    }
    base += rows[i];
  }
}

// The 16-bit types' fields: mantissa bits, the exponent of infinities and NaN,
// and the places by which the mantissa of a row's largest exponent is shifted up.
template <bool BF16>
struct Half16 {
  static constexpr int kMant = BF16 ? 7 : 10;
  static constexpr int kExpMax = BF16 ? 255 : 31;
  static constexpr int kBias = BF16 ? 127 : 15;
  static constexpr int kTop = 45 - kMant;  // the largest element below 2^46
  static constexpr int kUnit = 45 + kBias;  // s = kUnit - the largest exponent
};

// The largest finite magnitudes (as bits) of eight elements into m, two at a time.
template <bool BF16>
__device__ __forceinline__ void amax8(const uint4& u, uint32_t& m) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = w[i] & 0x7FFF7FFFu;
    const uint32_t over = (a + (0x00010001u << Half16<BF16>::kMant)) & 0x80008000u;  // not finite
    m = __vmaxu2(m, a & ~((over >> 15) * 0xFFFFu));
  }
}

__device__ __forceinline__ float pow2(int e) {  // e in -126..127
  return __uint_as_float(uint32_t(e + 127) << 23);
}

// The E2M1 codes of the five balanced base-8 digits of V (0 <= V < 2^13), digit i
// in nibble i, all signs flipped where `flip` is 0x88888.  With U = V + 4 (1 + 8 +
// ... + 8^4), digit i is ((U >> 3 i) & 7) - 4.
__device__ __forceinline__ uint32_t digit_codes(uint32_t V, uint32_t flip) {
  uint32_t t = V + 18724u;
  // 3-bit fields to nibbles
  t = (t & 0x0FFFu) | ((t & 0x7000u) << 4);
  t = (t & 0x7003Fu) | ((t & 0x0FC0u) << 2);
  t = (t & 0x70707u) | ((t & 0x3838u) << 1);
  // t - 4 as sign and magnitude (in halves): 4..7 -> 0..3, 0..3 -> -4..-1
  const uint32_t s = ~t & 0x44444u;
  const uint32_t neg = s >> 2;
  const uint32_t mag = ((t ^ (neg * 3u)) & 0x33333u) + neg;
  return (mag | (s << 1)) ^ flip;
}

// Has an element no digits?  Infinities and NaN, and in a BF16 row what may end
// below the lowest digit's unit (bits: without the sign; least: of the smallest
// element that has digits, see below).
template <bool BF16>
__device__ __forceinline__ bool no_digits(uint32_t bits, uint32_t least) {
  return bits >= uint32_t(Half16<BF16>::kExpMax) << Half16<BF16>::kMant ||
         (BF16 && bits < least && bits != 0);
}

// An element's mantissa lies max(exponent, 1) - top + kTop places above the unit,
// top the row's largest such exponent: none below exponent top - kTop.
template <bool BF16>
__device__ __forceinline__ uint32_t least_bits(int top) {
  using H = Half16<BF16>;
  return top > H::kTop + 1 ? uint32_t(top - H::kTop) << H::kMant : 0u;
}

// The codes of an element's sixteen digits, upper and lower eight.
template <bool BF16>
__device__ __forceinline__ void element_codes(uint32_t bits, int top, bool none, uint32_t& hi,
                                              uint32_t& lo) {
  using H = Half16<BF16>;
  const int ex = int(bits >> H::kMant) & H::kExpMax;
  uint32_t mant = (bits & ((1u << H::kMant) - 1u)) | (ex ? 1u << H::kMant : 0u);
  mant = none ? 0u : mant;
  const int s = mant ? max(ex, 1) + H::kTop - top : 0;
  const int q = (s * 43) >> 7;  // s / 3
  const uint64_t c = uint64_t(digit_codes(mant << (s - 3 * q), (bits & 0x8000u) ? 0x88888u : 0u))
                     << (4 * q);
  hi = uint32_t(c >> 32);
  lo = uint32_t(c);
}

// 8 x 8 nibbles: w[i] nibble j <-> w[j] nibble i.
__device__ __forceinline__ void transpose_nibbles(uint32_t (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // halves of 16 bits: rows i, i + 4
    const uint32_t a = w[i], b = w[i + 4];
    w[i] = __byte_perm(a, b, 0x5410);
    w[i + 4] = __byte_perm(a, b, 0x7632);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if ((i & 2) == 0) {  // bytes: rows i, i + 2
      const uint32_t a = w[i], b = w[i + 2];
      w[i] = __byte_perm(a, b, 0x6240);
      w[i + 2] = __byte_perm(a, b, 0x7351);
    }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {  // nibbles: rows i, i + 1
    const uint32_t a = w[i], b = w[i + 1];
    w[i] = (a & 0x0F0F0F0Fu) | ((b & 0x0F0F0F0Fu) << 4);
    w[i + 1] = ((a >> 4) & 0x0F0F0F0Fu) | (b & 0xF0F0F0F0u);
  }
}

// Sixteen scale bytes of a weight row in shared memory, in pieces of W bytes
// (the alignment every row keeps).  Pieces behind the row's end are read from
// its last one; the caller clears them.
template <int W>
__device__ __forceinline__ void load_scales(const uint8_t* row, int at, int row_bytes,
                                            uint32_t (&v)[4]) {
  if constexpr (W == 16) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + at);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  } else if constexpr (W == 8) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint2 u = *reinterpret_cast<const uint2*>(row + min(at + 8 * i, row_bytes - 8));
      v[2 * i] = u.x, v[2 * i + 1] = u.y;
    }
  } else if constexpr (W == 4) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const uint32_t*>(row + min(at + 4 * i, row_bytes - 4));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = *reinterpret_cast<const uint16_t*>(row + min(at + 4 * i, row_bytes - 2));
      const uint32_t hi =
          *reinterpret_cast<const uint16_t*>(row + min(at + 4 * i + 2, row_bytes - 2));
      v[i] = lo | hi << 16;
    }
  }
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// What the elements without digits in the 256-wide blocks `odd` of a token row add
// to weight row `row`, in ascending order.
template <bool BF16>
__device__ __noinline__ double odd_part(const GemvArgs& p, const uint16_t* x, uint32_t odd,
                                        uint32_t least, long long row) {
  double sum = 0.;
  for (; odd; odd &= odd - 1) {
    const int k0 = (__ffs(odd) - 1) * 256;
    for (int k = k0; k < min(k0 + 256, p.K); ++k) {
      const uint32_t b = x[k];
      if (!no_digits<BF16>(b & 0x7FFFu, least)) continue;
      const float v = BF16 ? __uint_as_float(b << 16) : __half2float(__ushort_as_half(uint16_t(b)));
      const uint32_t code = (p.w[row * (p.K / 2) + k / 2] >> (4 * (k & 1))) & 15;
      const uint32_t m = code & 7;
      const float mag = m < 2 ? 0.5f * m : (1.f + 0.5f * (m & 1)) * pow2(int(m >> 1) - 1);
      const uint32_t e4 = p.scale[row * (p.K / 16) + k / 16];
      const float sc = (e4 & 0x78) ? (1.f + (e4 & 7) / 8.f) * pow2(int(e4 >> 3 & 15) - 7)
                                   : (e4 & 7) * pow2(-9);
      sum += double(v) * double(((code & 8) ? -mag : mag) * sc);
    }
  }
  return sum;
}

template <bool BF16, int W>
__global__ void __launch_bounds__(kGemvThreads, 1)
    nvfp4_gemv_kernel(const __grid_constant__ GemvArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Setup S;
  __shared__ uint64_t full[kMaxStages], sf_full[kMaxStages], empty[kMaxStages];
  __shared__ uint64_t tfull[2], tempty[2], raw_full[2], raw_empty[2], xfull[2], xempty[2];
  __shared__ uint64_t drain[kChains];
  __shared__ uint32_t tmem_slot;
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;                 // the stages
  uint8_t* xs = ring + p.stages * kStageBytes;    // the digits
  const int nst = (p.K + kStageK - 1) / kStageK;  // stages of a tile
  const int xblock = p.xrows * 128;               // digit rows of one stage's inputs
  uint8_t* raw = xs + p.xbufs * nst * xblock;     // tiles' scales as they are stored
  const int row_bytes = p.K / 16;
  const uint32_t ring_u32 = smem_u32(ring), xs_u32 = smem_u32(xs);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&sf_full[s], 4);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], p.issuers);
      mbar_init(&tempty[b], 4);
      mbar_init(&xfull[b], 1);
      mbar_init(&xempty[b], 4);
      mbar_init(&raw_full[b], 1);
      mbar_init(&raw_empty[b], 4);
    }
    for (int c = 0; c < kChains; ++c) mbar_init(&drain[c], 1);
    fence_barrier_init();
    tma_prefetch_desc(&p.tmW);
    S.abort = 0;
  }
  if (warp == kProducer) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  if (tid < 2 * kMaxPassRows) S.xrow[tid / kMaxPassRows][tid % kMaxPassRows] = -2;
  if (tid == 0) S.changed = -1;
  pdl_wait();
  pdl_trigger();
  // ---- passes: routed rows grouped by expert, at most rp rows each
  if (p.R <= 32) {
    if (warp == 0) group_few_rows(p, S);
  } else {
    for (int e = tid; e < MOE_MAX_EXPERTS; e += kGemvThreads) S.count[e] = 0;
    for (int r = tid; r < p.R; r += kGemvThreads) S.id[r] = int16_t(expert_of(p, r));
    __syncthreads();
    if (warp == 0) group_rows(p, S);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot, col_sfb = uint32_t(p.col_sfb);
  // rows without an expert get zeros
  for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
    if (S.id[r] >= 0) continue;
    uint16_t* y = static_cast<uint16_t*>(p.y) + r * p.ldy;
    for (int n = tid; n < p.N; n += kGemvThreads) y[n] = 0;
  }

  const int blocks = (p.N + kUnitRows - 1) / kUnitRows;
  // (at most 1024 * 2048 units: 32 bits hold their product with the grid)
  const uint32_t units = uint32_t(S.passes) * uint32_t(blocks);
  const int u0 = int(units * blockIdx.x / gridDim.x);
  const int u1 = int(units * (blockIdx.x + 1) / gridDim.x);

  // Every role walks the same tiles: u -> pass, first unit inside the pass,
  // two units where this CTA has both of a pass.
  if (warp == kProducer) {
    // ------------------------------------------------------------ producer
    int stage = 0, it = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = u0, two; u < u1 && ok; u += two, ++it) {
      const int pass = u / blocks, block = u - pass * blocks;
      two = u + 1 < u1 && block + 1 < blocks ? 2 : 1;
      const int row = uniform(int(S.pass_e[pass])) * p.N + block * kUnitRows;
      const int slot = it % p.raws;
      ok = uniform(wait_for(p, &raw_empty[slot], ((it / p.raws) & 1) ^ 1u, &S.abort));
      if (!ok) break;
      {
        // the rows' scales: the 16-byte blocks that hold them, and the
        // tensor's last bytes, fewer than 16, by plain loads
        const long long a = (long long)(row)*row_bytes;
        const long long end = a + min(two * kUnitRows, p.N - block * kUnitRows) * row_bytes;
        const long long a16 = a & ~15LL, whole = p.scale_bytes & ~15LL;
        const long long b16 = min((end + 15) & ~15LL, whole);
        uint8_t* dst = raw + slot * p.raw_bytes;
        if (elect_one()) {
          for (long long i = b16; i < end; ++i) dst[i - a16] = p.scale[i];
          mbar_arrive_expect_tx(&raw_full[slot], uint32_t(b16 - a16));
          if (b16 > a16)
            bulk_load(smem_u32(dst), p.scale + a16, uint32_t(b16 - a16), &raw_full[slot]);
        }
        __syncwarp();
      }
      for (int k = 0; k < nst; ++k) {
        ok = uniform(wait_for(p, &empty[stage], phase ^ 1u, &S.abort));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t bar = smem_u32(&full[stage]), st = ring_u32 + stage * kStageBytes;
          mbar_arrive_expect_tx(&full[stage], two * 8192);
          tma_load_3d<1>(st, &p.tmW, bar, k * 128, row, 0);
          if (two == 2) tma_load_3d<1>(st + 8192, &p.tmW, bar, k * 128, row + kUnitRows, 0);
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {
      const long long t0 = clock64();  // let the copies in flight land
      while (clock64() - t0 < 4000000) {
      }
    }
  } else if (warp < kChains) {
    // --------------------------------------------------------- MMA issuers
    // Warp w takes the stages whose number in the CTA's sequence is w modulo
    // `issuers`, which divides the ring: a ring stage has one issuer for good,
    // so no wait can be answered by a phase that another issuer left open.
    // The warp walks with warp-uniform values, one lane issues.
    if (warp < p.issuers) {
      int it = 0, seen = -1, passes = -1;  // tiles; the pass, and how many before it
      int stage = warp, k0 = warp;        // this warp's next stage, and its first of the tile
      uint32_t phase = 0;
      bool ok = true;
      for (int u = u0, two; u < u1 && ok; u += two) {
        const int pass = u / blocks, block = u - pass * blocks;
        two = u + 1 < u1 && block + 1 < blocks ? 2 : 1;
        if (pass != seen) {
          seen = pass;
          ++passes;
          if (!uniform(wait_for(p, &xfull[passes % p.xbufs], (passes / p.xbufs) & 1, &S.abort)))
            break;
        }
        const uint32_t idesc = nvfp4_idesc(uniform(int(S.pass_n[pass])) * kDigits);
        const uint32_t d = tmem + uint32_t(((it & 1) * p.issuers + warp) * p.xrows);
        const uint32_t xb = xs_u32 + passes % p.xbufs * nst * xblock;
        if (!uniform(wait_for(p, &tempty[it & 1], ((it >> 1) & 1) ^ 1u, &S.abort))) break;
        tc_fence_after();
        int k = k0;
        for (; k < nst; k += p.issuers) {
          ok = uniform(wait_for(p, &full[stage], phase, &S.abort) &&
                       wait_for(p, &sf_full[stage], phase, &S.abort));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sfa = tmem + col_sfb + 16 + stage * 16;
          const int steps = min(4, (p.K - k * kStageK + 63) / 64);
          const uint64_t ad = smem_desc_k_sw128(ring_u32 + stage * kStageBytes);
          const uint64_t bd = smem_desc_k_sw128(xb + k * xblock);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < steps)
                umma_nvfp4(d, ad + j * 2, bd + j * 2, idesc, sfa + j * 4, tmem + col_sfb,
                           k > k0 || j > 0);
            umma_commit(&empty[stage]);
          }
          __syncwarp();
          stage += p.issuers;
          if (stage >= p.stages) {
            stage -= p.stages;
            phase ^= 1u;
          }
        }
        k0 = k - nst;
        if (ok && elect_one()) umma_commit(&tfull[it & 1]);
        __syncwarp();
        ++it;
      }
      if (elect_one()) umma_commit(&drain[warp]);
      __syncwarp();
      int zero = 0;
      mbar_wait(&drain[warp], 0, &zero);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ epilogue
    const int cw = warp - 4;
    int it = 0, passes = 0;
    for (int ub = u0; ub < u1; ++passes) {
      const int pass = ub / blocks, b = passes % p.xbufs;
      const int ue = min(u1, (pass + 1) * blocks);  // this CTA's units of the pass
      const int n_rows = S.pass_n[pass], e = S.pass_e[pass];
      const int16_t* rows = S.sorted + S.pass_at[pass];
      const float s2 = p.scale2[e];
      const int chains = min(p.issuers, nst);  // accumulators in use
      wait_for(p, &xfull[b], (passes / p.xbufs) & 1, &S.abort);  // the rows' s
      for (int u = ub, two; u < ue; u += two) {
        two = u + 1 < ue ? 2 : 1;
        const int n0 = (u - pass * blocks) * kUnitRows;
        const int valid = min(two * kUnitRows, p.N - n0);  // weight rows of the tile
        const int r = cw * 32 + lane;
        const bool ok = wait_for(p, &tfull[it & 1], (it >> 1) & 1, &S.abort);
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t(cw * 32) << 16) +
                           uint32_t((it & 1) * p.issuers * p.xrows);
        const int chain0 = int(uint32_t(it * nst) % uint32_t(p.issuers));  // of the tile's first stage
        for (int n = 0; n < n_rows && cw * 32 < valid; ++n) {
          // chain c: the stages c, c + issuers, ... of the tile
          uint32_t acc[kChains][kDigits];
#pragma unroll
          for (int c = 0; c < kChains; ++c) {
            int w = c < chains ? chain0 + c : 0;
            w = w >= p.issuers ? w - p.issuers : w;
            tmem_ld_32x32b_x16(d + uint32_t(w * p.xrows + n * kDigits), acc[c]);
          }
          tmem_ld_wait_regs(acc);
          float v[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[h] = 0.f;
#pragma unroll
            for (int i = kHalf - 1; i >= 0; --i) {
              float t = __uint_as_float(acc[0][h * kHalf + i]);
#pragma unroll
              for (int c = 1; c < kChains; ++c)
                if (c < chains) t += __uint_as_float(acc[c][h * kHalf + i]);
              v[h] = fmaf(v[h], 8.f, t);
            }
          }
          // digits count halves: times 2^(1 - s), in whatever range the factors lie
          const double unscale =
              __longlong_as_double((long long)(1024 - Half16<BF16>::kUnit + S.top[b][n]) << 52);
          double sum = double(fmaf(v[1], 16777216.f, v[0])) * unscale;
          if (r < valid && ok && !S.abort) {
            const long long src = p.per_slot ? rows[n] : rows[n] / p.top_k;
            if (S.odd[b][n])
              sum += odd_part<BF16>(p, static_cast<const uint16_t*>(p.x) + src * p.ldx,
                                    S.odd[b][n], least_bits<BF16>(S.top[b][n]),
                                    (long long)(e)*p.N + n0 + r);
            float out = float(sum * double(s2));
            if (p.relu2) out = out <= 0.f ? 0.f : out * out;  // NaN stays NaN
            const long long o = rows[n] * p.ldy + n0 + r;
            if constexpr (BF16)
              static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(out);
            else
              static_cast<__half*>(p.y)[o] = __float2half_rn(out);
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[it & 1]);
        ++it;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&xempty[b]);
      ub = ue;
    }
  } else if (warp >= 12) {
    // -------------------------------------------------------------- digits
    const int cw = warp - 12;
    int passes = 0;
    for (int ub = u0; ub < u1; ++passes) {
      const int pass = ub / blocks, b = passes % p.xbufs;
      const int n_rows = S.pass_n[pass];
      const int16_t* rows = S.sorted + S.pass_at[pass];
      // a row's 256-wide blocks over 8, 4 or 2 warps
      const int per = n_rows > 2 ? 2 : n_rows > 1 ? 4 : 8;
      const int n = cw / per, part = cw % per;
      const int want = n < n_rows ? (p.per_slot ? rows[n] : rows[n] / p.top_k) : -1;
      // the pass that had this buffer is done with it: its epilogues are, so its MMAs are
      wait_for(p, &xempty[b], ((passes / p.xbufs) & 1) ^ 1u, &S.abort);
      if (lane == 0 && part == 0 && want >= 0 && S.xrow[b][n] != want) S.changed = pass;
      named_barrier(1, kConverters);
      if (S.changed == pass) {
        const uint16_t* xr = static_cast<const uint16_t*>(p.x) + (want < 0 ? 0 : want) * p.ldx;
        // a lane's first two chunks of 8 elements stay in registers
        const int k0 = part * 256 + lane * 8, kstep = per * 256;
        uint4 held[2];
        if (want >= 0) {
          uint32_t m = 0;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            held[i] = k0 + i * kstep < p.K
                          ? *reinterpret_cast<const uint4*>(xr + k0 + i * kstep)
                          : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 2; ++i) amax8<BF16>(held[i], m);
          for (int k = k0 + 2 * kstep; k < p.K; k += kstep)
            amax8<BF16>(*reinterpret_cast<const uint4*>(xr + k), m);
          m = __reduce_max_sync(0xffffffffu, max(m & 0xFFFFu, m >> 16));
          if (lane == 0) {
            S.amax[n][part] = m;
            if (part == 0) S.odd[b][n] = 0;
          }
        }
        named_barrier(1, kConverters);
        if (want >= 0) {
          using H = Half16<BF16>;
          uint32_t m = 0;
          for (int i = 0; i < per; ++i) m = max(m, S.amax[n][i]);
          // the largest exponent's mantissas end 2^kTop above the lowest digit's unit
          const int top = max(int(m >> H::kMant), 1);
          const uint32_t least = least_bits<BF16>(top);
          if (lane == 0 && part == 0) {
            S.xrow[b][n] = want;
            S.top[b][n] = top;
          }
          auto put = [&](int k, const uint4& u) {
            const uint32_t x2[4] = {u.x, u.y, u.z, u.w};
            uint32_t hi[8], lo[8], low = 0;
            bool odd = false;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint32_t bits = (x2[i / 2] >> (16 * (i & 1))) & 0xFFFFu;
              const bool none = no_digits<BF16>(bits & 0x7FFFu, least);
              odd |= none;
              element_codes<BF16>(bits, top, none, hi[i], lo[i]);
              low |= lo[i];
            }
            if (odd) atomicOr(&S.odd[b][n], 1u << (k / 256));
            transpose_nibbles(hi);
            if (__any_sync(0xffffffffu, low)) transpose_nibbles(lo);  // (rare in BF16 rows)
            // digit i of eight inputs: 4 bytes of row n * 16 + i, swizzled as TMA would
            uint8_t* dst = xs + (b * nst + k / kStageK) * xblock + n * kDigits * 128 + (lane & 3) * 4;
#pragma unroll
            for (int i = 0; i < kHalf; ++i) {
              uint8_t* d = dst + i * 128 + ((lane >> 2) ^ i) * 16;
              *reinterpret_cast<uint32_t*>(d) = lo[i];
              *reinterpret_cast<uint32_t*>(d + kHalf * 128) = hi[i];
            }
          };
          // zeros behind K, to the end of the last stage
          // (one copy of the code: it runs cold)
#pragma unroll 1
          for (int k = k0, i = 0; k < nst * kStageK; k += kstep, ++i) {
            uint4 u = i == 0 ? held[0] : held[1];
            if (i > 1)
              u = k < p.K ? *reinterpret_cast<const uint4*>(xr + k) : make_uint4(0, 0, 0, 0);
            put(k, u);
          }
        }
        fence_proxy_async_smem();
        named_barrier(1, kConverters);
      }
      if (warp == 12 && lane == 0) mbar_arrive(&xfull[b]);
      ub = (pass + 1) * blocks;
    }
  } else {
    // -------------------------------------------------------------- scales
    // Each warp fills its own lane quarter of TMEM, and every quarter holds
    // all rows' scales: lane l writes those of rows l, l + 32, l + 64, l + 96.
    const uint32_t quarter = tmem + (uint32_t((warp & 3) * 32) << 16);
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0x38383838u;  // the tokens' scales: ones
    tmem_st_32x32b_x16(quarter + col_sfb, v);
    tmem_st_wait();  // (a CTA without units frees the columns next)
    int stage = 0, it = 0;
    uint32_t phase = 0;
    for (int u = u0, two; u < u1; u += two, ++it) {
      const int pass = u / blocks, block = u - pass * blocks;
      two = u + 1 < u1 && block + 1 < blocks ? 2 : 1;
      const int valid = min(two * kUnitRows, p.N - block * kUnitRows);
      const int slot = it % p.raws;
      const long long a = ((long long)(S.pass_e[pass]) * p.N + block * kUnitRows) * row_bytes;
      const uint8_t* rows = raw + slot * p.raw_bytes + int(a & 15) + lane * row_bytes;
      wait_for(p, &raw_full[slot], (it / p.raws) & 1, &S.abort);
      for (int k = 0; k < nst; ++k) {
        uint32_t w[4][4];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          load_scales<W>(rows + 32 * c * row_bytes, k * 16, row_bytes, w[c]);
        // scales are unsigned; none behind K or the tile's last row
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int left = row_bytes - k * 16 - 4 * j;  // 2 where K ends inside
          const uint32_t keep = left >= 4 ? 0x7F7F7F7Fu : left > 0 ? 0x7F7Fu : 0u;
#pragma unroll
          for (int c = 0; c < 4; ++c) v[4 * j + c] = lane + 32 * c < valid ? w[c][j] & keep : 0u;
        }
        wait_for(p, &empty[stage], phase ^ 1u, &S.abort);
        tc_fence_after();
        tmem_st_32x32b_x16(quarter + col_sfb + 16 + stage * 16, v);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[stage]);
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (lane == 0) mbar_arrive(&raw_empty[slot]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kProducer) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Static shared memory of the kernel, at most.
constexpr int kGemvStatic = int(sizeof(Setup)) + 512;

// All variants on the current device, before the first launch (loads the kernels,
// too): a call of another type or width than the first one's finds its own ready.
cudaError_t set_up_variants() {
  cudaError_t e = cudaSuccess;
  for (auto* fn : {nvfp4_gemv_kernel<true, 16>, nvfp4_gemv_kernel<true, 8>,
                   nvfp4_gemv_kernel<true, 4>, nvfp4_gemv_kernel<true, 2>,
                   nvfp4_gemv_kernel<false, 16>, nvfp4_gemv_kernel<false, 8>,
                   nvfp4_gemv_kernel<false, 4>, nvfp4_gemv_kernel<false, 2>})
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kGemvSmemMax - kGemvStatic);
  return e;
}

template <bool BF16, int W>
cudaError_t launch_gemv(const GemvArgs& a, int grid, int smem, cudaStream_t stream) {
  // a programmatic dependent launch: the set-up up to pdl_wait overlaps the
  // kernel before
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(kGemvThreads);
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, nvfp4_gemv_kernel<BF16, W>, a);
}

template <int W>
cudaError_t launch_any(bool bf16, const GemvArgs& a, int grid, int smem, cudaStream_t stream) {
  return bf16 ? launch_gemv<true, W>(a, grid, smem, stream)
              : launch_gemv<false, W>(a, grid, smem, stream);
}

}  // namespace
}  // namespace moe

extern "C" moe_status moe_nvfp4_gemv(const void* x, int64_t ldx, int32_t x_per_slot,
                                     const int32_t* idx, int32_t num_tokens, int32_t top_k,
                                     const void* w, const void* w_scale, const float* w_scale2,
                                     int32_t num_experts, int32_t in_features,
                                     int32_t out_features, int32_t dtype, int32_t activation,
                                     void* y, int64_t ldy, int32_t* status, void* stream) {
  using namespace moe;
  if (num_experts < 1 || num_experts > MOE_MAX_EXPERTS || top_k < 1 || top_k > MOE_MAX_TOP_K)
    return MOE_ERR_INVALID_CONFIG;
  if (in_features < 32 || in_features > MOE_NVFP4_MAX_K || in_features % 32 || out_features < 1 ||
      out_features > MOE_GROUPED_MAX_FEATURES)
    return MOE_ERR_INVALID_CONFIG;
  if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_FP16) return MOE_ERR_INVALID_CONFIG;
  if (activation != MOE_ACT_NONE && activation != MOE_ACT_RELU2) return MOE_ERR_INVALID_CONFIG;
  if (x_per_slot != 0 && x_per_slot != 1) return MOE_ERR_INVALID_CONFIG;
  if (ldx < in_features || (ldx & 7) || ldy < out_features) return MOE_ERR_INVALID_CONFIG;
  if (num_tokens < 0 || int64_t(num_tokens) * top_k > MOE_NVFP4_MAX_ROWS)
    return MOE_ERR_TOKENS_OUT_OF_RANGE;
  if (num_tokens == 0) return MOE_OK;
  if (!x || !idx || !w || !w_scale || !w_scale2 || !y) return MOE_ERR_NULL_POINTER;
  if (!aligned_to(x, 16) || !aligned_to(w, 16) || !aligned_to(w_scale, 16) ||
      !aligned_to(w_scale2, 4) || !aligned_to(idx, 4) || !aligned_to(y, 2) ||
      !aligned_to(status, 4))
    return MOE_ERR_MISALIGNED;
  int dev = 0, sms = 0;
  const moe_status st = current_device(&dev, &sms);
  if (st != MOE_OK) return st;
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[dev].load(std::memory_order_acquire)) {
    if (set_up_variants() != cudaSuccess) {
      cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    ready[dev].store(true, std::memory_order_release);
  }

  GemvArgs a = {};
  const int K = in_features, N = out_features;
  const uint64_t rows = uint64_t(num_experts) * N;
  if (!make_map_3d(&a.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, K / 2, rows, 1, K / 2, K / 2,
                   kUnitRows))
    return MOE_ERR_CUDA;
  a.x = x;
  a.ldx = ldx;
  a.per_slot = x_per_slot;
  a.idx = idx;
  a.R = num_tokens * top_k;
  a.top_k = top_k;
  a.scale = static_cast<const uint8_t*>(w_scale);
  a.scale_bytes = (long long)(rows) * (K / 16);
  a.scale2 = w_scale2;
  a.w = static_cast<const uint8_t*>(w);
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.relu2 = activation == MOE_ACT_RELU2;
  a.y = y;
  a.ldy = ldy;
  a.status = status;
  // Rows of a pass: more rows share one read of the weights, but each takes
  // shared memory from the ring and accumulator columns.  128 experts of 2688 x
  // 1856, k = 6, us with passes of 1 / 2 / 4 rows, uniform routing (and with
  // popularity rank^-1.2): 4 tokens 16.1 / 17.8 / 19.0 (15.2 / 17.4 / 21.3), 8 tokens
  // 26.4 / 26.6 / 30.5 (24.2 / 22.6 / 31.2), 16 tokens 44.8 / 39.1 / 43.3 (36.6 / 31.9 /
  // 39.1), 32 tokens 82 / 57.1 / 61.4 (65 / 48.5 / 50.3), 64 tokens 162 / 105 / 75.5 (123
  // / 82.9 / 70.3), 128 tokens 279 / 176 / 132 (237 / 145 / 118).
  a.rp = 4 * a.R <= num_experts ? 1 : a.R < 3 * num_experts ? 2 : kMaxPassRows;
  if (a.rp > num_tokens) a.rp = num_tokens > 1 ? 2 : 1;  // ids of a token are distinct, as a rule
  // What shares the memory: digits of one or two passes, scales of one or two
  // tiles, the ring.  The first that leaves the ring its stages; fewer rows a pass
  // where none does.  (One token, 2688 x 1856: 9 stages and one tile's scales 9.5
  // us, 8 and two tiles' 9.7.  8 tokens: 6 stages and two passes' digits 26.5, 8
  // and one pass's 28.6.  64 tokens, 4096 x 1024: 3 stages and 4 rows a pass 93, 4
  // and 2 rows 118.)
  struct Share {
    int xbufs, raws, stages;
  };
  constexpr Share kShares[] = {{2, 2, 9}, {2, 1, 9}, {2, 2, 6}, {2, 1, 6}, {1, 2, 6}, {1, 1, 4}};
  const int nst = (K + kStageK - 1) / kStageK;
  a.raw_bytes = 128 * (K / 16) + 32;
  for (a.stages = 0;; a.rp /= 2) {
    a.xrows = a.rp * kDigits;
    for (const Share& s : kShares) {
      a.xbufs = s.xbufs;
      a.raws = s.raws;
      a.stages = (kGemvSmemMax - kGemvStatic - 1024 - a.xbufs * nst * a.xrows * 128 -
                  a.raws * a.raw_bytes) /
                 kStageBytes;
      if (a.stages >= s.stages) break;
    }
    if (a.stages >= (a.rp == kMaxPassRows ? kWideChains : 4) || a.rp == 1) break;
  }
  // (three MMA warps where accumulators of 64 columns leave none for a fourth's)
  const bool wide = a.rp == kMaxPassRows;
  if (a.stages > (wide ? kWideStages : kMaxStages)) a.stages = wide ? kWideStages : kMaxStages;
  a.issuers = wide                                      ? kWideChains
              : a.stages / 3 * 3 > a.stages / 4 * 4 ? 3
                                                        : 4;
  a.stages = a.stages / a.issuers * a.issuers;
  a.col_sfb = 2 * a.issuers * a.xrows;
  const long long most = (long long)(a.R) * ((N + kUnitRows - 1) / kUnitRows);
  const int grid = int(most < sms ? most : sms);
  const int smem = 1024 + a.stages * kStageBytes + a.xbufs * nst * a.xrows * 128 +
                   a.raws * a.raw_bytes;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool bf16 = dtype == MOE_DTYPE_BF16;
  const int row_bytes = K / 16;  // of scales: even
  const cudaError_t err = row_bytes % 16 == 0  ? launch_any<16>(bf16, a, grid, smem, cs)
                          : row_bytes % 8 == 0 ? launch_any<8>(bf16, a, grid, smem, cs)
                          : row_bytes % 4 == 0 ? launch_any<4>(bf16, a, grid, smem, cs)
                                               : launch_any<2>(bf16, a, grid, smem, cs);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
