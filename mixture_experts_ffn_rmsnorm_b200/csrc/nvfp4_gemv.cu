// Matrix-vector products of a few tokens with their experts' NVFP4 matrices
// (moe_nvfp4_gemv): the W4A16 form of a decode step's expert projections
// (MoeLayer's W4A16 kernels).
//
//   y[t, j, n] = act(s2[e] * sum_k E2M1(w[e, n, k]) * E4M3(s[e, n, k / 16]) * x[t(, j), k]),
//   e = idx[t, j].
//
// Bound: HBM.  A step reads the chosen experts' 9/16 byte per weight once and
// little else; at 4 bits the arithmetic is the next limit (an SM gets about
// 40 weights a cycle at the full bandwidth), so the multiply-adds run as
// mma.sync m16n8k16 (16 weight rows x up to 8 tokens) on f16 operands that
// are exact: E2M1 times E4M3 has at most 6 significant bits and lies in
// [2^-10, 2688]; an FP16 token is one already, and a BF16 token row becomes
// one under a power-of-two scale of its own that puts its largest magnitude
// in [2^14, 2^15): every element above 2^-29 of the largest keeps all its
// bits, and what a smaller one loses is at most 2^-39 of the largest, far
// below the float32 sum's own rounding.  tcgen05 would need the
// unpacked weights in shared memory, written and read once more per product.
//
// Layout: routed rows with the same expert share a pass of up to 8 rows over
// its matrix.  All passes' blocks of 16 weight rows ("units") form one list,
// cut into contiguous ranges, one per CTA, so each CTA streams one contiguous
// piece of at most a few matrices.  One warp loads units into a ring of
// shared-memory stages (TMA boxes of 128 bytes x 16 rows, the scales as one
// bulk copy); four groups of four warps each take a unit, split its K by
// blocks of 128 over their warps and add up their four partial results in a
// fixed order.  Results do not depend on the grid.
#include <cuda_fp16.h>

#include "handle_free.h"
#include "ptx_pair.cuh"

namespace moe {
namespace {

constexpr int kGroups = 4;        // consumer groups
constexpr int kGroupWarps = 4;    // warps of a group
constexpr int kConsumers = kGroups * kGroupWarps * 32;
constexpr int kGemvThreads = kConsumers + 32;
constexpr int kUnitRows = 16;
constexpr int kMaxStages = 12;
constexpr int kMaxRows = MOE_NVFP4_MAX_ROWS;
constexpr int kGemvSmemMax = 232448;

struct GemvArgs {
  CUtensorMap tmW;  // [E * N, K / 2] bytes in spans of 128: a box is the whole spans of 16 rows
  CUtensorMap tmT;  // the same as rows: a box is 128 bytes of 16 rows (the part of a span at the end)
  const void* x;
  long long ldx;
  int per_slot;
  const int* idx;
  int R, top_k;
  const uint8_t* scale;
  long long scale_bytes;  // E * N * K / 16
  const float* scale2;
  int E, K, N;
  int relu2;
  void* y;
  long long ldy;
  int* status;
  int rp;           // rows of a pass, at most (1, 2, 4 or 8)
  int stages;
  int stage_bytes;  // multiple of 1024
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
  int xrow[8];    // token rows staged (-1: zeros)
  float xinv[8];  // 2^-s of each staged row
  int changed;    // the last pass whose token rows differ from the staged ones
  volatile int abort;
};

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight E2M1 values of a word (low nibble first) as four f16 pairs.
__device__ __forceinline__ void unpack_e2m1(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 values as an f16 pair (exact; NaN stays NaN).
__device__ __forceinline__ uint32_t unpack_e4m3(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bounded wait.  Once one has run out, every wait of the CTA returns at once:
// the warps go on through their barriers and store nothing.
__device__ __forceinline__ bool wait_for(const GemvArgs& p, uint64_t* bar, uint32_t parity,
                                         volatile int* abort) {
  if (mbar_wait(bar, parity, abort)) return true;
  *abort = 1;
  if (p.status) atomicOr(p.status, kStatusWaitTimeout);
  return false;
}

// Largest finite magnitude of 8 BF16 values.
__device__ __forceinline__ float amax8(const uint4& u) {
  float m = 0.f;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = fabsf(__uint_as_float(w[i] << 16));
    const float hi = fabsf(__uint_as_float(w[i] & 0xFFFF0000u));
    if (lo <= 3.4028235e38f) m = fmaxf(m, lo);
    if (hi <= 3.4028235e38f) m = fmaxf(m, hi);
  }
  return m;
}

// 8 BF16 values times a power of two, as f16.
__device__ __forceinline__ uint4 scaled_f16(const uint4& u, float s) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * s,
                                        __uint_as_float(w[i] & 0xFFFF0000u) * s);
    o[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
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

// The operands of one 128-wide block that a lane takes from a stage: 32
// weights of two rows and their two scales each, as f16 pairs.
struct Block {
  uint4 wa, wb;
  uint32_t sa, sb;
};

template <bool BF16>
__global__ void __launch_bounds__(kGemvThreads, 1)
    nvfp4_gemv_kernel(const __grid_constant__ GemvArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Setup S;
  __shared__ uint64_t full[kMaxStages], empty[kMaxStages];
  __shared__ float part[kGroups][2][kGroupWarps][8 * kUnitRows];
  __shared__ float s_amax[8][2];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* ring = smem_raw + pad;
  const int nkb = (p.K + 127) / 128;
  const int xblock = p.rp * 256;  // bytes of a 128-wide block of the staged token rows
  const int scale_at = (p.K / 2 + 127) / 128 * 2048;  // scales behind a stage's boxes
  uint8_t* xs = ring + p.stages * p.stage_bytes;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kGroupWarps);
    }
    fence_barrier_init();
    tma_prefetch_desc(&p.tmW);
    tma_prefetch_desc(&p.tmT);
  }
  if (tid < 8) S.xrow[tid] = -2;
  if (tid == 0) S.abort = 0;
  pdl_wait();
  pdl_trigger();
  // ---- passes: routed rows grouped by expert, at most rp rows each
  if (p.R <= 32) {
    if (warp == 0) group_few_rows(p, S);
  } else {
    for (int e = tid; e < MOE_MAX_EXPERTS; e += kGemvThreads) S.count[e] = 0;
    for (int r = tid; r < p.R; r += kGemvThreads) S.id[r] = expert_of(p, r);
    __syncthreads();
    if (warp == 0) group_rows(p, S);
  }
  __syncthreads();
  // rows without an expert get zeros
  for (int r = blockIdx.x; r < p.R; r += gridDim.x) {
    if (S.id[r] >= 0) continue;
    uint16_t* y = static_cast<uint16_t*>(p.y) + r * p.ldy;
    for (int n = tid; n < p.N; n += kGemvThreads) y[n] = 0;
  }

  const int blocks = (p.N + kUnitRows - 1) / kUnitRows;
  const long long units = (long long)(S.passes) * blocks;
  const int u0 = int(units * blockIdx.x / gridDim.x);
  const int u1 = int(units * (blockIdx.x + 1) / gridDim.x);

  if (warp == kConsumers / 32) {
    // ------------------------------------------------------------ producer
    // One lane issues a unit's two or three copies (with a box per 128-byte
    // span, spread over the lanes, their issue alone took 0.8 us a unit).
    const uint32_t ring_u32 = smem_u32(ring);
    const int spans = p.K / 256;
    const bool rest = p.K % 256 != 0;
    const uint32_t wbytes = (spans + rest) * 2048;
    const int row_bytes = p.K / 16;
    const long long whole = p.scale_bytes & ~15LL;
    int stage = 0, pass = u0 / blocks, block = u0 - pass * blocks;
    uint32_t phase = 0;
    for (int u = u0; u < u1; ++u) {
      const long long row = (long long)(S.pass_e[pass]) * p.N + block * kUnitRows;
      if (++block == blocks) {
        block = 0;
        ++pass;
      }
      if (!wait_for(p, &empty[stage], phase ^ 1u, &S.abort)) {
        const long long t0 = clock64();  // let the copies in flight land
        while (clock64() - t0 < 4000000) {
        }
        break;
      }
      // the scales of 16 rows are contiguous: the 16-byte blocks that hold them
      const long long a = row * row_bytes;
      const long long end = min(a + (long long)(kUnitRows)*row_bytes, p.scale_bytes);
      const long long a16 = a & ~15LL;
      long long b16 = (end + 15) & ~15LL;
      if (b16 > whole) {  // the tensor's last bytes, fewer than 16: plain loads
        b16 = whole;
        if (b16 + lane < end)
          ring[stage * p.stage_bytes + scale_at + (b16 - a16) + lane] = p.scale[b16 + lane];
        __syncwarp();
      }
      if (lane == 0) {
        const uint32_t st = ring_u32 + stage * p.stage_bytes;
        const uint32_t bar = smem_u32(&full[stage]);
        const uint32_t sbytes = uint32_t(b16 - a16);
        mbar_arrive_expect_tx(&full[stage], wbytes + sbytes);
        if (spans) tma_load_3d<1>(st, &p.tmW, bar, 0, int32_t(row), 0);
        if (rest) tma_load_3d<1>(st + spans * 2048, &p.tmT, bar, spans * 128, int32_t(row), 0);
        if (sbytes) bulk_load(st + scale_at, p.scale + a16, sbytes, &full[stage]);
      }
      __syncwarp();
      if (++stage == p.stages) {
        stage = 0;
        phase ^= 1u;
      }
    }
    return;
  }

  // -------------------------------------------------------------- consumers
  const int group = warp / kGroupWarps, gw = warp % kGroupWarps;
  const int g = lane >> 2, tig = lane & 3;
  // mma row g is weight row prow (and g + 8 is prow + 8): the two rows that a
  // quarter of a warp reads together differ in bit 2, so that the swizzle
  // puts their 16-byte blocks into different banks
  const int prow = (g >> 1) | ((g & 1) << 2);
  int buf = 0, staged = -1;
  for (int ub = u0; ub < u1;) {
    const int pass = ub / blocks;
    const int ue = min(u1, (pass + 1) * blocks);  // this CTA's units of the pass
    const int n_rows = S.pass_n[pass];
    const int16_t* rows = S.sorted + S.pass_at[pass];
    const int e = S.pass_e[pass];

    // ---- the pass's token rows as f16 fragments in shared memory
    {
      const int n = tid >> 6, i = tid & 63;  // 64 threads a row
      const int r = n < n_rows ? rows[n] : -1;
      const int want = n < n_rows ? (p.per_slot ? r : r / p.top_k) : -1;
      named_barrier(1, kConsumers);  // the pass before is done with xs
      if (i == 0 && S.xrow[n] != want) S.changed = pass;
      named_barrier(1, kConsumers);
      if (staged < 0 || S.changed == pass) {
        const uint16_t* xr = static_cast<const uint16_t*>(p.x) + (want < 0 ? 0 : want) * p.ldx;
        float s = 1.f;
        if constexpr (BF16) {
          float m = 0.f;
          if (want >= 0)
            for (int k = i * 8; k < p.K; k += 512)
              m = fmaxf(m, amax8(*reinterpret_cast<const uint4*>(xr + k)));
#pragma unroll
          for (int d = 16; d; d /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          if (lane == 0) s_amax[n][(tid >> 5) & 1] = m;
          named_barrier(1, kConsumers);
          m = fmaxf(s_amax[n][0], s_amax[n][1]);
          // m in [2^ex, 2^(ex + 1)): s = 2^(14 - ex), at most 2^126
          const int ex = m > 0.f ? max(int(__float_as_uint(m) >> 23), 1) - 127 : 14;
          const int sh = min(14 - ex, 126);
          s = __uint_as_float(uint32_t(sh + 127) << 23);
          if (i == 0) S.xinv[n] = __uint_as_float(uint32_t(127 - sh) << 23);
        } else if (i == 0) {
          S.xinv[n] = 1.f;
        }
        if (i == 0) S.xrow[n] = want;
        if (n < p.rp) {
          // chunk c = 8 elements: block c / 16, lane n * 4 + (c / 4) % 4, quarter c % 4
          for (int c = i; c < nkb * 16; c += 64) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (want >= 0 && c * 8 < p.K) {
              v = *reinterpret_cast<const uint4*>(xr + c * 8);
              if constexpr (BF16) v = scaled_f16(v, s);
            }
            *reinterpret_cast<uint4*>(xs + (c >> 4) * xblock + (c & 3) * (p.rp * 64) +
                                      (n * 4 + ((c >> 2) & 3)) * 16) = v;
          }
        }
        named_barrier(1, kConsumers);
        staged = pass;
      }
    }

    const float s2 = p.scale2[e];
    for (int u = ub + ((group - (ub - u0)) & (kGroups - 1)); u < ue; u += kGroups) {
      const int at = u - u0;
      const int stage = at % p.stages;
      const uint32_t parity = (at / p.stages) & 1;
      const int n0 = (u - pass * blocks) * kUnitRows;
      const long long row = (long long)(e)*p.N + n0;
      const uint8_t* st = ring + stage * p.stage_bytes;
      const uint8_t* sc = st + scale_at + int((row * (p.K / 16)) & 15) + tig * 2;
      const uint8_t* sca = sc + prow * (p.K / 16);
      const uint8_t* scb = sc + (prow + 8) * (p.K / 16);
      wait_for(p, &full[stage], parity, &S.abort);
      auto load = [&](int b) {
        Block k;
        const uint8_t* box = st + (b >> 1) * 2048 + prow * 128 + (((b & 1) * 4 + tig) ^ prow) * 16;
        k.wa = *reinterpret_cast<const uint4*>(box);
        k.wb = *reinterpret_cast<const uint4*>(box + 1024);
        k.sa = k.sb = 0;  // zero scales behind K: the boxes hold zeros there
        if (b * 128 + tig * 32 < p.K) {
          k.sa = unpack_e4m3(*reinterpret_cast<const uint16_t*>(sca + b * 8));
          k.sb = unpack_e4m3(*reinterpret_cast<const uint16_t*>(scb + b * 8));
        }
        return k;
      };
      float c[2][4] = {};
      Block next = {};
      if (gw < nkb) next = load(gw);
      for (int b = gw; b < nkb; b += kGroupWarps) {
        const Block k = next;
        if (b + kGroupWarps < nkb) next = load(b + kGroupWarps);
        const uint32_t a_w[4] = {k.wa.x, k.wa.y, k.wa.z, k.wa.w};
        const uint32_t b_w[4] = {k.wb.x, k.wb.y, k.wb.z, k.wb.w};
        const uint8_t* xb = xs + b * xblock + lane * 16;
        uint4 x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[j] = g < p.rp ? *reinterpret_cast<const uint4*>(xb + j * (p.rp * 64))
                          : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t fa = __byte_perm(k.sa, 0, j < 2 ? 0x1010 : 0x3232);
          const uint32_t fb = __byte_perm(k.sb, 0, j < 2 ? 0x1010 : 0x3232);
          uint32_t ha[4], hb[4];
          unpack_e2m1(a_w[j], ha);
          unpack_e2m1(b_w[j], hb);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            ha[i] = mul_f16x2(ha[i], fa);
            hb[i] = mul_f16x2(hb[i], fb);
          }
          mma_16816(c[0], ha[0], hb[0], ha[1], hb[1], x[j].x, x[j].y);
          mma_16816(c[1], ha[2], hb[2], ha[3], hb[3], x[j].z, x[j].w);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      // the four warps' partial sums, [token][weight row]
      float* mine = part[group][buf][gw];
      mine[(2 * tig) * kUnitRows + prow] = c[0][0] + c[1][0];
      mine[(2 * tig + 1) * kUnitRows + prow] = c[0][1] + c[1][1];
      mine[(2 * tig) * kUnitRows + prow + 8] = c[0][2] + c[1][2];
      mine[(2 * tig + 1) * kUnitRows + prow + 8] = c[0][3] + c[1][3];
      named_barrier(2 + group, kGroupWarps * 32);
      const int t = tid & 127;
      const int tok = t / kUnitRows, n = n0 + t % kUnitRows;
      if (tok < n_rows && n < p.N && !S.abort) {
        float v = part[group][buf][0][t];
#pragma unroll
        for (int w = 1; w < kGroupWarps; ++w) v += part[group][buf][w][t];
        // one rounding to float32, in whatever range the three factors lie
        v = float(double(v) * double(s2) * double(S.xinv[tok]));
        if (p.relu2) v = v <= 0.f ? 0.f : v * v;  // NaN stays NaN
        const long long o = rows[tok] * p.ldy + n;
        if constexpr (BF16)
          static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(v);
        else
          static_cast<__half*>(p.y)[o] = __float2half_rn(v);
      }
      buf ^= 1;
    }
    ub = ue;
  }
}

template <bool BF16>
cudaError_t launch_gemv(const GemvArgs& a, int dev, int grid, int smem, cudaStream_t stream) {
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, nvfp4_gemv_kernel<BF16>);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(nvfp4_gemv_kernel<BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kGemvSmemMax - int(fa.sharedSizeBytes));
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_release);
  }
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
  return cudaLaunchKernelEx(&cfg, nvfp4_gemv_kernel<BF16>, a);
}

// Static shared memory of the kernel, rounded up.
constexpr int kGemvStatic = int(sizeof(Setup)) + 2 * 8 * kMaxStages +
                            int(sizeof(float)) * kGroups * 2 * kGroupWarps * 8 * kUnitRows + 256;

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

  GemvArgs a = {};
  const int K = in_features, N = out_features;
  const uint64_t rows = uint64_t(num_experts) * N;
  if (!make_map_3d(&a.tmT, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, K / 2, rows, 1, K / 2, K / 2,
                   kUnitRows) ||
      (K >= 256 && !make_map_spans(&a.tmW, w, rows, K / 2, K / 256, kUnitRows)))
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
  a.E = num_experts;
  a.K = K;
  a.N = N;
  a.relu2 = activation == MOE_ACT_RELU2;
  a.y = y;
  a.ldy = ldy;
  a.status = status;
  // a stage: 16 rows of weights in whole boxes, then their scales (up to 15
  // bytes more on either side).  Beside the stages lie a pass's token rows:
  // as many as an expert can have when ids are distinct, at most 8 (the
  // mma's columns), and fewer where those would leave less than two stages.
  const int boxes = (K / 2 + 127) / 128;
  a.stage_bytes = (boxes * 2048 + K + 32 + 1023) / 1024 * 1024;
  const int nkb = (K + 127) / 128;
  const int room = kGemvSmemMax - kGemvStatic - 1024 - 1024;
  a.rp = num_tokens > 4 ? 8 : num_tokens > 2 ? 4 : num_tokens;
  while (a.rp > 1 && room - nkb * a.rp * 256 < 2 * a.stage_bytes) a.rp /= 2;
  const int xbytes = nkb * a.rp * 256;
  a.stages = (room - xbytes) / a.stage_bytes;
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  const long long most = (long long)(a.R) * ((N + kUnitRows - 1) / kUnitRows);
  const int grid = int(most < sms ? most : sms);
  const int smem = 1024 + a.stages * a.stage_bytes + xbytes;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t err = dtype == MOE_DTYPE_BF16 ? launch_gemv<true>(a, dev, grid, smem, cs)
                                                  : launch_gemv<false>(a, dev, grid, smem, cs);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}
