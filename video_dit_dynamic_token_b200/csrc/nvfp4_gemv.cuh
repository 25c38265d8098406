// Products of few bf16 rows with NVFP4 weights (lx_nvfp4_gemv):
//
//   y[m, n] = bf16(fl32(acc * gw) + bias[n]),  acc = sum_k x[m, k] e2m1(w[n, k]) e4m3(s[n, k / 16])
//
// for M <= 16 rows, x kept in bf16 precision (the modulation vectors of a
// timestep, a guided pair, single new tokens).  The weights are read once: N K / 2
// bytes of codes and N K / 16 of scales, which is what bounds large ones (30720 x 5120, cold:
// one row 21.5 us = 4.1 TB/s, 120 of the 148 SMs having a tile; 8 and 16 rows 23.3).
// Small ones are bound by the start, the digits and the joining of sums (5120 x 5120, two
// rows: 8.6 us with the weights in the L2 cache, 11.0 without; 256 x 512, one row: 5.9).
//
// Decoding 4-bit weights costs more issue slots than an SM has at the rate they
// arrive (42 weights per clock; mma.sync on weights decoded to fp16 took 38 to 55 us
// for 30720 x 5120, the format's conversion instruction or 5 instructions per weight
// bounding it), so the block-scaled tensor core reads the codes as they are, and x
// takes the weights' format: each row becomes P rows of signed octal digits.
//
// Digits.  With 2^e the largest power of two in the finite magnitudes of a row of x,
// x 2^(21-e) = H + L 2^-21 with integers
// |H| <= 2^22 and |L| <= 2^20, both by rounding in fp32 (the remainder x 2^(21-e) - H is
// exact).  Each is a sum of 8 octal digits in {-4 .. 3}, read off the octal digits of
// H + 44444444 (octal); every digit is an E2M1 value.  So
//   acc = 2^(e-21) (sum_i 8^i D_(P-8+i) + 2^-21 sum_i 8^i D_i)
// with D the fp32 sums of one row of the MMA, which has 128: P = 16 rows (H and L) for
// each of up to 8 rows of x, and P = 8 (H alone) for up to 16.  x has 8 significant
// bits, so elements down to 2^-35 (2^-14) of the largest are exact and smaller ones are
// rounded by at most 2^-43 (2^-22) of it.
// Elements that are not finite have zero digits; the rows that hold them add x w for
// those k at the end.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "attn.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace lx {

constexpr int kGvMaxRows = 16;                // rows of x
constexpr int kGvTile = 256;                  // weight rows of a CTA (columns of the MMA)
constexpr int kGvSplit = 8;                   // most CTAs that share a tile's K (a cluster)
constexpr uint32_t kGvBBytes = 256 * 128;     // stage: 256 weight rows x 256 codes
constexpr uint32_t kGvSfBytes = 2 * 4 * 512;  // their scales
constexpr int kGvSlice = 1024;                // elements of x per CTA of the digit pass
constexpr int kGvThreads = 320;
constexpr uint32_t kGvTmemCols = 512;   // sums 0 .. 255; ones 256 .. 259; scales 288 + 32 per stage

// Stage: weights, scales, then one 128-byte row per digit row (a multiple of the
// 8-row swizzle pattern).  The MMA reads 128 digit rows: what lies behind the M P that
// are written is read too and not used, hence the slack behind the last stage.
template <int P>
struct GemvSmem {
  __host__ __device__ static constexpr uint32_t x_bytes(int M) { return 128u * (uint32_t)(M * P); }
  __host__ __device__ static constexpr uint32_t stage(int M) { return kGvBBytes + kGvSfBytes + x_bytes(M); }
  __host__ __device__ static constexpr int stages(int M) { return stage(M) <= 40 * 1024 ? 5 : 4; }
  __host__ __device__ static constexpr uint32_t bytes(int M) {
    return 1024 + (uint32_t)stages(M) * stage(M) + 128 * 128 - x_bytes(M);
  }
};
constexpr int kGvMaxStages = 5;
// Up to this many elements of x, and up to this many weights, the product kernel writes the
// digits itself, each CTA those of its range of K (8 bytes of shared memory an element): one
// launch and no workspace, 4 us less of the host's time, which such calls wait for (two rows x
// 5120 x 5120: 8.6 us on the device instead of 8.4; 0.7 more for 8 x 1280).  Beyond, and for more than 8 rows, they
// come from a pass of their own, as every CTA would read all of x and write its part again (two
// rows x 30720 x 5120: 24.3 us, with the pass 21.6).  On the device and with the host, own digits and the
// pass, by elements of x: 10240 (8 x 1280) 7.9 and 8.2, 7.3 and 10.0; 12800 (5 x 2560) 9.2 and 9.4, 7.6
// and 10.1; 13824 (one row) 11.1 and 11.1, 10.9 and 11.1; 15360 (3 x 5120) 11.2 and 11.2, 9.7 and 10.2.
constexpr int kGvOwnDigits = 10240;
constexpr long long kGvOwnWeights = 1 << 25;
constexpr uint32_t kGvSmemLimit = 227 * 1024 - 2048;
struct GemvOwnSmem {
  static constexpr uint32_t stage = kGvBBytes + kGvSfBytes;
  __host__ __device__ static constexpr uint32_t x_bytes(int M, int per) { return 2048u * (uint32_t)(M * per); }
  __host__ __device__ static constexpr uint32_t slack(int M) { return 128 * 128 - 2048u * (uint32_t)M; }
  __host__ __device__ static constexpr int stages(int M, int per) {
    const int fit = (int)((kGvSmemLimit - 1024 - x_bytes(M, per) - slack(M)) / stage);
    return fit < kGvMaxStages ? fit : kGvMaxStages;
  }
  __host__ __device__ static constexpr uint32_t bytes(int M, int per) {
    return 1024 + (uint32_t)stages(M, per) * stage + x_bytes(M, per) + slack(M);
  }
};
static_assert(GemvOwnSmem::stages(1, kGvOwnDigits / 256) >= 3 &&
                  3 * GemvOwnSmem::stage + GemvOwnSmem::x_bytes(1, kGvOwnDigits / 256) >= (128 + kGvMaxRows) * 1024 &&
                  4 * GemvOwnSmem::stage >= (128 + kGvMaxRows) * 1024 &&
                  GemvOwnSmem::stages(1, kGvOwnDigits / 512) >= 4,
              "room for the stages and the sums");
static_assert(GemvSmem<16>::bytes(1) <= 227 * 1024 - 2048 && GemvSmem<16>::bytes(2) <= 227 * 1024 - 2048 &&
                  GemvSmem<16>::bytes(8) <= 227 * 1024 - 2048 && GemvSmem<8>::bytes(16) <= 227 * 1024 - 2048,
              "shared memory per CTA");
static_assert(GemvSmem<16>::bytes(1) >= 1024 + (128 + kGvMaxRows) * 1024, "room for the sums");

// ref of a row as the digit pass leaves it: biased exponent of the largest finite
// magnitude, bit 16 set when the row holds an element that is not finite
constexpr int kGvBadRow = 1 << 16;

struct GemvArgs {
  const __nv_bfloat16* x;
  const int* ref;       // [M]
  const uint8_t* wc;
  const uint8_t* wsf;
  const float* gw;
  const float* bias;
  __nv_bfloat16* y;
  long long ldx, ldy, N;
  int M, K, per;        // per: 256-element stages of a CTA
  int stages;           // ring slots
  unsigned long long limit_ns;
};

__device__ __forceinline__ float pow2f(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

// Eight octal digits (24 bits) as nibbles, then as bytes that hold the E2M1 codes of
// digit - 4: two words, digits 0 .. 3 and 4 .. 7.
__device__ __forceinline__ void octal_codes(uint32_t x, uint32_t& lo, uint32_t& hi) {
  x += (x & 0xFFF000u) * 15u;
  x += (x & 0x0FC00FC0u) * 3u;
  x += x & 0x38383838u;
  lo = __byte_perm(0x0A0C0D0Eu, 0x05040200u, x);        // -4 -3 -2 -1 | 0 1 2 3
  hi = __byte_perm(0x0A0C0D0Eu, 0x05040200u, x >> 16);
}

// Digit codes of 8 neighbouring elements: word[d] holds digit d of element i in nibble i.
// f0 f1 = 2^(21-e) (in two factors: it may pass fp32's range).
template <int P>
__device__ __forceinline__ void gemv_digits8(const uint4& v, float f0, float f1, uint32_t (&word)[P]) {
  constexpr float kMagic23 = 12582912.f;                 // 1.5 2^23: adding it leaves the rounded integer in the low bits
  constexpr uint32_t kBias = 044444444u - 0x4B400000u;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t pr[P / 4][4];   // [group of 4 digits][pair of elements]: a byte per digit
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float x = (h ? bf16hi(w[j]) : bf16lo(w[j])) * f0;
      const float t = fmaf(x, f1, kMagic23);
      uint32_t c[P / 4];
      octal_codes(__float_as_uint(t) + kBias, c[P / 4 - 2], c[P / 4 - 1]);
      if constexpr (P == 16) {
        const float rest = fmaf(x, f1, -(t - kMagic23));  // exact
        octal_codes(__float_as_uint(fmaf(rest, 2097152.f, kMagic23)) + kBias, c[0], c[1]);
      }
#pragma unroll
      for (int q = 0; q < P / 4; ++q) pr[q][j] = h ? pr[q][j] + 16u * c[q] : c[q];
    }
#pragma unroll
  for (int q = 0; q < P / 4; ++q) {
    const uint32_t a = __byte_perm(pr[q][0], pr[q][1], 0x5140), b = __byte_perm(pr[q][2], pr[q][3], 0x5140);
    const uint32_t c = __byte_perm(pr[q][0], pr[q][1], 0x7362), d = __byte_perm(pr[q][2], pr[q][3], 0x7362);
    word[4 * q] = __byte_perm(a, b, 0x5410);
    word[4 * q + 1] = __byte_perm(a, b, 0x7632);
    word[4 * q + 2] = __byte_perm(c, d, 0x5410);
    word[4 * q + 3] = __byte_perm(c, d, 0x7632);
  }
}

// v with zeros in place of elements that are not finite
__device__ __forceinline__ uint4 finite_only(uint4 v) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
    if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Largest finite magnitude (bits of a bf16) of pieces first, first + step, ... of a row, and bits that
// are set where an element is not finite; over the warp.
__device__ __forceinline__ void gemv_row_max(const uint4* row, int first, int pieces, int step, uint32_t& top,
                                             uint32_t& bad) {
  for (int v = first; v < pieces; v += 8 * step) {   // eight loads on their way together, also the last
    uint4 t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = v + i * step < pieces ? row[v + i * step] : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (v - (int)(threadIdx.x & 31) + i * step >= pieces) break;   // (a warp together)
      const uint4 f = finite_only(t[i]);
      bad |= (f.x ^ t[i].x) | (f.y ^ t[i].y) | (f.z ^ t[i].z) | (f.w ^ t[i].w);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(f.x & 0x7FFF7FFFu, f.y & 0x7FFF7FFFu),
                                   __vmaxu2(f.z & 0x7FFF7FFFu, f.w & 0x7FFF7FFFu)));
    }
  }
  top = __reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16));
  bad = __reduce_or_sync(0xffffffffu, bad);
}

__device__ __forceinline__ int gemv_ref(uint32_t top, uint32_t bad) { return max(1, (int)(top >> 7)) | (bad ? kGvBadRow : 0); }

// grid (M, ceil(K / kGvSlice)), 128 threads of 8 elements.  Every CTA reads the whole
// row (it is short) for its largest element.  codes: [M P][K / 2], row m P + d holds
// digit d of x's row m.
template <int P>
__global__ void __launch_bounds__(128) nvfp4_gemv_digits_kernel(const __nv_bfloat16* __restrict__ x, long long ldx, int K,
                                                                uint8_t* __restrict__ codes, int* __restrict__ ref) {
  // launched before the work ahead of it on the stream has ended; once that has, the
  // product kernel may start to load the weights
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");
  const int m = blockIdx.x;
  const uint4* row = reinterpret_cast<const uint4*>(x + m * ldx);
  const int k = blockIdx.y * kGvSlice + threadIdx.x * 8;
  const uint4 mine = k < K ? row[k / 8] : make_uint4(0, 0, 0, 0);
  uint32_t top = 0, bad = 0;
  gemv_row_max(row, threadIdx.x, K / 8, 128, top, bad);
  __shared__ uint32_t s_top[4], s_bad[4];
  if ((threadIdx.x & 31) == 0) {
    s_top[threadIdx.x >> 5] = top;
    s_bad[threadIdx.x >> 5] = bad;
  }
  __syncthreads();
  top = max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3]));
  bad = s_bad[0] | s_bad[1] | s_bad[2] | s_bad[3];
  const int info = gemv_ref(top, bad), e = 21 + 127 - (info & 0xFFFF);  // 2^e, in two factors
  if (blockIdx.y == 0 && threadIdx.x == 0) ref[m] = info;
  if (k >= K) return;
  uint32_t word[P];
  gemv_digits8<P>(bad ? finite_only(mine) : mine, pow2f(e >> 1), pow2f(e - (e >> 1)), word);
#pragma unroll
  for (int d = 0; d < P; ++d)
    *reinterpret_cast<uint32_t*>(codes + (long long)(m * P + d) * (K / 2) + k / 2) = word[d];
}

__device__ __forceinline__ void mma_nvf4_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};"
      "\n\ttcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], da, db, %4, [%6], [%7], p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb)
      : "memory");
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One CTA: the digit rows (the MMA's 128 rows) against 256 weight rows over a range of
// K; one CTA per SM.  Stages of 256 codes go through a ring:
//   warp 0: loads; those of the weights do not wait for the digit pass;
//   warp 1: MMAs;
//   warps 2 .. 9: two sets in turn move a stage's scales from shared memory to TMEM (a row
//           of the tiled layout per lane, the same in all four lane quarters), then the
//           sums.  One set takes 1,000 clocks a stage, whose MMAs take 420.  tcgen05.cp
//           does the same in the tensor pipe, where each copy of 512 bytes took 70
//           clocks between MMAs of 105.
// All ten warps then turn digit sums into outputs.  The digits' own scales are 1.  OWN: warps
// 2 .. 9 write the digits of the CTA's whole range first, under the first loads of the
// weights.  (Stage by stage, for any number of rows, that cost up to 40 us more for 16.)  The CTAs of a cluster split K and add their sums over
// distributed shared memory, in rank order.
template <int P, bool OWN>
__global__ void __launch_bounds__(kGvThreads, 1) nvfp4_gemv_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                   const __grid_constant__ CUtensorMap tmX,
                                                                   const GemvArgs a) {
  using S = GemvSmem<P>;
  extern __shared__ uint8_t gv_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gv_smem_raw) + 1023) & ~uintptr_t(1023));
  // full/empty: a ring slot's loads; sf: its scales are in TMEM
  __shared__ __align__(8) uint64_t bar_full[kGvMaxStages], bar_empty[kGvMaxStages], bar_sf[kGvMaxStages], bar_acc,
      bar_drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int never_abort;
  float* dsum = reinterpret_cast<float*>(sm);              // [digit row][256], in place of the stages once used
  float* part = dsum + 128 * 256;                          // [row of x][256]

  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int M = a.M, rows = M * P, stages = a.stages;
  const uint32_t stage_bytes = OWN ? GemvOwnSmem::stage : S::stage(M);
  uint8_t* own = sm + stages * stage_bytes;                // OWN: digits, 128-byte rows, M P a stage
  __shared__ uint32_t s_top[8], s_bad[8];                  // OWN: of a row of x
  const int KS = a.K / 64, nkb = (KS + 3) / 4;
  const int tile = blockIdx.x / ranks;
  const int kb0 = rank * a.per, n = min(a.per, nkb - kb0);   // stages of this CTA (at least one)
  const bool has1 = (long long)tile * 256 + 128 < a.N;       // the second scale tile exists

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tmW);
    if constexpr (!OWN) prefetch_tensormap(&tmX);
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1 + 4);   // the MMA and the set of scale warps whose stage it is not
      mbar_init(&bar_sf[s], 4);
    }
    mbar_init(&bar_acc, 1);
    mbar_init(&bar_drain, 1);
    abort_flag = 0;
    never_abort = 0;
    if constexpr (OWN)
      for (int m = 0; m < 8; ++m) s_top[m] = s_bad[m] = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kGvTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = tmem_slot;
  int info = 0;                                              // of row `lane` of x

  if (warp == 0) {
    // OWN: x first, which would otherwise wait in the memory system behind the weights
    if constexpr (OWN) asm volatile("bar.sync 2, 288;" ::: "memory");
    if (lane == 0) {
      // ================= loads =================
      auto load_w = [&](int i) {
        const int s = i % stages, kb = kb0 + i;
        uint8_t* st = sm + s * stage_bytes;
        const uint32_t sfb = (uint32_t)min(4, KS - 4 * kb) * 512u;     // k-steps of 64 in the stage
        mbar_arrive_expect_tx(&bar_full[s], kGvBBytes + (OWN ? 0u : S::x_bytes(M)) + (has1 ? 2u : 1u) * sfb);
        tma_load_2d(st, &tmW, &bar_full[s], kb * 128, tile * 256);
        bulk_load(st + kGvBBytes, a.wsf + ((long long)(2 * tile) * KS + kb * 4) * 512, sfb, &bar_full[s]);
        if (has1)
          bulk_load(st + kGvBBytes + 2048, a.wsf + ((long long)(2 * tile + 1) * KS + kb * 4) * 512, sfb, &bar_full[s]);
      };
      auto load_x = [&](int i) {
        const int s = i % stages;
        tma_load_2d(sm + s * stage_bytes + kGvBBytes + kGvSfBytes, &tmX, &bar_full[s], (kb0 + i) * 128, 0);
      };
      const int first = min(n, stages);
      // OWN: the work ahead may have written the weights; else the digit pass has waited for it
      if constexpr (OWN) asm volatile("griddepcontrol.wait;" ::: "memory");
      for (int i = 0; i < first; ++i) load_w(i);
      if constexpr (!OWN) {
        asm volatile("griddepcontrol.wait;" ::: "memory");             // the digits are complete
        for (int i = 0; i < first; ++i) load_x(i);
      }
      bool ok = true;
      int i = first;
      for (; i < n; ++i) {
        ok = mbar_wait(&bar_empty[i % stages], (uint32_t)((i / stages) - 1) & 1u, &abort_flag, a.limit_ns);
        if (!ok) break;
        load_w(i);
        if constexpr (!OWN) load_x(i);
      }
      if (!ok) {
        abort_flag = 1;
        report_error(-6);
      }
      // drain: every issued load lands before the CTA may exit
      for (int j = max(0, i - stages); j < i; ++j)
        mbar_wait(&bar_full[j % stages], (uint32_t)(j / stages) & 1u, &never_abort, a.limit_ns);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      // ================= MMA =================
      // One thread issues them all, so its instructions per stage count: descriptors as low words
      // (the high word is common), slot and phase kept as they go (1,000 clocks a stage without
      // that, 850 with it; the MMAs take 450)
      const uint64_t d0 = smem_desc(smem_u32(sm), 16, 1024, SW_128B);
      const uint32_t hi = (uint32_t)(d0 >> 32), own_lo = (uint32_t)smem_desc(smem_u32(own), 16, 1024, SW_128B);
      const int last = KS - 4 * (kb0 + n - 1);       // k-steps of the last stage, if fewer than 4
      bool ok = true;
      uint32_t ph = 0;
      int s = 0;
      for (int i = 0; i < n; ++i) {
        ok = mbar_wait(&bar_full[s], ph, &abort_flag, a.limit_ns) && mbar_wait(&bar_sf[s], ph, &abort_flag, a.limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t wlo = (uint32_t)d0 + s * (stage_bytes >> 4), xlo = OWN ? own_lo + i * (M * P * 128 >> 4) : wlo + ((kGvBBytes + kGvSfBytes) >> 4);
        const uint32_t tsf = tb + 288u + 32u * s;
        const int steps = i + 1 < n ? 4 : last;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          if (kk < steps)
            mma_nvf4_lo(tb, xlo + 2u * kk, wlo + 2u * kk, hi, kNvIdesc, tb + 256u, tsf + kk * 8u, (i | kk) != 0 ? 1u : 0u);
        mma_commit(&bar_empty[s]);
        if (++s == stages) s = 0, ph ^= 1u;
      }
      if (ok) mma_commit(&bar_acc);
      if (!ok) {
        abort_flag = 1;
        report_error(-6);
      }
      // drain: every issued MMA completes before TMEM is released
      mma_commit(&bar_drain);
      mbar_wait(&bar_drain, 0, &never_abort, a.limit_ns);
    }
    __syncwarp();
  } else {
    // ================= scales to TMEM: stages in turn =================
    const int quarter = warp & 3, set = (warp - 2) >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    asm volatile("griddepcontrol.wait;" ::: "memory");                 // the digits and exponents are complete
    if constexpr (OWN) {
      // the largest elements: 8 / M warps a row
      const uint32_t w = warp - 2, per_row = 8u / (uint32_t)M;
      if (w < per_row * M) {
        const int m = w % (uint32_t)M;
        uint32_t top = 0, bad = 0;
        gemv_row_max(reinterpret_cast<const uint4*>(a.x + m * a.ldx), (int)(w / (uint32_t)M) * 32 + lane, a.K / 8,
                     (int)per_row * 32, top, bad);
        if (lane == 0) {
          atomicMax(&s_top[m], top);
          atomicOr(&s_bad[m], bad);
        }
      }
      asm volatile("bar.arrive 2, 288;" ::: "memory");
      asm volatile("bar.sync 1, 256;" ::: "memory");
      info = gemv_ref(s_top[min(lane, M - 1)], s_bad[min(lane, M - 1)]);
      // digits of this CTA's range, a row of 256 elements by a warp
      for (int q = (int)w; q < n * M; q += 8) {
        const int i = q / M, m = q - i * M, k = (kb0 + i) * 256 + lane * 8;
        const int f = __shfl_sync(0xffffffffu, info, m), e = 21 + 127 - (f & 0xFFFF);
        const uint4 v = k < a.K ? *reinterpret_cast<const uint4*>(a.x + m * a.ldx + k) : make_uint4(0, 0, 0, 0);
        uint32_t word[P];
        gemv_digits8<P>(f & kGvBadRow ? finite_only(v) : v, pow2f(e >> 1), pow2f(e - (e >> 1)), word);
        uint8_t* dst = own + (i * M + m) * (P * 128) + (lane & 3) * 4;
#pragma unroll
        for (int d = 0; d < P; ++d)   // the 16-byte pieces in the MMA's 128-byte swizzle
          *reinterpret_cast<uint32_t*>(dst + d * 128 + (((lane >> 2) ^ (d & 7)) << 4)) = word[d];
      }
      fence_proxy_async_smem();
      asm volatile("bar.sync 1, 256;" ::: "memory");
    } else {
      info = a.ref[min(lane, M - 1)];
    }
    if (set == 0) {
      uint32_t one[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) one[i] = 0x38383838u;               // E4M3 1.0
      tmem_st16(tb + lanes + 256u, one);
    }
    bool ok = true;
    int slot = stages - 1;
    uint32_t ph = 1;
    for (int i = 0; i < n; ++i) {
      if (++slot == stages) slot = 0, ph ^= 1u;
      const int s = slot, steps = min(4, KS - 4 * (kb0 + i));
      ok = warp_wait(&bar_full[s], ph, &abort_flag, a.limit_ns);
      if (!ok) break;
      if ((i & 1) != set) {
        // The other set's: this one only keeps up with the phases.  The slot may not be filled again
        // before it has, as a phase's parity does not show a turn of the ring.  (A set holds back its
        // own stages by bar_sf, which the MMA waits for.)
        if (lane == 0) mbar_arrive(&bar_empty[s]);
        continue;
      }
      const uint4* sf = reinterpret_cast<const uint4*>(sm + s * stage_bytes + kGvBBytes) + lane;
      uint32_t v[32];
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 t = make_uint4(0, 0, 0, 0);
          if (kk < steps && (h == 0 || has1)) t = sf[h * 128 + kk * 32];
          v[kk * 8 + h * 4] = t.x;
          v[kk * 8 + h * 4 + 1] = t.y;
          v[kk * 8 + h * 4 + 2] = t.z;
          v[kk * 8 + h * 4 + 3] = t.w;
        }
      tmem_st32(tb + lanes + 288u + (uint32_t)s * 32u, v);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_sf[s]);
    }
    // ================= sums: digit rows -> shared memory =================
    if (ok) ok = warp_wait(&bar_acc, 0, &abort_flag, a.limit_ns);
    if (!ok) {
      abort_flag = 1;
      report_error(-6);
    }
    tc_fence_after();
    if (ok && quarter * 32 < rows) {
#pragma unroll 1
      for (int c = 128 * set; c < 128 * set + 128; c += 64) {
        uint32_t v[2][32];
        tmem_ld32(tb + lanes + (uint32_t)c, v[0]);
        tmem_ld32(tb + lanes + (uint32_t)c + 32u, v[1]);
        tmem_wait_ld();
        reg_fence32(v[0]);
        reg_fence32(v[1]);
        // lane r writes row r: a turn of the 16-byte pieces keeps the banks apart
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4* dst = reinterpret_cast<uint4*>(dsum + (quarter * 32 + lane) * 256 + c + 32 * h);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j ^ (lane & 7)] = make_uint4(v[h][4 * j], v[h][4 * j + 1], v[h][4 * j + 2], v[h][4 * j + 3]);
        }
      }
    }
  }
  // ================= one fp32 per output, by all warps =================
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kGvTmemCols);
  }
  if (warp >= 2) {
    // four columns of every fourth row of x a thread
    const int col = 4 * ((threadIdx.x - 64) & 63);
    for (int m = (threadIdx.x - 64) >> 6; m < M; m += 4) {
      const int f = __shfl_sync(0xffffffffu, info, m), e = (f & 0xFFFF) - 127;
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < P / 8; ++h) {   // the low digits first
        const float* row = dsum + (m * P + 8 * h) * 256;
        float4 x[8];                      // digit d (row 8 i + d): piece (col / 4) ^ d of its row
#pragma unroll
        for (int d = 0; d < 8; ++d) x[d] = *reinterpret_cast<const float4*>(row + d * 256 + (((col >> 2) ^ d) << 2));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u = 0.f;
#pragma unroll
          for (int d = 7; d >= 0; --d) u = fmaf(u, 8.f, i == 0 ? x[d].x : i == 1 ? x[d].y : i == 2 ? x[d].z : x[d].w);
          v[i] = fmaf(v[i], 0x1p-21f, u);
        }
      }
      const float a1 = pow2f(e >> 1), a2 = pow2f(e - (e >> 1) - 21);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] * a1 * a2;
      *reinterpret_cast<float4*>(part + m * 256 + col) = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (__any_sync(0xffffffffu, lane < M && (info & kGvBadRow)))   // (the same for all warps)
      asm volatile("bar.sync 1, 256;" ::: "memory");               // a thread reads what its neighbours wrote
    // elements of x that are not finite: their products, one by one
    for (uint32_t bad = __ballot_sync(0xffffffffu, lane < M && (info & kGvBadRow)); bad; bad &= bad - 1) {
      const int m = __ffs(bad) - 1;
      const int col = threadIdx.x - 64;
      const long long nr = (long long)tile * 256 + col;
      if (nr >= a.N) continue;
      const int end = min((kb0 + n) * 256, a.K), row = col & 127;
      const uint8_t* sf = a.wsf + (nr / 128) * KS * 512 + (row % 32) * 16 + (row / 32) * 4;
      float v = part[m * 256 + col];
      for (int k = kb0 * 256; k < end; ++k) {
        const float xv = __bfloat162float(a.x[m * a.ldx + k]);
        if (fabsf(xv) < INFINITY) continue;
        const uint32_t c = (a.wc[nr * (a.K / 2) + k / 2] >> (4 * (k & 1))) & 15u, mag = c & 7u;
        float wv = mag < 4 ? 0.5f * mag : (mag < 6 ? (float)(mag - 2) : 2.f * (mag - 4));
        wv *= e4m3_to_f32(sf[(k / 64) * 512 + (k / 16) % 4]);
        v = fmaf(xv, (c & 8u) ? -wv : wv, v);
      }
      part[m * 256 + col] = v;
    }
  }
  // every CTA of the cluster adds a share of the outputs, four at a time, in rank order
  asm volatile("griddepcontrol.wait;" ::: "memory");   // for the warps that have not waited yet
  cluster_sync();
  const float gw = *a.gw;
  const uint32_t base = smem_u32(part);
  for (int o = (int)(rank * kGvThreads + threadIdx.x); o < M * 64; o += (int)ranks * kGvThreads) {
    float4 v[kGvSplit];
#pragma unroll
    for (uint32_t r = 0; r < kGvSplit; ++r) {
      if (r >= ranks) break;
      uint32_t at;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + 16u * (uint32_t)o), "r"(r));
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[r].x), "=f"(v[r].y), "=f"(v[r].z), "=f"(v[r].w)
                   : "r"(at)
                   : "memory");
    }
    float s[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (uint32_t r = 1; r < kGvSplit; ++r) {
      if (r >= ranks) break;
      s[0] += v[r].x;
      s[1] += v[r].y;
      s[2] += v[r].z;
      s[3] += v[r].w;
    }
    const long long first = (long long)tile * 256 + 4 * (o & 63);
    __nv_bfloat16* y = a.y + (o >> 6) * a.ldy + first;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < a.N) y[i] = __float2bfloat16(__fadd_rn(__fmul_rn(s[i], gw), a.bias ? a.bias[first + i] : 0.f));
  }
  // no CTA leaves while another may still read its sums
  cluster_sync();
}

}  // namespace lx
