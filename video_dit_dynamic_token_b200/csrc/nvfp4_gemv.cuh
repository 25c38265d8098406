// Products of few bf16 rows with NVFP4 weights (lx_nvfp4_gemv):
//
//   y[m, n] = bf16(fl32(acc * gw) + bias[n]),  acc = sum_k x[m, k] e2m1(w[n, k]) e4m3(s[n, k / 16])
//
// for M <= 16 rows, x kept in bf16 precision (the modulation vectors of a
// timestep, a guided pair, single new tokens).  The weights are read once: N K / 2
// bytes of codes and N K / 16 of scales, which is what bounds it.
//
// Decoding 4-bit weights costs more issue slots than an SM has at the rate they
// arrive (42 weights per clock; mma.sync on weights decoded to fp16 took 38 to 55 us
// for 30720 x 5120, the format's conversion instruction or 5 instructions per weight
// bounding it), so the block-scaled tensor core reads the codes as they are, and x
// takes the weights' format: each row becomes 8 rows of signed octal digits.
//
// Digits.  Within a block of 16 along k, whose largest finite magnitude lies in
// [2^e, 2^(e+1)), x = X 2^(e-21) with an integer |X| <= 2^22 (x has 8 significant
// bits: elements down to 2^-14 of the largest are exact, smaller ones are rounded by at
// most 2^(e-22)).  X = sum_i d_i 8^i with d_i in {-4 .. 3}, read off the octal digits
// of X + 44444444 (octal); every d_i is an E2M1 value, and the block's scale 2^(e - ref + 8)
// an E4M3 one, ref the exponent of the row's largest element (blocks more than
// 2^17 below it use the smallest scale; their rounding is 2^(ref-39)).  So
//   acc = 2^(ref-29) sum_i 8^i D_i,  D_i = sum_k (w s) (d_i 2^(e-ref+8))
// with D_i the fp32 sums of one MMA column each: 8 M columns.  Elements that are not
// finite have zero digits; the rows that hold them add x w for those k in the epilogue.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "attn.cuh"
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace lx {

constexpr int kGvMaxRows = 16;                // rows of x
constexpr int kGvSplit = 8;                   // most CTAs that share a row tile's K (a cluster)
constexpr int kGvSlice = 1024;                // elements of x per CTA of the digit pass
constexpr uint32_t kGvABytes = 128 * 128;     // stage: 128 weight rows x 256 codes
constexpr uint32_t kGvSfBytes = 4 * 512;      // their scales; as many for the digits

// columns of the MMA (a multiple of 16) and what follows from them
__host__ __device__ constexpr int gemv_cols(int M) { return (8 * M + 15) / 16 * 16; }
__host__ __device__ constexpr uint32_t gemv_stage(int cols) { return kGvABytes + 2 * kGvSfBytes + 128u * (uint32_t)cols; }
// two CTAs share an SM: 4 stages of 22 to 26 KB up to 48 columns, 3 of up to 36 KB beyond
__host__ __device__ constexpr int gemv_stages(int cols) { return cols <= 48 ? 4 : 3; }
__host__ __device__ constexpr uint32_t gemv_smem(int cols) { return 1024 + (uint32_t)gemv_stages(cols) * gemv_stage(cols); }

// ref of a row as the digit pass leaves it: biased exponent, bit 16 set when the row
// holds an element that is not finite
constexpr int kGvBadRow = 1 << 16;

struct GemvArgs {
  const __nv_bfloat16* x;
  const uint8_t* wc;
  const uint8_t* wsf;
  const uint8_t* xsf;   // scales of the digits, tiled like the weights'
  const int* ref;       // [M]
  const float* gw;
  const float* bias;
  __nv_bfloat16* y;
  long long ldx, ldy, N;
  int M, K, per;        // per: 256-element stages of a CTA
  unsigned long long limit_ns;
};

__device__ __forceinline__ float pow2f(int e) {  // 2^e, -149 <= e <= 127
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

// ---------------------------------------------------------------- digits of x
// grid (M, ceil(K / kGvSlice)), 128 threads of 8 elements.  Every CTA reads the whole
// row (it is short) for the row's largest element.
__global__ void __launch_bounds__(128) nvfp4_gemv_digits_kernel(const __nv_bfloat16* __restrict__ x, long long ldx, int K,
                                                                uint8_t* __restrict__ codes, uint8_t* __restrict__ sf,
                                                                int* __restrict__ ref) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the weights may start to load
  const int m = blockIdx.x;
  const uint4* row = reinterpret_cast<const uint4*>(x + m * ldx);
  uint32_t top = 0, bad = 0;
#pragma unroll 4
  for (int v = threadIdx.x; v < K / 8; v += 128) {
    const uint4 t = row[v];
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      if (lo < 0x7F80u) top = max(top, lo); else bad = 1;
      if (hi < 0x7F80u) top = max(top, hi); else bad = 1;
    }
  }
  __shared__ uint32_t s_top, s_bad;
  if (threadIdx.x == 0) s_top = 0, s_bad = 0;
  __syncthreads();
  top = __reduce_max_sync(0xffffffffu, top);
  bad = __reduce_or_sync(0xffffffffu, bad);
  if ((threadIdx.x & 31) == 0) {
    atomicMax(&s_top, top);
    atomicOr(&s_bad, bad);
  }
  __syncthreads();
  const int eref = max(1, (int)(s_top >> 7));
  if (blockIdx.y == 0 && threadIdx.x == 0) ref[m] = eref | (s_bad ? kGvBadRow : 0);

  const int k = blockIdx.y * kGvSlice + threadIdx.x * 8;
  const bool live = k < K;
  const uint4 t = live ? row[k / 8] : make_uint4(0, 0, 0, 0);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
  uint32_t b[8];
  uint32_t big = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    b[i] = (w[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    if ((b[i] & 0x7FFFu) >= 0x7F80u) b[i] = 0;
    big = max(big, b[i] & 0x7FFFu);
  }
  big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));             // the block's other 8 elements
  const int e = max(max(1, (int)(big >> 7)), eref - 17);
  uint32_t word[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ex = (b[i] >> 7) & 0xFF, sh = 14 - (e - max(1, ex));
    const int mant = (b[i] & 0x7F) | (ex ? 0x80 : 0);
    int X = sh >= 0 ? mant << sh : (sh > -10 ? (mant + (1 << (-sh - 1))) >> -sh : 0);
    X = (b[i] & 0x8000u) ? -X : X;
    const uint32_t o = (uint32_t)(X + 044444444);
#pragma unroll
    for (int d = 0; d < 8; ++d)                                      // codes of -4 .. 3
      word[d] |= ((0x5420ACDEu >> (((o >> (3 * d)) & 7u) * 4)) & 15u) << (4 * i);
  }
  if (!live) return;
  const int se = 8 + e - eref;                                       // scale 2^se, -9 <= se <= 8
  const uint8_t s8 = (uint8_t)(se >= -6 ? (se + 7) << 3 : 1 << (se + 9));
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    const int r = m * 8 + d;
    *reinterpret_cast<uint32_t*>(codes + (long long)r * (K / 2) + k / 2) = word[d];
    if ((threadIdx.x & 1) == 0) sf[(long long)(k / 64) * 512 + (r % 32) * 16 + (r / 32) * 4 + (k / 16) % 4] = s8;
  }
}

// ---------------------------------------------------------------- products
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// One CTA: 128 weight rows (the MMA's rows) against the digit columns over a range
// of K; the CTAs of a cluster split K and add their sums over distributed shared
// memory, in rank order.  Stages of 256 codes go through a ring: warp 0 loads
// (the weights do not wait for the digit pass), warp 1 copies the scales into TMEM
// and issues the MMAs, warps 2 .. 5 read the sums, thread = weight row.
constexpr int kGvThreads = 192;
constexpr uint32_t kGvTmemCols = 256;   // sums 0 .. 127; scales 128 + 32 per stage

__global__ void __launch_bounds__(kGvThreads, 2) nvfp4_gemv_kernel(const __grid_constant__ CUtensorMap tmW,
                                                                   const __grid_constant__ CUtensorMap tmX,
                                                                   const GemvArgs a) {
  extern __shared__ uint8_t gv_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(gv_smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t bar_full[4], bar_empty[4], bar_acc, bar_drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int never_abort;
  float* part = reinterpret_cast<float*>(sm);   // sums [row of x][128], in place of the stages once they are used

  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cols = gemv_cols(a.M), stages = gemv_stages(cols);
  const uint32_t stage_bytes = gemv_stage(cols), b_bytes = 128u * (uint32_t)cols;
  const int KS = a.K / 64, nkb = (KS + 3) / 4;
  const int kb0 = min((int)rank * a.per, nkb), kb1 = min(kb0 + a.per, nkb), n = kb1 - kb0;
  const int tile = (int)(blockIdx.x / ranks);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    mbar_init(&bar_acc, 1);
    mbar_init(&bar_drain, 1);
    abort_flag = 0;
    never_abort = 0;
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

  if (warp == 0) {
    if (lane == 0) {
      // ================= loads =================
      prefetch_tensormap(&tmW);
      prefetch_tensormap(&tmX);
      auto steps = [&](int kb) { return min(4, KS - 4 * kb); };      // k-steps of 64 in a stage
      auto load_w = [&](int i) {
        const int s = i % stages, kb = kb0 + i;
        uint8_t* st = sm + s * stage_bytes;
        const uint32_t sfb = (uint32_t)steps(kb) * 512u;
        mbar_arrive_expect_tx(&bar_full[s], kGvABytes + b_bytes + 2 * sfb);
        tma_load_2d(st, &tmW, &bar_full[s], kb * 128, tile * 128);
        bulk_load(st + kGvABytes, a.wsf + ((long long)tile * KS + kb * 4) * 512, sfb, &bar_full[s]);
      };
      auto load_x = [&](int i) {
        const int s = i % stages, kb = kb0 + i;
        uint8_t* st = sm + s * stage_bytes + kGvABytes + kGvSfBytes;
        bulk_load(st, a.xsf + (long long)kb * 4 * 512, (uint32_t)steps(kb) * 512u, &bar_full[s]);
        tma_load_2d(st + kGvSfBytes, &tmX, &bar_full[s], kb * 128, 0);
      };
      const int first = min(n, stages);
      for (int i = 0; i < first; ++i) load_w(i);
      asm volatile("griddepcontrol.wait;" ::: "memory");              // the digits are complete
      for (int i = 0; i < first; ++i) load_x(i);
      bool ok = true;
      int i = first;
      for (; i < n; ++i) {
        ok = mbar_wait(&bar_empty[i % stages], (uint32_t)((i / stages) - 1) & 1u, &abort_flag, a.limit_ns);
        if (!ok) break;
        load_w(i);
        load_x(i);
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
      // ================= scales -> TMEM, MMA =================
      // block-scaled instruction: A, B = E2M1 (1), K-major, UE4M3 scales, 128 rows x cols
      const uint32_t idesc = (1u << 7) | (1u << 10) | ((uint32_t)(cols >> 3) << 17) | (8u << 24);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        const int s = i % stages, steps = min(4, KS - 4 * (kb0 + i));
        ok = mbar_wait(&bar_full[s], (uint32_t)(i / stages) & 1u, &abort_flag, a.limit_ns);
        if (!ok) break;
        tc_fence_after();
        const uint32_t st = smem_u32(sm + s * stage_bytes);
        const uint32_t sfa = st + kGvABytes, sfb = sfa + kGvSfBytes, bt = sfb + kGvSfBytes;
        for (int kk = 0; kk < steps; ++kk) {
          const uint32_t ta = tb + 128u + (uint32_t)s * 32u + (uint32_t)kk * 4u, tx = ta + 16u;
          tmem_cp_32x128b_x4(ta, smem_desc(sfa + kk * 512u, 128, 128, SW_NONE));
          tmem_cp_32x128b_x4(tx, smem_desc(sfb + kk * 512u, 128, 128, SW_NONE));
          mma_nvf4(tb, smem_desc(st + kk * 32u, 16, 1024, SW_128B), smem_desc(bt + kk * 32u, 16, 1024, SW_128B), idesc, ta,
                   tx, (i | kk) != 0 ? 1u : 0u);
        }
        mma_commit(&bar_empty[s]);
      }
      if (ok && n > 0) mma_commit(&bar_acc);
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
    // ================= sums: 8 digit columns of a row -> one fp32 =================
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int row = (warp & 3) * 32 + lane;
    const uint32_t taddr = tb + ((uint32_t)((warp & 3) * 32) << 16);
    bool ok = n == 0 || warp_wait(&bar_acc, 0, &abort_flag, a.limit_ns);
    if (!ok) {
      abort_flag = 1;
      report_error(-6);
    }
    tc_fence_after();
    const long long nr = (long long)tile * 128 + row;
    for (int m0 = 0; m0 < a.M; m0 += 2) {
      uint32_t d[16];
      if (n > 0 && ok) {
        tmem_ld16(taddr + 8 * m0, d);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(d[i]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int m = m0 + h;
        if (m >= a.M) break;
        const int info = a.ref[m], e = (info & 0xFFFF) - 127;
        float v = 0.f;
        if (n > 0 && ok) {
          v = __uint_as_float(d[8 * h + 7]);
#pragma unroll
          for (int i = 6; i >= 0; --i) v = fmaf(v, 8.f, __uint_as_float(d[8 * h + i]));
          v = v * pow2f(e >> 1) * pow2f(e - (e >> 1) - 29);
        }
        if ((info & kGvBadRow) && nr < a.N) {
          const long long end = min((long long)kb1 * 256, (long long)a.K);
          for (long long k = (long long)kb0 * 256; k < end; ++k) {
            const float xv = __bfloat162float(a.x[m * a.ldx + k]);
            if (fabsf(xv) < INFINITY) continue;
            const uint32_t c = (a.wc[nr * (a.K / 2) + k / 2] >> (4 * (k & 1))) & 15u, mag = c & 7u;
            const uint32_t s8 = a.wsf[((long long)tile * KS + k / 64) * 512 + (row % 32) * 16 + (row / 32) * 4 + (k / 16) % 4];
            float wv = mag < 4 ? 0.5f * mag : (mag < 6 ? (float)(mag - 2) : 2.f * (mag - 4));
            wv *= e4m3_to_f32(s8);
            v = fmaf(xv, (c & 8u) ? -wv : wv, v);
          }
        }
        part[m * 128 + row] = v;
      }
    }
  }
  tc_fence_before();
  cluster_sync();
  // every CTA of the cluster adds a share of the outputs, in rank order
  const float gw = *a.gw;
  const uint32_t base = smem_u32(part);
  for (int i = (int)(rank * kGvThreads + threadIdx.x); i < 128 * a.M; i += (int)ranks * kGvThreads) {
    const int m = i >> 7;
    const long long nr = (long long)tile * 128 + (i & 127);
    float s = 0.f;
    for (uint32_t r = 0; r < ranks; ++r) {
      uint32_t at;
      float v;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + 4u * (uint32_t)i), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
      s += v;
    }
    if (nr < a.N) a.y[m * a.ldy + nr] = __float2bfloat16(__fadd_rn(__fmul_rn(s, gw), a.bias ? a.bias[nr] : 0.f));
  }
  // no CTA leaves while another may still read its sums
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, kGvTmemCols);
  }
}

}  // namespace lx
