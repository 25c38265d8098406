// Products of few bf16 rows with NVFP4 weights (lx_nvfp4_gemv):
//
//   y[m, n] = bf16(fl32(acc * gw) + bias[n]),  acc = sum_k x[m, k] e2m1(w[n, k]) e4m3(s[n, k / 16])
//
// for M <= 16 rows, x kept in bf16 precision (the modulation vectors of a
// timestep, a guided pair, single new tokens).  The weights are read once: N K / 2
// bytes of codes and N K / 16 of scales, which is what bounds it.
//
// Arithmetic.  A weight times its block scale, e2m1 (2 significant bits) times
// e4m3 (4), is exact in fp16, so a thread decodes two codes with one
// conversion, scales them with one HMUL2, and mma.sync m16n8k16 multiplies 16
// weight rows by 8 (NT = 1) or 16 (NT = 2) columns of x with fp32 sums; the
// tensor core is idle most of the time, it only saves the issue slots that
// fp32 FMAs per weight and row would take.  x is put into fp16 by a power of
// two per row and 128 elements that brings the largest of them to [2^14, 2^15):
// its 8 significant bits fit, and elements more than 2^28 below that largest
// one lose bits (by less than 2^-39 of it).  The power is taken out again in
// fp32 after the chunk.
//
// Layout.  A CTA of 8 warps owns 128 weight rows (one tile of the scale layout)
// and a range of K; the CTAs of a cluster split K and add their fp32 sums over
// distributed shared memory, in rank order.  A warp owns 16 rows: those whose
// scales lie in 64 neighbouring bytes, rows 32 c + 4 w .. 4 w + 3, c = 0 .. 3.
// Thread (g, q) of a warp (g = lane / 4, q = lane % 4) holds codes
// [32 q, 32 q + 32) of a 128-element chunk of its two rows, one 16-byte load
// each: MMA step s takes its codes 4 s .. 4 s + 3, so k is permuted, the same way
// for x, whose fp16 copy in shared memory is laid out in fragment order.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include "nvfp4.cuh"
#include "ptx.cuh"

namespace lx {

constexpr int kGvMaxRows = 16;   // rows of x
constexpr int kGvSeg = 32;       // chunks of x staged at a time (divided by NT)
constexpr int kGvAhead = 4;      // chunks of weights in flight per thread
constexpr int kGvSplit = 8;      // most CTAs that share a row tile's K

struct GemvArgs {
  const __nv_bfloat16* x;
  const uint8_t* wc;
  const uint8_t* wsf;
  const float* gw;
  const float* bias;
  __nv_bfloat16* y;
  long long ldx, ldy, N;
  int M, K, per;        // per: 128-element chunks of a CTA
};

// Two E2M1 codes (byte b of w, low nibble first) as fp16.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 b0, b1, b2, b3;\n mov.b32 {b0, b1, b2, b3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, b0;\n cvt.rn.f16x2.e2m1x2 %1, b1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, b2;\n cvt.rn.f16x2.e2m1x2 %3, b3;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t s) {
  uint32_t h;
  asm("{\n .reg .b16 a;\n cvt.u16.u32 a, %1;\n cvt.rn.f16x2.e4m3x2 %0, a;\n}" : "=r"(h) : "r"(s));
  return h;
}
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldg_stream_v4(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ float pow2f(int e) {  // 2^e, -149 <= e <= 127
  return e >= -126 ? __uint_as_float((uint32_t)(e + 127) << 23) : __uint_as_float(1u << (e + 149));
}

template <int NT>
struct GemvSmem {
  static constexpr int SEG = kGvSeg / NT;
  static constexpr int X_BYTES = SEG * 128 * 8 * NT * 2;   // fragments of x
  static constexpr int S_OFF = X_BYTES;                     // 2^-shift [chunk][row]
  static constexpr int P_OFF = S_OFF + SEG * 8 * NT * 4;    // partial sums [row of x][128]
  static constexpr int BYTES = P_OFF + 128 * 8 * NT * 4;
};

struct GemvChunk {
  uint4 a, b;        // codes of the two rows
  uint32_t sa, sb;   // two E4M3 scales each
};

template <int NT>
__global__ void __launch_bounds__(256) nvfp4_gemv_kernel(const GemvArgs p) {
  using S = GemvSmem<NT>;
  constexpr int M8 = 8 * NT;
  extern __shared__ __align__(16) uint8_t gv_smem[];
  uint4* xs = reinterpret_cast<uint4*>(gv_smem);
  float* sx = reinterpret_cast<float*>(gv_smem + S::S_OFF);
  float* part = reinterpret_cast<float*>(gv_smem + S::P_OFF);

  uint32_t rank, ranks;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
  const long long tile = blockIdx.x / ranks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int KS = p.K / 64, nch = (p.K + 127) / 128;
  const int c_lo = min((int)rank * p.per, nch), c_hi = min(c_lo + p.per, nch);

  // this thread's two rows, and where their codes and scales lie
  const int ra = 32 * (g >> 2) + 4 * warp + (g & 3);
  const long long na = min(tile * 128 + ra, p.N - 1), nb = min(tile * 128 + ra + 64, p.N - 1);
  const uint8_t* pa = p.wc + na * (p.K / 2) + q * 16;
  const uint8_t* pb = p.wc + nb * (p.K / 2) + q * 16;
  const uint8_t* ps = p.wsf + (tile * KS + (q >> 1)) * 512 + (4 * warp + (g & 3)) * 16 + (g >> 2) * 4 + (q & 1) * 2;

  auto load = [&](int c) {
    GemvChunk w{};
    if (c < c_hi && 2 * c + (q >> 1) < KS) {   // the last chunk may be half a chunk
      w.a = ldg_stream_v4(pa + (long long)c * 64);
      w.b = ldg_stream_v4(pb + (long long)c * 64);
      const uint8_t* s = ps + (long long)c * 1024;
      w.sa = __ldg(reinterpret_cast<const unsigned short*>(s));
      w.sb = __ldg(reinterpret_cast<const unsigned short*>(s + 8));
    }
    return w;
  };

  float acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;

  GemvChunk ring[kGvAhead];
#pragma unroll
  for (int i = 0; i < kGvAhead; ++i) ring[i] = load(c_lo + i);

  for (int seg = c_lo; seg < c_hi; seg += S::SEG) {
    const int n = min(S::SEG, c_hi - seg);
    if (seg != c_lo) __syncthreads();
    // stage x: half a warp per (chunk, row), 8 elements a lane
    for (int u = threadIdx.x >> 4; u < n * M8; u += 16) {
      const int c = u / M8, m = u % M8, gi = threadIdx.x & 15;
      const int k = (seg + c) * 128 + gi * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (m < p.M && k < p.K) v = *reinterpret_cast<const uint4*>(p.x + m * p.ldx + k);
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t top = 0;   // largest finite magnitude, as bf16 bits
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
        if (lo < 0x7F80u) top = max(top, lo);
        if (hi < 0x7F80u) top = max(top, hi);
      }
#pragma unroll
      for (int o = 8; o; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const int shift = 141 - max(1, (int)(top >> 7));    // top * 2^shift in [2^14, 2^15)
      const float f0 = pow2f(shift >> 1), f1 = pow2f(shift - (shift >> 1));
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 t = __floats2half2_rn(bf16lo(w[i]) * f0 * f1, bf16hi(w[i]) * f0 * f1);
        h[i] = *reinterpret_cast<const uint32_t*>(&t);
      }
      xs[((c * 4 + (gi & 3)) * M8 + m) * 4 + (gi >> 2)] = make_uint4(h[0], h[1], h[2], h[3]);
      if (gi == 0) sx[c * M8 + m] = pow2f(-shift);
    }
    __syncthreads();

    for (int c0 = 0; c0 < n; c0 += kGvAhead) {
#pragma unroll
      for (int i = 0; i < kGvAhead; ++i) {
        const int c = c0 + i;
        if (c >= n) break;
        const GemvChunk w = ring[i];
        ring[i] = load(seg + c + kGvAhead);
        const uint32_t ha = e4m3x2_to_f16(w.sa), hb = e4m3x2_to_f16(w.sb);
        const uint32_t sa[2] = {__byte_perm(ha, ha, 0x1010), __byte_perm(ha, ha, 0x3232)};
        const uint32_t sb[2] = {__byte_perm(hb, hb, 0x1010), __byte_perm(hb, hb, 0x3232)};
        const uint32_t wa[4] = {w.a.x, w.a.y, w.a.z, w.a.w}, wb[4] = {w.b.x, w.b.y, w.b.z, w.b.w};
        float d[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) d[t][e] = 0.f;
#pragma unroll
        for (int s2 = 0; s2 < 4; ++s2) {     // one word of each row: two MMA steps
          uint32_t fa[4], fb[4];
          e2m1x8_to_f16(wa[s2], fa);
          e2m1x8_to_f16(wb[s2], fb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fa[e] = hmul2_u(fa[e], sa[s2 >> 1]);
            fb[e] = hmul2_u(fb[e], sb[s2 >> 1]);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 xf = xs[((c * 4 + s2) * M8 + t * 8 + g) * 4 + q];
            mma_f16_16816(d[t], fa[0], fb[0], fa[1], fb[1], xf.x, xf.y);
            mma_f16_16816(d[t], fa[2], fb[2], fa[3], fb[3], xf.z, xf.w);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float2 f = *reinterpret_cast<const float2*>(&sx[c * M8 + t * 8 + 2 * q]);
          acc[t][0] = fmaf(d[t][0], f.x, acc[t][0]);
          acc[t][1] = fmaf(d[t][1], f.y, acc[t][1]);
          acc[t][2] = fmaf(d[t][2], f.x, acc[t][2]);
          acc[t][3] = fmaf(d[t][3], f.y, acc[t][3]);
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < NT; ++t) {
    part[(t * 8 + 2 * q) * 128 + ra] = acc[t][0];
    part[(t * 8 + 2 * q + 1) * 128 + ra] = acc[t][1];
    part[(t * 8 + 2 * q) * 128 + ra + 64] = acc[t][2];
    part[(t * 8 + 2 * q + 1) * 128 + ra + 64] = acc[t][3];
  }
  // every CTA of the cluster adds a share of the outputs, in rank order
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  const float gw = *p.gw;
  const uint32_t base = smem_u32(part);
  for (int i = (int)(rank * 256 + threadIdx.x); i < 128 * p.M; i += (int)(ranks * 256)) {
    const int m = i >> 7;
    const long long n = tile * 128 + (i & 127);
    float s = 0.f;
    for (uint32_t r = 0; r < ranks; ++r) {
      uint32_t at;
      float v;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(base + 4u * (uint32_t)i), "r"(r));
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
      s += v;
    }
    if (n < p.N) p.y[m * p.ldy + n] = __float2bfloat16(__fadd_rn(__fmul_rn(s, gw), p.bias ? p.bias[n] : 0.f));
  }
  // no CTA leaves while another may still read its sums
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace lx
