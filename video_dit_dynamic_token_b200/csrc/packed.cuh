// Attention over packed sequences (lx_attn_packed) and behind a shared prefix
// (lx_attn_prefix): bf16 operands, fp32 scores and statistics, tcgen05 + TMA + TMEM.
//
//   o_t = sum_u p_u v_u / sum_u p_u,  p_u = exp(scale q_t.k_u - m),
//   lse_t = m + log sum_u p_u,
// over the keys u that row t of its sequence sees: u < lk, and with the causal
// rule u <= t + lk - lq; behind a prefix, every prefix key as well.  A row
// that sees no key has o = 0 and lse = -inf.
//
// Rows of a tile: the G query heads of one key/value head are packed into the
// 128 rows of an MMA tile, row r = (token r / G, head r % G), TQ = 128 / G
// tokens a tile, so that grouped heads read K and V once and a single token
// still fills G rows.
//
// A work item is one CTA: NQ row tiles of one sequence (or of all tokens, for
// the prefix) against a range of 128-key tiles of one key/value head.
//   NQ = 2: prompts.  Two row tiles share each K/V tile; while one tile's
//           softmax runs, the tensor core works for the other.  One CTA per SM.
//   NQ = 1: few rows.  One row tile, two CTAs per SM, and the key range cut
//           into splits when there are fewer items than CTA slots; each split
//           leaves its unnormalised fp32 rows and (max, sum), and
//           packed_combine_kernel joins them.
//
// Roles: warps 0 .. 4 NQ - 1 softmax (thread = row; warpgroup g owns row tile
// g), then one TMA warp and one MMA warp.  TMEM: S_g (128 fp32 columns, reused
// for P as 64 columns of bf16 pairs) and O_g (D fp32 columns).  The MMA warp's
// order per key tile j is PV_g(j), S_g(j+1) for each g: S_g(j+1) may overwrite
// the columns of P_g(j) because the tensor core runs a CTA's MMAs in order, and
// the commit of S_g(j+1) also says that PV_g(j) is complete, so the softmax
// may rescale O_g without another barrier.
//
// The running maximum moves only when it grows by more than 2^8 (a shift that
// leaves the quotient unchanged: P stays below 256 and its bf16 rounding is
// relative), so O is rarely rescaled.  P is rounded to bf16, the type of V and
// of the output; the row sum takes the unrounded fp32 values.
//
// Values in masked places: scores are replaced by -inf by selection, and V rows
// past a sequence's end are zeroed in shared memory before they are used.  A
// key that the causal rule hides from some rows of a tile and not from others
// has P = 0 there, and 0 * V is NaN when V is not finite: a row that ends
// non-finite and has such keys is computed again by packed_exact_row.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include "attn.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace lx {

constexpr int kPkKeys = 128;         // keys of a tile
constexpr int kPkSplitKeys = 2;      // a split covers at least this many tiles
constexpr int kPkSlots = 2 * 148;    // CTA slots of a B200 at two CTAs per SM
constexpr float kPkLazy = 8.0f;      // log2 growth of the row maximum that forces a rescale

template <int D, int NQ>
struct PackCfg {
  static constexpr int NATOM = D / 64;                 // 128-byte swizzle atoms per row
  static constexpr int TILE_BYTES = 128 * D * 2;       // a Q, K or V tile
  // ring of K and V tiles: 5 x 32 KB beside 64 KB of Q (NQ = 2); 2 x 32 KB beside
  // 32 KB of Q in half an SM (NQ = 1); twice as many for D = 64
  static constexpr int RING = NQ == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 2 : 4);
  static constexpr int OFF_RING = NQ * TILE_BYTES;
  static constexpr int SMEM = 1024 + OFF_RING + RING * TILE_BYTES;
  static constexpr int WARPS = 4 * NQ + 2;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr uint32_t S_COL = 0;                 // + 128 g
  static constexpr uint32_t O_COL = 128 * NQ;          // + D g
  static constexpr uint32_t TMEM_COLS = 256 * NQ;
  static constexpr uint32_t IDESC_S = instr_desc(IDESC_DF32, IDESC_BF16, IDESC_BF16, 0, 0, 128, kPkKeys);
  static constexpr uint32_t IDESC_PV = instr_desc(IDESC_DF32, IDESC_BF16, IDESC_BF16, 0, 1, 128, D);
};

struct PackParams {
  const int32_t* cu_q;   // [n + 1] first query row of each sequence, then the end
  const int32_t* cu_k;   // [n + 1] the same for key rows
  const int32_t* len_k;  // [n] keys in use from cu_k[i] on, or null: all up to cu_k[i + 1]
  int n, Tq, Tk, Lp;     // sequences; rows of Q; rows of K and V; prefix keys (0: none)
  int G, Hkv, TQ, causal;
  float scale_log2;      // scale * log2(e)
  BhldView q, k, v;      // for packed_exact_row
  __nv_bfloat16* o;
  long long osH, osL;
  float* lse;            // [Hq][Tq] or null
  float* part;           // NQ = 1: [max_np + max_ns][Tq * Hq][D] unnormalised rows
  float2* ml;            // NQ = 1: [max_np + max_ns][Tq * Hq] (max, sum), max in the log2 domain
  int* chunk;            // NQ = 1: tiles per split, for the combine kernel
  int max_np, max_ns;    // most splits of the prefix, of a sequence
  unsigned long long limit_ns;
};

struct PackSeq {
  int q0, lq, k0, lk;
};

// Rows and keys of sequence i; a sequence whose entries do not fit the tensors is
// reported and left out (lq = 0).
__device__ __forceinline__ PackSeq pack_seq(const PackParams& p, int i) {
  const int a = p.cu_q[i], b = p.cu_q[i + 1], c = p.cu_k[i], d = p.cu_k[i + 1];
  PackSeq s{a, b - a, c, d - c};
  bool ok = a >= 0 && a <= b && b <= p.Tq && c >= 0 && c <= d && d <= p.Tk;
  if (p.len_k) {
    const int len = p.len_k[i];
    ok = ok && len >= 0 && len <= d - c;
    s.lk = len;
  }
  if (!ok) {
    report_error(-7);
    s = PackSeq{0, 0, 0, 0};
  }
  return s;
}

// The token range of all sequences (the rows that share the prefix).
__device__ __forceinline__ PackSeq pack_all(const PackParams& p) {
  const int a = p.cu_q[0], b = p.cu_q[p.n];
  if (a < 0 || a > b || b > p.Tq) {
    report_error(-7);
    return PackSeq{0, 0, 0, 0};
  }
  return PackSeq{a, b - a, 0, p.Lp};
}

__device__ __forceinline__ int pack_div(int a, int b) { return (a + b - 1) / b; }
__device__ __forceinline__ int pack_tiles(int keys) { return (keys + kPkKeys - 1) / kPkKeys; }
// number of splits of T key tiles at c tiles each, at least one and at most `most`
__device__ __forceinline__ int pack_splits(int T, int c, int most) { return max(1, min(most, pack_div(T, c))); }

struct PackItem {
  int q0, q_end;    // first token of the item, end of its sequence (rows of Q)
  int t0, off;      // its index in the sequence; causal: token t sees keys <= t + off
  int k0, lk;       // first key row, keys
  int lo, hi;       // key tiles [lo, hi)
  int head;         // key/value head
  int slot;         // where a partial result goes; -1: the item finishes its rows
  bool prefix;
};

// Block-wide inclusive scan of v (every thread calls it); total to *total.
template <int WARPS>
__device__ __forceinline__ int pack_scan(int v, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = s;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    const int x = warp_sums[w];
    if (w < warp) before += x;
    all += x;
  }
  *total = all;
  return s + before;
}

// Finds this CTA's item.  Every thread reads a share of the sequence table, so
// that lengths stay on the device; false: no item (the grid is an upper bound).
template <int NQ, int WARPS>
__device__ bool pack_find(const PackParams& p, PackItem* shared_item, int* warp_sums, int* found) {
  constexpr int T = 32 * WARPS;
  const int TT = NQ * p.TQ;
  if (threadIdx.x == 0) *found = 0;
  if constexpr (NQ == 2) {
    // one item per row tile pair, the last rows of the last sequence first: with
    // the causal rule the long items start first
    const int x = blockIdx.x;
    int run = 0;
    for (int base = 0; base < p.n; base += T) {
      const int i = p.n - 1 - base - (int)threadIdx.x;
      const PackSeq s = i >= 0 ? pack_seq(p, i) : PackSeq{0, 0, 0, 0};
      const int mine = pack_div(s.lq, TT);
      int total;
      const int incl = pack_scan<WARPS>(mine, warp_sums, &total);
      const int r = x - run - (incl - mine);
      if (r >= 0 && r < mine) {
        const int tile = mine - 1 - r;
        PackItem it;
        it.t0 = tile * TT;
        it.q0 = s.q0 + it.t0;
        it.q_end = s.q0 + s.lq;
        it.off = s.lk - s.lq;
        it.k0 = s.k0;
        it.lk = s.lk;
        it.lo = 0;
        it.hi = pack_tiles(s.lk);
        it.head = blockIdx.y;
        it.slot = -1;
        it.prefix = false;
        *shared_item = it;
        *found = 1;
      }
      run += total;
      if (x < run) break;
    }
  } else {
    // items of one key/value head: prefix tiles x splits, then each sequence's
    // tiles x splits; the split length c follows from the total work, so that
    // the items fill the CTA slots
    __shared__ unsigned long long work;
    __shared__ int items, longest;
    if (threadIdx.x == 0) work = 0, items = 0, longest = 0;
    __syncthreads();
    {
      unsigned long long w = 0;
      int m = 0, l = 0;
      for (int i = threadIdx.x; i < p.n; i += T) {
        const PackSeq s = pack_seq(p, i);
        const int a = pack_div(s.lq, TT), t = pack_tiles(s.lk);
        w += (unsigned long long)a * t;
        m += a;
        if (a) l = max(l, t);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      m = __reduce_add_sync(0xffffffffu, m);
      l = __reduce_max_sync(0xffffffffu, l);
      if ((threadIdx.x & 31) == 0) {
        atomicAdd(&work, w);
        atomicAdd(&items, m);
        atomicMax(&longest, l);
      }
    }
    __syncthreads();
    const PackSeq all = p.Lp ? pack_all(p) : PackSeq{0, 0, 0, 0};
    const int pa = pack_div(all.lq, TT), pt = pack_tiles(p.Lp);
    const int slots = max(1, kPkSlots / p.Hkv);          // of one head
    const int n_items = items + pa, share = 2 * n_items <= slots ? slots - n_items : slots;
    const unsigned long long n_work = work + (unsigned long long)pa * pt;
    int c = (int)((n_work + share - 1) / share);
    c = max(max(c, kPkSplitKeys), pack_div(longest, p.max_ns));
    if (p.Lp) c = max(c, pack_div(pt, p.max_np));
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.chunk) *p.chunk = c;
    const int np = p.Lp ? pack_splits(pt, c, p.max_np) : 0;
    const int head = blockIdx.x % p.Hkv;
    int x = blockIdx.x / p.Hkv;
    if (x < pa * np) {
      if (threadIdx.x == 0) {
        const int tile = x / np, sp = x % np, per = pack_div(pt, np);
        PackItem it;
        it.t0 = tile * TT;
        it.q0 = all.q0 + it.t0;
        it.q_end = all.q0 + all.lq;
        it.off = 0;
        it.k0 = 0;
        it.lk = p.Lp;
        it.lo = min(sp * per, pt);
        it.hi = min(it.lo + per, pt);
        it.head = head;
        it.slot = sp;
        it.prefix = true;
        *shared_item = it;
        *found = 1;
      }
    } else {
      x -= pa * np;
      int run = 0;
      for (int base = 0; base < p.n; base += T) {
        const int i = base + (int)threadIdx.x;
        const PackSeq s = i < p.n ? pack_seq(p, i) : PackSeq{0, 0, 0, 0};
        const int a = pack_div(s.lq, TT), t = pack_tiles(s.lk), ns = pack_splits(t, c, p.max_ns);
        const int mine = (p.Lp && t == 0) ? 0 : a * ns;  // behind a prefix a sequence may have no keys of its own
        int total;
        const int incl = pack_scan<WARPS>(mine, warp_sums, &total);
        const int r = x - run - (incl - mine);
        if (r >= 0 && r < mine) {
          const int tile = r / ns, sp = r % ns, per = pack_div(t, ns);
          PackItem it;
          it.t0 = tile * TT;
          it.q0 = s.q0 + it.t0;
          it.q_end = s.q0 + s.lq;
          it.off = s.lk - s.lq;
          it.k0 = s.k0;
          it.lk = s.lk;
          it.lo = min(sp * per, t);
          it.hi = min(it.lo + per, t);
          it.head = head;
          it.slot = (p.Lp || ns > 1) ? np + sp : -1;
          it.prefix = false;
          *shared_item = it;
          *found = 1;
        }
        run += total;
        if (x < run) break;
      }
    }
  }
  __syncthreads();
  return *found != 0;
}

// One row over keys [lo, hi), a warp together: lane holds D / 32 neighbouring
// channels.  Returns the unnormalised row, its maximum (log2 domain) and sum.
template <int D>
__device__ __noinline__ void packed_exact_row(const __nv_bfloat16* q, const __nv_bfloat16* k, long long ksL,
                                              const __nv_bfloat16* v, long long vsL, int lo, int hi, float scale_log2,
                                              float (&o)[D / 32], float& m, float& l) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  float qf[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qf[e] = __bfloat162float(q[lane * E + e]);
    o[e] = 0.f;
  }
  m = -INFINITY;
  l = 0.f;
  for (int u = lo; u < hi; ++u) {
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(qf[e], __bfloat162float(k[u * ksL + lane * E + e]), s);
#pragma unroll
    for (int w = 16; w; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    s *= scale_log2;
    const float mn = fmaxf(m, s), at = mn == -INFINITY ? 0.f : mn;
    const float a = m == -INFINITY ? 0.f : ex2f(m - at), x = ex2f(s - at);
    l = fmaf(l, a, x);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = fmaf(x, __bfloat162float(v[u * vsL + lane * E + e]), o[e] * a);
    m = mn;
  }
}

__device__ __forceinline__ float pack_lse(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

template <int D, int NQ>
__global__ void __launch_bounds__(PackCfg<D, NQ>::THREADS, NQ == 1 ? 2 : 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKp,
                       const __grid_constant__ CUtensorMap tmVp, const PackParams p) {
  using C = PackCfg<D, NQ>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // full/empty: a ring slot; sfull[g]: S_g complete; pfull[g]: P_g written; odone[g]: O_g complete
  __shared__ uint64_t bar_q, bar_full[C::RING], bar_empty[C::RING], bar_sfull[NQ], bar_pfull[NQ], bar_odone[NQ],
      bar_drain;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ int never_abort, found;
  __shared__ int warp_sums[C::WARPS];
  __shared__ PackItem item;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (!pack_find<NQ, C::WARPS>(p, &item, warp_sums, &found)) return;
  const PackItem it = item;

  // key tiles of each row tile: up to the last key that its last token sees
  int nt[NQ];
  int most = 0;
#pragma unroll
  for (int g = 0; g < NQ; ++g) {
    const int first = g * p.TQ, tokens = min(p.TQ, it.q_end - it.q0 - first);
    int hi = it.hi;
    if (p.causal && !it.prefix) hi = min(hi, pack_tiles(max(0, min(it.lk, it.t0 + first + tokens + it.off))));
    nt[g] = tokens > 0 ? max(0, hi - it.lo) : 0;
    most = max(most, nt[g]);
  }

  if (threadIdx.x == 0) {
    mbar_init(&bar_q, 1);
    for (int s = 0; s < C::RING; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 1);
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&bar_sfull[g], 1);
      mbar_init(&bar_pfull[g], 4);  // one arrival per softmax warp
      mbar_init(&bar_odone[g], 1);
    }
    mbar_init(&bar_drain, 1);
    abort_flag = 0;
    never_abort = 0;
    fence_barrier_init();
  }
  constexpr int TMA_WARP = 4 * NQ, MMA_WARP = 4 * NQ + 1;
  if (warp == MMA_WARP) {
    tmem_alloc(&tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;

  if (warp == TMA_WARP) {
    // ================= loads: Q, then K(0), V(0), K(1), V(1), ... =================
    const bool leader = elect_one();
    const CUtensorMap* mk = it.prefix ? &tmKp : &tmK;
    const CUtensorMap* mv = it.prefix ? &tmVp : &tmV;
    int issued = 0;
    bool ok = true, q_issued = false;
    if (most > 0) {
      if (leader) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(mk);
        prefetch_tensormap(mv);
        const uint32_t qbytes = (uint32_t)(p.G * p.TQ * 128);
        int live = 0;
        for (int g = 0; g < NQ; ++g) live += nt[g] > 0;
        mbar_arrive_expect_tx(&bar_q, live * C::NATOM * qbytes);
        for (int g = 0; g < NQ; ++g)
          if (nt[g] > 0)
            for (int a = 0; a < C::NATOM; ++a)
              tma_load_4d(sm + g * C::TILE_BYTES + a * 128 * 128, &tmQ, &bar_q, a * 64, 0, it.q0 + g * p.TQ, it.head);
      }
      q_issued = true;
      for (int m = 0; ok && m < 2 * most; ++m) {
        const int slot = m % C::RING;
        if (m >= C::RING) {
          ok = warp_wait(&bar_empty[slot], (uint32_t)((m / C::RING) - 1) & 1u, &abort_flag, p.limit_ns);
          if (!ok) break;
        }
        if (leader) {
          uint8_t* dst = sm + C::OFF_RING + slot * C::TILE_BYTES;
          const int row = it.k0 + (it.lo + (m >> 1)) * kPkKeys;
          mbar_arrive_expect_tx(&bar_full[slot], C::TILE_BYTES);
          for (int a = 0; a < C::NATOM; ++a)
            tma_load_4d(dst + a * 128 * 128, (m & 1) ? mv : mk, &bar_full[slot], a * 64, row, it.head, 0);
        }
        __syncwarp();
        ++issued;
      }
    }
    if (leader) {
      if (!ok) {
        abort_flag = 1;
        report_error(-6);
      }
      // drain: every issued load lands before the CTA may exit
      if (q_issued) mbar_wait(&bar_q, 0, &never_abort, p.limit_ns);
      for (int m = max(0, issued - C::RING); m < issued; ++m)
        mbar_wait(&bar_full[m % C::RING], (uint32_t)(m / C::RING) & 1u, &never_abort, p.limit_ns);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ================= MMA: per key tile j and row tile g, O_g += P_g(j) V(j), then S_g(j+1) =================
    const uint32_t sbase = smem_u32(sm);
    const bool leader = elect_one();
    bool ok = true;
    auto wait_full = [&](int m) {
      return warp_wait(&bar_full[m % C::RING], (uint32_t)(m / C::RING) & 1u, &abort_flag, p.limit_ns);
    };
    auto issue_s = [&](int g, int j) {  // S_g = Q_g K(j)^T
      const int slot = (2 * j) % C::RING;
      const uint64_t dq = smem_desc(sbase + g * C::TILE_BYTES, 16, 1024, SW_128B);
      const uint64_t dk = smem_desc(sbase + C::OFF_RING + slot * C::TILE_BYTES, 16, 1024, SW_128B);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t step = (uint64_t)(((kk / 4) * 128 * 128 + (kk % 4) * 32) >> 4);
        mma_ss<KIND_F16>(tbase + C::S_COL + 128 * g, dq + step, dk + step, C::IDESC_S, kk > 0 ? 1u : 0u);
      }
      mma_commit(&bar_sfull[g]);
    };
    if (most > 0) {
      ok = warp_wait(&bar_q, 0, &abort_flag, p.limit_ns) && wait_full(0);
      if (ok) {
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int g = 0; g < NQ; ++g)
            if (nt[g] > 0) issue_s(g, 0);
          mma_commit(&bar_empty[0]);
        }
        __syncwarp();
      }
      for (int j = 0; ok && j < most; ++j) {
        const int vslot = (2 * j + 1) % C::RING;
        ok = wait_full(2 * j + 1);
        if (!ok) break;
        // V rows past the sequence's end belong to somebody else: zero them
        const int left = it.lk - (it.lo + j) * kPkKeys;
        if (left < kPkKeys) {
          uint8_t* vt = sm + C::OFF_RING + vslot * C::TILE_BYTES;
          for (int a = 0; a < C::NATOM; ++a)
            for (int b = left * 128 + lane * 16; b < kPkKeys * 128; b += 512)
              *reinterpret_cast<uint4*>(vt + a * 128 * 128 + b) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        bool k_ready = false;
        const int last = (NQ == 2 && nt[NQ - 1] > j) ? NQ - 1 : 0;         // last row tile that uses V(j)
        const int last_s = (NQ == 2 && nt[NQ - 1] > j + 1) ? NQ - 1 : 0;   // last row tile that uses K(j+1)
#pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (j >= nt[g]) continue;
          ok = warp_wait(&bar_pfull[g], (uint32_t)j & 1u, &abort_flag, p.limit_ns);
          if (ok && j + 1 < nt[g] && !k_ready) {
            ok = wait_full(2 * j + 2);
            k_ready = true;
          }
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t dv = smem_desc(sbase + C::OFF_RING + vslot * C::TILE_BYTES, 128 * 128, 1024, SW_128B);
#pragma unroll
            for (int kk = 0; kk < kPkKeys / 16; ++kk)
              mma_ts<KIND_F16>(tbase + C::O_COL + D * g, tbase + C::S_COL + 128 * g + 8 * kk,
                               dv + (uint64_t)((kk * 16 * 128) >> 4), C::IDESC_PV, (j > 0 || kk > 0) ? 1u : 0u);
            if (j + 1 == nt[g]) mma_commit(&bar_odone[g]);
            if (g == last) mma_commit(&bar_empty[vslot]);
            if (j + 1 < nt[g]) {
              issue_s(g, j + 1);
              if (g == last_s) mma_commit(&bar_empty[(2 * j + 2) % C::RING]);
            }
          }
          __syncwarp();
        }
      }
    }
    if (leader) {
      if (!ok) {
        abort_flag = 1;
        report_error(-6);
      }
      // drain: every issued MMA completes before TMEM is released
      mma_commit(&bar_drain);
      mbar_wait(&bar_drain, 0, &never_abort, p.limit_ns);
    }
    __syncwarp();
  } else {
    // ================= softmax, rescale, epilogue: thread = row =================
    const int g = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int tok = g * p.TQ + row / p.G;                // token of the item
    const int head = it.head * p.G + row % p.G;
    const bool valid = row < p.TQ * p.G && it.q0 + tok < it.q_end;
    const bool warp_live = __any_sync(0xffffffffu, valid);
    // keys [0, seen) of the sequence are visible to this row
    const int seen = (p.causal && !it.prefix) ? max(0, min(it.lk, it.t0 + tok + it.off + 1)) : it.lk;
    const int my_nt = NQ == 2 ? (g ? nt[NQ - 1] : nt[0]) : nt[0];
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tbase + lanes + C::S_COL + 128 * g, o_addr = tbase + lanes + C::O_COL + D * g;
    const float sc = p.scale_log2;
    float m_use = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < my_nt; ++j) {
      ok = warp_wait(&bar_sfull[g], (uint32_t)j & 1u, &abort_flag, p.limit_ns);
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
        const int nv = seen - (it.lo + j) * kPkKeys;      // visible columns of this tile
        if (__any_sync(0xffffffffu, nv < kPkKeys)) {
#pragma unroll
          for (int u = 0; u < 128; ++u)
            if (u >= nv) sv[u] = 0xFF800000u;             // -inf
        }
        const float* f = reinterpret_cast<const float*>(sv);
        float t8[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float a = fmaxf(f[i], f[i + 8]);
#pragma unroll
          for (int u = 16; u < 112; u += 16) a = fmax3(a, f[i + u], f[i + u + 8]);
          t8[i] = fmax3(a, f[i + 112], f[i + 120]);
        }
        const float mx = fmaxf(fmax3(t8[0], t8[1], t8[2]), fmax3(t8[3], t8[4], fmax3(t8[5], t8[6], t8[7]))) * sc;
        const bool grow = mx > m_use + kPkLazy;           // also the first finite maximum
        if (__any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? ex2f(m_use - mx) : 1.f;   // 0 from -inf
          if (grow) m_use = mx;
          l_run *= alpha;
          if (j > 0) {
            const uint64_t a2 = f2pack(alpha, alpha);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(o_addr + c, o);
              tmem_wait_ld();
              reg_fence32(o);
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                float x, y;
                f2unpack(mul2(f2pack(__uint_as_float(o[i]), __uint_as_float(o[i + 1])), a2), x, y);
                o[i] = __float_as_uint(x);
                o[i + 1] = __float_as_uint(y);
              }
              tmem_st32(o_addr + c, o);
            }
          }
        }
        const float at = m_use == -INFINITY ? 0.f : m_use;  // nothing visible yet: exp2(-inf - 0) = 0
        const uint64_t sc2 = f2pack(sc, sc), nm2 = f2pack(-at, -at);
        uint64_t sum2[4] = {0, 0, 0, 0};
        uint32_t pk[64];
#pragma unroll
        for (int u = 0; u < 128; u += 2) {
          float x0, x1;
          f2unpack(fma2(f2pack(__uint_as_float(sv[u]), __uint_as_float(sv[u + 1])), sc2, nm2), x0, x1);
          const float p0 = ex2f(x0), p1 = ex2f(x1);
          sum2[(u >> 1) & 3] = add2(sum2[(u >> 1) & 3], f2pack(p0, p1));
          const __nv_bfloat162 hb = __floats2bfloat162_rn(p0, p1);
          pk[u >> 1] = *reinterpret_cast<const uint32_t*>(&hb);
        }
        tmem_st32(s_addr, *reinterpret_cast<uint32_t(*)[32]>(&pk[0]));
        tmem_st32(s_addr + 32, *reinterpret_cast<uint32_t(*)[32]>(&pk[32]));
        float a0, a1, b0, b1;
        f2unpack(add2(sum2[0], sum2[1]), a0, a1);
        f2unpack(add2(sum2[2], sum2[3]), b0, b1);
        l_run += (a0 + a1) + (b0 + b1);
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar_pfull[g]);
    }
    if (ok && my_nt > 0) {
      ok = warp_wait(&bar_odone[g], 0, &abort_flag, p.limit_ns);
      tc_fence_after();
    }
    if (!ok) {
      abort_flag = 1;
      report_error(-6);
    } else if (warp_live) {
      const int from = it.lo * kPkKeys;                          // keys [from, to) were computed
      const int to = min(it.lk, (it.lo + my_nt) * kPkKeys);
      const bool any = valid && seen > from && my_nt > 0;        // this row saw a key
      const float inv = it.slot < 0 ? 1.0f / l_run : 1.0f;
      const long long tr = it.q0 + tok;
      __nv_bfloat16* orow = p.o + head * p.osH + tr * p.osL;
      const long long R = (long long)p.Tq * p.Hkv * p.G, prow = it.slot * R + tr * (p.Hkv * p.G) + head;
      float* part = it.slot < 0 ? nullptr : p.part + prow * D;
      float check = 0.f;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (my_nt > 0) {
          tmem_ld32(o_addr + c, o);
          tmem_wait_ld();
          reg_fence32(o);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = any ? __uint_as_float(o[i]) : 0.f;
          check = fmaf(x, 0.f, check);
          o[i] = __float_as_uint(any ? x * inv : 0.f);
        }
        if (!valid) continue;
        if (it.slot < 0) {
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const __nv_bfloat162 hb = __floats2bfloat162_rn(__uint_as_float(o[8 * w + 2 * i]),
                                                              __uint_as_float(o[8 * w + 2 * i + 1]));
              h[i] = *reinterpret_cast<const uint32_t*>(&hb);
            }
            *reinterpret_cast<uint4*>(orow + c + 8 * w) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        } else {
#pragma unroll
          for (int w = 0; w < 8; ++w)
            *reinterpret_cast<uint4*>(part + c + 4 * w) = make_uint4(o[4 * w], o[4 * w + 1], o[4 * w + 2], o[4 * w + 3]);
        }
      }
      if (valid) {
        if (it.slot >= 0)
          p.ml[prow] = any ? make_float2(m_use, l_run) : make_float2(-INFINITY, 0.f);
        else if (p.lse)
          p.lse[(long long)head * p.Tq + tr] = any ? pack_lse(m_use, l_run) : -INFINITY;
      }
      // rows that a hidden key's non-finite V may have spoilt
      uint32_t redo = __ballot_sync(0xffffffffu, any && check != check && seen < to);
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        const int s_seen = __shfl_sync(0xffffffffu, seen, src), s_head = __shfl_sync(0xffffffffu, head, src);
        const int s_tr = __shfl_sync(0xffffffffu, (int)tr, src);
        const __nv_bfloat16* kb = p.k.p + it.head * p.k.sH + (long long)it.k0 * p.k.sL;
        const __nv_bfloat16* vb = p.v.p + it.head * p.v.sH + (long long)it.k0 * p.v.sL;
        constexpr int E = D / 32;
        bool spoilt = false;
        for (int u = s_seen; u < to; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x = __bfloat162float(vb[u * p.v.sL + lane * E + e]);
            spoilt |= !(fabsf(x) < INFINITY);
          }
        if (!__any_sync(0xffffffffu, spoilt)) continue;
        float o[E], m, l;
        packed_exact_row<D>(p.q.p + s_head * p.q.sH + (long long)s_tr * p.q.sL, kb, p.k.sL, vb, p.v.sL, from, s_seen,
                            sc, o, m, l);
        const long long s_prow = it.slot * R + (long long)s_tr * (p.Hkv * p.G) + s_head;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (it.slot < 0)
            p.o[s_head * p.osH + s_tr * p.osL + lane * E + e] = __float2bfloat16(o[e] / l);
          else
            p.part[s_prow * D + lane * E + e] = o[e];
        }
        if (lane == 0) {
          if (it.slot >= 0)
            p.ml[s_prow] = make_float2(m, l);
          else if (p.lse)
            p.lse[(long long)s_head * p.Tq + s_tr] = pack_lse(m, l);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

// Joins the splits of each row: a warp per row, lane = D / 32 channels, splits in
// ascending order (the result does not depend on which item finished first).
template <int D>
__global__ void __launch_bounds__(256) packed_combine_kernel(const PackParams p) {
  constexpr int E = D / 32;
  const int Hq = p.Hkv * p.G, lane = threadIdx.x & 31;
  const long long R = (long long)p.Tq * Hq, row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= R) return;
  const int tok = (int)(row / Hq), head = (int)(row % Hq);
  // the last sequence that starts at or before this token
  int lo = 0, hi = p.n;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + lane * step;
    const unsigned le = __ballot_sync(0xffffffffu, at < hi && p.cu_q[at] <= tok);
    const int k = le ? 31 - __clz(le) : 0;
    const int nl = lo + k * step;
    hi = min(hi, nl + step);
    lo = nl;
  }
  const PackSeq s = pack_seq(p, lo);
  if (tok < s.q0 || tok >= s.q0 + s.lq) return;
  if (p.Lp) {  // a malformed table may leave rows without their prefix part
    const PackSeq all = pack_all(p);
    if (tok < all.q0 || tok >= all.q0 + all.lq) return;
  }
  const int c = *p.chunk, t = pack_tiles(s.lk);
  const int np = p.Lp ? pack_splits(pack_tiles(p.Lp), c, p.max_np) : 0;
  const int ns = (p.Lp && t == 0) ? 0 : pack_splits(t, c, p.max_ns);
  if (!p.Lp && ns == 1) return;   // its item finished the row
  float m = -INFINITY;
  for (int i = lane; i < np + ns; i += 32) m = fmaxf(m, p.ml[i * R + row].x);
#pragma unroll
  for (int w = 16; w; w >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
  const float at = m == -INFINITY ? 0.f : m;
  float o[E], l = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 4
  for (int i = 0; i < np + ns; ++i) {
    const float2 x = p.ml[i * R + row];
    const float w = ex2f(x.x - at);
    l = fmaf(w, x.y, l);
    const float* src = p.part + (i * R + row) * D + lane * E;
    if constexpr (E == 4) {
      const float4 y = *reinterpret_cast<const float4*>(src);
      o[0] = fmaf(w, y.x, o[0]);
      o[1] = fmaf(w, y.y, o[1]);
      o[2] = fmaf(w, y.z, o[2]);
      o[3] = fmaf(w, y.w, o[3]);
    } else {
      const float2 y = *reinterpret_cast<const float2*>(src);
      o[0] = fmaf(w, y.x, o[0]);
      o[1] = fmaf(w, y.y, o[1]);
    }
  }
  const int seen = p.causal ? max(0, min(s.lk, tok - s.q0 + s.lk - s.lq + 1)) : s.lk;
  const bool any = p.Lp > 0 || seen > 0;
  __nv_bfloat16* dst = p.o + head * p.osH + tok * p.osL + lane * E;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + e) =
        any ? __floats2bfloat162_rn(o[e] / l, o[e + 1] / l) : __floats2bfloat162_rn(0.f, 0.f);
  if (lane == 0 && p.lse) p.lse[(long long)head * p.Tq + tok] = any ? pack_lse(m, l) : -INFINITY;
}

}  // namespace lx
