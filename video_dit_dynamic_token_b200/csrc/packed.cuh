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
// A work item keeps two streams of a CTA busy, each with a row tile of Q, its
// softmax warpgroup and its accumulator in TMEM; while one stream's softmax runs, the
// tensor core works for the other.  Two row tiles of a sequence (2 TQ tokens) share
// the same 128-key tiles, loaded once.  A single row tile (narrow), such as a single token or
// the rest of a longer sequence, is taken for two neighbouring key/value heads; where their
// number is odd, for one, whose keys are split between the streams.  (Splitting for all:
// decoding 48 sequences 113 us instead of 108, 64 behind a prefix 58 instead of 52; pairs
// for an odd number, the last one half empty: 39 instead of 31 us with one head.)
// Key ranges (splits) also spread long sequences over the SMs when there are few items:
// a split leaves its unnormalised fp32 rows and (max, sum), and packed_combine_kernel
// joins them.  A row whose keys are one split is finished by its item, and only sequences that are
// split have partial rows (200 prompts of 77 tokens, 40 heads: 368 us with a place for every row, 212).
//
// One CTA per SM.  The grid has a block for every item there can be; a running CTA takes
// over blocks that have not started (cluster launch control), so that items are
// handed out as CTAs become free, and the loads and first scores of an item run under the
// end of the one before it.
//
// Roles: warps 0 .. 7 softmax (thread = row; warpgroup g is stream g); in the last
// warpgroup one warp that takes items and loads, and an MMA warp for each stream; each
// walks the items by itself.  TMEM: S_g (128 fp32 columns; P of the first and of the
// second half of the keys, 32 columns of bf16 pairs each, takes the place of the half's
// first columns) and O_g (D fp32 columns).  A stream's order per key tile j is the product
// of the first half of P(j) with V, that of the second half, S(j+1): the first product
// runs under the second half's exponentials, S(j+1) may overwrite P(j) because the tensor
// core runs a thread's MMAs in order, and its commit also says that O has P(j) V(j), so
// the softmax may rescale O without another barrier.  What bounds a long row: a stream's chain
// of 3,500 clocks per tile (scores to P 2,300, of which the exponentials 1,600; P to scores
// 1,000), two of which overlap; its MMAs take 1,024.  Measured and slower for the 480p grid (9.9
// ms): half tiles with two score buffers 12.1; the first half of S(j+1) issued between the
// halves of P V 10.7 (64-column MMAs take 1.5 times as long per column, Q being read twice as
// often); 16 softmax warps 11.3 and more.
//
// The reference that the exponents are taken against is not the running maximum but
// follows it: it moves only when the maximum of a tile has passed it by more than 2^8, so
// that O is rarely rescaled.  A shift leaves the quotient unchanged: P is at most 2^8 and its
// rounding to bf16, the type of V and of the output, is relative; the row sum takes the
// unrounded fp32 values.
//
// Values in masked places: scores are replaced by -inf by selection, and V rows
// past a sequence's end are zeroed in shared memory before they are used.  A
// key that the causal rule hides from some rows of a tile and not from others
// has P = 0 there, and 0 * V is NaN when V is not finite: a row that ends
// non-finite and has such keys is computed again by packed_exact_row (up to 32 rows a warp, one after
// another: 0.4 s for a sequence of 75,600 keys, 8.5 s for a million; other waits go on meanwhile).
//
// Measured (D = 128, in a graph, inputs colder than L2): a causal sequence of 32,760 tokens with
// 40 heads 10.0 to 10.4 ms (1.1 PFLOP/s); 16,000 video tokens over prompts of 77 to 512 keys 134 to 140 us
// (2.5 TB/s); one token in each of 48 sequences of 200 to 8,000 keys, 40 heads on 8, 106 us
// (4.4 TB/s); 64 tokens behind 8,192 shared keys 46 us; three prompts of 5 to 77 tokens 7.8.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cstdint>
#include "attn.cuh"
#include "ptx.cuh"
#include "quant.cuh"

namespace lx {

constexpr int kPkKeys = 128;         // keys of a tile
constexpr int kPkHalf = 64;          // keys of a product with V
constexpr int kPkSplitKeys = 1;      // a split covers at least this many tiles (2: four tokens behind 200 keys 15.9, not 14.1 us)
// from this many tiles on, three splits for a CTA's share of the work (64 tokens behind 8,192 keys,
// 16 over 1,000 to 4,000: 4 46.3 and 40.5 us, 6 44.4 and 46.8, 9 42.1 and 50.4; 75,600 shared keys:
// two splits 195 us, three 172, four 186)
constexpr int kPkFine = 6;
constexpr int kPkSMs = 148;
constexpr int kPkItems = 4;          // items published ahead of their last reader
constexpr float kPkLazy = 8.0f;      // log2 growth of the row maximum that moves the reference

template <int D>
struct PackCfg {
  static constexpr int NATOM = D / 64;                 // 128-byte swizzle atoms per row
  static constexpr int TILE_BYTES = 128 * D * 2;       // a Q, K or V tile
  static constexpr int RING = D == 128 ? 5 : 8;        // K and V tiles beside the two of Q
  static constexpr int OFF_RING = 2 * TILE_BYTES;
  static constexpr int SMEM = 1024 + OFF_RING + RING * TILE_BYTES;
  static constexpr int READERS = 10;                   // warps that read an item: softmax, MMA
  static constexpr int THREADS = 384;                  // softmax warpgroups; loads, two MMA warps, one idle
  // registers per thread: 168 at launch, then moved to the softmax, whose threads hold a
  // half row of scores and of P: 128 x 72 + 256 x 216 = 384 x 168
  static constexpr int REGS_AUX = 72, REGS_SOFTMAX = 216;
  static constexpr uint32_t S_COL = 0;                 // + 128 g
  static constexpr uint32_t O_COL = 256;               // + D g
  static constexpr uint32_t TMEM_COLS = 512;
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
  int sectors;           // rows of o start at multiples of 32 bytes
  float* lse;            // [Hq][Tq] or null
  // Partial rows, [..][Hq] for each of `room` tokens: with a prefix [max_np + max_ns][Tq]; else
  // [ns][lq] for each sequence that is split, one after the other.
  float* part;           // [room][Hq][D] unnormalised rows; null where nothing is split
  float2* ml;            // [room][Hq] (max, sum), max in the log2 domain
  int* chunk;            // tiles per split, whether nothing is split, most splits; for the combine kernel
  int* start;            // [n] first partial row of a sequence that is split, in tokens (no prefix)
  int room;              // (no prefix)
  int max_np, max_ns;    // most splits of the prefix, of a sequence
  int wide;              // more than a row tile of tokens a sequence on average, no prefix
  int pair, units;       // key/value heads of a narrow item (1 or 2), Hkv / pair
  int group;             // units worked on at a time
  unsigned long long limit_ns;
};

struct PackSeq {
  int q0, lq, k0, lk;
};

// Rows and keys of sequence i; a sequence whose entries do not fit the tensors is
// reported and left out (lq = 0, k0 = -1).
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
    s = PackSeq{0, 0, -1, 0};
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
// Row tile pairs of `rows` tokens; a rest of at most TQ tokens is a narrow item.
__device__ __forceinline__ int pack_pairs(const PackParams& p, int rows) { return (rows + p.TQ - 1) / (2 * p.TQ); }
__device__ __forceinline__ int pack_narrow(const PackParams& p, int rows) {
  return rows > 2 * p.TQ * pack_pairs(p, rows) ? 1 : 0;
}
// Splits of T key tiles, c tiles each and at most `most`; at least two where the streams
// of a narrow item share a head and all rows are in it.
__device__ __forceinline__ int pack_splits(const PackParams& p, int rows, int T, int c, int most) {
  if (p.pair == 1 && rows <= p.TQ) c = min(c, max(kPkSplitKeys, pack_div(T, 2)));
  return max(1, min(most, pack_div(T, c)));
}
// Items of `rows` tokens in ns splits, for p.pair heads together.
__device__ __forceinline__ int pack_count(const PackParams& p, int rows, int ns) {
  return p.pair * pack_pairs(p, rows) * ns + pack_narrow(p, rows) * (p.pair == 2 ? ns : pack_div(ns, 2));
}

struct PackItem {
  int q0, q_end;         // first token of the item, end of its sequence (rows of Q)
  int t0, off;           // its index in the sequence; causal: token t sees keys <= t + off
  int k0, lk;            // first key row, keys
  int lo[2], nt[2];      // first key tile and number of key tiles of each stream
  int nh[2];             // number of halves with a key that some row sees
  int slot[2];           // where a stream's partial result goes; -1: it finishes its rows; -2: no rows
  int head[2];           // key/value head of each stream
  int prefix;            // keys of the prefix (no causal rule)
  int row0, step;        // partial row of token t (a row of Q) in slot x: row0 + x step + t
  int narrow;            // both streams have the item's rows, and a head or a range of keys each
  int stop;              // no further item
};

// What a CTA works out once from the sequence table: the number of items of a unit
// (p.pair key/value heads), and for up to 128 chunks of sequences the items before each.
constexpr int kPkChunks = 128;
struct PackTable {
  unsigned long long work, hidden;   // steps; those that the causal rule spares
  int longest;
  int c, np, pi;           // tiles per split, prefix splits, prefix items
  int total;               // items of a unit
  int most;                // splits of a sequence
  int bad;                 // a sequence was left out
  int need;                // partial rows of the sequences that are split, in tokens (no prefix)
  int before[kPkChunks + 1];
  int rows[kPkChunks + 1];        // partial rows before each chunk (bits of an unsigned while they are added up)
};
constexpr int kPkManyRows = 1 << 18;   // more tokens than `room` holds; counts stop there

// Splits and items of a sequence, and its partial rows in tokens (no prefix).
__device__ __forceinline__ int pack_seq_splits(const PackParams& p, const PackSeq& s, int c, int most) {
  return pack_splits(p, s.lq, pack_tiles(s.lk), c, most);
}
__device__ __forceinline__ int pack_seq_items(const PackParams& p, const PackSeq& s, int ns) {
  if (p.Lp && s.lk == 0) return 0;   // behind a prefix a sequence may have no keys of its own
  return pack_count(p, s.lq, ns);
}
__device__ __forceinline__ int pack_seq_rows(const PackSeq& s, int ns) {
  return ns == 1 ? 0 : (int)min((long long)s.lq * ns, (long long)kPkManyRows);
}
// Steps of a CTA over T key tiles for `rows` tokens of p.pair heads.
__device__ __forceinline__ unsigned long long pack_steps(const PackParams& p, int rows, int T) {
  return (unsigned long long)(p.pair * pack_pairs(p, rows)) * T +
         pack_narrow(p, rows) * (p.pair == 2 ? T : (T + 1) / 2);
}

// Items and partial rows of all sequences for splits of tb.c tiles, and their sums; before and rows are zero.
// seq(i): sequence i.
template <int THREADS, class Seq>
__device__ __forceinline__ void pack_count_all(const PackParams& p, PackTable& tb, const Seq& seq) {
  const int tid = threadIdx.x, cs = pack_div(p.n, kPkChunks);
  const bool pool = p.part && !p.Lp;   // partial rows of split sequences only
  for (int i = tid; i < p.n; i += THREADS) {
    const PackSeq s = seq(i);
    const int ns = pack_seq_splits(p, s, tb.c, tb.most), m = pack_seq_items(p, s, ns);
    if (m) atomicAdd(&tb.before[i / cs + 1], m);
    if (s.k0 < 0) tb.bad = 1;
    if (pool && ns > 1)   // 2^13 sequences in a chunk at most
      atomicAdd(reinterpret_cast<unsigned*>(&tb.rows[i / cs + 1]), (unsigned)pack_seq_rows(s, ns));
  }
  __syncthreads();
  if (tid < (pool ? 64 : 32)) {   // inclusive sums of 4 chunks a lane: items by warp 0, partial rows by warp 1
    const int lane = tid & 31, first = 1 + lane * (kPkChunks / 32);
    int* sums = tid < 32 ? tb.before : tb.rows;
    int v[kPkChunks / 32], s = 0;
#pragma unroll
    for (int j = 0; j < kPkChunks / 32; ++j)
      v[j] = s += tid < 32 ? sums[first + j] : (int)min((unsigned)sums[first + j], (unsigned)kPkManyRows);
    int run = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += t;
    }
#pragma unroll
    for (int j = 0; j < kPkChunks / 32; ++j) sums[first + j] = run - s + v[j];
    if (tid == 31) tb.total = run + tb.pi;
    if (tid == 63) tb.need = run;
  }
  __syncthreads();
}

// What few calls need, out of the line (in it, it cost the smallest calls 0.5 us):
// - More partial rows than there is room for: longer splits, at last none (then only heads without a
//   neighbour are split, whose streams share the keys).
// - A table that descends may count rows more than once, and then has more items than the grid has
//   blocks, or than 31 bits hold: none of them is worked on.
template <int THREADS>
__device__ __noinline__ void pack_refit(const PackParams& p, PackTable& tb) {
  const int tid = threadIdx.x;
  auto seq = [&](int i) { return pack_seq(p, i); };
  while (tb.need > p.room) {
    __syncthreads();
    if (tid == 0) {
      if (tb.c >= tb.longest) tb.most = 1;
      const long long c = tb.c;
      tb.c = (int)min((long long)tb.longest, max(c * tb.need / max(p.room, 1), c + c / 8 + 1));
    }
    for (int i = tid; i <= kPkChunks; i += THREADS) tb.before[i] = 0, tb.rows[i] = 0;
    __syncthreads();
    pack_count_all<THREADS>(p, tb, seq);
  }
  if (!tb.bad) return;
  if (tid == 0) tb.work = 0;
  __syncthreads();
  unsigned long long all = 0;
  for (int i = tid; i < p.n; i += THREADS) {
    const PackSeq s = pack_seq(p, i);
    all += pack_seq_items(p, s, pack_seq_splits(p, s, tb.c, tb.most));
  }
  if (all) atomicAdd(&tb.work, all);
  __syncthreads();
  if (tid == 0 && (tb.work + tb.pi) * p.units > gridDim.x) tb.total = tb.need = 0;
  __syncthreads();
}

// Every thread reads a share of the table, so that lengths stay on the device.
template <int THREADS>
__device__ void pack_prepare(const PackParams& p, PackTable& tb) {
  const int tid = threadIdx.x;
  if (tid == 0) {
    tb.work = 0, tb.hidden = 0, tb.longest = 0, tb.np = 0, tb.pi = 0;
    tb.c = 1 << 29;   // one split
    tb.bad = tb.need = 0;
    tb.most = p.max_ns;
  }
  for (int i = tid; i <= kPkChunks; i += THREADS) tb.before[i] = 0, tb.rows[i] = 0;
  const PackSeq mine = tid < p.n ? pack_seq(p, tid) : PackSeq{0, 0, 0, 0};   // read once where it covers the table
  __syncthreads();
  if (p.part) {
    // the split length c follows from the work: a CTA's share of it, or a third of
    // that where it is long, so that uneven items still end together
    unsigned long long w = 0, hid = 0;
    int l = 0;
    for (int i = tid; i < p.n; i += THREADS) {
      const PackSeq s = i < THREADS ? mine : pack_seq(p, i);
      const int t = pack_tiles(s.lk);
      w += pack_steps(p, s.lq, t);
      if (p.causal) hid += pack_steps(p, s.lq, min(t, pack_tiles(s.lq))) / 2;
      if (s.lq) l = max(l, t);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      w += __shfl_xor_sync(0xffffffffu, w, o);
      hid += __shfl_xor_sync(0xffffffffu, hid, o);
    }
    l = __reduce_max_sync(0xffffffffu, l);
    if ((tid & 31) == 0 && w) {
      atomicAdd(&tb.work, w);
      atomicAdd(&tb.hidden, hid);
      atomicMax(&tb.longest, l);
    }
    __syncthreads();
    if (tid == 0) {
      const int pt = pack_tiles(p.Lp), rows = p.Lp ? pack_all(p).lq : 0;
      const unsigned long long work = (tb.work + pack_steps(p, rows, pt)) * p.units;
      int c = (int)((work + kPkSMs - 1) / kPkSMs);
      if (c > kPkFine) c = max(kPkFine, pack_div(c, 3));
      c = max(max(c, kPkSplitKeys), pack_div(tb.longest, p.max_ns));
      if (p.Lp) c = max(c, pack_div(pt, p.max_np));
      // Row tiles full of tokens pay for a split with their partial rows, about as much as 7
      // tiles.  Times in tiles, fitted to single prompts of 2,000 to 16,128 tokens with 1 to 10
      // heads (split, whole; 1.9 us a tile): 10 heads x 4,000 103, 66 us; 10 x 2,000 51, 36;
      // 2 x 16,128 210, 223; 1 x 8,000 52, 118.  With D = 64 (split, whole): 10 x 4,000 93, 64;
      // 10 x 2,300 50, 41; 2 x 16,128 198, 225; 1 x 8,000 45, 113; 12 x 8,000 265, 184.  The estimate is too
      // high for few short items, with either D: 2 x 2,300 stay whole, 40 us instead of 23 (D = 128: 42, 26),
      // and so do 2 x 8,000 without the causal rule, 119 instead of 76 (126, 89).
      if (p.wide) {
        const long long C = (long long)((work - tb.hidden * p.units + kPkSMs - 1) / kPkSMs), l = tb.longest;
        if (max(l, C + l / 2) <= C + C / 2 + 7 * ((C + c - 1) / c) + 8) c = max(1, tb.longest);
      }
      tb.c = c;
      if (p.Lp) {
        tb.np = pack_splits(p, rows, pt, c, p.max_np);
        tb.pi = pack_count(p, rows, tb.np);
      }
    }
    __syncthreads();
  }
  pack_count_all<THREADS>(p, tb, [&](int i) { return i < THREADS ? mine : pack_seq(p, i); });
  if (tb.bad || tb.need > p.room) pack_refit<THREADS>(p, tb);
  if (tid == 0 && p.part) {
    // by every CTA, all the same: which block numbers ever start is the launch control's affair
    p.chunk[0] = tb.c;
    p.chunk[1] = tb.total == 0 || (!p.Lp && tb.need == 0);   // nothing to join
    p.chunk[2] = tb.most;
  }
}

// Item number `id` (a warp together); stop past the last one.  In the order of a unit's
// items the prefix comes first, then the last rows of the last sequence (with the causal
// rule the long items start first); p.group units, whose K and V fit the L2 cache
// together, take turns in it.
__device__ __forceinline__ void pack_item(const PackParams& p, const PackTable& tb, int id, PackItem& it) {
  const int lane = threadIdx.x & 31;
  it.stop = 1;
  if (id / p.units >= tb.total) return;   // total * units items in all
  it.stop = 0;
  const int first = id / (tb.total * p.group) * p.group, turns = min(p.group, p.units - first);
  id -= first * tb.total;
  const int unit = first + id % turns;
  int x = id / turns;
  PackSeq s{0, 0, 0, 0};
  int ns, base = -1;                    // splits; slot of the first one
  it.row0 = 0;
  it.step = p.Tq;
  it.prefix = x < tb.pi;
  if (it.prefix) {
    s = pack_all(p);
    ns = tb.np;
    base = 0;
  } else {
    x = tb.total - 1 - x;
    // the chunk, then the sequence in it
    int ch = 0;
#pragma unroll
    for (int j = 0; j < kPkChunks / 32; ++j) ch += __popc(__ballot_sync(0xffffffffu, tb.before[1 + j * 32 + lane] <= x));
    x -= tb.before[ch];
    int rows = tb.need ? tb.rows[ch] : 0;   // partial rows before the sequence
    const int cs = pack_div(p.n, kPkChunks), end = min(p.n, (ch + 1) * cs);
    int seq = 0;
    for (int b = ch * cs; b < end; b += 32) {
      const int i = b + lane;
      const PackSeq mine = i < end ? pack_seq(p, i) : PackSeq{0, 0, 0, 0};
      const int splits = pack_seq_splits(p, mine, tb.c, tb.most), m = pack_seq_items(p, mine, splits);
      int run = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, run > x);
      const int src = hit ? __ffs(hit) - 1 : 32;
      if (tb.need) rows += __reduce_add_sync(0xffffffffu, lane < src ? pack_seq_rows(mine, splits) : 0);
      if (hit) {
        seq = b + src;
        s.q0 = __shfl_sync(0xffffffffu, mine.q0, src);
        s.lq = __shfl_sync(0xffffffffu, mine.lq, src);
        s.k0 = __shfl_sync(0xffffffffu, mine.k0, src);
        s.lk = __shfl_sync(0xffffffffu, mine.lk, src);
        x -= __shfl_sync(0xffffffffu, run - m, src);
        break;
      }
      x -= __shfl_sync(0xffffffffu, run, 31);
    }
    ns = pack_seq_splits(p, s, tb.c, tb.most);
    if (p.Lp || ns > 1) base = tb.np;
    if (!p.Lp && ns > 1) {
      it.row0 = rows - s.q0;
      it.step = s.lq;
      if (lane == 0) p.start[seq] = rows;   // by each of its items, all the same
    }
  }
  const int T = pack_tiles(s.lk), per = pack_div(T, ns), pairs = pack_pairs(p, s.lq);
  // first the pairs of row tiles, then the narrow rest; sequences are walked from the end,
  // so that the order within one is turned round as well
  const int wide = p.pair * pairs * ns, two = p.pair - 1;
  it.narrow = x >= wide;
  const int y = it.narrow ? x - wide : x >> two;
  it.t0 = (it.narrow ? pairs : y / ns) * 2 * p.TQ;
  it.q0 = s.q0 + it.t0;
  it.q_end = s.q0 + s.lq;
  it.off = s.lk - s.lq;
  it.k0 = s.k0;
  it.lk = s.lk;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int first_tok = it.narrow ? 0 : g * p.TQ;
    const int tokens = min(p.TQ, it.q_end - it.q0 - first_tok);
    const int sp = !it.narrow ? y % ns : (two ? y : 2 * y + g);
    it.head[g] = p.pair * unit + (two & (it.narrow ? g : x));
    const int lo = min(sp * per, T), hi = min(lo + per, T);
    // keys up to the last one that the tile's last token sees
    int keys = min(s.lk, hi * kPkKeys);
    if (p.causal && !it.prefix) keys = min(keys, it.t0 + first_tok + tokens + it.off);
    const bool live = tokens > 0 && sp < ns;
    it.lo[g] = lo;
    it.nh[g] = live ? pack_div(max(0, keys - lo * kPkKeys), kPkHalf) : 0;
    it.nt[g] = (it.nh[g] + 1) / 2;
    it.slot[g] = !live ? -2 : (base < 0 ? -1 : base + sp);
  }
}

// ---------------------------------------------------------------- cluster launch control
// Asks for a block that has not started; the answer (16 bytes) arrives at `bar`.
__device__ __forceinline__ void clc_request(void* answer, uint64_t* bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                   smem_u32(answer)),
               "r"(smem_u32(bar))
               : "memory");
}
// The block taken over, or -1 when none was left.
__device__ __forceinline__ int clc_answer(const void* answer) {
  uint32_t ok, x = 0;
  asm volatile(
      "{\n\t.reg .b128 r;\n\t.reg .pred p;\n\tld.shared.b128 r, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\tselp.u32 %0, 1, 0, p;\n\t"
      "mov.u32 %1, 0;\n\t@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, r;\n\t}"
      : "=r"(ok), "=r"(x)
      : "r"(smem_u32(answer))
      : "memory");
  return ok ? (int)x : -1;
}

// ---------------------------------------------------------------- MMA issue
// One thread issues every MMA of a stream, so the instructions per MMA count: operands
// are the low words of their descriptors (the high word is common).
__device__ __forceinline__ void mma_f16_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};"
      "\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts_lo(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 db, {%2, %3};"
      "\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}

// 32 bytes, a whole sector (the address a multiple of 32).
__device__ __forceinline__ void st_global_32b(void* p, const uint32_t* x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

// As warp_wait, but the limit starts again while `state` moves: rows that are computed again
// (packed_exact_row) may take longer than any wait, and count their keys in it, in twos; an odd
// number ends all waits.  (One loop in the line: a second wait after the first one's limit made
// all waits 3 % slower.)
__device__ __forceinline__ bool pack_wait(uint64_t* bar, uint32_t parity, const volatile int* state, uint64_t limit_ns) {
  bool ok = mbar_test_wait(bar, parity) || mbar_try_wait(bar, parity);
  if (!ok) {
    uint64_t t0 = globaltimer_ns();
    int seen = 0;
    for (uint32_t it = 1;; ++it) {
      if (mbar_try_wait(bar, parity)) {
        ok = true;
        break;
      }
      if ((it & 63u) == 0u) {
        const int now = *state;
        if (now & 1) break;
        if (globaltimer_ns() - t0 > limit_ns) {
          if (now == seen) break;
          seen = now;
          t0 = globaltimer_ns();
        }
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

// One row over keys [lo, hi), a warp together: lane holds D / 32 neighbouring
// channels.  Returns the unnormalised row, its maximum (log2 domain) and sum.
template <int D>
__device__ __noinline__ void packed_exact_row(const __nv_bfloat16* q, const __nv_bfloat16* k, long long ksL,
                                              const __nv_bfloat16* v, long long vsL, int lo, int hi, float scale_log2,
                                              int* state, float (&o)[D / 32], float& m, float& l) {
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
  constexpr int N = 4;   // keys at a time, whose loads and sums overlap
  for (int u = lo; u < hi; u += N) {
    if (lane == 0 && ((u - lo) & 1023) == 0) atomicAdd(state, 2);   // every millisecond
    float s[N], vf[N][E], mn = m;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool in = u + i < hi;
        s[i] = fmaf(qf[e], in ? __bfloat162float(k[(u + i) * ksL + lane * E + e]) : 0.f, s[i]);
        vf[i][e] = in ? __bfloat162float(v[(u + i) * vsL + lane * E + e]) : 0.f;
      }
    }
#pragma unroll
    for (int w = 16; w; w >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], w);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      s[i] = u + i < hi ? s[i] * scale_log2 : -INFINITY;
      mn = fmaxf(mn, s[i]);
    }
    const float at = mn == -INFINITY ? 0.f : mn, a = m == -INFINITY ? 0.f : ex2f(m - at);
    l *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= a;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = ex2f(s[i] - at);
      l += x;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(x, vf[i][e], o[e]);
    }
    m = mn;
  }
}

__device__ __forceinline__ float pack_lse(float m, float l) { return (m + log2f(l)) * 0.6931471805599453f; }

template <int D>
__global__ void __launch_bounds__(PackCfg<D>::THREADS, 1)
    packed_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKp,
                       const __grid_constant__ CUtensorMap tmVp, const __grid_constant__ PackParams p) {
  using C = PackCfg<D>;
  constexpr int NQ = 2;   // streams
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // full/empty: a ring slot; qfull/qempty[g]: the tile Q_g; sfull[g]: S complete; pfull[g][b]: half b of P
  // written; odone[g]: O complete; ifull/iempty: an item slot; clc: an answer of the launch control
  __shared__ uint64_t bar_full[C::RING], bar_empty[C::RING], bar_qfull[NQ], bar_qempty[NQ], bar_sfull[NQ],
      bar_pfull[NQ][2], bar_odone[NQ], bar_ifull[kPkItems], bar_iempty[kPkItems], bar_clc, bar_drain[NQ];
  __shared__ __align__(16) uint4 clc;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int busy[NQ][4];   // a warp is at its exponentials
  __shared__ volatile int abort_flag;    // odd: all waits end; else keys computed again (pack_wait)
  __shared__ int never_abort;
  __shared__ PackTable table;
  __shared__ PackItem items[kPkItems];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int TMA_WARP = 4 * NQ, MMA_WARP = 4 * NQ + 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::RING; ++s) {
      mbar_init(&bar_full[s], 1);
      mbar_init(&bar_empty[s], 2);   // both streams
    }
    for (int g = 0; g < NQ; ++g) {
      mbar_init(&bar_qfull[g], 1);
      mbar_init(&bar_qempty[g], 1);
      mbar_init(&bar_sfull[g], 1);
      for (int b = 0; b < 2; ++b) mbar_init(&bar_pfull[g][b], 4);  // one arrival per softmax warp
      mbar_init(&bar_odone[g], 1);
    }
    for (int s = 0; s < kPkItems; ++s) {
      mbar_init(&bar_ifull[s], 1);
      mbar_init(&bar_iempty[s], C::READERS);
    }
    mbar_init(&bar_clc, 1);
    for (int g = 0; g < NQ; ++g) mbar_init(&bar_drain[g], 1);
    abort_flag = 0;
    never_abort = 0;
    for (int i = 0; i < 8; ++i) busy[i >> 2][i & 3] = 0;
    fence_barrier_init();
  }
  // the work ahead of this kernel may still run up to here
  asm volatile("griddepcontrol.wait;" ::: "memory");
  pack_prepare<C::THREADS>(p, table);
  if ((int)blockIdx.x / p.units >= table.total) return;   // the grid is an upper bound
  if (warp == MMA_WARP) {
    tmem_alloc(&tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_slot;

  // the k-th item, for the warps that read items; done_item when it is not read any more
  auto next_item = [&](int k) {
    return pack_wait(&bar_ifull[k % kPkItems], (uint32_t)(k / kPkItems) & 1u, &abort_flag, p.limit_ns);
  };
  auto done_item = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar_iempty[k % kPkItems]);
  };
  if (warp >= 4 * NQ) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_AUX));
    if (warp == TMA_WARP) {
      // ================= items and loads: Q, then K(0), V(0), K(1), V(1), ... =================
      const bool leader = elect_one();
      if (leader) {
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
      }
      int m = 0;                 // loads into the ring so far
      int uq[NQ];                // loads of each Q tile
  #pragma unroll
      for (int g = 0; g < NQ; ++g) uq[g] = 0;
      bool ok = true, asked = false;
      int id = blockIdx.x;
      int k = 0;
      for (;; ++k) {
        PackItem it;
        pack_item(p, table, id, it);
        if (k >= kPkItems) {
          ok = pack_wait(&bar_iempty[k % kPkItems], (uint32_t)(k / kPkItems - 1) & 1u, &abort_flag, p.limit_ns);
          if (!ok) break;
        }
        if (leader) {
          items[k % kPkItems] = it;
          mbar_arrive(&bar_ifull[k % kPkItems]);
          if (!it.stop) {        // ask for the next one now: the answer comes under this item's loads
            mbar_arrive_expect_tx(&bar_clc, 16);
            clc_request(&clc, &bar_clc);
          }
        }
        __syncwarp();
        if (it.stop) break;
        asked = true;
        const CUtensorMap* mk = it.prefix ? &tmKp : &tmK;
        const CUtensorMap* mv = it.prefix ? &tmVp : &tmV;
  #pragma unroll
        for (int g = 0; g < NQ; ++g) {
          if (it.nt[g] == 0) continue;
          if (uq[g] > 0) {
            ok = pack_wait(&bar_qempty[g], (uint32_t)(uq[g] - 1) & 1u, &abort_flag, p.limit_ns);
            if (!ok) break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&bar_qfull[g], (uint32_t)(C::NATOM * p.G * p.TQ * 128));
            for (int a = 0; a < C::NATOM; ++a)
              tma_load_4d(sm + g * C::TILE_BYTES + a * 128 * 128, &tmQ, &bar_qfull[g], a * 64, 0,
                          it.q0 + (it.narrow ? 0 : g * p.TQ), it.head[g]);
          }
          __syncwarp();
          ++uq[g];
        }
        if (!ok) break;
        // shared key tiles: K(j), V(j); of its own for each stream: K_0(j), K_1(j), V_0(j), V_1(j)
        const int most = max(it.nt[0], it.nt[1]);
        auto load = [&](const CUtensorMap* map, int j, int g) {
          const int slot = m % C::RING;
          if (m >= C::RING &&
              !pack_wait(&bar_empty[slot], (uint32_t)((m / C::RING) - 1) & 1u, &abort_flag, p.limit_ns))
            return false;
          if (leader) {
            uint8_t* dst = sm + C::OFF_RING + slot * C::TILE_BYTES;
            mbar_arrive_expect_tx(&bar_full[slot], C::TILE_BYTES);
            for (int a = 0; a < C::NATOM; ++a)
              tma_load_4d(dst + a * 128 * 128, map, &bar_full[slot], a * 64, it.k0 + (it.lo[g] + j) * kPkKeys,
                          it.head[g], 0);
          }
          __syncwarp();
          ++m;
          return true;
        };
        for (int j = 0; ok && j < most; ++j) {
          if (!it.narrow) {
            ok = load(mk, j, 0) && load(mv, j, 0);
          } else {
            const bool b1 = j < it.nt[1];
            ok = load(mk, j, 0) && (!b1 || load(mk, j, 1)) && load(mv, j, 0) && (!b1 || load(mv, j, 1));
          }
        }
        if (!ok) break;
        ok = pack_wait(&bar_clc, (uint32_t)k & 1u, &abort_flag, p.limit_ns);
        if (!ok) break;
        asked = false;
        const int next = clc_answer(&clc);
        fence_proxy_async_smem();   // read before the next answer overwrites it
        id = next < 0 ? 0x7FFFFFFF : next;
        __syncwarp();
      }
      asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // no block is left to start
      if (leader) {
        if (!ok) {
          abort_flag = 1;
          report_error(-6);
        }
        // drain: every issued load and answer lands before the CTA may exit
        if (asked) mbar_wait(&bar_clc, (uint32_t)k & 1u, &never_abort, p.limit_ns);
  #pragma unroll
        for (int g = 0; g < NQ; ++g)
          if (uq[g] > 0) mbar_wait(&bar_qfull[g], (uint32_t)(uq[g] - 1) & 1u, &never_abort, p.limit_ns);
        for (int j = max(0, m - C::RING); j < m; ++j)
          mbar_wait(&bar_full[j % C::RING], (uint32_t)(j / C::RING) & 1u, &never_abort, p.limit_ns);
      }
      __syncwarp();
      } else if (warp >= MMA_WARP && warp < MMA_WARP + 2) {
      // ================= MMA of stream g: per tile j, O += P(j) V(j) in two halves, then S(j+1) =================
      const int g = warp - MMA_WARP;
      const uint32_t sbase = smem_u32(sm), scol = tbase + C::S_COL + 128 * g, ocol = tbase + C::O_COL + D * g;
      // descriptors: the high word is the same for all, the low word holds address and leading offset
      const uint64_t dkm = smem_desc(sbase + C::OFF_RING, 16, 1024, SW_128B);
      const uint32_t hi = (uint32_t)(dkm >> 32), ring_k = (uint32_t)dkm;
      const uint32_t ring_v = (uint32_t)smem_desc(sbase + C::OFF_RING, 128 * 128, 1024, SW_128B);
      const uint32_t dq = (uint32_t)smem_desc(sbase + g * C::TILE_BYTES, 16, 1024, SW_128B);
      bool ok = true;
      int m = 0, uq = 0;         // ring position of this item's first load; Q tiles used
      int up[2] = {0, 0};        // halves of P used
      // Both streams walk all loads in order and both free each slot: a stream that only
      // waited for its own tiles could be a turn of the ring ahead or behind on a
      // slot, which a phase's parity does not show.
      int seen = 0;
      auto wait_load = [&](int at) {
        return pack_wait(&bar_full[at % C::RING], (uint32_t)(at / C::RING) & 1u, &abort_flag, p.limit_ns);
      };
      auto skip_to = [&](int at) {   // loads of the other stream: nothing to do with them
        for (; seen < at; ++seen) {
          if (!wait_load(seen)) return false;
          if (lane == 0) mbar_arrive(&bar_empty[seen % C::RING]);
        }
        return true;
      };
      auto wait_full = [&](int at) {
        if (!skip_to(at) || !wait_load(at)) return false;
        seen = at + 1;
        return true;
      };
      for (int k = 0; ok; ++k) {
        ok = next_item(k);
        if (!ok) break;
        const PackItem& it = items[k % kPkItems];
        const int t0 = it.nt[0], t1 = it.nt[1], n = it.nh[g];
        const bool stop = it.stop, narrow = it.narrow;
        const int keys = it.lk - it.lo[g] * kPkKeys;   // from the first tile on
        done_item(k);
        if (stop) break;
        // ring position of K(j) and V(j); narrow: t0 >= t1, four loads a step while both streams run
        int at = m + (narrow ? g : 0);
        m += narrow ? 2 * (t0 + t1) : 2 * max(t0, t1);
        if (n == 0) {
          ok = skip_to(m);
          continue;
        }
        ok = wait_full(at) && pack_wait(&bar_qfull[g], (uint32_t)(uq++) & 1u, &abort_flag, p.limit_ns);
        if (!ok) break;
        tc_fence_after();
        const int nt = (n + 1) / 2;
        auto issue_s = [&](int slot, bool last) {   // S(j) = Q K(j)^T
          const uint32_t dk = ring_k + slot * (C::TILE_BYTES >> 4);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t step = ((kk / 4) * 128 * 128 + (kk % 4) * 32) >> 4;
            mma_f16_lo(scol, dq + step, dk + step, hi, C::IDESC_S, kk > 0);
          }
          mma_commit(&bar_sfull[g]);
          mma_commit(&bar_empty[slot]);
          if (last) mma_commit(&bar_qempty[g]);
        };
        if (elect_one()) issue_s(at % C::RING, nt == 1);
        __syncwarp();
        for (int j = 0; j < nt; ++j) {
          // V of this tile, and K of the next
          const int va = narrow ? at + (j < t1 ? 2 : 1) : at + 1, vslot = va % C::RING;
          at = narrow ? (j + 1 < t1 ? at + 4 : (j < t1 ? at + 4 - g : at + 2)) : at + 2;
          ok = wait_full(va) && (j + 1 >= nt || wait_full(at));
          if (!ok) break;
          // V rows past the sequence's end belong to somebody else: zero them
          const int left = keys - j * kPkKeys;
          if (left < kPkKeys) {
            uint8_t* vt = sm + C::OFF_RING + vslot * C::TILE_BYTES;
            for (int a = 0; a < C::NATOM; ++a)
              for (int y = left * 128 + lane * 16; y < kPkKeys * 128; y += 512)
                *reinterpret_cast<uint4*>(vt + a * 128 * 128 + y) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
          }
          const uint32_t dv = ring_v + vslot * (C::TILE_BYTES >> 4);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            if (b && 2 * j + 1 >= n) break;        // no visible key in the second half
            ok = pack_wait(&bar_pfull[g][b], (uint32_t)(up[b]++) & 1u, &abort_flag, p.limit_ns);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kPkHalf / 16; ++kk)
                mma_f16_ts_lo(ocol, scol + 64 * b + 8 * kk, dv + (uint32_t)(((64 * b + kk * 16) * 128) >> 4), hi,
                              C::IDESC_PV, b || kk || j > 0);
              if (2 * j + b + 1 == n || b) {
                mma_commit(&bar_empty[vslot]);
                if (j + 1 == nt)
                  mma_commit(&bar_odone[g]);
                else
                  issue_s(at % C::RING, j + 2 == nt);
              }
            }
            __syncwarp();
          }
          if (!ok) break;
        }
        ok = ok && skip_to(m);
      }
      if (elect_one()) {
        if (!ok) {
          abort_flag = 1;
          report_error(-6);
        }
        // drain: every issued MMA completes before TMEM is released
        mma_commit(&bar_drain[g]);
        mbar_wait(&bar_drain[g], 0, &never_abort, p.limit_ns);
      }
      __syncwarp();
    }
  } else {
    // ================= softmax, rescale, epilogue: thread = row =================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    const int g = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const int row_tok = row / p.G, row_head = row % p.G;
    const bool row_in = row < p.TQ * p.G;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_addr = tbase + lanes + C::S_COL + 128 * g, o_addr = tbase + lanes + C::O_COL + D * g;
    const float sc = p.scale_log2;
    int us = 0, uo = 0;        // S tiles and O tiles read
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = next_item(k);
      const PackItem& it = items[k % kPkItems];
      if (!ok || it.stop) break;
      const int slot = it.slot[g];
      const int tok = row_tok + (it.narrow ? 0 : g * p.TQ);   // token of the item
      const bool valid = row_in && it.q0 + tok < it.q_end && slot > -2;
      const bool warp_live = __any_sync(0xffffffffu, valid);
      // keys [0, seen) of the sequence are visible to this row
      const int seen = (p.causal && !it.prefix) ? max(0, min(it.lk, it.t0 + tok + it.off + 1)) : it.lk;
      const int my_nh = it.nh[g], lo = it.lo[g], ahead = seen - lo * kPkKeys;
      const int my_nt = (my_nh + 1) / 2;
      float m_use = -INFINITY, l_run = 0.f, top;   // reference, sum, maximum of the tile
      const int whole = __reduce_min_sync(0xffffffffu, ahead);   // keys that all rows of the warp see
      for (int j = 0; j < my_nt; ++j) {
        ok = pack_wait(&bar_sfull[g], (uint32_t)(us++) & 1u, &abort_flag, p.limit_ns);
        if (!ok) break;
        const bool two = 2 * j + 1 < my_nh;
        if (!warp_live) {          // no rows: the scores only have to be handed back
          if (lane == 0) {
            mbar_arrive(&bar_pfull[g][0]);
            if (two) mbar_arrive(&bar_pfull[g][1]);
          }
          continue;
        }
        tc_fence_after();
        uint32_t sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(*reinterpret_cast<uint32_t(*)[32]>(&sv[32 * c]));
        if (j * kPkKeys + kPkKeys > whole) {              // some row does not see all of this tile
          const int nv = ahead - j * kPkKeys;
#pragma unroll
          for (int b = 0; b < kPkKeys; b += kPkHalf) {
            if (b + kPkHalf + j * kPkKeys > whole) {
#pragma unroll
              for (int c = b; c < b + kPkHalf; ++c)
                if (c >= nv) sv[c] = 0xFF800000u;         // -inf
            }
          }
        }
        const float* f = reinterpret_cast<const float*>(sv);
        auto maximum = [&]() {
          float t8[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float a = fmaxf(f[i], f[i + 8]);
#pragma unroll
            for (int c = 16; c < 112; c += 16) a = fmax3(a, f[i + c], f[i + c + 8]);
            t8[i] = fmax3(a, f[i + 112], f[i + 120]);
          }
          return fmaxf(fmax3(t8[0], t8[1], t8[2]), fmax3(t8[3], t8[4], fmax3(t8[5], t8[6], t8[7]))) * sc;
        };
        // takes `top` as the reference of the rows that it has passed, and the sums with it
        auto move = [&]() {
          const bool grow = top > m_use + kPkLazy;        // also the first finite maximum
          const float alpha = grow ? ex2f(m_use - top) : 1.f;   // 0 from -inf
          if (grow) m_use = top;
          l_run *= alpha;
          if (j == 0) return;
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
        };
        top = maximum();
        if (__any_sync(0xffffffffu, top > m_use + kPkLazy)) move();
        uint32_t pk[32];
        uint64_t sum2[4];
        // P of columns [from, from + 2 pairs): exponentials, their sums, bf16 pairs
        auto exponentials = [&](int from, int pairs) {
          const float at = m_use == -INFINITY ? 0.f : m_use;  // nothing visible yet: exp2(-inf - 0) = 0
          const uint64_t sc2 = f2pack(sc, sc), nm2 = f2pack(-at, -at);
#pragma unroll
          for (int i = 0; i < pairs; ++i) {
            const int c = from + 2 * i;
            float x0, x1;
            f2unpack(fma2(f2pack(f[c], f[c + 1]), sc2, nm2), x0, x1);
            float p0, p1;                      // in this order (reordered by the compiler: 2 % slower)
            asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(x0));
            asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(x1));
            sum2[i & 3] = add2(sum2[i & 3], f2pack(p0, p1));
            const __nv_bfloat162 hb = __floats2bfloat162_rn(p0, p1);
            pk[(c & 63) >> 1] = *reinterpret_cast<const uint32_t*>(&hb);
          }
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) sum2[i] = 0;
        // The two warps of a scheduler (one of each stream) take turns with their exponentials: both
        // at once leave the special function unit idle while both wait for their MMAs (480p grid
        // 10.5 ms without, 9.9 with).  Nothing depends on it: after 100 looks, longer than a turn of
        // 1,600 clocks, or where both look at once, they go ahead together.
        for (int spin = 0; spin < 100 && busy[1 - g][quarter]; ++spin) {}
        if (lane == 0) busy[g][quarter] = 1;
        exponentials(0, 32);
        tmem_st32(s_addr, pk);
        if (two) {
          // the first half is on its way while the second starts
          exponentials(64, 8);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar_pfull[g][0]);
          exponentials(80, 24);
          tmem_st32(s_addr + 64, pk);
        }
        if (lane == 0) busy[g][quarter] = 0;
        float a0, a1, b0, b1;
        f2unpack(add2(sum2[0], sum2[1]), a0, a1);
        f2unpack(add2(sum2[2], sum2[3]), b0, b1);
        l_run += (a0 + a1) + (b0 + b1);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar_pfull[g][two ? 1 : 0]);
      }
      if (ok && my_nh > 0) {
        ok = pack_wait(&bar_odone[g], (uint32_t)(uo++) & 1u, &abort_flag, p.limit_ns);
        tc_fence_after();
      }
      if (ok && !warp_live) {
        done_item(k);
        continue;
      }
      if (!ok) break;
      const int head = it.head[g] * p.G + row_head;
      const int from = lo * kPkKeys;                          // keys [from, to) were computed
      const int to = min(it.lk, from + my_nh * kPkHalf);
      const bool any = valid && seen > from && my_nh > 0;        // this row saw a key
      const long long tr = it.q0 + tok;
      // partial row of token t and query head h
      auto part_row = [&](long long t, int h) { return ((long long)slot * it.step + it.row0 + t) * (p.Hkv * p.G) + h; };
      const long long prow = part_row(tr, head);
      // rows without a key, rows with hidden keys: neither in most items
      const bool odd = !__all_sync(0xffffffffu, any || !valid) || __any_sync(0xffffffffu, any && seen < to);
      float check = 0.f;
      const float inv = any ? 1.0f / l_run : 0.f;
      const uint64_t inv2 = f2pack(inv, inv);
      __nv_bfloat16* to_row = p.o + head * p.osH + tr * p.osL;
      float* to_part = p.part + prow * D;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        if (my_nh > 0) {
          tmem_ld32(o_addr + c, o);
          tmem_wait_ld();
          reg_fence32(o);
        }
        if (odd) {
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = any ? __uint_as_float(o[i]) : 0.f;
            check = fmaf(x, 0.f, check);
            o[i] = __float_as_uint(x);
          }
        }
        // a lane writes whole 32-byte sectors of its row
        if (slot < 0) {
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              f2unpack(mul2(f2pack(__uint_as_float(o[16 * w + 2 * i]), __uint_as_float(o[16 * w + 2 * i + 1])), inv2), x0, x1);
              const __nv_bfloat162 hb = __floats2bfloat162_rn(x0, x1);
              y[i] = *reinterpret_cast<const uint32_t*>(&hb);
            }
            __nv_bfloat16* dst = to_row + c + 16 * w;
            if (valid) {
              if (p.sectors) {
                st_global_32b(dst, y);
              } else {
                *reinterpret_cast<uint4*>(dst) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(dst + 8) = make_uint4(y[4], y[5], y[6], y[7]);
              }
            }
          }
        } else if (valid) {
#pragma unroll
          for (int w = 0; w < 4; ++w) st_global_32b(to_part + c + 8 * w, o + 8 * w);
        }
      }
      if (valid) {
        if (slot >= 0)
          p.ml[prow] = any ? make_float2(m_use, l_run) : make_float2(-INFINITY, 0.f);
        else if (p.lse)
          p.lse[(long long)head * p.Tq + tr] = any ? pack_lse(m_use, l_run) : -INFINITY;
      }
      // rows that a hidden key's non-finite V may have spoilt
      uint32_t redo = __ballot_sync(0xffffffffu, any && check != check && seen < to);
      if (redo) __syncwarp();   // the rows' own stores come first
      while (redo) {
        const int src = __ffs(redo) - 1;
        redo &= redo - 1;
        const int s_seen = __shfl_sync(0xffffffffu, seen, src), s_head = __shfl_sync(0xffffffffu, head, src);
        const int s_tr = __shfl_sync(0xffffffffu, (int)tr, src);
        const __nv_bfloat16* kb = p.k.p + it.head[g] * p.k.sH + (long long)it.k0 * p.k.sL;
        const __nv_bfloat16* vb = p.v.p + it.head[g] * p.v.sH + (long long)it.k0 * p.v.sL;
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
                            sc, const_cast<int*>(&abort_flag), o, m, l);
        const long long s_prow = part_row(s_tr, s_head);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (slot < 0)
            p.o[s_head * p.osH + s_tr * p.osL + lane * E + e] = __float2bfloat16(o[e] / l);
          else
            p.part[s_prow * D + lane * E + e] = o[e];
        }
        if (lane == 0) {
          if (slot >= 0)
            p.ml[s_prow] = make_float2(m, l);
          else if (p.lse)
            p.lse[(long long)s_head * p.Tq + s_tr] = pack_lse(m, l);
        }
      }
      done_item(k);
    }
    if (!ok) {
      abort_flag = 1;
      report_error(-6);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, C::TMEM_COLS);
  }
}

// Joins the splits of each row: a warp per row (three CTAs per SM walk them), lane = D / 32 channels, splits in
// ascending order (the result does not depend on which item finished first).
template <int D>
__global__ void __launch_bounds__(256) packed_combine_kernel(const PackParams p) {
  constexpr int E = D / 32;
  const int Hq = p.Hkv * p.G, lane = threadIdx.x & 31;
  const long long R = (long long)p.Tq * Hq;
  asm volatile("griddepcontrol.wait;\n\tgriddepcontrol.launch_dependents;" ::: "memory");   // the partial rows are complete
  if (p.chunk[1]) return;
  const int c = p.chunk[0], most = p.chunk[2];
  const long long turn = (long long)gridDim.x * 8;
  for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < R; row += turn) {
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
    const int start = p.Lp ? 0 : p.start[lo];   // (on its way with the lengths)
    const PackSeq s = pack_seq(p, lo);
    if (tok < s.q0 || tok >= s.q0 + s.lq) continue;
    int rows = 0;
    if (p.Lp) {  // a malformed table may leave rows without their prefix part
      const PackSeq all = pack_all(p);
      if (tok < all.q0 || tok >= all.q0 + all.lq) continue;
      rows = all.lq;
    }
    const int np = p.Lp ? pack_splits(p, rows, pack_tiles(p.Lp), c, p.max_np) : 0;
    const int ns = (p.Lp && s.lk == 0) ? 0 : pack_seq_splits(p, s, c, most);
    if (!p.Lp && ns == 1) {   // its items finished its rows: on to the first one behind them
      row += ((long long)(s.q0 + s.lq) * Hq - 1 - row) / turn * turn;
      continue;
    }
    // (where a wait ran out, an item may not have said where its partial rows are)
    if (!p.Lp && (start < 0 || start + (long long)s.lq * ns > p.room)) continue;
    // its partial rows, and how far apart the splits' are
    const long long first = p.Lp ? row : (long long)(start + tok - s.q0) * Hq + head;
    const long long apart = p.Lp ? R : (long long)s.lq * Hq;
    float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    // 32 splits at a time, a weight in each lane; the rows of 8 are on their way together, with
    // the maxima and sums (one after another: 10.8 us instead of 8.3 for 2,560 rows of 12 splits)
    for (int b = 0; b < np + ns; b += 32) {
      const int count = min(32, np + ns - b);
      const long long base = (long long)b * apart + first;
      const float2 x = lane < count ? p.ml[base + lane * apart] : make_float2(-INFINITY, 0.f);
      float w = 0.f;
      for (int i = 0; i < count; i += 8) {
        float y[8][E];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float* src = p.part + (base + (i + u) * apart) * D + lane * E;
          if constexpr (E == 4) {
            const float4 z = i + u < count ? *reinterpret_cast<const float4*>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
            y[u][0] = z.x, y[u][1] = z.y, y[u][2] = z.z, y[u][3] = z.w;
          } else {
            const float2 z = i + u < count ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
            y[u][0] = z.x, y[u][1] = z.y;
          }
        }
        if (i == 0) {
          float top = fmaxf(m, x.x);
#pragma unroll
          for (int v = 16; v; v >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, v));
          const float at = top == -INFINITY ? 0.f : top, a = ex2f(m - at);   // 0 from -inf
          w = ex2f(x.x - at);
          float sum = w * x.y;
#pragma unroll
          for (int v = 16; v; v >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, v);
          l = fmaf(l, a, sum);
          m = top;
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] *= a;
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const float wu = __shfl_sync(0xffffffffu, w, (i + u) & 31);
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(wu, y[u][e], o[e]);
        }
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
}

}  // namespace lx
