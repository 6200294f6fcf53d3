// Attention of chunks of new tokens over a paged KV cache, for sm_100a.
//
// A batch of ragged chunks: sequence b holds n_b = seqlens[b] keys in its pages, and the packed
// query rows [cu[b], cu[b + 1]) are its last new_b positions: row i sits at pos = n_b - new_b + i.
// Query head h reads key/value head h / G (G = Hq / Hkv). For each of them
//   O = softmax(scale * q . k_j) V over the visible keys,  LSE = ln sum_j exp(scale * q . k_j);
// key j < n_b is visible when j <= pos + win_r (win_r = 0 under causal masking; -1: no bound) and
// when j >= pos - win_l (-1: no bound) or j < sinks: a sliding window beside which the sequence's
// first keys stay visible. A row that sees no key gets O = 0 and LSE = -inf.
//
// Rows of a tile: the G query heads of a key/value head share its keys, so a 128-row tile holds
// tq = 128 / G consecutive tokens times their G heads (row = token * G + head), and a block of
// work is kTiles such tiles that share every K/V load. Its keys are visited in 128-key tiles: the
// sink tiles before the window, then the window's (all tiles without one).
//
// Work split: for each group of hg heads, the key tiles of all blocks are listed block after block;
// the lists of all groups, one after another, are cut into P equal contiguous pieces. A piece takes
// hg CTAs, one for each head of the group, next to each other; in all one CTA per SM. So every CTA
// visits the same number of key tiles (within one), for decoding steps, long prompts and mixtures
// alike, and the heads' rows of a token, which lie side by side in a page, are read at about the
// same time: DRAM serves 512 bytes and more at a stretch, not 128 or 256. A block that lies in one
// piece is finished by its CTA;
// otherwise each of its pieces writes a partial (O / l, log2 l + m) and fa_chunk_merge_kernel joins
// them by their log-sum-exp. (The CTA that finished a block last used to join it: one CTA reading
// all partials of 64 rows took 60 us of a 178 us call, 32 query heads over 131072 keys.)
//
// Both products run on the tensor core, with the forward's roles and order of issue: S_t(v + 1)
// ahead of P V_t(v), a row's 128 scores split over two warps that exchange their maxima, P in
// TMEM, O rescaled only when a row's maximum has grown by more than 2^8, O divided by the sum of
// the rounded weights.
//
// E4M3 pages (kF8): the codes of a K or V tile and their power-of-two scales are loaded as they
// are, and eight warps write the tile's values, code * 2^e, as bf16 into the operand buffers: exact,
// since a code has 4 significant bits. The products then are those of bf16 pages holding these
// values, bit for bit; 8-bit products would have to split Q and P into three terms each, which pays
// for few rows (fa_chunk_few.cuh) and not where the tensor core and the softmax set the pace.
//
// What bounds it: over bf16 pages few rows read the cache at 1.40 us a tile of 128 keys (64 KB a
// CTA, 6.9 TB/s in all); two tiles of rows take 2.2 us a key tile at d = 128 (1130 TFLOP/s, the
// forward's rate: the softmax's instruction stream, tensor pipe 58%) and 2.1 at d = 64; over E4M3
// pages 2.9, of which the conversion's arithmetic is 0.5 (without it 2.3). A call adds 12 to 25 us:
// launch 3, set-up until the first scores 6 (cold instructions), first tile 1.5, join 3 to 8.
// Measured steps: one thread that walks over the blocks for all roles in place of every role (63 ->
// 46 us, window with sinks, with the masks as bits); the page entry of the next tile read one tile
// ahead (144 -> 120 us, mixed chunks over E4M3 pages); set-up by four warps and not all (5 us).
// Not kept: K and V converted by four warps each (rings of one and two tiles: 3.3 us for 2.4),
// blocks weighted by their rows in the work split (116 us for 113).
#pragma once

#include "fa_cache.cuh"
#include "fa_decode.cuh"
#include "fa_fwd.cuh"

namespace fa {

// Division of 0 <= n < 2^31 by a number known on the host: n / d = (n + hi(n m)) >> s with
// s = ceil(log2 d), m = ceil(2^(32 + s) / d) - 2^32.
struct FastDiv {
  unsigned m, s;
  __device__ __forceinline__ int operator()(int n) const { return (int)((__umulhi((unsigned)n, m) + (unsigned)n) >> s); }
};

struct ChunkParams {
  int B, total, Hq, Hkv, G;
  int tq;          // tokens per 128-row tile: 128 / G
  int page_size;
  FastDiv by_page, by_group, by_tokens;  // page_size, G, tokens of a block (kTiles * tq)
  int box_rows;    // rows of one page box: the largest power of two that divides page_size, <= 128
  int max_pages, num_pages;
  float scale_log2;  // scale * log2(e)
  int win_l, win_r;  // -1 = unbounded, else < 2^30, as positions; causal already folded into win_r = 0
  int sinks;         // first keys that stay visible left of the window
  int pieces;        // P: the pieces of a head group's list
  int hg;            // heads of a group, on CTAs next to each other
  int ctas;          // P * hg
  const int* block_table;  // (B, max_pages)
  const int* seqlens;      // (B)
  const int* cu;           // (B + 1)
  __nv_bfloat16* o;        // (total, Hq, d)
  float* lse;              // (Hq, total), natural log
  float* o_part;           // (2 ctas, kTiles, d / 4, 128, 4) fp32: a warp's rows lie side by side
  float* lse_part;         // (2 ctas, kTiles * 128), log2 domain
  int4* split;             // (ctas) the block that starts in the CTA's piece and goes on: first packed row,
                           // tokens (0: none), head, 2 * (pieces it goes on through) + (its first partial
                           // is slot 2 cta + 1)
};

template <int D, bool kF8, int kTiles>
struct ChunkCfg {
  static constexpr int kSoftWarps = 8 * kTiles;       // row split: two warps per 32 rows
  static constexpr int kSoftThreads = 32 * kSoftWarps;
  static constexpr int kConvThreads = kF8 ? 256 : 0;  // (with 128: 2.7 us a tile for 2.4)
  static constexpr int kConvWarps = kConvThreads / 32;
  static constexpr int kThreads = 128 + kSoftThreads + kConvThreads;
  static constexpr int kBlockReaders = 2 + kSoftWarps + kConvThreads / 32;  // the loads', the MMAs', ...
  static constexpr int kRegs = 65536 / kThreads / 8 * 8;  // a thread's at launch
  // (the load and MMA roles spill below 80: 56 cost more there than 104 gained the softmax)
  static constexpr int kLoadRegs = kF8 && kTiles == 2 ? 56 : 80, kConvRegs = kTiles == 2 ? 48 : 64;
  static constexpr int kSoftRegs = kTiles == 2 ? (kF8 ? 88 : 96) : kF8 ? 128 : 0;  // 0: as launched
  static_assert(kSoftRegs * kSoftThreads + kLoadRegs * 128 + kConvRegs * kConvThreads <= kRegs * kThreads, "registers");
  static constexpr int kBoxes = D / 64;               // 128-byte boxes per bf16 row
  static constexpr int kTileBytes = 128 * D * 2;      // a bf16 tile of Q, K or V
  static constexpr int kRawBytes = 128 * D;           // the codes of a K or V tile
  static constexpr int kRawSlotBytes = kRawBytes + 1024;  // codes, then the scales of each page box at 128 bytes
  static constexpr int kSlots = kF8 ? (D == 64 ? 5 : 3) : (D == 64 ? 10 : kTiles == 2 ? 4 : 5);
  static constexpr int kRawSlots = kF8 ? (D == 64 ? 9 : kTiles == 2 ? 3 : 5) : 0;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kTiles * kTileBytes;
  static constexpr int kOffRaw = kOffKV + kSlots * kTileBytes;
  static constexpr int kOffX = kOffRaw + kRawSlots * kRawSlotBytes;
  static constexpr int kXBytes = 4096 * kTiles;       // per tile: maxima [parity][half][row], sums [sum][half][row]
  static constexpr int kOffBar = kOffX + kXBytes;
  static constexpr int kSmemBytes = kOffBar + 1536 + 1024;  // barriers + alignment slack
  static constexpr bool kShareS = kTiles == 2 && D == 128;  // one S buffer for both tiles
  static constexpr uint32_t kColS0 = 0, kColS1 = kShareS ? 0 : 128;
  static constexpr uint32_t kColP0 = kShareS ? 128 : 384, kColP1 = kShareS ? 192 : 448;
  static constexpr uint32_t kColO0 = 256, kColO1 = 256 + D;
  static constexpr uint32_t kTmemCols = 512;
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

// A sequence: first packed row, rows and keys. Offsets or lengths out of range make it empty
// (reported by report_bad_batch).
struct ChunkSeq {
  int c0, rows, n;
};
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b) {
  ChunkSeq s;
  s.c0 = p.cu[b];
  const int c1 = p.cu[b + 1], n = p.seqlens[b];
  s.rows = (s.c0 < 0 || c1 < s.c0 || c1 > p.total) ? 0 : c1 - s.c0;
  s.n = (n < 0 || n > (long long)p.max_pages * p.page_size) ? 0 : n;
  return s;
}

// Keys visible to some row of a block, and the tiles that hold them: tile v of the block is key
// tile v for v < ns (sinks left of the window), lo + v - ns from there on; cnt >= 1 in all (a
// block that sees nothing visits one tile with every key masked).
struct ChunkKeys {
  int vis_lo, vis_hi;  // window part (vis_hi < 0: nothing visible)
  int ns, lo, cnt;
  __device__ __forceinline__ int tile(int v) const { return v < ns ? v : lo + v - ns; }
};
__device__ __forceinline__ ChunkKeys chunk_keys(const ChunkParams& p, int n, int pos0, int pos1) {
  ChunkKeys k;
  k.vis_lo = p.win_l >= 0 ? max(0, pos0 - p.win_l) : 0;
  k.vis_hi = p.win_r >= 0 ? min(n - 1, pos1 + p.win_r) : n - 1;
  k.ns = 0;
  k.lo = 0;
  k.cnt = 1;
  if (pos1 < 0 || k.vis_hi < 0) {
    k.vis_hi = -1;
    return k;
  }
  k.lo = min(k.vis_lo, k.vis_hi) >> 7;
  k.ns = min((int)(((long long)min(p.sinks, n) + 127) >> 7), k.lo);
  k.cnt = k.ns + (k.vis_hi >> 7) - k.lo + 1;
  return k;
}

// A block as its roles need it: head h, sequence b of n keys, ntok tokens from packed row c0 on, the
// first at position pos0; key tiles [v0, v1) of it belong to this CTA's piece.
struct ChunkBlock {
  int h, b, n, c0, ntok, pos0;
  ChunkKeys keys;
  int v0, v1;  // v1 = 0: the end of the list
  int slot;    // of its partial result; -1: the block lies in the piece as a whole
};
// One thread walks over the piece's blocks and hands them to the other roles through a ring.
constexpr int kBlockRing = 4;

template <class Cfg>
struct ChunkBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[Cfg::kSlots], kv_empty[Cfg::kSlots];
  uint64_t raw_full[Cfg::kRawSlots + 1], raw_empty[Cfg::kRawSlots + 1];
  uint64_t s_full[2], s_empty[2], p_full[2], pv_done[2];
  uint64_t block_full[kBlockRing], block_empty[kBlockRing];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  long long u0, u1, th;     // the piece, the length of one head's list
  long long first_start;    // the piece's first block: its position on the list of all heads
  int first_h, first_b, first_blk;
  ChunkSeq first_seq;
  long long sums[3][4];     // scans
  int many[4];
  ChunkBlock block[kBlockRing];
};

// A walk over the blocks of one piece: block blk of sequence b for head h.
template <int kTiles>
struct ChunkWalk {
  long long u0, u1;  // the piece's range of the list of all heads
  int h, b, blk;
  ChunkSeq s;
  ChunkKeys keys;
  long long start;  // position of the block's first tile on the list of all heads
  int i0, ntok;

  __device__ __forceinline__ void set(const ChunkParams& p) {
    const int tokens = kTiles * p.tq;
    i0 = blk * tokens;
    ntok = min(tokens, s.rows - i0);
    const int pos0 = s.n - s.rows + i0;
    keys = chunk_keys(p, s.n, pos0, pos0 + ntok - 1);
  }
  __device__ __forceinline__ bool valid() const { return start < u1; }
  __device__ __forceinline__ bool whole() const { return start >= u0 && start + keys.cnt <= u1; }
  template <class Bars>
  __device__ __forceinline__ void begin(const ChunkParams& p, const Bars* bars) {
    u0 = bars->u0;
    u1 = bars->u1;
    start = bars->first_start;
    if (!valid()) return;
    h = bars->first_h;
    b = bars->first_b;
    blk = bars->first_blk;
    s = bars->first_seq;
    set(p);
  }
  __device__ __forceinline__ void next(const ChunkParams& p) {
    start += keys.cnt;
    if (!valid()) return;
    if (++blk * kTiles * p.tq >= s.rows) {
      blk = 0;
      do {
        if (++b == p.B) {
          b = 0;
          h += p.hg;
        }
        s = chunk_seq(p, b);
      } while (s.rows == 0);
    }
    set(p);
  }
  __device__ __forceinline__ ChunkBlock block() const {
    return {h, b, s.n, s.c0 + i0, ntok, s.n - s.rows + i0, keys, (int)max(0LL, u0 - start),
            (int)min((long long)keys.cnt, u1 - start), whole() ? -1 : 2 * (int)blockIdx.x + (start > u0 ? 1 : 0)};
  }
};

// The list of all head groups, T tiles, in pieces: the first T % pieces of them one tile longer.
struct ChunkSplit {
  long long each, more;
  __device__ __forceinline__ ChunkSplit(long long T, int pieces) {
    if (T < (1LL << 31)) {  // (a 64-bit division is some 100 instructions)
      each = (unsigned)T / (unsigned)pieces;
    } else {
      each = T / pieces;
    }
    more = T - each * pieces;
  }
  __device__ __forceinline__ long long lo(int r) const { return each * r + min((long long)r, more); }
  __device__ __forceinline__ int of(long long u) const {  // the piece that holds tile u
    const long long head = more * (each + 1);
    return u < head ? (int)(u / (each + 1)) : (int)(more + (u - head) / each);
  }
};

// Publishes the piece's blocks, and the block that the piece hands on to the next one (for the merge).
template <int kTiles, class Bars>
__device__ __forceinline__ void chunk_publish(const ChunkParams& p, Bars* bars, Abort ab) {
  ChunkWalk<kTiles> w;
  int4 split = make_int4(0, 0, 0, 0);
  uint32_t i = 0;
  auto put = [&](const ChunkBlock& b) {
    const uint32_t slot = i % kBlockRing;
    mbar_wait(smem_u32(&bars->block_empty[slot]), ((i / kBlockRing) & 1) ^ 1, ab);
    bars->block[slot] = b;
    mbar_arrive(smem_u32(&bars->block_full[slot]));
    ++i;
  };
  for (w.begin(p, bars); w.valid() && !ab.raised(); w.next(p)) {
    put(w.block());
    if (!w.whole() && w.start >= w.u0) {
      const long long T = bars->th * (p.Hkv / p.hg);
      const int last = ChunkSplit(T, (int)min((long long)p.pieces, T)).of(w.start + w.keys.cnt - 1);
      split = make_int4(w.s.c0 + w.i0, w.ntok, w.h, 2 * (last - (int)blockIdx.x / p.hg) + (w.start > w.u0 ? 1 : 0));
    }
  }
  if (!ab.raised()) put(ChunkBlock{});
  if (dbg_range(ab, blockIdx.x, 1, p.ctas)) p.split[blockIdx.x] = split;
}
// Block i of the piece (all lanes of a warp, or one thread); null: there is none, or the CTA gave up.
template <class Bars>
__device__ __forceinline__ const ChunkBlock* chunk_take(Bars* bars, uint32_t i, Abort ab) {
  const uint32_t slot = i % kBlockRing;
  const bool ok = mbar_wait(smem_u32(&bars->block_full[slot]), (i / kBlockRing) & 1, ab);
  return ok && bars->block[slot].v1 > 0 ? &bars->block[slot] : nullptr;
}
template <class Bars>
__device__ __forceinline__ void chunk_release(Bars* bars, uint32_t i) {
  mbar_arrive(smem_u32(&bars->block_empty[i % kBlockRing]));
}
// True for all `threads` threads at the barrier when it is for each of them.
__device__ __forceinline__ bool all_agree(bool x, uint32_t id, uint32_t threads) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// The set-up of one CTA by 128 threads (tid 0..127 here): which piece is its own, and where the
// piece's first block lies. Blocks are counted per run of sequences, then key tiles per run of
// blocks. (All the CTA's warps used to take part: what bounds this is the issue of its
// instructions, several thousand cycles with 20 warps.)
constexpr int kPlanThreads = 128;
__device__ __forceinline__ long long plan_scan(long long x, long long (&sums)[4], int tid, long long& total) {
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, x, off);
    if ((tid & 31) >= off) x += v;
  }
  if ((tid & 31) == 31) sums[tid >> 5] = x;
  named_bar_sync(1, kPlanThreads);
  const long long a = sums[0], b = a + sums[1], c = b + sums[2];
  total = c + sums[3];
  const int w = tid >> 5;
  return x + (w == 0 ? 0 : w == 1 ? a : w == 2 ? b : c);
}
template <int kTiles, class Bars>
__device__ __forceinline__ void chunk_plan(const ChunkParams& p, Bars* bars, int* run_base, int tid) {
  const int run = (p.B + kPlanThreads - 1) / kPlanThreads;
  const int rb0 = min(p.B, tid * run), rb1 = min(p.B, rb0 + run);
  const int tokens = kTiles * p.tq;
  auto blocks_of = [&](const ChunkSeq& s) { return p.by_tokens(s.rows + tokens - 1); };
  auto tiles_of = [&](const ChunkSeq& s, int blk) {
    const int i0 = blk * tokens, pos0 = s.n - s.rows + i0;
    return chunk_keys(p, s.n, pos0, pos0 + min(tokens, s.rows - i0) - 1).cnt;
  };
  // Few blocks per run (decoding steps, short chunks): their tiles are counted at once.
  constexpr int kFew = 4;
  long long blocks = 0, tiles = 0, nb, th;
  for (int b = rb0; b < rb1; ++b) {
    const ChunkSeq s = chunk_seq(p, b);
    const int m = blocks_of(s);
    blocks += m;
    for (int k = 0; k < m && blocks <= kFew; ++k) tiles += tiles_of(s, k);
  }
  const bool many = __any_sync(0xffffffffu, blocks > kFew);
  if ((tid & 31) == 0) bars->many[tid >> 5] = many;
  long long incl = plan_scan(tiles, bars->sums[0], tid, th);
  int b = rb0, blk = 0;      // this thread's first block, and how many it has
  long long mine = blocks;
  if (bars->many[0] | bars->many[1] | bars->many[2] | bars->many[3]) {
    // The blocks of all sequences are dealt out evenly; a thread's first is found by the run that holds it.
    const long long blocks_incl = plan_scan(blocks, bars->sums[1], tid, nb);
    run_base[tid] = (int)(blocks_incl - blocks);
    named_bar_sync(1, kPlanThreads);
    const long long each = (nb + kPlanThreads - 1) / kPlanThreads;
    const long long q0 = min(nb, each * tid);
    mine = min(nb, q0 + each) - q0;
    if (mine > 0) {
      int lo = 0;
#pragma unroll
      for (int step = kPlanThreads / 2; step > 0; step >>= 1)
        if (run_base[lo + step] <= q0) lo += step;
      b = min(lo * run, p.B - 1);
      blk = (int)(q0 - run_base[lo]);
    }
  }
  // visit the thread's blocks in order; f(sequence, block, its rows and keys, tiles) until it returns false
  auto visit = [&](auto f) {
    int bb = b, kk = blk;
    for (long long q = 0; q < mine && bb < p.B;) {
      const ChunkSeq s = chunk_seq(p, bb);
      const int nbb = blocks_of(s);
      if (kk >= nbb) {
        kk -= nbb;
        ++bb;
        continue;
      }
      if (!f(bb, kk, s, tiles_of(s, kk))) return;
      ++kk;
      ++q;
    }
  };
  if (bars->many[0] | bars->many[1] | bars->many[2] | bars->many[3]) {
    tiles = 0;
    visit([&](int, int, const ChunkSeq&, int cnt) {
      tiles += cnt;
      return true;
    });
    incl = plan_scan(tiles, bars->sums[2], tid, th);
  }
  const long long excl = incl - tiles;
  const long long T = th * (p.Hkv / p.hg);
  const int pe = (int)min((long long)p.pieces, T), r = blockIdx.x / p.hg;
  long long u0 = T, u1 = T;
  if (r < pe && T > 0) {
    const ChunkSplit split(T, pe);
    u0 = split.lo(r);
    u1 = split.lo(r + 1);
  }
  if (tid == 0) {
    bars->u0 = u0;
    bars->u1 = u1;
    bars->th = th;
    if (u0 >= u1) bars->first_start = u1;
  }
  if (u0 >= u1) return;
  const int h = u0 < (1LL << 31) && th < (1LL << 31) ? (int)((unsigned)u0 / (unsigned)th) : (int)(u0 / th);
  const long long w0 = u0 - (long long)h * th;
  if (excl <= w0 && w0 < incl) {
    long long at = excl;
    visit([&](int bb, int kk, const ChunkSeq& s, int cnt) {
      if (w0 >= at + cnt) {
        at += cnt;
        return true;
      }
      bars->first_h = h * p.hg + blockIdx.x % p.hg;
      bars->first_b = bb;
      bars->first_blk = kk;
      bars->first_seq = s;
      bars->first_start = at + (long long)h * th;
      return false;
    });
  }
}

// E4M3 codes, four in a word, to bf16 values times f (two packed factors per row: f, and g for
// scales whose exponent does not fit one factor). A code's exponent and mantissa bits, shifted
// into a bf16's, are the value times 2^-120 (subnormals included); f makes up for it.
__device__ __forceinline__ uint32_t e4m3_pair_bits(uint32_t spread) {  // bytes at bits 8..15 and 24..31
  return ((spread >> 4) & 0x07f007f0u) | (spread & 0x80008000u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two-dimensional tiled load (the scales of E4M3 pages).
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::
          "r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}

// Which of 64 keys from kbase on a row sees: those in [kmin, kmax] and the first `sinks` up to kmax.
__device__ __forceinline__ uint32_t bits_below(int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ void chunk_visible(int kbase, int kmin, int kmax, int sinks, uint32_t (&m)[2]) {
  const int from = kmin - kbase, end = kmax + 1 - kbase, first = min(sinks, kmax + 1) - kbase;
#pragma unroll
  for (int w = 0; w < 2; ++w)
    m[w] = (bits_below(end - 32 * w) & ~bits_below(from - 32 * w)) | bits_below(first - 32 * w);
}

// Exponentials of 32 scores (16 pairs from pair k0 on) against the reference maximum, packed to bf16
// pairs and summed twice, as fwd_exp_chunk, but all on MUFU: the forward's degree-3 polynomial (off by
// 7.5e-5) would show in the log-sum-exp of rows of a few keys, and a degree-5 one for one pair in four,
// eight or sixteen was not faster here (111 to 117 us against 111, mixed chunks over E4M3 pages).
template <bool kPosScale, int kC>
__device__ __forceinline__ void chunk_exp(const float (&x)[kC], int k0, float c, float m_use, uint32_t (&pk)[16],
                                          float2& sum, float2& rsum) {
  const float2 neg_m = make_float2(-m_use, -m_use), c2 = make_float2(c, c);
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 xv = make_float2(x[2 * (k0 + k)], x[2 * (k0 + k) + 1]);
    const float2 a = kPosScale ? fma2(xv, c2, neg_m) : add2(xv, neg_m);
    const float2 pv = make_float2(ex2_approx(a.x), ex2_approx(a.y));
    sum = add2(sum, pv);
    pk[k] = pack_bf16x2(pv.x, pv.y);
    rsum = add_bf16x2_f32x2(pk[k], rsum);
  }
}

template <int D, bool kF8, int kTiles>
__global__ void __launch_bounds__(ChunkCfg<D, kF8, kTiles>::kThreads, 1)
    fa_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmKs,
                    const __grid_constant__ CUtensorMap tmVs, const ChunkParams p) {
  using Cfg = ChunkCfg<D, kF8, kTiles>;
  using Bars = ChunkBars<Cfg>;
  static_assert(sizeof(Bars) <= 1536, "barrier block");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem_base - smem_u32(smem_raw));
  const uint32_t smem_end = smem_u32(smem_raw) + Cfg::kSmemBytes;  // for the FA_DEBUG bounds checks
  Bars* bars = reinterpret_cast<Bars*>(smem_gen + Cfg::kOffBar);
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = lane_id();
  const Abort ab{&bars->abort_flag};
  const long long max_keys = (long long)p.max_pages * p.page_size;

  griddep_launch_dependents();  // the merge takes an SM as soon as its CTA is done, and waits there
  // (Launched as a programmatic dependent itself: up to griddep_wait nothing of global memory is touched.)
  // set-up, a part per warp: barriers (a lane each), TMEM, tensor maps, and the piece of this CTA
  if (warp == 2) {
    if (lane == 0) bars->abort_flag = 0;
    constexpr int kBars = offsetof(Bars, mma_done) / 8 + 1, kPer = (kBars + 31) / 32;
    constexpr int kKv = offsetof(Bars, kv_full) / 8, kRaw = offsetof(Bars, raw_full) / 8, kS = offsetof(Bars, s_full) / 8;
    const uint32_t first = bar(bars->q_full[0]);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int i = lane + 32 * j;
      int count = 1;
      if (kF8 && i >= kKv && i < kKv + Cfg::kSlots) count = Cfg::kConvWarps;               // kv_full: converting warps
      if (kF8 && i >= kRaw + Cfg::kRawSlots + 1 && i < kS) count = Cfg::kConvWarps;         // raw_empty
      if (i >= kS + 2 && i < kS + 6) count = 256;                                           // s_empty, p_full
      if (i >= kBars - 1 - kBlockRing && i < kBars - 1) count = Cfg::kBlockReaders;         // block_empty
      if (i < kBars) mbar_init(first + i * 8, count);
    }
    fence_barrier_init();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), Cfg::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  } else if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
  } else if (warp >= 4 && warp < 8) {
    // (over the Q buffer: no load is in flight yet)
    griddep_wait();
    chunk_plan<kTiles>(p, bars, reinterpret_cast<int*>(smem_gen), tid - 128);
    fence_proxy_async_smem();  // the Q loads may overwrite it
  }
  griddep_wait();  // what ran before on the stream is done and visible
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  const uint32_t sKV = smem_base + Cfg::kOffKV, sRaw = smem_base + Cfg::kOffRaw;
  auto sQ = [&](int t) { return smem_base + Cfg::kOffQ + t * Cfg::kTileBytes; };

  // Registers: the launch gives each thread the same number (Cfg::kRegs); the producer and MMA warps
  // and the converting ones hand some back, and the softmax warps take them. The sum stays within
  // the launch's.
  if (warp < 4) {
  if constexpr (Cfg::kSoftRegs > 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kLoadRegs) : "memory");
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer (all lanes)
    // Lane l loads page box l % groups of 64-column box l / groups (E4M3: lanes from 16 on the
    // scales of a box). Boxes of keys that no row of the block sees are filled with zeros by a
    // coordinate past the pool: their page entries are not read.
    const int groups = 128 / p.box_rows;
    const int grp = (kF8 ? lane & 15 : lane) % groups, col = (kF8 ? lane & 15 : lane) / groups;
    const bool loads = col < (kF8 ? 1 : Cfg::kBoxes), scales = kF8 && lane >= 16;
    const uint32_t box_off = (uint32_t)grp * p.box_rows;
    uint32_t n = 0, qn[2] = {0, 0};  // K/V tiles issued, Q tiles issued
    constexpr int kRing = kF8 ? Cfg::kRawSlots : Cfg::kSlots;
    // page and row of this lane's box of tile v of block w; row -1: no page (zeros)
    auto place = [&](const ChunkBlock& w, int v, int& page, int& row) {
      const int key = w.keys.tile(v) * 128 + (int)box_off, last = key + p.box_rows - 1;
      row = -1;  // no page
      if (!loads || key > w.keys.vis_hi || (last < w.keys.vis_lo && key >= p.sinks)) return;
      const int in_seq = p.by_page(key);
      const long long ti = (long long)w.b * p.max_pages + in_seq;
      if (!dbg_range(ab, ti, 1, (long long)p.B * p.max_pages)) return;
      page = p.block_table[ti];
      row = key - in_seq * p.page_size;
    };
    int page = 0, row = 0;
    const ChunkBlock* block;
    for (uint32_t i = 0; (block = chunk_take(bars, i, ab)) && !ab.raised(); ++i) {
      const ChunkBlock& w = *block;
      const int nact = (kTiles == 2 && w.ntok > p.tq) ? 2 : 1;
      if (lane == 0) {
        for (int t = 0; t < nact; ++t) {
          mbar_wait(bar(bars->q_empty[t]), (qn[t] & 1) ^ 1, ab);
          const int tok = w.c0 + t * p.tq;
          bool ok = true;
          for (int bx = 0; bx < Cfg::kBoxes; ++bx)
            ok = ok && dbg_tma(ab, bx * 64, 0, w.h, tok, D, p.G, p.Hkv, p.total, 2, sQ(t) + bx * 16384, 16384,
                               smem_base, smem_end);
          if (!ok) break;
          mbar_arrive_expect_tx(bar(bars->q_full[t]), (uint32_t)(p.tq * p.G * D * 2));
#pragma unroll
          for (int bx = 0; bx < Cfg::kBoxes; ++bx)
            tma_load_4d(sQ(t) + bx * 16384, &tmQ, bar(bars->q_full[t]), bx * 64, 0, w.h, tok);
          ++qn[t];
        }
      }
      __syncwarp();
      place(w, w.v0, page, row);
      const int h = w.h;
      for (int v = w.v0; v < w.v1 && !ab.raised(); ++v) {
        // (looked at only now: the entry was read while the tile before was loaded)
        int pg = p.num_pages, rw = 0;
        if (row >= 0) {
          if (page >= 0 && page < p.num_pages) {
            pg = page;
            rw = row;
          } else {
            atomicOr(&g_fa_error, kErrBadInput);
          }
        }
        if (v + 1 < w.v1) place(w, v + 1, page, row);  // the next tile's page, read while this one waits
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const uint32_t slot = n % kRing, phase = (n / kRing) & 1;
          uint64_t& full = kF8 ? bars->raw_full[slot] : bars->kv_full[slot];
          mbar_wait(kF8 ? bar(bars->raw_empty[slot]) : bar(bars->kv_empty[slot]), phase ^ 1, ab);
          if (FA_DEBUG) {  // (page num_pages, the zero fill, lies just past the pool)
            const uint32_t to = kF8 ? sRaw + slot * Cfg::kRawSlotBytes + box_off * D
                                    : sKV + slot * Cfg::kTileBytes + col * 16384 + box_off * 128;
            const bool ok = !loads || dbg_tma(ab, kF8 ? 0 : col * 64, h, rw, pg, D, p.Hkv, p.page_size,
                                              p.num_pages + 1, kF8 ? 1 : 2, to, p.box_rows * (kF8 ? D : 128),
                                              smem_base, smem_end);
            if (!__all_sync(0xffffffffu, ok)) break;
          }
          if (lane == 0)
            mbar_arrive_expect_tx(bar(full), kF8 ? (uint32_t)(Cfg::kRawBytes + 128) : (uint32_t)Cfg::kTileBytes);
          __syncwarp();
          if constexpr (kF8) {
            const uint32_t base = sRaw + slot * Cfg::kRawSlotBytes;
            if (loads && !scales)
              tma_load_4d(base + box_off * D, kv ? &tmV : &tmK, bar(full), 0, h, rw, pg);
            else if (loads)
              tma_load_2d(base + Cfg::kRawBytes + grp * 128, kv ? &tmVs : &tmKs, bar(full), rw, pg * p.Hkv + h);
          } else if (loads) {
            tma_load_4d(sKV + slot * Cfg::kTileBytes + col * 16384 + box_off * 128, kv ? &tmV : &tmK, bar(full),
                        col * 64, h, rw, pg);
          }
        }
      }
      __syncwarp();
      if (lane == 0) chunk_release(bars, i);
    }
    // every load issued lands before the CTA exits
    for (uint32_t i = n > kRing ? n - kRing : 0; i < n; ++i)
      mbar_drain(kF8 ? bar(bars->raw_full[i % kRing]) : bar(bars->kv_full[i % kRing]), (i / kRing) & 1);
    if (lane == 0)
      for (int t = 0; t < 2; ++t)
        if (qn[t] > 0) mbar_drain(bar(bars->q_full[t]), (qn[t] - 1) & 1);
  } else if (warp == 3) {
    if (lane == 0) chunk_publish<kTiles>(p, bars, ab);
  } else if (warp == 2) {
    if (blockIdx.x == 0) report_bad_batch(p.cu, p.seqlens, p.B, p.total, max_keys, lane, 32);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (elect_one()) {
      constexpr uint32_t idS = idesc_bf16_f32(128, 128, false, false);  // S = Q K^T (both K-major)
      constexpr uint32_t idO = idesc_bf16_f32(128, D, false, true);     // O += P V (V MN-major)
      const uint32_t tS[2] = {tmem + Cfg::kColS0, tmem + Cfg::kColS1};
      const uint32_t tO[2] = {tmem + Cfg::kColO0, tmem + Cfg::kColO1};
      const uint32_t tP[2] = {tmem + Cfg::kColP0, tmem + Cfg::kColP1};
      uint32_t kvn = 0, qn[2] = {0, 0}, pn[2] = {0, 0}, sn[2] = {0, 0};
      auto kv_wait = [&](uint32_t n) {
        const uint32_t s = n % Cfg::kSlots;
        mbar_wait(bar(bars->kv_full[s]), (n / Cfg::kSlots) & 1, ab);
        tc_fence_after_sync();
        return s;
      };
      auto issue_s = [&](int t, uint32_t ks, bool last) {  // once the S before it in the buffer has been read
        const int buf = Cfg::kShareS ? 0 : t;
        mbar_wait(bar(bars->s_empty[buf]), (sn[buf] & 1) ^ 1, ab);
        ++sn[buf];
        tc_fence_after_sync();
        const uint32_t k_smem = sKV + ks * Cfg::kTileBytes;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_ss(tS[t], sdesc_kmajor(sQ(t) + off), sdesc_kmajor(k_smem + off), idS, kk > 0);
        }
        mma_commit(bar(bars->s_full[t]));
        if (last) mma_commit(bar(bars->q_empty[t]));  // the block's last read of Q_t
      };
      auto issue_pv = [&](int t, uint32_t vs, bool first) {
        mbar_wait(bar(bars->p_full[t]), pn[t] & 1, ab);
        ++pn[t];
        tc_fence_after_sync();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tO[t], tP[t] + kk * 8, sdesc_mnmajor(sKV + vs * Cfg::kTileBytes + kk * 2048, 16384), idO,
                 !first || kk > 0);
        mma_commit(bar(bars->pv_done[t]));
      };
      const ChunkBlock* block;
      for (uint32_t i = 0; (block = chunk_take(bars, i, ab)); ++i) {
        const ChunkBlock& w = *block;
        const int nact = (kTiles == 2 && w.ntok > p.tq) ? 2 : 1, nv = w.v1 - w.v0;
        for (int t = 0; t < nact; ++t) mbar_wait(bar(bars->q_full[t]), (qn[t]++) & 1, ab);
        tc_fence_after_sync();
        uint32_t ks = kv_wait(kvn);
        for (int t = 0; t < nact; ++t) issue_s(t, ks, nv == 1);
        mma_commit(bar(bars->kv_empty[ks]));
        for (int v = 0; v < nv; ++v) {
          const bool more = v + 1 < nv;
          const uint32_t vs = kv_wait(kvn + 1);
          kvn += 2;
          if (more) ks = kv_wait(kvn);
          for (int t = 0; t < nact; ++t) {
            if (more) issue_s(t, ks, v + 2 == nv);
            if (more && t == nact - 1) mma_commit(bar(bars->kv_empty[ks]));
            issue_pv(t, vs, v == 0);
          }
          mma_commit(bar(bars->kv_empty[vs]));
        }
        chunk_release(bars, i);
      }
      mma_commit(bar(bars->mma_done));
      mbar_drain(bar(bars->mma_done), 0);
    }
  }
  } else if (warp < 4 + Cfg::kSoftWarps) {
    if constexpr (Cfg::kSoftRegs > 0)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kSoftRegs) : "memory");
    // ---------------------------------------------------------------- softmax + epilogue
    constexpr int kC = 64;                                    // scores of a row per thread and key tile
    const int t = kTiles == 2 ? ((warp - 4) >> 2) & 1 : 0;    // tile of the block
    const int half = (warp - 4) >> (kTiles == 2 ? 3 : 2);     // columns [64 half, 64 half + 64)
    const int row = (tid - 128) & 127;                        // TMEM lane and row within the tile
    const uint32_t lane_field = (uint32_t)((row & ~31) << 16);
    const uint32_t tS = tmem + lane_field + (t ? Cfg::kColS1 : Cfg::kColS0) + kC * half;
    const uint32_t tO = tmem + lane_field + (t ? Cfg::kColO1 : Cfg::kColO0);
    const uint32_t tP = tmem + lane_field + (t ? Cfg::kColP1 : Cfg::kColP0) + (kC / 2) * half;
    float* xm = reinterpret_cast<float*>(smem_gen + Cfg::kOffX) + t * 1024;  // [parity][half][row]
    float* xl = xm + 512;                                                    // [sum][half][row]
    uint32_t sn = 0, pvn = 0, xu = 0, vn = 0;  // vn: key tiles of this CTA so far (K/V stream position 2 vn)
    auto pair_sync = [&]() { named_bar_sync(4 + 4 * t + (row >> 5), 64); };
    const float c = p.scale_log2;
    const bool pos_scale = c > 0.0f;
    const int tok_in_tile = p.by_group(row), head_in_group = row - tok_in_tile * p.G;

    for (uint32_t bi = 0;; ++bi) {
      const ChunkBlock* block = chunk_take(bars, bi, ab);
      // (both warps of a pair go on, or neither: they meet at its barrier)
      if (!all_agree(block != nullptr, 4 + 4 * t + (row >> 5), 64)) break;
      const ChunkBlock& w = *block;
      const int nv = w.v1 - w.v0;
      const int tile_tok = min(p.tq, w.ntok - t * p.tq);  // tokens of this tile (<= 0: no such tile)
      const int rows = tile_tok * p.G;                    // its rows
      const bool act = tile_tok > 0, live = (row & ~31) < rows;  // (live: some row of this warp)
      const int pos_lo = w.pos0 + t * p.tq, pos_hi = pos_lo + tile_tok - 1;
      const int pos = pos_lo + tok_in_tile;
      const bool mine = row < rows;
      const int kmax = (!mine || pos < 0) ? -1
                       : p.win_r >= 0     ? min(w.n - 1, pos + p.win_r)
                                          : w.n - 1;
      const int kmin = p.win_l >= 0 ? max(0, pos - p.win_l) : 0;
      float m_run = -INFINITY, l_run = 0.0f, lr_run = 0.0f;

      for (int v = 0; act && v < nv; ++v) {
        const int key0 = w.keys.tile(w.v0 + v) * 128;
        mbar_wait(bar(bars->s_full[t]), sn & 1, ab);
        ++sn;
        tc_fence_after_sync();
        if (!live) {  // no row of this warp: keep the barriers' counts
          mbar_arrive(bar(bars->s_empty[Cfg::kShareS ? 0 : t]));
          if (v > 0) {
            mbar_wait(bar(bars->pv_done[t]), pvn & 1, ab);
            ++pvn;
          }
          mbar_arrive(bar(bars->p_full[t]));
          continue;
        }
        uint32_t r[kC / 32][32];
#pragma unroll
        for (int q4 = 0; q4 < kC / 32; ++q4) tmem_ld32(tS + q4 * 32, r[q4]);
#pragma unroll
        for (int q4 = 0; q4 < kC / 32; ++q4) tmem_wait_ld(r[q4]);
        tc_fence_before_sync();  // the S buffer may now take the next scores
        mbar_arrive(bar(bars->s_empty[Cfg::kShareS ? 0 : t]));
        float x[kC];
#pragma unroll
        for (int cc = 0; cc < kC; ++cc) x[cc] = __uint_as_float(r[cc >> 5][cc & 31]);

        const int k1 = key0 + 127, kbase = key0 + kC * half;
        const bool all = pos_lo >= 0 && k1 < w.n && (p.win_r < 0 || k1 <= pos_lo + p.win_r) &&
                         (p.win_l < 0 || key0 >= pos_hi - p.win_l || k1 < p.sinks);
        bool none = false;  // no score of this warp is visible
        uint32_t m[2] = {~0u, ~0u};
        if (!all) {
          chunk_visible(kbase, kmin, kmax, p.sinks, m);
          none = __all_sync(0xffffffffu, (m[0] | m[1]) == 0u);
          if (!none && !__all_sync(0xffffffffu, (m[0] & m[1]) == ~0u)) {
#pragma unroll
            for (int cc = 0; cc < kC; ++cc) x[cc] = (m[cc >> 5] >> (cc & 31)) & 1u ? x[cc] : -INFINITY;
          }
        }
        float m_tile = -INFINITY;
        if (!none) {
          if (pos_scale) {
            m_tile = fwd_tile_max<true>(x, false, 0, 0, 0, c);
          } else {  // masked scores stay -inf whatever the scale's sign (a visible -inf does not)
#pragma unroll
            for (int cc = 0; cc < kC; ++cc) {
              x[cc] = (m[cc >> 5] >> (cc & 31)) & 1u ? x[cc] * c : -INFINITY;
              m_tile = fmaxf(m_tile, x[cc]);
            }
          }
        }
        {
          float* slot = xm + (xu & 1) * 256;
          slot[half * 128 + row] = m_tile;
          pair_sync();
          m_tile = fmaxf(m_tile, slot[(half ^ 1) * 128 + row]);
          ++xu;
        }
        float alpha;
        bool updated;
        fwd_update_max(m_tile, m_run, alpha, updated);
        const float m_use = (m_run == -INFINITY) ? 0.0f : m_run;
        if (v > 0) {  // P V of the tile before has read P_t, and O_t is quiescent
          mbar_wait(bar(bars->pv_done[t]), pvn & 1, ab);
          ++pvn;
          tc_fence_after_sync();
        }
        float2 sum = make_float2(0.0f, 0.0f), rsum = make_float2(0.0f, 0.0f);
        if (none) {
          uint32_t pk[16] = {};
#pragma unroll
          for (int q4 = 0; q4 < kC / 32; ++q4) tmem_st16(tP + q4 * 16, pk);
        } else {
#pragma unroll
          for (int q4 = 0; q4 < kC / 32; ++q4) {
            uint32_t pk[16];
            if (pos_scale)
              chunk_exp<true>(x, q4 * 16, c, m_use, pk, sum, rsum);
            else
              chunk_exp<false>(x, q4 * 16, c, m_use, pk, sum, rsum);
            tmem_st16(tP + q4 * 16, pk);
          }
        }
        l_run = l_run * alpha + (sum.x + sum.y);
        lr_run = lr_run * alpha + (rsum.x + rsum.y);
        if (__any_sync(0xffffffffu, updated && v > 0)) {
#pragma unroll 1
          for (int cc = (D / 2) * half; cc < (D / 2) * (half + 1); cc += 32) {
            uint32_t o[32];
            tmem_ld32(tO + cc, o);
            tmem_wait_ld(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + cc, o);
          }
        }
        if constexpr (!kF8) {
          // V rows that no row of the block sees may hold anything, a NaN among it: 0 (their
          // weights are 0). The live warps of each tile write the same zeros before their P V.
          const int keys_end = w.keys.vis_hi - key0 + 1;  // rows from here on
          const int win_from = w.keys.vis_lo - key0, sink_end = p.sinks - key0;  // and rows [sink_end, win_from)
          if (keys_end < 128 || (win_from > 0 && sink_end < 128)) {
            const uint32_t vi = 2 * (vn + v) + 1, vs = vi % Cfg::kSlots;
            mbar_wait(bar(bars->kv_full[vs]), (vi / Cfg::kSlots) & 1, ab);
            const int lw = min(4, (rows + 31) >> 5);  // live warps per half
            const int li = (half * lw + (row >> 5)) * 32 + lane, chunk = li & (Cfg::kBoxes * 8 - 1);
            const uint32_t to = sKV + vs * Cfg::kTileBytes + (chunk >> 3) * 16384 + (chunk & 7) * 16;
            auto clear = [&](int from, int end) {
              for (int vr = from + li / (Cfg::kBoxes * 8); vr < end; vr += 64 * lw / (Cfg::kBoxes * 8))
                st_shared_v4(to + vr * 128, 0u, 0u, 0u, 0u);
            };
            const int end = max(0, min(128, keys_end));
            clear(end, 128);
            clear(max(0, sink_end), min(win_from, end));
            fence_proxy_async_smem();
          }
        }
        tmem_wait_st();
        tc_fence_before_sync();
        mbar_arrive(bar(bars->p_full[t]));
      }

      // ---- epilogue: O / (sum of the weights applied) and the log-sum-exp, final or partial
      const bool whole = w.slot < 0;
      if (act) {
        mbar_wait(bar(bars->pv_done[t]), pvn & 1, ab);
        ++pvn;
        tc_fence_after_sync();
      }
      if (act && live) {
        xl[half * 128 + row] = l_run;
        xl[256 + half * 128 + row] = lr_run;
        pair_sync();
        const float l_tot = l_run + xl[(half ^ 1) * 128 + row];
        const float l_o = lr_run + xl[256 + (half ^ 1) * 128 + row];
        const float inv_l = l_o > 0.0f ? 1.0f / l_o : 0.0f;
        const float lse2 = l_tot > 0.0f ? m_run + lg2_approx(l_tot) : (l_tot == l_tot ? -INFINITY : l_tot);
        const bool dead = !(l_o > 0.0f) && l_o == l_o;  // no visible key (a NaN sum is not one)
        const long long tok = (long long)w.c0 + t * p.tq + tok_in_tile;
        const int head = w.h * p.G + head_in_group;
        const long long ptile = (long long)w.slot * kTiles + t;
        const long long o_size = (long long)p.total * p.Hq * D, part_rows = 2LL * p.ctas * kTiles * 128;
#pragma unroll 1
        for (int cc = (D / 2) * half; cc < (D / 2) * (half + 1); cc += 32) {
          uint32_t o[32];
          tmem_ld32(tO + cc, o);
          tmem_wait_ld(o);
          if (!mine) continue;
          const float mul = l_o == l_o ? inv_l : l_o;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = dead ? 0u : __float_as_uint(__uint_as_float(o[e]) * mul);
          if (whole) {
            const long long oi = (tok * p.Hq + head) * D + cc;
            if (dbg_range(ab, oi, 32, o_size)) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                uint4 q;
                q.x = pack_bf16x2(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
                q.y = pack_bf16x2(__uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
                q.z = pack_bf16x2(__uint_as_float(o[e + 4]), __uint_as_float(o[e + 5]));
                q.w = pack_bf16x2(__uint_as_float(o[e + 6]), __uint_as_float(o[e + 7]));
                *reinterpret_cast<uint4*>(p.o + oi + e) = q;
              }
            }
          } else if (dbg_range(ab, ptile * 128 * D + (cc / 4 * 128 + row) * 4, 28 * 128 + 4, part_rows * D)) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              reinterpret_cast<uint4*>(p.o_part + ptile * 128 * D)[(cc + e) / 4 * 128 + row] =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (mine && half == 0) {
          const long long li = (long long)head * p.total + tok;
          if (!whole) {
            if (dbg_range(ab, ptile * 128 + row, 1, part_rows)) p.lse_part[ptile * 128 + row] = lse2;
          } else if (dbg_range(ab, li, 1, (long long)p.Hq * p.total)) {
            p.lse[li] = lse2 == -INFINITY ? -INFINITY : lse2 * kLn2;
          }
        }
        tc_fence_before_sync();
      }
      vn += nv;
      __syncwarp();
      if (lane == 0) chunk_release(bars, bi);
    }
  } else {
    if constexpr (kF8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kConvRegs) : "memory");
      // ---------------------------------------------------------------- E4M3 codes -> bf16 operand tiles
      constexpr int kPerRow = D / 16;  // 16-byte pieces of codes in a row
      constexpr int kRowStep = Cfg::kConvThreads / kPerRow;
      const int ct = tid - 128 - Cfg::kSoftThreads;
      const int c = ct % kPerRow;      // this thread's piece, in rows ct / kPerRow + k * kRowStep
      const int box_shift = 31 - __clz(p.box_rows), odd = c >> 2;
      uint32_t n = 0;
      const ChunkBlock* block;
      for (uint32_t i = 0; (block = chunk_take(bars, i, ab)); ++i) {
        const ChunkBlock& w = *block;
        for (int v = w.v0; v < w.v1; ++v) {
          const int key0 = w.keys.tile(v) * 128;
          const int hi = w.keys.vis_hi - key0, lo = w.keys.vis_lo - key0, sinks = p.sinks - key0;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv, ++n) {
            const uint32_t rs = n % Cfg::kRawSlots, ks = n % Cfg::kSlots;
            mbar_wait(bar(bars->raw_full[rs]), (n / Cfg::kRawSlots) & 1, ab);
            mbar_wait(bar(bars->kv_empty[ks]), ((n / Cfg::kSlots) & 1) ^ 1, ab);
            const uint8_t* raw = smem_gen + Cfg::kOffRaw + rs * Cfg::kRawSlotBytes;
            const uint8_t* scale = raw + Cfg::kRawBytes;
            const uint32_t dst = sKV + ks * Cfg::kTileBytes;
            // (all loads ahead of the stores, which the compiler would keep them behind)
            uint4 xs[128 / kRowStep];
            uint32_t ss[128 / kRowStep];
#pragma unroll
            for (int k = 0; k < 128 / kRowStep; ++k) {
              const int row = ct / kPerRow + k * kRowStep;
              xs[k] = reinterpret_cast<const uint4*>(raw)[row * kPerRow + c];
              ss[k] = scale[((row >> box_shift) << 7) + (row & (p.box_rows - 1))];
            }
#pragma unroll
            for (int k = 0; k < 128 / kRowStep; ++k) {
              const int row = ct / kPerRow + k * kRowStep;
              uint4 x = xs[k];
              uint32_t s = ss[k];
              // V rows that no row of the block sees may hold anything: 0 (their weights are 0)
              if (kv && (row > hi || (row < lo && row >= sinks))) {
                x = make_uint4(0u, 0u, 0u, 0u);
                s = 127u;
              }
              const uint32_t f = (min(s, 134u) + 120u) << 7, ff = f | (f << 16);  // 2^(s - 127 + 120), bf16
              const uint32_t in[4] = {x.x, x.y, x.z, x.w};
              uint32_t r[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                r[2 * e] = mul_bf16x2(e4m3_pair_bits(__byte_perm(in[e], 0u, 0x1404)), ff);
                r[2 * e + 1] = mul_bf16x2(e4m3_pair_bits(__byte_perm(in[e], 0u, 0x3424)), ff);
              }
              if (s > 134u) {  // scales above 2^7: a second factor; NaN for s = 255
                const uint32_t g = s == (uint32_t)kScaleNan ? 0x7fc0u : (s - 134u + 127u) << 7;
#pragma unroll
                for (int e = 0; e < 8; ++e) r[e] = mul_bf16x2(r[e], g | (g << 16));
              }
              // two 16-byte chunks; the upper half of a row's threads stores its odd chunk first, so
              // that the eight threads of a row (d = 128) touch all banks in each store
              const uint32_t to = dst + (uint32_t)(c >> 2) * 16384u + row * 128;
              const uint32_t a0 = to + (((2 * (c & 3) + odd) ^ (row & 7)) << 4);
              const uint32_t a1 = to + (((2 * (c & 3) + 1 - odd) ^ (row & 7)) << 4);
              st_shared_v4(a0, odd ? r[4] : r[0], odd ? r[5] : r[1], odd ? r[6] : r[2], odd ? r[7] : r[3]);
              st_shared_v4(a1, odd ? r[0] : r[4], odd ? r[1] : r[5], odd ? r[2] : r[6], odd ? r[3] : r[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(bars->raw_empty[rs]));
              mbar_arrive(bar(bars->kv_full[ks]));
            }
          }
        }
        __syncwarp();
        if (lane == 0) chunk_release(bars, i);
      }
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

// Joins the blocks that are spread over several pieces: CTA (r, y) takes the block that starts in
// CTA r's piece and goes on, if there is one, and of it rows [8 y, 8 y + 8): a thread takes four columns of
// one row. A row's partials are weighted by 2^(their log-sum-exp - the largest), in piece order: the
// same sum in every run. Bound by the latency of the partials, which lie in L2: kBatch of them, with
// their log-sum-exps, are on their way at once (few rows are spread over many pieces, two tiles of
// rows over two or three). Launched as the main kernel's programmatic dependent: an SM takes it as
// soon as its CTA of the main kernel is done.
constexpr int kMergeThreads = 256, kMergeRows = 8;
template <int D, int kTiles>
__global__ void __launch_bounds__(kMergeThreads) fa_chunk_merge_kernel(const ChunkParams p) {
  constexpr int kBatch = kTiles == 2 ? 4 : 16;
  const Abort none{nullptr};
  griddep_wait();  // the pieces have been written
  const int pf = blockIdx.x;
  const int4 s = p.split[pf];
  const int m = (s.w >> 1) + 1, first = blockIdx.y * kMergeRows, nrows = min(kMergeRows, s.y * p.G - first);
  if (nrows <= 0 || !dbg_range(none, pf, (m - 1) * p.hg + 1, p.ctas)) return;
  // a warp's threads: rows side by side (their number rounded up to a power of two), then columns
  const int shift = nrows <= 1 ? 0 : 32 - __clz(nrows - 1);
  for (int e = threadIdx.x; e < (D / 4) << shift; e += kMergeThreads) {
    const int rr = first + (e & ((1 << shift) - 1)), c4 = e >> shift;
    if (rr - first >= nrows) continue;
    const int itok = p.by_group(rr), t = itok >= p.tq ? 1 : 0, srow = rr - t * p.tq * p.G;
    float mx = -INFINITY, wsum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int from = 0; from < m; from += kBatch) {
      float4 o4[kBatch];
      float lse[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        lse[i] = -INFINITY;
        o4[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (from + i >= m) continue;
        const long long tile = (2LL * (pf + (from + i) * p.hg) + (from + i == 0 ? (s.w & 1) : 0)) * kTiles + t;
        lse[i] = ld_global_cg(p.lse_part + tile * 128 + srow);
        o4[i] = ld_global_cg(reinterpret_cast<const float4*>(p.o_part + tile * 128 * D) + c4 * 128 + srow);
      }
      float most = mx;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) most = fmaxf(most, lse[i]);
      const float ref = most == -INFINITY ? 0.0f : most, down = ex2_approx(mx - ref);  // (0 at first)
      wsum *= down;
      acc = make_float4(acc.x * down, acc.y * down, acc.z * down, acc.w * down);
      mx = most;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = ex2_approx(lse[i] - ref);
        wsum += w;
        acc.x = fmaf(w, o4[i].x, acc.x);
        acc.y = fmaf(w, o4[i].y, acc.y);
        acc.z = fmaf(w, o4[i].z, acc.z);
        acc.w = fmaf(w, o4[i].w, acc.w);
      }
    }
    const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
    const int head = s.z * p.G + rr - itok * p.G;
    const long long tok = (long long)s.x + itok, oi = (tok * p.Hq + head) * D + c4 * 4;
    const long long li = (long long)head * p.total + tok;
    if (dbg_range(none, oi, 4, (long long)p.total * p.Hq * D))
      *reinterpret_cast<uint2*>(p.o + oi) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (c4 == 0 && dbg_range(none, li, 1, (long long)p.Hq * p.total))
      p.lse[li] = wsum == 0.0f ? -INFINITY : ((mx == -INFINITY ? 0.0f : mx) + lg2_approx(wsum)) * kLn2;
  }
}

}  // namespace fa
