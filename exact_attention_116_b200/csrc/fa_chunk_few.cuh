// Attention of a few new tokens over a paged E4M3 cache, for sm_100a: fa_chunk.cuh's operation, list
// of key tiles, pieces and partials, for blocks of at most 16 rows (tokens times the query heads of
// a key/value head) and d = 128: decoding steps.
//
// The codes go from the cache to the tensor core as they lie. Both products are transposed, so that
// the cache is operand A and the few rows are its narrow partner:
//   S^T (128 keys x 16 rows) = K Q^T,   O^T (128 columns x 16 rows) += V^T W^T.
// A key is then a lane, and its scales, 2^ek and 2^ev, are scalars of the lane's thread:
//   score(row, key) = S * 2^ek * scale,   W(row, key) = P(row, key) * 2^(ev - E).
// Q and W are sums of three E5M2 numbers, each the remainder of the ones before rounded to 3
// significant bits: bf16 queries (8 bits) exactly, weights to 9 bits (bf16 keeps 8), with the range
// of E5M2 below the largest: a query's elements down to 2^-31 of its row's largest, W down to 2^-26 of
// the row's largest and its 9 bits down to 2^-17 of it. Products of E4M3 and E5M2 codes are exact, sums
// are fp32. The three terms of Q go into one accumulator, those of W are 3 x 16 columns of one product
// (V is read once).
//
// Against bf16 operand tiles made from the codes (fa_chunk.cuh): no conversion, which took 2.4 us a
// tile of 128 keys on one SM, and half the shared-memory traffic. Bound by HBM: 33 KB a tile in
// 0.82 us, 6.0 TB/s in all; a step of 48 sequences (873 MB) in 148 to 150 us, 135 at the copy rate. How it got
// there: one tile at a time 218 us, 128- or 256-byte reads of neighbouring heads at about the same
// time 207, all waits of a step ahead of its loads 184, a lane per wait and straight-line code for
// the number of row pairs 153, one reference per row for scores and values 150 (16 rows: 240 to 230;
// with a second reference for each row's values 286). With 16 rows a pair of tiles takes 4500 cycles, all
// in the softmax.
//
// Per tile a thread handles one key: x = score - the row's reference m (log2), P = 2^x rounded to 9
// bits, summed before (log-sum-exp) and after the rounding (divisor of O). E is fixed at the block's first
// keys (their largest ev, within [-14, 24]), and m is the row's largest score + ev, less E: so every row's
// largest W is near 2^10, whatever the values are that other rows see or that it gives no weight. (With m
// from the scores alone and E the block's largest ev, a key with values 2^28 times larger that one of the
// rows sees took all bits from the weights of the others.) P itself is then about 2^(E - ev), in fp32's
// range with 2^-26 to spare below for ev from E - 96 to E + 100. Where a block's values differ by more, m is
// held to the scores' maximum less 96 and plus 100: O loses bits, or its largest weights end at E5M2's
// largest number, and the log-sum-exp stands. The references move only when some x + ev exceeds E + 5, which one barrier's vote tells; then
// the exact maxima are taken and O is rescaled. W <= 2^(5 + 10), E5M2 ends at 1.75 * 2^15.
//
// Warps: 0 loads; 1 issues MMAs; 4-7 softmax and epilogue (and the set-up); 8-11 split the next
// block's queries, ahead.
#pragma once

#include "fa_chunk.cuh"

namespace fa {

constexpr int kFewRows = 16, kFewTerms = 3, kFewSlots = 5;
constexpr int kFewBufs = 4;        // tiles of scores and of weights in flight: two pairs
constexpr int kFewThreads = 384;
constexpr int kFewD = 128;
constexpr float kFewGrow = 5.0f;   // log2: how far P * 2^ev may exceed 2^E
constexpr int kFewShift = 10;      // W = P * 2^(ev - E + 10)
constexpr int kFewLeastE = -14, kFewMostE = 24, kFewNoE = -1000;  // (-1000: not fixed yet)
constexpr int kFewSpan = 96;       // P <= 2^(96 + 5): sums of 2^26 of them stay in fp32's range
constexpr int kFewRise = 100;      // and a row's largest P >= 2^-100

struct FewCfg {
  static constexpr int kSlotBytes = 128 * kFewD + 1024;  // codes, then the scales of each page box at 128 bytes
  static constexpr int kQBytes = kFewTerms * kFewRows * kFewD, kWBytes = kFewTerms * kFewRows * 128;
  static constexpr int kOffK = 0, kOffV = kFewSlots * kSlotBytes;
  static constexpr int kOffQ = 2 * kFewSlots * kSlotBytes;  // two buffers
  static constexpr int kOffW = kOffQ + 2 * kQBytes;
  static constexpr int kOffX = kOffW + kFewBufs * kWBytes;         // maxima and sums: [warp][row], three of them
  static constexpr int kOffBar = kOffX + 1024;
  static constexpr int kSmemBytes = kOffBar + 1536 + 1024;
  static constexpr uint32_t kColS = 0, kColO = 64, kTmemCols = 128;  // S: buffers of 16 columns
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
};

struct FewBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t full[2][kFewSlots], empty[2][kFewSlots];  // K, V tiles
  uint64_t s_full[kFewBufs], s_empty[kFewBufs], w_full[kFewBufs], pv_done[kFewBufs];
  uint64_t block_full[kBlockRing], block_empty[kBlockRing];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort_flag;
  long long u0, u1, th, first_start;  // (as ChunkBars)
  int first_h, first_b, first_blk;
  ChunkSeq first_seq;
  long long sums[3][4];
  int many[4];
  ChunkBlock block[kBlockRing];
  float q_factor[2][kFewRows];  // log2 score per unit of S, before the key's scale
};

// kind::f8f6f4 with E4M3 A and E5M2 B.
__host__ __device__ constexpr uint32_t idesc_e4m3_e5m2(uint32_t M, uint32_t N, bool a_mn_major) {
  return idesc_e4m3_f32(M, N, a_mn_major, false) | (1u << 10);
}

// x to s significant bits, nearest: c - (c - x) with c = (2^(24 - s) + 1) x.
template <int kBits>
__device__ __forceinline__ float2 round_bits2(float2 x) {
  constexpr float k = (float)(1 << (24 - kBits)) + 1.0f;
  const float2 c = mul2(x, make_float2(k, k));
  const float2 e = fma2(x, make_float2(-1.0f, -1.0f), c);
  return fma2(e, make_float2(-1.0f, -1.0f), c);
}
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, make_float2(-1.0f, -1.0f), a); }
__device__ __forceinline__ uint32_t pack_e5m2x2(float2 x) {  // x.x in the low byte
  uint16_t d;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(d) : "f"(x.y), "f"(x.x));
  return d;
}
// x as three E5M2 pairs whose sum is x to 9 bits.
__device__ __forceinline__ void split_e5m2(float2 x, uint32_t (&t)[kFewTerms]) {
  const float2 a = round_bits2<3>(x), r = sub2(x, a), b = round_bits2<3>(r);
  t[0] = pack_e5m2x2(a);
  t[1] = pack_e5m2x2(b);
  t[2] = pack_e5m2x2(sub2(r, b));
}
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// True for all 128 softmax threads when it is for one.
__device__ __forceinline__ bool few_vote(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float exp2_int(int e) { return e < -126 ? 0.0f : __int_as_float((e + 127) << 23); }

__global__ void __launch_bounds__(kFewThreads, 1)
    fa_chunk_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const __grid_constant__ CUtensorMap tmKs, const __grid_constant__ CUtensorMap tmVs,
                        const __nv_bfloat16* q, long long q_stride, const ChunkParams p) {
  using Cfg = FewCfg;
  constexpr int D = kFewD;
  static_assert(sizeof(FewBars) <= 1536, "barrier block");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem_base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* smem_gen = smem_raw + (smem_base - smem_u32(smem_raw));
  const uint32_t smem_end = smem_u32(smem_raw) + Cfg::kSmemBytes;  // for the FA_DEBUG bounds checks
  FewBars* bars = reinterpret_cast<FewBars*>(smem_gen + Cfg::kOffBar);
  auto bar = [&](uint64_t& b) { return smem_u32(&b); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = lane_id();
  const Abort ab{&bars->abort_flag};

  griddep_launch_dependents();
  if (warp == 2) {
    if (lane == 0) bars->abort_flag = 0;
    constexpr int kBars = offsetof(FewBars, mma_done) / 8 + 1;
    constexpr int kEmptyK = offsetof(FewBars, empty) / 8, kS = offsetof(FewBars, s_full) / 8;
    const uint32_t first = bar(bars->q_full[0]);
#pragma unroll
    for (int j = 0; j < (kBars + 31) / 32; ++j) {
      const int i = lane + 32 * j;
      int count = 1;
      if (i < 2) count = 128;                                  // q_full: the splitting threads
      else if (i < 4) count = 5;                               // q_empty: the MMAs, the softmax warps
      else if (i >= kEmptyK && i < kEmptyK + kFewSlots) count = 5;  // K tile: the same (its scales)
      else if (i >= kS + kFewBufs && i < kS + 3 * kFewBufs) count = 4;           // s_empty, w_full: the softmax warps
      else if (i >= kBars - 1 - kBlockRing && i < kBars - 1) count = 11;  // block_empty: loads, MMAs, softmax, queries
      if (i < kBars) mbar_init(first + i * 8, count);
    }
    fence_barrier_init();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), Cfg::kTmemCols);
    tmem_relinquish();
    tc_fence_before_sync();
  } else if (warp == 0) {
    if (lane == 0) {
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
      prefetch_tmap(&tmKs);
      prefetch_tmap(&tmVs);
    }
  } else if (warp >= 4 && warp < 8) {
    // (over the W buffers: nothing is in them yet)
    griddep_wait();
    chunk_plan<1>(p, bars, reinterpret_cast<int*>(smem_gen + Cfg::kOffW), tid - 128);
    fence_proxy_async_smem();
  }
  griddep_wait();  // what ran before on the stream is done and visible
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bars->tmem_base;
  auto sT = [&](int kv, uint32_t slot) { return smem_base + (kv ? Cfg::kOffV : Cfg::kOffK) + slot * Cfg::kSlotBytes; };
  const int box_shift = 31 - __clz(p.box_rows);

  if (warp == 0 || warp == 2) {
    // ---------------------------------------------------------------- TMA producers (all lanes): K and V
    // (One warp took 1100 cycles to place and issue the four loads of a tile.) Lane l < 16 loads the
    // codes of page box l of a tile, lane 16 + l its scales; boxes of keys that no row sees are filled
    // with zeros (page num_pages), as in fa_chunk_kernel.
    const int groups = 128 / p.box_rows, grp = lane & 15;
    const bool loads = grp < groups, scales = lane >= 16;
    const uint32_t box_off = (uint32_t)grp * p.box_rows;
    const int kv = warp == 2 ? 1 : 0;
    const CUtensorMap *tm = kv ? &tmV : &tmK, *tms = kv ? &tmVs : &tmKs;
    uint32_t n = 0;
    const ChunkBlock* block;
    for (uint32_t bi = 0; (block = chunk_take(bars, bi, ab)) && !ab.raised(); ++bi) {
      const ChunkBlock& w = *block;
      auto place = [&](int v, int& page, int& row) {
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
      place(w.v0, page, row);
      for (int v = w.v0; v < w.v1 && !ab.raised(); ++v, ++n) {
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
        if (v + 1 < w.v1) place(v + 1, page, row);  // the next tile's page, read while this one waits
        const uint32_t slot = n % kFewSlots, phase = (n / kFewSlots) & 1;
        mbar_wait(bar(bars->empty[kv][slot]), phase ^ 1, ab);
        const uint32_t to = sT(kv, slot) + box_off * D;
        if (FA_DEBUG) {
          const bool ok = !loads || dbg_tma(ab, 0, w.h, rw, pg, D, p.Hkv, p.page_size, p.num_pages + 1, 1, to,
                                            p.box_rows * D, smem_base, smem_end);
          if (!__all_sync(0xffffffffu, ok)) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(bar(bars->full[kv][slot]), 128 * D + 128);
        __syncwarp();
        if (loads && !scales)
          tma_load_4d(to, tm, bar(bars->full[kv][slot]), 0, w.h, rw, pg);
        else if (loads)
          tma_load_2d(sT(kv, slot) + 128 * D + grp * 128, tms, bar(bars->full[kv][slot]), rw, pg * p.Hkv + w.h);
      }
      __syncwarp();
      if (lane == 0) chunk_release(bars, bi);
    }
    for (uint32_t i = n > kFewSlots ? n - kFewSlots : 0; i < n; ++i)  // every load issued lands before the CTA exits
      mbar_drain(bar(bars->full[kv][i % kFewSlots]), (i / kFewSlots) & 1);
  } else if (warp == 3) {
    if (lane == 0) chunk_publish<1>(p, bars, ab);
    __syncwarp();
    if (blockIdx.x == 0)
      report_bad_batch(p.cu, p.seqlens, p.B, p.total, (long long)p.max_pages * p.page_size, lane, 32);
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    if (elect_one()) {
      constexpr uint32_t idS = idesc_e4m3_e5m2(128, kFewRows, false);            // K: rows of 128 bytes
      constexpr uint32_t idO = idesc_e4m3_e5m2(D, kFewTerms * kFewRows, true);   // V^T: columns are contiguous
      uint32_t n = 0, blocks = 0;
      auto issue_s = [&](uint32_t i, uint32_t qb, bool last) {
        const uint32_t slot = i % kFewSlots, buf = i % kFewBufs;
        mbar_wait(bar(bars->full[0][slot]), (i / kFewSlots) & 1, ab);
        mbar_wait(bar(bars->s_empty[buf]), ((i / kFewBufs) & 1) ^ 1, ab);
        tc_fence_after_sync();
        const uint32_t k_smem = sT(0, slot), q_smem = smem_base + Cfg::kOffQ + qb * Cfg::kQBytes;
#pragma unroll
        for (int term = 0; term < kFewTerms; ++term)
#pragma unroll
          for (int kk = 0; kk < D / 32; ++kk)
            mma_ss_f8(tmem + Cfg::kColS + buf * kFewRows, sdesc_kmajor(k_smem + kk * 32),
                      sdesc_kmajor(q_smem + term * (kFewRows * D) + kk * 32), idS, term > 0 || kk > 0);
        mma_commit(bar(bars->s_full[buf]));
        mma_commit(bar(bars->empty[0][slot]));
        if (last) mma_commit(bar(bars->q_empty[qb]));
      };
      const ChunkBlock* block;
      for (; (block = chunk_take(bars, blocks, ab)); ++blocks) {
        const ChunkBlock& w = *block;
        const int nv = w.v1 - w.v0;
        const uint32_t qb = blocks & 1;
        mbar_wait(bar(bars->q_full[qb]), (blocks >> 1) & 1, ab);
        tc_fence_after_sync();
        for (int v = 0; v < min(nv, kFewBufs); ++v) issue_s(n + v, qb, v + 1 == nv);
        for (int v = 0; v < nv; ++v, ++n) {
          const uint32_t slot = n % kFewSlots, buf = n % kFewBufs;
          mbar_wait(bar(bars->full[1][slot]), (n / kFewSlots) & 1, ab);
          mbar_wait(bar(bars->w_full[buf]), (n / kFewBufs) & 1, ab);
          tc_fence_after_sync();
          const uint32_t w_smem = smem_base + Cfg::kOffW + buf * Cfg::kWBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss_f8(tmem + Cfg::kColO, sdesc_mnmajor(sT(1, slot) + kk * 4096, 16384), sdesc_kmajor(w_smem + kk * 32),
                      idO, v > 0 || kk > 0);
          mma_commit(bar(bars->pv_done[buf]));
          mma_commit(bar(bars->empty[1][slot]));
          if (v + kFewBufs < nv) issue_s(n + kFewBufs, qb, v + kFewBufs + 1 == nv);
        }
        chunk_release(bars, blocks);
      }
      mma_commit(bar(bars->mma_done));
      mbar_drain(bar(bars->mma_done), 0);
    }
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- softmax + epilogue: a key, then a column of O
    const int key_in = tid - 128, wq = warp - 4;
    const uint32_t lane_field = (uint32_t)(wq * 32) << 16;
    const uint32_t scale_at = 128 * D + ((key_in >> box_shift) << 7) + (key_in & (p.box_rows - 1));
    float* sX = reinterpret_cast<float*>(smem_gen + Cfg::kOffX);  // [3][warp][row]
    int* sE = reinterpret_cast<int*>(smem_gen + Cfg::kOffX + 768);  // [warp]
    const uint32_t w_at = (uint32_t)key_in;  // byte of this key in a row of W, before the swizzle
    uint32_t n = 0, blocks = 0;
    auto pv_wait = [&](uint32_t i) {     // W V of tile i has been added
      mbar_wait(bar(bars->pv_done[i % kFewBufs]), (i / kFewBufs) & 1, ab);
      tc_fence_after_sync();
    };
    // One block of at most 2 kPairs rows.
    auto block_rows = [&](auto np, const ChunkBlock& w) {
      constexpr int kPairs = decltype(np)::value;
      const int nv = w.v1 - w.v0, rows = w.ntok * p.G, v0 = w.v0;
      const int pos0 = w.pos0, pos1 = pos0 + w.ntok - 1, keys = w.n;
      const int tile_ns = w.keys.ns, tile_lo = w.keys.lo;
      // keys [lo_all, hi_all] are seen by every row (bounds of the window fit 32 bits: fa_chunk_paged)
      const int hi_all = pos0 < 0 ? -1 : p.win_r >= 0 ? min(keys - 1, pos0 + p.win_r) : keys - 1;
      const int lo_all = p.win_l >= 0 ? pos1 - p.win_l : 0;
      const uint32_t qb = blocks & 1;
      float2 c2[kPairs], m2[kPairs], l2[kPairs], lr2[kPairs];
      mbar_wait(bar(bars->q_full[qb]), (blocks >> 1) & 1, ab);
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        c2[k] = *reinterpret_cast<const float2*>(&bars->q_factor[qb][2 * k]);
        m2[k] = l2[k] = lr2[k] = make_float2(0.0f, 0.0f);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(bars->q_empty[qb]));
      int E = kFewNoE;
      uint32_t unset = (1u << rows) - 1u;  // rows that have seen no key: their reference is not one yet

      // Two tiles at a time: this thread has key key_in of each. (One at a time took 1900 cycles a tile,
      // most of them the latencies of the chain from the scores to the weights.)
      for (int v = 0; v < nv; v += 2) {
        const bool two = v + 1 < nv;
        const uint32_t n1 = n + (two ? 1 : 0);  // the last of the tiles
        uint32_t slot[2], buf[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          slot[u] = (u ? n1 : n) % kFewSlots;
          buf[u] = (u ? n1 : n) % kFewBufs;
        }
        {
          // the waits of this step, a lane each: scores (the later tile's come last), K and V (for their
          // scales), and that the weights' buffers have been read (the same)
          const uint32_t i = lane == 1 || lane == 3 ? n : n1;
          const uint32_t k_bar = bar(bars->full[0][i % kFewSlots]), v_bar = bar(bars->full[1][i % kFewSlots]);
          uint32_t at = bar(bars->s_full[buf[1]]), parity = (n1 / kFewBufs) & 1;
          if (lane >= 1 && lane < 5) {
            at = lane < 3 ? k_bar : v_bar;
            parity = (i / kFewSlots) & 1;
          } else if (lane == 5 && n1 >= kFewBufs) {
            at = bar(bars->pv_done[buf[1]]);
            parity ^= 1;
          }
          mbar_wait(at, parity, ab);
          __syncwarp();
        }
        tc_fence_after_sync();
        constexpr int kHalves = kPairs > 4 ? 2 : 1;
        uint32_t r[2][kHalves][8], ks[2], vs[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf)
            tmem_ld8(tmem + lane_field + Cfg::kColS + buf[u] * kFewRows + hf * 8, r[u][hf]);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          ks[u] = smem_gen[sT(0, slot[u]) - smem_base + scale_at];
          vs[u] = smem_gen[sT(1, slot[u]) - smem_base + scale_at];
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int hf = 0; hf < kHalves; ++hf) tmem_wait_ld(r[u][hf]);
        tc_fence_before_sync();
        __syncwarp();
        if (lane < (two ? 2 : 1)) {
          mbar_arrive(bar(bars->s_empty[(n + lane) % kFewBufs]));
          mbar_arrive(bar(bars->empty[0][(n + lane) % kFewSlots]));
        }

        // scores against the references, -inf where masked; is the key seen at all?
        float2 a[2][kPairs];
        bool seen[2], over = unset != 0 || E == kFewNoE;
        int ev[2];  // less E, at least -96 (a key without values: -96)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float kf = ks[u] == (uint32_t)kScaleNan ? __int_as_float(0x7fc00000)
                                                        : __int_as_float((int)max(ks[u], 1u) << 23);
          const int tile = v0 + v + u, key0 = (tile < tile_ns ? tile : tile_lo + tile - tile_ns) * 128, key = key0 + key_in;
          const bool on = u == 0 || two, all = key0 + 127 <= hi_all && (key0 >= lo_all || key0 + 127 < p.sinks);
          seen[u] = on && all;
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const float2 x = make_float2(__uint_as_float(r[u][k / 4][2 * (k % 4)]),
                                         __uint_as_float(r[u][k / 4][2 * (k % 4) + 1]));
            a[u][k] = fma2(mul2(x, c2[k]), make_float2(kf, kf), make_float2(-m2[k].x, -m2[k].y));
          }
          if (!(on && all)) {
#pragma unroll
            for (int k = 0; k < kPairs; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int pos = pos0 + p.by_group(2 * k + e);
                const bool vis = on && pos >= 0 && key < keys && (p.win_r < 0 || key <= pos + p.win_r) &&
                                 (p.win_l < 0 || key >= pos - p.win_l || key < p.sinks) && 2 * k + e < rows;
                seen[u] |= vis;
                if (!vis) (e ? a[u][k].y : a[u][k].x) = -INFINITY;
              }
          }
          float most = -INFINITY;
#pragma unroll
          for (int k = 0; k < kPairs; ++k) most = max3(most, a[u][k].x, a[u][k].y);
          const bool has = seen[u] && vs[u] != (uint32_t)kScaleNan;
          ev[u] = has ? max((int)vs[u] - 127 - E, -kFewSpan) : -kFewSpan;
          over |= most + (float)ev[u] > kFewGrow;
        }
        if (few_vote(over)) {
          if (E == kFewNoE) {  // the first keys with values fix it
            const int em = __reduce_max_sync(0xffffffffu, max(ev[0], ev[1]));
            if (lane == 0) sE[wq] = em;
            named_bar_sync(2, 128);
            const int most_ev = max(max(sE[0], sE[1]), max(sE[2], sE[3])) + kFewNoE;
            if (most_ev > kFewNoE - kFewSpan) {
              E = min(max(most_ev, kFewLeastE), kFewMostE);
#pragma unroll
              for (int u = 0; u < 2; ++u)
                if (ev[u] > -kFewSpan) ev[u] = max(ev[u] + kFewNoE - E, -kFewSpan);
            }
          }
          // exact maxima over the tiles' keys of x + ev - E; the sums and O follow the new references (P of the
          // largest score stays above 2^-100: the log-sum-exp stands whatever the values are)
          const float ev_0 = (float)min(ev[0], kFewRise), ev_1 = (float)min(ev[1], kFewRise);
          const float2 ev0 = make_float2(ev_0, ev_0), ev1 = make_float2(ev_1, ev_1);
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            const float2 y0 = add2(a[0][k], ev0), y1 = add2(a[1][k], ev1);
            const float2 x = make_float2(warp_max_f32(fmaxf(y0.x, y1.x)), warp_max_f32(fmaxf(y0.y, y1.y)));
            if (lane == 0) *reinterpret_cast<float2*>(&sX[wq * kFewRows + 2 * k]) = x;
          }
          named_bar_sync(2, 128);
          float2 alpha[kPairs];
#pragma unroll
          for (int k = 0; k < kPairs; ++k) {
            float2 x = make_float2(-INFINITY, -INFINITY);
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const float2 y = *reinterpret_cast<const float2*>(&sX[q4 * kFewRows + 2 * k]);
              x = make_float2(fmaxf(x.x, y.x), fmaxf(x.y, y.y));
            }
            float2 up;  // rise of the references; a first one may lie anywhere
            auto rise = [&](float most_r, int row, float& up_r, float& alpha_r) {
              const bool first = (unset >> row) & 1;
              up_r = first ? (most_r == -INFINITY ? 0.0f : most_r) : fmaxf(most_r, 0.0f);
              alpha_r = first ? 1.0f : ex2_approx(-up_r);
              if (most_r != -INFINITY) unset &= ~(1u << row);
            };
            rise(x.x, 2 * k, up.x, alpha[k].x);
            rise(x.y, 2 * k + 1, up.y, alpha[k].y);
            m2[k] = add2(m2[k], up);
            a[0][k] = sub2(a[0][k], up);
            a[1][k] = sub2(a[1][k], up);
            float2 fall = alpha[k];
            if (fmaxf(up.x, up.y) > 120.0f) {  // the sums may fall from 2^96 to 2^-100: a factor beyond fp32, in halves
              fall = make_float2(fminf(ex2_approx(-0.5f * up.x), 1.0f), fminf(ex2_approx(-0.5f * up.y), 1.0f));
              l2[k] = mul2(l2[k], fall);
              lr2[k] = mul2(lr2[k], fall);
            }
            l2[k] = mul2(l2[k], fall);
            lr2[k] = mul2(lr2[k], fall);
          }
          if (v > 0) {
            pv_wait(n - 1);
#pragma unroll
            for (int term = 0; term < kFewTerms; ++term)
#pragma unroll
              for (int hf = 0; hf < kHalves; ++hf) {
                uint32_t o[8];
                const uint32_t at = tmem + lane_field + Cfg::kColO + term * kFewRows + hf * 8;
                tmem_ld8(at, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  if (hf * 4 + k >= kPairs) continue;
                  o[2 * k] = __float_as_uint(__uint_as_float(o[2 * k]) * alpha[hf * 4 + k].x);
                  o[2 * k + 1] = __float_as_uint(__uint_as_float(o[2 * k + 1]) * alpha[hf * 4 + k].y);
                }
                tmem_st8(at, o);
              }
            tmem_wait_st();
          }
          named_bar_sync(2, 128);  // sX and sE have been read
        }
        // weights: rounded, summed, and in three terms into their buffers
        float vf[2];
#pragma unroll
        for (int u = 0; u < 2; ++u)
          vf[u] = !seen[u]                        ? 0.0f
                  : vs[u] == (uint32_t)kScaleNan ? __int_as_float(0x7fc00000)
                                                 : exp2_int(min((int)vs[u] - 127 - E + kFewShift, 127));
#pragma unroll
        for (int k = 0; k < kPairs; ++k) {
          uint32_t t[2][kFewTerms];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float2 pe = make_float2(ex2_approx(a[u][k].x), ex2_approx(a[u][k].y));
            l2[k] = add2(l2[k], pe);
            const float2 pr = round_bits2<9>(pe);
            lr2[k] = add2(lr2[k], pr);
            split_e5m2(mul2(pr, make_float2(vf[u], vf[u])), t[u]);
          }
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            if (u == 1 && !two) continue;  // (the buffer is not this block's)
            const uint32_t w_smem = smem_base + Cfg::kOffW + buf[u] * Cfg::kWBytes;
#pragma unroll
            for (int term = 0; term < kFewTerms; ++term)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int row = term * kFewRows + 2 * k + e;
                st_shared_u8(w_smem + row * 128 + (w_at ^ ((row & 7) << 4)), e ? t[u][term] >> 8 : t[u][term]);
              }
          }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (!seen[u] && (u == 0 || two)) {  // the row of a key that no row sees may hold anything: 0
#pragma unroll
            for (int k = 0; k < D / 16; ++k) st_shared_v4(sT(1, slot[u]) + key_in * D + k * 16, 0u, 0u, 0u, 0u);
          }
        fence_proxy_async_smem();
        tc_fence_before_sync();
        __syncwarp();
        if (lane < (two ? 2 : 1)) mbar_arrive(bar(bars->w_full[(n + lane) % kFewBufs]));
        n = n1 + 1;
      }

      // ---- epilogue: this thread's column of every row
      const bool whole = w.slot < 0;
#pragma unroll
      for (int k = 0; k < kPairs; ++k) {
        float2 a = l2[k], b = lr2[k];
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          a = add2(a, make_float2(__shfl_xor_sync(0xffffffffu, a.x, off), __shfl_xor_sync(0xffffffffu, a.y, off)));
          b = add2(b, make_float2(__shfl_xor_sync(0xffffffffu, b.x, off), __shfl_xor_sync(0xffffffffu, b.y, off)));
        }
        if (lane == 0) {
          *reinterpret_cast<float2*>(&sX[wq * kFewRows + 2 * k]) = a;
          *reinterpret_cast<float2*>(&sX[(4 + wq) * kFewRows + 2 * k]) = b;
        }
      }
      named_bar_sync(2, 128);
      pv_wait(n - 1);
      const float e_unit = exp2_int(E - kFewShift);
      const long long o_size = (long long)p.total * p.Hq * D, part_rows = 2LL * p.ctas * 128;
#pragma unroll
      for (int hf = 0; hf < (kPairs > 4 ? 2 : 1); ++hf) {
        float o[8];
#pragma unroll
        for (int term = 0; term < kFewTerms; ++term) {
          uint32_t x[8];
          tmem_ld8(tmem + lane_field + Cfg::kColO + term * kFewRows + hf * 8, x);
          tmem_wait_ld(x);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = term == 0 ? __uint_as_float(x[i]) : o[i] + __uint_as_float(x[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          constexpr int kLast = 2 * kPairs;
          const int row = hf * 8 + i;
          if (row >= kLast || row >= rows) break;
          float l = 0.0f, lr = 0.0f;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            l += sX[u * kFewRows + row];
            lr += sX[(4 + u) * kFewRows + row];
          }
          const bool dead = !(lr > 0.0f) && lr == lr;  // no visible key (a NaN sum is not one)
          const float value = dead ? 0.0f : o[i] * e_unit / lr;
          const float m = (row & 1) ? m2[row < kLast ? row >> 1 : 0].y : m2[row < kLast ? row >> 1 : 0].x;
          const float lse2 = l > 0.0f ? m + lg2_approx(l) : (l == l ? -INFINITY : l);
          const int itok = p.by_group(row), head = w.h * p.G + row - itok * p.G;
          const long long tok = (long long)w.c0 + itok;
          if (whole) {
            const long long oi = (tok * p.Hq + head) * D + key_in, li = (long long)head * p.total + tok;
            if (dbg_range(ab, oi, 1, o_size)) p.o[oi] = __float2bfloat16_rn(value);
            if (key_in == 0 && dbg_range(ab, li, 1, (long long)p.Hq * p.total))
              p.lse[li] = lse2 == -INFINITY ? -INFINITY : lse2 * kLn2;
          } else {
            const long long pi = (long long)w.slot * 128;
            if (dbg_range(ab, pi + row, 1, part_rows)) {
              p.o_part[pi * D + ((key_in >> 2) * 128 + row) * 4 + (key_in & 3)] = value;
              if (key_in == 0) p.lse_part[pi + row] = lse2;
            }
          }
        }
      }
      tc_fence_before_sync();
      named_bar_sync(2, 128);  // the sums have been read
    };
    for (;; ++blocks) {
      const ChunkBlock* block = chunk_take(bars, blocks, ab);
      if (!all_agree(block != nullptr, 2, 128)) break;  // (the warps meet at this barrier: all go on, or none)
      const ChunkBlock& w = *block;
      const int rows = w.ntok * p.G;
      // (straight-line code for the number of row pairs: a branch per pair kept the chains of different
      // pairs and tiles from overlapping)
      if (rows <= 2)
        block_rows(std::integral_constant<int, 1>(), w);
      else if (rows <= 4)
        block_rows(std::integral_constant<int, 2>(), w);
      else if (rows <= 8)
        block_rows(std::integral_constant<int, 4>(), w);
      else
        block_rows(std::integral_constant<int, 8>(), w);
      if (lane == 0) chunk_release(bars, blocks);
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- queries: eight threads a row, 16 elements each
    const int ct = tid - 256, row = ct >> 3, c = ct & 7;
    uint32_t blocks = 0;
    const ChunkBlock* block;
    for (; (block = chunk_take(bars, blocks, ab)); ++blocks) {
      const ChunkBlock& w = *block;
      const uint32_t qb = blocks & 1;
      const int itok = p.by_group(row), head = w.h * p.G + row - itok * p.G;
      const long long qi = ((long long)w.c0 + itok) * q_stride + (long long)head * D + c * 16;
      uint4 x[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
      if (row < w.ntok * p.G) {
        x[0] = *reinterpret_cast<const uint4*>(q + qi);
        x[1] = *reinterpret_cast<const uint4*>(q + qi + 8);
      }
      const uint32_t in[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) most = __vmaxu2(most, in[i] & 0x7fff7fffu);
#pragma unroll
      for (int off = 4; off > 0; off >>= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, off));
      // the row's largest magnitude goes to [2^14, 2^15); an infinity or a NaN stays one (as NaN)
      const int top = (int)(max(most & 0xffffu, most >> 16) >> 7);
      const int up = min(14 + 127 - top, 126);
      const float f = top == 255 ? __int_as_float(0x7fc00000) : exp2_int(up);
      mbar_wait(bar(bars->q_empty[qb]), ((blocks >> 1) & 1) ^ 1, ab);
      uint32_t out[kFewTerms][4];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t t[kFewTerms];
        split_e5m2(mul2(make_float2(bf16lo_to_f32(in[i]), bf16hi_to_f32(in[i])), make_float2(f, f)), t);
#pragma unroll
        for (int term = 0; term < kFewTerms; ++term)
          out[term][i >> 1] = (i & 1) ? out[term][i >> 1] | t[term] << 16 : t[term];
      }
      const uint32_t to = smem_base + Cfg::kOffQ + qb * Cfg::kQBytes + row * D + ((c ^ (row & 7)) << 4);
#pragma unroll
      for (int term = 0; term < kFewTerms; ++term)
        st_shared_v4(to + term * (kFewRows * D), out[term][0], out[term][1], out[term][2], out[term][3]);
      if (c == 0) bars->q_factor[qb][row] = p.scale_log2 * exp2_int(-up);
      fence_proxy_async_smem();
      mbar_arrive(bar(bars->q_full[qb]));
      __syncwarp();
      if (lane == 0) chunk_release(bars, blocks);
    }
  }

  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace fa
