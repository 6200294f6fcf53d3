// Writing new key and value rows into a paged cache, and reading rows back, for sm_100a.
//
// A batch of ragged chunks: sequence b owns the packed rows [cu[b], cu[b + 1]) of k_new, v_new
// (total, H, d); they are the last new_b = cu[b + 1] - cu[b] of its seqlens[b] keys, so row i sits
// at position seqlens[b] - new_b + i, in row position % page_size of page
// block_table[b][position / page_size].
//
// bf16 pages take the rows as they are. E4M3 pages hold codes and, per (token, head), one scale
// byte s standing for 2^(s - 127): with a = max |x| over the row's d values,
//   e = the least integer >= -110 with a <= 448 * 2^e,   code = E4M3(x * 2^-e),   s = e + 127.
// Scaling by a power of two is exact, so a value is rounded once, to nearest even with 4
// significant bits, and reading it back, code * 2^e, is exact in bf16 (the least code times the
// least scale is 2^-119, a normal number). The one exception is the top binade: with e = 120 a
// value above 248 * 2^120 would round to 2^128, beyond bf16, so codes stop at 240 there (still
// within 2^-4 of the value). A power of two instead of a / 448 costs no precision
// (the codes float), only up to one binade at the small end of their range. A row with a NaN or an
// infinity has no such scale: it gets s = 255, and its values read back as NaN.
// The codes are laid out like bf16 pages, (num_pages, page_size, H, d); the scales as
// (num_pages, H, page_size), so that the scales of a head's consecutive keys are contiguous.
//
// Both kernels move each byte once, in 16-byte pieces, and are bound by HBM, or by the launch and
// the chain offsets -> length -> page -> row when there are few rows. One warp takes kCacheWarpElems
// values of one token, of K or of V; the loads of new rows do not wait for the token's place.
// Measured: reading 49573 tokens of 16 heads x 128 back 97 to 103 us (609 MB, 95 at the copy rate; K and
// V by one warp 112, 512 values a warp 118, no streaming hints 101); writing 16625 tokens of 8 heads
// 22.6 us (102 MB, 15.8 at the copy rate, and a launch; finding the places and the scattered scale
// bytes cost 2 us each); a step's 64 tokens 4.2 us, a launch and its chain.
#pragma once

#include "sm100_ptx.cuh"

namespace fa {

constexpr int kCacheThreads = 256;
constexpr int kCacheWarpElems = 1024;  // of one token's H * d values, per warp
constexpr int kScaleMin = 17;          // scale byte of 2^-110
constexpr int kScaleTop = 247;         // 2^120, the largest a finite row gets
constexpr int kScaleNan = 255;

struct CacheParams {
  int B, total, H, page_size, max_pages, num_pages;
  int parts;             // warps per token: ceil(H d / kCacheWarpElems)
  long long row_stride;  // elements between two tokens of the packed rows
  const int* block_table;
  const int* seqlens;
  const int* cu;
  void* rows[2];    // packed K, V rows (total, H, d) bf16
  void* cache[2];   // pages
  uint8_t* scale[2];  // (num_pages, H, page_size), E4M3 pages only
};

// Offsets and lengths of a ragged batch over a paged cache: reports (kErrBadInput) offsets that
// do not start at 0, decrease or pass `total`, and lengths outside [0, max_pages * page_size].
// Called by `threads` threads of one block, `tid` of them.
__device__ __forceinline__ void report_bad_batch(const int* cu, const int* seqlens, int B, int total,
                                                 long long max_keys, int tid, int threads) {
  bool bad = tid == 0 && (cu[0] != 0 || cu[B] > total);
  for (int i = tid; i < B; i += threads)
    bad |= cu[i + 1] < cu[i] || seqlens[i] < 0 || seqlens[i] > max_keys;
  if (bad) atomicOr(&g_fa_error, kErrBadInput);
}

// Where a packed token lives: 1 and its page and row, 0 for a row without a place (its position is
// negative or its length or page out of range), -1 for a row of no sequence.
__device__ __forceinline__ int cache_place(const CacheParams& p, int token, int& page, int& row) {
  const int b = seg_of(p.cu, p.B, token);
  const int c0 = p.cu[b], c1 = p.cu[b + 1], n = p.seqlens[b];
  if (token < c0 || token >= c1 || c0 < 0 || c1 > p.total) return -1;
  if (n < 0 || n > (long long)p.max_pages * p.page_size) return 0;  // (a length near -2^31 would wrap below)
  const int pos = n - (c1 - c0) + (token - c0);
  if (pos < 0) return 0;
  page = p.block_table[(size_t)b * p.max_pages + pos / p.page_size];
  row = pos % p.page_size;
  if (page < 0 || page >= p.num_pages) {
    atomicOr(&g_fa_error, kErrBadInput);
    return 0;
  }
  return 1;
}

// Scale byte of a row whose largest magnitude has the bf16 bits `most` (sign cleared): 448 is
// 1.75 * 2^8, so e is the exponent of `most` minus 8, plus one when its mantissa is above 1.75.
__device__ __forceinline__ int e4m3_scale_byte(uint32_t most) {
  if (most >= 0x7f80u) return kScaleNan;
  const int s = (int)(most >> 7) - 8 + ((most & 127u) > 96u ? 1 : 0);
  return s > kScaleMin ? s : kScaleMin;
}

__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}

// One warp: kCacheWarpElems values of one token, of K (blockIdx.y = 0) or V. kF8 picks E4M3 pages, D
// the lanes per row.
template <int D, bool kF8>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_write_kernel(const CacheParams p) {
  constexpr int kIters = kCacheWarpElems / 256;  // 32 lanes of 8 values
  constexpr int kLanes = D / 8;                  // lanes of one row
  const Abort none{nullptr};
  griddep_wait();  // launched as a programmatic dependent: what ran before on the stream is done
  if (blockIdx.x == 0 && blockIdx.y == 0)
    report_bad_batch(p.cu, p.seqlens, p.B, p.total, (long long)p.max_pages * p.page_size, threadIdx.x, kCacheThreads);
  const long long unit = (long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  const int lane = lane_id(), kv = blockIdx.y;
  const int token = (int)(unit / p.parts), part = (int)(unit - (long long)token * p.parts);
  if (token >= p.total) return;
  const int width = p.H * D, first = part * kCacheWarpElems + lane * 8;
  const __nv_bfloat16* rows =
      static_cast<const __nv_bfloat16*>(kv ? p.rows[1] : p.rows[0]) + (long long)token * p.row_stride;
  void* cache = kv ? p.cache[1] : p.cache[0];
  uint8_t* scale = kv ? p.scale[1] : p.scale[0];
  uint4 x[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int at = first + i * 256;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (at < width) x[i] = ld_global_cs(rows + at);
  }
  int page = 0, row = 0;
  if (cache_place(p, token, page, row) <= 0) return;
  const long long base = ((long long)page * p.page_size + row) * width;
  const long long size = (long long)p.num_pages * p.page_size * width;
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int at = first + i * 256;
    if constexpr (!kF8) {
      if (at < width && dbg_range(none, base + at, 8, size))
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(cache) + base + at) = x[i];
    } else {
      uint32_t most = __vmaxu2(max_abs_bf16x2(x[i].x, x[i].y), max_abs_bf16x2(x[i].z, x[i].w));
#pragma unroll
      for (int off = kLanes / 2; off > 0; off >>= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, off));
      const int s = e4m3_scale_byte(max(most & 0xffffu, most >> 16));
      // 2^-e = 2^(127 - s): its float exponent field is 254 - s; s = 255 makes every code NaN
      const float inv = s == kScaleNan ? __int_as_float(0x7fc00000) : __int_as_float((254 - s) << 23);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint2 codes;
      codes.x = pack_e4m3x4(bf16lo_to_f32(w[0]) * inv, bf16hi_to_f32(w[0]) * inv, bf16lo_to_f32(w[1]) * inv,
                            bf16hi_to_f32(w[1]) * inv);
      codes.y = pack_e4m3x4(bf16lo_to_f32(w[2]) * inv, bf16hi_to_f32(w[2]) * inv, bf16lo_to_f32(w[3]) * inv,
                            bf16hi_to_f32(w[3]) * inv);
      if (s == kScaleTop) {  // 256 (0x78) becomes 240 (0x77)
        codes.x = (codes.x & 0x80808080u) | __vminu4(codes.x & 0x7f7f7f7fu, 0x77777777u);
        codes.y = (codes.y & 0x80808080u) | __vminu4(codes.y & 0x7f7f7f7fu, 0x77777777u);
      }
      if (at < width && dbg_range(none, base + at, 8, size)) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(cache) + base + at) = codes;
        if ((lane & (kLanes - 1)) == 0) scale[((long long)page * p.H + at / D) * p.page_size + row] = (uint8_t)s;
      }
    }
  }
}

// Two E4M3 codes (16 bits) -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  float2 v;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tcvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

template <int D, bool kF8>
__global__ void __launch_bounds__(kCacheThreads) fa_cache_read_kernel(const CacheParams p) {
  constexpr int kVec = kF8 ? 16 : 8;                     // values of a 16-byte piece of a page
  constexpr int kIters = kCacheWarpElems / (32 * kVec);
  const Abort none{nullptr};
  griddep_wait();  // launched as a programmatic dependent: what ran before on the stream is done
  if (blockIdx.x == 0 && blockIdx.y == 0)
    report_bad_batch(p.cu, p.seqlens, p.B, p.total, (long long)p.max_pages * p.page_size, threadIdx.x, kCacheThreads);
  const long long unit = (long long)blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  const int lane = lane_id(), kv = blockIdx.y;
  const int token = (int)(unit / p.parts), part = (int)(unit - (long long)token * p.parts);
  if (token >= p.total) return;
  int page = 0, row = 0;
  const int placed = cache_place(p, token, page, row);
  if (placed < 0) return;
  const int width = p.H * D, first = part * kCacheWarpElems + lane * kVec;
  const long long base = ((long long)page * p.page_size + row) * width;
  const long long size = (long long)p.num_pages * p.page_size * width;
  const char* cache = static_cast<const char*>(kv ? p.cache[1] : p.cache[0]);
  const uint8_t* scale = kv ? p.scale[1] : p.scale[0];
  __nv_bfloat16* rows = static_cast<__nv_bfloat16*>(kv ? p.rows[1] : p.rows[0]) + (long long)token * p.row_stride;
  uint4 x[kIters];
  int s[kIters];
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int at = first + i * 32 * kVec;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    s[i] = kScaleMin;
    if (placed && at < width && dbg_range(none, base + at, kVec, size)) {
      x[i] = ld_global_cs(cache + (base + at) * (kF8 ? 1 : 2));
      if (kF8) s[i] = scale[((long long)page * p.H + at / D) * p.page_size + row];
    }
  }
#pragma unroll
  for (int i = 0; i < kIters; ++i) {
    const int at = first + i * 32 * kVec;
    if (at >= width) continue;
    if constexpr (!kF8) {
      __stcs(reinterpret_cast<uint4*>(rows + at), x[i]);
    } else {
      // 2^(s - 127); a scale byte below 1 would need a subnormal float: no row is written with one
      const float unit_f = s[i] == kScaleNan ? __int_as_float(0x7fc00000) : __int_as_float(max(s[i], 1) << 23);
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      uint32_t r[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = e4m3x2_to_f32(w[e] & 0xffffu), c = e4m3x2_to_f32(w[e] >> 16);
        r[2 * e] = pack_bf16x2(a.x * unit_f, a.y * unit_f);
        r[2 * e + 1] = pack_bf16x2(c.x * unit_f, c.y * unit_f);
      }
      __stcs(reinterpret_cast<uint4*>(rows + at), make_uint4(r[0], r[1], r[2], r[3]));
      __stcs(reinterpret_cast<uint4*>(rows + at + 8), make_uint4(r[4], r[5], r[6], r[7]));
    }
  }
}

}  // namespace fa
