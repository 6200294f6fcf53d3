// Host side of the fa_sm100 C ABI: argument validation, TMA tensor maps, per-device
// kernel attributes, launches on the caller's stream and device-side error reporting.
// The kernels live in fa_fwd.cuh / fa_bwd.cuh and are compiled into this one translation
// unit (they share the device error word).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <mutex>

#include "fa_sm100.h"
#include "fa_bwd.cuh"
#include "fa_bwd_dq.cuh"
#include "fa_cache.cuh"
#include "fa_chunk.cuh"
#include "fa_chunk_few.cuh"
#include "fa_decode.cuh"
#include "fa_fwd.cuh"

namespace {

constexpr int kMaxDevices = 64;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

std::mutex g_mu;
EncodeTiledFn g_encode = nullptr;
int g_sm_count[kMaxDevices] = {0};
bool g_attr_done[kMaxDevices] = {false};
bool g_chunk_done[kMaxDevices] = {false};
bool g_is_sm100[kMaxDevices] = {false};

EncodeTiledFn encode_fn() {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_encode) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
  }
  return g_encode;
}

bool log_enabled() {
  static int on = -1;
  if (on < 0) {
    const char* e = std::getenv("FA_LOG");
    on = (e && e[0] == '1') ? 1 : 0;
  }
  return on == 1;
}

// Per-device set-up: SM count, sm_100 check, dynamic shared memory opt-in of every kernel.
// Shared-memory attributes of every (ALiBi, packed) variant of the bf16 kernels of head dim D.
template <int D, bool kAlibi, bool kVarlen>
bool variant_attributes() {
  const auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  const int smem = fa::BwdCfg<D>::kSmemBytes, smem_dq = fa::BwdDqCfg<D>::kSmemBytes;
  const int smem_fwd = fa::FwdCfg<D>::kSmemBytes + (kVarlen ? fa::kFwdSortBytes : 0);
  return cudaFuncSetAttribute(fa::fa_fwd_kernel<D, false, kAlibi, kVarlen>, attr, smem_fwd) == cudaSuccess &&
         cudaFuncSetAttribute(fa::fa_bwd_kernel<D, true, kAlibi, kVarlen>, attr, smem) == cudaSuccess &&
         cudaFuncSetAttribute(fa::fa_bwd_kernel<D, false, kAlibi, kVarlen>, attr, smem) == cudaSuccess &&
         cudaFuncSetAttribute(fa::fa_bwd_dq_kernel<D, kAlibi, kVarlen>, attr, smem_dq) == cudaSuccess;
}

template <int D>
bool bwd_attributes() {
  return variant_attributes<D, false, false>() && variant_attributes<D, true, false>() &&
         variant_attributes<D, false, true>() && variant_attributes<D, true, true>();
}

// Dynamic shared memory size of the decode kernel, and the largest shared-memory carveout (one
// CTA takes nearly all of an SM's).
template <int D>
bool decode_attributes() {
  for (const void* k : {(const void*)fa::fa_decode_kernel<D, 4>, (const void*)fa::fa_decode_kernel<D, 8>})
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, fa::DecTcCfg<D>::kSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared) !=
            cudaSuccess)
      return false;
  return true;
}

template <int D, bool kF8, int kTiles>
bool chunk_attribute() {
  return cudaFuncSetAttribute(fa::fa_chunk_kernel<D, kF8, kTiles>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              fa::ChunkCfg<D, kF8, kTiles>::kSmemBytes) == cudaSuccess;
}

template <int D>
bool chunk_attributes() {
  return chunk_attribute<D, false, 1>() && chunk_attribute<D, false, 2>() && chunk_attribute<D, true, 1>() &&
         chunk_attribute<D, true, 2>();
}

int device_setup(int* dev_out, int* sm_count) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_attr_done[dev]) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return FA_ERR_CUDA;
    g_is_sm100[dev] = (major == 10 && minor == 0);
    g_sm_count[dev] = sms;
    if (g_is_sm100[dev]) {
      if (cudaFuncSetAttribute(fa::fa_fwd_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               fa::FwdCfg<128, true>::kSmemBytes) != cudaSuccess ||
          !decode_attributes<64>() || !decode_attributes<128>() ||
          !bwd_attributes<64>() || !bwd_attributes<128>())
        return FA_ERR_CUDA;
    }
    g_attr_done[dev] = true;
  }
  if (!g_is_sm100[dev]) return FA_ERR_UNSUPPORTED;
  *dev_out = dev;
  *sm_count = g_sm_count[dev];
  return FA_OK;
}

// The same for the chunk kernels, at the first call that needs them: setting an attribute loads its kernel,
// 0.5 ms for these nine. (A process's first forward takes 19.0 ms of set-up with them here, 19.5 with them
// above, and 14.4 in a library without the paged calls, whose module is a quarter smaller.)
int chunk_setup(int* dev, int* sm_count) {
  const int st = device_setup(dev, sm_count);
  if (st) return st;
  std::lock_guard<std::mutex> lk(g_mu);
  if (g_chunk_done[*dev]) return FA_OK;
  if (cudaFuncSetAttribute(fa::fa_chunk_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           fa::FewCfg::kSmemBytes) != cudaSuccess ||
      !chunk_attributes<64>() || !chunk_attributes<128>())
    return FA_ERR_CUDA;
  g_chunk_done[*dev] = true;
  return FA_OK;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct Shape {
  int B, N, H, d;
  size_t elems() const { return (size_t)B * N * H * d; }
  size_t tensor_bytes() const { return elems() * 2; }
  size_t rowvec_bytes() const { return (size_t)B * H * N * 4; }
  int n_pad() const { return (N + 127) / 128 * 128; }
};

// Sizes, head dim, windows and scale. Windows are normalised: causal forces win_r = 0,
// and a bound that reaches the whole sequence becomes -1 (unbounded).
int check_problem(int B, int N, int H, int d, float scale, int causal, int* win_l, int* win_r) {
  if (B < 1 || N < 1 || H < 1 || d < 1) return FA_ERR_INVALID_ARG;
  if (*win_l < -1 || *win_r < -1) return FA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  // TMA: strides < 2^40 bytes; item counts and coordinates stay in int.
  const double row_stride = (double)N * H * d * 2;
  if (row_stride >= 1099511627776.0) return FA_ERR_INVALID_ARG;
  if ((double)B * H * ((N + 127) / 128) >= 2147483647.0) return FA_ERR_INVALID_ARG;
  if (causal) *win_r = 0;
  if (*win_l >= N - 1) *win_l = -1;
  if (*win_r >= N - 1) *win_r = -1;
  return FA_OK;
}

// 4-D map over a (B, N, H, d) bf16 tensor: dims (d, N, H, B), box (64, 128, 1, 1), 128B swizzle.
int make_map(CUtensorMap* m, const void* base, const Shape& s) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.N, (cuuint64_t)s.H, (cuuint64_t)s.B};
  const cuuint64_t strides[3] = {(cuuint64_t)s.H * s.d * 2, (cuuint64_t)s.d * 2, (cuuint64_t)s.N * s.H * s.d * 2};
  const cuuint32_t box[4] = {64, 128, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_INVALID_ARG;
}

// 4-D map over a (B, N, H, d) tensor of E4M3 codes: dims (d, N, H, B), box (128, 128, 1, 1)
// (128 bytes x 128 rows), 128B swizzle.
int make_map_u8(CUtensorMap* m, const void* base, const Shape& s) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.N, (cuuint64_t)s.H, (cuuint64_t)s.B};
  const cuuint64_t strides[3] = {(cuuint64_t)s.H * s.d, (cuuint64_t)s.d, (cuuint64_t)s.N * s.H * s.d};
  const cuuint32_t box[4] = {128, 128, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_INVALID_ARG;
}

// 4-D map over a paged (num_pages, page_size, H, d) bf16 cache: dims (d, H, page_size, num_pages),
// box (64, 1, 64, 1) (128 bytes x 64 rows of one head and one page), 128B swizzle.
int make_map_cache(CUtensorMap* m, const void* base, int num_pages, int page_size, int H, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)page_size, (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2, (cuuint64_t)page_size * H * d * 2};
  const cuuint32_t box[4] = {64, 1, 64, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_INVALID_ARG;
}

// 4-D map over the (B, N, H, d) fp32 dQ accumulator for TMA reduce-add: box (32, 128, 1, 1)
// (128 bytes x 128 rows), 128B swizzle.
int make_map_f32_acc(CUtensorMap* m, const void* base, const Shape& s) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const cuuint64_t dims[4] = {(cuuint64_t)s.d, (cuuint64_t)s.N, (cuuint64_t)s.H, (cuuint64_t)s.B};
  const cuuint64_t strides[3] = {(cuuint64_t)s.H * s.d * 4, (cuuint64_t)s.d * 4, (cuuint64_t)s.N * s.H * s.d * 4};
  const cuuint32_t box[4] = {32, 128, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_INVALID_ARG;
}

struct Workspace {
  float* dq_acc;
  float* lse2;
  float* dvec;
  int* next_item;
};

size_t workspace_bytes(const Shape& s) {
  return align256(s.elems() * 4) + 2 * align256((size_t)s.B * s.H * s.n_pad() * 4) + 256;
}

// Layout: dQ accumulator | -LSE*log2(e) | -D | work counter, each 256-byte aligned.
Workspace carve(void* ws, const Shape& s) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  Workspace w;
  w.dq_acc = reinterpret_cast<float*>(p);
  p += align256(s.elems() * 4);
  w.lse2 = reinterpret_cast<float*>(p);
  p += align256((size_t)s.B * s.H * s.n_pad() * 4);
  w.dvec = reinterpret_cast<float*>(p);
  p += align256((size_t)s.B * s.H * s.n_pad() * 4);
  w.next_item = reinterpret_cast<int*>(p);
  return w;
}

int launch_status() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// ---------------------------------------------------------------- launches (arguments already checked)

// The forward's work counter: slots of fa::g_fwd_next_item are handed out in turn per device,
// so calls in flight at the same time (on different streams) count in different slots as long
// as fewer than kFwdCounterSlots of them overlap. Each launch zeroes its slot first.
std::atomic<unsigned> g_fwd_slot_seq[kMaxDevices];

// The counter-reset kernel, then the forward kernel as its programmatic dependent (it sets up
// while the reset runs and waits for it before taking its first item).
template <int D, bool kF8, bool kAlibi, bool kVarlen>
int fwd_launch(int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
               const CUtensorMap& mo, const fa::FwdParams& p) {
  fa::fa_fwd_counter_reset_kernel<<<1, 32, 0, stream>>>(p.counter_slot);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(fa::FwdCfg<D, kF8>::kThreads);
  cfg.dynamicSmemBytes = fa::FwdCfg<D, kF8>::kSmemBytes + (kVarlen ? fa::kFwdSortBytes : 0);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, fa::fa_fwd_kernel<D, kF8, kAlibi, kVarlen>, mq, mk, mv, mo, p) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <int D>
int fwd_variant(bool alibi, bool varlen, int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk,
                const CUtensorMap& mv, const CUtensorMap& mo, const fa::FwdParams& p) {
  if (alibi && varlen) return fwd_launch<D, false, true, true>(grid, stream, mq, mk, mv, mo, p);
  if (alibi) return fwd_launch<D, false, true, false>(grid, stream, mq, mk, mv, mo, p);
  if (varlen) return fwd_launch<D, false, false, true>(grid, stream, mq, mk, mv, mo, p);
  return fwd_launch<D, false, false, false>(grid, stream, mq, mk, mv, mo, p);
}

// Pair ranks of the forward's final phase (all heads, shortest last): enough for two items per
// CTA, so that the end of the run is made of short items; all of them when that is more.
int fwd_tail_ranks(const Shape& s, int num_pairs, int sm_count) {
  const int bh = s.B * s.H;
  const int k = (2 * sm_count + bh - 1) / bh;
  return k < num_pairs ? k : num_pairs;
}

// Heads per scheduling group of the forward: as many as keep the K/V of one group within
// 24 MiB (two groups in flight stay well inside L2), at least 1.
int fwd_head_group(const Shape& s, int elem_bytes) {
  const double kv_per_head = 2.0 * s.N * s.d * elem_bytes;
  const double g = (24.0 * 1024 * 1024) / kv_per_head;
  const int bh = s.B * s.H;
  return g < 1.0 ? 1 : (g >= bh ? bh : (int)g);
}

// Offsets of a packed batch: cu[0] = 0, non-decreasing, cu[nseg] = n; a violation is reported
// through fa_check (the kernels clamp every bound, so bad offsets cannot send work out of range).
__global__ void __launch_bounds__(256) fa_check_cu_kernel(const int* cu, int nseg, int n) {
  bool bad = false;
  if (threadIdx.x == 0) bad = cu[0] != 0 || cu[nseg] != n;
  for (int i = threadIdx.x; i < nseg; i += blockDim.x) bad |= cu[i + 1] < cu[i];
  if (__syncthreads_or(bad) && threadIdx.x == 0) atomicOr(&fa::g_fa_error, fa::kErrBadInput);
}

int launch_check_cu(const int* cu, int nseg, int n, cudaStream_t stream) {
  fa_check_cu_kernel<<<1, 256, 0, stream>>>(cu, nseg, n);
  return launch_status();
}

// alibi != nullptr: (B, H) ALiBi slopes (bf16 inputs).
int launch_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const Shape& s, float scale,
               int causal, int win_l, int win_r, int sm_count, cudaStream_t stream,
               int dev, const float* const* descales = nullptr, const float* alibi = nullptr, const int* cu = nullptr,
               int nseg = 0) {
  CUtensorMap mq, mk, mv, mo;
  int st;
  auto in_map = descales ? make_map_u8 : make_map;
  if ((st = in_map(&mq, q, s)) || (st = in_map(&mk, k, s)) || (st = in_map(&mv, v, s)) ||
      (st = make_map(&mo, o, s)))
    return st;
  fa::FwdParams p;
  p.cu_seqlens = cu;
  p.nseg = nseg;
  p.q_descale = descales ? descales[0] : nullptr;
  p.k_descale = descales ? descales[1] : nullptr;
  p.v_descale = descales ? descales[2] : nullptr;
  p.alibi_slopes = alibi;
  p.B = s.B;
  p.N = s.N;
  p.H = s.H;
  p.scale_log2 = scale * fa::kLog2e;
  p.win_l = win_l;
  p.win_r = win_r;
  p.causal = causal ? 1 : 0;
  p.num_pairs = (s.N + 255) / 256;
  p.num_items = s.B * s.H * p.num_pairs;
  p.lse = lse;
  if (cu) {  // packed batch: the cost-sorted pairs in one group (their order already ends short)
    p.head_group = s.B * s.H;
    p.tail_ranks = 0;
  } else {
    p.head_group = fwd_head_group(s, descales ? 1 : 2);
    p.tail_ranks = fwd_tail_ranks(s, p.num_pairs, sm_count);
  }
  p.counter_slot = (int)(g_fwd_slot_seq[dev].fetch_add(1, std::memory_order_relaxed) % fa::kFwdCounterSlots);
  // Test-only fault knob: the forward withholds one internal signal so that a bounded wait in
  // the kernel runs out (it must report FA_ERR_TIMEOUT through fa_check, not hang).
  const char* drop = std::getenv("FA_DEBUG_DROP_S_SIGNAL");
  p.debug_drop_s_signal = (drop && drop[0] == '1') ? 1 : 0;
  const int grid = p.num_items < sm_count ? p.num_items : sm_count;
  if (log_enabled())
    std::fprintf(stderr, "[fa] fwd B=%d N=%d H=%d d=%d causal=%d win=(%d,%d) items=%d grid=%d smem=%d\n", s.B, s.N,
                 s.H, s.d, p.causal, win_l, win_r, p.num_items, grid,
                 s.d == 64 ? fa::FwdCfg<64>::kSmemBytes : fa::FwdCfg<128>::kSmemBytes);
  if (descales)
    st = fwd_launch<128, true, false, false>(grid, stream, mq, mk, mv, mo, p);
  else if (s.d == 64)
    st = fwd_variant<64>(alibi != nullptr, cu != nullptr, grid, stream, mq, mk, mv, mo, p);
  else
    st = fwd_variant<128>(alibi != nullptr, cu != nullptr, grid, stream, mq, mk, mv, mo, p);
  return st ? st : launch_status();
}

int launch_pre(const void* o, const float* lse, const void* dO, const Shape& s, const Workspace& w,
               cudaStream_t stream) {
  const long long rows_per_cta = s.d == 64 ? fa::PreCfg<64>::kRows : fa::PreCfg<128>::kRows;
  const long long blocks = (long long)s.B * s.H * (s.n_pad() / rows_per_cta);
  if (s.d == 64)
    fa::fa_bwd_pre_kernel<64><<<(unsigned)blocks, 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dO), lse, w.lse2, w.dvec, w.dq_acc,
        w.next_item, s.B, s.N, s.H, s.n_pad());
  else
    fa::fa_bwd_pre_kernel<128><<<(unsigned)blocks, 256, 0, stream>>>(
        static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dO), lse, w.lse2, w.dvec, w.dq_acc,
        w.next_item, s.B, s.N, s.H, s.n_pad());
  return launch_status();
}

// Packed sequences travel with the backward's other options.
struct BwdOptions {
  const float* alibi = nullptr;
  const int* cu = nullptr;
  int nseg = 0;
};

fa::BwdParams bwd_params(const Shape& s, float scale, int causal, int win_l, int win_r, const Workspace& w,
                         const BwdOptions& opt, int sm_count_hint) {
  fa::BwdParams p;
  p.alibi_slopes = opt.alibi;
  p.cu_seqlens = opt.cu;
  p.nseg = opt.nseg;
  p.B = s.B;
  p.N = s.N;
  p.H = s.H;
  p.N_pad = s.n_pad();
  p.scale = scale;
  p.scale_log2 = scale * fa::kLog2e;
  p.win_l = win_l;
  p.win_r = win_r;
  p.causal = causal ? 1 : 0;
  p.num_kv_tiles = (s.N + 127) / 128;
  p.num_items = s.B * s.H * p.num_kv_tiles;
  // Head groups of the main kernel: the Q, dO (bf16) and dQ accumulator (fp32) rows of a group,
  // 8 N d bytes per head, within 32 MiB; the last KV tiles (the shortest under causal masking,
  // enough for four items per CTA) dealt over all heads at the end.
  const double per_head = 8.0 * s.N * s.d;
  const double g = (32.0 * 1024 * 1024) / per_head;
  const int bh = s.B * s.H;
  p.head_group = g < 1.0 ? 1 : (g >= bh ? bh : (int)g);
  const int sms = sm_count_hint > 0 ? sm_count_hint : 148;
  const int k = (4 * sms + bh - 1) / bh;
  p.tail_tiles = k < p.num_kv_tiles ? k : p.num_kv_tiles;
  p.dq_acc = w.dq_acc;
  p.lse2 = w.lse2;
  p.dvec = w.dvec;
  p.next_item = w.next_item;
  return p;
}

template <int D, bool kDQ, bool kAlibi, bool kVarlen>
void main_launch(int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                 const CUtensorMap& mdo, const CUtensorMap& mdk, const CUtensorMap& mdv, const CUtensorMap& mdq,
                 const fa::BwdParams& p) {
  fa::fa_bwd_kernel<D, kDQ, kAlibi, kVarlen><<<grid, fa::BwdCfg<D>::kThreads, fa::BwdCfg<D>::kSmemBytes, stream>>>(
      mq, mk, mv, mdo, mdk, mdv, mdq, p);
}

template <int D, bool kDQ>
void main_kernel(bool alibi, bool varlen, int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk,
                 const CUtensorMap& mv, const CUtensorMap& mdo, const CUtensorMap& mdk, const CUtensorMap& mdv,
                 const CUtensorMap& mdq, const fa::BwdParams& p) {
  if (alibi && varlen) main_launch<D, kDQ, true, true>(grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else if (alibi) main_launch<D, kDQ, true, false>(grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else if (varlen) main_launch<D, kDQ, false, true>(grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else main_launch<D, kDQ, false, false>(grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
}

template <int D, bool kAlibi, bool kVarlen>
void dq_launch(int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
               const CUtensorMap& mdo, const CUtensorMap& mdq, const fa::BwdParams& p) {
  fa::fa_bwd_dq_kernel<D, kAlibi, kVarlen><<<grid, fa::BwdDqCfg<D>::kThreads, fa::BwdDqCfg<D>::kSmemBytes, stream>>>(
      mq, mk, mv, mdo, mdq, p);
}

template <int D>
void dq_kernel(bool alibi, bool varlen, int grid, cudaStream_t stream, const CUtensorMap& mq, const CUtensorMap& mk,
               const CUtensorMap& mv, const CUtensorMap& mdo, const CUtensorMap& mdq, const fa::BwdParams& p) {
  if (alibi && varlen) dq_launch<D, true, true>(grid, stream, mq, mk, mv, mdo, mdq, p);
  else if (alibi) dq_launch<D, true, false>(grid, stream, mq, mk, mv, mdo, mdq, p);
  else if (varlen) dq_launch<D, false, true>(grid, stream, mq, mk, mv, mdo, mdq, p);
  else dq_launch<D, false, false>(grid, stream, mq, mk, mv, mdo, mdq, p);
}

// Main backward kernel; with_dq = false computes dK and dV only (the deterministic backward).
int launch_main(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, const Shape& s,
                float scale, int causal, int win_l, int win_r, const Workspace& w, int sm_count,
                cudaStream_t stream, bool with_dq = true, const BwdOptions& opt = BwdOptions()) {
  CUtensorMap mq, mk, mv, mdo, mdk, mdv, mdq;
  int st;
  if ((st = make_map(&mq, q, s)) || (st = make_map(&mk, k, s)) || (st = make_map(&mv, v, s)) ||
      (st = make_map(&mdo, dO, s)) || (st = make_map(&mdk, dk, s)) || (st = make_map(&mdv, dv, s)) ||
      (st = make_map_f32_acc(&mdq, w.dq_acc, s)))
    return st;
  const fa::BwdParams p = bwd_params(s, scale, causal, win_l, win_r, w, opt, sm_count);
  const int grid = p.num_items < sm_count ? p.num_items : sm_count;
  if (log_enabled())
    std::fprintf(stderr, "[fa] bwd B=%d N=%d H=%d d=%d causal=%d win=(%d,%d) items=%d grid=%d smem=%d\n", s.B, s.N,
                 s.H, s.d, p.causal, win_l, win_r, p.num_items, grid,
                 s.d == 64 ? fa::BwdCfg<64>::kSmemBytes : fa::BwdCfg<128>::kSmemBytes);
  const bool a = opt.alibi != nullptr, vl = opt.cu != nullptr;
  if (s.d == 64 && with_dq)
    main_kernel<64, true>(a, vl, grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else if (s.d == 64)
    main_kernel<64, false>(a, vl, grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else if (with_dq)
    main_kernel<128, true>(a, vl, grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  else
    main_kernel<128, false>(a, vl, grid, stream, mq, mk, mv, mdo, mdk, mdv, mdq, p);
  return launch_status();
}

// dQ of the deterministic backward: one item per (b, h, Q tile), dQ accumulated in TMEM.
int launch_dq(const void* q, const void* k, const void* v, const void* dO, void* dq, const Shape& s, float scale,
              int causal, int win_l, int win_r, const Workspace& w, int sm_count, cudaStream_t stream,
              const BwdOptions& opt = BwdOptions()) {
  CUtensorMap mq, mk, mv, mdo, mdq;
  int st;
  if ((st = make_map(&mq, q, s)) || (st = make_map(&mk, k, s)) || (st = make_map(&mv, v, s)) ||
      (st = make_map(&mdo, dO, s)) || (st = make_map(&mdq, dq, s)))
    return st;
  const fa::BwdParams p = bwd_params(s, scale, causal, win_l, win_r, w, opt, sm_count);
  const int grid = p.num_items < sm_count ? p.num_items : sm_count;
  if (s.d == 64)
    dq_kernel<64>(opt.alibi != nullptr, opt.cu != nullptr, grid, stream, mq, mk, mv, mdo, mdq, p);
  else
    dq_kernel<128>(opt.alibi != nullptr, opt.cu != nullptr, grid, stream, mq, mk, mv, mdo, mdq, p);
  return launch_status();
}

int launch_convert(void* dq, const Shape& s, const Workspace& w, cudaStream_t stream) {
  const long long n8 = (long long)(s.elems() / 8);
  const long long blocks = (n8 + 255) / 256;
  fa::fa_dq_convert_kernel<<<(unsigned)blocks, 256, 0, stream>>>(w.dq_acc, static_cast<__nv_bfloat16*>(dq), n8);
  return launch_status();
}

// Common checks of the backward calls: problem, pointers, workspace.
int check_workspace(void* workspace, size_t bytes, const Shape& s) {
  if (!workspace || !aligned(workspace, 256) || bytes < workspace_bytes(s)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}


// ---------------------------------------------------------------- paged caches: ragged chunks

// Host checks shared by the calls on a ragged batch over a paged cache.
int check_paged(int B, int total, int H, int d, int num_pages, int page_size, int max_pages, const void* k_cache,
                const void* v_cache, const void* k_scale, const void* v_scale, const int* block_table,
                const int* seqlens, const int* cu) {
  if (B < 1 || total < 0 || H < 1 || num_pages < 1 || page_size < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  // TMA strides and coordinates; positions, packed rows and head counts stay in int with room to spare
  if ((double)num_pages * page_size * H * d * 2 >= 1099511627776.0 || (double)num_pages * H >= 2147483647.0 ||
      (double)max_pages * page_size > 1073741824.0 || total > 1073741824 || (double)H * d > 1073741824.0)
    return FA_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !block_table || !seqlens || !cu) return FA_ERR_INVALID_ARG;
  if ((k_scale == nullptr) != (v_scale == nullptr)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 16) || !aligned(v_scale, 16) ||
      !aligned(block_table, 4) || !aligned(seqlens, 4) || !aligned(cu, 4))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

struct Span {
  const void* p;
  size_t n;
};

bool any_overlap(const Span& a, const Span* others, int count) {
  for (int i = 0; i < count; ++i)
    if (a.p && others[i].p && overlap(a.p, a.n, others[i].p, others[i].n)) return true;
  return false;
}

// Bytes from the first to the last of `total` packed rows of `width` elements, `stride` apart.
size_t rows_bytes(int total, size_t width, long long stride) {
  return total < 1 ? 0 : ((size_t)(total - 1) * (size_t)stride + width) * 2;
}

// Do two sets of `total` such rows, of equal stride, meet? When their spans do, exactly if one's first row
// starts less than a row behind, or before, the start of some row of the other.
bool rows_overlap(const void* a, const void* b, int total, size_t width, long long stride) {
  const size_t n = rows_bytes(total, width, stride);
  if (n == 0 || !overlap(a, n, b, n)) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t low = (size_t)(x < y ? y - x : x - y) % ((size_t)stride * 2);
  return low < 2 * width || low > 2 * ((size_t)stride - width);
}

// A launch that may begin while the kernel before it on the stream ends (its kernels wait for that one
// before they touch global memory, in every thread, so that the end of one implies the end of those
// before it; so does the decode kernel, or its prep kernel). It saves 2 us a call: a step over bf16 pages 76.9 -> 74.6 us, a read of 609 MB 98.8 -> 96.5.
template <class... Params, class... Args>
int launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, args...) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return FA_OK;
}

template <bool kWrite>
int launch_cache(const fa::CacheParams& p, int d, cudaStream_t stream) {
  const long long units = (long long)p.total * p.parts, per_block = fa::kCacheThreads / 32;
  const long long blocks = (units + per_block - 1) / per_block;
  if (blocks >= 2147483647LL) return FA_ERR_INVALID_ARG;
  const bool f8 = p.scale[0] != nullptr;
  void (*kernel)(fa::CacheParams);
  if (kWrite)
    kernel = d == 64 ? (f8 ? fa::fa_cache_write_kernel<64, true> : fa::fa_cache_write_kernel<64, false>)
                     : (f8 ? fa::fa_cache_write_kernel<128, true> : fa::fa_cache_write_kernel<128, false>);
  else
    kernel = d == 64 ? (f8 ? fa::fa_cache_read_kernel<64, true> : fa::fa_cache_read_kernel<64, false>)
                     : (f8 ? fa::fa_cache_read_kernel<128, true> : fa::fa_cache_read_kernel<128, false>);
  return launch_dependent(kernel, dim3((unsigned)blocks, 2), fa::kCacheThreads, 0, stream, p);
}

// Writing (kWrite) or reading the rows [cu[b], cu[b + 1]) of every sequence.
template <bool kWrite>
int cache_rows(void* k_rows, void* v_rows, long long row_stride, void* k_cache, void* v_cache, void* k_scale,
               void* v_scale, const int* block_table, const int* seqlens, const int* cu, int B, int total, int H,
               int d, int num_pages, int page_size, int max_pages, fa_stream_t stream) {
  int st = check_paged(B, total, H, d, num_pages, page_size, max_pages, k_cache, v_cache, k_scale, v_scale,
                       block_table, seqlens, cu);
  if (st) return st;
  if (total > 0 && (!k_rows || !v_rows)) return FA_ERR_INVALID_ARG;
  if (!aligned(k_rows, 16) || !aligned(v_rows, 16) || row_stride < (long long)H * d || row_stride % 8 != 0 ||
      row_stride > 1073741824LL)
    return FA_ERR_INVALID_ARG;
  const bool f8 = k_scale != nullptr;
  const size_t rb = rows_bytes(total, (size_t)H * d, row_stride);
  const size_t cells = (size_t)num_pages * page_size * H, cb = cells * d * (f8 ? 1 : 2);
  const Span caches[4] = {{k_cache, cb}, {v_cache, cb}, {k_scale, cells}, {v_scale, cells}};
  const Span rows[2] = {{k_rows, rb}, {v_rows, rb}};
  const Span plan[3] = {{block_table, (size_t)B * max_pages * 4}, {seqlens, (size_t)B * 4}, {cu, (size_t)(B + 1) * 4}};
  for (int i = 0; i < 4; ++i) {
    if (any_overlap(caches[i], rows, 2)) return FA_ERR_INVALID_ARG;
    if (kWrite && (any_overlap(caches[i], caches + i + 1, 3 - i) || any_overlap(caches[i], plan, 3)))
      return FA_ERR_INVALID_ARG;
  }
  if (!kWrite && (any_overlap(rows[0], plan, 3) || any_overlap(rows[1], plan, 3))) return FA_ERR_INVALID_ARG;
  // (K and V rows may be slices of one tensor, whose spans interleave. Read back, no row may meet another.)
  if (!kWrite && rows_overlap(k_rows, v_rows, total, (size_t)H * d, row_stride)) return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  if (total == 0) return FA_OK;
  fa::CacheParams p;
  p.B = B;
  p.total = total;
  p.H = H;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.parts = (int)(((long long)H * d + fa::kCacheWarpElems - 1) / fa::kCacheWarpElems);
  p.row_stride = row_stride;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.cu = cu;
  p.rows[0] = k_rows;
  p.rows[1] = v_rows;
  p.cache[0] = k_cache;
  p.cache[1] = v_cache;
  p.scale[0] = static_cast<uint8_t*>(k_scale);
  p.scale[1] = static_cast<uint8_t*>(v_scale);
  return launch_cache<kWrite>(p, d, reinterpret_cast<cudaStream_t>(stream));
}

int encode_map(CUtensorMap* m, CUtensorMapDataType type, int rank, const void* base, const cuuint64_t* dims,
               const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return FA_ERR_CUDA;
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = enc(m, type, (cuuint32_t)rank, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FA_OK : FA_ERR_INVALID_ARG;
}

// Queries (total, Hkv, G, d), rows q_stride elements apart: a box is 64 columns of tq tokens' G heads.
int make_map_chunk_q(CUtensorMap* m, const void* q, int total, int Hkv, int G, int d, long long q_stride, int tq) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)G, (cuuint64_t)Hkv, (cuuint64_t)total};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)G * d * 2, (cuuint64_t)q_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)tq};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Pages (num_pages, page_size, H, d): box_rows rows of one head, 64 bf16 columns (swizzled) or all
// d codes of E4M3 pages (as they lie, or swizzled for the tensor core).
int make_map_pages(CUtensorMap* m, const void* base, int num_pages, int page_size, int H, int d, int box_rows,
                   bool f8, bool swizzle) {
  const cuuint64_t e = f8 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)page_size, (cuuint64_t)num_pages};
  const cuuint64_t strides[3] = {d * e, (cuuint64_t)H * d * e, (cuuint64_t)page_size * H * d * e};
  const cuuint32_t box[4] = {f8 ? (cuuint32_t)d : 64u, 1, (cuuint32_t)box_rows, 1};
  return encode_map(m, f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, base, dims, strides,
                    box, f8 && !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Scales (num_pages * H, page_size): box_rows consecutive keys of one head.
int make_map_scales(CUtensorMap* m, const void* base, int num_pages, int page_size, int H, int box_rows) {
  const cuuint64_t dims[2] = {(cuuint64_t)page_size, (cuuint64_t)num_pages * H};
  const cuuint64_t strides[1] = {(cuuint64_t)page_size};
  const cuuint32_t box[2] = {(cuuint32_t)box_rows, 1};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, base, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// One or two 128-row tiles per block of the chunk kernel: two share every K/V load, which long chunks
// need; with few rows to a sequence the second would stand idle. Measured with one / two (us in a graph, 8
// sequences of 4000 keys, 32 query heads over 8), by rows of a sequence:
//                    4           32          64          96          128         256
//   bf16, d = 128   33.6/35.7   36.6/37.3   38.6/38.7   41.3/39.9   44.0/40.5   66.1/51.5
//   E4M3, d = 128               42.0/42.2   43.6/43.5   45.8/44.8   48.9/46.3   80.3/62.7
//   bf16, d = 64    28.4/31.1   31.1/32.9   32.7/33.3   33.6/33.8   35.5/34.3   58.2/45.0
//   E4M3, d = 64    33.5/34.6   35.9/36.5   36.6/37.0   37.5/37.3   39.3/37.9   64.8/46.9
// The rows are the batch's average (the lengths are on the device): among 255 steps, a chunk of 1000 tokens
// takes 820 / 1121 with all contexts 4K (bf16, d = 128), 1037 / 761 with 32K under the chunk and 1K else.
int chunk_tiles(int B, int total, int G) { return (double)total * G <= 64.0 * B ? 1 : 2; }

// Heads whose CTAs run next to each other: the most of 4, 2 and 1 that divides the heads and the SMs.
// Measured with 1 / 2 / 4 heads (us): a step of 8 sequences of 4096 to 8192 keys, 16 heads, bf16 pages
// 76.9 / 77.0 / 75.3; 16 rows over 131072 keys, 8 heads 100 / 98.4 / 97.0; a step of 48 sequences, 8
// heads, E4M3 pages (128-byte rows) 223 / 207 / 207.
int chunk_head_group(int Hkv, int sms) {
  for (int hg = 4; hg > 1; hg /= 2)
    if (Hkv % hg == 0 && sms % hg == 0) return hg;
  return 1;
}

// Rows of a few tokens over E4M3 pages take the transposed kernel: when a sequence's rows fit its
// 16-row blocks on average (the lengths are on the device; padded rows count). Measured with it / with
// fa_chunk_kernel (us in a graph): a step of 48 sequences of 2000 to 15630 keys, 4 query heads to each of 8,
// 1 token 148 / 367, 3 tokens 216 / 368, 4 tokens 225 / 368; 16 heads to each of 4 136 / 191; 16 sequences,
// a head each of 16, 74 / 181. A longer chunk in such a batch is cut into several blocks, which read its
// keys again: a chunk of 20 tokens among 63 steps, all over 4K keys, 171 / 233, one of 512 among 199 over 8K
// 1171 / 1469, but one of 512 over 32K among 199 steps over 1K 1569 / 681 (in two calls: 333 and 90), one
// of 16 over 64K among 15 over 300, 8 heads to each of 8, 313 / 92 (in two: 77 and 21).
bool chunk_few(bool f8, int d, int B, int total, int G) {
  return f8 && d == fa::kFewD && G <= fa::kFewRows && (double)total <= (double)B * (fa::kFewRows / G);
}

// (fa::FastDiv says what the numbers are)
fa::FastDiv fast_div(unsigned d) {
  unsigned s = 0;
  while ((1ull << s) < d) ++s;
  return {(unsigned)((((1ull << 32) << s) + d - 1) / d - (1ull << 32)), s};
}

struct ChunkWorkspace {
  size_t o_bytes, lse_bytes, split_bytes;
  size_t bytes() const { return o_bytes + lse_bytes + split_bytes; }
};
ChunkWorkspace chunk_workspace(int pieces, int tiles, int d) {
  const size_t rows = (size_t)2 * pieces * tiles * 128;  // two partial slots per piece
  return {align256(rows * d * 4), align256(rows * 4), align256((size_t)pieces * 16)};
}

template <int D, bool kF8, int kTiles>
int chunk_launch(int grid, const CUtensorMap* m, const fa::ChunkParams& p, cudaStream_t stream) {
  using Cfg = fa::ChunkCfg<D, kF8, kTiles>;
  return launch_dependent(fa::fa_chunk_kernel<D, kF8, kTiles>, dim3(grid), Cfg::kThreads, Cfg::kSmemBytes, stream, m[0],
                          m[1], m[2], m[3], m[4], p);
}

// The join of blocks that are spread over several pieces, as the main kernel's programmatic dependent.
template <int D, int kTiles>
int chunk_merge_launch(int ctas, const fa::ChunkParams& p, cudaStream_t stream) {
  const long long rows = std::min<long long>((long long)p.total * p.G, kTiles * 128);
  return launch_dependent(fa::fa_chunk_merge_kernel<D, kTiles>,
                          dim3(ctas, (unsigned)((rows + fa::kMergeRows - 1) / fa::kMergeRows)), fa::kMergeThreads, 0,
                          stream, p);
}

template <int D>
int chunk_variant(bool f8, int tiles, int grid, const CUtensorMap* m, const fa::ChunkParams& p, cudaStream_t stream) {
  if (f8) return tiles == 1 ? chunk_launch<D, true, 1>(grid, m, p, stream) : chunk_launch<D, true, 2>(grid, m, p, stream);
  return tiles == 1 ? chunk_launch<D, false, 1>(grid, m, p, stream) : chunk_launch<D, false, 2>(grid, m, p, stream);
}

}  // namespace

// ---------------------------------------------------------------- backward without allocation
//
// Scratch for fa_bwd_static_workspace: a fixed array in the library's device image. Host code
// sees only a stand-in symbol; the device address is looked up once per device (with that
// device current) and cached. No cudaMalloc, cudaFree or allocating library call is made.
namespace {
constexpr size_t kStaticWorkspaceBytes = size_t(32) << 20;
static __device__ __align__(256) unsigned char g_static_workspace[kStaticWorkspaceBytes];
void* g_static_workspace_ptr[kMaxDevices] = {nullptr};

int static_workspace_address(int dev, void** out) {
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_static_workspace_ptr[dev]) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_workspace) != cudaSuccess || p == nullptr) {
      cudaGetLastError();
      return FA_ERR_CUDA;
    }
    g_static_workspace_ptr[dev] = p;
  }
  *out = g_static_workspace_ptr[dev];
  return FA_OK;
}
}  // namespace

extern "C" {

const char* fa_status_string(int status) {
  switch (status) {
    case FA_OK: return "FA_OK";
    case FA_ERR_INVALID_ARG: return "FA_ERR_INVALID_ARG: invalid argument";
    case FA_ERR_UNSUPPORTED: return "FA_ERR_UNSUPPORTED: head dim or device not supported";
    case FA_ERR_CUDA: return "FA_ERR_CUDA: CUDA runtime error";
    case FA_ERR_TIMEOUT: return "FA_ERR_TIMEOUT: a device-side wait timed out";
    case FA_ERR_NO_MEMORY: return "FA_ERR_NO_MEMORY: workspace allocation failed";
    case FA_ERR_DEVICE: return "FA_ERR_DEVICE: a device-side check failed";
    default: return "FA_ERR_UNKNOWN";
  }
}

size_t fa_bwd_workspace_bytes(int B, int N, int H, int d) {
  int wl = -1, wr = -1;
  if (check_problem(B, N, H, d, 1.0f, 0, &wl, &wr) != FA_OK) return 0;
  return workspace_bytes(Shape{B, N, H, d});
}

int fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int N, int H, int d, float scale,
           int causal, int win_l, int win_r, fa_stream_t stream) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4))
    return FA_ERR_INVALID_ARG;
  const Shape s{B, N, H, d};
  const size_t tb = s.tensor_bytes(), lb = s.rowvec_bytes();
  if (overlap(o, tb, q, tb) || overlap(o, tb, k, tb) || overlap(o, tb, v, tb) || overlap(lse, lb, q, tb) ||
      overlap(lse, lb, k, tb) || overlap(lse, lb, v, tb) || overlap(lse, lb, o, tb))
    return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  return launch_fwd(q, k, v, o, lse, s, scale, causal, win_l, win_r, sms, reinterpret_cast<cudaStream_t>(stream),
                    dev);
}

int fa_fwd_ex(const void* q, const void* k, const void* v, const float* alibi_slopes, void* o, float* lse, int B,
              int N, int H, int d, float scale, int causal, int win_l, int win_r, fa_stream_t stream) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(alibi_slopes, 4))
    return FA_ERR_INVALID_ARG;
  const Shape s{B, N, H, d};
  const size_t tb = s.tensor_bytes(), lb = s.rowvec_bytes(), ab = (size_t)B * H * 4;
  if (overlap(o, tb, q, tb) || overlap(o, tb, k, tb) || overlap(o, tb, v, tb) || overlap(lse, lb, q, tb) ||
      overlap(lse, lb, k, tb) || overlap(lse, lb, v, tb) || overlap(lse, lb, o, tb))
    return FA_ERR_INVALID_ARG;
  if (alibi_slopes && (overlap(o, tb, alibi_slopes, ab) || overlap(lse, lb, alibi_slopes, ab)))
    return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  return launch_fwd(q, k, v, o, lse, s, scale, causal, win_l, win_r, sms, reinterpret_cast<cudaStream_t>(stream),
                    dev, nullptr, alibi_slopes);
}

int fa_fwd_varlen(const void* q, const void* k, const void* v, const int* cu_seqlens, const float* alibi_slopes,
                  void* o, float* lse, int B, int total, int H, int d, float scale, int causal, int win_l,
                  int win_r, fa_stream_t stream) {
  if (B < 1 || !cu_seqlens || !aligned(cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  int st = check_problem(1, total, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(alibi_slopes, 4))
    return FA_ERR_INVALID_ARG;
  const Shape s{1, total, H, d};
  const size_t tb = s.tensor_bytes(), lb = s.rowvec_bytes(), ab = (size_t)H * 4, cb = (size_t)(B + 1) * 4;
  const void* ins[5] = {q, k, v, cu_seqlens, alibi_slopes};
  const size_t in_bytes[5] = {tb, tb, tb, cb, alibi_slopes ? ab : 0};
  for (int i = 0; i < 5; ++i)
    if (overlap(o, tb, ins[i], in_bytes[i]) || overlap(lse, lb, ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
  if (overlap(o, tb, lse, lb)) return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if ((st = launch_check_cu(cu_seqlens, B, total, cs))) return st;
  return launch_fwd(q, k, v, o, lse, s, scale, causal, win_l, win_r, sms, cs, dev, nullptr, alibi_slopes, cu_seqlens,
                    B);
}

int fa_fwd_fp8(const void* q, const void* k, const void* v, const float* q_descale, const float* k_descale,
               const float* v_descale, void* o, float* lse, int B, int N, int H, int d, float scale, int causal,
               int win_l, int win_r, fa_stream_t stream) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !q_descale || !k_descale || !v_descale || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(q_descale, 4) || !aligned(k_descale, 4) || !aligned(v_descale, 4))
    return FA_ERR_INVALID_ARG;
  const Shape s{B, N, H, d};
  const size_t ib = s.elems(), ob = s.tensor_bytes(), lb = s.rowvec_bytes(), db = (size_t)B * H * 4;
  const void* ins[6] = {q, k, v, q_descale, k_descale, v_descale};
  const size_t in_bytes[6] = {ib, ib, ib, db, db, db};
  for (int i = 0; i < 6; ++i)
    if (overlap(o, ob, ins[i], in_bytes[i]) || overlap(lse, lb, ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
  if (overlap(o, ob, lse, lb)) return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  const float* descales[3] = {q_descale, k_descale, v_descale};
  return launch_fwd(q, k, v, o, lse, s, scale, causal, win_l, win_r, sms, reinterpret_cast<cudaStream_t>(stream),
                    dev, descales);
}

}  // extern "C"

namespace {

// The decode kernel, compiled for up to 4 or up to 8 new rows, launched as the programmatic
// dependent of the kernel before it on the stream: the prep kernel, which follows all that came
// before in full, or with one piece whatever the caller launched last (the kernel then waits for it).
template <int D>
int launch_decode(dim3 grid, const CUtensorMap& mk, const CUtensorMap& mv, const fa::DecParams& p,
                  cudaStream_t cs) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(fa::kDecMmaThreads);
  cfg.dynamicSmemBytes = fa::DecTcCfg<D>::kSmemBytes;
  cfg.stream = cs;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = p.Sq <= 4 ? cudaLaunchKernelEx(&cfg, fa::fa_decode_kernel<D, 4>, mk, mv, p)
                                  : cudaLaunchKernelEx(&cfg, fa::fa_decode_kernel<D, 8>, mk, mv, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_CUDA;
  }
  return launch_status();
}

// Workspace of a call with P > 1 pieces per head: partial O (fp32) and partial LSE for the
// B + P - 1 (sequence, piece) slots, one arrival counter per (b, h).
size_t decode_workspace_bytes(int B, int Sq, int H, int d, int pieces) {
  if (pieces <= 1) return 0;
  const size_t rows = ((size_t)B + pieces - 1) * H * Sq;
  return align256(rows * d * 4) + align256(rows * 4) + align256((size_t)B * H * 4);
}

// CTAs of the decode kernel that fit on one SM at a time (0 on error).
template <int D>
int decode_ctas_per_sm() {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fa::fa_decode_kernel<D, 8>, fa::kDecMmaThreads,
                                                    fa::DecTcCfg<D>::kSmemBytes) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return n;
}

// Pieces per head when the caller passes 0: as many as fill every CTA slot of the GPU once
// (H x P <= resident CTAs), at least 1, no more than the batch can have tiles, at most 65535.
int decode_auto_pieces(int B, int Sq, int H, int d, int max_keys, int sm_count) {
  const int per_sm = d == 64 ? decode_ctas_per_sm<64>() : decode_ctas_per_sm<128>();
  long long pieces = (long long)std::max(per_sm, 1) * sm_count / H;
  const long long tiles = (long long)B * ((max_keys + fa::kDecTile - 1) / fa::kDecTile);
  pieces = std::min(pieces, std::min(tiles, 65535LL));
  return pieces < 1 ? 1 : (int)pieces;
}

}  // namespace

extern "C" {

int fa_decode_splits(int B, int Sq, int H, int d, int max_keys) {
  if (B < 1 || Sq < 1 || H < 1 || max_keys < 1 || d < 1) return -FA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || Sq > fa::kDecMaxSq) return -FA_ERR_UNSUPPORTED;
  int dev, sms, st;
  if ((st = device_setup(&dev, &sms))) return -st;
  return decode_auto_pieces(B, Sq, H, d, max_keys, sms);
}

size_t fa_decode_workspace_bytes(int B, int Sq, int H, int d, int splits) {
  if (B < 1 || Sq < 1 || H < 1 || (d != 64 && d != 128) || splits < 0) return 0;
  return decode_workspace_bytes(B, Sq, H, d, splits);
}

int fa_decode_paged(const void* q, void* k_cache, void* v_cache, const void* k_new, const void* v_new,
                    const int* block_table, const int* seqlens, void* o, float* lse, int B, int Sq, int H, int d,
                    int num_pages,
                    int page_size, int max_pages, float scale, int causal, int win_l, int win_r, int splits,
                    void* workspace, size_t workspace_bytes_, fa_stream_t stream) {
  if (B < 1 || H < 1 || Sq < 1 || num_pages < 1 || max_pages < 1 || page_size < 1 || splits < 0)
    return FA_ERR_INVALID_ARG;
  if (win_l < -1 || win_r < -1 || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (Sq > fa::kDecMaxSq || page_size % fa::kDecTile != 0) return FA_ERR_UNSUPPORTED;
  if ((double)num_pages * page_size * H * d * 2 >= 1099511627776.0 ||
      (double)max_pages * page_size >= 2147483647.0)
    return FA_ERR_INVALID_ARG;
  if (splits > 65535 || (long long)B * H >= 2147483647LL) return FA_ERR_INVALID_ARG;  // grid and counter limits
  if (!q || !k_cache || !v_cache || !block_table || !seqlens || !o || !lse) return FA_ERR_INVALID_ARG;
  if ((k_new == nullptr) != (v_new == nullptr)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
      !aligned(block_table, 4) || !aligned(seqlens, 4) || !aligned(k_new, 16) || !aligned(v_new, 16))
    return FA_ERR_INVALID_ARG;
  if (causal) win_r = 0;
  const size_t qb = (size_t)B * Sq * H * d * 2, cb = (size_t)num_pages * page_size * H * d * 2;
  const size_t lb = (size_t)B * H * Sq * 4, tb = (size_t)B * max_pages * 4, sb = (size_t)B * 4;
  const void* ins[7] = {q, k_cache, v_cache, block_table, seqlens, k_new, v_new};
  const size_t in_bytes[7] = {qb, cb, cb, tb, sb, k_new ? qb : 0, v_new ? qb : 0};
  for (int i = 0; i < 7; ++i)
    if (overlap(o, qb, ins[i], in_bytes[i]) || overlap(lse, lb, ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
  if (overlap(o, qb, lse, lb) || overlap(k_cache, cb, v_cache, cb)) return FA_ERR_INVALID_ARG;
  for (int i = 0; i < 7; ++i)  // the caches are written when new rows are given: nothing may alias them
    if (k_new && i != 1 && i != 2 &&
        (overlap(k_cache, cb, ins[i], in_bytes[i]) || overlap(v_cache, cb, ins[i], in_bytes[i])))
      return FA_ERR_INVALID_ARG;
  int dev, sms, st;
  if ((st = device_setup(&dev, &sms))) return st;
  if (splits == 0) splits = decode_auto_pieces(B, Sq, H, d, max_pages * page_size, sms);
  const size_t wbytes = decode_workspace_bytes(B, Sq, H, d, splits);
  if (wbytes > 0 && workspace) {
    if (!aligned(workspace, 256) || workspace_bytes_ < wbytes) return FA_ERR_INVALID_ARG;
    for (int i = 0; i < 7; ++i)
      if (overlap(workspace, wbytes, ins[i], in_bytes[i])) return FA_ERR_INVALID_ARG;
    if (overlap(workspace, wbytes, o, qb) || overlap(workspace, wbytes, lse, lb)) return FA_ERR_INVALID_ARG;
  }
  CUtensorMap mk, mv;
  if ((st = make_map_cache(&mk, k_cache, num_pages, page_size, H, d)) ||
      (st = make_map_cache(&mv, v_cache, num_pages, page_size, H, d)))
    return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  void* ws = workspace;
  if (wbytes > 0 && !ws) {
    if (cudaMallocAsync(&ws, wbytes, cs) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_NO_MEMORY;
    }
  }
  fa::DecParams p;
  p.B = B;
  p.Sq = Sq;
  p.H = H;
  p.page_size = page_size;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = scale * fa::kLog2e;
  p.win_l = win_l;
  p.win_r = win_r;
  p.pieces = splits;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_part = static_cast<float*>(ws);
  const size_t part_rows = ((size_t)B + splits - 1) * H * Sq;  // (sequence, piece) slots
  const size_t part_bytes = align256(part_rows * d * 4);
  const size_t lse_part_bytes = align256(part_rows * 4);
  p.lse_part = wbytes ? reinterpret_cast<float*>(static_cast<char*>(ws) + part_bytes) : nullptr;
  p.arrivals = wbytes ? reinterpret_cast<int*>(static_cast<char*>(ws) + part_bytes + lse_part_bytes) : nullptr;
  p.k_new = static_cast<const __nv_bfloat16*>(k_new);
  p.v_new = static_cast<const __nv_bfloat16*>(v_new);
  p.k_cache = static_cast<__nv_bfloat16*>(k_cache);
  p.v_cache = static_cast<__nv_bfloat16*>(v_cache);
  st = FA_OK;
  if (splits > 1) {
    const int count = B * H;
    const int blocks = (int)std::min<long long>((count + 255) / 256, sms);
    fa::fa_decode_prep_kernel<<<blocks, 256, 0, cs>>>(p.arrivals, count);
    st = launch_status();
  }
  if (!st) {
    const dim3 grid(H, splits);  // heads fastest: concurrent CTAs share cache rows
    if (d == 64)
      st = launch_decode<64>(grid, mk, mv, p, cs);
    else
      st = launch_decode<128>(grid, mk, mv, p, cs);
  }
  if (wbytes > 0 && !workspace && cudaFreeAsync(ws, cs) != cudaSuccess && !st) st = FA_ERR_CUDA;
  return st;
}

int fa_cache_write(const void* k_new, const void* v_new, long long row_stride, void* k_cache, void* v_cache,
                   void* k_scale, void* v_scale, const int* block_table, const int* seqlens, const int* cu_seqlens,
                   int B, int total, int H, int d, int num_pages, int page_size, int max_pages, fa_stream_t stream) {
  return cache_rows<true>(const_cast<void*>(k_new), const_cast<void*>(v_new), row_stride, k_cache, v_cache, k_scale,
                          v_scale, block_table, seqlens, cu_seqlens, B, total, H, d, num_pages, page_size, max_pages,
                          stream);
}

int fa_cache_read(const void* k_cache, const void* v_cache, const void* k_scale, const void* v_scale,
                  const int* block_table, const int* seqlens, const int* cu_seqlens, void* k, void* v,
                  long long row_stride, int B, int total, int H, int d, int num_pages, int page_size, int max_pages,
                  fa_stream_t stream) {
  return cache_rows<false>(k, v, row_stride, const_cast<void*>(k_cache), const_cast<void*>(v_cache),
                           const_cast<void*>(k_scale), const_cast<void*>(v_scale), block_table, seqlens, cu_seqlens,
                           B, total, H, d, num_pages, page_size, max_pages, stream);
}

size_t fa_chunk_workspace_bytes(int B, int total, int Hq, int Hkv, int d) {
  if (B < 1 || total < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (d != 64 && d != 128)) return 0;
  int dev, sms;
  if (chunk_setup(&dev, &sms)) return 0;
  return chunk_workspace(sms, chunk_tiles(B, total, Hq / Hkv), d).bytes();
}

int fa_chunk_paged(const void* q, long long q_stride, const void* k_cache, const void* v_cache, const void* k_scale,
                   const void* v_scale, const int* block_table, const int* seqlens, const int* cu_seqlens, void* o,
                   float* lse, int B, int total, int Hq, int Hkv, int d, int num_pages, int page_size, int max_pages,
                   float scale, int causal, int win_l, int win_r, int sinks, void* workspace,
                   size_t workspace_bytes_, fa_stream_t stream) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || win_l < -1 || win_r < -1 || sinks < 0 || !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
  int st = check_paged(B, total, Hkv, d, num_pages, page_size, max_pages, k_cache, v_cache, k_scale, v_scale,
                       block_table, seqlens, cu_seqlens);
  if (st) return st;
  const int G = Hq / Hkv;
  if (G > 128) return FA_ERR_UNSUPPORTED;
  if (total > 0 && (!q || !o || !lse)) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4) || q_stride < (long long)Hq * d || q_stride % 8 != 0 ||
      q_stride > 1073741824LL || (double)total * Hq >= 1099511627776.0)
    return FA_ERR_INVALID_ARG;
  const bool f8 = k_scale != nullptr;
  const int max_keys = max_pages * page_size;
  if (causal) win_r = 0;
  if (win_l >= max_keys) win_l = -1;
  if (win_r >= max_keys) win_r = -1;
  if (win_l < 0) sinks = 0;  // no left bound: every first key is visible anyway
  const size_t cells = (size_t)num_pages * page_size * Hkv, cb = cells * d * (f8 ? 1 : 2);
  const size_t ob = (size_t)total * Hq * d * 2, lb = (size_t)total * Hq * 4;
  const Span ins[8] = {{q, rows_bytes(total, (size_t)Hq * d, q_stride)}, {k_cache, cb}, {v_cache, cb},
                       {k_scale, cells}, {v_scale, cells}, {block_table, (size_t)B * max_pages * 4},
                       {seqlens, (size_t)B * 4}, {cu_seqlens, (size_t)(B + 1) * 4}};
  if (any_overlap({o, ob}, ins, 8) || any_overlap({lse, lb}, ins, 8) || (o && lse && overlap(o, ob, lse, lb)))
    return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = chunk_setup(&dev, &sms))) return st;
  if (total == 0) return FA_OK;
  const bool few = chunk_few(f8, d, B, total, G);
  const int tiles = chunk_tiles(B, total, G), tq = (few ? fa::kFewRows : 128) / G;
  const ChunkWorkspace wb = chunk_workspace(sms, tiles, d);
  if (workspace) {
    const Span ws{workspace, wb.bytes()};
    if (!aligned(workspace, 256) || workspace_bytes_ < wb.bytes() || any_overlap(ws, ins, 8) ||
        overlap(workspace, ws.n, o, ob) || overlap(workspace, ws.n, lse, lb))
      return FA_ERR_INVALID_ARG;
  }
  // CTAs: one per SM, and no more than the key tiles there can be; heads in groups (fa_chunk.cuh)
  const int hg = chunk_head_group(Hkv, sms);
  const double blocks = (double)(total / ((few ? 1 : tiles) * tq)) + std::min(B, total);
  const int key_tiles = (max_keys + 127) / 128;
  const double most = blocks * (Hkv / hg) * key_tiles;
  const int pieces = most < sms / hg ? (int)most : sms / hg, ctas = pieces * hg;
  int box_rows = 16;
  while (box_rows < 128 && page_size % (2 * box_rows) == 0) box_rows *= 2;
  CUtensorMap m[5];
  if ((!few && (st = make_map_chunk_q(&m[0], q, total, Hkv, G, d, q_stride, tq))) ||
      (st = make_map_pages(&m[1], k_cache, num_pages, page_size, Hkv, d, box_rows, f8, few)) ||
      (st = make_map_pages(&m[2], v_cache, num_pages, page_size, Hkv, d, box_rows, f8, few)))
    return st;
  m[3] = m[1];
  m[4] = m[2];
  if (f8 && ((st = make_map_scales(&m[3], k_scale, num_pages, page_size, Hkv, box_rows)) ||
             (st = make_map_scales(&m[4], v_scale, num_pages, page_size, Hkv, box_rows))))
    return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  void* ws = workspace;
  if (!ws && cudaMallocAsync(&ws, wb.bytes(), cs) != cudaSuccess) {
    cudaGetLastError();
    return FA_ERR_NO_MEMORY;
  }
  fa::ChunkParams p;
  p.B = B;
  p.total = total;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.tq = tq;
  p.page_size = page_size;
  p.by_page = fast_div(page_size);
  p.by_group = fast_div(G);
  p.by_tokens = fast_div((few ? 1 : tiles) * tq);
  p.box_rows = box_rows;
  p.max_pages = max_pages;
  p.num_pages = num_pages;
  p.scale_log2 = scale * fa::kLog2e;
  p.win_l = win_l;
  p.win_r = win_r;
  p.sinks = sinks;
  p.pieces = pieces;
  p.hg = hg;
  p.ctas = ctas;
  p.block_table = block_table;
  p.seqlens = seqlens;
  p.cu = cu_seqlens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.o_part = static_cast<float*>(ws);
  p.lse_part = reinterpret_cast<float*>(static_cast<char*>(ws) + wb.o_bytes);
  p.split = reinterpret_cast<int4*>(static_cast<char*>(ws) + wb.o_bytes + wb.lse_bytes);
  if (log_enabled())
    std::fprintf(stderr,
                 "[fa] chunk B=%d total=%d Hq=%d Hkv=%d d=%d f8=%d tiles=%d few=%d pieces=%d hg=%d box=%d win=(%d,%d) "
                 "sinks=%d\n",
                 B, total, Hq, Hkv, d, f8, tiles, few, pieces, hg, box_rows, win_l, win_r, sinks);
  if (few) {
    st = launch_dependent(fa::fa_chunk_few_kernel, dim3(ctas), fa::kFewThreads, fa::FewCfg::kSmemBytes, cs, m[1], m[2],
                          m[3], m[4], static_cast<const __nv_bfloat16*>(q), q_stride, p);
  } else {
    st = d == 64 ? chunk_variant<64>(f8, tiles, ctas, m, p, cs) : chunk_variant<128>(f8, tiles, ctas, m, p, cs);
  }
  // (with one key tile per block at most, or one piece, no block is spread over pieces)
  if (!st && pieces > 1 && key_tiles > 1)
    st = d == 64 ? (tiles == 1 ? chunk_merge_launch<64, 1>(ctas, p, cs) : chunk_merge_launch<64, 2>(ctas, p, cs))
                 : (tiles == 1 ? chunk_merge_launch<128, 1>(ctas, p, cs) : chunk_merge_launch<128, 2>(ctas, p, cs));
  if (!workspace && cudaFreeAsync(ws, cs) != cudaSuccess && !st) st = FA_ERR_CUDA;
  return st;
}

int fa_cache_write_args(const fa_cache_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_cache_write(a->k_rows, a->v_rows, a->row_stride, a->k_cache, a->v_cache, a->k_scale, a->v_scale,
                        a->block_table, a->seqlens, a->cu_seqlens, a->B, a->total, a->H, a->d, a->num_pages,
                        a->page_size, a->max_pages, a->stream);
}

int fa_cache_read_args(const fa_cache_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_cache_read(a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->block_table, a->seqlens, a->cu_seqlens,
                       const_cast<void*>(a->k_rows), const_cast<void*>(a->v_rows), a->row_stride, a->B, a->total, a->H,
                       a->d, a->num_pages, a->page_size, a->max_pages, a->stream);
}

int fa_chunk_paged_args(const fa_chunk_args* a) {
  if (!a) return FA_ERR_INVALID_ARG;
  return fa_chunk_paged(a->q, a->q_stride, a->k_cache, a->v_cache, a->k_scale, a->v_scale, a->block_table, a->seqlens,
                        a->cu_seqlens, a->o, a->lse, a->B, a->total, a->Hq, a->Hkv, a->d, a->num_pages, a->page_size,
                        a->max_pages, a->scale, a->causal, a->win_l, a->win_r, a->sinks, a->workspace,
                        a->workspace_bytes, a->stream);
}

int fa_bwd_preprocess(const void* o, const float* lse, const void* dO, int B, int N, int H, int d, void* workspace,
                      size_t workspace_bytes_, fa_stream_t stream) {
  int wl = -1, wr = -1;
  int st = check_problem(B, N, H, d, 1.0f, 0, &wl, &wr);
  if (st) return st;
  const Shape s{B, N, H, d};
  if (!o || !lse || !dO || !aligned(o, 16) || !aligned(dO, 16) || !aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes_, s))) return st;
  const size_t tb = s.tensor_bytes(), wb = workspace_bytes(s), lb = s.rowvec_bytes();
  if (overlap(workspace, wb, o, tb) || overlap(workspace, wb, dO, tb) || overlap(workspace, wb, lse, lb))
    return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  return launch_pre(o, lse, dO, s, carve(workspace, s), reinterpret_cast<cudaStream_t>(stream));
}

int fa_bwd_main(const void* q, const void* k, const void* v, const void* dO, void* dk, void* dv, int B, int N, int H,
                int d, float scale, int causal, int win_l, int win_r, void* workspace, size_t workspace_bytes_,
                fa_stream_t stream) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  const Shape s{B, N, H, d};
  if (!q || !k || !v || !dO || !dk || !dv) return FA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(dO, 16) || !aligned(dk, 16) ||
      !aligned(dv, 16))
    return FA_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes_, s))) return st;
  const size_t tb = s.tensor_bytes(), wb = workspace_bytes(s);
  const void* ins[4] = {q, k, v, dO};
  for (const void* in : ins)
    if (overlap(dk, tb, in, tb) || overlap(dv, tb, in, tb) || overlap(workspace, wb, in, tb)) return FA_ERR_INVALID_ARG;
  if (overlap(dk, tb, dv, tb) || overlap(workspace, wb, dk, tb) || overlap(workspace, wb, dv, tb))
    return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  return launch_main(q, k, v, dO, dk, dv, s, scale, causal, win_l, win_r, carve(workspace, s), sms,
                     reinterpret_cast<cudaStream_t>(stream));
}

int fa_bwd_dq_convert(void* dq, int B, int N, int H, int d, void* workspace, size_t workspace_bytes_,
                      fa_stream_t stream) {
  int wl = -1, wr = -1;
  int st = check_problem(B, N, H, d, 1.0f, 0, &wl, &wr);
  if (st) return st;
  const Shape s{B, N, H, d};
  if (!dq || !aligned(dq, 16)) return FA_ERR_INVALID_ARG;
  if ((st = check_workspace(workspace, workspace_bytes_, s))) return st;
  if (overlap(workspace, workspace_bytes(s), dq, s.tensor_bytes())) return FA_ERR_INVALID_ARG;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  return launch_convert(dq, s, carve(workspace, s), reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"

static int bwd_impl(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                    void* dq, void* dk, void* dv, int B, int N, int H, int d, float scale, int causal, int win_l,
                    int win_r, void* workspace, size_t workspace_bytes_, fa_stream_t stream, bool deterministic,
                    const float* alibi = nullptr, const int* cu = nullptr, int nseg = 0) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  const Shape s{B, N, H, d};
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  const void* ptrs[8] = {q, k, v, o, dO, dq, dk, dv};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return FA_ERR_INVALID_ARG;
  if (!aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  const size_t tb = s.tensor_bytes(), lb = s.rowvec_bytes();
  const void* ins[5] = {q, k, v, o, dO};
  void* outs[3] = {dq, dk, dv};
  for (void* out : outs) {
    for (const void* in : ins)
      if (overlap(out, tb, in, tb)) return FA_ERR_INVALID_ARG;
    if (overlap(out, tb, lse, lb)) return FA_ERR_INVALID_ARG;
  }
  if (overlap(dq, tb, dk, tb) || overlap(dq, tb, dv, tb) || overlap(dk, tb, dv, tb)) return FA_ERR_INVALID_ARG;
  if (alibi) {
    if (!aligned(alibi, 4)) return FA_ERR_INVALID_ARG;
    for (void* out : outs)
      if (overlap(out, tb, alibi, (size_t)B * H * 4)) return FA_ERR_INVALID_ARG;
  }
  if (workspace) {
    if ((st = check_workspace(workspace, workspace_bytes_, s))) return st;
    if (alibi && overlap(workspace, workspace_bytes(s), alibi, (size_t)B * H * 4)) return FA_ERR_INVALID_ARG;
    const size_t wb = workspace_bytes(s);
    for (const void* in : ins)
      if (overlap(workspace, wb, in, tb)) return FA_ERR_INVALID_ARG;
    for (void* out : outs)
      if (overlap(workspace, wb, out, tb)) return FA_ERR_INVALID_ARG;
    if (overlap(workspace, wb, lse, lb)) return FA_ERR_INVALID_ARG;
  }
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  void* ws = workspace;
  const size_t wbytes = workspace_bytes(s);
  if (!ws) {
    if (cudaMallocAsync(&ws, wbytes, cs) != cudaSuccess) {
      cudaGetLastError();
      return FA_ERR_NO_MEMORY;
    }
  }
  const Workspace w = carve(ws, s);
  st = launch_pre(o, lse, dO, s, w, cs);
  BwdOptions opt;
  opt.alibi = alibi;
  opt.cu = cu;
  opt.nseg = nseg;
  if (!st && cu) st = launch_check_cu(cu, nseg, N, cs);
  if (deterministic) {
    if (!st) st = launch_main(q, k, v, dO, dk, dv, s, scale, causal, win_l, win_r, w, sms, cs, false, opt);
    if (!st) st = launch_dq(q, k, v, dO, dq, s, scale, causal, win_l, win_r, w, sms, cs, opt);
  } else {
    if (!st) st = launch_main(q, k, v, dO, dk, dv, s, scale, causal, win_l, win_r, w, sms, cs, true, opt);
    if (!st) st = launch_convert(dq, s, w, cs);
  }
  if (!workspace && cudaFreeAsync(ws, cs) != cudaSuccess && !st) st = FA_ERR_CUDA;
  return st;
}

extern "C" {

int fa_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO, void* dq,
           void* dk, void* dv, int B, int N, int H, int d, float scale, int causal, int win_l, int win_r,
           void* workspace, size_t workspace_bytes_, fa_stream_t stream) {
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, N, H, d, scale, causal, win_l, win_r, workspace,
                  workspace_bytes_, stream, false);
}

int fa_bwd_ex(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
              const float* alibi_slopes, void* dq, void* dk, void* dv, int B, int N, int H, int d, float scale,
              int causal, int win_l, int win_r, int deterministic, void* workspace, size_t workspace_bytes_,
              fa_stream_t stream) {
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, N, H, d, scale, causal, win_l, win_r, workspace,
                  workspace_bytes_, stream, deterministic != 0, alibi_slopes);
}

int fa_bwd_varlen(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                  const int* cu_seqlens, const float* alibi_slopes, void* dq, void* dk, void* dv, int B, int total,
                  int H, int d, float scale, int causal, int win_l, int win_r, int deterministic, void* workspace,
                  size_t workspace_bytes_, fa_stream_t stream) {
  if (B < 1 || !cu_seqlens || !aligned(cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  const size_t tb = (size_t)total * H * d * 2, cb = (size_t)(B + 1) * 4;
  void* outs[3] = {dq, dk, dv};
  for (void* out : outs)
    if (out && total > 0 && H > 0 && d > 0 && overlap(out, tb, cu_seqlens, cb)) return FA_ERR_INVALID_ARG;
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, 1, total, H, d, scale, causal, win_l, win_r, workspace,
                  workspace_bytes_, stream, deterministic != 0, alibi_slopes, cu_seqlens, B);
}

int fa_bwd_deterministic(const void* q, const void* k, const void* v, const void* o, const float* lse,
                         const void* dO, void* dq, void* dk, void* dv, int B, int N, int H, int d, float scale,
                         int causal, int win_l, int win_r, void* workspace, size_t workspace_bytes_,
                         fa_stream_t stream) {
  return bwd_impl(q, k, v, o, lse, dO, dq, dk, dv, B, N, H, d, scale, causal, win_l, win_r, workspace,
                  workspace_bytes_, stream, true);
}

int fa_bwd_static_workspace(const void* q, const void* k, const void* v, const void* o, const float* lse,
                            const void* dO, void* dq, void* dk, void* dv, int B, int N, int H, int d, float scale,
                            int causal, int win_l, int win_r, fa_stream_t stream) {
  int st = check_problem(B, N, H, d, scale, causal, &win_l, &win_r);
  if (st) return st;
  const Shape s{B, N, H, d};
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv) return FA_ERR_INVALID_ARG;
  const void* ptrs[8] = {q, k, v, o, dO, dq, dk, dv};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return FA_ERR_INVALID_ARG;
  if (!aligned(lse, 4)) return FA_ERR_INVALID_ARG;
  const size_t tb = s.tensor_bytes(), lb = s.rowvec_bytes();
  const void* ins[5] = {q, k, v, o, dO};
  void* outs[3] = {dq, dk, dv};
  for (void* out : outs) {
    for (const void* in : ins)
      if (overlap(out, tb, in, tb)) return FA_ERR_INVALID_ARG;
    if (overlap(out, tb, lse, lb)) return FA_ERR_INVALID_ARG;
  }
  if (overlap(dq, tb, dk, tb) || overlap(dq, tb, dv, tb) || overlap(dk, tb, dv, tb)) return FA_ERR_INVALID_ARG;
  if (workspace_bytes(s) > kStaticWorkspaceBytes) return FA_ERR_UNSUPPORTED;
  int dev, sms;
  if ((st = device_setup(&dev, &sms))) return st;
  void* ws = nullptr;
  if ((st = static_workspace_address(dev, &ws))) return st;
  cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  const Workspace w = carve(ws, s);  // the preprocess launch zeroes dQ and rewrites LSE2 / D
  st = launch_pre(o, lse, dO, s, w, cs);
  if (!st) st = launch_main(q, k, v, dO, dk, dv, s, scale, causal, win_l, win_r, w, sms, cs);
  if (!st) st = launch_convert(dq, s, w, cs);
  return st;
}

int fa_check(fa_stream_t stream) {
  if (cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  int err = 0;
  if (cudaMemcpyFromSymbol(&err, fa::g_fa_error, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  if (err == 0) return FA_OK;
  const int zero = 0;
  if (cudaMemcpyToSymbol(fa::g_fa_error, &zero, sizeof(int)) != cudaSuccess) return FA_ERR_CUDA;
  return (err & fa::kErrWaitTimeout) ? FA_ERR_TIMEOUT : FA_ERR_DEVICE;
}

}  // extern "C"
