// C ABI of the exact attention library (declared in include/attn.h): argument validation,
// device checks, TMA descriptor encoding and kernel launches.  No allocation happens here and
// no pointer is kept after a call returns.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <algorithm>
#include <cstring>
#include <mutex>

#include "../../include/attn.h"
#include "bwd_sm100.cuh"
#include "common.cuh"
#include "decode.cuh"
#include "decode_prefix.cuh"
#include "decode_tc.cuh"
#include "fwd_f32.cuh"
#include "fwd_sm100.cuh"
#include "pages.cuh"
#include "qk_norm_rope.cuh"

namespace attn {
namespace {

constexpr int kMaxDevices = 64;
constexpr float kLog2e = 1.4426950408889634f;

struct DeviceInfo {
  bool probed = false;
  bool sm100 = false;
  int num_sms = 0;
  bool fwd_configured = false;
  bool bwd_configured = false;
  bool dtc_configured = false;
  bool pfx_configured = false;
  bool pages_configured = false;
};

std::mutex g_mutex;
DeviceInfo g_devices[kMaxDevices];
thread_local const char* g_last_detail = "no error";

// Maps a CUDA runtime result to a status, remembering the runtime's text for
// attn_last_error_detail().
int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return ATTN_OK;
  g_last_detail = cudaGetErrorString(e);
  return ATTN_ERR_CUDA;
}
PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;

// Work-unit counters of the persistent prefill and backward kernels, one per stream that launches
// them: calls on one stream run one after another and can share a counter, calls on different
// streams may overlap and must not.  A counter is zero between launches (the last CTA of a launch
// to take from it sets it back).  Past kCounterSlots streams on one device, a stream shares the
// counter of an earlier one.
constexpr int kCounterSlots = 1024;
static __device__ unsigned int g_unit_counters[kCounterSlots];

struct CounterTable {
  unsigned int* base = nullptr;
  cudaStream_t stream[kCounterSlots] = {};
  int used = 0;
};
CounterTable g_counter_tables[kMaxDevices];

// The counter of `st` on the current device.
int unit_counter(cudaStream_t st, unsigned int** out) {
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev));
  if (rc != ATTN_OK) return rc;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mutex);
  CounterTable& tab = g_counter_tables[dev];
  if (tab.base == nullptr) {
    void* p = nullptr;
    rc = cuda_status(cudaGetSymbolAddress(&p, g_unit_counters));
    if (rc != ATTN_OK) return rc;
    tab.base = static_cast<unsigned int*>(p);
  }
  int slot = -1;
  for (int i = 0; i < tab.used; ++i)
    if (tab.stream[i] == st) {
      slot = i;
      break;
    }
  if (slot < 0) {
    if (tab.used < kCounterSlots) {
      slot = tab.used++;
      tab.stream[slot] = st;
    } else {
      slot = static_cast<int>(reinterpret_cast<uintptr_t>(st) % kCounterSlots);
    }
  }
  *out = tab.base + slot;
  return ATTN_OK;
}

// Looks up the current device once: compute capability 10.x and the SM count; raises the
// dynamic shared memory limit of the tensor-core kernel on first use.
int current_device(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cuda_status(cudaGetLastError());
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceInfo& info = g_devices[dev];
  if (!info.probed) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return ATTN_ERR_CUDA;
    info.sm100 = (major == 10 && minor == 0);
    info.num_sms = sms;
    info.probed = true;
  }
  if (!info.sm100) return ATTN_ERR_UNSUPPORTED;
  *out = &info;
  return ATTN_OK;
}

int configure_fwd(DeviceInfo* info) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!info->fwd_configured) {
    void (*kernels[6])(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, fwd::Params) = {
        fwd::fwd_bf16_sm100_kernel<false, false>, fwd::fwd_bf16_sm100_kernel<true, false>,
        fwd::fwd_bf16_sm100_kernel<false, true>,  fwd::fwd_bf16_sm100_kernel<true, true>,
        fwd::fwd_fp8_sm100_kernel<false>,         fwd::fwd_fp8_sm100_kernel<true>};
    for (auto* kern : kernels) {
      const int rc = cuda_status(cudaFuncSetAttribute(
          kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(fwd::kSmemBytes)));
      if (rc != ATTN_OK) return rc;
    }
    void (*sparse_kernels[2])(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, fwd::Params) = {
        fwd::fwd_bf16_sparse_sm100_kernel<false>, fwd::fwd_bf16_sparse_sm100_kernel<true>};
    for (auto* kern : sparse_kernels) {
      const int rc = cuda_status(cudaFuncSetAttribute(kern,
                                                      cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      static_cast<int>(fwd::kSmemBytesSparse)));
      if (rc != ATTN_OK) return rc;
    }
    info->fwd_configured = true;
  }
  if (g_encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess || fn == nullptr)
      return ATTN_ERR_CUDA;
    g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Raises the dynamic shared memory limit of the tensor-core decode kernels on first use (and
// looks up the tensor-map encoder, as configure_fwd does).
int configure_decode_tc(DeviceInfo* info) {
  int rc = configure_fwd(info);
  if (rc != ATTN_OK) return rc;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!info->dtc_configured) {
    void (*kernels[8])(CUtensorMap, CUtensorMap, CUtensorMap, float*, float*, int, int, int, int,
                       int, float, dec::Paged) = {
        dtc::decode_tc_kernel<1, false>, dtc::decode_tc_kernel<2, false>,
        dtc::decode_tc_kernel<4, false>, dtc::decode_tc_kernel<8, false>,
        dtc::decode_tc_kernel<1, true>,  dtc::decode_tc_kernel<2, true>,
        dtc::decode_tc_kernel<4, true>,  dtc::decode_tc_kernel<8, true>};
    for (auto* kern : kernels) {
      rc = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(dtc::kSmemBytes)));
      if (rc != ATTN_OK) return rc;
    }
    info->dtc_configured = true;
  }
  return ATTN_OK;
}

// Raises the dynamic shared memory limit of the backward kernels on first use.
int configure_bwd(DeviceInfo* info) {
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!info->bwd_configured) {
    int rc = cuda_status(cudaFuncSetAttribute(bwd::bwd_dkdv_kernel,
                                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(bwd::kSmemKVBytes)));
    if (rc != ATTN_OK) return rc;
    rc = cuda_status(cudaFuncSetAttribute(bwd::bwd_dq_kernel,
                                          cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(bwd::kSmemQBytes)));
    if (rc != ATTN_OK) return rc;
    info->bwd_configured = true;
  }
  return ATTN_OK;
}

// Backward workspace, in this order: LSE * log2(e) and D per query row (fp32, rows padded to
// whole 128-row tiles); the dS block offsets of the key blocks (int32, num_kblocks + 1); the
// dS^T blocks (bf16 128 x 128, one per visible (key block, query tile) pair and query head).
struct BwdLayout {
  size_t npad, pairs, off_bytes, ds_offset, total;
};

BwdLayout bwd_layout(int B, int Hq, int Nq, int Nk, const MaskSpec& m) {
  BwdLayout L{};
  const int nqt = (Nq + bwd::kT - 1) / bwd::kT, nkb = (Nk + bwd::kT - 1) / bwd::kT;
  L.npad = static_cast<size_t>(nqt) * bwd::kT;
  size_t pairs = 0;
  for (int kb = 0; kb < nkb; ++kb) {
    const int c0 = kb * bwd::kT, c1 = (c0 + bwd::kT < Nk ? c0 + bwd::kT : Nk) - 1;
    pairs += static_cast<size_t>(bwd::query_tiles(m, c0, c1, Nk - Nq, Nq).count());
  }
  L.pairs = pairs;
  const size_t vec = 2 * static_cast<size_t>(B) * Hq * L.npad * sizeof(float);
  L.off_bytes = (static_cast<size_t>(nkb) + 1) * sizeof(int);
  L.ds_offset = (vec + L.off_bytes + 255) & ~size_t(255);
  L.total = L.ds_offset + static_cast<size_t>(B) * Hq * pairs * bwd::kT * bwd::kT * 2;
  return L;
}

// Common argument rules of the forward entry points.
int check_fwd_args(const void* q, const void* k, const void* v, const void* o, int B, int Hq,
                   int Hkv, int Nq, int Nk, int mask_kind, int window, int n_sink, float scale) {
  if (B < 0 || Nq < 0 || Nk < 0 || Hq < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  // a pointer may be NULL only when its tensor holds no element
  const bool q_empty = B == 0 || Nq == 0, kv_empty = B == 0 || Nk == 0;
  if ((!q_empty && (q == nullptr || o == nullptr)) || (!kv_empty && (k == nullptr || v == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (mask_kind < ATTN_MASK_FULL || mask_kind > ATTN_MASK_LOCAL_GLOBAL) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_SLIDING && window < 1) return ATTN_ERR_INVALID_ARG;
  if (mask_kind == ATTN_MASK_LOCAL_GLOBAL && window < 0) return ATTN_ERR_INVALID_ARG;
  if (n_sink < 0) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

MaskSpec make_mask(int mask_kind, int window, int n_sink, int Nk) {
  MaskSpec m;
  m.kind = mask_kind;
  const bool windowed = mask_kind == ATTN_MASK_SLIDING || mask_kind == ATTN_MASK_LOCAL_GLOBAL;
  m.window = windowed ? window : 0;
  m.n_sink = windowed ? n_sink : 0;
  m.Nk = Nk;
  return m;
}

// O = 0 and LSE = -inf for rows that can see no key at all (Nk = 0).
template <typename T>
__global__ void fill_empty_kernel(T* o, float* lse, size_t rows, int d) {
  const size_t i = blockIdx.x * static_cast<size_t>(blockDim.x) + threadIdx.x;
  if (i < rows * d) o[i] = T(0.f);
  if (lse != nullptr && i < rows) lse[i] = -INFINITY;
}

template <typename T>
int launch_fill_empty(T* o, float* lse, size_t rows, int d, cudaStream_t stream) {
  const size_t n = rows * static_cast<size_t>(d);
  if (n == 0) return ATTN_OK;
  const unsigned blocks = static_cast<unsigned>((n + 255) / 256);
  fill_empty_kernel<T><<<blocks, 256, 0, stream>>>(o, lse, rows, d);
  return cuda_status(cudaGetLastError());
}

// 3-D tiled TMA map over a [heads][rows][128] bf16 tensor: box of 64 columns x box_rows rows,
// 128-byte swizzle (the layout tcgen05.mma descriptors read).  Rows past `rows` read as zero
// and are not written.
int encode_map(CUtensorMap* map, const void* base, int rows, int heads, uint32_t box_rows = 128) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(fwd::kD), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(fwd::kD) * 2,
                                 static_cast<cuuint64_t>(rows) * fwd::kD * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// 3-D tiled TMA map over [heads][rows][128] E4M3 codes (one byte each), read as boxes of the full
// 128-byte row width x 128 rows x 1 head with the 128-byte swizzle.
int encode_map_e4m3(CUtensorMap* map, const void* base, int rows, int heads) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(fwd::kD), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(fwd::kD),
                                 static_cast<cuuint64_t>(rows) * fwd::kD};
  const cuuint32_t box[3] = {128, 128, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims,
                        strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// 3-D tiled TMA map over a token-major packed [rows][heads][128] bf16 tensor, read as boxes of
// 64 columns x 1 head x 128 rows (same shared-memory layout as encode_map).
int encode_map_packed(CUtensorMap* map, const void* base, int rows, int heads,
                      uint32_t box_rows = 128) {
  // dimensions (d, rows, heads): rows second, so that a box is a 64 x 128 block of one head as
  // in the dense map (a box that is one element wide in its second dimension copies measurably
  // slower); the row stride (heads * d) exceeds the head stride (d)
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(fwd::kD), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads) * fwd::kD * 2,
                                 static_cast<cuuint64_t>(fwd::kD) * 2};
  const cuuint32_t box[3] = {64, box_rows, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// TMA map of a prefill output (bf16, d = 128): dense [heads][rows][128] or packed
// [rows][heads][128], written as boxes of 32 columns x 32 rows x 1 head staged with the 64-byte
// swizzle (one box per softmax warp and column quarter).
int encode_map_out(CUtensorMap* map, void* base, int rows, int heads, bool packed) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(fwd::kD), static_cast<cuuint64_t>(rows),
                              static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[2] = {
      packed ? static_cast<cuuint64_t>(heads) * fwd::kD * 2 : static_cast<cuuint64_t>(fwd::kD) * 2,
      packed ? static_cast<cuuint64_t>(fwd::kD) * 2 : static_cast<cuuint64_t>(rows) * fwd::kD * 2};
  const cuuint32_t box[3] = {32, 32, 1};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estride,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

constexpr int kMaxSplits = 256;

int decode_splits(int B, int Hkv, int Nk, int G, int requested, int num_sms) {
  int max_chunk;
  switch (G) {
    case 1: max_chunk = dec::max_chunk<1>(); break;
    case 2: max_chunk = dec::max_chunk<2>(); break;
    case 4: max_chunk = dec::max_chunk<4>(); break;
    default: max_chunk = dec::max_chunk<8>(); break;
  }
  const int min_splits = Nk > 0 ? (Nk + max_chunk - 1) / max_chunk : 1;
  int s = requested;
  if (s <= 0) {
    // chunks of whole 128-key tiles, at most the tensor-core kernel's dtc::kMaxChunk keys, and
    // small enough for about 4 CTAs per SM (2 are resident at a time)
    const long long groups = B * Hkv > 0 ? static_cast<long long>(B) * Hkv : 1;
    const long long want = (4LL * num_sms + groups - 1) / groups;
    long long chunk = Nk > 0 ? (Nk + want - 1) / want : 1;
    chunk = (chunk + dtc::kTile - 1) / dtc::kTile * dtc::kTile;
    if (chunk > dtc::kMaxChunk) chunk = dtc::kMaxChunk;
    s = Nk > 0 ? static_cast<int>((Nk + chunk - 1) / chunk) : 1;
  }
  if (s < min_splits) s = min_splits;
  if (s < 1) s = 1;
  if (s > kMaxSplits) s = kMaxSplits;
  return s;
}

size_t decode_ws_bytes(int B, int Hq, int splits) {
  const size_t rows = static_cast<size_t>(B) * Hq * splits;
  return rows * dec::kD * sizeof(float) + ((rows * sizeof(float) + 15) & ~size_t(15));
}

template <int G>
void launch_decode_split(dim3 grid, int chunk, cudaStream_t stream, const __nv_bfloat16* q,
                         const __nv_bfloat16* k, const __nv_bfloat16* v, float* ws_o,
                         float* ws_lse, int Hq, int Hkv, int Nk, int splits, float c,
                         const dec::Paged* pg) {
  const size_t smem = static_cast<size_t>(dec::smem_floats(G, chunk)) * sizeof(float);
  if (pg == nullptr)
    dec::decode_split_kernel<G><<<grid, dec::kThreads, smem, stream>>>(
        q, k, v, ws_o, ws_lse, Hq, Hkv, Nk, chunk, splits, c);
  else if ((1 << pg->page_shift) >= 2 * dec::unroll<G>())
    dec::decode_split_paged_kernel<G, 2><<<grid, dec::kThreads, smem, stream>>>(
        q, k, v, ws_o, ws_lse, Hq, Hkv, Nk, chunk, splits, c, *pg);
  else
    dec::decode_split_paged_kernel<G, 1><<<grid, dec::kThreads, smem, stream>>>(
        q, k, v, ws_o, ws_lse, Hq, Hkv, Nk, chunk, splits, c, *pg);
}

// Split kernel + combine over a contiguous cache (pg == nullptr; Nk keys per sequence) or a
// paged one (Nk = the longest sequence).  Arguments are already checked.
int decode_run(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
               int Hkv, int Nk, float scale, int num_splits, void* workspace,
               size_t workspace_bytes, cudaStream_t st, const DeviceInfo* info,
               const dec::Paged* pg) {
  const int G = Hq / Hkv;
  const int splits = decode_splits(B, Hkv, Nk, G, num_splits, info->num_sms);
  const size_t need = decode_ws_bytes(B, Hq, splits);
  if (workspace == nullptr || workspace_bytes < need || !aligned16(workspace))
    return ATTN_ERR_WORKSPACE;
  int chunk = (Nk + splits - 1) / splits;
  // paged: chunks of whole 32-key groups (the kernel's one-lookup-per-iteration path needs the
  // chunk starts aligned); a multiple of 32 keeps chunk <= the kernel's largest chunk, and
  // splits past the last key see no keys
  if (pg != nullptr) chunk = (chunk + 31) & ~31;
  float* ws_o = static_cast<float*>(workspace);
  float* ws_lse = ws_o + static_cast<size_t>(B) * Hq * splits * dec::kD;
  const float c = scale * kLog2e;
  const dim3 grid(splits, Hkv, B);
  if (chunk <= dtc::kMaxChunk && (pg == nullptr || pg->page_shift >= dtc::kMinTcPageShift)) {
    // chunks of at most kMaxChunk keys, contiguous or in pages of at least 64 keys: the
    // tensor-core split kernel
    int rc = configure_decode_tc(const_cast<DeviceInfo*>(info));
    if (rc != ATTN_OK) return rc;
    CUtensorMap tq, tk, tv;
    if (encode_map(&tq, q, B * Hq, 1, dtc::kN) != ATTN_OK) return ATTN_ERR_UNSUPPORTED;
    if (pg == nullptr) {
      if (encode_map(&tk, k, Nk, B * Hkv) != ATTN_OK || encode_map(&tv, v, Nk, B * Hkv) != ATTN_OK)
        return ATTN_ERR_UNSUPPORTED;
    } else {
      const long long rows = static_cast<long long>(pg->num_pages) << pg->page_shift;
      const uint32_t piece = (1u << pg->page_shift) < 32u ? (1u << pg->page_shift) : 32u;
      if (rows > 0x7fffffffLL || encode_map_packed(&tk, k, static_cast<int>(rows), Hkv, piece) != ATTN_OK ||
          encode_map_packed(&tv, v, static_cast<int>(rows), Hkv, piece) != ATTN_OK)
        return ATTN_ERR_UNSUPPORTED;
    }
    const dec::Paged pgv = pg != nullptr ? *pg : dec::Paged{};
    const bool paged = pg != nullptr;
#define ATTN_LAUNCH_DTC(GG)                                                                      \
  do {                                                                                           \
    if (paged)                                                                                   \
      dtc::decode_tc_kernel<GG, true><<<grid, dtc::kThreads, dtc::kSmemBytes, st>>>(             \
          tq, tk, tv, ws_o, ws_lse, Hq, Hkv, Nk, chunk, splits, c, pgv);                         \
    else                                                                                         \
      dtc::decode_tc_kernel<GG, false><<<grid, dtc::kThreads, dtc::kSmemBytes, st>>>(            \
          tq, tk, tv, ws_o, ws_lse, Hq, Hkv, Nk, chunk, splits, c, pgv);                         \
  } while (0)
    switch (G) {
      case 1: ATTN_LAUNCH_DTC(1); break;
      case 2: ATTN_LAUNCH_DTC(2); break;
      case 4: ATTN_LAUNCH_DTC(4); break;
      default: ATTN_LAUNCH_DTC(8); break;
    }
#undef ATTN_LAUNCH_DTC
    rc = cuda_status(cudaGetLastError());
    if (rc != ATTN_OK) return rc;
    dec::decode_combine_kernel<<<B * Hq, dec::kD, 0, st>>>(
        ws_o, ws_lse, static_cast<__nv_bfloat16*>(o), lse, splits);
    return cuda_status(cudaGetLastError());
  }
  const auto* qb = static_cast<const __nv_bfloat16*>(q);
  const auto* kb = static_cast<const __nv_bfloat16*>(k);
  const auto* vb = static_cast<const __nv_bfloat16*>(v);
  switch (G) {
    case 1: launch_decode_split<1>(grid, chunk, st, qb, kb, vb, ws_o, ws_lse, Hq, Hkv, Nk, splits, c, pg); break;
    case 2: launch_decode_split<2>(grid, chunk, st, qb, kb, vb, ws_o, ws_lse, Hq, Hkv, Nk, splits, c, pg); break;
    case 4: launch_decode_split<4>(grid, chunk, st, qb, kb, vb, ws_o, ws_lse, Hq, Hkv, Nk, splits, c, pg); break;
    default: launch_decode_split<8>(grid, chunk, st, qb, kb, vb, ws_o, ws_lse, Hq, Hkv, Nk, splits, c, pg); break;
  }
  int rc = cuda_status(cudaGetLastError());
  if (rc != ATTN_OK) return rc;
  dec::decode_combine_kernel<<<B * Hq, dec::kD, 0, st>>>(ws_o, ws_lse,
                                                         static_cast<__nv_bfloat16*>(o), lse, splits);
  return cuda_status(cudaGetLastError());
}

__global__ void timeout_probe_kernel(long long limit) {
  __shared__ uint64_t bar;
  __shared__ int abort_flag;
  if (threadIdx.x == 0) {
    dev::mbar_init(dev::smem_u32(&bar), 1);
    abort_flag = 0;
    dev::fence_barrier_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) wait_bounded(dev::smem_u32(&bar), 0, &abort_flag, limit);
  __syncthreads();
}

// The CTAs of a prefill launch.  With an even group size a CTA takes the same 128 rows of two
// query heads that read one kv head, so its two query tiles see the same keys and every key
// tile feeds both; otherwise a CTA takes 256 consecutive rows of one head.
struct FwdSchedule {
  int head_pair, num_qblocks;
  long long units;
};

FwdSchedule fwd_schedule(int batch, int Hq, int Hkv, int rows) {
  FwdSchedule sc;
  sc.head_pair = (Hq / Hkv) % 2 == 0 ? 1 : 0;
  const int per_cta = sc.head_pair ? fwd::kBM : fwd::kRowsPerCta;
  sc.num_qblocks = (rows + per_cta - 1) / per_cta;
  sc.units = static_cast<long long>(sc.num_qblocks) * batch * (sc.head_pair ? Hq / 2 : Hq);
  return sc;
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" {

int attn_abi_version(void) { return 1; }

const char* attn_last_error_detail(void) { return g_last_detail; }

const char* attn_status_string(int status) {
  switch (status) {
    case ATTN_OK: return "ok";
    case ATTN_ERR_INVALID_ARG: return "invalid argument";
    case ATTN_ERR_UNSUPPORTED: return "unsupported configuration (head dim, group size, alignment or device)";
    case ATTN_ERR_CUDA: return "CUDA runtime error";
    case ATTN_ERR_WORKSPACE: return "decode workspace missing or too small";
    case ATTN_ERR_DEVICE_TIMEOUT: return "a bounded device-side wait expired";
    default: return "unknown status";
  }
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
             int Hkv, int Nq, int Nk, int d, int mask_kind, int window, int n_sink, float scale,
             attn_stream_t stream) {
  int rc = check_fwd_args(q, k, v, o, B, Hq, Hkv, Nq, Nk, mask_kind, window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  if (d != fwd::kD) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || Nq == 0) return ATTN_OK;
  if (Nk == 0)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse,
                             static_cast<size_t>(B) * Hq * Nq, d, st);
  const FwdSchedule sc = fwd_schedule(B, Hq, Hkv, Nq);
  if (sc.units > 0x7fffffffLL - 4096) return ATTN_ERR_UNSUPPORTED;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;

  CUtensorMap tq, tk, tv, to;
  if (encode_map(&tq, q, Nq, B * Hq) != ATTN_OK || encode_map(&tk, k, Nk, B * Hkv) != ATTN_OK ||
      encode_map(&tv, v, Nk, B * Hkv) != ATTN_OK || encode_map_out(&to, o, Nq, B * Hq, false) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  fwd::Params p{};
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.mask = make_mask(mask_kind, window, n_sink, Nk);
  // scale = 0 makes every visible weight equal; a tiny positive c gives exactly that (every
  // exp2 argument rounds to 0) while masked scores (-inf) still map to weight 0
  p.c = scale * kLog2e;
  if (p.c == 0.f) p.c = 1e-30f;
  p.num_qblocks = sc.num_qblocks;
  p.head_pair = sc.head_pair;
  p.units = static_cast<int>(sc.units);
  if ((rc = unit_counter(st, &p.unit_counter)) != ATTN_OK) return rc;
  p.front_heavy = (mask_kind == ATTN_MASK_LOCAL_GLOBAL && n_sink > 0) ? 1 : 0;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cu_q = nullptr;
  p.cu_k = nullptr;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(sc.units, info->num_sms)));
  if (scale < 0.f)
    fwd::fwd_bf16_sm100_kernel<true, false><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  else
    fwd::fwd_bf16_sm100_kernel<false, false><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  return cuda_status(cudaGetLastError());
}

int attn_fwd_block_sparse(const void* q, const void* k, const void* v, void* o, float* lse,
                          const uint8_t* block_mask, int mask_heads, int B, int Hq, int Hkv,
                          int Nq, int Nk, int d, int mask_kind, int window, int n_sink,
                          float scale, attn_stream_t stream) {
  int rc = check_fwd_args(q, k, v, o, B, Hq, Hkv, Nq, Nk, mask_kind, window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  if (mask_heads != 1 && mask_heads != Hq) return ATTN_ERR_INVALID_ARG;
  if (B > 0 && Nq > 0 && Nk > 0 && block_mask == nullptr) return ATTN_ERR_INVALID_ARG;
  if (d != fwd::kD) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_UNSUPPORTED;
  const int mask_qtiles = (Nq + fwd::kBM - 1) / fwd::kBM, mask_ktiles = (Nk + fwd::kBN - 1) / fwd::kBN;
  if (mask_ktiles > fwd::kMaxSparseTiles) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || Nq == 0) return ATTN_OK;
  if (Nk == 0)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse,
                             static_cast<size_t>(B) * Hq * Nq, d, st);
  const FwdSchedule sc = fwd_schedule(B, Hq, Hkv, Nq);
  if (sc.units > 0x7fffffffLL - 4096) return ATTN_ERR_UNSUPPORTED;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;
  CUtensorMap tq, tk, tv, to;
  if (encode_map(&tq, q, Nq, B * Hq) != ATTN_OK || encode_map(&tk, k, Nk, B * Hkv) != ATTN_OK ||
      encode_map(&tv, v, Nk, B * Hkv) != ATTN_OK || encode_map_out(&to, o, Nq, B * Hq, false) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  fwd::Params p{};
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.mask = make_mask(mask_kind, window, n_sink, Nk);
  p.c = scale * kLog2e;
  if (p.c == 0.f) p.c = 1e-30f;
  p.num_qblocks = sc.num_qblocks;
  p.head_pair = sc.head_pair;
  p.units = static_cast<int>(sc.units);
  if ((rc = unit_counter(st, &p.unit_counter)) != ATTN_OK) return rc;
  p.front_heavy = (mask_kind == ATTN_MASK_FULL || mask_kind == ATTN_MASK_LOCAL_GLOBAL) ? 1 : 0;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.block_mask = block_mask;
  p.mask_heads = mask_heads;
  p.mask_qtiles = mask_qtiles;
  p.mask_ktiles = mask_ktiles;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(sc.units, info->num_sms)));
  if (scale < 0.f)
    fwd::fwd_bf16_sparse_sm100_kernel<true><<<grid, fwd::kThreads, fwd::kSmemBytesSparse, st>>>(tq, tk, tv, to, p);
  else
    fwd::fwd_bf16_sparse_sm100_kernel<false><<<grid, fwd::kThreads, fwd::kSmemBytesSparse, st>>>(tq, tk, tv, to, p);
  return cuda_status(cudaGetLastError());
}

int attn_fwd_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                    const int* cu_seqlens_q, const int* cu_seqlens_k, int num_seqs, int Hq,
                    int Hkv, int total_q, int total_k, int max_seqlen_q, int d, int mask_kind,
                    int window, int n_sink, float scale, attn_stream_t stream) {
  if (num_seqs < 0 || total_q < 0 || total_k < 0 || max_seqlen_q < 0) return ATTN_ERR_INVALID_ARG;
  if (num_seqs > 0 && (cu_seqlens_q == nullptr || cu_seqlens_k == nullptr)) return ATTN_ERR_INVALID_ARG;
  // the packed tensors play the role of one batch row each for the common checks
  int rc = check_fwd_args(q, k, v, o, num_seqs > 0 ? 1 : 0, Hq, Hkv, total_q, total_k, mask_kind,
                          window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  if (d != fwd::kD) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens_q) & 3u) || (reinterpret_cast<uintptr_t>(cu_seqlens_k) & 3u))
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return ATTN_OK;
  if (total_k == 0)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse, static_cast<size_t>(total_q) * Hq, d, st);
  const FwdSchedule sc = fwd_schedule(num_seqs, Hq, Hkv, max_seqlen_q);
  if (sc.units > 0x7fffffffLL - 4096) return ATTN_ERR_UNSUPPORTED;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;
  CUtensorMap tq, tk, tv, to;
  if (encode_map_packed(&tq, q, total_q, Hq) != ATTN_OK || encode_map_packed(&tk, k, total_k, Hkv) != ATTN_OK ||
      encode_map_packed(&tv, v, total_k, Hkv) != ATTN_OK ||
      encode_map_out(&to, o, total_q, Hq, true) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  fwd::Params p{};
  p.B = num_seqs;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = total_q;
  p.Nk = total_k;
  p.G = Hq / Hkv;
  p.mask = make_mask(mask_kind, window, n_sink, total_k);
  p.c = scale * kLog2e;
  if (p.c == 0.f) p.c = 1e-30f;
  p.num_qblocks = sc.num_qblocks;
  p.head_pair = sc.head_pair;
  p.units = static_cast<int>(sc.units);
  if ((rc = unit_counter(st, &p.unit_counter)) != ATTN_OK) return rc;
  p.front_heavy = (mask_kind == ATTN_MASK_LOCAL_GLOBAL && n_sink > 0) ? 1 : 0;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(sc.units, info->num_sms)));
  if (scale < 0.f)
    fwd::fwd_bf16_sm100_kernel<true, true><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  else
    fwd::fwd_bf16_sm100_kernel<false, true><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  return cuda_status(cudaGetLastError());
}

int attn_fwd_fp8(const void* q, const void* k, const void* v, void* o, float* lse,
                 const float* descale_q, const float* descale_k, const float* descale_v, int B,
                 int Hq, int Hkv, int Nq, int Nk, int d, int mask_kind, int window, int n_sink,
                 float scale, attn_stream_t stream) {
  int rc = check_fwd_args(q, k, v, o, B, Hq, Hkv, Nq, Nk, mask_kind, window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  const bool q_empty = B == 0 || Nq == 0, kv_empty = B == 0 || Nk == 0;
  if (!q_empty && (descale_q == nullptr || (!kv_empty && (descale_k == nullptr ||
                                                          descale_v == nullptr))))
    return ATTN_ERR_INVALID_ARG;
  if (d != fwd::kD) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (q_empty) return ATTN_OK;
  if (Nk == 0)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse, static_cast<size_t>(B) * Hq * Nq, d, st);
  const FwdSchedule sc = fwd_schedule(B, Hq, Hkv, Nq);
  if (sc.units > 0x7fffffffLL - 4096) return ATTN_ERR_UNSUPPORTED;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;
  CUtensorMap tq, tk, tv, to;
  if (encode_map_e4m3(&tq, q, Nq, B * Hq) != ATTN_OK || encode_map_e4m3(&tk, k, Nk, B * Hkv) != ATTN_OK ||
      encode_map_e4m3(&tv, v, Nk, B * Hkv) != ATTN_OK || encode_map_out(&to, o, Nq, B * Hq, false) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  fwd::Params p{};
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.mask = make_mask(mask_kind, window, n_sink, Nk);
  p.c = scale * kLog2e;
  if (p.c == 0.f) p.c = 1e-30f;
  p.num_qblocks = sc.num_qblocks;
  p.head_pair = sc.head_pair;
  p.units = static_cast<int>(sc.units);
  if ((rc = unit_counter(st, &p.unit_counter)) != ATTN_OK) return rc;
  p.front_heavy = (mask_kind == ATTN_MASK_LOCAL_GLOBAL && n_sink > 0) ? 1 : 0;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cu_q = nullptr;
  p.cu_k = nullptr;
  p.descale_q = descale_q;
  p.descale_k = descale_k;
  p.descale_v = descale_v;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(sc.units, info->num_sms)));
  if (scale < 0.f)
    fwd::fwd_fp8_sm100_kernel<true><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  else
    fwd::fwd_fp8_sm100_kernel<false><<<grid, fwd::kThreads, fwd::kSmemBytes, st>>>(tq, tk, tv, to, p);
  return cuda_status(cudaGetLastError());
}

int attn_fwd_f32(const float* q, const float* k, const float* v, float* o, float* lse, int B,
                 int Hq, int Hkv, int Nq, int Nk, int d, int mask_kind, int window, int n_sink,
                 float scale, attn_stream_t stream) {
  int rc = check_fwd_args(q, k, v, o, B, Hq, Hkv, Nq, Nk, mask_kind, window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0 || Nq == 0) return ATTN_OK;
  if (Nk == 0) return launch_fill_empty(o, lse, static_cast<size_t>(B) * Hq * Nq, d, st);
  if (Hq > 65535 || B > 65535) return ATTN_ERR_UNSUPPORTED;
  f32::Params p;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.mask = make_mask(mask_kind, window, n_sink, Nk);
  p.c = scale * kLog2e;
  // the kv head's whole K and V in shared memory (at most 512 keys, about 200 KB): one warp per
  // query row; otherwise the tiled kernel
  const size_t small_bytes = d == 64 ? f32::small_smem_bytes<64>(Nk) : f32::small_smem_bytes<128>(Nk);
  if (Nk <= 32 * f32::kSmallMaxChunks && small_bytes <= 200 * 1024) {
    const dim3 grid((Nq + f32::kSmallWarps - 1) / f32::kSmallWarps, Hq, B);
    if (d == 64) {
      rc = cuda_status(cudaFuncSetAttribute(f32::fwd_f32_small_kernel<64>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(small_bytes)));
      if (rc != ATTN_OK) return rc;
      f32::fwd_f32_small_kernel<64><<<grid, f32::kSmallWarps * 32, small_bytes, st>>>(q, k, v, o, lse, p);
    } else {
      rc = cuda_status(cudaFuncSetAttribute(f32::fwd_f32_small_kernel<128>,
                                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(small_bytes)));
      if (rc != ATTN_OK) return rc;
      f32::fwd_f32_small_kernel<128><<<grid, f32::kSmallWarps * 32, small_bytes, st>>>(q, k, v, o, lse, p);
    }
    return cuda_status(cudaGetLastError());
  }
  if (d == 64) {
    dim3 grid((Nq + f32::rows_per_cta<64>() - 1) / f32::rows_per_cta<64>(), Hq, B);
    f32::fwd_f32_kernel<64><<<grid, f32::kWarps * 32, 0, st>>>(q, k, v, o, lse, p);
  } else {
    dim3 grid((Nq + f32::rows_per_cta<128>() - 1) / f32::rows_per_cta<128>(), Hq, B);
    f32::fwd_f32_kernel<128><<<grid, f32::kWarps * 32, 0, st>>>(q, k, v, o, lse, p);
  }
  return cuda_status(cudaGetLastError());
}

int attn_decode_num_splits(int B, int Hq, int Hkv, int Nk, int d) {
  (void)d;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nk < 0) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* info = nullptr;
  const int num_sms = current_device(&info) == ATTN_OK ? info->num_sms : 148;
  return decode_splits(B, Hkv, Nk, Hq / Hkv, 0, num_sms);
}

size_t attn_decode_workspace_bytes(int B, int Hq, int Hkv, int Nk, int d, int num_splits) {
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || Nk < 0 || d != dec::kD) return 0;
  DeviceInfo* info = nullptr;
  const int num_sms = current_device(&info) == ATTN_OK ? info->num_sms : 148;
  const int splits = decode_splits(B, Hkv, Nk, Hq / Hkv, num_splits, num_sms);
  return decode_ws_bytes(B, Hq, splits);
}

int attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                int Hkv, int Nk, int d, float scale, int num_splits, void* workspace,
                size_t workspace_bytes, attn_stream_t stream) {
  if (B < 0 || Nk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (B > 0 && (q == nullptr || o == nullptr || (Nk > 0 && (k == nullptr || v == nullptr))))
    return ATTN_ERR_INVALID_ARG;
  if (num_splits < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  if (d != dec::kD) return ATTN_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  int rc = current_device(&info);
  if (rc != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return ATTN_OK;
  if (Nk == 0)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse, static_cast<size_t>(B) * Hq, d, st);
  if (B > 65535 || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  return decode_run(q, k, v, o, lse, B, Hq, Hkv, Nk, scale, num_splits, workspace,
                    workspace_bytes, st, info, nullptr);
}

int attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, void* o,
                      float* lse, const int* block_table, const int* seq_lens, int B, int Hq,
                      int Hkv, int num_pages, int page_size, int max_pages_per_seq,
                      int max_seq_len, int d, float scale, int num_splits, void* workspace,
                      size_t workspace_bytes, attn_stream_t stream) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_pages < 0 || max_pages_per_seq < 0 ||
      max_seq_len < 0)
    return ATTN_ERR_INVALID_ARG;
  if (page_size < dec::kMinPageSize || page_size > (1 << 20) || (page_size & (page_size - 1)) != 0)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(max_seq_len) > static_cast<long long>(max_pages_per_seq) * page_size)
    return ATTN_ERR_INVALID_ARG;
  if (num_splits < 0 || !std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  const bool any_keys = max_seq_len > 0 && num_pages > 0;
  if (B > 0 && (q == nullptr || o == nullptr || seq_lens == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (B > 0 && any_keys && (k_cache == nullptr || v_cache == nullptr || block_table == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (d != dec::kD) return ATTN_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o))
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  int rc = current_device(&info);
  if (rc != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return ATTN_OK;
  if (!any_keys)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse, static_cast<size_t>(B) * Hq, d, st);
  if (B > 65535 || Hkv > 65535) return ATTN_ERR_UNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < page_size) ++shift;
  const dec::Paged pg{block_table, seq_lens, max_pages_per_seq, num_pages, shift};
  return decode_run(q, k_cache, v_cache, o, lse, B, Hq, Hkv, max_seq_len, scale, num_splits,
                    workspace, workspace_bytes, st, info, &pg);
}

size_t attn_bwd_workspace_bytes(int B, int Hq, int Nq, int Nk, int mask_kind, int window,
                                int n_sink) {
  if (B < 1 || Hq < 1 || Nq < 0 || Nk < 0) return 0;
  if (mask_kind < ATTN_MASK_FULL || mask_kind > ATTN_MASK_LOCAL_GLOBAL || n_sink < 0 ||
      (mask_kind == ATTN_MASK_SLIDING && window < 1) ||
      (mask_kind == ATTN_MASK_LOCAL_GLOBAL && window < 0))
    return 0;
  return bwd_layout(B, Hq, Nq, Nk, make_mask(mask_kind, window, n_sink, Nk)).total;
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse,
             const void* dout, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Nq,
             int Nk, int d, int mask_kind, int window, int n_sink, float scale, void* workspace,
             size_t workspace_bytes, attn_stream_t stream) {
  int rc = check_fwd_args(q, k, v, o, B, Hq, Hkv, Nq, Nk, mask_kind, window, n_sink, scale);
  if (rc != ATTN_OK) return rc;
  const bool q_empty = B == 0 || Nq == 0, kv_empty = B == 0 || Nk == 0;
  if (!q_empty && (lse == nullptr || dout == nullptr || dq == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!kv_empty && (dk == nullptr || dv == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (d != bwd::kD) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dout) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return ATTN_OK;
  const size_t q_bytes = static_cast<size_t>(B) * Hq * Nq * d * 2;
  const size_t kv_bytes = static_cast<size_t>(B) * Hkv * Nk * d * 2;
  // no query: every key gets zero gradients; no key: every query does
  if (Nq == 0 || Nk == 0) {
    if (Nq == 0 && Nk > 0) {
      if ((rc = cuda_status(cudaMemsetAsync(dk, 0, kv_bytes, st))) != ATTN_OK) return rc;
      return cuda_status(cudaMemsetAsync(dv, 0, kv_bytes, st));
    }
    if (Nq > 0) return cuda_status(cudaMemsetAsync(dq, 0, q_bytes, st));
    return ATTN_OK;
  }
  const int nqt = (Nq + bwd::kT - 1) / bwd::kT, nkb = (Nk + bwd::kT - 1) / bwd::kT;
  const long long units_q = static_cast<long long>((nqt + 1) / 2) * B * Hq;  // query-tile pairs
  const long long units_kv = static_cast<long long>(nkb) * B * Hkv;
  if (units_q > 0x7fffffffLL - 4096 || units_kv > 0x7fffffffLL - 4096) return ATTN_ERR_UNSUPPORTED;
  const MaskSpec mask = make_mask(mask_kind, window, n_sink, Nk);
  const BwdLayout L = bwd_layout(B, Hq, Nq, Nk, mask);
  if (static_cast<double>(B) * Hq * static_cast<double>(L.pairs) > 2147483647.0)
    return ATTN_ERR_UNSUPPORTED;  // dS block index of the dQ kernel's tensor map
  if (workspace == nullptr || workspace_bytes < L.total || !aligned16(workspace))
    return ATTN_ERR_WORKSPACE;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;  // the tensor-map encoder
  if ((rc = configure_bwd(info)) != ATTN_OK) return rc;
  CUtensorMap tq, tk, tv, tdo;
  if (encode_map(&tq, q, Nq, B * Hq) != ATTN_OK || encode_map(&tk, k, Nk, B * Hkv) != ATTN_OK ||
      encode_map(&tv, v, Nk, B * Hkv) != ATTN_OK || encode_map(&tdo, dout, Nq, B * Hq) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  bwd::Params p;
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.Nq = Nq;
  p.Nk = Nk;
  p.G = Hq / Hkv;
  p.mask = mask;
  p.scale = scale;
  p.c = scale * kLog2e;
  p.num_kblocks = nkb;
  p.num_qtiles = nqt;
  p.npad = nqt * bwd::kT;
  float* lse2 = static_cast<float*>(workspace);
  float* dsum = lse2 + static_cast<size_t>(B) * Hq * p.npad;
  p.lse2 = lse2;
  p.dsum = dsum;
  p.dq = static_cast<__nv_bfloat16*>(dq);
  p.dk = static_cast<__nv_bfloat16*>(dk);
  p.dv = static_cast<__nv_bfloat16*>(dv);
  p.ds_off = reinterpret_cast<int*>(dsum + static_cast<size_t>(B) * Hq * p.npad);
  p.ds = reinterpret_cast<__nv_bfloat16*>(static_cast<uint8_t*>(workspace) + L.ds_offset);
  p.ds_pairs = static_cast<long long>(L.pairs);
  if ((rc = unit_counter(st, &p.unit_counter)) != ATTN_OK) return rc;
  // dS^T blocks as a 3-D tensor (queries, keys, block) for the dQ kernel's TMA loads
  CUtensorMap tds;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(bwd::kT), static_cast<cuuint64_t>(bwd::kT),
                                static_cast<cuuint64_t>(B) * Hq * (L.pairs > 0 ? L.pairs : 1)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(bwd::kT) * 2,
                                   static_cast<cuuint64_t>(bwd::kT) * bwd::kT * 2};
    const cuuint32_t box[3] = {64, 128, 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    if (g_encode(&tds, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.ds, dims, strides, box, estride,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ATTN_ERR_UNSUPPORTED;
  }
  // the same blocks as the dK/dV kernel writes them: boxes of 32 queries x 32 keys, one per row
  // warp and sub-step, staged with the 64-byte swizzle
  CUtensorMap tds_out;
  {
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(bwd::kT), static_cast<cuuint64_t>(bwd::kT),
                                static_cast<cuuint64_t>(B) * Hq * (L.pairs > 0 ? L.pairs : 1)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(bwd::kT) * 2,
                                   static_cast<cuuint64_t>(bwd::kT) * bwd::kT * 2};
    const cuuint32_t box[3] = {32, 32, 1};
    const cuuint32_t estride[3] = {1, 1, 1};
    if (g_encode(&tds_out, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.ds, dims, strides, box, estride,
                 CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_64B,
                 CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return ATTN_ERR_UNSUPPORTED;
  }
  // dQ, dK and dV as boxes of 32 columns x 32 rows staged with the 64-byte swizzle
  CUtensorMap tdq, tdk, tdv;
  if (encode_map_out(&tdq, dq, Nq, B * Hq, false) != ATTN_OK ||
      encode_map_out(&tdk, dk, Nk, B * Hkv, false) != ATTN_OK ||
      encode_map_out(&tdv, dv, Nk, B * Hkv, false) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  const long long prow = static_cast<long long>(B) * Hq * p.npad;
  // one wave (4 blocks of 8 warps per SM at 64 registers a thread), grid-stride over the row groups
  const long long prep_blocks = std::min<long long>((prow + bwd::kPrepRowsPerBlock - 1) /
                                                        bwd::kPrepRowsPerBlock,
                                                    4LL * info->num_sms);
  bwd::bwd_prep_kernel<<<static_cast<unsigned>(prep_blocks), 256, 0, st>>>(
      static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(dout), lse, lse2,
      dsum, Nq, p.npad, prow, mask, nkb, p.ds_off);
  if ((rc = cuda_status(cudaGetLastError())) != ATTN_OK) return rc;
  // persistent: one CTA per SM walking the key-block units
  bwd::bwd_dkdv_kernel<<<static_cast<unsigned>(std::min<long long>(units_kv, info->num_sms)),
                         bwd::kThreads, bwd::kSmemKVBytes, st>>>(tq, tk, tv, tdo, tds_out, tdk,
                                                                 tdv, p);
  if ((rc = cuda_status(cudaGetLastError())) != ATTN_OK) return rc;
  bwd::bwd_dq_kernel<<<static_cast<unsigned>(std::min<long long>(units_q, info->num_sms)),
                       bwd::kThreads, bwd::kSmemQBytes, st>>>(tds, tk, tdq, p);
  return cuda_status(cudaGetLastError());
}

int attn_get_device_error(attn_stream_t stream) {
  int rc = cuda_status(cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream)));
  if (rc != ATTN_OK) return rc;
  int flag = 0;
  if ((rc = cuda_status(cudaMemcpyFromSymbol(&flag, g_device_error, sizeof(int)))) != ATTN_OK)
    return rc;
  if (flag != 0) {
    const int zero = 0;
    if ((rc = cuda_status(cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)))) != ATTN_OK)
      return rc;
    return flag;
  }
  return ATTN_OK;
}

int attn_debug_timeout_probe(long long limit_cycles, attn_stream_t stream) {
  if (limit_cycles < 1 || limit_cycles > (1ll << 34)) return ATTN_ERR_INVALID_ARG;
  DeviceInfo* info = nullptr;
  int rc = current_device(&info);
  if (rc != ATTN_OK) return rc;
  timeout_probe_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(limit_cycles);
  return cuda_status(cudaGetLastError());
}

}  // extern "C"

// ------------------------------------------------------------------------------------------
// Decode without allocation: the same split-K decode, with its partial results kept in a
// fixed array that the library owns instead of a caller-provided workspace.
// ------------------------------------------------------------------------------------------
namespace attn {
namespace {

// Every GPU that loads this library holds this array until the process exits.
static __device__ __align__(256) unsigned char g_noalloc_scratch[ATTN_DECODE_NOALLOC_MAX_BYTES];

void* g_noalloc_ptr[kMaxDevices] = {};

// Device address of g_noalloc_scratch on the current device, looked up once per device (in
// host code the array's name is only a host-side stand-in, never a device address).  The
// address is kept for the process's life: the header rules out use across a device reset.
int noalloc_scratch(void** out) {
  int dev = 0;
  int rc = cuda_status(cudaGetDevice(&dev));
  if (rc != ATTN_OK) return rc;
  if (dev < 0 || dev >= kMaxDevices) return ATTN_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_noalloc_ptr[dev] == nullptr) {
    void* p = nullptr;
    rc = cuda_status(cudaGetSymbolAddress(&p, g_noalloc_scratch));
    if (rc != ATTN_OK) return rc;
    g_noalloc_ptr[dev] = p;
  }
  *out = g_noalloc_ptr[dev];
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" int attn_decode_noalloc(const void* q, const void* k, const void* v, void* o,
                                   float* lse, int B, int Hq, int Hkv, int Nk, int d,
                                   float scale, int num_splits, attn_stream_t stream) {
  // same argument rules as attn_decode; the scratch size is checked before anything runs
  if (B < 0 || Nk < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATTN_ERR_INVALID_ARG;
  if (num_splits < 0) return ATTN_ERR_INVALID_ARG;
  if (d != dec::kD) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  int rc = current_device(&info);
  if (rc != ATTN_OK) return rc;
  const int G = Hq / Hkv;
  if (G != 1 && G != 2 && G != 4 && G != 8) return ATTN_ERR_UNSUPPORTED;
  if (B > 0 && Nk > 0) {
    const int splits = decode_splits(B, Hkv, Nk, G, num_splits, info->num_sms);
    if (decode_ws_bytes(B, Hq, splits) > ATTN_DECODE_NOALLOC_MAX_BYTES) return ATTN_ERR_WORKSPACE;
  }
  void* scratch = nullptr;
  if ((rc = noalloc_scratch(&scratch)) != ATTN_OK) return rc;
  return attn_decode(q, k, v, o, lse, B, Hq, Hkv, Nk, d, scale, num_splits, scratch,
                     ATTN_DECODE_NOALLOC_MAX_BYTES, stream);
}

// ------------------------------------------------------------------------------------------
// Around attention: queries and keys on their way to it, the paged cache's bookkeeping, and decode
// behind shared prefixes.
// ------------------------------------------------------------------------------------------
namespace attn {
namespace {

// A [B][H][N][d] view: 16-byte rows for the vector loads (strides of single entries do not count).
bool view_ok(const void* base, const long long* st, int B, int H, int N, int size) {
  const long long mask = 16 / size - 1;
  return aligned16(base) && (B <= 1 || (st[0] & mask) == 0) && (H <= 1 || (st[1] & mask) == 0) &&
         (N <= 1 || (st[2] & mask) == 0);
}

qkn::View make_view(const long long* st) { return qkn::View{st[1], st[2]}; }  // (b, h, n) of a packed view

// Argument rules shared by the norm + rotation calls; fills what they share of the parameters.
int qkn_common(qkn::Params& p, const void* q_weight, const void* k_weight, const float* rope,
               const int* positions, const int* sections, int dtype, int B, int N, int Hq, int Hkv,
               int d, int rot_dim, int max_pos, int num_axes, float eps) {
  if (B < 0 || N < 0 || Hq < 1 || Hkv < 1) return ATTN_ERR_INVALID_ARG;
  if (dtype != ATTN_DTYPE_BF16 && dtype != ATTN_DTYPE_F32) return ATTN_ERR_INVALID_ARG;
  if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0 || max_pos < 0) return ATTN_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > qkn::kMaxAxes) return ATTN_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return ATTN_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return ATTN_ERR_UNSUPPORTED;
  const bool empty = B == 0 || N == 0;
  if (rot_dim > 0 && !empty && (rope == nullptr || positions == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (!aligned16(rope) || !aligned16(q_weight) || !aligned16(k_weight)) return ATTN_ERR_UNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return ATTN_ERR_UNSUPPORTED;
  if (static_cast<long long>(B) * N > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  int at = 0;
  for (int a = 0; a < num_axes; ++a) {
    if (num_axes > 1) {
      if (sections == nullptr || sections[a] < 0 || sections[a] > rot_dim / 2 - at) return ATTN_ERR_INVALID_ARG;
      at += sections[a];
    } else {
      at = rot_dim / 2;
    }
    p.end[a] = at;
  }
  if (at != rot_dim / 2) return ATTN_ERR_INVALID_ARG;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.rope = rope;
  p.pos = positions;
  p.axes = num_axes;
  p.rot = rot_dim;
  p.max_pos = max_pos;
  p.B = B;
  p.N = N;
  p.H[0] = Hq;
  p.H[1] = Hkv;
  p.eps = eps;
  return ATTN_OK;
}

// One token of a [B][H][1][d] call per batch row: the same as one row of B tokens, which fills tiles.
void qkn_flatten(qkn::Params& p, long long* st, int views, const long long* strides) {
  std::copy(strides, strides + 3 * views + 2, st);
  p.pos_axis = st[3 * views];
  p.pos_b = st[3 * views + 1];
  if (p.N != 1 || p.B <= 1 || p.pos_b != 1) return;
  for (int v = 0; v < views; ++v) st[3 * v + 2] = st[3 * v];
  p.N = p.B;
  p.B = 1;
}

// [B][H][N][d] view as (d, H, N, B), in tiles of kTokens tokens x `heads` heads.
int encode_map_heads(CUtensorMap* map, const void* base, const long long* st, int B, int H, int N, int d,
                     int dtype, int heads) {
  const int size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N),
                              static_cast<cuuint64_t>(B)};
  // the stride of a dimension of one entry does not count (and may be anything)
  const cuuint64_t strides[3] = {H > 1 ? static_cast<cuuint64_t>(st[1]) * size : 16u,
                                 N > 1 ? static_cast<cuuint64_t>(st[2]) * size : 16u,
                                 B > 1 ? static_cast<cuuint64_t>(st[0]) * size : 16u};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(d), static_cast<cuuint32_t>(heads), qkn::kTokens, 1};
  const cuuint32_t estride[4] = {1, 1, 1, 1};
  CUresult r = g_encode(map, dtype == ATTN_DTYPE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                        4, const_cast<void*>(base), dims, strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

// Blocks of a tiled call: a whole number for each group of heads (a block's tiles all have the same heads),
// every tile of its own up to `most` blocks.
int qkn_tile_blocks(const qkn::Params& p, int heads, int most, int* chunks, int* cq, unsigned* blocks) {
  *cq = (p.H[0] + heads - 1) / heads;
  const long long ch = *cq + static_cast<long long>((p.H[1] + heads - 1) / heads);
  if (ch > most) return ATTN_ERR_UNSUPPORTED;  // more groups of heads than blocks
  const long long runs = static_cast<long long>(p.B) * ((p.N + qkn::kTokens - 1) / qkn::kTokens);
  *chunks = static_cast<int>(ch);
  *blocks = static_cast<unsigned>(ch * std::min<long long>(runs, most / ch));
  return ATTN_OK;
}

constexpr int kQknBwdBlocks = 148 * qkn::kTileBlocksBwd;  // and rows of partial weight gradients

// kernel KERNEL<type, d, interleaved, rot_dim == d, several axes> for a call
#define ATTN_QKN_PICK_D(KERNEL, T, D)                                                        \
  (full ? (multi ? (inter ? KERNEL<T, D, true, true, true> : KERNEL<T, D, false, true, true>)  \
                 : (inter ? KERNEL<T, D, true, true, false> : KERNEL<T, D, false, true, false>)) \
        : (multi ? (inter ? KERNEL<T, D, true, false, true> : KERNEL<T, D, false, false, true>)  \
                 : (inter ? KERNEL<T, D, true, false, false> : KERNEL<T, D, false, false, false>)))
#define ATTN_QKN_PICK(KERNEL)                                                                \
  (dtype == ATTN_DTYPE_BF16                                                                  \
       ? (d == 128 ? ATTN_QKN_PICK_D(KERNEL, __nv_bfloat16, 128) : ATTN_QKN_PICK_D(KERNEL, __nv_bfloat16, 64)) \
       : (d == 128 ? ATTN_QKN_PICK_D(KERNEL, float, 128) : ATTN_QKN_PICK_D(KERNEL, float, 64)))

// Launch with the next kernel of the stream allowed to start early: that kernel waits for this one's
// results by itself (griddepcontrol.wait).
template <typename... A>
int launch_early(void (*kern)(A...), dim3 blocks, unsigned threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kern, args...));
}

bool page_size_ok(int page_size) {
  return page_size >= 8 && page_size <= (1 << 20) && (page_size & (page_size - 1)) == 0;
}
int log2_int(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// Decode behind shared prefixes: one CTA per SM of a B200, and the workspace is sized for that.
constexpr int kPfxCtas = 148;

struct PfxLayout {
  long long thin_row0, own_row0, rows;
  size_t lse_offset, plan_offset, total;
};

PfxLayout pfx_layout(int B, int Hq, int Hkv, int num_groups) {
  PfxLayout L{};
  const int G = Hq / Hkv;
  L.thin_row0 = 2ll * B * Hq + static_cast<long long>(kPfxCtas) * pfx::kWideCtaRows;
  L.own_row0 = L.thin_row0 + 2ll * B * Hq + static_cast<long long>(kPfxCtas) * pfx::kThinCtaRows;
  L.rows = L.own_row0 + 2ll * B * Hq + 2ll * G * kPfxCtas;
  L.lse_offset = static_cast<size_t>(L.rows) * pfx::kD * sizeof(float);
  L.plan_offset = (L.lse_offset + static_cast<size_t>(L.rows) * sizeof(float) + 15) & ~size_t(15);
  L.total = L.plan_offset + (4 + 2 * static_cast<size_t>(num_groups) + B) * sizeof(int);
  return L;
}

// Shapes that the prefix decode takes (the lines of steps are counted in 32 bits).
int pfx_shapes(int B, int Hq, int Hkv, int num_groups, int max_prefix_len, int max_seq_len, int d) {
  if (B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || num_groups < 0 || max_prefix_len < 0 || max_seq_len < 0)
    return ATTN_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  if (d != pfx::kD || (G != 1 && G != 2 && G != 4 && G != 8)) return ATTN_ERR_UNSUPPORTED;
  // the kernels look up to two tiles past a length
  if (max_prefix_len > 0x7fffffff - 512 || max_seq_len > 0x7fffffff - 512) return ATTN_ERR_UNSUPPORTED;
  const double blocks = std::min<double>(B, B / (256 / G) + static_cast<double>(num_groups));
  const double cost = Hkv * (blocks * ((max_prefix_len / 128 + 1.0) * pfx::kCostBoth + pfx::kCostWideJob) +
                             static_cast<double>(B) * ((max_seq_len / 128 + 1.0) * pfx::kCostThinMax + pfx::kCostThinJob));
  // grid (Hkv, B) of the joining kernel, and its 16-byte units of partial rows in 32 bits
  if (B > 65535 || (6.0 * B * Hq + 148.0 * 512) * 32 > 2.0e9) return ATTN_ERR_UNSUPPORTED;
  return cost < 2.0e9 ? ATTN_OK : ATTN_ERR_UNSUPPORTED;
}

int configure_pfx(DeviceInfo* info) {
  int rc = configure_fwd(info);  // the tensor-map encoder
  if (rc != ATTN_OK) return rc;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (!info->pfx_configured) {
    for (auto* kern : {pfx::decode_prefix_kernel<false>, pfx::decode_prefix_kernel<true>}) {
      rc = cuda_status(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            static_cast<int>(pfx::kSmemBytes)));
      if (rc != ATTN_OK) return rc;
    }
    info->pfx_configured = true;
  }
  return ATTN_OK;
}

// [B][heads][128] queries of one token each, read as boxes of 64 columns x G heads x seqs sequences
int encode_map_decode_q(CUtensorMap* map, const void* base, int heads, int B, int G, int seqs) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(pfx::kD), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(B)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(pfx::kD) * 2,
                                 static_cast<cuuint64_t>(heads) * pfx::kD * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(seqs)};
  const cuuint32_t estride[3] = {1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims,
                        strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

// Page pool [rows][heads][128], rows a multiple of 8, as (64 columns, 8 rows, 2 column halves, groups of 8
// rows, heads), read as boxes of box_rows rows of one head, both halves (the tile layout of
// decode_prefix.cuh).  A group index past the last reads as zero.
int encode_map_pages(CUtensorMap* map, const void* base, int rows, int heads, uint32_t box_rows) {
  const cuuint64_t row = static_cast<cuuint64_t>(heads) * pfx::kD * 2;
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(rows) / 8, static_cast<cuuint64_t>(heads)};
  const cuuint64_t strides[4] = {row, 128, 8 * row, static_cast<cuuint64_t>(pfx::kD) * 2};
  const cuuint32_t box[5] = {64, 8, 2, box_rows / 8, 1};
  const cuuint32_t estride[5] = {1, 1, 1, 1, 1};
  CUresult r = g_encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(base), dims,
                        strides, box, estride, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn

extern "C" {

int attn_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, const void* q_weight,
                      const void* k_weight, const float* rope, const int* positions,
                      const long long* strides, const int* sections, int dtype, int B, int N, int Hq,
                      int Hkv, int d, int rot_dim, int max_pos, int num_axes, int interleaved,
                      float eps, attn_stream_t stream) {
  qkn::Params p{};
  int rc = qkn_common(p, q_weight, k_weight, rope, positions, sections, dtype, B, N, Hq, Hkv, d,
                      rot_dim, max_pos, num_axes, eps);
  if (rc != ATTN_OK) return rc;
  if (strides == nullptr) return ATTN_ERR_INVALID_ARG;
  const bool empty = B == 0 || N == 0;
  if (!empty && (q == nullptr || k == nullptr || q_out == nullptr || k_out == nullptr))
    return ATTN_ERR_INVALID_ARG;
  const int size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  if (!view_ok(q, strides, B, Hq, N, size) || !view_ok(k, strides + 3, B, Hkv, N, size) ||
      !view_ok(q_out, strides + 6, B, Hq, N, size) || !view_ok(k_out, strides + 9, B, Hkv, N, size))
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  if (empty) return ATTN_OK;
  if ((rc = configure_fwd(info)) != ATTN_OK) return rc;  // the tensor-map encoder
  long long st[14];
  qkn_flatten(p, st, 4, strides);
  const int heads = qkn::kUnroll * (512 / (d * size));
  int chunks = 0, cq = 0;
  unsigned blocks = 0;
  if ((rc = qkn_tile_blocks(p, heads, qkn::kTileBlocks * info->num_sms, &chunks, &cq, &blocks)) != ATTN_OK) return rc;
  CUtensorMap tq, tk, tqo, tko;
  if ((rc = encode_map_heads(&tq, q, st, p.B, Hq, p.N, d, dtype, heads)) != ATTN_OK ||
      (rc = encode_map_heads(&tk, k, st + 3, p.B, Hkv, p.N, d, dtype, heads)) != ATTN_OK ||
      (rc = encode_map_heads(&tqo, q_out, st + 6, p.B, Hq, p.N, d, dtype, heads)) != ATTN_OK ||
      (rc = encode_map_heads(&tko, k_out, st + 9, p.B, Hkv, p.N, d, dtype, heads)) != ATTN_OK)
    return rc;
  const bool full = rot_dim == d, multi = num_axes > 1, inter = interleaved != 0;
  auto* kern = ATTN_QKN_PICK(qkn::qk_norm_rope_kernel);
  kern<<<blocks, qkn::kTileThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(tq, tk, tqo, tko, p);
  return cuda_status(cudaGetLastError());
}

size_t attn_qk_norm_rope_bwd_workspace_bytes(int d) {
  return d == 64 || d == 128 ? static_cast<size_t>(kQknBwdBlocks) * d * sizeof(float) : 0;
}

int attn_qk_norm_rope_bwd(const void* q, const void* k, const void* dq_out, const void* dk_out,
                          void* dq, void* dk, const void* q_weight, const void* k_weight,
                          float* dq_weight, float* dk_weight, const float* rope,
                          const int* positions, const long long* strides, const int* sections,
                          int dtype, int B, int N, int Hq, int Hkv, int d, int rot_dim, int max_pos,
                          int num_axes, int interleaved, float eps, void* workspace,
                          size_t workspace_bytes, attn_stream_t stream) {
  qkn::Params p{};
  int rc = qkn_common(p, q_weight, k_weight, rope, positions, sections, dtype, B, N, Hq, Hkv, d,
                      rot_dim, max_pos, num_axes, eps);
  if (rc != ATTN_OK) return rc;
  if (strides == nullptr) return ATTN_ERR_INVALID_ARG;
  const bool empty = B == 0 || N == 0;
  if (!empty && (dq_out == nullptr || dk_out == nullptr || dq == nullptr || dk == nullptr ||
                 (q_weight != nullptr && q == nullptr) || (k_weight != nullptr && k == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  // a weight has a gradient, and only a weight has one
  if ((q_weight == nullptr) != (dq_weight == nullptr) || (k_weight == nullptr) != (dk_weight == nullptr))
    return ATTN_ERR_INVALID_ARG;
  const int size = dtype == ATTN_DTYPE_BF16 ? 2 : 4;
  if ((q_weight != nullptr && !view_ok(q, strides, B, Hq, N, size)) ||
      (k_weight != nullptr && !view_ok(k, strides + 3, B, Hkv, N, size)) ||
      !view_ok(dq_out, strides + 6, B, Hq, N, size) || !view_ok(dk_out, strides + 9, B, Hkv, N, size) ||
      !view_ok(dq, strides + 12, B, Hq, N, size) || !view_ok(dk, strides + 15, B, Hkv, N, size))
    return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u)
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  const bool weighted = q_weight != nullptr || k_weight != nullptr;
  if (weighted && (workspace == nullptr || !aligned16(workspace) ||
                   workspace_bytes < attn_qk_norm_rope_bwd_workspace_bytes(d)))
    return ATTN_ERR_WORKSPACE;
  cudaStream_t strm = reinterpret_cast<cudaStream_t>(stream);
  int chunks = 1, cq = 0;
  unsigned blocks = 0;
  if (!empty) {
    if ((rc = configure_fwd(info)) != ATTN_OK) return rc;  // the tensor-map encoder
    long long st[20];
    qkn_flatten(p, st, 6, strides);
    p.dw = weighted ? static_cast<float*>(workspace) : nullptr;
    const int heads = qkn::kUnrollBwd * (512 / (d * size));
    if ((rc = qkn_tile_blocks(p, heads, std::min(qkn::kTileBlocksBwd * info->num_sms, kQknBwdBlocks), &chunks, &cq,
                              &blocks)) != ATTN_OK)
      return rc;
    CUtensorMap t[6];
    const void* views[6] = {q, k, dq_out, dk_out, dq, dk};
    for (int i = 0; i < 6; ++i) {
      if ((i == 0 && q_weight == nullptr) || (i == 1 && k_weight == nullptr)) {
        t[i] = CUtensorMap{};  // not read
        continue;
      }
      if ((rc = encode_map_heads(&t[i], views[i], st + 3 * i, p.B, i % 2 ? Hkv : Hq, p.N, d, dtype, heads)) != ATTN_OK)
        return rc;
    }
    const bool full = rot_dim == d, multi = num_axes > 1, inter = interleaved != 0;
    auto* kern = ATTN_QKN_PICK(qkn::qk_norm_rope_bwd_kernel);
    kern<<<blocks, qkn::kTileThreads, 0, strm>>>(t[0], t[1], t[2], t[3], t[4], t[5], p);
    if ((rc = cuda_status(cudaGetLastError())) != ATTN_OK) return rc;
  }
  if (weighted)
    rc = launch_early<const float*, int, int, int, int, float*, float*>(
        qkn::qk_norm_dw_kernel, dim3(d / 8, 2), 8 * qkn::kSumRows, strm, static_cast<const float*>(workspace),
        static_cast<int>(blocks), chunks, cq, d, dq_weight, dk_weight);
  return rc;
}

int attn_qk_norm_rope_paged(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                            void* v_cache, const void* q_weight, const void* k_weight,
                            const float* rope, const int* positions, const int* slots,
                            const long long* strides, const int* sections, int T, int Hq, int Hkv,
                            int num_pages, int page_size, int d, int rot_dim, int max_pos,
                            int num_axes, int interleaved, float eps, attn_stream_t stream) {
  qkn::Params p{};
  int rc = qkn_common(p, q_weight, k_weight, rope, positions, sections, ATTN_DTYPE_BF16, 1, T, Hq,
                      Hkv, d, rot_dim, max_pos, num_axes, eps);
  if (rc != ATTN_OK) return rc;
  if (strides == nullptr || num_pages < 0 || !page_size_ok(page_size)) return ATTN_ERR_INVALID_ARG;
  if (d != 128) return ATTN_ERR_UNSUPPORTED;
  if (T > 0 && (q == nullptr || k == nullptr || v == nullptr || q_out == nullptr || slots == nullptr))
    return ATTN_ERR_INVALID_ARG;
  if (T > 0 && num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return ATTN_ERR_INVALID_ARG;
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (!view_ok(q, strides, 1, Hq, T, 2) || !view_ok(k, strides + 3, 1, Hkv, T, 2) ||
      !view_ok(v, strides + 6, 1, Hkv, T, 2) || !view_ok(q_out, strides + 9, 1, Hq, T, 2) ||
      !aligned16(k_cache) || !aligned16(v_cache) || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  if (T == 0) return ATTN_OK;
  p.x[0] = q;
  p.x[1] = k;
  p.v = v;
  p.out[0] = q_out;
  p.xs[0] = make_view(strides);
  p.xs[1] = make_view(strides + 3);
  p.vs = make_view(strides + 6);
  p.os[0] = make_view(strides + 9);
  p.pos_axis = strides[12];
  p.pos_b = 0;
  p.slots = slots;
  p.cache[0] = k_cache;
  p.cache[1] = v_cache;
  p.slots_total = num_pages * page_size;
  // a warp per item (its heads of one token) up to kBlocks blocks per SM, one at least for every group of heads
  const int heads = qkn::kUnroll * 2;
  const long long chunks = (Hq + heads - 1) / heads + 2ll * ((Hkv + heads - 1) / heads);
  const long long want = (T * chunks + qkn::kWarps - 1) / qkn::kWarps, least = (chunks + qkn::kWarps - 1) / qkn::kWarps;
  const long long blocks = std::max(std::min<long long>(want, qkn::kBlocks * info->num_sms), least);
  if (blocks > (1 << 20)) return ATTN_ERR_UNSUPPORTED;
  const bool full = rot_dim == d, multi = num_axes > 1, inter = interleaved != 0;
  auto* kern = ATTN_QKN_PICK_D(qkn::qk_norm_rope_paged_kernel, __nv_bfloat16, 128);
  kern<<<static_cast<unsigned>(blocks), qkn::kThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cuda_status(cudaGetLastError());
}

int attn_page_update(int* block_table, const int* old_lens, const int* new_lens, int* free_pages,
                     const long long* ring_in, long long* ring_out, int* cu_seqlens, int* slots,
                     int* positions, const int* pos_offset, int B, int max_pages_per_seq,
                     int page_size, int num_pages, int max_tokens, attn_stream_t stream) {
  if (B < 0 || max_pages_per_seq < 0 || num_pages < 0 || max_tokens < 0 || !page_size_ok(page_size))
    return ATTN_ERR_INVALID_ARG;
  if (ring_in == nullptr || ring_out == nullptr || cu_seqlens == nullptr ||
      (B > 0 && (old_lens == nullptr || new_lens == nullptr)) ||
      (B > 0 && max_pages_per_seq > 0 && block_table == nullptr) ||
      (num_pages > 0 && free_pages == nullptr) ||
      (max_tokens > 0 && (slots == nullptr || positions == nullptr)))
    return ATTN_ERR_INVALID_ARG;
  // the blocks read one ring state while one of them writes the other
  if (ring_in < ring_out + 3 && ring_out < ring_in + 3) return ATTN_ERR_INVALID_ARG;
  if (B > pages::kMaxRequests || static_cast<long long>(num_pages) * page_size > 0x7fffffffLL)
    return ATTN_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(ring_in) | reinterpret_cast<uintptr_t>(ring_out)) & 7u) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  int rc = current_device(&info);
  if (rc != ATTN_OK) return rc;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!info->pages_configured) {
      rc = cuda_status(cudaFuncSetAttribute(pages::page_update_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            (3 * pages::kMaxRequests + 1) * static_cast<int>(sizeof(int))));
      if (rc != ATTN_OK) return rc;
      info->pages_configured = true;
    }
  }
  pages::Params p{};
  p.table = block_table;
  p.old_lens = old_lens;
  p.new_lens = new_lens;
  p.free_pages = free_pages;
  p.ring_in = ring_in;
  p.ring_out = ring_out;
  p.cu = cu_seqlens;
  p.slots = slots;
  p.positions = positions;
  p.offset = pos_offset;
  p.B = B;
  p.max_pages = max_pages_per_seq;
  p.page_shift = log2_int(page_size);
  p.cap = num_pages;
  p.max_tokens = max_tokens;
  // a thread per token, and 32 a request for the pages (the device alone knows how many move)
  const int want = std::max((max_tokens - 1) / pages::kThreads + 1, (B + pages::kWarps - 1) / pages::kWarps);
  const int blocks = std::max(1, std::min(want, info->num_sms));
  const size_t smem = (3 * static_cast<size_t>(B) + 1) * sizeof(int);
  pages::page_update_kernel<<<blocks, pages::kThreads, smem, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return cuda_status(cudaGetLastError());
}

size_t attn_decode_shared_prefix_workspace_bytes(int B, int Hq, int Hkv, int num_groups,
                                                 int max_prefix_len, int max_seq_len, int d) {
  if (pfx_shapes(B, Hq, Hkv, num_groups, max_prefix_len, max_seq_len, d) != ATTN_OK) return 0;
  return pfx_layout(B, Hq, Hkv, num_groups).total;
}

int attn_decode_shared_prefix(const void* q, const void* k_cache, const void* v_cache, void* o,
                              float* lse, const int* prefix_table, const int* prefix_lens,
                              const int* group_starts, const int* block_table, const int* seq_lens,
                              int B, int Hq, int Hkv, int num_groups, int num_pages, int page_size,
                              int max_prefix_pages, int max_prefix_len, int max_pages_per_seq,
                              int max_seq_len, int d, float scale, void* workspace,
                              size_t workspace_bytes, attn_stream_t stream) {
  int rc = pfx_shapes(B, Hq, Hkv, num_groups, max_prefix_len, max_seq_len, d);
  if (rc != ATTN_OK) return rc;
  if (num_pages < 0 || max_prefix_pages < 0 || max_pages_per_seq < 0 || !page_size_ok(page_size))
    return ATTN_ERR_INVALID_ARG;
  if (max_prefix_len > static_cast<long long>(max_prefix_pages) * page_size ||
      max_seq_len > static_cast<long long>(max_pages_per_seq) * page_size)
    return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return ATTN_ERR_INVALID_ARG;
  const bool prefixes = num_groups > 0 && max_prefix_len > 0, own = max_seq_len > 0;
  if (B > 0) {
    if (q == nullptr || o == nullptr) return ATTN_ERR_INVALID_ARG;
    if ((prefixes || own) && num_pages > 0 && (k_cache == nullptr || v_cache == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (num_groups > 0 && (prefix_lens == nullptr || group_starts == nullptr)) return ATTN_ERR_INVALID_ARG;
    if (prefixes && prefix_table == nullptr) return ATTN_ERR_INVALID_ARG;
    if (seq_lens == nullptr || (own && block_table == nullptr)) return ATTN_ERR_INVALID_ARG;
  }
  if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return ATTN_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o)) return ATTN_ERR_UNSUPPORTED;
  if (lse != nullptr && (reinterpret_cast<uintptr_t>(lse) & 3u)) return ATTN_ERR_UNSUPPORTED;
  DeviceInfo* info = nullptr;
  if ((rc = current_device(&info)) != ATTN_OK) return rc;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (B == 0) return ATTN_OK;
  if (!prefixes && !own)
    return launch_fill_empty(static_cast<__nv_bfloat16*>(o), lse, static_cast<size_t>(B) * Hq, d, st);
  if (num_pages == 0) return ATTN_ERR_INVALID_ARG;  // keys, but no page to hold one
  const PfxLayout L = pfx_layout(B, Hq, Hkv, num_groups);
  if (workspace == nullptr || workspace_bytes < L.total || !aligned16(workspace)) return ATTN_ERR_WORKSPACE;
  if ((rc = configure_pfx(info)) != ATTN_OK) return rc;

  pfx::Params p{};
  p.B = B;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = Hq / Hkv;
  p.S = 128 / p.G;
  p.num_groups = prefixes ? num_groups : 0;
  p.max_prefix_len = max_prefix_len;
  p.max_prefix_pages = max_prefix_pages;
  p.max_seq_len = max_seq_len;
  p.max_pages = max_pages_per_seq;
  p.num_pages = num_pages;
  p.page_shift = log2_int(page_size);
  p.thin_cost = pfx::cost_thin_step(p.page_shift);
  p.prefix_table = prefix_table;
  p.prefix_lens = prefix_lens;
  p.group_starts = group_starts;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  // scale = 0 makes every weight equal; a tiny positive c gives exactly that (see attn_fwd)
  p.c = scale * kLog2e;
  if (p.c == 0.f) p.c = 1e-30f;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + L.lse_offset);
  p.plan = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + L.plan_offset);
  p.thin_row0 = L.thin_row0;
  p.own_row0 = L.own_row0;

  CUtensorMap tq, tq_thin, tq_own, tk, tv;
  const int rows = num_pages * page_size;
  const uint32_t piece = static_cast<uint32_t>(std::min(page_size, pfx::kTile));
  if (encode_map_decode_q(&tq, q, Hq, B, p.G, p.S) != ATTN_OK ||
      encode_map_decode_q(&tq_thin, q, Hq, B, p.G, pfx::kThinRows / p.G) != ATTN_OK ||
      encode_map_decode_q(&tq_own, q, Hq, B, p.G, 1) != ATTN_OK ||
      encode_map_pages(&tk, k_cache, rows, Hkv, piece) != ATTN_OK ||
      encode_map_pages(&tv, v_cache, rows, Hkv, piece) != ATTN_OK)
    return ATTN_ERR_UNSUPPORTED;
  const int ctas = std::min(info->num_sms, kPfxCtas);
  if (scale < 0.f)
    pfx::decode_prefix_kernel<true><<<ctas, pfx::kThreads, pfx::kSmemBytes, st>>>(tq, tq_thin, tq_own, tk, tv, p);
  else
    pfx::decode_prefix_kernel<false><<<ctas, pfx::kThreads, pfx::kSmemBytes, st>>>(tq, tq_thin, tq_own, tk, tv, p);
  if ((rc = cuda_status(cudaGetLastError())) != ATTN_OK) return rc;
  // sets of warps per block: as many as the SMs hold at 32 warps each
  int split = 4;
  while (split > 1 && static_cast<long long>(B) * Hq * split > 32ll * info->num_sms) split /= 2;
  void (*combine)(pfx::Params, __nv_bfloat16*, float*) = nullptr;
#define ATTN_PFX_COMBINE(G)                                                  \
  combine = split == 4   ? pfx::decode_prefix_combine_kernel<G, 4>           \
            : split == 2 ? pfx::decode_prefix_combine_kernel<G, 2>           \
                         : pfx::decode_prefix_combine_kernel<G, 1>
  switch (p.G) {
    case 1: ATTN_PFX_COMBINE(1); break;
    case 2: ATTN_PFX_COMBINE(2); break;
    case 4: ATTN_PFX_COMBINE(4); break;
    default: ATTN_PFX_COMBINE(8); break;
  }
#undef ATTN_PFX_COMBINE
  return launch_early<pfx::Params, __nv_bfloat16*, float*>(combine, dim3(Hkv, B), 32 * p.G * split, st, p,
                                                           static_cast<__nv_bfloat16*>(o), lse);
}

}  // extern "C"
