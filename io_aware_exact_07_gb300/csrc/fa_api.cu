// C ABI of the attention library (declared in include/fa.h): argument
// validation, TMA tensor-map encoding, kernel launches, test hooks and the
// device status word. No device memory is allocated here.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cstdlib>
#include <mutex>
#include <new>
#include <vector>

#include "../../include/fa.h"
#include "fa_decode.h"
#include "fa_fp8.h"
#include "fa_kernels.h"
#include "fa_paged.h"

namespace {

// First device-side error since the last clear (one per device that loads the library).
__device__ unsigned int g_fa_status;

constexpr int kMaxDevices = 64;
std::atomic<unsigned long long> g_timeout_ns{4000000000ull};
std::atomic<int> g_inject_stall{0};

struct DeviceInfo {
  bool ready = false;
  int num_sms = 0;
  int major = 0;
  unsigned int* status = nullptr;
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_dev_mutex;

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;
std::once_flag g_encode_once;

EncodeTiledFn encoder() {
  std::call_once(g_encode_once, []() {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
  });
  return g_encode;
}

// Per-device set-up, done once per device with that device current.
fa_status device_info(DeviceInfo** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_dev_mutex);
  DeviceInfo& di = g_dev[dev];
  if (!di.ready) {
    cudaDeviceProp prop;
    if (cudaGetDeviceProperties(&prop, dev) != cudaSuccess) return FA_ERR_CUDA;
    di.num_sms = prop.multiProcessorCount;
    di.major = prop.major;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_fa_status) != cudaSuccess) return FA_ERR_CUDA;
    di.status = static_cast<unsigned int*>(p);
    di.ready = true;
  }
  if (di.major != 10) return FA_ERR_UNSUPPORTED;
  *out = &di;
  return FA_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int p8_of(float p) {
  if (!(p >= 0.f) || !(p < 1.f)) return -1;
  const int v = static_cast<int>(std::floor(static_cast<double>(p) * 256.0 + 0.5));
  return v >= 256 ? -1 : v;
}

fa_status check_common(int B, int H, int N, int d, float scale, float dropout_p, int Hkv) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(B) * H * N;
  if (rows >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (p8_of(dropout_p) < 0) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

// [B*H, N, d] bf16 tensor, boxes of 64 columns x 128 rows, 128-byte swizzle,
// out-of-range elements read as zero.
bool encode_map(CUtensorMap* m, const void* base, int BH, int N, int d) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(N),
                        static_cast<cuuint64_t>(BH)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                           static_cast<cuuint64_t>(N) * static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[3] = {64, 128, 1};
  cuuint32_t elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [outer, rows, inner] tensor of bytes (e4m3 codes) with rows of `inner`
// bytes spaced `row_stride` bytes apart: 128-byte x 128-row boxes, 128-byte
// swizzle, out-of-range elements read as zero.
bool encode_map_u8(CUtensorMap* m, const void* base, int outer, int rows, int inner,
                   int row_stride) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(row_stride),
                           static_cast<cuuint64_t>(rows) * static_cast<cuuint64_t>(row_stride)};
  cuuint32_t box[3] = {128, 128, 1};
  cuuint32_t elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Packed tokens [T, H, d] bf16, `stride` elements apart: boxes of 64 columns x heads x tokens,
// 128-byte swizzle.
bool encode_map_tokens(CUtensorMap* m, const void* base, int T, int H, int d, int64_t stride,
                       int heads, int tokens) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H),
                        static_cast<cuuint64_t>(T)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(stride) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(heads), static_cast<cuuint32_t>(tokens)};
  cuuint32_t elem[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             elem, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Pages of a cache, [num_pages, H_kv, page_size, d] in the cache's strides: boxes of 64 bf16
// columns (128-byte swizzle) or of d codes (as they are) x rows; out-of-range pages read as zero.
bool encode_map_pages(CUtensorMap* m, const void* base, const fa::PagedArgs& c, bool e4m3,
                      int rows) {
  EncodeTiledFn enc = encoder();
  if (enc == nullptr) return false;
  const cuuint64_t es = e4m3 ? 1 : 2;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.d), static_cast<cuuint64_t>(c.page_size),
                        static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.num_pages)};
  cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.stride_row) * es,
                           static_cast<cuuint64_t>(c.stride_head) * es,
                           static_cast<cuuint64_t>(c.stride_page) * es};
  cuuint32_t box[4] = {static_cast<cuuint32_t>(e4m3 ? c.d : 64), static_cast<cuuint32_t>(rows), 1,
                       1};
  cuuint32_t elem[4] = {1, 1, 1, 1};
  return enc(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void*>(base), dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
             e4m3 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

fa::MaskParams make_mask(int B, int H, int Hkv, int N, int causal, const uint8_t* bm,
                         const int32_t* sl, int wl = -1, int wr = -1) {
  fa::MaskParams m;
  m.B = B;
  m.H = H;
  m.Hkv = Hkv;
  m.N = N;
  m.nb = (N + fa::kTile - 1) / fa::kTile;
  m.causal = causal ? 1 : 0;
  m.wl = wl;
  m.wr = wr;
  m.block_mask = bm;
  m.seqlens_k = sl;
  m.Nk = N;
  m.q_off = 0;
  return m;
}

fa::DropParams make_drop(float p, uint64_t seed, uint64_t offset) {
  fa::DropParams d;
  d.p8 = p8_of(p);
  d.keep_scale = static_cast<float>(1.0 / (1.0 - d.p8 / 256.0));
  d.seed_lo = static_cast<uint32_t>(seed);
  d.seed_hi = static_cast<uint32_t>(seed >> 32);
  d.off_lo = static_cast<uint32_t>(offset);
  d.off_hi = static_cast<uint32_t>(offset >> 32);
  // Philox4x32 key schedule (Salmon et al., SC'11): the key grows by the two
  // Weyl constants every round.
  for (int r = 0; r < 10; ++r) {
    d.rk[r].x = d.seed_lo + static_cast<uint32_t>(r) * 0x9E3779B9u;
    d.rk[r].y = d.seed_hi + static_cast<uint32_t>(r) * 0xBB67AE85u;
  }
  return d;
}

// Launch kinds the stall hook (fa_test_inject_stall) can target.
enum StallTarget { kStallNone = 0, kStallForward = 1, kStallDkdv = 2, kStallDq = 3 };

// 1 if the stall hook is armed for `target` (and then disarm it), else 0.
int take_stall(StallTarget target) {
  if (target == kStallNone) return 0;
  int expected = static_cast<int>(target);
  return g_inject_stall.compare_exchange_strong(expected, 0) ? 1 : 0;
}

fa::SyncParams make_sync(const DeviceInfo* di, StallTarget target) {
  fa::SyncParams s;
  s.status = di->status;
  s.timeout_ns = g_timeout_ns.load();
  s.inject_stall = take_stall(target);
  return s;
}

// Limits of the calls with positions on a key axis: sums of two positions, an offset and a window
// stay within 32 bits.
constexpr int kMaxAxis = 1 << 28;
constexpr int kMaxDistances = 1 << 16;  // distances of a bias, left + right + 1

size_t round256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Backward workspace for fa_bwd_noalloc: room for D = rowsum(dO * O) of up to
// kNoAllocMaxRows query rows (B*H*N), 16 MiB. It is part of the library's
// device image, so every GPU that loads the library holds it until the
// process exits. In host code `g_noalloc_dsum` is only a host-side stand-in
// for the array; its device address comes from cudaGetSymbolAddress below.
constexpr size_t kNoAllocMaxRows = static_cast<size_t>(1) << 22;
__device__ __align__(256) float g_noalloc_dsum[kNoAllocMaxRows];
void* g_noalloc_addr[kMaxDevices] = {};
std::mutex g_noalloc_mutex;

}  // namespace

extern "C" {

static fa_status fwd_impl(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                          int H, int Hkv, int N, int d, float scale, int causal, int wl, int wr,
                          float dropout_p, uint64_t seed, uint64_t offset,
                          const uint8_t* block_mask, const int32_t* seqlens_k, void* stream) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Hkv);
  if (st != FA_OK) return st;
  if (wl < -1 || wr < -1) return FA_ERR_INVALID_ARG;
  if (!q || !k || !v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  CUtensorMap tq, tk, tv;
  if (!encode_map(&tq, q, B * H, N, d) || !encode_map(&tk, k, B * Hkv, N, d) ||
      !encode_map(&tv, v, B * Hkv, N, d))
    return FA_ERR_CUDA;
  fa::FwdArgs a;
  a.mask = make_mask(B, H, Hkv, N, causal, block_mask, seqlens_k, wl, wr);
  a.drop = make_drop(dropout_p, seed, offset);
  a.sync = make_sync(di, kStallForward);
  a.scale_log2 = scale * fa::kLog2e;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.mode = wl >= 0 || wr >= 0 ? fa::kWindow : fa::kPlain;
  a.rel = fa::RelParams{};
  cudaError_t e = fa::launch_fwd(tq, tk, tv, a, d, a.drop.p8 > 0, di->num_sms,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                 int N, int d, float scale, int causal, float dropout_p, uint64_t seed,
                 uint64_t offset, const uint8_t* block_mask, const int32_t* seqlens_k,
                 void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, H, N, d, scale, causal, -1, -1, dropout_p, seed, offset,
                  block_mask, seqlens_k, stream);
}

fa_status fa_fwd_gqa(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                     int H, int H_kv, int N, int d, float scale, int causal, float dropout_p,
                     uint64_t seed, uint64_t offset, const uint8_t* block_mask,
                     const int32_t* seqlens_k, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, H_kv, N, d, scale, causal, -1, -1, dropout_p, seed,
                  offset, block_mask, seqlens_k, stream);
}

fa_status fa_fwd_window(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                        int H, int H_kv, int N, int d, float scale, int causal, int window_left,
                        int window_right, float dropout_p, uint64_t seed, uint64_t offset,
                        const uint8_t* block_mask, const int32_t* seqlens_k, void* stream) {
  return fwd_impl(q, k, v, o, lse, B, H, H_kv, N, d, scale, causal, window_left, window_right,
                  dropout_p, seed, offset, block_mask, seqlens_k, stream);
}

size_t fa_bwd_workspace_size(int B, int H, int N, int d) {
  (void)d;
  if (B < 1 || H < 1 || N < 1) return 0;
  return round256(static_cast<size_t>(B) * H * N * sizeof(float));
}

// Shared validation and set-up of the backward stages. `need` selects which
// pointers must be present: 1 = preprocess (o, dout), 2 = dK/dV, 4 = dQ.
static fa_status bwd_prepare(const void* q, const void* k, const void* v, const void* o,
                             const void* dout, const float* lse, void* dq, void* dk, void* dv,
                             int B, int H, int Hkv, int N, int d, float scale, int causal,
                             int wl, int wr, float dropout_p, uint64_t seed, uint64_t offset,
                             const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                             size_t workspace_bytes, int need, fa::BwdArgs* a, CUtensorMap* maps,
                             DeviceInfo** di) {
  fa_status st = check_common(B, H, N, d, scale, dropout_p, Hkv);
  if (st != FA_OK) return st;
  if (wl < -1 || wr < -1) return FA_ERR_INVALID_ARG;
  if (need & 1) {
    if (!o || !dout || !aligned16(o) || !aligned16(dout)) return FA_ERR_INVALID_ARG;
  }
  if (need & 6) {
    if (!q || !k || !v || !dout || !lse) return FA_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, dout})
      if (!aligned16(p)) return FA_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  }
  if ((need & 2) && (!dk || !dv || !aligned16(dk) || !aligned16(dv))) return FA_ERR_INVALID_ARG;
  if ((need & 4) && (!dq || !aligned16(dq))) return FA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < fa_bwd_workspace_size(B, H, N, d) ||
      !aligned16(workspace))
    return FA_ERR_WORKSPACE;
  if ((st = device_info(di)) != FA_OK) return st;
  if (need & 6) {
    if (!encode_map(&maps[0], q, B * H, N, d) || !encode_map(&maps[1], k, B * Hkv, N, d) ||
        !encode_map(&maps[2], v, B * Hkv, N, d) || !encode_map(&maps[3], dout, B * H, N, d))
      return FA_ERR_CUDA;
  }
  a->mask = make_mask(B, H, Hkv, N, causal, block_mask, seqlens_k, wl, wr);
  a->drop = make_drop(dropout_p, seed, offset);
  a->sync = make_sync(*di, kStallNone);
  a->scale = scale;
  a->scale_log2 = scale * fa::kLog2e;
  a->o = static_cast<const __nv_bfloat16*>(o);
  a->dout = static_cast<const __nv_bfloat16*>(dout);
  a->lse = lse;
  a->dsum = static_cast<float*>(workspace);
  a->dq = static_cast<__nv_bfloat16*>(dq);
  a->dk = static_cast<__nv_bfloat16*>(dk);
  a->dv = static_cast<__nv_bfloat16*>(dv);
  a->mode = wl >= 0 || wr >= 0 ? fa::kWindow : fa::kPlain;
  a->rel = fa::RelParams{};
  a->row_sums = nullptr;
  a->pieces = 1;
  a->key_tiles = nullptr;
  return FA_OK;
}

static fa_status bwd_impl(const void* q, const void* k, const void* v, const void* o,
                          const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                          int H, int Hkv, int N, int d, float scale, int causal, int wl, int wr,
                          float dropout_p, uint64_t seed, uint64_t offset,
                          const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                          size_t workspace_bytes, void* stream) {
  fa::BwdArgs a;
  CUtensorMap m[4];
  DeviceInfo* di = nullptr;
  fa_status st = bwd_prepare(q, k, v, o, dout, lse, dq, dk, dv, B, H, Hkv, N, d, scale, causal,
                             wl, wr, dropout_p, seed, offset, block_mask, seqlens_k, workspace,
                             workspace_bytes, 7, &a, m, &di);
  if (st != FA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool drop = a.drop.p8 > 0;
  cudaError_t e = fa::launch_bwd_preprocess(a, d, di->num_sms, s);
  if (e == cudaSuccess) {
    a.sync.inject_stall = take_stall(kStallDkdv);
    e = fa::launch_bwd_dkdv(m[0], m[1], m[2], m[3], a, d, drop, di->num_sms, s);
  }
  if (e == cudaSuccess) {
    a.sync.inject_stall = take_stall(kStallDq);
    e = fa::launch_bwd_dq(m[0], m[1], m[2], m[3], a, d, drop, di->num_sms, s);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dout,
                 const float* lse, void* dq, void* dk, void* dv, int B, int H, int N, int d,
                 float scale, int causal, float dropout_p, uint64_t seed, uint64_t offset,
                 const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                 size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, H, H, N, d, scale, causal, -1, -1,
                  dropout_p, seed, offset, block_mask, seqlens_k, workspace, workspace_bytes,
                  stream);
}

fa_status fa_bwd_gqa(const void* q, const void* k, const void* v, const void* o, const void* dout,
                     const float* lse, void* dq, void* dk, void* dv, int B, int H, int H_kv, int N,
                     int d, float scale, int causal, float dropout_p, uint64_t seed,
                     uint64_t offset, const uint8_t* block_mask, const int32_t* seqlens_k,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, H, H_kv, N, d, scale, causal, -1, -1,
                  dropout_p, seed, offset, block_mask, seqlens_k, workspace, workspace_bytes,
                  stream);
}

fa_status fa_bwd_window(const void* q, const void* k, const void* v, const void* o,
                        const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                        int H, int H_kv, int N, int d, float scale, int causal, int window_left,
                        int window_right, float dropout_p, uint64_t seed, uint64_t offset,
                        const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return bwd_impl(q, k, v, o, dout, lse, dq, dk, dv, B, H, H_kv, N, d, scale, causal, window_left,
                  window_right, dropout_p, seed, offset, block_mask, seqlens_k, workspace,
                  workspace_bytes, stream);
}

fa_status fa_bwd_preprocess(const void* o, const void* dout, int B, int H, int N, int d,
                            void* workspace, size_t workspace_bytes, void* stream) {
  fa::BwdArgs a;
  CUtensorMap m[4];
  DeviceInfo* di = nullptr;
  fa_status st = bwd_prepare(nullptr, nullptr, nullptr, o, dout, nullptr, nullptr, nullptr,
                             nullptr, B, H, H, N, d, 1.f, 0, -1, -1, 0.f, 0, 0, nullptr, nullptr,
                             workspace, workspace_bytes, 1, &a, m, &di);
  if (st != FA_OK) return st;
  return fa::launch_bwd_preprocess(a, d, di->num_sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_bwd_dkdv(const void* q, const void* k, const void* v, const void* dout,
                      const float* lse, void* dk, void* dv, int B, int H, int N, int d,
                      float scale, int causal, float dropout_p, uint64_t seed, uint64_t offset,
                      const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                      size_t workspace_bytes, void* stream) {
  fa::BwdArgs a;
  CUtensorMap m[4];
  DeviceInfo* di = nullptr;
  fa_status st = bwd_prepare(q, k, v, nullptr, dout, lse, nullptr, dk, dv, B, H, H, N, d, scale,
                             causal, -1, -1, dropout_p, seed, offset, block_mask, seqlens_k,
                             workspace, workspace_bytes, 2, &a, m, &di);
  if (st != FA_OK) return st;
  a.sync.inject_stall = take_stall(kStallDkdv);
  return fa::launch_bwd_dkdv(m[0], m[1], m[2], m[3], a, d, a.drop.p8 > 0, di->num_sms,
                             static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_bwd_dq(const void* q, const void* k, const void* v, const void* dout,
                    const float* lse, void* dq, int B, int H, int N, int d, float scale,
                    int causal, float dropout_p, uint64_t seed, uint64_t offset,
                    const uint8_t* block_mask, const int32_t* seqlens_k, void* workspace,
                    size_t workspace_bytes, void* stream) {
  fa::BwdArgs a;
  CUtensorMap m[4];
  DeviceInfo* di = nullptr;
  fa_status st = bwd_prepare(q, k, v, nullptr, dout, lse, dq, nullptr, nullptr, B, H, H, N, d,
                             scale, causal, -1, -1, dropout_p, seed, offset, block_mask,
                             seqlens_k, workspace, workspace_bytes, 4, &a, m, &di);
  if (st != FA_OK) return st;
  a.sync.inject_stall = take_stall(kStallDq);
  return fa::launch_bwd_dq(m[0], m[1], m[2], m[3], a, d, a.drop.p8 > 0, di->num_sms,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_bwd_noalloc(const void* q, const void* k, const void* v, const void* o,
                         const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                         int H, int N, int d, float scale, int causal, float dropout_p,
                         uint64_t seed, uint64_t offset, const uint8_t* block_mask,
                         const int32_t* seqlens_k, void* stream) {
  if (B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (static_cast<size_t>(B) * static_cast<size_t>(H) * static_cast<size_t>(N) > kNoAllocMaxRows)
    return FA_ERR_WORKSPACE;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return FA_ERR_CUDA;
  void* scratch = nullptr;
  {
    // First call on this device (with it current): look up the array's device address.
    std::lock_guard<std::mutex> lock(g_noalloc_mutex);
    if (g_noalloc_addr[dev] == nullptr) {
      void* p = nullptr;
      if (cudaGetSymbolAddress(&p, g_noalloc_dsum) != cudaSuccess || p == nullptr)
        return FA_ERR_CUDA;
      g_noalloc_addr[dev] = p;
    }
    scratch = g_noalloc_addr[dev];
  }
  // D is written in full by the first backward kernel before it is read, so
  // the array's contents from an earlier call never matter and nothing is cleared.
  return fa_bwd(q, k, v, o, dout, lse, dq, dk, dv, B, H, N, d, scale, causal, dropout_p, seed,
                offset, block_mask, seqlens_k, scratch, kNoAllocMaxRows * sizeof(float), stream);
}

// Work split of fa_decode: the (K/V head, key tile) pairs, B * H_kv * n_t of
// them, cut into equal runs of per_cta pairs, one run per CTA; seg_max bounds
// the number of runs that cut one K/V head (1: no head is cut, no combine).
struct DecodePlan {
  int n_t, per_cta, grid, seg_max;
};

static fa_status decode_plan(int B, int H, int Hkv, int Nq, int Nk, int d, int num_ctas,
                             DecodePlan* p) {
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || num_ctas < 0) return FA_ERR_INVALID_ARG;
  if (Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H * Nq >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(H / Hkv) * Nq > fa::kTile) return FA_ERR_UNSUPPORTED;
  p->n_t = (Nk + fa::kTile - 1) / fa::kTile;
  const long long total = static_cast<long long>(B) * Hkv * p->n_t;
  if (total >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  long long ctas = num_ctas;
  long long per = 0;
  if (ctas == 0) {
    DeviceInfo* di = nullptr;
    const fa_status st = device_info(&di);
    if (st != FA_OK) return st;
    ctas = di->num_sms;
    // Whole K/V heads per CTA when that still keeps enough SMs streaming to
    // saturate HBM (measured: 4/5 of them at d = 128, where one CTA streams
    // about 54 GB/s; all but 1/20 at d = 64, where a CTA is slower than its
    // share of HBM): no head is cut, so there are no partial results to write
    // and no combine launch. Otherwise equal runs over all SMs, cutting heads.
    const long long heads = static_cast<long long>(B) * Hkv;
    const long long k = (heads + ctas - 1) / ctas;  // heads per CTA
    const long long busy = (heads + k - 1) / k;      // CTAs that get a head
    if (d == 128 ? busy * 5 >= ctas * 4 : busy * 20 >= ctas * 19) per = k * p->n_t;
  }
  if (ctas > total) ctas = total;
  if (per == 0) per = (total + ctas - 1) / ctas;
  p->per_cta = static_cast<int>(per);
  p->grid = static_cast<int>((total + per - 1) / per);
  if (per % p->n_t == 0) {
    p->seg_max = 1;  // every run holds whole heads
  } else {
    const int bound = (p->n_t - 1) / p->per_cta + 2;
    p->seg_max = bound < p->grid ? bound : p->grid;
  }
  return FA_OK;
}

static size_t decode_ws_bytes(int B, int H, int Nq, int d, const DecodePlan& p) {
  if (p.seg_max <= 1) return 0;
  const size_t slots = static_cast<size_t>(B) * H * Nq * p.seg_max;
  return round256(slots * d * sizeof(float)) + round256(slots * sizeof(float));
}

size_t fa_decode_workspace_size(int B, int H, int H_kv, int Nq, int Nk, int d, int num_ctas) {
  DecodePlan p;
  if (decode_plan(B, H, H_kv, Nq, Nk, d, num_ctas, &p) != FA_OK) return 0;
  return decode_ws_bytes(B, H, Nq, d, p);
}

// Checks that the decode calls share.
static fa_status check_decode(const void* q, const void* k, const void* v, const void* o,
                              const float* lse, float scale, int window_left,
                              const int32_t* seqlens_k) {
  if (window_left < -1) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  for (const void* p : {q, k, v, o})
    if (!p || !aligned16(p)) return FA_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(seqlens_k) & 3u) != 0) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status fa_decode(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                    int B, int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                    int window_left, const int32_t* seqlens_k, int num_ctas, void* workspace,
                    size_t workspace_bytes, void* stream) {
  DecodePlan p;
  fa_status st = decode_plan(B, H, H_kv, Nq, Nk, d, num_ctas, &p);
  if (st != FA_OK) return st;
  if ((st = check_decode(q, k_cache, v_cache, o, lse, scale, window_left, seqlens_k)) != FA_OK)
    return st;
  const size_t ws = decode_ws_bytes(B, H, Nq, d, p);
  if (ws > 0 && (workspace == nullptr || workspace_bytes < ws || !aligned16(workspace)))
    return FA_ERR_WORKSPACE;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  CUtensorMap tq, tk, tv;
  if (!encode_map(&tq, q, 1, B * H * Nq, d) || !encode_map(&tk, k_cache, B * H_kv, Nk, d) ||
      !encode_map(&tv, v_cache, B * H_kv, Nk, d))
    return FA_ERR_CUDA;
  fa::DecodeArgs a;
  a.B = B;
  a.H = H;
  a.Hkv = H_kv;
  a.Nq = Nq;
  a.Nk = Nk;
  a.causal = causal ? 1 : 0;
  a.wl = window_left;
  a.seqlens_k = seqlens_k;
  a.n_t = p.n_t;
  a.per_cta = p.per_cta;
  a.seg_max = p.seg_max;
  a.scale_log2 = scale * fa::kLog2e;
  a.sync = make_sync(di, kStallForward);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.rel = fa::RelParams{};
  a.whole = 0;
  a.pieces = nullptr;
  const size_t slots = static_cast<size_t>(B) * H * Nq * p.seg_max;
  a.o_part = ws > 0 ? static_cast<float*>(workspace) : nullptr;
  a.lse_part = ws > 0 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                                 round256(slots * d * sizeof(float)))
                      : nullptr;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = fa::launch_decode(tq, tk, tv, a, d, p.grid, s);
  if (e == cudaSuccess && p.seg_max > 1) e = fa::launch_decode_combine(a, d, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Workspace of fa_paged_attn: one header per CTA, then the pieces' lse and outputs.
struct PagedWorkspace {
  int ctas, rows;
  bool whole;  // a step over few keys: no head is cut, nothing is left behind
  size_t lse_off, o_off, bytes;
};
static PagedWorkspace paged_workspace(int G, int d, int max_q, long long max_keys, int num_sms) {
  PagedWorkspace w;
  const long long rows = static_cast<long long>(G) * max_q;
  w.whole = rows <= fa::kStepRows && max_keys <= fa::kWholeKeys;
  w.ctas = num_sms < 256 ? num_sms : 256;  // the chunk kernel plans with a thread per CTA
  w.rows = rows <= fa::kStepRows ? static_cast<int>((rows + 7) / 8 * 8) : fa::kTile;
  const size_t slots = 2 * static_cast<size_t>(w.ctas) * w.rows;
  w.lse_off = round256(static_cast<size_t>(w.ctas) * 16);
  w.o_off = w.lse_off + round256(slots * sizeof(float));
  w.bytes = w.whole ? 0 : w.o_off + round256(slots * d * sizeof(float));
  return w;
}

// Plan of fa_decode_rel: the CTAs find their shares from the lengths on the device. Few query rows
// per K/V head run on the paged cache's step kernel, more as tiles of 128 rows. us with the one and
// the other: d = 64, 32 ragged sequences of up to 4096 keys, 16 K/V heads, 1 row 53 and 84, 16 rows
// 76 and 87, 20 rows 96 and 87; 4 of up to 500 keys 16 rows 10.2 and 10.5; d = 128, the same with 8
// K/V heads 8 rows 55.7 and 55.4, 12 rows 63 and 56; 1 of 131001 keys 8 rows 87 and 91, 16 89 and 91.
struct RelDecodePlan {
  bool step;
  int grid, whole;
  PagedWorkspace w;                // step
  size_t lse_off, pieces_off, bytes;
};

static fa_status rel_decode_plan(int B, int H, int Hkv, int Nq, int Nk, int d, int num_ctas,
                                 RelDecodePlan* p) {
  DecodePlan q;  // for its checks
  const fa_status st = decode_plan(B, H, Hkv, Nq, Nk, d, num_ctas > 0 ? num_ctas : 1, &q);
  if (st != FA_OK) return st;
  if (num_ctas < 0 || Nk > kMaxAxis) return FA_ERR_INVALID_ARG;
  int ctas = num_ctas;
  if (ctas == 0) {
    DeviceInfo* di = nullptr;
    const fa_status dev = device_info(&di);
    if (dev != FA_OK) return dev;
    ctas = di->num_sms;
  }
  const long long heads = static_cast<long long>(B) * Hkv;
  const size_t rows = static_cast<size_t>(H / Hkv) * Nq;
  p->step = rows <= static_cast<size_t>(fa::rel_step_rows(d));
  if (p->step) {
    p->w = paged_workspace(H / Hkv, d, Nq, num_ctas > 0 ? kMaxAxis : Nk, ctas);
    p->grid = p->w.ctas;
    p->whole = p->w.whole;
    p->bytes = p->w.bytes;
    return FA_OK;
  }
  p->whole = num_ctas == 0 && Nk <= fa::kWholeKeys;
  const long long most = p->whole ? heads : heads * q.n_t;
  p->grid = static_cast<int>(ctas < most ? ctas : most);
  const size_t slots = (heads + p->grid) * rows;
  p->lse_off = round256(slots * d * sizeof(float));
  p->pieces_off = p->lse_off + round256(slots * sizeof(float));
  p->bytes = p->whole ? 0 : p->pieces_off + round256(heads * sizeof(int2));
  return FA_OK;
}

size_t fa_decode_rel_workspace_size(int B, int H, int H_kv, int Nq, int Nk, int d, int num_ctas) {
  RelDecodePlan p;
  if (rel_decode_plan(B, H, H_kv, Nq, Nk, d, num_ctas, &p) != FA_OK) return 0;
  return p.bytes;
}

static fa_status check_lines(const float* lines, int left, int right);

fa_status fa_decode_rel(const void* q, const void* k_cache, const void* v_cache, void* o,
                        float* lse, int B, int H, int H_kv, int Nq, int Nk, int d, float scale,
                        int causal, int window_left, const int32_t* seqlens_k,
                        const float* rel_lines, int rel_left, int rel_right, int num_ctas,
                        void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_lines(rel_lines, rel_left, rel_right);
  if (st != FA_OK) return st;
  RelDecodePlan p;
  if ((st = rel_decode_plan(B, H, H_kv, Nq, Nk, d, num_ctas, &p)) != FA_OK) return st;
  if ((st = check_decode(q, k_cache, v_cache, o, lse, scale, window_left, seqlens_k)) != FA_OK)
    return st;
  if (p.bytes > 0 && (workspace == nullptr || workspace_bytes < p.bytes || !aligned16(workspace)))
    return FA_ERR_WORKSPACE;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  const fa::RelParams rel{rel_lines, rel_left, rel_right};
  if (window_left >= Nk) window_left = -1;  // hides nothing
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (p.step) {
    fa::PagedAttnArgs a = {};
    a.c.k = static_cast<uint8_t*>(const_cast<void*>(k_cache));
    a.c.v = static_cast<uint8_t*>(const_cast<void*>(v_cache));
    a.c.Hkv = H_kv;
    a.c.d = d;
    a.c.stride_page = static_cast<long long>(H_kv) * Nk * d;
    a.c.stride_head = static_cast<long long>(Nk) * d;
    a.c.stride_row = d;
    a.c.kv_lens = seqlens_k;
    a.c.B = B;
    a.c.T = B * Nq;
    a.c.max_q = Nq;
    a.c.status = di->status;
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.H = H;
    a.G = H / H_kv;
    a.o = static_cast<__nv_bfloat16*>(o);
    a.lse = lse;
    a.scale_log2 = scale * fa::kLog2e;
    a.causal = causal ? 1 : 0;
    a.wl = window_left;
    a.whole = p.whole;
    if (!p.whole) {
      a.headers = ws;
      a.lse_part = reinterpret_cast<float*>(ws + p.w.lse_off);
      a.o_part = reinterpret_cast<float*>(ws + p.w.o_off);
    }
    a.rel = rel;
    a.Nk = Nk;
    return fa::launch_rel_step(a, p.grid, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
  }
  CUtensorMap tq, tk, tv;
  if (!encode_map(&tq, q, 1, B * H * Nq, d) || !encode_map(&tk, k_cache, B * H_kv, Nk, d) ||
      !encode_map(&tv, v_cache, B * H_kv, Nk, d))
    return FA_ERR_CUDA;
  fa::DecodeArgs a = {};
  a.B = B;
  a.H = H;
  a.Hkv = H_kv;
  a.Nq = Nq;
  a.Nk = Nk;
  a.causal = causal ? 1 : 0;
  a.wl = window_left;
  a.seqlens_k = seqlens_k;
  a.scale_log2 = scale * fa::kLog2e;
  a.sync = make_sync(di, kStallForward);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.rel = rel;
  a.whole = p.whole;
  if (!p.whole) {
    a.o_part = reinterpret_cast<float*>(ws);
    a.lse_part = reinterpret_cast<float*>(ws + p.lse_off);
    a.pieces = reinterpret_cast<int2*>(ws + p.pieces_off);
    a.ctas = p.grid;
  }
  cudaError_t e = fa::launch_decode(tq, tk, tv, a, d, p.grid, s);
  if (e == cudaSuccess && !p.whole) e = fa::launch_decode_combine(a, d, s);
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

static fa_status check_lines(const float* lines, int left, int right) {
  if (lines == nullptr || !aligned16(lines)) return FA_ERR_INVALID_ARG;
  if (left < 0 || right < 0 || left >= kMaxDistances || right >= kMaxDistances)
    return FA_ERR_INVALID_ARG;
  return left + right + 1 <= kMaxDistances ? FA_OK : FA_ERR_UNSUPPORTED;
}

int fa_rel_line_length(int left, int right) {
  if (left < 0 || right < 0 || left >= kMaxDistances || right >= kMaxDistances ||
      left + right + 1 > kMaxDistances)
    return 0;
  return fa::RelParams{nullptr, left, right}.stride();
}

// n^a >= b^c * m^d in whole numbers of any size.
static bool power_at_least(uint32_t n, int a, uint32_t b, int c, uint32_t m, int d) {
  typedef std::vector<uint32_t> Big;  // little-endian
  auto times = [](Big& x, uint32_t y) {
    uint64_t carry = 0;
    for (uint32_t& w : x) {
      carry += static_cast<uint64_t>(w) * y;
      w = static_cast<uint32_t>(carry);
      carry >>= 32;
    }
    if (carry != 0) x.push_back(static_cast<uint32_t>(carry));
  };
  Big l(1, 1u), r(1, 1u);
  for (int i = 0; i < a; ++i) times(l, n);
  for (int i = 0; i < d; ++i) times(r, m);
  for (int i = 0; i < c; ++i) times(r, b);
  if (l.size() != r.size()) return l.size() > r.size();
  for (size_t i = l.size(); i-- > 0;)
    if (l[i] != r[i]) return l[i] > r[i];
  return true;
}

int fa_rel_buckets(int32_t* map_host, int capacity, int num_buckets, int max_distance,
                   int bidirectional, int* left) {
  const int half = bidirectional ? num_buckets / 2 : num_buckets;
  const int exact = half / 2, steps = half - exact;
  if (left == nullptr || num_buckets > 1024 || half < 2 || (bidirectional && num_buckets % 2) ||
      max_distance <= exact || max_distance >= kMaxDistances / 2)
    return 0;
  // Bucket exact + t begins at the smallest n with (n / exact)^steps >= (max_distance / exact)^t,
  // that is n^steps >= max_distance^t exact^(steps - t): a comparison of whole numbers, so that no
  // logarithm's rounding decides where a bucket begins. (Doubles say where to look first.)
  std::vector<int32_t> side;  // buckets of distances 0, 1, ... up to where the last one begins
  try {
    for (int n = 0; n < exact; ++n) side.push_back(n);
    for (int t = 1; t < steps; ++t) {
      int n = static_cast<int>(exact * std::pow(static_cast<double>(max_distance) / exact,
                                                static_cast<double>(t) / steps)) - 1;
      if (n < exact) n = exact;
      while (!power_at_least(n, steps, exact, steps - t, max_distance, t)) ++n;
      while (static_cast<int>(side.size()) < n) side.push_back(exact + t - 1);
    }
    side.push_back(half - 1);
  } catch (const std::bad_alloc&) {
    return 0;
  }
  const int reach = static_cast<int>(side.size()) - 1;
  const int total = bidirectional ? 2 * reach + 1 : reach + 1;
  *left = reach;
  if (map_host != nullptr) {
    if (capacity < total) return 0;
    for (int i = 0; i <= reach; ++i) map_host[reach - i] = side[i];
    if (bidirectional)
      for (int i = 1; i <= reach; ++i) map_host[reach + i] = half + side[i];
  }
  return total;
}

fa_status fa_rel_bias(const void* table, int table_type, const int32_t* map, int left, int right,
                      int num_buckets, int H, float* lines, void* stream) {
  fa_status st = check_lines(lines, left, right);
  if (st != FA_OK) return st;
  if (H < 1 || num_buckets < 1 || !table || !map) return FA_ERR_INVALID_ARG;
  if (table_type != FA_TABLE_F32 && table_type != FA_TABLE_BF16) return FA_ERR_UNSUPPORTED;
  if (num_buckets > kMaxDistances || H > 65535) return FA_ERR_UNSUPPORTED;
  const uintptr_t unit = table_type == FA_TABLE_F32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(table) & unit) != 0 ||
      (reinterpret_cast<uintptr_t>(map) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  fa::RelLinesArgs a;
  a.table = table;
  a.bf16 = table_type == FA_TABLE_BF16;
  a.map = map;
  a.left = left;
  a.right = right;
  a.num_buckets = num_buckets;
  a.H = H;
  a.lines = lines;
  a.status = di->status;
  return fa::launch_rel_lines(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK
                                                                                   : FA_ERR_CUDA;
}

// Checks that the calls with positions share; fills the mask and the bias.
static fa_status cross_args(int B, int H, int Hkv, int Nq, int Nk, int d, float scale, int causal,
                            int q_offset, int wl, int wr, float dropout_p,
                            const int32_t* seqlens_k, const float* lines, int left, int right,
                            fa::MaskParams* m, fa::RelParams* rel, int* mode) {
  fa_status st = check_common(B, H, Nq, d, scale, dropout_p, Hkv);
  if (st != FA_OK) return st;
  if (Nk < 1 || static_cast<long long>(B) * Hkv * Nk >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  if (Nq > kMaxAxis || Nk > kMaxAxis || q_offset > kMaxAxis || q_offset < -kMaxAxis)
    return FA_ERR_INVALID_ARG;
  if (wl < -1 || wr < -1) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(seqlens_k) & 3u) != 0) return FA_ERR_INVALID_ARG;
  // a window as wide as all positions hides nothing
  const int widest = Nq + Nk + std::abs(q_offset);
  *m = make_mask(B, H, Hkv, Nq, causal, nullptr, seqlens_k, wl >= widest ? -1 : wl,
                 wr >= widest ? -1 : wr);
  m->Nk = Nk;
  m->q_off = q_offset;
  *mode = fa::kCross;
  *rel = fa::RelParams{};
  if (lines != nullptr) {
    if ((st = check_lines(lines, left, right)) != FA_OK) return st;
    if (H > 65535) return FA_ERR_UNSUPPORTED;
    *rel = fa::RelParams{lines, left, right};
    *mode = fa::kRel;
  }
  return FA_OK;
}

fa_status fa_fwd_cross(const void* q, const void* k, const void* v, void* o, float* lse, int B,
                       int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                       int q_offset, int window_left, int window_right, float dropout_p,
                       uint64_t seed, uint64_t offset, const int32_t* seqlens_k,
                       const float* rel_lines, int rel_left, int rel_right, void* stream) {
  fa::FwdArgs a;
  fa_status st = cross_args(B, H, H_kv, Nq, Nk, d, scale, causal, q_offset, window_left,
                            window_right, dropout_p, seqlens_k, rel_lines, rel_left, rel_right,
                            &a.mask, &a.rel, &a.mode);
  if (st != FA_OK) return st;
  for (const void* p : {q, k, v, static_cast<const void*>(o)})
    if (!p || !aligned16(p)) return FA_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  CUtensorMap tq, tk, tv;
  if (!encode_map(&tq, q, B * H, Nq, d) || !encode_map(&tk, k, B * H_kv, Nk, d) ||
      !encode_map(&tv, v, B * H_kv, Nk, d))
    return FA_ERR_CUDA;
  a.drop = make_drop(dropout_p, seed, offset);
  a.sync = make_sync(di, kStallForward);
  a.scale_log2 = scale * fa::kLog2e;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  cudaError_t e = fa::launch_fwd(tq, tk, tv, a, d, a.drop.p8 > 0, di->num_sms,
                                 static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Workspace of fa_bwd_cross: D, the list of key tiles, the parts of dK and dV where key tiles are cut
// into pieces, and for the gradient of a bias table what the dQ kernel leaves of each query row, the
// near tiles' diagonal sums and the far fields' sums.
struct CrossWorkspace {
  int first, n_diag;  // near tile pairs: kt - qt = first .. first + n_diag - 1
  size_t tiles_off, part_off, rows_off, diag_off, line_off, far_off, bytes;
};
static CrossWorkspace cross_workspace(int B, int H, int Nq, int Nk, int d, int causal, int q_offset,
                                      bool grad, int left, int right) {
  CrossWorkspace w = {};
  const size_t rows = static_cast<size_t>(B) * H * Nq;
  w.tiles_off = round256(rows * sizeof(float));
  // (room for a K/V head per query head)
  const size_t tiles = static_cast<size_t>(B) * H * ((static_cast<size_t>(Nk) + fa::kTile - 1) / fa::kTile);
  w.part_off = w.tiles_off + round256((tiles + 1) * sizeof(int32_t));
  w.bytes = w.part_off;
  // pieces have two query tiles or more, and for all H_kv there are at most kMaxPieces
  const size_t k_tiles = (static_cast<size_t>(Nk) + fa::kTile - 1) / fa::kTile;
  const size_t q_tiles = (static_cast<size_t>(Nq) + fa::kTile - 1) / fa::kTile;
  if (2 * B * k_tiles <= fa::kMaxPieces && H * q_tiles >= fa::kMinCutTiles) {
    size_t units = tiles * q_tiles / 2;
    if (units > fa::kMaxPieces) units = fa::kMaxPieces;
    w.bytes += units * 2 * fa::kTile * d * sizeof(float);
  }
  if (!grad) return w;
  w.rows_off = w.bytes;
  w.diag_off = w.rows_off + round256(rows * 4 * fa::kRelRowSums * sizeof(float));
  // near: -left - 127 < 128 (kt - qt) - q_offset < right + 127, between the first and last tiles,
  // and under a causal mask not wholly to the right of the queries
  constexpr long long T = fa::kTile;
  auto floor_div = [](long long x) { return x >= 0 ? x / T : -((-x + T - 1) / T); };
  const long long n_q = (Nq + T - 1) / T, n_k = (Nk + T - 1) / T;
  long long lo = floor_div(static_cast<long long>(q_offset) - left - (T - 1)) + 1;
  long long hi = -floor_div(-(static_cast<long long>(q_offset) + right + (T - 1))) - 1;
  if (causal && hi > floor_div(static_cast<long long>(q_offset) + T - 1))
    hi = floor_div(static_cast<long long>(q_offset) + T - 1);
  if (lo < 1 - n_q) lo = 1 - n_q;
  if (hi > n_k - 1) hi = n_k - 1;
  w.first = static_cast<int>(lo);
  w.n_diag = hi < lo ? 0 : static_cast<int>(hi - lo + 1);
  w.line_off = w.diag_off + round256((static_cast<size_t>(H) * w.n_diag + fa::kRelMaxCtas) *
                                    fa::kRelDiagFloats * sizeof(float));
  w.far_off = w.line_off + round256(static_cast<size_t>(H) * (left + right + 1 + 4 * (T - 1)) *
                                    sizeof(float));
  const size_t chunks = (static_cast<size_t>(Nq) + fa::kRelRows - 1) / fa::kRelRows;
  w.bytes = w.far_off + round256(static_cast<size_t>(B) * H * chunks * 2 * sizeof(float));
  return w;
}

size_t fa_bwd_cross_workspace_size(int B, int H, int Nq, int Nk, int d, int causal, int q_offset,
                                   int rel_grad, int rel_left, int rel_right) {
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || (d != 64 && d != 128) || Nq > kMaxAxis ||
      Nk > kMaxAxis || q_offset > kMaxAxis || q_offset < -kMaxAxis ||
      static_cast<long long>(B) * H * Nq >= (1ll << 31))
    return 0;
  if (rel_grad && fa_rel_line_length(rel_left, rel_right) == 0) return 0;
  return cross_workspace(B, H, Nq, Nk, d, causal, q_offset, rel_grad != 0, rel_left, rel_right).bytes;
}

fa_status fa_bwd_cross(const void* q, const void* k, const void* v, const void* o,
                       const void* dout, const float* lse, void* dq, void* dk, void* dv, int B,
                       int H, int H_kv, int Nq, int Nk, int d, float scale, int causal,
                       int q_offset, int window_left, int window_right, float dropout_p,
                       uint64_t seed, uint64_t offset, const int32_t* seqlens_k,
                       const float* rel_lines, int rel_left, int rel_right,
                       const int32_t* rel_map, int num_buckets, float* dtable, void* workspace,
                       size_t workspace_bytes, void* stream) {
  fa::RelGradArgs g;
  fa::BwdArgs& a = g.b;
  fa_status st = cross_args(B, H, H_kv, Nq, Nk, d, scale, causal, q_offset, window_left,
                            window_right, dropout_p, seqlens_k, rel_lines, rel_left, rel_right,
                            &a.mask, &a.rel, &a.mode);
  if (st != FA_OK) return st;
  for (const void* p : {q, k, v, o, dout, static_cast<const void*>(dq),
                        static_cast<const void*>(dk), static_cast<const void*>(dv)})
    if (!p || !aligned16(p)) return FA_ERR_INVALID_ARG;
  if (!lse || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  const bool grad = dtable != nullptr;
  if (grad) {
    if (!rel_lines || !rel_map || num_buckets < 1) return FA_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(rel_map) | reinterpret_cast<uintptr_t>(dtable)) & 3u) != 0)
      return FA_ERR_INVALID_ARG;
    if (num_buckets > kMaxDistances) return FA_ERR_UNSUPPORTED;
  }
  const CrossWorkspace w = cross_workspace(B, H, Nq, Nk, d, a.mask.causal, q_offset, grad, rel_left,
                                           rel_right);
  if (workspace == nullptr || workspace_bytes < w.bytes || !aligned16(workspace))
    return FA_ERR_WORKSPACE;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  CUtensorMap m[4];
  if (!encode_map(&m[0], q, B * H, Nq, d) || !encode_map(&m[1], k, B * H_kv, Nk, d) ||
      !encode_map(&m[2], v, B * H_kv, Nk, d) || !encode_map(&m[3], dout, B * H, Nq, d))
    return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.drop = make_drop(dropout_p, seed, offset);
  a.sync = make_sync(di, kStallNone);
  a.scale = scale;
  a.scale_log2 = scale * fa::kLog2e;
  a.o = static_cast<const __nv_bfloat16*>(o);
  a.dout = static_cast<const __nv_bfloat16*>(dout);
  a.lse = lse;
  a.dsum = reinterpret_cast<float*>(ws);
  a.dq = static_cast<__nv_bfloat16*>(dq);
  a.dk = static_cast<__nv_bfloat16*>(dk);
  a.dv = static_cast<__nv_bfloat16*>(dv);
  a.row_sums = grad ? reinterpret_cast<float*>(ws + w.rows_off) : nullptr;
  a.key_tiles = seqlens_k != nullptr ? reinterpret_cast<int32_t*>(ws + w.tiles_off) : nullptr;
  a.pieces = fa::dkdv_pieces(
      static_cast<long long>(B) * H_kv * ((Nk + fa::kTile - 1) / fa::kTile),
      static_cast<long long>(H / H_kv) * ((Nq + fa::kTile - 1) / fa::kTile), di->num_sms);
  a.dkdv_part = reinterpret_cast<float*>(ws + w.part_off);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool drop = a.drop.p8 > 0;
  cudaError_t e = fa::launch_bwd_preprocess(a, d, di->num_sms, s);
  if (e == cudaSuccess) e = fa::launch_row_d(m[0], m[1], m[2], m[3], a, d, drop, di->num_sms, s);
  if (e == cudaSuccess) {
    a.sync.inject_stall = take_stall(kStallDkdv);
    e = fa::launch_bwd_dkdv(m[0], m[1], m[2], m[3], a, d, drop, di->num_sms, s);
  }
  if (e == cudaSuccess && a.pieces > 1) e = fa::launch_dkdv_merge(a, d, s);
  if (e == cudaSuccess) {
    a.sync.inject_stall = take_stall(kStallDq);
    e = fa::launch_bwd_dq(m[0], m[1], m[2], m[3], a, d, drop, di->num_sms, s);
  }
  if (e == cudaSuccess && grad) {
    a.sync.inject_stall = 0;
    g.map = rel_map;
    g.num_buckets = num_buckets;
    g.dtable = dtable;
    g.first = w.first;
    g.n_diag = w.n_diag;
    g.diag_sums = reinterpret_cast<float*>(ws + w.diag_off);
    g.line_sums = reinterpret_cast<float*>(ws + w.line_off);
    g.far_sums = reinterpret_cast<float*>(ws + w.far_off);
    e = fa::launch_rel_grad(m[0], m[1], m[2], m[3], g, d, drop, di->num_sms, s);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_fp8_workspace_size(int B, int H, int d) {
  // B*H amaxes of Q, and of K plus 128 columns of V per K/V head: at most 130 B*H
  if (B < 1 || H < 1 || d != 128) return 0;
  return round256(static_cast<size_t>(B) * H * (2 + 128) * sizeof(unsigned int));
}

int fa_fp8_vt_stride(int N) { return N < 1 ? 0 : (N + 15) / 16 * 16; }

fa_status fa_fp8_quantize_gqa(const void* q, const void* k, const void* v, const float* signs,
                              int B, int H, int Hkv, int N, int d, void* q8, void* k8, void* vt8,
                              float* s_q, float* s_k, float* s_v, void* workspace,
                              size_t workspace_bytes, void* stream) {
  if (B < 1 || H < 1 || N < 1 || Hkv < 1 || H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H * N >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  const void* ptrs[] = {q, k, v, q8, k8, vt8, s_q, s_k, s_v};  // signs may be null
  for (const void* p : ptrs)
    if (p == nullptr) return FA_ERR_INVALID_ARG;
  const void* tensors[] = {q, k, v, q8, k8, vt8};
  for (const void* p : tensors)
    if (!aligned16(p)) return FA_ERR_INVALID_ARG;
  if (workspace == nullptr || workspace_bytes < fa_fp8_workspace_size(B, H, d) ||
      !aligned16(workspace))
    return FA_ERR_WORKSPACE;
  DeviceInfo* di = nullptr;
  fa_status st = device_info(&di);
  if (st != FA_OK) return st;
  fa::Fp8QuantArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.k = static_cast<const __nv_bfloat16*>(k);
  a.v = static_cast<const __nv_bfloat16*>(v);
  a.signs = signs;
  a.B = B;
  a.H = H;
  a.Hkv = Hkv;
  a.N = N;
  a.Np = fa_fp8_vt_stride(N);
  a.amax = static_cast<unsigned int*>(workspace);
  a.q8 = static_cast<uint8_t*>(q8);
  a.k8 = static_cast<uint8_t*>(k8);
  a.vt8 = static_cast<uint8_t*>(vt8);
  a.s_q = s_q;
  a.s_k = s_k;
  a.s_v = s_v;
  return fa::launch_fp8_quantize(a, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_fwd_fp8_gqa(const void* q8, const void* k8, const void* vt8, const float* s_q,
                         const float* s_k, const float* s_v, void* o, float* lse, int B, int H,
                         int Hkv, int N, int d, float scale, int causal, const int32_t* seqlens_k,
                         void* stream) {
  fa_status st = check_common(B, H, N, d, scale, 0.f, Hkv);
  if (st != FA_OK) return st;
  if (d != 128) return FA_ERR_UNSUPPORTED;
  if (!q8 || !k8 || !vt8 || !s_q || !s_k || !s_v || !o || !lse) return FA_ERR_INVALID_ARG;
  if (!aligned16(q8) || !aligned16(k8) || !aligned16(vt8) || !aligned16(o))
    return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  const int Np = fa_fp8_vt_stride(N);
  CUtensorMap tq, tk, tv;
  if (!encode_map_u8(&tq, q8, B * H, N, 128, 128) ||
      !encode_map_u8(&tk, k8, B * Hkv, N, 128, 128) ||
      !encode_map_u8(&tv, vt8, B * Hkv, 128, Np, Np))
    return FA_ERR_CUDA;
  fa::Fp8FwdArgs a;
  a.mask = make_mask(B, H, Hkv, N, causal, nullptr, seqlens_k);
  a.sync = make_sync(di, kStallForward);
  a.scale_log2 = scale * fa::kLog2e;
  a.s_q = s_q;
  a.s_k = s_k;
  a.s_v = s_v;
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  return fa::launch_fwd_fp8(tq, tk, tv, a, di->num_sms, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_fp8_quantize(const void* q, const void* k, const void* v, const float* signs, int B,
                          int H, int N, int d, void* q8, void* k8, void* vt8, float* s_q,
                          float* s_k, float* s_v, void* workspace, size_t workspace_bytes,
                          void* stream) {
  return fa_fp8_quantize_gqa(q, k, v, signs, B, H, H, N, d, q8, k8, vt8, s_q, s_k, s_v, workspace,
                             workspace_bytes, stream);
}

fa_status fa_fwd_fp8(const void* q8, const void* k8, const void* vt8, const float* s_q,
                     const float* s_k, const float* s_v, void* o, float* lse, int B, int H, int N,
                     int d, float scale, int causal, const int32_t* seqlens_k, void* stream) {
  return fa_fwd_fp8_gqa(q8, k8, vt8, s_q, s_k, s_v, o, lse, B, H, H, N, d, scale, causal,
                        seqlens_k, stream);
}

// Shared validation of the paged calls; fills `a` on success.
static fa_status paged_args(const void* k, const void* v, const uint8_t* ks, const uint8_t* vs,
                            int type, int num_pages, int page_size, int Hkv, int d, int64_t sp,
                            int64_t sh, int64_t sr, const int32_t* table, int64_t table_stride,
                            int max_pages, const int32_t* kv_lens, const int32_t* cu, int B, int T,
                            int max_q, fa::PagedArgs* a) {
  if (num_pages < 1 || page_size < 1 || Hkv < 1 || B < 1 || T < 0 || max_pages < 1 || max_q < 0)
    return FA_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return FA_ERR_UNSUPPORTED;
  if (type != FA_CACHE_BF16 && type != FA_CACHE_E4M3) return FA_ERR_UNSUPPORTED;
  if (page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  const bool e4m3 = type == FA_CACHE_E4M3;
  if (static_cast<long long>(max_pages) * page_size >= (1ll << 31) - 256) return FA_ERR_INVALID_ARG;
  if (!k || !v || !table || !kv_lens || (e4m3 && (!ks || !vs))) return FA_ERR_INVALID_ARG;
  if (!aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
  if (e4m3 && (!aligned16(ks) || !aligned16(vs))) return FA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(table), static_cast<const void*>(kv_lens),
                        static_cast<const void*>(cu)})
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return FA_ERR_INVALID_ARG;
  const int64_t unit = e4m3 ? 16 : 8;              // elements in 16 bytes
  const int64_t most = (1ll << 40) / (e4m3 ? 1 : 2);
  for (const int64_t x : {sp, sh, sr})
    if (x < unit || x % unit != 0 || x >= most) return FA_ERR_INVALID_ARG;
  if (table_stride < max_pages) return FA_ERR_INVALID_ARG;
  if (cu == nullptr && static_cast<long long>(B) * max_q != T) return FA_ERR_INVALID_ARG;
  a->k = static_cast<uint8_t*>(const_cast<void*>(k));
  a->v = static_cast<uint8_t*>(const_cast<void*>(v));
  a->k_scale = const_cast<uint8_t*>(ks);
  a->v_scale = const_cast<uint8_t*>(vs);
  a->num_pages = num_pages;
  a->page_size = page_size;
  // 2^(s - 1) < page_size <= 2^s: m = ceil(2^(31 + s) / page_size) has 32 bits, and the excess
  // pos * (m * page_size - 2^(31 + s)) < 2^31 * page_size <= 2^(31 + s) of the product does
  // not reach the next whole quotient.
  int s = 0;
  while ((1ll << s) < page_size) ++s;
  a->page_mul = static_cast<unsigned>(((1ull << (31 + s)) + page_size - 1) / page_size);
  a->page_shift = s - 1;
  a->Hkv = Hkv;
  a->d = d;
  a->stride_page = sp;
  a->stride_head = sh;
  a->stride_row = sr;
  a->table = table;
  a->table_stride = table_stride;
  a->max_pages = max_pages;
  a->kv_lens = kv_lens;
  a->cu = cu;
  a->B = B;
  a->T = T;
  a->max_q = max_q;
  a->status = nullptr;
  return FA_OK;
}

fa_status fa_paged_write(const void* k_new, const void* v_new, void* k_pages, void* v_pages,
                         uint8_t* k_scale, uint8_t* v_scale, int type, int num_pages,
                         int page_size, int H_kv, int d, int64_t stride_page, int64_t stride_head,
                         int64_t stride_row, const int32_t* page_table, int64_t table_stride,
                         int max_pages, const int32_t* kv_lens, const int32_t* cu_seqlens_q, int B,
                         int T, int max_q, int64_t k_stride, int64_t v_stride, void* stream) {
  fa::PagedWriteArgs a;
  fa_status st = paged_args(k_pages, v_pages, k_scale, v_scale, type, num_pages, page_size, H_kv,
                            d, stride_page, stride_head, stride_row, page_table, table_stride,
                            max_pages, kv_lens, cu_seqlens_q, B, T, max_q, &a.c);
  if (st != FA_OK) return st;
  const int64_t row = static_cast<int64_t>(H_kv) * d;
  if (k_stride < row || v_stride < row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return FA_ERR_INVALID_ARG;
  if (T == 0) return FA_OK;
  if (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new)) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  a.c.status = di->status;
  a.k_new = static_cast<const __nv_bfloat16*>(k_new);
  a.v_new = static_cast<const __nv_bfloat16*>(v_new);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  cudaError_t e = fa::launch_paged_write(a, type == FA_CACHE_E4M3,
                                         static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_paged_read(const void* k_pages, const void* v_pages, const uint8_t* k_scale,
                        const uint8_t* v_scale, int type, int num_pages, int page_size, int H_kv,
                        int d, int64_t stride_page, int64_t stride_head, int64_t stride_row,
                        const int32_t* page_table, int64_t table_stride, int max_pages,
                        const int32_t* kv_lens, int B, int N, void* k_out, void* v_out,
                        void* stream) {
  fa::PagedReadArgs a;
  fa_status st = paged_args(k_pages, v_pages, k_scale, v_scale, type, num_pages, page_size, H_kv,
                            d, stride_page, stride_head, stride_row, page_table, table_stride,
                            max_pages, kv_lens, nullptr, B, 0, 0, &a.c);
  if (st != FA_OK) return st;
  if (N < 1 || !k_out || !v_out || !aligned16(k_out) || !aligned16(v_out))
    return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  a.c.status = di->status;
  a.k_out = static_cast<__nv_bfloat16*>(k_out);
  a.v_out = static_cast<__nv_bfloat16*>(v_out);
  a.N = N;
  cudaError_t e = fa::launch_paged_read(a, type == FA_CACHE_E4M3,
                                        static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

size_t fa_paged_workspace_size(int H, int H_kv, int d, int max_q, int max_keys) {
  DeviceInfo* di = nullptr;
  if (H < 1 || H_kv < 1 || H % H_kv != 0 || (d != 64 && d != 128) || max_q < 1 ||
      max_keys < 1 || device_info(&di) != FA_OK)
    return 0;
  return paged_workspace(H / H_kv, d, max_q, max_keys, di->num_sms).bytes;
}

fa_status fa_paged_attn(const void* q, const void* k_pages, const void* v_pages,
                        const uint8_t* k_scale, const uint8_t* v_scale, void* o, float* lse,
                        int type, int num_pages, int page_size, int H, int H_kv, int d,
                        int64_t stride_page, int64_t stride_head, int64_t stride_row,
                        const int32_t* page_table, int64_t table_stride, int max_pages,
                        const int32_t* kv_lens, const int32_t* cu_seqlens_q, int B, int T,
                        int max_q, int64_t q_stride, float scale, int causal, int window_left,
                        void* workspace, size_t workspace_bytes, void* stream) {
  fa::PagedAttnArgs a;
  fa_status st = paged_args(k_pages, v_pages, k_scale, v_scale, type, num_pages, page_size, H_kv,
                            d, stride_page, stride_head, stride_row, page_table, table_stride,
                            max_pages, kv_lens, cu_seqlens_q, B, T, max_q, &a.c);
  if (st != FA_OK) return st;
  if (H < 1 || H % H_kv != 0 || max_q < 1 || window_left < -1) return FA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return FA_ERR_INVALID_ARG;
  if (q_stride < static_cast<int64_t>(H) * d || q_stride % 8 != 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(T) * H >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  // positions reach from -max_q (more new tokens than positions) to the tables' room
  const long long max_keys = static_cast<long long>(max_pages) * page_size;
  if (max_keys + max_q >= (1ll << 31) - 256) return FA_ERR_INVALID_ARG;
  if (window_left >= max_keys) window_left = -1;  // hides nothing
  if (H / H_kv > 128) return FA_ERR_UNSUPPORTED;
  if (T == 0) return FA_OK;
  if (!q || !o || !lse || !aligned16(q) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  if ((st = device_info(&di)) != FA_OK) return st;
  const PagedWorkspace w = paged_workspace(H / H_kv, d, max_q, max_keys, di->num_sms);
  if (w.bytes > 0 && (workspace == nullptr || workspace_bytes < w.bytes || !aligned16(workspace)))
    return FA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.headers = ws;
  a.lse_part = w.whole ? nullptr : reinterpret_cast<float*>(ws + w.lse_off);
  a.o_part = w.whole ? nullptr : reinterpret_cast<float*>(ws + w.o_off);
  a.c.status = di->status;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.q_stride = q_stride;
  a.H = H;
  a.G = H / H_kv;
  a.tt = fa::kTile / a.G;
  a.g_magic = (65536u + static_cast<unsigned>(a.G) - 1u) / static_cast<unsigned>(a.G);
  a.o = static_cast<__nv_bfloat16*>(o);
  a.lse = lse;
  a.scale_log2 = scale * fa::kLog2e;
  a.causal = causal ? 1 : 0;
  a.wl = window_left;
  a.whole = w.whole;
  a.sync = fa::SyncParams{};
  const bool e4m3 = type == FA_CACHE_E4M3;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (w.rows <= fa::kStepRows) {
    e = fa::launch_paged_step(a, e4m3, w.ctas, cs);
  } else {
    a.sync = make_sync(di, kStallForward);
    int box = 128;  // rows of a page that a key tile can take at once
    while (page_size % box != 0) box /= 2;
    CUtensorMap tq, tk, tv;
    if (!encode_map_tokens(&tq, q, T, H, d, q_stride, a.G, a.tt) ||
        !encode_map_pages(&tk, k_pages, a.c, e4m3, box) ||
        !encode_map_pages(&tv, v_pages, a.c, e4m3, box))
      return FA_ERR_CUDA;
    e = fa::launch_paged_chunk(tq, tk, tv, a, e4m3, box, w.ctas, cs);
  }
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// The calls above from blocks of arguments; x[i] for i in `ints` are ints.
#define FA_BLOCK_INTS(...)                                                    \
  if (x == nullptr) return FA_ERR_INVALID_ARG;                                \
  for (const int i : {__VA_ARGS__})                                           \
    if (x[i] != static_cast<int32_t>(x[i])) return FA_ERR_INVALID_ARG;        \
  auto p = [&](int i) { return reinterpret_cast<void*>(x[i]); };              \
  [[maybe_unused]] auto u8 = [&](int i) { return reinterpret_cast<uint8_t*>(x[i]); };  \
  auto i32 = [&](int i) { return reinterpret_cast<const int32_t*>(x[i]); };   \
  auto n = [&](int i) { return static_cast<int>(x[i]); };

fa_status fa_paged_write_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(6, 7, 8, 9, 10, 16, 19, 20, 21)
  return fa_paged_write(p(0), p(1), p(2), p(3), u8(4), u8(5), n(6), n(7), n(8), n(9), n(10), x[11],
                        x[12], x[13], i32(14), x[15], n(16), i32(17), i32(18), n(19), n(20), n(21),
                        x[22], x[23], stream);
}

fa_status fa_paged_read_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(4, 5, 6, 7, 8, 14, 16, 17)
  return fa_paged_read(p(0), p(1), u8(2), u8(3), n(4), n(5), n(6), n(7), n(8), x[9], x[10], x[11],
                       i32(12), x[13], n(14), i32(15), n(16), n(17), p(18), p(19), stream);
}

fa_status fa_paged_attn_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(7, 8, 9, 10, 11, 12, 18, 21, 22, 23, 26, 27)
  double scale;
  memcpy(&scale, x + 25, sizeof(scale));
  if (x[29] < 0) return FA_ERR_INVALID_ARG;
  return fa_paged_attn(p(0), p(1), p(2), u8(3), u8(4), p(5), static_cast<float*>(p(6)), n(7), n(8),
                       n(9), n(10), n(11), n(12), x[13], x[14], x[15], i32(16), x[17], n(18),
                       i32(19), i32(20), n(21), n(22), n(23), x[24], static_cast<float>(scale),
                       n(26), n(27), p(28), static_cast<size_t>(x[29]), stream);
}

fa_status fa_fwd_cross_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(5, 6, 7, 8, 9, 10, 12, 13, 14, 15, 21, 22)
  double scale, drop;
  memcpy(&scale, x + 11, sizeof(scale));
  memcpy(&drop, x + 16, sizeof(drop));
  return fa_fwd_cross(p(0), p(1), p(2), p(3), static_cast<float*>(p(4)), n(5), n(6), n(7), n(8),
                      n(9), n(10), static_cast<float>(scale), n(12), n(13), n(14), n(15),
                      static_cast<float>(drop), static_cast<uint64_t>(x[17]),
                      static_cast<uint64_t>(x[18]), i32(19), static_cast<float*>(p(20)), n(21),
                      n(22), stream);
}

fa_status fa_bwd_cross_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(9, 10, 11, 12, 13, 14, 16, 17, 18, 19, 25, 26, 28)
  double scale, drop;
  memcpy(&scale, x + 15, sizeof(scale));
  memcpy(&drop, x + 20, sizeof(drop));
  if (x[31] < 0) return FA_ERR_INVALID_ARG;
  return fa_bwd_cross(p(0), p(1), p(2), p(3), p(4), static_cast<float*>(p(5)), p(6), p(7), p(8),
                      n(9), n(10), n(11), n(12), n(13), n(14), static_cast<float>(scale), n(16),
                      n(17), n(18), n(19), static_cast<float>(drop), static_cast<uint64_t>(x[21]),
                      static_cast<uint64_t>(x[22]), i32(23), static_cast<float*>(p(24)), n(25),
                      n(26), i32(27), n(28), static_cast<float*>(p(29)), p(30),
                      static_cast<size_t>(x[31]), stream);
}

fa_status fa_rel_bias_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(1, 3, 4, 5, 6)
  return fa_rel_bias(p(0), n(1), i32(2), n(3), n(4), n(5), n(6), static_cast<float*>(p(7)), stream);
}

fa_status fa_decode_rel_block(const int64_t* x, void* stream) {
  FA_BLOCK_INTS(5, 6, 7, 8, 9, 10, 12, 13, 16, 17, 18)
  double scale;
  memcpy(&scale, x + 11, sizeof(scale));
  if (x[20] < 0) return FA_ERR_INVALID_ARG;
  return fa_decode_rel(p(0), p(1), p(2), p(3), static_cast<float*>(p(4)), n(5), n(6), n(7), n(8),
                       n(9), n(10), static_cast<float>(scale), n(12), n(13), i32(14),
                       static_cast<float*>(p(15)), n(16), n(17), n(18), p(19),
                       static_cast<size_t>(x[20]), stream);
}
#undef FA_BLOCK_INTS

int fa_dropout_p8(float dropout_p) { return p8_of(dropout_p); }

fa_status fa_debug_dropout_keep(uint8_t* keep, int B, int H, int N, float dropout_p,
                                uint64_t seed, uint64_t offset, void* stream) {
  if (keep == nullptr || B < 1 || H < 1 || N < 1) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H * N >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  if (p8_of(dropout_p) < 0) return FA_ERR_INVALID_ARG;
  DeviceInfo* di = nullptr;
  fa_status st = device_info(&di);
  if (st != FA_OK) return st;
  cudaError_t e = fa::launch_debug_dropout(keep, B, H, N, make_drop(dropout_p, seed, offset),
                                           static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_debug_philox(const uint32_t* counters, uint32_t* out, int n, uint32_t key0,
                          uint32_t key1, void* stream) {
  if (counters == nullptr || out == nullptr || n < 0) return FA_ERR_INVALID_ARG;
  if (!aligned16(counters) || !aligned16(out)) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  DeviceInfo* di = nullptr;
  fa_status st = device_info(&di);
  if (st != FA_OK) return st;
  cudaError_t e =
      fa::launch_debug_philox(counters, out, n, key0, key1, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_butterfly_mask(uint8_t* mask_host, int nb) {
  if (mask_host == nullptr || nb < 1 || nb > 65536) return FA_ERR_INVALID_ARG;
  // Partner of block r at stride 2^k is r XOR 2^k; the diagonal is stride 0.
  for (int r = 0; r < nb; ++r) {
    for (int c = 0; c < nb; ++c) {
      const unsigned x = static_cast<unsigned>(r ^ c);
      mask_host[static_cast<size_t>(r) * nb + c] =
          static_cast<uint8_t>(x == 0u || (x & (x - 1u)) == 0u);
    }
  }
  return FA_OK;
}

fa_status fa_device_status(void* stream, int clear) {
  DeviceInfo* di = nullptr;
  fa_status st = device_info(&di);
  if (st != FA_OK) return st;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  unsigned int v = 0;
  if (cudaMemcpy(&v, di->status, sizeof(v), cudaMemcpyDeviceToHost) != cudaSuccess)
    return FA_ERR_CUDA;
  if (clear) {
    const unsigned int zero = 0;
    if (cudaMemcpy(di->status, &zero, sizeof(zero), cudaMemcpyHostToDevice) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return static_cast<fa_status>(v);
}

void fa_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns ? ns : 1); }

void fa_test_inject_stall(int mode) {
  g_inject_stall.store(mode >= kStallForward && mode <= kStallDq ? mode : kStallNone);
}

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported head dimension or device";
    case FA_ERR_CUDA: return "CUDA call failed";
    case FA_ERR_WORKSPACE: return "workspace missing or too small";
    case FA_ERR_TIMEOUT: return "device-side wait timed out";
  }
  return "unknown status";
}

}  // extern "C"
