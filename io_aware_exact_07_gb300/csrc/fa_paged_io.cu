// Writing new key and value rows into a paged cache, and reading a paged cache back
// into contiguous rows (IO-aware in the sense of the method: a quantised cache halves
// the bytes that attention over it, bound by reading K and V, has to move).
//
// A row is the d values of one K/V head at one position. Quantised rows are e4m3 codes
// with one power-of-two scale per row: E is the smallest exponent in [kScaleMin,
// kScaleMax] with max |x| <= 448 * 2^E (0 for a row of zeros), and the codes are
// x * 2^-E rounded to the nearest, ties to even, saturating at 448. A power of two costs
// e4m3 no precision (its significand does not depend on the scale), makes x * 2^-E and
// code * 2^E exact, so that only the one rounding to e4m3 is lost, and lets the scale be
// one byte. A row that holds a NaN or an infinity is marked by its scale byte and reads
// back as NaN.
//
// Both kernels move each byte once and compute little: HBM bounds large calls, the
// launch and three dependent loads (offsets, page table, rows) the smallest.
#include <cuda_fp8.h>

#include "fa_paged.h"

namespace fa {

namespace {

constexpr int kIoWarps = 8;
constexpr int kReadRows = 16;  // rows per warp; a page holds a multiple of it

// Exponent of the scale of a row whose largest magnitude has the bf16 bits `top`
// (finite): with top = 1.m * 2^x, 448 = 1.75 * 2^8 is exceeded from m = 97 / 128 on, where
// adding 31 carries into the exponent.
__device__ __forceinline__ int scale_exponent(uint32_t top) {
  const int e = static_cast<int>((top + 31u) >> 7) - 127 - 8;
  return top == 0u ? 0 : max(kScaleMin, min(kScaleMax, e));
}

// The codes of four bf16 values times f, f.
__device__ __forceinline__ uint32_t codes4(uint32_t a, uint32_t b, uint64_t ff) {
  float x0, x1, x2, x3;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u)), ff), x0, x1);
  f2_unpack(f2_mul(f2_pack(__uint_as_float(b << 16), __uint_as_float(b & 0xFFFF0000u)), ff), x2, x3);
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x2, x3), __NV_SATFINITE, __NV_E4M3);
  return prmt(lo, hi, 0x5410u);
}

}  // namespace

// One warp takes rows of one token: D / 8 lanes hold a row (16 bytes each), so a pass covers
// 2 (d = 128) or 4 (d = 64) of the token's 2 Hkv rows (K's heads, then V's). The rows of all
// PASSES passes are loaded first, so that they and the chain of loads that finds their place
// (offsets, length, page table) are in flight together. The blocks from `blocks` on take no
// rows: their threads look over a sequence each, since offsets and lengths out of range are to be
// reported where no token leads to them too.
template <int D, bool E4M3, int PASSES>
__global__ void __launch_bounds__(kIoWarps * 32)
    fa_paged_write_kernel(const PagedWriteArgs a, int warps_per_token, unsigned blocks) {
  constexpr int kLanes = D / 8;
  constexpr int kRows = 32 / kLanes;
  const int lane = threadIdx.x & 31;
  if (blockIdx.x >= blocks) {
    const unsigned b = (blockIdx.x - blocks) * (kIoWarps * 32) + threadIdx.x;
    if (b < static_cast<unsigned>(a.c.B)) paged_seq(a.c, static_cast<int>(b));
    return;
  }
  const long long task = static_cast<long long>(blockIdx.x) * kIoWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(task / warps_per_token);
  const int sub = static_cast<int>(task - static_cast<long long>(t) * warps_per_token);
  if (t >= a.c.T) return;
  const int u = lane % kLanes;  // 16-byte unit of the row
  const int r0 = sub * PASSES * kRows + lane / kLanes;
  uint4 x[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = r0 + i * kRows;
    const bool is_v = r >= a.c.Hkv;
    x[i] = make_uint4(0u, 0u, 0u, 0u);
    if (r < 2 * a.c.Hkv)
      x[i] = *reinterpret_cast<const uint4*>((is_v ? a.v_new + t * a.v_stride : a.k_new + t * a.k_stride) +
                                             (is_v ? r - a.c.Hkv : r) * D + u * 8);
  }
  const int b = paged_find_seq(a.c, t);
  if (b >= a.c.B) return;  // a token behind the last sequence
  const PagedSeq s = paged_seq(a.c, b);
  const int pos = s.len - s.nq + (t - s.t0);
  if (t < s.t0 || t >= s.t0 + s.nq || pos < 0) return;
  const int page = paged_page(a.c, b, pos);
  if (page < 0) return;
  const int slot = page_row(a.c, pos);
  const long long at0 = page * a.c.stride_page + slot * a.c.stride_row + u * 8;
  const long long scale0 = static_cast<long long>(page) * a.c.Hkv * a.c.page_size + slot;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = r0 + i * kRows;
    const bool real = r < 2 * a.c.Hkv;
    const bool is_v = r >= a.c.Hkv;
    const int h = is_v ? r - a.c.Hkv : r;
    const long long at = at0 + h * a.c.stride_head;
    uint8_t* base = is_v ? a.c.v : a.c.k;
    if constexpr (!E4M3) {
      if (real) *reinterpret_cast<uint4*>(base + at * 2) = x[i];
    } else {
      constexpr uint32_t kAbs = 0x7FFF7FFFu;
      uint32_t m2 = __vimax3_u16x2(x[i].x & kAbs, x[i].y & kAbs, x[i].z & kAbs);
      m2 = __vmaxu2(m2, x[i].w & kAbs);
      uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
      if constexpr (kLanes == 16) {  // a row each for the halves of the warp
        const uint32_t lo = __reduce_max_sync(0xffffffffu, lane < 16 ? top : 0u);
        const uint32_t hi = __reduce_max_sync(0xffffffffu, lane < 16 ? 0u : top);
        top = lane < 16 ? lo : hi;
      } else {
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const bool finite = top < 0x7F80u;
      const int e = finite ? scale_exponent(top) : 0;
      const uint64_t ff = f2_pack(pow2i(-e), pow2i(-e));
      uint2 w = make_uint2(codes4(x[i].x, x[i].y, ff), codes4(x[i].z, x[i].w, ff));
      if (!finite) w = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
      if (real) {
        *reinterpret_cast<uint2*>(base + at) = w;
        if (u == 0)
          (is_v ? a.c.v_scale : a.c.k_scale)[scale0 + static_cast<long long>(h) * a.c.page_size] =
              static_cast<uint8_t>(finite ? e + 127 : kScaleNaN);
      }
    }
  }
}

// One warp copies kReadRows positions of one K/V head, which lie in one page.
template <int D, bool E4M3>
__global__ void __launch_bounds__(kIoWarps * 32) fa_paged_read_kernel(const PagedReadArgs a,
                                                                      int groups) {
  const int lane = threadIdx.x & 31;
  long long task = static_cast<long long>(blockIdx.x) * kIoWarps + (threadIdx.x >> 5);
  const int g = static_cast<int>(task % groups);
  task /= groups;
  const int h = static_cast<int>(task % a.c.Hkv);
  task /= a.c.Hkv;
  const int b = static_cast<int>(task >> 1);
  if (b >= a.c.B) return;
  const bool is_v = (task & 1) != 0;
  const int j0 = g * kReadRows;
  const int len = paged_seq(a.c, b).len;
  const int page = j0 < len ? paged_page(a.c, b, j0) : -1;
  const int slot = page_row(a.c, j0);
  // rows of this group that the cache holds; the others are written as zeros
  const int have = page < 0 ? 0 : min(kReadRows, len - j0);
  const int rows = min(kReadRows, a.N - j0);
  const long long src = page * a.c.stride_page + h * a.c.stride_head + slot * a.c.stride_row;
  __nv_bfloat16* dst = (is_v ? a.v_out : a.k_out) +
                       ((static_cast<long long>(b) * a.c.Hkv + h) * a.N + j0) * D;
  const uint8_t* base = is_v ? a.c.v : a.c.k;
  if constexpr (!E4M3) {
    constexpr int kUnits = D / 8;                    // 16-byte units of a row
    constexpr int kPasses = kReadRows * kUnits / 32;
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = (i * 32 + lane) / kUnits, u = lane % kUnits;
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (r < have)
        x[i] = *reinterpret_cast<const uint4*>(base + (src + r * a.c.stride_row + u * 8) * 2);
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = (i * 32 + lane) / kUnits, u = lane % kUnits;
      if (r < rows) *reinterpret_cast<uint4*>(dst + r * D + u * 8) = x[i];
    }
  } else {
    constexpr int kUnits = D / 8;                    // 8-byte units of a row of codes
    constexpr int kPasses = kReadRows * kUnits / 32;
    const uint8_t* scales = (is_v ? a.c.v_scale : a.c.k_scale) +
                            (static_cast<long long>(page) * a.c.Hkv + h) * a.c.page_size + slot;
    uint2 x[kPasses];
    int sc[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = (i * 32 + lane) / kUnits, u = lane % kUnits;
      x[i] = make_uint2(0u, 0u);
      sc[i] = 127;
      if (r < have) {
        x[i] = *reinterpret_cast<const uint2*>(base + src + r * a.c.stride_row + u * 8);
        sc[i] = scales[r];
      }
    }
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int r = (i * 32 + lane) / kUnits, u = lane % kUnits;
      const uint32_t f = e4m3_factor(sc[i]);
      if (r < rows)
        *reinterpret_cast<uint4*>(dst + r * D + u * 8) = make_uint4(
            e4m3_lo(x[i].x, f), e4m3_hi(x[i].x, f), e4m3_lo(x[i].y, f), e4m3_hi(x[i].y, f));
    }
  }
}

namespace {

template <int D, bool E4M3, int PASSES>
cudaError_t launch_write(const PagedWriteArgs& a, cudaStream_t stream) {
  constexpr int kRows = PASSES * 256 / D;  // rows of a warp
  const int warps_per_token = (2 * a.c.Hkv + kRows - 1) / kRows;
  const long long blocks = (static_cast<long long>(a.c.T) * warps_per_token + kIoWarps - 1) / kIoWarps;
  const long long checks = (a.c.B + kIoWarps * 32ll - 1) / (kIoWarps * 32);
  if (blocks + checks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  fa_paged_write_kernel<D, E4M3, PASSES>
      <<<static_cast<unsigned>(blocks + checks), kIoWarps * 32, 0, stream>>>(
          a, warps_per_token, static_cast<unsigned>(blocks));
  return cudaGetLastError();
}

// A warp takes 16 rows of 128 values or 64 at once where that leaves some ten warps for each
// SM, and as few as it can where the rows have to spread over the SMs. 18300 tokens of 8 heads
// to e4m3 with 1, 2, 4, 8, 16 passes, d = 128: 47, 29, 25, 25, 43 us (23 now, of 17 that the bytes
// take: the quantising instructions and a chain of loads per warp bound it; bf16 23 of 22); with 1
// and 8 passes 2400 tokens take 6.6 and 5.3 us, 1200 tokens 4.2 and 4.3.
template <int D, bool E4M3>
cudaError_t launch_write(const PagedWriteArgs& a, cudaStream_t stream) {
  const long long rows = 2ll * a.c.T * a.c.Hkv;
  return rows >= 32768 ? launch_write<D, E4M3, D / 16>(a, stream) : launch_write<D, E4M3, 1>(a, stream);
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteArgs& a, bool e4m3, cudaStream_t stream) {
  if (a.c.T <= 0) return cudaSuccess;
  if (a.c.d == 64)
    return e4m3 ? launch_write<64, true>(a, stream) : launch_write<64, false>(a, stream);
  return e4m3 ? launch_write<128, true>(a, stream) : launch_write<128, false>(a, stream);
}

cudaError_t launch_paged_read(const PagedReadArgs& a, bool e4m3, cudaStream_t stream) {
  const int groups = (a.N + kReadRows - 1) / kReadRows;
  const long long tasks = 2ll * a.c.B * a.c.Hkv * groups;
  const long long blocks = (tasks + kIoWarps - 1) / kIoWarps;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  auto kern = a.c.d == 64 ? (e4m3 ? fa_paged_read_kernel<64, true> : fa_paged_read_kernel<64, false>)
                          : (e4m3 ? fa_paged_read_kernel<128, true> : fa_paged_read_kernel<128, false>);
  kern<<<static_cast<unsigned>(blocks), kIoWarps * 32, 0, stream>>>(a, groups);
  return cudaGetLastError();
}

}  // namespace fa
