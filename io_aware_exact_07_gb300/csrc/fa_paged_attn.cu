// Attention of new tokens over a paged key/value cache, in its simplest form: one warp
// per query row (token and head) walks the keys it sees with the online softmax
// (running maximum m and sum l; the page "Attention Kernel", section on FlashAttention's
// IO-aware insight), the row's d values spread over the lanes. Bound by the shuffles of
// each key's dot product.
#include "fa_paged.h"

namespace fa {

namespace {
constexpr int kWarps = 8;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) fa_paged_attn_kernel(const PagedAttnArgs a) {
  constexpr int kPer = D / 32;  // columns per lane
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int t = static_cast<int>(row / a.H), h = static_cast<int>(row % a.H);
  if (t >= a.c.T) return;
  const int b = paged_find_seq(a.c, t);
  if (b >= a.c.B) return;
  const PagedSeq s = paged_attn_seq(a.c, b);
  if (t < s.t0 || t >= s.t0 + s.nq) return;
  const int pos = s.len - s.nq + (t - s.t0);
  const int hi = a.causal ? min(s.len, pos + 1) : s.len;
  const int lo = a.wl >= 0 ? max(0, pos - a.wl) : 0;
  const int hk = h / (a.H / a.c.Hkv);
  auto load = [&](const uint8_t* base, const uint8_t* scales, int page, int slot, float* x) {
    const long long at = page * a.c.stride_page + hk * a.c.stride_head + slot * a.c.stride_row + lane * kPer;
    if constexpr (E4M3) {
      const uint32_t f = e4m3_factor(scales[(static_cast<long long>(page) * a.c.Hkv + hk) * a.c.page_size + slot]);
      uint32_t w = 0;
      for (int i = 0; i < kPer; ++i) w |= static_cast<uint32_t>(base[at + i]) << (8 * i);
      const uint32_t p0 = e4m3_lo(w, f), p1 = e4m3_hi(w, f);
      x[0] = __uint_as_float(p0 << 16);
      x[1] = __uint_as_float(p0 & 0xFFFF0000u);
      if constexpr (kPer == 4) {
        x[2] = __uint_as_float(p1 << 16);
        x[3] = __uint_as_float(p1 & 0xFFFF0000u);
      }
    } else {
      for (int i = 0; i < kPer; ++i)
        x[i] = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(base)[at + i]);
    }
  };
  float q[kPer], o[kPer], x[kPer];
  for (int i = 0; i < kPer; ++i) {
    q[i] = __bfloat162float(a.q[t * a.q_stride + h * D + lane * kPer + i]);
    o[i] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int j = lo; j < hi; ++j) {
    const int page = paged_page(a.c, b, j), slot = j % a.c.page_size;
    for (int i = 0; i < kPer; ++i) x[i] = 0.f;
    if (page >= 0) load(a.c.k, a.c.k_scale, page, slot, x);
    float z = 0.f;
    for (int i = 0; i < kPer; ++i) z += q[i] * x[i];
    for (int k = 16; k > 0; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
    z *= a.scale_log2;
    const float mn = fmaxf(m, z), alpha = exp2f(m - mn), p = exp2f(z - mn);
    for (int i = 0; i < kPer; ++i) x[i] = 0.f;
    if (page >= 0) load(a.c.v, a.c.v_scale, page, slot, x);
    for (int i = 0; i < kPer; ++i) o[i] = o[i] * alpha + p * x[i];
    l = l * alpha + p;
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < kPer; ++i)
    a.o[(static_cast<long long>(t) * a.H + h) * D + lane * kPer + i] = __float2bfloat16(o[i] * inv);
  if (lane == 0)
    a.lse[static_cast<long long>(t) * a.H + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

cudaError_t launch_paged_attn(const PagedAttnArgs& a, bool e4m3, cudaStream_t stream) {
  const long long rows = static_cast<long long>(a.c.T) * a.H;
  const long long blocks = (rows + kWarps - 1) / kWarps;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
  auto kern = a.c.d == 64 ? (e4m3 ? fa_paged_attn_kernel<64, true> : fa_paged_attn_kernel<64, false>)
                          : (e4m3 ? fa_paged_attn_kernel<128, true> : fa_paged_attn_kernel<128, false>);
  kern<<<static_cast<unsigned>(blocks), kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace fa
