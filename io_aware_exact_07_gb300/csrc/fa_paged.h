// Internal interface between the C-ABI layer (fa_api.cu) and the kernels over a
// paged key/value cache, and the device code they share: where a sequence's new
// tokens stand, which page holds a position, and the e4m3 rows of a quantised cache.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "fa_common.cuh"

namespace fa {

constexpr unsigned kStatusInvalid = 1u;  // a length, offset or page number out of range

// The exponent E of an e4m3 row's power-of-two scale lies in [kScaleMin, kScaleMax]
// and is stored as E + 127; byte kScaleNaN marks a row that held a NaN or an infinity.
constexpr int kScaleMin = -117;
constexpr int kScaleMax = 7;
constexpr int kScaleNaN = 255;

// A paged cache and the batch of sequences in it (pointers are device pointers).
// Page p holds, for each K/V head h, page_size rows of d values: row r starts at
// element p * stride_page + h * stride_head + r * stride_row of k and of v.
struct PagedArgs {
  uint8_t* k;                   // bf16 values or e4m3 codes
  uint8_t* v;
  uint8_t* k_scale;             // [num_pages, Hkv, page_size] scale bytes (e4m3), else null
  uint8_t* v_scale;
  int num_pages, page_size, Hkv, d;
  unsigned page_mul;            // pos / page_size = pos * page_mul >> 32 + page_shift,
  int page_shift;               // 0 <= pos < 2^31
  long long stride_page, stride_head, stride_row;  // in elements
  const int32_t* table;         // [B, max_pages], row b at b * table_stride
  long long table_stride;
  int max_pages;
  const int32_t* kv_lens;       // [B] lengths, the new tokens included
  const int32_t* cu;            // [B + 1] first new token of each sequence, or null: max_q each
  int B, T, max_q;
  unsigned int* status;         // device status word
};

// New tokens [t0, t0 + nq) of a sequence of len positions: token t0 + i stands at
// position len - nq + i.
struct PagedSeq {
  int t0, nq, len;
};

// Offsets that do not lie in order within [0, T] leave the sequence without new
// tokens, and a length outside [0, max_pages * page_size] counts as 0; both are recorded.
__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs& a, int b) {
  PagedSeq s;
  if (a.cu == nullptr) {
    s.t0 = b * a.max_q;
    s.nq = a.max_q;
  } else {
    const int lo = a.cu[b], hi = a.cu[b + 1];
    s.t0 = lo;
    s.nq = hi - lo;
    if (lo < 0 || hi < lo || hi > a.T) {
      record_error(a.status, kStatusInvalid);
      s.t0 = s.nq = 0;
    }
  }
  s.len = a.kv_lens[b];
  if (s.len < 0 || s.len > a.max_pages * a.page_size) {
    record_error(a.status, kStatusInvalid);
    s.len = 0;
  }
  return s;
}

// The same for attention, whose caller bounds the new tokens of a sequence by max_q: one
// with more has none (recorded).
__device__ __forceinline__ PagedSeq paged_attn_seq(const PagedArgs& a, int b) {
  PagedSeq s = paged_seq(a, b);
  if (s.nq > a.max_q) {
    record_error(a.status, kStatusInvalid);
    s.nq = 0;
  }
  return s;
}

__device__ __forceinline__ int page_index(const PagedArgs& a, int pos) {
  return static_cast<int>(__umulhi(static_cast<unsigned>(pos), a.page_mul) >> a.page_shift);
}
// Row of position pos >= 0 in its page.
__device__ __forceinline__ int page_row(const PagedArgs& a, int pos) {
  return pos - page_index(a, pos) * a.page_size;
}

// Page that holds position pos of sequence b, or -1 (recorded) where the table
// names none of the pool's pages.
__device__ __forceinline__ int paged_page(const PagedArgs& a, int b, int pos) {
  const int p = a.table[b * a.table_stride + page_index(a, pos)];
  if (p >= 0 && p < a.num_pages) return p;
  record_error(a.status, kStatusInvalid);
  return -1;
}

// Sequence of new token t: the number of sequences whose tokens end at or before it,
// counted by the whole (converged) warp; B for a token behind the last sequence.
__device__ __forceinline__ int paged_find_seq(const PagedArgs& a, int t) {
  if (a.cu == nullptr) return t / a.max_q;
  int n = 0;
  for (int b = threadIdx.x & 31; b < a.B; b += 32) n += a.cu[b + 1] <= t;
  return static_cast<int>(__reduce_add_sync(0xffffffffu, static_cast<unsigned>(n)));
}

// bf16 pair (f, f) of the factor 2^(120 + E) that turns the bits of e4m3_bits() into
// the values code * 2^E; a NaN for a row marked kScaleNaN. Bytes above kScaleMax + 127,
// which no written row has, count as that.
__device__ __forceinline__ uint32_t e4m3_factor(int scale_byte) {
  const int s = scale_byte < kScaleMax + 127 ? scale_byte : kScaleMax + 127;
  return scale_byte == kScaleNaN ? 0x7FC07FC0u : static_cast<uint32_t>((s + 120) << 7) * 0x10001u;
}

// Two e4m3 codes, in the high byte of each half of x (the low bytes do not matter), as
// bf16 bits of value * 2^-120: the sign stays, the four exponent and three mantissa bits
// move to the low end of bf16's exponent and the high end of its mantissa. Exact for
// e4m3's subnormals too, which become bf16 subnormals.
__device__ __forceinline__ uint32_t e4m3_bits(uint32_t x) {
  return (x & 0x80008000u) | ((x >> 4) & 0x07F007F0u);
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Codes 0, 1 (lo) and 2, 3 (hi) of a word as bf16 pairs of code * 2^E. The product is
// exact: a code has four significant bits, and code * 2^E is a normal bf16 for every E
// of a written row.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w, uint32_t factor) {
  return mul_bf16x2(e4m3_bits(prmt(w, 0u, 0x1404u)), factor);
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w, uint32_t factor) {
  return mul_bf16x2(e4m3_bits(prmt(w, 0u, 0x3424u)), factor);
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t saddr) {
  uint2 r;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(saddr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t saddr) {
  uint32_t r;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(saddr) : "memory");
  return r;
}

__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t saddr) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(saddr) : "memory");
  return r;
}
__device__ __forceinline__ void st_shared_u32(uint32_t saddr, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(a) : "memory");
}
__device__ __forceinline__ void st_shared_v2(uint32_t saddr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(saddr), "r"(a), "r"(b) : "memory");
}
// Copies 16 bytes into shared memory, or fills them with zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}

// The four e4m3 codes of a word as f16 pairs, exactly (f16 holds every e4m3 value).
__device__ __forceinline__ void e4m3_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float pow2i(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

struct PagedWriteArgs {
  PagedArgs c;
  const __nv_bfloat16* k_new;   // token t at t * k_stride, heads and d contiguous
  const __nv_bfloat16* v_new;
  long long k_stride, v_stride;
};
struct PagedReadArgs {
  PagedArgs c;
  __nv_bfloat16* k_out;         // [B, Hkv, N, d]
  __nv_bfloat16* v_out;
  int N;
};
struct PagedAttnArgs {
  PagedArgs c;
  const __nv_bfloat16* q;       // token t at t * q_stride, [H, d] contiguous
  long long q_stride;
  int H;
  int G, tt;                    // H / Hkv; tokens of a 128-row query tile, 128 / G
  unsigned g_magic;             // ceil(2^16 / G): r / G = r * g_magic >> 16 for r < 128
  __nv_bfloat16* o;             // [T, H, d]
  float* lse;                   // [T, H]
  float scale_log2;             // scale * log2(e)
  int causal;
  int wl;                       // sliding window (-1: none)
  int whole;                    // step kernel: no head is cut between CTAs
  // Workspace of calls whose work is cut between CTAs: a header per CTA and two pieces,
  // each of `rows` query rows: o_part [ctas, 2, rows, d], lse_part [ctas, 2, rows] (log2).
  void* headers;                // [ctas] int4
  float* o_part;
  float* lse_part;
  SyncParams sync;
};
constexpr int kStepRows = 24;   // most query rows per K/V head of the step kernel
// Page tables with room for so many keys: heads are not cut, and neither the merge nor its
// workspace is needed (8 sequences, 4 K/V heads, d = 64, cut and whole: up to 512 keys 9.3 and
// 7.8 us, up to 1000 9.0 and 9.6, 2000 10.4 and 13.9).
constexpr int kWholeKeys = 512;

cudaError_t launch_paged_write(const PagedWriteArgs& a, bool e4m3, cudaStream_t stream);
cudaError_t launch_paged_read(const PagedReadArgs& a, bool e4m3, cudaStream_t stream);
cudaError_t launch_paged_step(const PagedAttnArgs& a, bool e4m3, int ctas, cudaStream_t stream);
// tq: [T, H, d] with boxes of (64 columns, H / Hkv heads, 128 / (H / Hkv) tokens); tk, tv:
// [num_pages, Hkv, page_size, d] with boxes of 64 bf16 columns or d codes times box_rows rows.
cudaError_t launch_paged_chunk(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                               const PagedAttnArgs& a, bool e4m3, int box_rows, int ctas,
                               cudaStream_t stream);

}  // namespace fa
