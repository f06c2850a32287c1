// Attention of few new tokens per sequence over a paged cache (a decode step: one new
// token, or a handful of drafted ones): at most 24 query rows per K/V head, G = H / Hkv
// heads times nq tokens. The page "FlashAttention — L3 Cross-Paper Synthesis" (section 3)
// names this case, bound by reading K and V, as left unoptimised. HBM is the bound, so the
// kernel is a stream of K and V through shared memory, each byte read once per K/V head:
//
//  - Every warp is on its own: it takes 16 or 32 keys of each block of keys, brings their K and
//    V rows into its own ring of stages with cp.async, and keeps its own softmax state, so
//    that the main loop has no block barrier and loads run ahead across heads and sequences.
//    16 keys lie in one page (its size is a multiple of 16), so one table entry serves them.
//  - S^T = K Q^T and O^T += V^T P^T with m16n8k16 products: the keys (then the columns of V)
//    are the 16 rows, the query rows the 8 columns (1 to 3 times). With so few query rows
//    the products are below what bounds the kernel (a 128-row tensor-memory tile would be
//    three quarters empty, and its softmax walks all of it); keeping S and P in registers
//    saves the handshakes that a short sequence cannot hide. With more rows the products, some
//    7 cycles each and SM, come near what the bytes take, and e4m3 is bound by them and the
//    conversion. us, and those of the bytes, 24 sequences of 8192 keys, 8 K/V heads, 16 and 24
//    rows: d = 128 bf16 129 and 136 of 119, e4m3 92 and 112 of 60; d = 64 71 and 77 of 60, 61 and
//    73 of 30. The border of 24 rows was measured when e4m3 took 10 to 20 % more than now; here and
//    with 128-row tiles, 24 rows: d = 128, 8192 bf16 keys 138 and 132, 1024 keys 35 and 38, e4m3
//    122 and 147, 34 and 50; d = 64 79 and 82, 22 and 31, e4m3 86 and 107; 128 sequences of 200
//    keys 48 and 55, 4 of 3000 13 and 17. 32 rows: 8192 keys 156 and 133, 1024 44 and 38, e4m3 160
//    and 148, d = 64 94 and 82, 128 of 200 keys 60 and 55.
//  - The order of the columns d within a product is free as long as both operands share
//    it: a thread takes the 16 bytes of a row that it can load at once.
//  - e4m3 codes become f16 between shared memory and the product, which the hardware converts
//    exactly; the products run in f16, with Q scaled by a power of two per row to fit. A key's
//    K scale goes to its score, its V scale to its weight: P carries it (and the running
//    maximum counts it), the softmax's sum takes it out again. Turning the codes into bf16
//    with their scales, by integer operations, takes 2.5 instructions a code instead of 0.6.
//  - The (sequence, K/V head, key block) list is cut into equal runs, one per CTA, by
//    the lengths found on the device. A head that falls into one run is written directly;
//    one cut by a run's end leaves normalised pieces, merged by a second, small kernel with
//    the two-block rule of the online softmax. Where the page table has room for few keys,
//    runs are of whole heads and there is nothing to merge.
#include "fa_paged_plan.cuh"

namespace fa {

namespace {

constexpr int kGroup = 16;                  // keys of a product, which lie in one page
constexpr int kMergeWarps = 8;
constexpr int kSmemMax = 232448;
// A multiple of 16 that no length reaches (they stay below 2^31 - 256), and from which a warp's
// keys of a block can be counted on in 32 bits.
constexpr unsigned kFarKey = 0x7FFFFF00u;
// A quantised cache's maxima count V's scales (2^-117 .. 2^7), its sums do not: a weight may be
// 2^-133 of the largest and still count for 2^-9 of the sum. So weights are computed times 2^kUp,
// which fp32 has room for above the 2^15 of f16; only what is below 2^-49 of the sum then falls
// below 2^-126. (Exponentials of their own for keys with small scales, behind a test in every
// step, cost 2 to 4 % with 9 rows and more, this 1 %.) The sum is held times 2^-kDown: its terms
// are 2^132 at most (a weight of 2^15 with a scale of 2^-117), a row's largest is 1 at least, and
// 2^31 of them stay in range.
constexpr int kUp = 40, kDown = 40;

template <int D, bool E4M3, int NT>
struct StepL {
  // More warps hide the latency of a warp's chain of steps where its keys are few bytes, as
  // far as registers and the merge buffer leave room. 16 sequences of 16384 keys, 8 K/V heads,
  // 4 rows with 8, 12, 16 warps: e4m3 d = 128 112, 96, 97 us; bf16 d = 64 91, 91, 87; bf16 d =
  // 128 with 8: 160; e4m3 d = 64 (kU = 2) with 12, 16: 59, 58, and 128 of 200 keys 21, 23.5. 24
  // of 8192 keys, 20 rows, d = 64: 95, 89, 152.
  static constexpr int kWarps = NT >= 2 ? (D == 64 ? 12 : 8) : E4M3 ? 12 : D == 64 ? 16 : 8;
  static constexpr int kThreads = kWarps * 32;
  // Groups of a warp's step. From codes to O a group is a long chain, of which a scheduler's
  // three warps hide too little: two at once overlap, and share the vote, the walk and the
  // waits. e4m3, 16 sequences of 16384 keys, 8 K/V heads, one and two groups: 4 rows, d = 128 94
  // and 88 us, d = 64 71 and 60; 16 rows 135 and 112, 89 and 74; 24 rows 149 and 134, 105 and 87.
  // (bf16, d = 64, whose bytes bound it, gains nothing; at d = 128 there is no room.)
  static constexpr int kU = E4M3 ? 2 : 1;
  static constexpr int kChunk = kU * kGroup;
  static constexpr int kBlock = kWarps * kChunk;          // keys of a block
  static constexpr int kRows = 8 * NT;                    // query rows
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int kUnits = kRowBytes / 16;           // 16-byte units of a row
  static constexpr int kGroupBytes = kGroup * kRowBytes;  // 16 K rows, or V rows
  static constexpr int kTileBytes = kU * kGroupBytes;     // those of a step
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kScaleBytes = E4M3 ? 32 * kU : 0;  // K's and V's scale bytes, 16 each a group
  static constexpr int kPitch = D + 4;                    // merge buffer row, in floats
  // From 17 rows on Q lies in shared memory, one copy for all warps. Where the merge's buffer
  // would leave no room for the ring, two warps first join their states in registers, and it
  // takes half (20 rows, d = 64, where it fits without: 58.6 us, with 62.4).
  static constexpr bool kQShared = NT == 3;
  static constexpr int kFold = kU == 2 || (NT == 3 && kRowBytes == 256) ? 2 : 1;
  static constexpr int kStates = kWarps / kFold;
  static constexpr int kQBytes = kQShared ? kRows * (D * 2 + 4) : 0;  // rows, and their exponents
  static constexpr int kMergeBytes = kStates * kRows * kPitch * 4;
  static constexpr int kMlBytes = kWarps * kRows * 8;
  static constexpr int kFixed = kMergeBytes + kMlBytes + kQBytes + 256;
  static constexpr int kFit = (kSmemMax - kFixed) / (kWarps * (kStageBytes + kScaleBytes));
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  static_assert(kStages >= 2, "the ring needs two stages");
  static constexpr int kRingOff = 0;
  static constexpr int kScaleOff = kWarps * kStages * kStageBytes;
  static constexpr int kMergeOff = kScaleOff + kWarps * kStages * kScaleBytes;
  static constexpr int kMlOff = kMergeOff + kMergeBytes;
  static constexpr int kQOff = kMlOff + kMlBytes;
  static constexpr int kPlanOff = kQOff + kQBytes;
  static constexpr int kSmemBytes = kPlanOff + 256;
  static_assert(kSmemBytes <= kSmemMax, "more shared memory than one CTA may hold");
  static_assert(kChunk <= 0x7FFFFFFF - kFarKey, "keys of a step beyond 31 bits");
};

// Where unit `u` (16 bytes) of row `row` lies in a tile. The exclusive-or spreads the rows
// that one load instruction touches over all banks: K rows come in pairs (2 p, 2 p + 1),
// 4 units each; V as eight rows with one unit each (bf16), or as four rows (2 c) with two
// units each (e4m3). At e4m3 and d = 64, where a row has 4 units, V's even rows come first.
template <int D, bool E4M3>
__device__ __forceinline__ int k_unit(int row, int u) {
  if constexpr (!E4M3) return row * (D / 8) + (u ^ (((row & 1) << 2) | ((row >> 1) & 3)));
  if constexpr (D == 128) return row * 8 + (u ^ ((row & 1) << 2));
  return row * 4 + u;
}
template <int D, bool E4M3>
__device__ __forceinline__ int v_unit(int row, int u) {
  if constexpr (!E4M3) return row * (D / 8) + (u ^ (((row & 1) << 2) | ((row >> 1) & 3)));
  if constexpr (D == 128) return row * 8 + (u ^ (((row >> 1) & 3) << 1));
  const int slot = (row >> 1) | ((row & 1) << 3);
  return slot * 4 + (u ^ (((slot >> 1) & 1) << 1));
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float* c, uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ int ld_shared_u8(uint32_t saddr) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(saddr) : "memory");
  return static_cast<int>(r);
}

// The factor 2^x, x <= 0, of a softmax sum, and of the products with V that go with it. The
// maxima of a quantised cache count V's scales, its sums do not: 2^x may be below 2^-126 and
// still leave something of a sum, so there it is applied in two halves.
template <bool HALVES>
struct Factor {
  float part;
  __device__ __forceinline__ explicit Factor(float x) : part(ex2_approx(HALVES ? 0.5f * x : x)) {}
  __device__ __forceinline__ float all() const { return HALVES ? part * part : part; }
  __device__ __forceinline__ float of(float sum) const {
    return HALVES ? sum * part * part : sum * part;
  }
};

// Key blocks [first, first + n) of a sequence that hold a key some new token sees: with a
// sliding window the first token sees the lowest. A sequence with new tokens has at least
// one block (its rows have to be written), one without has none.
struct Span {
  int first, n;
};
template <int kBlock>
__device__ __forceinline__ Span span_of(const PagedAttnArgs& a, const PagedSeq& s) {
  Span r;
  const int lo = a.wl >= 0 ? s.len - s.nq - a.wl : 0;
  r.first = lo > 0 ? lo / kBlock : 0;
  r.n = (s.len - 1) / kBlock + 1 - r.first;  // (len + kBlock - 1 may have 33 bits)
  if (r.n < 1) r.n = 1;
  if (s.nq <= 0) r.n = 0;
  return r;
}

// A place in the list of (sequence, K/V head, key block).
template <int kBlock>
struct Walk {
  int b, h;          // sequence (B past the end), K/V head
  int blk, end;      // key block, end of the sequence's blocks
  int first;
  PagedSeq s;
  __device__ __forceinline__ void load(const PagedAttnArgs& a) {
    s = paged_attn_seq(a.c, b);
    const Span sp = span_of<kBlock>(a, s);
    first = sp.first;
    end = first + sp.n;
  }
  // Next place; past the last sequence an empty one that is never left.
  __device__ __forceinline__ void next(const PagedAttnArgs& a) {
    if (b >= a.c.B || ++blk < end) return;
    if (++h == a.c.Hkv) {
      h = 0;
      do {
        ++b;
        if (b >= a.c.B) {
          s.nq = s.len = first = blk = 0;
          end = 0x7FFFFFFF;
          return;
        }
        load(a);
      } while (first == end);
    }
    blk = first;
  }
};

}  // namespace

template <int D, bool E4M3, int NT>
__global__ void __launch_bounds__(StepL<D, E4M3, NT>::kThreads, 1) fa_paged_step_kernel(const PagedAttnArgs a) {
  using L = StepL<D, E4M3, NT>;
  using Walk = Walk<L::kBlock>;
  constexpr int kWarps = L::kWarps, kThreads = L::kThreads, kBlock = L::kBlock;
  constexpr int kU = L::kU, kChunk = L::kChunk;
  extern __shared__ __align__(1024) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g8 = lane >> 2, c4 = lane & 3;
  const int G = a.G;
  pdl_launch_dependents();

  // ---- this CTA's run [lo, hi) of the list: of key blocks, or (whole) of K/V heads
  struct Plan {
    long long warp_sums[kWarps];
    int b;
    int rem_h, rem_blk;
  };
  Plan* plan = reinterpret_cast<Plan*>(smem + L::kPlanOff);
  static_assert(sizeof(Plan) <= 256, "plan area");
  bool whole = a.whole != 0;
  int most = 0, heads = 0;  // blocks of this thread's longest sequence, its K/V heads
  auto weight = [&](int b) -> long long {
    if (b >= a.c.B) return 0;
    const int n = span_of<kBlock>(a, paged_attn_seq(a.c, b)).n;
    most = max(most, n);
    if (n > 0) heads += a.c.Hkv;
    return static_cast<long long>(whole ? min(n, 1) : n) * a.c.Hkv;
  };
  long long total = 0, x0 = 0;
  auto add_up = [&]() {
    total = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += kThreads) {
      const long long x = weight(b0 + tid);
      if (b0 == 0) x0 = x;
      long long sum;
      block_scan<kWarps>(x, plan->warp_sums, &sum);
      total += sum;
    }
  };
  add_up();
  long long per = (total + gridDim.x - 1) / gridDim.x;
  // About as many heads as CTAs, of about the same length: a head each, since five sixths of
  // the SMs can draw all that HBM gives where a warp's work per byte is least, and cutting
  // costs pieces and their merge. 128 heads (152 CTAs), cut and whole: 16384 bf16 keys of 128
  // 161 and 156 us, 4096 keys 48 and 44, 1000 keys 15.6 and 13.9, with 20 rows 56 and 51 for 4096.
  // Where the warps' work counts there is nothing to gain: e4m3 16384 keys 88.5 and 88.0, 4096
  // 31.4 and 30.2, 1000 12.8 and 13.7; d = 64 1000 bf16 keys 10.7 and 12.0, 4096 29.5 and 27.6.
  if constexpr (!E4M3 && D == 128) {
    long long all;
    block_scan<kWarps>(heads, plan->warp_sums, &all);
    const bool uneven = 5ll * most > 6 * per;
    if (!whole && all <= gridDim.x && !__syncthreads_or(uneven)) {
      whole = true;
      add_up();
      per = 1;
    }
  }
  const long long lo = per * blockIdx.x;
  const long long hi = lo + per < total ? lo + per : total;
  PieceHeader* headers = static_cast<PieceHeader*>(a.headers);
  if (lo >= hi) {
    if (tid == 0 && !a.whole) headers[blockIdx.x] = PieceHeader{-1, 0, 0, 1};
    return;
  }
  {
    long long base = 0;
    for (int b0 = 0; b0 < a.c.B && base <= lo; b0 += kThreads) {
      const long long x = b0 == 0 ? x0 : weight(b0 + tid);
      long long sum;
      const long long at = base + block_scan<kWarps>(x, plan->warp_sums, &sum);
      if (at <= lo && lo < at + x) {
        const long long n = x / a.c.Hkv;  // blocks (1 if whole) of a head
        plan->b = b0 + tid;
        plan->rem_h = static_cast<int>((lo - at) / n);
        plan->rem_blk = static_cast<int>((lo - at) % n);
      }
      base += sum;
    }
  }
  __syncthreads();
  Walk cw;  // the block being computed
  cw.b = plan->b;
  cw.h = plan->rem_h;
  cw.load(a);
  const bool starts_mid = plan->rem_blk != 0;
  cw.blk = cw.first + plan->rem_blk;

  // ---- loads
  const uint32_t ring = smem_u32(smem + L::kRingOff) + warp * L::kStages * L::kStageBytes;
  const uint32_t scale_ring = smem_u32(smem + L::kScaleOff) + warp * L::kStages * L::kScaleBytes;
  constexpr int kRowsPer = 32 / L::kUnits;        // rows that the lanes cover at once
  constexpr int kLoads = kGroup / kRowsPer;
  const int lrow = lane / L::kUnits, lunit = lane % L::kUnits;
  constexpr int kEs = E4M3 ? 1 : 2;
  const long long row_bytes = a.c.stride_row * kEs;
  Walk lw = cw;  // the block to load next
  // First of the warp's keys of a block; those of the last one may begin beyond 31 bits.
  auto chunk_of = [&](const Walk& w) {
    const unsigned j = static_cast<unsigned>(w.blk) * kBlock + static_cast<unsigned>(warp * kChunk);
    return static_cast<int>(min(j, kFarKey));
  };
  int lpage[kU];  // pages of its groups
  auto find_pages = [&]() {
#pragma unroll
    for (int g = 0; g < kU; ++g) {
      const int j = chunk_of(lw) + g * kGroup;
      lpage[g] = j < lw.s.len ? paged_page(a.c, lw.b, j) : -1;
    }
  };
  find_pages();
  auto issue = [&](int stage) {
#pragma unroll
    for (int g = 0; g < kU; ++g) {
      const int j = chunk_of(lw) + g * kGroup;
      const int have = lpage[g] >= 0 ? lw.s.len - j : 0;  // rows of the group that the cache holds
      const int slot = page_row(a.c, j);
      const int page = lpage[g] >= 0 ? lpage[g] : 0;
      const long long at = (page * a.c.stride_page + lw.h * a.c.stride_head +
                            (slot + lrow) * a.c.stride_row) * kEs + lunit * 16;
      const uint32_t dk = ring + stage * L::kStageBytes + g * L::kGroupBytes, dv = dk + L::kTileBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int r = lrow + i * kRowsPer;
        const bool real = r < have;
        const long long off = real ? at + i * kRowsPer * row_bytes : 0;
        cp_async16(dk + k_unit<D, E4M3>(r, lunit) * 16, a.c.k + off, real);
        cp_async16(dv + v_unit<D, E4M3>(r, lunit) * 16, a.c.v + off, real);
      }
      if constexpr (E4M3) {
        if (lane < 2) {  // the 16 rows' scale bytes lie next to each other
          const long long so =
              (static_cast<long long>(page) * a.c.Hkv + lw.h) * a.c.page_size + slot;
          cp_async16(scale_ring + stage * L::kScaleBytes + g * 32 + lane * 16,
                     (lane ? a.c.v_scale : a.c.k_scale) + so, have > 0);
        }
      }
    }
    lw.next(a);
    find_pages();
  };
  // ---- query rows of a K/V head: row r = t * G + g; the rows' columns in the order of the
  // products, two registers per 16 columns. Column from which 16 bytes of a thread's row serve
  // products 2 i and 2 i + 1.
  auto q_col = [&](int i) {
    return E4M3 ? (i >> 1) * 64 + c4 * 16 + (i & 1) * 8 : i * 32 + c4 * 8;
  };
  auto q_load = [&](const Walk& w, int r, int col) {
    const int t = r / G;
    const __nv_bfloat16* p = a.q + (w.s.t0 + t) * a.q_stride + (w.h * G + (r - t * G)) * D;
    return r < w.s.nq * G ? *reinterpret_cast<const uint4*>(p + col) : make_uint4(0u, 0u, 0u, 0u);
  };
  // e4m3: Q's rows as f16, each times 2^k that puts its largest magnitude (bf16 bits `top`)
  // into [2^14, 2^15): f16 then holds all that bf16 held but for elements below 2^-29 of it.
  auto q_exponent = [](uint32_t top) {
    return max(-114, min(60, 14 + 127 - static_cast<int>(top >> 7)));
  };
  auto top_of = [](const uint4& x) {
    constexpr uint32_t kAbs = 0x7FFF7FFFu;
    const uint32_t m =
        __vmaxu2(__vmaxu2(x.x & kAbs, x.y & kAbs), __vmaxu2(x.z & kAbs, x.w & kAbs));
    return max(m & 0xFFFFu, m >> 16);
  };
  auto to_f16 = [](uint4 x, float f) {
    auto one = [&](uint32_t y) {
      return pack_f16x2(__uint_as_float(y << 16) * f, __uint_as_float(y & 0xFFFF0000u) * f);
    };
    return make_uint4(one(x.x), one(x.y), one(x.z), one(x.w));
  };
  float c_row[NT][2];  // what a row's scores are multiplied with, rows 2 c4, 2 c4 + 1 of each eight
  // Q in registers ...
  constexpr int kQRegs = L::kQShared ? 1 : D / 32;
  uint4 q[NT][kQRegs] = {}, qn[NT][kQRegs];
  auto load_q = [&](const Walk& w, uint4(&x)[NT][kQRegs]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < kQRegs; ++i) x[n][i] = q_load(w, n * 8 + g8, q_col(i));
  };
  auto ready_q = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      c_row[n][0] = c_row[n][1] = a.scale_log2;
      if constexpr (E4M3) {
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kQRegs; ++i) top = max(top, top_of(q[n][i]));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int k = q_exponent(top);
#pragma unroll
        for (int i = 0; i < kQRegs; ++i) q[n][i] = to_f16(q[n][i], pow2i(k));
#pragma unroll
        for (int e = 0; e < 2; ++e)
          c_row[n][e] *= pow2i(-__shfl_sync(0xffffffffu, k, (2 * c4 + e) * 4));
      }
    }
  };
  // ... or in shared memory: the block's threads bring 16-byte units of it, spread over the
  // banks for the eight lanes (two rows, four units) that read at once.
  const uint32_t sQ = smem_u32(smem + L::kQOff), sQExp = sQ + L::kRows * D * 2;
  auto q_unit = [](int r, int u) {
    return r * (D / 8) + (u ^ (E4M3 ? (r & 1) : ((r & 1) << 2)));
  };
  constexpr int kQAll = L::kRows * (D / 8);
  constexpr int kQUnits = L::kQShared ? (kQAll + kThreads - 1) / kThreads : 1;
  uint4 qs[kQUnits];
  auto load_q_shared = [&](const Walk& w) {
#pragma unroll
    for (int i = 0; i < kQUnits; ++i) {
      const int x = tid + i * kThreads;
      if (x < kQAll) qs[i] = q_load(w, x / (D / 8), x % (D / 8) * 8);
    }
  };
  auto store_q_shared = [&]() {
#pragma unroll
    for (int i = 0; i < kQUnits; ++i) {
      const int x = tid + i * kThreads, r = x / (D / 8), u = x % (D / 8);
      if (x >= kQAll) break;
      uint4 y = qs[i];
      if constexpr (E4M3) {
        uint32_t top = top_of(y);
#pragma unroll
        for (int k = D / 16; k > 0; k >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, k));
        const int k = q_exponent(top);
        y = to_f16(y, pow2i(k));
        if (u == 0) st_shared_u32(sQExp + r * 4, __float_as_uint(a.scale_log2 * pow2i(-k)));
      }
      st_shared_v4(sQ + q_unit(r, u) * 16, y.x, y.y, y.z, y.w);
    }
  };
  auto ready_q_shared = [&]() {  // after a barrier
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        c_row[n][e] = E4M3 ? __uint_as_float(ld_shared_u32(sQExp + (n * 8 + 2 * c4 + e) * 4))
                           : a.scale_log2;
  };
  auto get_q = [&](int n, int i) {  // the registers of products 2 i and 2 i + 1
    if constexpr (L::kQShared)
      return ld_shared_v4(sQ + q_unit(n * 8 + g8, q_col(i) >> 3) * 16);
    else
      return q[n][i];
  };
  if constexpr (L::kQShared) {
    load_q_shared(cw);
    store_q_shared();
    __syncthreads();
    ready_q_shared();
  } else {
    load_q(cw, q);
    ready_q();
  }

  long long steps = hi - lo;  // blocks
  if (whole) {
    Walk t = cw;
    steps = 0;
    for (long long u = lo; u < hi; ++u) {
      steps += t.end - t.first;
      t.blk = t.end - 1;
      t.next(a);
    }
  }
#pragma unroll
  for (int s = 0; s < L::kStages - 1; ++s) {
    if (s < steps) issue(s);
    cp_async_commit();
  }

  float o[NT][D / 16][4];
  float m_ref[NT][2], l_sum[NT][2];  // rows 2 c4, 2 c4 + 1 of each group of eight
  auto clear = [&]() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m_ref[n][e] = -INFINITY;
        l_sum[n][e] = 0.f;
      }
    }
  };
  clear();
  bool first_piece = true, ended0 = false;
  int slot1_row = -1, slot1_h = 0, slot1_rows = 0;
  float* merge = reinterpret_cast<float*>(smem + L::kMergeOff);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMlOff);
  int stage = 0;
  int piece_blk = cw.blk;  // first block of the piece
  for (long long i = 0; i < steps; ++i) {
    cp_async_wait<L::kStages - 2>();
    __syncwarp();  // the stage has landed for every lane; the last one has been read by all
    if (i + L::kStages - 1 < steps) issue(stage == 0 ? L::kStages - 1 : stage - 1);
    cp_async_commit();
    Walk nw = cw;
    nw.next(a);
    const bool ends = nw.b != cw.b || nw.h != cw.h;  // the unit's last block
    if constexpr (!L::kQShared) {
      if (ends && i + 1 < steps) load_q(nw, qn);
    }

    const int j0 = chunk_of(cw);
    const int pos0 = cw.s.len - cw.s.nq;  // position of the first new token
    const int key_min = a.wl >= 0 ? pos0 - a.wl : 0;
    if (j0 < cw.s.len && j0 + kChunk > key_min) {
      const uint32_t sk = ring + stage * L::kStageBytes, sv = sk + L::kTileBytes;
      // ---- S^T = K Q^T: keys g8 and g8 + 8, query rows 2 c4 and 2 c4 + 1
      constexpr bool kTwo = NT <= 2;  // two chains of products each, where there are few
      float s[kU][NT][4], s2[kU][NT][4];
#pragma unroll
      for (int g = 0; g < kU; ++g) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[g][n][e] = s2[g][n][e] = 0.f;
        if constexpr (!E4M3) {
#pragma unroll
          for (int x = 0; x < D / 32; ++x) {
            const uint4 k0 = ld_shared_v4(sk + g * L::kGroupBytes + k_unit<D, E4M3>(g8, 4 * x + c4) * 16);
            const uint4 k1 = ld_shared_v4(sk + g * L::kGroupBytes + k_unit<D, E4M3>(g8 + 8, 4 * x + c4) * 16);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const uint4 y = get_q(n, x);
              mma16816<E4M3>(s[g][n], k0.x, k1.x, k0.y, k1.y, y.x, y.y);
              mma16816<E4M3>(kTwo ? s2[g][n] : s[g][n], k0.z, k1.z, k0.w, k1.w, y.z, y.w);
            }
          }
        } else {
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const uint4 k0 = ld_shared_v4(sk + g * L::kGroupBytes + k_unit<D, E4M3>(g8, 4 * x + c4) * 16);
            const uint4 k1 = ld_shared_v4(sk + g * L::kGroupBytes + k_unit<D, E4M3>(g8 + 8, 4 * x + c4) * 16);
            const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
            for (int w = 0; w < 4; w += 2) {
              uint32_t a0[4], a1[4];
              e4m3_to_f16(w0[w], a0[0], a0[2]);
              e4m3_to_f16(w1[w], a0[1], a0[3]);
              e4m3_to_f16(w0[w + 1], a1[0], a1[2]);
              e4m3_to_f16(w1[w + 1], a1[1], a1[3]);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const uint4 y = get_q(n, 2 * x + (w >> 1));
                mma16816<E4M3>(s[g][n], a0[0], a0[1], a0[2], a0[3], y.x, y.y);
                mma16816<E4M3>(kTwo ? s2[g][n] : s[g][n], a1[0], a1[1], a1[2], a1[3], y.z, y.w);
              }
            }
          }
        }
      }
      // ---- scores in log2 units, masks, running maximum, P. e4m3: keys g8 and g8 + 8 have K's
      // scale, V's exponent, and what takes V's scale out of the sum (a scale byte of 0, which
      // only a page that is none has, counts as 127).
      float v_inv[kU][2];
#pragma unroll
      for (int g = 0; g < kU; ++g) {
        float k_scale[2] = {1.f, 1.f}, v_exp[2] = {0.f, 0.f};
        if constexpr (E4M3) {
          const uint32_t ss = scale_ring + stage * L::kScaleBytes + g * 32 + g8;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kb = ld_shared_u8(ss + 8 * e);
            int vb = ld_shared_u8(ss + 16 + 8 * e);
            vb = vb == 0 ? 127 : min(vb, kScaleMax + 127);
            k_scale[e] = kb == kScaleNaN ? __uint_as_float(0x7FC00000u) : pow2i(min(kb, kScaleMax + 127) - 127);
            v_exp[e] = static_cast<float>(vb - 127);
            v_inv[g][e] = pow2i(127 - kUp - kDown - vb);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[g][n][e] = (s[g][n][e] + s2[g][n][e]) * (c_row[n][e & 1] * k_scale[e >> 1]) + v_exp[e >> 1];
      }
      constexpr float kLift = E4M3 ? kF16Lift : 0.f;
      const int last_lo = a.wl >= 0 ? cw.s.len - 1 - a.wl : 0;  // first key of the last token
      const int first_hi = a.causal ? pos0 + 1 : cw.s.len;      // end of the first token's keys
      if (j0 < last_lo || j0 + kChunk > first_hi) {
#pragma unroll
        for (int g = 0; g < kU; ++g)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int key = j0 + g * kGroup + g8 + (e >> 1) * 8;
              const int pos = pos0 + (n * 8 + 2 * c4 + (e & 1)) / G;
              if (key >= cw.s.len || (a.causal && key > pos) || (a.wl >= 0 && key < pos - a.wl))
                s[g][n][e] = -INFINITY;
            }
      }
      // largest of the thread's scores of rows 2 c4 + e
      auto largest = [&](int n, int e) {
        float mx = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
        for (int g = 1; g < kU; ++g) mx = fmaxf(mx, fmaxf(s[g][n][e], s[g][n][e + 2]));
        return mx;
      };
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) grow |= largest(n, e) > m_ref[n][e] + (kRescale + kLift);
      // The reference maximum moves rarely, so most steps need one vote instead of the row
      // maxima.
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = largest(n, e);
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
            const float m_new = fmaxf(m_ref[n][e], mx - kLift);
            const Factor<E4M3> f(m_new == -INFINITY ? 0.f : m_ref[n][e] - m_new);
            const float alpha = f.all();
            m_ref[n][e] = m_new;
            l_sum[n][e] = f.of(l_sum[n][e]);
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              o[n][x][e] *= alpha;
              o[n][x][e + 2] *= alpha;
            }
          }
      }
      uint32_t p0[kU][NT], p1[kU][NT];  // P^T as the second operand: keys 2 c4 (+ 8) .., query row g8
#pragma unroll
      for (int g = 0; g < kU; ++g)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float m = m_ref[n][e & 1];
            p[e] = ex2_approx(s[g][n][e] - (m == -INFINITY ? 0.f : E4M3 ? m - kUp : m));
          }
          if constexpr (E4M3) {
            l_sum[n][0] = fmaf(p[0], v_inv[g][0], fmaf(p[2], v_inv[g][1], l_sum[n][0]));
            l_sum[n][1] = fmaf(p[1], v_inv[g][0], fmaf(p[3], v_inv[g][1], l_sum[n][1]));
            const uint64_t down = f2_pack(pow2i(-kUp), pow2i(-kUp));
            f2_unpack(f2_mul(f2_pack(p[0], p[1]), down), p[0], p[1]);
            f2_unpack(f2_mul(f2_pack(p[2], p[3]), down), p[2], p[3]);
          } else {
            l_sum[n][0] += p[0] + p[2];
            l_sum[n][1] += p[1] + p[3];
          }
          // P is rounded to bf16 for the product (at most 2^-8 of each weight: its operands have one
          // type, which is V's), or to f16 (2^-11, or 2^-32 of the largest weight where that is
          // more); the sum keeps fp32
          p0[g][n] = movmatrix_t(E4M3 ? pack_f16x2(p[0], p[1]) : pack_bf16x2(p[0], p[1]));
          p1[g][n] = movmatrix_t(E4M3 ? pack_f16x2(p[2], p[3]) : pack_bf16x2(p[2], p[3]));
        }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int g = 0; g < kU; ++g) {
        if constexpr (!E4M3) {
          const int key = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            uint32_t v[4];
            ldmatrix4_t(sv + g * L::kGroupBytes + v_unit<D, E4M3>(key, 2 * x + ((lane >> 3) & 1)) * 16, v);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<E4M3>(o[n][x], v[0], v[1], v[2], v[3], p0[g][n], p1[g][n]);
          }
        } else {
          constexpr int kWords = D / 32;  // words of a thread's columns, D / 8 of them, per key
          uint32_t v[4][kWords];          // keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = 2 * c4 + (e & 1) + (e >> 1) * 8;
            if constexpr (D == 128) {
              const uint4 y = ld_shared_v4(sv + g * L::kGroupBytes + v_unit<D, E4M3>(key, g8) * 16);
              v[e][0] = y.x;
              v[e][1] = y.y;
              v[e][kWords - 2] = y.z;
              v[e][kWords - 1] = y.w;
            } else {
              const uint2 y = ld_shared_v2(sv + g * L::kGroupBytes + v_unit<D, E4M3>(key, g8 >> 1) * 16 + (g8 & 1) * 8);
              v[e][0] = y.x;
              v[e][1] = y.y;
            }
          }
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {  // columns (D / 8) g8 + 2 x and + 1
            // both columns' codes of two keys in one word, then as f16 pairs of keys
            constexpr uint32_t kSel[2] = {0x5140u, 0x7362u};
            uint32_t r[4];
            e4m3_to_f16(prmt(v[0][x >> 1], v[1][x >> 1], kSel[x & 1]), r[0], r[1]);
            e4m3_to_f16(prmt(v[2][x >> 1], v[3][x >> 1], kSel[x & 1]), r[2], r[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816<E4M3>(o[n][x], r[0], r[1], r[2], r[3], p0[g][n], p1[g][n]);
          }
        }
      }
    }
    stage = stage + 1 == L::kStages ? 0 : stage + 1;

    if (ends || i + 1 == steps) {
      // ---- merge the warps' states of this piece
      const int M = cw.s.nq * G;
      const bool more = ends && i + 1 < steps;
      if constexpr (L::kQShared) {
        if (more) load_q_shared(nw);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float l = l_sum[n][e];
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
          l_sum[n][e] = l;
        }
      // State `to` of the merge buffer: (m, l) and O of every row.
      auto put_state = [&](int to) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int r = n * 8 + 2 * c4 + e;
            if (r < M) {
              if (g8 == 0) ml[to * L::kRows + r] = make_float2(m_ref[n][e], l_sum[n][e]);
              float* dst = merge + (to * L::kRows + r) * L::kPitch;
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                dst[E4M3 ? (D / 8) * g8 + 2 * x : 16 * x + g8] = o[n][x][e];
                dst[E4M3 ? (D / 8) * g8 + 2 * x + 1 : 16 * x + g8 + 8] = o[n][x][e + 2];
              }
            }
          }
      };
      __syncthreads();  // the last merge's readers are done, and every warp is with Q
      if constexpr (L::kQShared) {
        if (more) store_q_shared();
      }
      if constexpr (L::kFold == 2) {
        if (warp >= L::kStates) put_state(warp - L::kStates);
        __syncthreads();
        if (warp < L::kStates) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int r = n * 8 + 2 * c4 + e;
              if (r < M) {
                const float2 z = ml[warp * L::kRows + r];
                const float m = fmaxf(m_ref[n][e], z.x), mu = m == -INFINITY ? 0.f : m;
                const Factor<E4M3> f0(m_ref[n][e] - mu), f1(z.x - mu);
                const float k0 = f0.all(), k1 = f1.all();
                m_ref[n][e] = m;
                l_sum[n][e] = f0.of(l_sum[n][e]) + f1.of(z.y);
                const float* src = merge + (warp * L::kRows + r) * L::kPitch;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                  const float y0 = src[E4M3 ? (D / 8) * g8 + 2 * x : 16 * x + g8];
                  const float y1 = src[E4M3 ? (D / 8) * g8 + 2 * x + 1 : 16 * x + g8 + 8];
                  o[n][x][e] = k0 * o[n][x][e] + k1 * y0;
                  o[n][x][e + 2] = k0 * o[n][x][e + 2] + k1 * y1;
                }
              }
            }
          __syncwarp();  // this state has been read by every lane
          put_state(warp);
        }
      } else {
        put_state(warp);
      }
      __syncthreads();
      const bool from_start = piece_blk == cw.first;
      const bool direct = from_start && ends;
      // slot 0: the piece began in an earlier CTA's run; slot 1: it goes on in the next's
      const int slot = from_start ? 1 : 0;
      for (int it = tid; it < M * (D / 4); it += kThreads) {
        const int r = it / (D / 4), d0 = (it % (D / 4)) * 4;
        float m = -INFINITY;
#pragma unroll
        for (int w = 0; w < L::kStates; ++w) m = fmaxf(m, ml[w * L::kRows + r].x);
        const float mu = m == -INFINITY ? 0.f : m;
        float l = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < L::kStates; ++w) {
          const float2 z = ml[w * L::kRows + r];
          const Factor<E4M3> f(z.x - mu);
          const float k = f.all();
          l += f.of(z.y);
          const float4 v = *reinterpret_cast<const float4*>(merge + (w * L::kRows + r) * L::kPitch + d0);
          y[0] += k * v.x;
          y[1] += k * v.y;
          y[2] += k * v.z;
          y[3] += k * v.w;
        }
        // l is 0 for a row that sees no key, and a NaN stays one. e4m3: l is 2^-kDown of the sum,
        // which is made good last (1 / l alone may be as small as 2^-123)
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = E4M3 ? y[k] * inv * pow2i(-kDown) : y[k] * inv;
        const float lse2 = l == 0.f ? -INFINITY : m + __log2f(l) + (E4M3 ? kDown : 0);  // log2
        if (direct) {
          const int t = r / G;
          const long long row = static_cast<long long>(cw.s.t0 + t) * a.H + cw.h * G + (r - t * G);
          *reinterpret_cast<uint2*>(a.o + row * D + d0) = make_uint2(
              pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
          if (d0 == 0) a.lse[row] = lse2 * kLn2;
        } else {
          const long long row = (2ll * blockIdx.x + slot) * L::kRows + r;
          *reinterpret_cast<float4*>(a.o_part + row * D + d0) =
              make_float4(y[0], y[1], y[2], y[3]);
          if (d0 == 0) a.lse_part[row] = lse2;
        }
      }
      if (first_piece && starts_mid) ended0 = ends;
      if (!ends && from_start) {
        slot1_row = cw.s.t0;
        slot1_h = cw.h;
        slot1_rows = M;
      }
      first_piece = false;
      clear();
      piece_blk = nw.blk;
      if (more) {
        if constexpr (L::kQShared) {
          ready_q_shared();
        } else {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int x = 0; x < kQRegs; ++x) q[n][x] = qn[n][x];
          ready_q();
        }
      }
    }
    cw = nw;
  }
  cp_async_wait<0>();
  if (tid == 0 && !a.whole)
    headers[blockIdx.x] = PieceHeader{slot1_row, slot1_h, slot1_rows, !starts_mid || ended0};
}

// Merge of the pieces of a head that runs' ends have cut: with lse_s and the normalised O_s
// of piece s, O = sum_s 2^(lse_s - m) O_s / sum_s 2^(lse_s - m), m = max_s lse_s. Block (c, r)
// takes query row r of the head that CTA c's run began and did not end; the next CTAs'
// pieces follow until one ends it. In the order of the pieces, so always the same result. A
// piece whose lse is a NaN takes no part in the maximum, and makes the sums NaN.
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) fa_paged_step_merge_kernel(const PagedAttnArgs a, int ctas,
                                                                       int rows) {
  constexpr int kPer = D / 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, r = blockIdx.y;
  __shared__ int n_more;
  __shared__ float mx[kMergeWarps], dens[kMergeWarps];
  __shared__ float acc_s[kMergeWarps][D];
  pdl_wait();
  const PieceHeader* headers = static_cast<const PieceHeader*>(a.headers);
  PieceHeader hd;
  // pieces: slot 1 of CTA c, slot 0 of the n - 1 after it
  const int n = 1 + pieces_after(headers, c, ctas, &n_more, &hd);
  if (hd.row0 < 0 || r >= hd.rows) return;
  const int G = a.G;
  auto row_of = [&](int i) { return (2ll * (c + i) + (i == 0 ? 1 : 0)) * rows + r; };
  // the warp's first piece is under way while the maximum is found
  float m = -INFINITY, den = 0.f, acc[kPer] = {}, lse0 = -INFINITY, part0[kPer] = {};
  if (warp < n) {
    lse0 = a.lse_part[row_of(warp)];
    load_part<kPer>(a.o_part + row_of(warp) * D + lane * kPer, part0);
  }
  for (int i = tid; i < n; i += kMergeWarps * 32) m = fmaxf(m, a.lse_part[row_of(i)]);
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
  if (lane == 0) mx[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kMergeWarps; ++w) m = fmaxf(m, mx[w]);
  const float mu = m == -INFINITY ? 0.f : m;
  auto add = [&](float lse, const float* part) {
    const float w = ex2_approx(lse - mu);
    den += w;
#pragma unroll
    for (int k = 0; k < kPer; ++k) acc[k] += w * part[k];
  };
  add(lse0, part0);
#pragma unroll 4
  for (int i = warp + kMergeWarps; i < n; i += kMergeWarps) {
    float part[kPer];
    load_part<kPer>(a.o_part + row_of(i) * D + lane * kPer, part);
    add(a.lse_part[row_of(i)], part);
  }
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc_s[warp][lane * kPer + k] = acc[k];
  if (lane == 0) dens[warp] = den;
  __syncthreads();
  if (tid < D) {
    float y = 0.f, l = 0.f;
#pragma unroll
    for (int w = 0; w < kMergeWarps; ++w) {
      y += acc_s[w][tid];
      l += dens[w];
    }
    const int t = r / G;
    const long long row = static_cast<long long>(hd.row0 + t) * a.H + hd.h * G + (r - t * G);
    a.o[row * D + tid] = __float2bfloat16(l == 0.f ? 0.f : y / l);
    if (tid == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2;
  }
}

namespace {

template <int D, bool E4M3, int NT>
cudaError_t launch_impl(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  using L = StepL<D, E4M3, NT>;
  auto kern = fa_paged_step_kernel<D, E4M3, NT>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kern), L::kSmemBytes, 0, ready);
  if (e != cudaSuccess) return e;
  kern<<<ctas, L::kThreads, L::kSmemBytes, stream>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.whole) return e;
  return launch_merge(fa_paged_step_merge_kernel<D>, dim3(ctas, a.G * a.c.max_q),
                      kMergeWarps * 32, stream, a, ctas, int(L::kRows));
}

template <int D, bool E4M3>
cudaError_t launch_rows(const PagedAttnArgs& a, int ctas, cudaStream_t stream) {
  const int rows = a.G * a.c.max_q;
  return rows <= 8    ? launch_impl<D, E4M3, 1>(a, ctas, stream)
         : rows <= 16 ? launch_impl<D, E4M3, 2>(a, ctas, stream)
                      : launch_impl<D, E4M3, 3>(a, ctas, stream);
}

}  // namespace

cudaError_t launch_paged_step(const PagedAttnArgs& a, bool e4m3, int ctas, cudaStream_t stream) {
  if (a.c.d == 64)
    return e4m3 ? launch_rows<64, true>(a, ctas, stream) : launch_rows<64, false>(a, ctas, stream);
  return e4m3 ? launch_rows<128, true>(a, ctas, stream) : launch_rows<128, false>(a, ctas, stream);
}

}  // namespace fa
